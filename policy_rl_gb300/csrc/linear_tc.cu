// linear_tc.cu -- bf16 matrix products with fused epilogues on the tensor
// cores (tcgen05), operands streamed by TMA.
//
// out(i, j) = sum_r A(i, r) B(j, r).  Each operand is read as it lies: with
// the sum's index contiguous ("K-major": x and W of the forward product, dz of
// the data gradient) or with its own index contiguous ("MN-major": W of the
// data gradient, both operands of the weight gradient), so nothing is
// transposed beforehand.
//
// A unit of work is one output tile (and one slice of the sum); a CTA, or a
// pair of CTAs, walks over units.  Warp 0 issues TMA loads into a ring of
// 64-deep stages, warp 1 issues the MMAs into one of two TMEM accumulators,
// and eight warps drain the other accumulator through the epilogue meanwhile:
// bias, pre-activation, activation, residual, rounding, and stores through
// swizzled staging by TMA.
//
// Why pairs: at the full MMA rate a CTA with a 128 x 256 tile would have to
// take in 48 KB of operands every 512 clocks, more than an SM receives (about
// 46 bytes a clock measured).  A pair (cta_group::2) computes 256 x 256 with
// each CTA holding its 128 rows of A and half of B: 32 KB per 512 clocks, with
// the accumulators still double-buffered.  Small products take single CTAs
// with 128 x 128 tiles, so that more SMs have work.
//
// Every wait on an mbarrier is bounded; on expiry the kernel sets the error
// word, stops issuing, drains what is in flight and frees its TMEM.
#include <algorithm>

#include "gemm.h"
#include "linear.h"
#include "ops.cuh"
#include "tc_tile.cuh"

namespace ppo {
namespace lin {
namespace {

using namespace ptx;
using ppo::tc::Guard;
using ppo::tc::drain_wait;
using ppo::tc::put_row_chunks;
using ppo::tc::wait_bar;

constexpr uint64_t kWaitNs = 2000000000ull;
constexpr int BM = 128, BK = 64;
constexpr int kEpiWarps = 8;
constexpr int kThreads = (2 + kEpiWarps) * kWarp;
// The tensor cores truncate their fp32 sums: measured, 7.6e-5 relative after
// 1,000 16-deep steps.  Sums that stay fp32 (the weight gradient over many
// thousand rows) are therefore taken out of TMEM every kWindow 64-deep steps
// and added in registers, rounded to nearest, while the next window's MMAs fill
// the other accumulator.
#ifndef KWIN
#define KWIN 8
#endif
constexpr int kWindow = KWIN;
constexpr int kStg = 8192;             // staging of an epilogue warp: two 32-row x 128-byte boxes

template <int CG, int BN>
struct TileCfg {
  static constexpr int A_BYTES = BM * BK * 2;
  static constexpr int B_ROWS = BN / CG;
  static constexpr int B_BYTES = B_ROWS * BK * 2;
  static constexpr int STAGE = A_BYTES + B_BYTES;
  static constexpr int S = 5;
  static constexpr int TMEM = 2 * BN;
  static constexpr size_t SMEM = 1024 + (size_t)S * STAGE + kEpiWarps * (size_t)kStg + 512;
  static_assert(SMEM <= 232448, "shared memory per CTA");
};

struct TcArgs {
  int64_t I, J, R;
  int tiles_i, tiles_j, k_tiles, kt_per_split;
  int window;                    // 64-deep steps that the tensor cores sum before a rounded add
  int64_t units;                 // tiles * splits
  Epilogue e;
  float* part;                   // [splits][I][ldp] partial products (nullable)
  int64_t ldp;
  int tma_out, tma_pre;          // the result (pre) leaves by TMA
  int vec_res, vec_aux;          // residual (pre_in) rows are 16-byte aligned
  int* err;
};

__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// TMA load whose completion counts on the even CTA's barrier
template <int CG>
__device__ __forceinline__ void load_2d(uint32_t dst, const void* tmap, int x, int y, uint32_t bar) {
  if constexpr (CG == 1) {
    tma_load_2d(dst, tmap, x, y, bar);
  } else {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"((uint64_t)tmap), "r"(x), "r"(y), "r"(bar)
        : "memory");
  }
}
template <int CG>
__device__ __forceinline__ void alloc(uint32_t slot, uint32_t ncols) {
  if constexpr (CG == 1) {
    tmem_alloc(slot, ncols);
  } else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot),
                 "r"(ncols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
}
template <int CG>
__device__ __forceinline__ void dealloc(uint32_t taddr, uint32_t ncols) {
  if constexpr (CG == 1) {
    tmem_dealloc(taddr, ncols);
  } else {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols)
                 : "memory");
  }
}
// arrives on `bar` (of both CTAs of a pair) when this thread's MMAs are done
template <int CG>
__device__ __forceinline__ void commit(uint32_t bar) {
  if constexpr (CG == 1) {
    tc_commit(bar);
  } else {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
        " [%0], %1;" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
  }
}
template <int CG>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                    uint32_t accumulate) {
  if constexpr (CG == 1) {
    tc_mma_bf16(d, a, b, idesc, accumulate);
  } else {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
  }
}

// 32 consecutive bf16 of a row, zeros from column `cols` on
__device__ __forceinline__ void load_row32(const void* base, int64_t ld, int64_t row, int64_t c0,
                                           int64_t cols, bool ok, bool vec, uint4 (&o)[4]) {
  const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(base) + row * ld + c0;
  if (vec && c0 + 32 <= cols) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      o[i] = ok ? *reinterpret_cast<const uint4*>(p + 8 * i) : make_uint4(0, 0, 0, 0);
  } else {
    uint32_t w[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const uint32_t lo = ok && c0 + 2 * i < cols ? __bfloat16_as_ushort(p[2 * i]) : 0;
      const uint32_t hi = ok && c0 + 2 * i + 1 < cols ? __bfloat16_as_ushort(p[2 * i + 1]) : 0;
      w[i] = lo | (hi << 16);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  }
}
__device__ __forceinline__ float2 pair_of(const uint4 (&o)[4], int k) {   // elements 2k, 2k + 1
  const uint4 q = o[k / 4];
  const uint32_t w = (k & 3) == 0 ? q.x : (k & 3) == 1 ? q.y : (k & 3) == 2 ? q.z : q.w;
  return unpack_bf16x2(w);
}
__device__ __forceinline__ void store_plain(void* base, int64_t ld, int64_t row, int64_t c0,
                                            int64_t cols, bool ok, const float (&v)[32]) {
  if (!ok) return;
  __nv_bfloat16* p = static_cast<__nv_bfloat16*>(base) + row * ld + c0;
#pragma unroll
  for (int j = 0; j < 32; ++j)
    if (c0 + j < cols) p[j] = __float2bfloat16_rn(v[j]);
}

// The activation with its code known outside the loop over a chunk's values
template <int ACT>
__device__ __forceinline__ void act_chunk(float (&v)[32]) {
#pragma unroll
  for (int j = 0; j < 32; ++j) v[j] = ops::act_value<true>(ACT, v[j]);
}
__device__ __forceinline__ void act_chunk(int act, float (&v)[32]) {
  switch (act) {
    case PPO_ACT_TANH: act_chunk<PPO_ACT_TANH>(v); break;
    case PPO_ACT_RELU: act_chunk<PPO_ACT_RELU>(v); break;
    case PPO_ACT_SILU: act_chunk<PPO_ACT_SILU>(v); break;
    case PPO_ACT_GELU: act_chunk<PPO_ACT_GELU>(v); break;
    default: break;
  }
}
template <int ACT>
__device__ __forceinline__ void slope_chunk(const uint4 (&aux)[4], float (&v)[32]) {
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    const float2 x = pair_of(aux, k);
    v[2 * k] *= ops::act_slope<true>(ACT, x.x);
    v[2 * k + 1] *= ops::act_slope<true>(ACT, x.y);
  }
}
__device__ __forceinline__ void slope_chunk(int act, const uint4 (&aux)[4], float (&v)[32]) {
  switch (act) {
    case PPO_ACT_TANH: slope_chunk<PPO_ACT_TANH>(aux, v); break;
    case PPO_ACT_RELU: slope_chunk<PPO_ACT_RELU>(aux, v); break;
    case PPO_ACT_SILU: slope_chunk<PPO_ACT_SILU>(aux, v); break;
    case PPO_ACT_GELU: slope_chunk<PPO_ACT_GELU>(aux, v); break;
    default: break;
  }
}

template <int CG, int BN, int MODE, bool AMN, bool BMN>
__global__ void __launch_bounds__(kThreads, 1)
lin_tc_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
              const __grid_constant__ CUtensorMap tmO, const __grid_constant__ CUtensorMap tmP,
              const TcArgs p) {
  using C = TileCfg<CG, BN>;
  constexpr int S = C::S;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  uint8_t* stg = gbase + (size_t)S * C::STAGE;
  uint8_t* ctrl = stg + kEpiWarps * (size_t)kStg;
  uint64_t* bars = reinterpret_cast<uint64_t*>(ctrl);   // full[S] empty[S] tfull[2] tempty[2] drain
  auto full = [&](int s) { return smem_u32(&bars[s]); };
  auto empty = [&](int s) { return smem_u32(&bars[S + s]); };
  auto tfull = [&](int a) { return smem_u32(&bars[2 * S + a]); };
  auto tempty = [&](int a) { return smem_u32(&bars[2 * S + 2 + a]); };
  const uint32_t drain = smem_u32(&bars[2 * S + 4]);
  uint32_t* tslot = reinterpret_cast<uint32_t*>(&bars[2 * S + 5]);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tslot + 1);
  volatile uint32_t* cnt = reinterpret_cast<volatile uint32_t*>(tslot + 2);   // issued, consumed

  const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp;
  const uint32_t rank = CG == 2 ? cluster_rank() : 0u;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull(a), 1);
      mbar_init(tempty(a), CG * kEpiWarps);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    cnt[0] = cnt[1] = 0;
    fence_mbar_init();
  }
  if (warp == 1) alloc<CG>(smem_u32(tslot), C::TMEM);
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tmA);
    prefetch_tmap(&tmB);
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync();   // the pair's barriers exist
  tc_fence_after();
  const uint32_t tmem = *tslot;
  const Guard g{abort_flag, p.err, kWaitNs};
  const int64_t group = blockIdx.x / CG, groups = gridDim.x / CG;
  const int64_t tiles = (int64_t)p.tiles_i * p.tiles_j;
  pdl_wait();
  pdl_trigger();
  auto sA = [&](int s) { return base + (uint32_t)(s * C::STAGE); };
  auto sB = [&](int s) { return base + (uint32_t)(s * C::STAGE + C::A_BYTES); };
  auto unit_of = [&](int64_t u, int& ti, int& tj, int& kt0, int& kt1, int& split) {
    split = (int)(u / tiles);
    const int64_t t = u - (int64_t)split * tiles;
    ti = (int)(t / p.tiles_j);
    tj = (int)(t - (int64_t)ti * p.tiles_j);
    kt0 = split * p.kt_per_split;
    kt1 = min(p.k_tiles, kt0 + p.kt_per_split);
  };

  if (warp == 0) {
    if (lane == 0) {
      uint32_t it = 0, ph = 0;
      int s = 0;
      bool ok = true;
      for (int64_t u = group; u < p.units && ok; u += groups) {
        int ti, tj, kt0, kt1, split;
        unit_of(u, ti, tj, kt0, kt1, split);
        const int i0 = (ti * CG + (int)rank) * BM, j0 = tj * BN + (int)rank * C::B_ROWS;
        for (int kt = kt0; kt < kt1; ++kt) {
          if (!wait_bar(empty(s), ph ^ 1, g)) { ok = false; break; }
          if (rank == 0) mbar_arrive_expect_tx(full(s), CG * C::STAGE);
          const uint32_t bar = CG == 2 ? map_rank(full(s), 0) : full(s);
          if constexpr (AMN) {
#pragma unroll
            for (int b = 0; b < BM / 64; ++b)
              load_2d<CG>(sA(s) + b * 8192, &tmA, i0 + 64 * b, kt * BK, bar);
          } else {
            load_2d<CG>(sA(s), &tmA, kt * BK, i0, bar);
          }
          if constexpr (BMN) {
#pragma unroll
            for (int b = 0; b < C::B_ROWS / 64; ++b)
              load_2d<CG>(sB(s) + b * 8192, &tmB, j0 + 64 * b, kt * BK, bar);
          } else {
            load_2d<CG>(sB(s), &tmB, kt * BK, j0, bar);
          }
          cnt[0] = ++it;
          if (++s == S) { s = 0; ph ^= 1; }
        }
      }
      // every stage released: no commit is still to arrive here when the CTA leaves
      if (ok)
        for (int j = 0; j < S; ++j) {
          if (!wait_bar(empty(s), ph ^ 1, g)) break;
          if (++s == S) { s = 0; ph ^= 1; }
        }
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      constexpr uint32_t idesc = idesc_bf16(CG * BM, BN, AMN, BMN);
      uint32_t it = 0, ph = 0, n = 0;
      int s = 0;
      bool ok = true;
      for (int64_t u = group; u < p.units && ok; u += groups) {
        int ti, tj, kt0, kt1, split;
        unit_of(u, ti, tj, kt0, kt1, split);
        for (int w0 = kt0; w0 < kt1 && ok; w0 += p.window, ++n) {
          const int acc = n & 1, w1 = min(kt1, w0 + p.window);
          if (!wait_bar(tempty(acc), ((n >> 1) & 1) ^ 1, g)) { ok = false; break; }
          tc_fence_after();
          const uint32_t d = tmem + (uint32_t)(acc * BN);
          for (int kt = w0; kt < w1; ++kt) {
            if (!wait_bar(full(s), ph, g)) { ok = false; break; }
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < BK / 16; ++kk) {
              const uint64_t da = AMN ? sdesc_sw128(sA(s) + kk * 2048, 8192, 1024)
                                      : sdesc_sw128(sA(s) + kk * 32, 16, 1024);
              const uint64_t db = BMN ? sdesc_sw128(sB(s) + kk * 2048, 8192, 1024)
                                      : sdesc_sw128(sB(s) + kk * 32, 16, 1024);
              mma<CG>(d, da, db, idesc, (kt != w0 || kk != 0) ? 1u : 0u);
            }
            commit<CG>(empty(s));
            cnt[1] = ++it;
            if (++s == S) { s = 0; ph ^= 1; }
          }
          if (ok) commit<CG>(tfull(acc));
        }
      }
    }
  } else {
    const int q = warp & 3, half = (warp - 2) / 4;
    constexpr int PART = BN / 2;                  // columns of an epilogue warp
    uint8_t* mine = stg + (warp - 2) * kStg;
    uint32_t n = 0, sc = 0;
    // one window: TMEM columns of this warp, or false when a wait gave up
    auto window = [&](uint32_t& taddr) {
      const int acc = n & 1;
      if (!wait_bar(tfull(acc), (n >> 1) & 1, g)) return false;
      tc_fence_after();
      taddr = tmem + (uint32_t)(acc * BN + half * PART) + ((uint32_t)(q * 32) << 16);
      return true;
    };
    // the window's columns are read: the MMAs may overwrite them
    auto release = [&]() {
      const int acc = n & 1;
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (CG == 2) arrive_cluster(map_rank(tempty(acc), 0));
        else mbar_arrive(tempty(acc));
      }
      ++n;
    };
    for (int64_t u = group; u < p.units; u += groups) {
      int ti, tj, kt0, kt1, split;
      unit_of(u, ti, tj, kt0, kt1, split);
      const int64_t row0 = (int64_t)(ti * CG + (int)rank) * BM + q * 32, row = row0 + lane;
      const bool rok = row < p.I, any = row0 < p.I;
      const int64_t col0 = (int64_t)tj * BN + half * PART;
      uint32_t taddr;
      if constexpr (MODE == kWeight) {
        // the windows' sums are added here, in fp32 with rounding to nearest
        float v[PART / 32][32];
        bool ok = true;
        for (int w0 = kt0; w0 < kt1; w0 += p.window) {
          if (!window(taddr)) { ok = false; break; }
          uint32_t r[32];
          tmem_ld32_async(taddr, r);
#pragma unroll
          for (int c = 0; c < PART / 32; ++c) {
            tmem_wait_ld(r);
            if (w0 == kt0) {
#pragma unroll
              for (int j = 0; j < 32; ++j) v[c][j] = __uint_as_float(r[j]);
            } else {
#pragma unroll
              for (int j = 0; j < 32; ++j) v[c][j] += __uint_as_float(r[j]);
            }
            if (c + 1 < PART / 32) tmem_ld32_async(taddr + (uint32_t)(32 * (c + 1)), r);
          }
          release();
        }
        if (!ok) break;
        // 32 columns (128 bytes) at a time through two boxes
#pragma unroll
        for (int c = 0; c < PART / 32; ++c, ++sc) {
          const int64_t cc = col0 + 32 * c;
          if (p.tma_out) {
            uint8_t* buf = mine + (sc & 1) * 4096;
            if (lane == 0) bulk_wait_read1();
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i)
              *reinterpret_cast<float4*>(buf + lane * 128 + ((i ^ (lane & 7)) << 4)) =
                  make_float4(v[c][4 * i], v[c][4 * i + 1], v[c][4 * i + 2], v[c][4 * i + 3]);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0 && any && cc < p.J) {
              tma_store_3d(&tmO, smem_u32(buf), (int)cc, (int)row0, split);
              bulk_commit();
            }
          } else if (rok) {
            float* o = p.part ? p.part + ((int64_t)split * p.I + row) * p.ldp
                              : static_cast<float*>(p.e.out) + row * p.e.ldo;
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (cc + j < p.J) o[cc + j] = v[c][j];
          }
        }
      } else {
        if (!window(taddr)) break;
        const bool use_res = p.e.res != nullptr;
        const bool use_aux = MODE == kData && p.e.act != PPO_ACT_NONE;
        const bool use_pre = MODE == kForward && p.e.pre != nullptr;
#pragma unroll 1
        for (int c = 0; c < PART; c += 64, ++sc) {
          const int64_t c64 = col0 + c;
          uint8_t* yb = mine + (use_pre ? 4096 : (sc & 1) * 4096);
          uint8_t* pb = mine;
          const bool cols = c64 < p.J;
          if (lane == 0) {      // the buffers' last stores have read them
            if (use_pre) bulk_wait_read0();
            else bulk_wait_read1();
          }
          __syncwarp();
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            const int64_t cc = c64 + 32 * hh;
            uint32_t r[32];
            tmem_ld32_async(taddr + (uint32_t)(c + 32 * hh), r);
            uint4 rs[4], ax[4];
            if (use_res) load_row32(p.e.res, p.e.ldres, row, cc, p.J, rok, p.vec_res, rs);
            if (use_aux) load_row32(p.e.pre, p.e.ldpre, row, cc, p.J, rok, p.vec_aux, ax);
            float v[32];
            tmem_wait_ld(r);
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
            if constexpr (MODE == kForward) {
              if (p.e.bias) {
                if (cc + 32 <= p.J) {
                  const float4* b4 = reinterpret_cast<const float4*>(p.e.bias + cc);
#pragma unroll
                  for (int j = 0; j < 8; ++j) {
                    const float4 b = __ldg(b4 + j);
                    v[4 * j] += b.x;
                    v[4 * j + 1] += b.y;
                    v[4 * j + 2] += b.z;
                    v[4 * j + 3] += b.w;
                  }
                } else {
#pragma unroll
                  for (int j = 0; j < 32; ++j)
                    if (cc + j < p.J) v[j] += __ldg(p.e.bias + cc + j);
                }
              }
              if (use_pre) {
                if (p.tma_pre) put_row_chunks(pb + lane * 128, lane, 4 * hh, v);
                else store_plain(p.e.pre, p.e.ldpre, row, cc, p.J, rok, v);
              }
              act_chunk(p.e.act, v);
            } else {
              if (use_aux) slope_chunk(p.e.act, ax, v);
            }
            if (use_res) {
#pragma unroll
              for (int k = 0; k < 16; ++k) {
                const float2 x = pair_of(rs, k);
                v[2 * k] += x.x;
                v[2 * k + 1] += x.y;
              }
            }
            if (p.tma_out) put_row_chunks(yb + lane * 128, lane, 4 * hh, v);
            else store_plain(p.e.out, p.e.ldo, row, cc, p.J, rok, v);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0 && any && cols) {
            if (use_pre && p.tma_pre) tma_store_2d(&tmP, smem_u32(pb), (int)c64, (int)row0);
            if (p.tma_out) tma_store_2d(&tmO, smem_u32(yb), (int)c64, (int)row0);
            bulk_commit();
          }
        }
      }
      if constexpr (MODE != kWeight) release();
    }
    if (lane == 0) bulk_wait0();   // this warp's stores are complete before the CTA exits
  }

  __syncthreads();
  if (rank == 0 && *abort_flag) {
    // loads issued by this CTA (and, with it, the other one) but never
    // consumed, and outstanding MMAs
    if (threadIdx.x == 0) {
      const uint32_t issued = cnt[0], consumed = cnt[1];
      for (uint32_t it = consumed; it < issued; ++it)
        drain_wait(full(it % S), (it / S) & 1, kWaitNs);
    }
    if (warp == 1 && lane == 0) {
      if constexpr (CG == 1) {
        tc_commit(drain);
      } else {
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(drain)
            : "memory");
      }
      drain_wait(drain, 0, kWaitNs);
    }
    __syncthreads();
  }
  if (rank == 1 && *abort_flag) {
    // the odd CTA's loads complete on the other CTA's barriers: let them land
    const uint64_t t0 = globaltimer();
    while (globaltimer() - t0 < 1000000ull) {
    }
  }
  if constexpr (CG == 2) cluster_sync();   // neither CTA leaves while the other still uses it
  if (warp == 1) {
    tc_fence_after();
    dealloc<CG>(tmem, C::TMEM);
  }
}

// ---- launch --------------------------------------------------------------------
// One launch with its tensor maps.  A K-major operand is read in boxes of
// 64 (sum) x 128 rows, an MN-major one in boxes of 64 (own index) x 64.
template <int CG, int BN, int MODE, bool AMN, bool BMN>
cudaError_t launch(const Product& g, TcArgs p, int sms, cudaStream_t st) {
  using C = TileCfg<CG, BN>;
  CUtensorMap ta, tb, to, tp;
  cudaError_t e;
  if (AMN) e = tc_make_tmap(&ta, g.A, g.I, g.R, g.sar, 64, BK);
  else e = tc_make_tmap(&ta, g.A, g.R, g.I, g.sai, BK, BM);
  if (e != cudaSuccess) return e;
  if (BMN) e = tc_make_tmap(&tb, g.B, g.J, g.R, g.sbr, 64, BK);
  else e = tc_make_tmap(&tb, g.B, g.R, g.J, g.sbj, BK, C::B_ROWS);
  if (e != cudaSuccess) return e;
  to = ta;
  tp = ta;
  if (p.tma_out) {
    if (MODE == kWeight) {
      const int64_t splits = (p.k_tiles + p.kt_per_split - 1) / p.kt_per_split;
      e = tc_make_tmap_f32(&to, p.part ? p.part : static_cast<float*>(p.e.out), p.J, p.I,
                           p.part ? splits : 1, p.part ? p.ldp : p.e.ldo);
    } else {
      e = tc_make_tmap(&to, p.e.out, p.J, p.I, p.e.ldo, 64, 32);
    }
    if (e != cudaSuccess) return e;
  }
  if (p.tma_pre) {
    e = tc_make_tmap(&tp, p.e.pre, p.J, p.I, p.e.ldpre, 64, 32);
    if (e != cudaSuccess) return e;
  }
  const auto kernel = lin_tc_kernel<CG, BN, MODE, AMN, BMN>;
  static thread_local int prepared = -1;   // the device whose shared-memory opt-in is made
  int dev = 0;
  e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (prepared != dev) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM);
    if (e != cudaSuccess) return e;
    prepared = dev;
  }
  const int64_t groups = std::min<int64_t>(p.units, sms / CG);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(groups * CG));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CG;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CG == 2 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, ta, tb, to, tp, p);
}

template <int CG, int BN>
cudaError_t launch_mode(const Product& g, const TcArgs& p, int mode, int sms, cudaStream_t st) {
  if (p.part || mode == kWeight) {
    if (mode == kWeight) return launch<CG, BN, kWeight, true, true>(g, p, sms, st);
    if (mode == kForward) return launch<CG, BN, kWeight, false, false>(g, p, sms, st);
    return launch<CG, BN, kWeight, false, true>(g, p, sms, st);
  }
  if (mode == kForward) return launch<CG, BN, kForward, false, false>(g, p, sms, st);
  return launch<CG, BN, kData, false, true>(g, p, sms, st);
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace

// The cheapest of the tile shapes and splits for a whole GB300, by the rounds
// its units take: a 64-deep step of a unit costs a pair of CTAs and a single
// CTA (128 x 128) about 300 and 200 ns, a unit's start and epilogue 2 us, and
// a split product writes and re-reads its partial products.
TcPlan tc_plan(int64_t I, int64_t J, int64_t R, bool must_split) {
  constexpr int kSms = 152;
  TcPlan best{};
  double best_cost = 0;
  const int64_t kt = cdiv(R, BK);
  for (int cg = 1; cg <= 2; ++cg) {
    const int64_t ti = cdiv(I, cg * BM), tj = cdiv(J, cg == 2 ? 256 : 128);
    const double step = cg == 2 ? 0.30 : 0.20;
    int64_t last = -1;
    for (int64_t s = 1; s <= 32 && s <= kt; ++s) {
      const int64_t per = cdiv(kt, s), used = cdiv(kt, per);
      if (used == last) continue;
      last = used;
      const int64_t rounds = cdiv(ti * tj * used, kSms / cg);
      double cost = rounds * (per * step + 2.0);
      if (used > 1 || must_split) cost += 3.0 + (double)(used + 1) * I * J * 4 * 2 / 5e6;
      if (used > 1 && (double)used * I * J * 4 > 64e6) break;   // partial products stay in L2
      if (best.cg == 0 || cost < best_cost) {
        best_cost = cost;
        best.cg = cg;
        best.kt_per_split = (int)per;
        best.splits = (int)used;
      }
    }
  }
  return best;
}

bool tc_fits(const Product& g) {
  // TMA coordinates and tile counts are 32-bit
  constexpr int64_t top = (1ll << 31) - 512;
  return g.I < top && g.J < top && g.R < top &&
         cdiv(g.I, BM) * cdiv(g.J, 128) < (1ll << 31);
}

cudaError_t tc_product(const Product& g, const Epilogue& e, const TcPlan& plan, float* part,
                       int* err, int sms, cudaStream_t st) {
  TcArgs p{};
  p.I = g.I;
  p.J = g.J;
  p.R = g.R;
  p.tiles_i = (int)cdiv(g.I, plan.cg * BM);
  p.tiles_j = (int)cdiv(g.J, plan.cg == 2 ? 256 : 128);
  p.k_tiles = (int)cdiv(g.R, BK);
  p.kt_per_split = plan.kt_per_split;
  p.window = e.mode == kWeight ? kWindow : p.k_tiles;
  p.units = (int64_t)p.tiles_i * p.tiles_j * plan.splits;
  p.e = e;
  p.part = part;
  p.ldp = (g.J + 3) / 4 * 4;
  p.err = err;
  auto al = [](const void* q, int64_t ld, int m) { return ops::al16(q) && ld % m == 0; };
  p.tma_out = part ? 1 : e.mode == kWeight ? al(e.out, e.ldo, 4) : al(e.out, e.ldo, 8);
  p.tma_pre = !part && e.mode == kForward && e.pre && al(e.pre, e.ldpre, 8);
  p.vec_res = al(e.res, e.ldres, 8);
  p.vec_aux = al(e.pre, e.ldpre, 8);
  if (plan.cg == 2) return launch_mode<2, 256>(g, p, e.mode, sms, st);
  return launch_mode<1, 128>(g, p, e.mode, sms, st);
}

}  // namespace lin
}  // namespace ppo
