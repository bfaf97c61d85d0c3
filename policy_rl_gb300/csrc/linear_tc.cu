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
// 64-deep stages, warp 1 issues the MMAs into one of two TMEM accumulators, and
// 16 warps (8 for single CTAs) drain the other accumulator through the epilogue
// meanwhile: bias, pre-activation, activation, residual, rounding.  An epilogue
// warp owns a box of 32 rows x 64 columns of the tile: the residual or pre_in
// box comes by TMA while the MMAs run, is overwritten by the result, and leaves
// by TMA.  A residual beside pre or pre_in has a box of 16 rows more, for which
// the ring gives up a stage.  In the weight gradient warps 2 and 3 add up the
// columns of dz from the stages that the MMAs have read, so that db costs no
// pass of its own.
//
// What bounds it: long sums their operands.  An SM takes in 47 bytes of them a
// clock by TMA (measured with and without an epilogue; the full MMA rate would
// want 64): 0.35 us per 64-deep step of a 256 x 256 tile, 1.76 PFLOP/s at 8,192 x
// 8,192 x 8,192.  Sums of 512 (8 steps) the epilogue, 16 warps in step, and the
// memory behind it: 32,768 x 512 -> 2,048 forward, 39 us by its operands, takes 53,
// with gelu and pre 69 (302 MB), with a residual too 86; 65,536 x 512 -> 2,048 data
// gradient 95 us, with gelu' 126 (604 MB).  The weight gradient of the former, 64
// units of 128 steps, would take 45 us by its operands and takes 57, its finish
// among them, with db 64: 0.4 to 0.45 us a step, for a reason not found (windows of
// 64 steps instead of 8 save 2 us).
// What a warp waits for matters more than what it computes: with a releasing
// arrival for each read accumulator (a memory barrier) the last figure was 157,
// forward with gelu and pre 84.  Measured and left, on the last figure: a fence and
// store for every 16 rows (145).  Before the arrival was relaxed, on
// 157: inputs fetched 16 rows at a time (+10) or half a unit earlier from a third
// box (+8: a stage less), inputs by cp.async (+4), one reciprocal for two (+3),
// divisions for each unit's place (+5), stores by the warps themselves, the
// accumulator held in 64 registers so that TMEM is free at once (spills), L2
// prefetches of the operands by TMA.
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
#include "lin_tile.cuh"

namespace ppo {
namespace lin {
namespace {

constexpr int kFirstEpi = 4;           // warps 0..3: producer, MMA, column sums
constexpr int kBox = 4096;             // 32 rows x 128 bytes, 128-byte swizzle
// The tensor cores truncate their fp32 sums: measured, 7.6e-5 relative after
// 1,000 16-deep steps.  Sums that stay fp32 (the weight gradient over many
// thousand rows), and those of more than 2^16 terms, are therefore taken out of TMEM every kWindow 64-deep steps
// and added in registers, rounded to nearest, while the next window's MMAs fill
// the other accumulator.
// (Measured at 32,768 rows: error 1.9e-7 and 108 us with windows of 2 steps,
// 4.8e-7 and 60 us with 8, 4.4e-6 and 58 us with 64.)
constexpr int kWindow = 8;
// LATE: a residual beside another box of input or output; its boxes, of 16
// rows, take the room of a stage
template <int CG, int BN, int MODE, bool LATE>
struct TileCfg {
  static constexpr int A_BYTES = BM * BK * 2;
  static constexpr int B_ROWS = BN / CG;
  static constexpr int B_BYTES = B_ROWS * BK * 2;
  static constexpr int STAGE = A_BYTES + B_BYTES;
  // the weight gradient stages no results: its boxes' room goes to the ring
  // (weight and bias gradient of 32,768 x 512 -> 2,048: 68 us with 5 stages, 60
  // with 7)
  static constexpr int S = MODE == kWeight ? 7 : LATE ? 4 : 5;
  static constexpr int EW = 4 * (BN / 64);   // epilogue warps: 32 rows x 64 columns each
  static constexpr int THREADS = (kFirstEpi + EW) * kWarp;
  static constexpr int BOXES = MODE == kWeight ? 0 : EW * kBox + (LATE ? EW * kBox / 2 : 0);
  static constexpr int TMEM = 2 * BN;
  static constexpr int CTRL = 512;
  static constexpr size_t SMEM = 1024 + (size_t)S * STAGE + BOXES + CTRL;
  static_assert(SMEM <= 232448, "shared memory per CTA");
};

struct TcArgs {
  int64_t I, J, R;
  int tiles_i, tiles_j, k_tiles, kt_per_split;
  int window;                    // 64-deep steps that the tensor cores sum before a rounded add
  int units;                     // tiles * splits
  Epilogue e;
  int64_t plane_a, plane_b;      // fp32 operands as three bf16 planes: their rows (0: bf16)
  float* part;                   // [splits][I][ldp] partial products (nullable)
  int64_t ldp;
  int in;                        // matrix read a unit ahead: 0 none, 1 the residual, 2 pre_in
  int tma_late;                  // the residual beside another box (LATE) moves by TMA
  int wide_out;                  // fp32 rows start on 32-byte boundaries
  int tma_in, tma_out, tma_pre;  // it (the result, pre) moves by TMA
  float* db_part;                // [splits * tiles_j][I] column sums of A (nullable)
  int* err;
};

template <int CG, int BN, int MODE, bool AMN, bool BMN, bool LATE, int SETS>
__global__ void __launch_bounds__(TileCfg<CG, BN, MODE, LATE>::THREADS, 1)
lin_tc_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
              const __grid_constant__ CUtensorMap tmO, const __grid_constant__ CUtensorMap tmP,
              const __grid_constant__ CUtensorMap tmI, const TcArgs p) {
  using C = TileCfg<CG, BN, MODE, LATE>;
  constexpr int S = C::S;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  uint8_t* boxes = gbase + (size_t)S * C::STAGE;
  uint8_t* ctrl = boxes + C::BOXES;
  // full[S] empty[S] tfull[2] tempty[2] drain summed[S] box[EW] late[EW]
  uint64_t* bars = reinterpret_cast<uint64_t*>(ctrl);
  auto full = [&](int s) { return smem_u32(&bars[s]); };
  auto empty = [&](int s) { return smem_u32(&bars[S + s]); };
  auto tfull = [&](int a) { return smem_u32(&bars[2 * S + a]); };
  auto tempty = [&](int a) { return smem_u32(&bars[2 * S + 2 + a]); };
  const uint32_t drain = smem_u32(&bars[2 * S + 4]);
  auto summed = [&](int i) { return smem_u32(&bars[2 * S + 5 + i]); };
  auto box_bar = [&](int w) { return smem_u32(&bars[3 * S + 5 + w]); };
  auto late_bar = [&](int w) { return smem_u32(&bars[3 * S + 5 + C::EW + w]); };
  constexpr int kBars = 3 * S + 5 + 2 * C::EW;
  static_assert(kBars * 8 + 16 <= C::CTRL, "control block");
  uint32_t* tslot = reinterpret_cast<uint32_t*>(&bars[kBars]);
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
      mbar_init(tempty(a), CG * C::EW / SETS);
    }
    mbar_init(drain, 1);
    for (int s = 0; s < S; ++s) mbar_init(summed(s), 2);
    for (int w = 0; w < 2 * C::EW; ++w) mbar_init(box_bar(w), 1);
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
  const int group = blockIdx.x / CG, groups = gridDim.x / CG;
  pdl_wait();
  pdl_trigger();
  auto sA = [&](int s) { return base + (uint32_t)(s * C::STAGE); };
  auto sB = [&](int s) { return base + (uint32_t)(s * C::STAGE + C::A_BYTES); };
  auto unit_of = [&](int u, int& ti, int& tj, int& kt0, int& kt1, int& split) {
    const int row = u / p.tiles_j;
    tj = u - row * p.tiles_j;
    split = row / p.tiles_i;
    ti = row - split * p.tiles_i;
    kt0 = split * p.kt_per_split;
    kt1 = min(p.k_tiles, kt0 + p.kt_per_split);
  };

  // 16 epilogue warps leave 96 registers a thread: their four warpgroups take
  // some from the first one (64 + 4 x 104 = 5 x 96, the launch's registers)
  constexpr bool kShift = C::EW == 16;
  if (warp < kFirstEpi) {
  if constexpr (kShift) regs_dec<64>();
  if (warp == 0) {
    if (lane == 0) {
      uint32_t it = 0, ph = 0;
      int s = 0;
      bool ok = true;
      for (int u = group; u < p.units && ok; u += groups) {
        int ti, tj, kt0, kt1, split;
        unit_of(u, ti, tj, kt0, kt1, split);
        const int i0 = (ti * CG + (int)rank) * BM, j0 = tj * BN + (int)rank * C::B_ROWS;
        for (int kt = kt0; kt < kt1; ++kt) {
          if (!wait_bar(empty(s), ph ^ 1, g)) { ok = false; break; }
          if (MODE == kWeight && p.db_part && !wait_bar(summed(s), ph ^ 1, g)) { ok = false; break; }
          // the sum's step, and the rows that the operands' planes start at: of
          // three planes the six products of 2^-16 and more, the small ones first
          // (the accumulator is truncated at its own size)
          int k = kt, pa = 0, pb = 0;
          if (MODE == kWeight && p.plane_a) {
            k = kt / kTerms;
            const int t = kt - k * kTerms;
            pa = (int)p.plane_a * (t == 0 ? 2 : t == 2 || t == 3 ? 1 : 0);
            pb = (int)p.plane_b * (t == 1 ? 2 : t == 2 || t == 4 ? 1 : 0);
          }
          if (rank == 0) mbar_arrive_expect_tx(full(s), CG * C::STAGE);
          const uint32_t bar = CG == 2 ? map_rank(full(s), 0) : full(s);
          if constexpr (AMN) {
#pragma unroll
            for (int b = 0; b < BM / 64; ++b)
              load_2d<CG>(sA(s) + b * 8192, &tmA, i0 + 64 * b, k * BK + pa, bar);
          } else {
            load_2d<CG>(sA(s), &tmA, k * BK, i0 + pa, bar);
          }
          if constexpr (BMN) {
#pragma unroll
            for (int b = 0; b < C::B_ROWS / 64; ++b)
              load_2d<CG>(sB(s) + b * 8192, &tmB, j0 + 64 * b, k * BK + pb, bar);
          } else {
            load_2d<CG>(sB(s), &tmB, k * BK, j0 + pb, bar);
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
      for (int u = group; u < p.units && ok; u += groups) {
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
    // column sums of A (MN-major: [2 blocks of 64 columns][64 of the sum][64]):
    // a warp takes a block, a lane 8 columns of every fourth row.  A tile row's
    // stages are shared out among its tiles_j tiles.
    if (MODE == kWeight && p.db_part) {
      uint32_t ph = 0;
      int s = 0;
      bool ok = true;
      for (int u = group; u < p.units && ok; u += groups) {
        int ti, tj, kt0, kt1, split;
        unit_of(u, ti, tj, kt0, kt1, split);
        float sum[8] = {};
        const int terms = p.plane_a ? kTerms : 1;
        int turn = kt0 / terms % p.tiles_j, term = 0;
        for (int kt = kt0; kt < kt1; ++kt) {
          if (!wait_bar(empty(s), ph, g)) { ok = false; break; }
          if (turn == tj && term < 3) {      // (the first three terms meet each plane of A once)
            const uint8_t* blk = gbase + (size_t)s * C::STAGE + (warp - 2) * 8192;
            float t[8] = {};
#pragma unroll
            for (int r = 0; r < BK; r += 4) {
              const int k = r + (lane >> 3);
              const uint4 w = *reinterpret_cast<const uint4*>(
                  blk + k * 128 + (((lane & 7) ^ (k & 7)) << 4));
              const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float2 f = unpack_bf16x2(ww[i]);
                t[2 * i] += f.x;
                t[2 * i + 1] += f.y;
              }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[i] += t[i];
          }
          if (++term == terms) {
            term = 0;
            if (++turn == p.tiles_j) turn = 0;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(summed(s));
          if (++s == S) { s = 0; ph ^= 1; }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 8);
          sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 16);
        }
        const int64_t col = (int64_t)(ti * CG + (int)rank) * BM + (warp - 2) * 64 + lane * 8;
        if (ok && lane < 8) {
          float* d = p.db_part + ((int64_t)split * p.tiles_j + tj) * p.I;
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (col + i < p.I) d[col + i] = sum[i];
        }
      }
    }
  }
  } else {
    if constexpr (kShift) regs_inc<104>();
    const int q = warp & 3, we = warp - kFirstEpi;
    // one set of warps reads every accumulator, 64 columns a warp, or two sets one
    // accumulator each, 128 columns a warp in turn
    const int set = SETS == 2 && we >= C::EW / 2, part = (we - set * (C::EW / 2)) / 4 * SETS;
    constexpr int PART = 64;                      // columns of an epilogue warp
    uint8_t* box = boxes + we * kBox;
    uint32_t n = 0;      // accumulators read
    uint32_t boxes_in = 0, late_in = 0;
    // one window: TMEM columns of this warp, or false when a wait gave up
    auto window = [&](uint32_t& taddr) {
      const int acc = SETS == 1 ? n & 1 : set;
      if (!wait_bar(tfull(acc), (SETS == 1 ? n >> 1 : n) & 1, g)) return false;
      tc_fence_after();
      taddr = tmem + (uint32_t)(acc * BN + part * PART) + ((uint32_t)(q * 32) << 16);
      return true;
    };
    // the window's columns are read: the MMAs may overwrite them
    auto release = [&]() {
      const int acc = SETS == 1 ? n & 1 : set;
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (CG == 2) arrive_cluster(map_rank(tempty(acc), 0));
        else mbar_arrive(tempty(acc));
      }
      ++n;
    };
    if constexpr (MODE == kWeight) {
      for (int u = group; u < p.units; u += groups) {
        int ti, tj, kt0, kt1, split;
        unit_of(u, ti, tj, kt0, kt1, split);
        const int64_t row = (int64_t)(ti * CG + (int)rank) * BM + q * 32 + lane;
        const int64_t col0 = (int64_t)tj * BN + part * PART;
        uint32_t taddr;
        // the windows' sums are added here, in fp32 with rounding to nearest
        float v[PART / 32][32];
        bool ok = true;
        for (int w0 = kt0; w0 < kt1; w0 += p.window) {
          if (!window(taddr)) { ok = false; break; }
#pragma unroll
          for (int c = 0; c < PART / 32; ++c) {
            uint32_t r[32];
            tmem_ld32_async(taddr + (uint32_t)(32 * c), r);
            tmem_wait_ld(r);
            if (w0 == kt0) {
#pragma unroll
              for (int j = 0; j < 32; ++j) v[c][j] = __uint_as_float(r[j]);
            } else {
#pragma unroll
              for (int j = 0; j < 32; ++j) v[c][j] += __uint_as_float(r[j]);
            }
          }
          release();
        }
        if (!ok) break;
        if (row < p.I) {
          float* o = p.part ? p.part + ((int64_t)split * p.I + row) * p.ldp
                            : static_cast<float*>(p.e.out) + row * p.e.ldo;
#pragma unroll
          for (int c = 0; c < PART / 32; ++c) {
            const int64_t cc = col0 + 32 * c;
#pragma unroll
            for (int i = 0; i < 4; ++i) {      // 32-byte pieces: whole sectors
              const int64_t c8 = cc + 8 * i;
              if (p.wide_out && c8 + 8 <= p.J) {
                uint32_t w[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j] = __float_as_uint(v[c][8 * i + j]);
                store_32b(o + c8, w);
              } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                  if (c8 + j < p.J) o[c8 + j] = v[c][8 * i + j];
              }
            }
          }
        }
      }
    } else {
      const int I = (int)p.I, J = (int)p.J;
      // the places (row, column) of this unit, the next and the one after, walked
      // without the divisions of unit_of
      struct Place {
        int r, c;
      };
      const int u0 = group + set * groups, first = u0 / p.tiles_j, step = SETS * groups / p.tiles_j;
      const int dr = step * (CG * BM), dc = (SETS * groups - step * p.tiles_j) * BN, wrap = p.tiles_j * BN;
      Place at{(first * CG + (int)rank) * BM + q * 32, (u0 - first * p.tiles_j) * BN + part * PART};
      auto after = [&](Place x) {
        x.r += dr;
        x.c += dc;
        if (x.c >= wrap) {
          x.c -= wrap;
          x.r += CG * BM;
        }
        return x;
      };
      // the input box of a unit (lane 0; nothing where the box is off the matrix;
      // rows of units past the last are)
      auto send = [&](const Place& x) {
        if (x.r >= I || x.c >= J) return;
        mbar_arrive_expect_tx(box_bar(we), kBox);
        tma_load_2d(smem_u32(box), &tmI, x.c, x.r, box_bar(we));
      };
      // and its residual's rows 16 h ..
      uint8_t* late = boxes + C::EW * kBox + we * (kBox / 2);
      const CUtensorMap* tmL = MODE == kForward ? &tmI : &tmP;      // (not used otherwise)
      auto send_late = [&](const Place& x, int h) {
        if (x.r + 16 * h >= I || x.c >= J) return;
        mbar_arrive_expect_tx(late_bar(we), kBox / 2);
        tma_load_2d(smem_u32(late), tmL, x.c, x.r + 16 * h, late_bar(we));
      };
      // this thread's row of a unit's box, towards L2
      auto fetch = [&](const Place& x) {
        if (x.r + lane >= I || x.c >= J) return;
        const int64_t r = x.r + lane;
        if (p.tma_in && p.in == 2) prefetch_l2(static_cast<const __nv_bfloat16*>(p.e.pre) + r * p.e.ldpre + x.c);
        if (p.tma_in && p.in == 1 || LATE && p.tma_late)
          prefetch_l2(static_cast<const __nv_bfloat16*>(p.e.res) + r * p.e.ldres + x.c);
      };
      Place soon = after(at), later = after(soon);
      // boxes in their order: SETS side by side of each unit
      auto beside = [&](const Place& x, int sub) { return Place{x.r, x.c + sub * PART}; };
      auto next_box = [&](int sub) { return sub + 1 < SETS ? beside(at, sub + 1) : soon; };
      if (lane == 0 && p.tma_in) send(at);
      if (LATE && lane == 0 && p.tma_late) send_late(at, 0);
      if (p.in || LATE) fetch(next_box(0));
      bool ok = true;
      for (int u = u0; u < p.units && ok;
           u += SETS * groups, at = soon, soon = later, later = after(later)) {
        uint32_t taddr;
        if (!window(taddr)) break;
#pragma unroll 1
        for (int sub = 0; sub < SETS; ++sub) {
          const int row0 = at.r, col0 = at.c + sub * PART;
          const bool there = row0 < I && col0 < J;
          if (there && p.in) {
            if (p.tma_in) {
              ok = wait_bar(box_bar(we), boxes_in & 1, g);
              ++boxes_in;
            } else {
              if (lane == 0) bulk_wait_read0();
              __syncwarp();
              box_load_slow(box, lane, p.in == 1 ? p.e.res : p.e.pre,
                            p.in == 1 ? p.e.ldres : p.e.ldpre, row0, col0, p.I, p.J, 32);
              __syncwarp();
            }
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
          }
          // towards L2: the box after the next
          if (there && (p.in || LATE)) fetch(SETS == 2 ? beside(soon, sub) : later);
          float2 bi[8];      // this thread's columns: c8 + 8 i, + 1
          const int c8 = col0 + 2 * (lane & 3);
          if constexpr (MODE == kForward) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              bi[i] = make_float2(0.f, 0.f);
              if (p.e.bias && there)
                bi[i] = col0 + PART <= J
                            ? __ldg(reinterpret_cast<const float2*>(p.e.bias + c8 + 8 * i))
                            : bias_slow(p.e.bias, c8 + 8 * i, J);
            }
          }
          // `rows` rows of the box to where they belong (by TMA: after a fence).  A TMA
          // store ends on 16 bytes, not on the matrix's last column: a box that reaches
          // past a width that is no multiple of 8 is stored by hand, or it would
          // overwrite what follows the row.
          const bool inside = col0 + PART <= J || (J & 7) == 0;
          auto leave = [&](uint8_t* from, const CUtensorMap* tm, bool tma, void* base, int64_t ld,
                           int r0, int rows) {
            if (tma && inside) {
              if (lane == 0 && r0 < I) tma_store_2d(tm, smem_u32(from), col0, r0);
            } else {
              box_store_slow(from, lane, base, ld, r0, col0, p.I, p.J, rows);
              __syncwarp();
            }
          };
          const bool two = MODE == kForward && p.e.pre;   // results: pre as well
#pragma unroll 1
          for (int hr = 0; hr < 2; ++hr) {      // 16 rows at a time
            uint32_t r[32];
            tmem_ld_16x64(taddr + (uint32_t)(sub * PART) + ((uint32_t)(16 * hr) << 16), r);
            if (sub == SETS - 1 && hr == 1) release();
            const int r0 = row0 + 16 * hr;
            // the residual's box takes the next rows
            auto late_next = [&]() {
              if (LATE && p.tma_late && lane == 0) {
                if (hr == 0) send_late(at, 1);
                else send_late(soon, 0);
              }
            };
            if (!there) {
              late_next();
              continue;
            }
            float2 v[16];      // v[2 i + b]: column group i, row lane / 4 + 8 b
#pragma unroll
            for (int k = 0; k < 16; ++k)
              v[k] = make_float2(__uint_as_float(r[2 * k]), __uint_as_float(r[2 * k + 1]));
            if constexpr (MODE == kForward) {
#pragma unroll
              for (int k = 0; k < 16; ++k) v[k] = ffma2(v[k], both(1.f), bi[k / 2]);
              if (p.e.pre) {
                // (halves: the last stores have read them)
                if (lane == 0) bulk_wait_read0();
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                  uint32_t w[4];
#pragma unroll
                  for (int j = 0; j < 4; ++j) w[j] = pack_bf16x2(v[2 * i + j].x, v[2 * i + j].y);
                  quad_put(box, lane, i, w);
                }
              }
              act_chunk(p.e.act, v);
            }
            uint8_t* half = two ? box + 2048 : box + 2048 * hr;
            if (p.in) {
              uint32_t x[16];
#pragma unroll
              for (int i = 0; i < 8; i += 2) quad_get(half, lane, i, x + 2 * i);
              if (MODE == kData && p.in == 2) {
                slope_chunk(p.e.act, x, v);
              } else {
#pragma unroll
                for (int k = 0; k < 16; ++k) v[k] = ffma2(v[k], both(1.f), unpack_bf16x2(x[k]));
              }
              __syncwarp();   // all have read the half
            } else if (hr == 0 && !two) {
              if (lane == 0) bulk_wait_read0();
              __syncwarp();
            }
            if constexpr (LATE) {
              if (p.tma_late) {
                if (r0 < I) {      // (rows off the matrix are not stored)
                  ok = __all_sync(0xffffffffu, wait_bar(late_bar(we), late_in & 1, g));
                  if (!ok) break;
                  ++late_in;
                }
              } else {
                box_load_slow(late, lane, p.e.res, p.e.ldres, r0, col0, p.I, p.J, 16);
                __syncwarp();
              }
#pragma unroll
              for (int i = 0; i < 8; i += 2) {
                uint32_t x[4];
                quad_get(late, lane, i, x);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                  v[2 * i + j] = ffma2(v[2 * i + j], both(1.f), unpack_bf16x2(x[j]));
              }
              fence_proxy_async_smem();      // (read by all lanes before it is written again)
              __syncwarp();
              late_next();
            }
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
              uint32_t w[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) w[j] = pack_bf16x2(v[2 * i + j].x, v[2 * i + j].y);
              quad_put(half, lane, i, w);
            }
            if (two || hr == 1) {
              fence_proxy_async_smem();
              __syncwarp();
              if (two) {
                leave(box, &tmP, p.tma_pre, p.e.pre, p.e.ldpre, r0, 16);
                leave(half, &tmO, p.tma_out, p.e.out, p.e.ldo, r0, 16);
              } else {
                leave(box, &tmO, p.tma_out, p.e.out, p.e.ldo, row0, 32);
              }
              if (lane == 0) bulk_commit();
            }
          }
          if (!ok) break;
          // the box takes the next unit's input
          if (p.tma_in && lane == 0) {
            bulk_wait_read0();
            send(next_box(sub));
          }
        }
      }
    }
    // a box that was sent for but not used (after an abort)
    if (MODE != kWeight && p.tma_in && lane == 0 && *abort_flag)
      drain_wait(box_bar(we), boxes_in & 1, 1000000ull);
    if (LATE && p.tma_late && lane == 0 && *abort_flag)
      drain_wait(late_bar(we), late_in & 1, 1000000ull);
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
template <int CG, int BN, int MODE, bool AMN, bool BMN, bool LATE = false, int SETS = 1>
cudaError_t launch(const Product& g, TcArgs p, int sms, cudaStream_t st) {
  using C = TileCfg<CG, BN, MODE, LATE>;
  CUtensorMap ta, tb, to, tp, ti;
  cudaError_t e;
  const int64_t pa = 3 * p.plane_a, pb = 3 * p.plane_b;   // all rows of planes
  if (AMN) e = tc_make_tmap(&ta, g.A, g.I, pa ? pa : g.R, g.sar, 64, BK);
  else e = tc_make_tmap(&ta, g.A, g.R, pa ? pa : g.I, g.sai, BK, BM);
  if (e != cudaSuccess) return e;
  if (BMN) e = tc_make_tmap(&tb, g.B, g.J, pb ? pb : g.R, g.sbr, 64, BK);
  else e = tc_make_tmap(&tb, g.B, g.R, pb ? pb : g.J, g.sbj, BK, C::B_ROWS);
  if (e != cudaSuccess) return e;
  to = ta;
  tp = ta;
  ti = ta;
  if (MODE != kWeight && p.tma_out) {
    e = tc_make_tmap(&to, p.e.out, p.J, p.I, p.e.ldo, 64,
                     MODE == kForward && p.e.pre ? 16 : 32);
    if (e != cudaSuccess) return e;
  }
  if (MODE != kWeight && p.tma_pre) {
    e = tc_make_tmap(&tp, p.e.pre, p.J, p.I, p.e.ldpre, 64, 16);
    if (e != cudaSuccess) return e;
  }
  if (MODE != kWeight && p.tma_in) {
    e = p.in == 1 ? tc_make_tmap(&ti, p.e.res, p.J, p.I, p.e.ldres, 64, 32)
                  : tc_make_tmap(&ti, p.e.pre, p.J, p.I, p.e.ldpre, 64, 32);
    if (e != cudaSuccess) return e;
  }
  if (LATE && p.tma_late) {
    e = tc_make_tmap(MODE == kForward ? &ti : &tp, p.e.res, p.J, p.I, p.e.ldres, 64, 16);
    if (e != cudaSuccess) return e;
  }
  const auto kernel = lin_tc_kernel<CG, BN, MODE, AMN, BMN, LATE, SETS>;
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
  cfg.blockDim = dim3(C::THREADS);
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
  return cudaLaunchKernelEx(&cfg, kernel, ta, tb, to, tp, ti, p);
}

template <int CG, int BN>
cudaError_t launch_mode(const Product& g, const TcArgs& p, int mode, int sms, cudaStream_t st) {
  if (p.part || mode == kWeight) {
    if (mode == kWeight) return launch<CG, BN, kWeight, true, true>(g, p, sms, st);
    if (mode == kForward) return launch<CG, BN, kWeight, false, false>(g, p, sms, st);
    return launch<CG, BN, kWeight, false, true>(g, p, sms, st);
  }
  const bool late = p.e.res && p.in != 1;
  // Two sets of epilogue warps where there is little to compute and there are
  // tiles enough: one set computes while the other waits (for TMEM, its input, a
  // fence, a store).  32,768 x 512 -> 2,048 forward 59 us with one set, 53 with two;
  // 65,536 x 512 -> 2,048 data gradient 105 and 95, with a residual 121 and 112;
  // 16,384 x 4,096 -> 2,048 forward with one 163 and 155; but 65 and 68 at 32,768 x
  // 512 -> 2,048, and 124 and 148 with gelu' of the data gradient.
  if constexpr (CG == 2) {
    const bool light = p.e.act == PPO_ACT_NONE || p.e.act == PPO_ACT_RELU;
    const bool short_in = mode == kForward && p.in && p.R < 1024;
    if (!late && light && !short_in && p.units >= 4 * (sms / CG))
      return mode == kForward ? launch<CG, BN, kForward, false, false, false, 2>(g, p, sms, st)
                              : launch<CG, BN, kData, false, true, false, 2>(g, p, sms, st);
  }
  if (mode == kForward)
    return late ? launch<CG, BN, kForward, false, false, true>(g, p, sms, st)
                : launch<CG, BN, kForward, false, false>(g, p, sms, st);
  return late ? launch<CG, BN, kData, false, true, true>(g, p, sms, st)
              : launch<CG, BN, kData, false, true>(g, p, sms, st);
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace

// The cheapest of the tile shapes and splits for a whole GB300, by the rounds
// its units take: a 64-deep step of a unit costs a pair of CTAs and a single
// CTA (128 x 128) about 300 and 200 ns, a unit's start and epilogue 2 us, and
// a split product writes and re-reads its partial products.
TcPlan tc_plan(int64_t I, int64_t J, int64_t R, bool must_split, int terms) {
  constexpr int kSms = 152;
  TcPlan best{};
  double best_cost = 0;
  const int64_t kt = cdiv(R, BK) * terms;
  for (int cg = 1; cg <= 2; ++cg) {
    const int64_t ti = cdiv(I, cg * BM), tj = cdiv(J, cg == 2 ? 256 : 128);
    const double step = cg == 2 ? 0.30 : 0.20;
    int64_t last = -1;
    for (int64_t s = 1; s <= 32 && s <= kt; ++s) {
      const int64_t per = cdiv(cdiv(kt, s), terms) * terms, used = cdiv(kt, per);
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

int64_t tc_sum_rows(const Product& g, const TcPlan& plan) {
  return (int64_t)plan.splits * cdiv(g.J, plan.cg == 2 ? 256 : 128);
}

cudaError_t tc_product(const Product& g, const Epilogue& e, const TcPlan& plan, float* part,
                       float* db_part, int* err, int sms, cudaStream_t st, int64_t plane_a,
                       int64_t plane_b) {
  TcArgs p{};
  p.I = g.I;
  p.J = g.J;
  p.R = g.R;
  p.tiles_i = (int)cdiv(g.I, plan.cg * BM);
  p.tiles_j = (int)cdiv(g.J, plan.cg == 2 ? 256 : 128);
  p.plane_a = plane_a;
  p.plane_b = plane_b;
  p.k_tiles = (int)cdiv(g.R, BK) * (plane_a ? kTerms : 1);
  p.kt_per_split = plan.kt_per_split;
  p.window = plane_a ? kTerms : e.mode == kWeight || part ? kWindow : p.k_tiles;
  const int64_t units = (int64_t)p.tiles_i * p.tiles_j * plan.splits;
  if (units > (1ll << 30)) return cudaErrorInvalidValue;
  p.units = (int)units;
  p.e = e;
  p.part = part;
  p.ldp = part_pitch(g.J);
  p.err = err;
  auto al = [](const void* q, int64_t ld, int m) { return ops::al16(q) && ld % m == 0; };
  p.tma_out = al(e.out, e.ldo, 8);
  p.tma_pre = e.mode == kForward && e.pre && al(e.pre, e.ldpre, 8);
  if (!part && e.mode != kWeight) {
    p.in = e.mode == kData && e.act != PPO_ACT_NONE ? 2 : e.res && !e.pre ? 1 : 0;
    p.tma_in = p.in == 1 ? al(e.res, e.ldres, 8) : p.in == 2 && al(e.pre, e.ldpre, 8);
    p.tma_late = e.res && p.in != 1 && al(e.res, e.ldres, 8);
  }
  p.db_part = db_part;
  const void* f32_out = part ? part : e.out;
  p.wide_out = ((reinterpret_cast<uintptr_t>(f32_out) | (uintptr_t)((part ? p.ldp : e.ldo) * 4)) & 31) == 0;
  if (plan.cg == 2) return launch_mode<2, 256>(g, p, e.mode, sms, st);
  return launch_mode<1, 128>(g, p, e.mode, sms, st);
}

}  // namespace lin
}  // namespace ppo
