// glinear_skinny.cu -- gated linear layers in bf16 for up to 64 rows: W streamed
// through the tensor cores once.
//
// The rows of x are the narrow operand: a CTA's 128 accumulator lanes are 64 rows of
// the gate's W and the 64 of the other projection's for the same columns, its 16, 32,
// 48 or 64 accumulator columns are x's rows, so that what it takes in by TMA is W and
// little else (a tile of 128 rows of x would cost as much again, most of it
// padding).  The sum is cut over the 1, 2 or 4 CTAs of a cluster, whatever fills the
// GPU; each leaves its part in its shared memory, and after a cluster barrier each
// adds up its share of x's rows from all of them, in order, and finishes it: bias,
// pre-activations, activation, product.
//
// What bounds it: W's bytes, and the start and end of a launch that lasts as long as
// two of those.  33 rows of 4,096 -> 4,096, W not in L2: 16.2 us, 10 by W's bytes (in
// tiles of 128 x 128 with the sum cut in two and a second launch 19.1); 4 rows 15.3 (22
// on the CUDA cores), 64 rows 17.0 (20.3), 40 x 4,096 -> 1,000 9.7 (11.4), 33 x 512 -> 2,048
// 5.4 (6.0).  Parts sent to the CTA that adds them up cost more than parts fetched by it:
// 19.8 element by element, 18.4 by bulk copies.
//
// Every wait on an mbarrier is bounded; on expiry the kernel sets the error
// word, stops issuing, drains what is in flight and frees its TMEM.
#include <algorithm>

#include "gemm.h"
#include "glinear.h"
#include "lin_tile.cuh"

namespace ppo {
namespace glin {
namespace {

using namespace lin;

constexpr int kThreads = 128;
constexpr int kCols = 64;              // gated columns of a tile
constexpr int kMostRows = 64;
constexpr int kMostCtas = 4;           // (40 x 4,096 -> 1,000: 11.4 us with four, 17 with eight)

template <int MP>
struct Cfg {
  static constexpr int A_BYTES = 2 * kCols * BK * 2;
  static constexpr int STAGE = A_BYTES + MP * BK * 2;
  static constexpr int S = 6;
  static constexpr int PART = MP * 2 * kCols * 4;      // [MP][128] sums
  static constexpr int TMEM = MP <= 32 ? 32 : 64;
  static constexpr size_t SMEM = 1024 + (size_t)S * STAGE + PART + 256;
  static_assert(SMEM <= 232448, "shared memory per CTA");
};

struct SkinnyArgs {
  int M, N, k_tiles;
  int act;
  const float* bias;
  void* pre;
  int64_t ldpre;
  void* y;
  int64_t ldy;
  int* err;
};

__device__ __forceinline__ float4 ld_cluster(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr));
  return v;
}
__device__ __forceinline__ void add4(float4& a, const float4& b) {
  a.x += b.x;
  a.y += b.y;
  a.z += b.z;
  a.w += b.w;
}

template <int MP>
__global__ void __launch_bounds__(kThreads, 1)
skinny_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const SkinnyArgs p) {
  using C = Cfg<MP>;
  constexpr int S = C::S;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  float* part = reinterpret_cast<float*>(gbase + (size_t)S * C::STAGE);
  uint64_t* bars = reinterpret_cast<uint64_t*>(gbase + (size_t)S * C::STAGE + C::PART);
  // full[S] empty[S] done drain
  auto full = [&](int s) { return smem_u32(&bars[s]); };
  auto empty = [&](int s) { return smem_u32(&bars[S + s]); };
  const uint32_t done = smem_u32(&bars[2 * S]), drain = smem_u32(&bars[2 * S + 1]);
  uint32_t* tslot = reinterpret_cast<uint32_t*>(&bars[2 * S + 2]);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tslot + 1);
  volatile uint32_t* cnt = reinterpret_cast<volatile uint32_t*>(tslot + 2);   // issued, consumed
  static_assert((2 * S + 2) * 8 + 16 <= 256, "control block");

  const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp;
  uint32_t ctas;
  asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(ctas));
  const uint32_t rank = lin::cluster_rank();
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    mbar_init(done, 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    cnt[0] = cnt[1] = 0;
    fence_mbar_init();
  }
  if (warp == 1) alloc<1>(smem_u32(tslot), C::TMEM);
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tmW);
    prefetch_tmap(&tmX);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  const Guard g{abort_flag, p.err, kWaitNs};
  const int j0 = (int)(blockIdx.x / ctas) * kCols;
  const int kt0 = (int)((int64_t)p.k_tiles * rank / ctas), kt1 = (int)((int64_t)p.k_tiles * (rank + 1) / ctas);
  pdl_wait();
  pdl_trigger();
  if (warp == 0 && lane == 0) {
    int s = 0;
    uint32_t it = 0, ph = 0;
    bool ok = true;
    for (int kt = kt0; kt < kt1; ++kt) {
      if (!wait_bar(empty(s), ph ^ 1, g)) { ok = false; break; }
      const uint32_t at = base + (uint32_t)(s * C::STAGE);
      mbar_arrive_expect_tx(full(s), C::STAGE);
      tma_load_2d(at, &tmW, kt * BK, j0, full(s));
      tma_load_2d(at + C::A_BYTES / 2, &tmW, kt * BK, p.N + j0, full(s));
      tma_load_2d(at + C::A_BYTES, &tmX, kt * BK, 0, full(s));
      cnt[0] = ++it;
      if (++s == S) { s = 0; ph ^= 1; }
    }
    // every stage released: no commit is still to arrive here when the CTA leaves
    if (ok)
      for (int j = 0; j < S; ++j) {
        if (!wait_bar(empty(s), ph ^ 1, g)) break;
        if (++s == S) { s = 0; ph ^= 1; }
      }
  } else if (warp == 1 && lane == 0) {
    constexpr uint32_t idesc = idesc_bf16(2 * kCols, MP, false, false);
    int s = 0;
    uint32_t it = 0, ph = 0;
    bool ok = true;
    for (int kt = kt0; kt < kt1; ++kt) {
      if (!wait_bar(full(s), ph, g)) { ok = false; break; }
      tc_fence_after();
      const uint32_t at = base + (uint32_t)(s * C::STAGE);
#pragma unroll
      for (int kk = 0; kk < BK / 16; ++kk)
        mma<1>(tmem, sdesc_sw128(at + kk * 32, 16, 1024), sdesc_sw128(at + C::A_BYTES + kk * 32, 16, 1024), idesc,
               (kt != kt0 || kk != 0) ? 1u : 0u);
      commit<1>(empty(s));
      cnt[1] = ++it;
      if (++s == S) { s = 0; ph ^= 1; }
    }
    if (ok) commit<1>(done);
  }
  __syncwarp();
  // this thread's W row against all rows of x
  const bool ok = wait_bar(done, 0, g);
  __syncwarp();
  if (__all_sync(0xffffffffu, ok)) {
    tc_fence_after();
    const uint32_t at = tmem + ((uint32_t)(warp * 32) << 16);
    float v[32];
#pragma unroll
    for (int c = 0; c < MP; c += 32) {
      if (MP - c >= 32) tmem_ld32(at + (uint32_t)c, v);
      else tmem_ld16(at + (uint32_t)c, v);
#pragma unroll
      for (int k = 0; k < 32 && c + k < MP; ++k) part[(c + k) * (2 * kCols) + threadIdx.x] = v[k];
    }
  }
  tc_fence_before();
  __syncthreads();
  if (*abort_flag) {
    // loads that were issued but never consumed, and outstanding MMAs
    if (threadIdx.x == 0) {
      const uint32_t issued = cnt[0], consumed = cnt[1];
      for (uint32_t it = consumed; it < issued; ++it) drain_wait(full(it % S), (it / S) & 1, kWaitNs);
    }
    if (warp == 1 && lane == 0) {
      tc_commit(drain);
      drain_wait(drain, 0, kWaitNs);
    }
    __syncthreads();
  }
  if (warp == 1) {
    tc_fence_after();
    dealloc<1>(tmem, C::TMEM);
  }
  cluster_sync();      // every CTA's part is there
  {
    // four columns a thread, eight rows of x at a time
    constexpr int kVec = kCols / 4;
    const int c = threadIdx.x % kVec * 4, j = j0 + c, n = min(4, p.N - j);
    uint32_t at[kMostCtas];
#pragma unroll
    for (int i = 0; i < kMostCtas; ++i) at[i] = map_rank(smem_u32(part), i < (int)ctas ? i : 0) + c * 4;
    float b0[4], b1[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      b0[e] = p.bias && e < n ? p.bias[j + e] : 0.f;
      b1[e] = p.bias && e < n ? p.bias[p.N + j + e] : 0.f;
    }
    for (int m = (int)rank + (int)ctas * (threadIdx.x / kVec); m < p.M; m += (int)ctas * (kThreads / kVec)) {
      float4 a[kMostCtas], u[kMostCtas];
#pragma unroll
      for (int i = 0; i < kMostCtas; ++i)
        if (i < (int)ctas) {
          a[i] = ld_cluster(at[i] + (uint32_t)m * (2 * kCols * 4));
          u[i] = ld_cluster(at[i] + (uint32_t)m * (2 * kCols * 4) + kCols * 4);
        }
#pragma unroll
      for (int i = 1; i < kMostCtas; ++i)
        if (i < (int)ctas) {
          add4(a[0], a[i]);
          add4(u[0], u[i]);
        }
      const float va[4] = {a[0].x, a[0].y, a[0].z, a[0].w}, vu[4] = {u[0].x, u[0].y, u[0].z, u[0].w};
      __nv_bfloat16* y = static_cast<__nv_bfloat16*>(p.y) + (int64_t)m * p.ldy + j;
      __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.pre) + (int64_t)m * p.ldpre + j;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (e >= n) break;
        const float ga = va[e] + b0[e], up = vu[e] + b1[e];
        if (p.pre) {
          o[e] = __float2bfloat16_rn(ga);
          o[p.N + e] = __float2bfloat16_rn(up);
        }
        y[e] = __float2bfloat16_rn(ops::act_value<false>(p.act, ga) * up);
      }
    }
  }
  cluster_sync();      // no CTA leaves while another reads its part
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

template <int MP>
cudaError_t launch(const Product& m, const Gate& g, int ctas, int* err, cudaStream_t st) {
  using C = Cfg<MP>;
  SkinnyArgs p{(int)g.M, (int)g.N, (int)cdiv(m.R, BK), g.act, g.bias, g.pre, g.ldpre, g.y, g.ldy, err};
  CUtensorMap tw, tx;
  cudaError_t e = tc_make_tmap(&tw, m.B, m.R, 2 * g.N, m.sbj, BK, kCols);
  if (e == cudaSuccess) e = tc_make_tmap(&tx, m.A, m.R, g.M, m.sai, BK, MP);
  if (e != cudaSuccess) return e;
  static thread_local int prepared = -1;   // the device whose shared-memory opt-in is made
  int dev = 0;
  e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (prepared != dev) {
    e = cudaFuncSetAttribute(skinny_kernel<MP>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM);
    if (e != cudaSuccess) return e;
    prepared = dev;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(cdiv(g.N, kCols) * ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)ctas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, skinny_kernel<MP>, tw, tx, p);
}

}  // namespace

int skinny_ctas(int64_t M, int64_t N, int64_t R) {
  constexpr int kSms = 152;
  // (longer sums drift in the accumulator; a column tile is a block)
  if (M > kMostRows || R > 1ll << 16 || N > 1ll << 24) return 0;
  const int64_t kt = cdiv(R, BK), tiles = cdiv(N, kCols);
  int best = 1;
  double cost = 0;
  for (int c = 1; c <= kMostCtas && c <= kt; c *= 2) {
    // rounds of the GPU's SMs, of steps of 0.2 us, a start of 3 and a join of 0.5
    const double t = (double)cdiv(tiles * c, kSms) * (cdiv(kt, c) * 0.2 + (c > 1 ? 3.5 : 3.0));
    if (c == 1 || t < cost) {
      best = c;
      cost = t;
    }
  }
  return best;
}
cudaError_t skinny_forward(const Product& m, const Gate& g, int ctas, int* err, cudaStream_t st) {
  if (g.M <= 16) return launch<16>(m, g, ctas, err, st);
  if (g.M <= 32) return launch<32>(m, g, ctas, err, st);
  if (g.M <= 48) return launch<48>(m, g, ctas, err, st);
  return launch<kMostRows>(m, g, ctas, err, st);
}

}  // namespace glin
}  // namespace ppo
