// glinear.cu -- gated linear layers: two projections of the same rows, the gate
// through its activation, and their product; and the gradient of both from that
// of the layer behind.
//
//   forward    pre = x W^T + b  [M][2N],  y = act(g) u,  g | u the halves of pre
//   backward   d = dz W2  [M][N],  dp = [ d u act'(g) | d act(g) ],  y = act(g) u
//
// bf16 products finish their tiles in the same kernel (glinear_tc.cu) where there are
// tiles enough.  Others leave fp32 sums, partial ones where the sum is split, and one
// kernel here finishes them: what it writes is rounded once, from fp32.  Forward
// products of few rows have kernels of their own.
// fp32, 4,999 x 512 -> 1,365, forward with pre and backward with y: 198 us, floor 66 as six
// bf16 products; of them the planes 14, the products 123, the gates 60 for the 300 MB
// that they read and write (75 with a choice of activation for each element and a division
// for each run).  Up to 64
// bf16 rows: glinear_skinny.cu.
#include <algorithm>

#include "glinear.h"
#include "lin_again.cuh"
#include "ops.cuh"
#include "tc_ptx.cuh"

namespace ppo {
namespace glin {
namespace {

using namespace ops;

constexpr int kThreads = 256;
constexpr int kSms = 152;

// A block takes runs of kRun columns of a row, its threads one column in kThreads of them,
// all loads first: rows may start anywhere.
constexpr int kPer = 4, kRun = kPer * kThreads;

// f(row, this thread's first column, how many of its columns there are) of this block's
// runs, all of about one length: blocks along y take a row's runs, those along x the rows
template <typename F>
__device__ __forceinline__ void each_run(const Gate& g, F f) {
  const int per = (int)((g.N + kRun - 1) / kRun);
  const int len = (int)((g.N + per - 1) / per + kWarp - 1) / kWarp * kWarp;
  for (int c = blockIdx.y; c < per; c += gridDim.y) {
    const int j = c * len + (int)threadIdx.x, end = min((int)g.N, (c + 1) * len);
    if (j >= end) continue;
    const int count = (end - j + kThreads - 1) / kThreads;
    for (int64_t i = blockIdx.x; i < g.M; i += gridDim.x) f(i, j, count);
  }
}
// kPer elements, kThreads apart, of which `count` are there
template <typename T>
__device__ __forceinline__ void run_load(const T* p, int count, float (&v)[kPer]) {
#pragma unroll
  for (int e = 0; e < kPer; ++e) v[e] = e < count ? (float)p[e * kThreads] : 0.f;
}
template <typename T>
__device__ __forceinline__ void run_store(T* p, int count, const float (&v)[kPer]) {
#pragma unroll
  for (int e = 0; e < kPer; ++e)
    if (e < count) round_to(v[e], p[e * kThreads]);
}
__device__ __forceinline__ void run_sums(const lin::PartialSums& s, int64_t i, int64_t j, int count,
                                         float (&v)[kPer]) {
  const float* p = s.part + i * s.ldp + j;
#pragma unroll
  for (int e = 0; e < kPer; ++e) v[e] = e < count ? __ldcg(p + e * kThreads) : 0.f;
  for (int k = 1; k < s.splits; ++k) {
    p += s.stride;
#pragma unroll
    for (int e = 0; e < kPer; ++e) v[e] += e < count ? __ldcg(p + e * kThreads) : 0.f;
  }
}
// What is not finite of a product of planes, looked at again.  (A pass of its own: with
// the call in the kernel's loop that loop spills, 106 us instead of 38.)
__device__ __forceinline__ bool run_finite(const float (&v)[kPer]) {
  bool f = true;
#pragma unroll
  for (int e = 0; e < kPer; ++e) f = f && isfinite(v[e]);
  return f;
}
__device__ __noinline__ void run_again(const lin::PartialSums& s, const lin::Again* again, int64_t i, int64_t j, int count,
                                       float* v) {
  for (int e = 0; e < count; ++e)
    if (!isfinite(v[e])) v[e] = lin::dot_again(again, i, j + e * kThreads, i * s.ldp + j + e * kThreads);
}

// act(a), and its slope, of a run: the choice is made once
template <int ACT>
__device__ __forceinline__ void act_run(const float (&a)[kPer], float (&v)[kPer], float (&s)[kPer]) {
#pragma unroll
  for (int e = 0; e < kPer; ++e) {
    v[e] = act_value<false>(ACT, a[e]);
    s[e] = act_slope<false>(ACT, a[e]);
  }
}
__device__ __forceinline__ void act_run(int act, const float (&a)[kPer], float (&v)[kPer], float (&s)[kPer]) {
  switch (act) {
    case PPO_ACT_TANH: act_run<PPO_ACT_TANH>(a, v, s); break;
    case PPO_ACT_RELU: act_run<PPO_ACT_RELU>(a, v, s); break;
    case PPO_ACT_SILU: act_run<PPO_ACT_SILU>(a, v, s); break;
    case PPO_ACT_GELU: act_run<PPO_ACT_GELU>(a, v, s); break;
    default: act_run<PPO_ACT_NONE>(a, v, s); break;
  }
}

template <typename T>
__device__ __forceinline__ void put_forward(const Gate& g, int64_t i, int j, int count, float (&a)[kPer],
                                            float (&u)[kPer]) {
  if (g.bias) {
    float b[kPer];
    run_load(g.bias + j, count, b);
#pragma unroll
    for (int e = 0; e < kPer; ++e) a[e] += b[e];
    run_load(g.bias + g.N + j, count, b);
#pragma unroll
    for (int e = 0; e < kPer; ++e) u[e] += b[e];
  }
  if (g.pre) {
    T* o = static_cast<T*>(g.pre) + i * g.ldpre + j;
    run_store(o, count, a);
    run_store(o + g.N, count, u);
  }
  float v[kPer], s[kPer];
  act_run(g.act, a, v, s);
#pragma unroll
  for (int e = 0; e < kPer; ++e) v[e] *= u[e];
  run_store(static_cast<T*>(g.y) + i * g.ldy + j, count, v);
}
template <typename T>
__device__ __forceinline__ void put_backward(const Gate& g, int64_t i, int j, int count, const float (&d)[kPer],
                                             const float (&a)[kPer], const float (&u)[kPer]) {
  float v[kPer], s[kPer], x[kPer];
  act_run(g.act, a, v, s);
  T* o = static_cast<T*>(g.dp) + i * g.lddp + j;
#pragma unroll
  for (int e = 0; e < kPer; ++e) x[e] = d[e] * s[e] * u[e];      // (d u may overflow where s is 0)
  run_store(o, count, x);
#pragma unroll
  for (int e = 0; e < kPer; ++e) x[e] = d[e] * v[e];
  run_store(o + g.N, count, x);
  if (!g.y) return;
#pragma unroll
  for (int e = 0; e < kPer; ++e) x[e] = v[e] * u[e];
  run_store(static_cast<T*>(g.y) + i * g.ldy + j, count, x);
}

__device__ __noinline__ void forward_again(const Gate& g, const lin::Again* again) {
  each_run(g, [&](int64_t i, int j, int count) {
    float a[kPer], u[kPer];
    run_sums(g.s, i, j, count, a);
    run_sums(g.s, i, g.N + j, count, u);
    if (run_finite(a) && run_finite(u)) return;
    run_again(g.s, again, i, j, count, a);
    run_again(g.s, again, i, g.N + j, count, u);
    put_forward<float>(g, i, j, count, a, u);
  });
}
template <typename T, bool PLANES>
__global__ void __launch_bounds__(kThreads)
gate_forward_kernel(const __grid_constant__ Gate g, const __grid_constant__ lin::Again again) {
  pdl_wait();
  bool left = false;
  each_run(g, [&](int64_t i, int j, int count) {
    float a[kPer], u[kPer];
    run_sums(g.s, i, j, count, a);
    run_sums(g.s, i, g.N + j, count, u);
    if (PLANES && !(run_finite(a) && run_finite(u))) left = true;
    else put_forward<T>(g, i, j, count, a, u);
  });
  if (PLANES && left) forward_again(g, &again);
}

__device__ __noinline__ void backward_again(const Gate& g, const lin::Again* again) {
  each_run(g, [&](int64_t i, int j, int count) {
    float d[kPer], a[kPer], u[kPer];
    run_sums(g.s, i, j, count, d);
    if (run_finite(d)) return;
    run_again(g.s, again, i, j, count, d);
    const float* p = static_cast<const float*>(g.pre_in) + i * g.ldin + j;
    run_load(p, count, a);
    run_load(p + g.N, count, u);
    put_backward<float>(g, i, j, count, d, a, u);
  });
}
template <typename T, bool PLANES>
__global__ void __launch_bounds__(kThreads)
gate_backward_kernel(const __grid_constant__ Gate g, const __grid_constant__ lin::Again again) {
  pdl_wait();
  bool left = false;
  each_run(g, [&](int64_t i, int j, int count) {
    const T* p = static_cast<const T*>(g.pre_in) + i * g.ldin + j;
    float d[kPer], a[kPer], u[kPer];
    run_load(p, count, a);
    run_load(p + g.N, count, u);
    run_sums(g.s, i, j, count, d);
    if (PLANES && !run_finite(d)) left = true;
    else put_backward<T>(g, i, j, count, d, a, u);
  });
  if (PLANES && left) backward_again(g, &again);
}

template <typename K>
cudaError_t finish(K kernel, const Gate& g, const lin::Product& m, cudaStream_t st) {
  const int64_t runs = std::min<int64_t>((g.N + kRun - 1) / kRun, 1024);
  const int64_t rows = std::min<int64_t>(g.M, std::max<int64_t>(1, 16 * kSms / runs));
  return launch_pdl(kernel, dim3((unsigned)rows, (unsigned)runs), dim3(kThreads), 0, st, g,
                    lin::Again{m, g.s.part, g.s.stride, g.s.splits, g.s.r_per_split});
}

// ---- a few rows ------------------------------------------------------------------------
// Forward of up to 8 rows: bound by reading W once, and for small W by the launch.  A
// group of wk warps (1, 2 or 4, along the sum) takes one output column, every lane 16
// bytes of both of its rows of W at a time and the same piece of the rows of x, which
// stay in L1; the lanes' sums are then folded until a lane holds a row's gate and its
// neighbour the other sum.  Rows off 16-byte boundaries go element by element.
constexpr int kFewRows = 8;
template <typename T, int MR>
__global__ void __launch_bounds__(kThreads)
gate_few_kernel(const __grid_constant__ lin::Product m, const __grid_constant__ Gate g, int vec, int wk) {
  constexpr int A = 2 * MR, E = 16 / (int)sizeof(T);
  constexpr int U = MR >= 4 ? 2 : 4;     // pieces of a W row in flight
  __shared__ float sums[kThreads / kWarp][A];
  pdl_wait();
  const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp;
  const int64_t j = (int64_t)blockIdx.x * (kThreads / kWarp / wk) + warp / wk;
  const int64_t jj = min(j, g.N - 1);      // (columns and rows past the last one repeat it)
  const T *x[MR], *w[2];
#pragma unroll
  for (int i = 0; i < MR; ++i) x[i] = static_cast<const T*>(m.A) + min((int64_t)i, g.M - 1) * m.sai;
  w[0] = static_cast<const T*>(m.B) + jj * m.sbj;
  w[1] = static_cast<const T*>(m.B) + (g.N + jj) * m.sbj;
  float2 pair[A];      // [row][gate, up]: sums of even and odd elements
#pragma unroll
  for (int i = 0; i < A; ++i) pair[i] = make_float2(0.f, 0.f);
  int64_t k = 0;
  if (vec) {
    const int64_t whole = m.R / E * E, step = (int64_t)wk * kWarp * E;
    for (k = ((int64_t)(warp % wk) * kWarp + lane) * E; k < whole; k += U * step) {
      Raw<T, E> rw[U][2];
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int c = 0; c < 2; ++c)
          rw[u][c] = k + u * step < whole ? __ldg(reinterpret_cast<const Raw<T, E>*>(w[c] + k + u * step))
                                          : Raw<T, E>{};
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (k + u * step >= whole) break;
        float fw[2][E];
        to_f32<T, E>(rw[u][0], fw[0]);
        to_f32<T, E>(rw[u][1], fw[1]);
#pragma unroll
        for (int i = 0; i < MR; ++i) {
          float fx[E];
          to_f32<T, E>(__ldg(reinterpret_cast<const Raw<T, E>*>(x[i] + k + u * step)), fx);
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int e = 0; e < E; e += 2)
              pair[2 * i + c] = ptx::ffma2(make_float2(fx[e], fx[e + 1]), make_float2(fw[c][e], fw[c][e + 1]),
                                           pair[2 * i + c]);
        }
      }
    }
    k = whole;
  }
  float acc[A];
#pragma unroll
  for (int i = 0; i < A; ++i) acc[i] = pair[i].x + pair[i].y;
#pragma unroll 4
  for (k += (int64_t)(warp % wk) * kWarp + lane; k < m.R; k += (int64_t)wk * kWarp) {
    const float f0 = (float)w[0][k], f1 = (float)w[1][k];
#pragma unroll
    for (int i = 0; i < MR; ++i) {
      const float f = (float)x[i][k];
      acc[2 * i] = fmaf(f, f0, acc[2 * i]);
      acc[2 * i + 1] = fmaf(f, f1, acc[2 * i + 1]);
    }
  }
  // lanes fold their sums: each keeps half of them and takes the other lane's share of
  // those, until one is left; `mine` is which
  int mine = 0;
#pragma unroll
  for (int n = A, off = 16; off >= 1; off >>= 1) {
    if (n > 1) {
      n >>= 1;
      const bool up = lane & off;
      mine += up ? n : 0;
#pragma unroll
      for (int i = 0; i < n; ++i) {
        const float give = up ? acc[i] : acc[i + n], keep = up ? acc[i + n] : acc[i];
        acc[i] = keep + __shfl_xor_sync(0xffffffffu, give, off);
      }
    } else {
      acc[0] += __shfl_xor_sync(0xffffffffu, acc[0], off);
    }
  }
  constexpr int kNext = kWarp / A;       // from a row's gate to its other sum, in lanes
  const bool holds = (lane & (kNext - 1)) == 0;
  if (wk > 1) {
    if (holds) sums[warp][mine] = acc[0];
    __syncthreads();
    if (warp % wk != 0) return;
    acc[0] = 0.f;
    for (int i = 0; i < wk; ++i) acc[0] += sums[warp + i][mine];
  }
  const int row = mine / 2, c = mine & 1;
  float v = acc[0];
  if (g.bias) v += g.bias[c * g.N + jj];
  const float u = __shfl_xor_sync(0xffffffffu, v, kNext);
  if (!holds || row >= g.M || j >= g.N) return;
  if (g.pre) round_to(v, static_cast<T*>(g.pre)[row * g.ldpre + c * g.N + j]);
  if (c == 0) round_to(act_value<false>(g.act, v) * u, static_cast<T*>(g.y)[row * g.ldy + j]);
}

template <typename T>
cudaError_t few(const lin::Product& m, const Gate& g, cudaStream_t st) {
  constexpr int E = 16 / (int)sizeof(T);
  const int vec = m.sai % E == 0 && m.sbj % E == 0;
  // warps along the sum until there are 4,096
  int wk = 1;
  while (wk < 4 && g.N * wk < 4096 && m.R >= 4 * wk * kWarp * E) wk *= 2;
  const int64_t per = kThreads / kWarp / wk;
  auto go = [&](auto kernel) {
    return launch_pdl(kernel, dim3((unsigned)((g.N + per - 1) / per)), dim3(kThreads), 0, st, m, g, vec, wk);
  };
  if (g.M <= 1) return go(gate_few_kernel<T, 1>);
  if (g.M <= 2) return go(gate_few_kernel<T, 2>);
  if (g.M <= 4) return go(gate_few_kernel<T, 4>);
  return go(gate_few_kernel<T, kFewRows>);
}
// bf16 in a graph, here / on the tensor cores: one row of 512 -> 2,048 2.7 us / 4.5, 3 rows
// 3.2 / 4.5, 8 rows 4.5 / 4.6; of 4,096 -> 4,096, W not in L2, one row 18.2 / 14.9, two rows
// 21.3 / 14.9.  Rows off 16-byte boundaries have to be copied first for those: of 1,397 -> 4,096
// one row 18.2 here, 4 to 64 rows 15.1 to 17.4 with W copied (of 1,400 8.1 to 10.6).
// (A pitch <= 0 stands for the row's length.)
template <typename T>
bool takes_few(int64_t M, int64_t N, int64_t K, int64_t ldx, int64_t ldw) {
  if (sizeof(T) == 4 || M > kFewRows) return M <= kFewRows;
  if (M <= 2 && ((ldx > 0 ? ldx : K) % 8 || (ldw > 0 ? ldw : K) % 8)) return true;
  return 2 * N * K <= (M <= 4 ? 1ll << 22 : 1ll << 21);
}

// ---- workspace ------------------------------------------------------------------------
// The status word and its padding; then the copies of bf16 operands off 16-byte
// boundaries, or fp32 operands' planes, and the partial products.  fp32 products that
// take the CUDA cores: the product's own workspace, whose status word is the
// call's, and the sums.
constexpr size_t kCtrl = 256;
size_t up256(size_t n) { return (n + 255) / 256 * 256; }

size_t linear_bytes(int64_t M, int64_t N, int64_t K) {
  size_t b = 0;
  return ppo_linear_workspace_bytes(PPO_DTYPE_F32, M, N, K, 0, 0, 0, &b) == PPO_OK ? up256(b) : 0;
}
size_t forward_bytes(int32_t dtype, int64_t M, int64_t N, int64_t K, int64_t ldx, int64_t ldw) {
  if (dtype == PPO_DTYPE_F32 && takes_few<float>(M, N, K, ldx, ldw)) return kCtrl;
  if (dtype == PPO_DTYPE_F32)
    return lin::takes_planes(lin::kForward, M, 2 * N, K)
               ? kCtrl + lin::planes_need(M, K, 2 * N, K, M, 2 * N, K)
               : linear_bytes(M, 2 * N, K) + (size_t)M * 2 * N * 4;
  if (takes_few<__nv_bfloat16>(M, N, K, ldx, ldw)) return kCtrl;
  return kCtrl + lin::packed_bytes(M, K, ldx) + lin::packed_bytes(2 * N, K, ldw) +
         (skinny_ctas(M, N, K) || fused_pairs(false, M, N, K) ? 0 : lin::tc_part_bytes(M, 2 * N, K, true));
}
size_t backward_bytes(int32_t dtype, int64_t M, int64_t N, int64_t J, int64_t lddz, int64_t ldw2) {
  if (dtype == PPO_DTYPE_F32)
    return lin::takes_planes(lin::kData, M, J, N) ? kCtrl + lin::planes_need(M, J, J, N, M, N, J)
                                                  : linear_bytes(M, J, N) + (size_t)M * N * 4;
  return kCtrl + lin::packed_bytes(M, J, lddz) + lin::packed_bytes(J, N, ldw2) +
         (fused_pairs(true, M, N, J) ? 0 : lin::tc_part_bytes(M, N, J, true));
}
bool gated_sizes_ok(int64_t M, int64_t N, int64_t K) {
  return N >= 1 && N < (1ll << 28) && lin::sizes_ok(M, 2 * N, K);
}

// The bf16 product's sums, taken out of the tensor cores as partial products.
cudaError_t tc_sums(const lin::Product& p, int mode, Gate& g, char* work, int* err, cudaStream_t st) {
  const lin::TcPlan plan = lin::tc_plan(p.I, p.J, p.R, true);
  lin::Epilogue e{};
  e.mode = mode;
  e.act = PPO_ACT_NONE;
  const int64_t ldp = lin::part_pitch(p.J);
  g.s = lin::PartialSums{reinterpret_cast<float*>(work), plan.splits, p.I * ldp, ldp, 0};
  return lin::tc_product(p, e, plan, reinterpret_cast<float*>(work), nullptr, err, num_sms(), st);
}

}  // namespace
}  // namespace glin
}  // namespace ppo

using namespace ppo;
using ops::al16;
using ops::extent_ok;
using ops::status_of;

namespace {

ppo_status checked(std::initializer_list<const void*> ptrs, const void* work, size_t work_bytes, size_t need) {
  for (const void* p : ptrs)
    if (!al16(p)) return PPO_ERR_ALIGN;
  if (!work || work_bytes < need) return PPO_ERR_INVALID;
  if (!al16(work)) return PPO_ERR_ALIGN;
  return ops::num_sms() > 0 ? PPO_OK : PPO_ERR_CUDA;
}

}  // namespace

extern "C" {

ppo_status ppo_gated_linear_workspace_bytes(int32_t dtype, int64_t M, int64_t N, int64_t K, int64_t J,
                                            int64_t ldx, int64_t ldw, int64_t lddz, int64_t ldw2,
                                            size_t* bytes) {
  if (!bytes || !ops::dtype_ok(dtype) || !glin::gated_sizes_ok(M, N, K) || J < 0 ||
      (J > 0 && !glin::gated_sizes_ok(M, N, J)))
    return PPO_ERR_INVALID;
  *bytes = std::max(glin::forward_bytes(dtype, M, N, K, ldx, ldw),
                    J > 0 ? glin::backward_bytes(dtype, M, N, J, lddz, ldw2) : (size_t)0);
  return PPO_OK;
}

ppo_status ppo_gated_linear_forward(int32_t dtype, const void* x, int64_t ldx, const void* w, int64_t ldw,
                                    const float* bias, int32_t act, int64_t M, int64_t N, int64_t K, void* y,
                                    int64_t ldy, void* pre, int64_t ldpre, void* work, size_t work_bytes,
                                    cudaStream_t st) {
  if (!x || !w || !y || !ops::act_ok(act) || !ops::dtype_ok(dtype) || !glin::gated_sizes_ok(M, N, K) ||
      !extent_ok(M, ldx, K) || !extent_ok(2 * N, ldw, K) || !extent_ok(M, ldy, N) ||
      (pre && !extent_ok(M, ldpre, 2 * N)))
    return PPO_ERR_INVALID;
  const ppo_status s = checked({x, w, bias, y, pre}, work, work_bytes,
                               glin::forward_bytes(dtype, M, N, K, ldx, ldw));
  if (s != PPO_OK) return s;
  glin::Gate g{};
  g.act = act;
  g.y = y;
  g.ldy = ldy;
  g.M = M;
  g.N = N;
  const lin::Product given{x, ldx, 1, w, ldw, 1, M, 2 * N, K};
  char* free = static_cast<char*>(work) + glin::kCtrl;
  if (dtype == PPO_DTYPE_F32 ? glin::takes_few<float>(M, N, K, ldx, ldw)
                             : glin::takes_few<__nv_bfloat16>(M, N, K, ldx, ldw)) {
    g.bias = bias;
    g.pre = pre;
    g.ldpre = ldpre;
    return status_of(dtype == PPO_DTYPE_F32 ? glin::few<float>(given, g, st) : glin::few<__nv_bfloat16>(given, g, st));
  }
  if (dtype == PPO_DTYPE_F32 && !lin::takes_planes(lin::kForward, M, 2 * N, K)) {
    // the sums go where pre does; without it, to the workspace
    const size_t own = glin::linear_bytes(M, 2 * N, K);
    float* sums = pre ? static_cast<float*>(pre) : reinterpret_cast<float*>(static_cast<char*>(work) + own);
    const int64_t ldp = pre ? ldpre : 2 * N;
    g.s = lin::PartialSums{sums, 1, 0, ldp, 0};
    const ppo_status e = ppo_linear_forward(dtype, x, ldx, w, ldw, bias, PPO_ACT_NONE, nullptr, 0, M, 2 * N, K,
                                            sums, ldp, nullptr, 0, work, own, st);
    return e != PPO_OK ? e : status_of(glin::finish(glin::gate_forward_kernel<float, false>, g, given, st));
  }
  g.bias = bias;
  g.pre = pre;
  g.ldpre = ldpre;
  if (dtype == PPO_DTYPE_F32) {
    const cudaError_t e = lin::planes_sums(given, lin::kForward, free, static_cast<int*>(work), st, &g.s);
    return status_of(e == cudaSuccess ? glin::finish(glin::gate_forward_kernel<float, true>, g, given, st) : e);
  }
  const lin::Copy ca = lin::on_16_bytes(x, ldx, M, K, free), cb = lin::on_16_bytes(w, ldw, 2 * N, K, free);
  cudaError_t err = lin::pack(ca, cb, st);
  if (err != cudaSuccess) return status_of(err);
  const lin::Product m{x, ldx, 1, w, ldw, 1, M, 2 * N, K};
  if (const int ctas = glin::skinny_ctas(M, N, K))
    return status_of(glin::skinny_forward(m, g, ctas, static_cast<int*>(work), st));
  if (const int pairs = glin::fused_pairs(false, M, N, K))
    return status_of(glin::fused_forward(m, g, pairs, static_cast<int*>(work), ops::num_sms(), st));
  err = glin::tc_sums(m, lin::kForward, g, free, static_cast<int*>(work), st);
  if (err == cudaSuccess) err = glin::finish(glin::gate_forward_kernel<__nv_bfloat16, false>, g, m, st);
  return status_of(err);
}

ppo_status ppo_gated_linear_backward_data(int32_t dtype, const void* dz, int64_t lddz, const void* w2,
                                          int64_t ldw2, const void* pre, int64_t ldpre, int32_t act,
                                          int64_t M, int64_t N, int64_t J, void* dp, int64_t lddp, void* y,
                                          int64_t ldy, void* work, size_t work_bytes, cudaStream_t st) {
  if (!dz || !w2 || !pre || !dp || !ops::act_ok(act) || !ops::dtype_ok(dtype) ||
      !glin::gated_sizes_ok(M, N, J) || !extent_ok(M, lddz, J) || !extent_ok(J, ldw2, N) ||
      !extent_ok(M, ldpre, 2 * N) || !extent_ok(M, lddp, 2 * N) || (y && !extent_ok(M, ldy, N)) ||
      (dp == pre && lddp != ldpre))
    return PPO_ERR_INVALID;
  const ppo_status s = checked({dz, w2, pre, dp, y}, work, work_bytes,
                               glin::backward_bytes(dtype, M, N, J, lddz, ldw2));
  if (s != PPO_OK) return s;
  glin::Gate g{};
  g.act = act;
  g.pre_in = pre;
  g.ldin = ldpre;
  g.dp = dp;
  g.lddp = lddp;
  g.y = y;
  g.ldy = ldy;
  g.M = M;
  g.N = N;
  const lin::Product given{dz, lddz, 1, w2, 1, ldw2, M, N, J};
  char* free = static_cast<char*>(work) + glin::kCtrl;
  if (dtype == PPO_DTYPE_F32 && !lin::takes_planes(lin::kData, M, J, N)) {
    const size_t own = glin::linear_bytes(M, J, N);
    float* sums = reinterpret_cast<float*>(static_cast<char*>(work) + own);
    g.s = lin::PartialSums{sums, 1, 0, N, 0};
    const ppo_status e = ppo_linear_backward_data(dtype, dz, lddz, w2, ldw2, nullptr, 0, PPO_ACT_NONE, nullptr,
                                                  0, M, J, N, sums, N, work, own, st);
    return e != PPO_OK ? e : status_of(glin::finish(glin::gate_backward_kernel<float, false>, g, given, st));
  }
  if (dtype == PPO_DTYPE_F32) {
    const cudaError_t e = lin::planes_sums(given, lin::kData, free, static_cast<int*>(work), st, &g.s);
    return status_of(e == cudaSuccess ? glin::finish(glin::gate_backward_kernel<float, true>, g, given, st) : e);
  }
  const lin::Copy ca = lin::on_16_bytes(dz, lddz, M, J, free), cb = lin::on_16_bytes(w2, ldw2, J, N, free);
  cudaError_t err = lin::pack(ca, cb, st);
  if (err != cudaSuccess) return status_of(err);
  const lin::Product m{dz, lddz, 1, w2, 1, ldw2, M, N, J};
  if (const int pairs = glin::fused_pairs(true, M, N, J))
    return status_of(glin::fused_backward(m, g, pairs, static_cast<int*>(work), ops::num_sms(), st));
  err = glin::tc_sums(m, lin::kData, g, free, static_cast<int*>(work), st);
  if (err == cudaSuccess) err = glin::finish(glin::gate_backward_kernel<__nv_bfloat16, false>, g, m, st);
  return status_of(err);
}

}  // extern "C"
