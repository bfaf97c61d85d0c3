// glinear.cu -- gated linear layers: two projections of the same rows, the gate
// through its activation, and their product; and the gradient of both from that
// of the layer behind.
//
//   forward    pre = x W^T + b  [M][2N],  y = act(g) u,  g | u the halves of pre
//   backward   d = dz W2  [M][N],  dp = [ d u act'(g) | d act(g) ],  y = act(g) u
//
// The products leave fp32 sums (partial ones where the sum is split), and one
// kernel finishes them: what it writes is rounded once, from fp32.
#include <algorithm>

#include "glinear.h"
#include "ops.cuh"

namespace ppo {
namespace glin {
namespace {

using namespace ops;

constexpr int kThreads = 256;
constexpr int kSms = 152;

template <typename T>
__global__ void __launch_bounds__(kThreads) gate_forward_kernel(const __grid_constant__ Gate g) {
  pdl_wait();
  const int64_t n = g.M * g.N;
  for (int64_t k = (int64_t)blockIdx.x * kThreads + threadIdx.x; k < n; k += (int64_t)gridDim.x * kThreads) {
    const int64_t i = k / g.N, j = k - i * g.N;
    float a = 0.f, u = 0.f;
    for (int s = 0; s < g.splits; ++s) {
      const float* p = g.part + s * g.stride + i * g.ldp + j;
      a += __ldcg(p);
      u += __ldcg(p + g.N);
    }
    if (g.bias) {
      a += g.bias[j];
      u += g.bias[g.N + j];
    }
    if (g.pre) {
      T* o = static_cast<T*>(g.pre) + i * g.ldpre + j;
      round_to(a, o[0]);
      round_to(u, o[g.N]);
    }
    round_to(act_value<false>(g.act, a) * u, static_cast<T*>(g.y)[i * g.ldy + j]);
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) gate_backward_kernel(const __grid_constant__ Gate g) {
  pdl_wait();
  const int64_t n = g.M * g.N;
  for (int64_t k = (int64_t)blockIdx.x * kThreads + threadIdx.x; k < n; k += (int64_t)gridDim.x * kThreads) {
    const int64_t i = k / g.N, j = k - i * g.N;
    float d = 0.f;
    for (int s = 0; s < g.splits; ++s) d += __ldcg(g.part + s * g.stride + i * g.ldp + j);
    const T* p = static_cast<const T*>(g.pre_in) + i * g.ldin + j;
    const float a = (float)p[0], u = (float)p[g.N], v = act_value<false>(g.act, a);
    T* o = static_cast<T*>(g.dp) + i * g.lddp + j;
    round_to(d * u * act_slope<false>(g.act, a), o[0]);
    round_to(d * v, o[g.N]);
    if (g.y) round_to(v * u, static_cast<T*>(g.y)[i * g.ldy + j]);
  }
}

int blocks_for(int64_t n) { return (int)std::min<int64_t>((n + kThreads - 1) / kThreads, 16 * kSms); }
template <typename T>
cudaError_t finish_forward(const Gate& g, cudaStream_t st) {
  return launch_pdl(gate_forward_kernel<T>, dim3((unsigned)blocks_for(g.M * g.N)), dim3(kThreads), 0, st, g);
}
template <typename T>
cudaError_t finish_backward(const Gate& g, cudaStream_t st) {
  return launch_pdl(gate_backward_kernel<T>, dim3((unsigned)blocks_for(g.M * g.N)), dim3(kThreads), 0, st, g);
}

// ---- workspace ------------------------------------------------------------------------
// The status word and its padding, then (bf16) the copies of operands off 16-byte
// boundaries and the partial products, or (fp32) the sums and the product's own
// workspace, whose status word is the call's.
constexpr size_t kCtrl = 256;
size_t up256(size_t n) { return (n + 255) / 256 * 256; }

size_t linear_bytes(int64_t M, int64_t N, int64_t K) {
  size_t b = 0;
  return ppo_linear_workspace_bytes(PPO_DTYPE_F32, M, N, K, 0, 0, 0, &b) == PPO_OK ? up256(b) : 0;
}
size_t forward_bytes(int32_t dtype, int64_t M, int64_t N, int64_t K, int64_t ldx, int64_t ldw) {
  if (dtype == PPO_DTYPE_F32) return linear_bytes(M, 2 * N, K) + (size_t)M * 2 * N * 4;
  return kCtrl + lin::packed_bytes(M, K, ldx) + lin::packed_bytes(2 * N, K, ldw) +
         lin::tc_part_bytes(M, 2 * N, K, true);
}
size_t backward_bytes(int32_t dtype, int64_t M, int64_t N, int64_t J, int64_t lddz, int64_t ldw2) {
  if (dtype == PPO_DTYPE_F32) return linear_bytes(M, J, N) + (size_t)M * N * 4;
  return kCtrl + lin::packed_bytes(M, J, lddz) + lin::packed_bytes(J, N, ldw2) +
         lin::tc_part_bytes(M, N, J, true);
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
  g.part = reinterpret_cast<float*>(work);
  g.splits = plan.splits;
  g.ldp = lin::part_pitch(p.J);
  g.stride = p.I * g.ldp;
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
  if (dtype == PPO_DTYPE_F32) {
    const size_t own = glin::linear_bytes(M, 2 * N, K);
    float* sums = pre ? static_cast<float*>(pre) : reinterpret_cast<float*>(static_cast<char*>(work) + own);
    g.part = sums;
    g.ldp = pre ? ldpre : 2 * N;
    g.splits = 1;
    const ppo_status e = ppo_linear_forward(dtype, x, ldx, w, ldw, bias, PPO_ACT_NONE, nullptr, 0, M, 2 * N, K,
                                            sums, g.ldp, nullptr, 0, work, own, st);
    return e != PPO_OK ? e : status_of(glin::finish_forward<float>(g, st));
  }
  g.bias = bias;
  g.pre = pre;
  g.ldpre = ldpre;
  char* free = static_cast<char*>(work) + glin::kCtrl;
  const lin::Copy ca = lin::on_16_bytes(x, ldx, M, K, free), cb = lin::on_16_bytes(w, ldw, 2 * N, K, free);
  cudaError_t err = lin::pack(ca, cb, st);
  if (err != cudaSuccess) return status_of(err);
  const lin::Product m{x, ldx, 1, w, ldw, 1, M, 2 * N, K};
  if (const int pairs = glin::fused_pairs(false, M, N, K))
    return status_of(glin::fused_forward(m, g, pairs, static_cast<int*>(work), ops::num_sms(), st));
  err = glin::tc_sums(m, lin::kForward, g, free, static_cast<int*>(work), st);
  if (err == cudaSuccess) err = glin::finish_forward<__nv_bfloat16>(g, st);
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
  if (dtype == PPO_DTYPE_F32) {
    const size_t own = glin::linear_bytes(M, J, N);
    float* sums = reinterpret_cast<float*>(static_cast<char*>(work) + own);
    g.part = sums;
    g.ldp = N;
    g.splits = 1;
    const ppo_status e = ppo_linear_backward_data(dtype, dz, lddz, w2, ldw2, nullptr, 0, PPO_ACT_NONE, nullptr,
                                                  0, M, J, N, sums, N, work, own, st);
    return e != PPO_OK ? e : status_of(glin::finish_backward<float>(g, st));
  }
  char* free = static_cast<char*>(work) + glin::kCtrl;
  const lin::Copy ca = lin::on_16_bytes(dz, lddz, M, J, free), cb = lin::on_16_bytes(w2, ldw2, J, N, free);
  cudaError_t err = lin::pack(ca, cb, st);
  if (err != cudaSuccess) return status_of(err);
  const lin::Product m{dz, lddz, 1, w2, 1, ldw2, M, N, J};
  if (const int pairs = glin::fused_pairs(true, M, N, J))
    return status_of(glin::fused_backward(m, g, pairs, static_cast<int*>(work), ops::num_sms(), st));
  err = glin::tc_sums(m, lin::kData, g, free, static_cast<int*>(work), st);
  if (err == cudaSuccess) err = glin::finish_backward<__nv_bfloat16>(g, st);
  return status_of(err);
}

}  // extern "C"
