// action.cu -- the policy over any number of actions: log-probability and
// entropy of a row of logits, and the clipped policy loss with its gradient.
//
// Of a row's logits l over the allowed actions, with m = max l and d = l - m:
//   s = sum e^d,  t = sum e^d d,   logp_j = d_j - log s,   H = log s - t / s,
// and with c and W the row's slope and weight (row_terms below) the gradient is
//   W (c (1[j = a] - p_j) + ent p_j (logp_j + H))
//     = e^(d_j) (A1 d_j + A0) + 1[j = a] W c,
//   A1 = W ent / s,   A0 = W (ent (H - log s) - c) / s.
#include <algorithm>
#include <math_constants.h>

#include "ops.cuh"

namespace ppo {
namespace {

using namespace ops;

constexpr int kRowThreads = 128;
constexpr int kMaxBlocks = 1216;     // blocks of a call: rows are walked by their stride
constexpr int kTerms = 8;            // sums of d_stats

struct ActionArgs {
  const void* l;
  int64_t ld, M;
  int V;
  const uint8_t* mask;
  int64_t ldm;
  const int32_t* action;
  const float *old, *adv, *ref, *weight;
  float scale, lo, hi, kl, ent;      // lo, hi: the ratio's bounds
  void* dl;
  int64_t lddl;
  float *logp, *entropy;
  double* part;                      // [blocks][kTerms]
};

// A row's statistics: maximum, sum of e^d, sum of e^d d.
struct Stat {
  float m, s, t;
};
// (d = -inf of an action that is not allowed: e^d d is 0 there, not NaN)
__device__ __forceinline__ float held(float d) { return fmaxf(d, -1e30f); }
// maximum that the deviations are taken from: 0 in a row without any
__device__ __forceinline__ float base_of(float m) { return m == -CUDART_INF_F ? 0.f : m; }

// What a row's gradient and sums need beyond its logits.
struct RowTerms {
  float a0, a1, hot;       // gradient: e^d (a1 d + a0), + hot at the action
  bool kept;
};
// x: the logit of the row's action (-inf where it is not allowed); one thread.
// Adds the row's terms to sums where they are wanted.
__device__ __forceinline__ RowTerms row_terms(const ActionArgs& p, int64_t row, const Stat& st, float x,
                                              bool has, double (&sums)[kTerms]) {
  RowTerms r{0.f, 0.f, 0.f, false};
  const float base = base_of(st.m), logs = logf(st.s);
  const float H = st.s == 0.f ? 0.f : logs - st.t / st.s;
  const float lp = has ? (x == -CUDART_INF_F ? x : (x - base) - logs) : 0.f;
  if (p.logp) p.logp[row] = lp;
  if (p.entropy) p.entropy[row] = H;
  if (!p.dl) return r;
  if (!has || lp == -CUDART_INF_F) {
    sums[7] += 1.0;
    return r;
  }
  const float w = p.weight ? p.weight[row] : 1.f;
  if (w == 0.f) return r;
  const float A = p.adv[row], u = lp - p.old[row], ratio = expf(u);
  const float s1 = ratio * A, s2 = fminf(fmaxf(ratio, p.lo), p.hi) * A;
  const float pg = s1 <= s2 ? -s1 : -s2;       // (NaN comes through s2)
  float c = s1 <= s2 ? -s1 : s1 != s1 ? s1 : 0.f, kl = 0.f;
  if (p.ref) {
    const float y = p.ref[row] - lp, em = expm1f(y);
    kl = em - y;
    c -= p.kl * em;
  }
  const float W = p.scale * w;
  const double Wd = (double)p.scale * w;
  sums[0] += Wd * ((double)pg + (double)p.kl * kl - (double)p.ent * H);
  sums[1] += Wd * pg;
  sums[2] += Wd * kl;
  sums[3] += Wd * H;
  sums[4] += ratio < p.lo || ratio > p.hi ? Wd : 0.0;
  sums[5] += Wd * (expm1f(u) - u);
  sums[6] += Wd;
  r.kept = true;
  r.hot = W * c;
  r.a1 = W * p.ent / st.s;
  r.a0 = W * (p.ent * (H - logs) - c) / st.s;
  return r;
}

// ---- a block for a row ---------------------------------------------------------------
__device__ __forceinline__ float block_max(float v, float* s) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  if (threadIdx.x % kWarp == 0) s[threadIdx.x / kWarp] = v;
  __syncthreads();
  v = s[0];
  for (int w = 1; w < kRowThreads / kWarp; ++w) v = fmaxf(v, s[w]);
  __syncthreads();
  return v;
}
__device__ __forceinline__ float block_sum(float v, float* s) {
  v = warp_sum(v);
  if (threadIdx.x % kWarp == 0) s[threadIdx.x / kWarp] = v;
  __syncthreads();
  v = 0.f;
  for (int w = 0; w < kRowThreads / kWarp; ++w) v += s[w];
  __syncthreads();
  return v;
}

template <typename T>
__global__ void __launch_bounds__(kRowThreads) action_rows_kernel(const ActionArgs p) {
  __shared__ float red[kRowThreads / kWarp];
  __shared__ RowTerms terms;
  double sums[kTerms] = {};
  pdl_wait();
  for (int64_t row = blockIdx.x; row < p.M; row += gridDim.x) {
    const T* l = static_cast<const T*>(p.l) + row * p.ld;
    const uint8_t* k = p.mask ? p.mask + row * p.ldm : nullptr;
    auto at = [&](int j) { return k && !k[j] ? -CUDART_INF_F : (float)l[j]; };
    const int a = p.action ? p.action[row] : -1;
    const bool has = a >= 0 && a < p.V;
    Stat st{-CUDART_INF_F, 0.f, 0.f};
    for (int j = threadIdx.x; j < p.V; j += kRowThreads) st.m = fmaxf(st.m, at(j));
    st.m = block_max(st.m, red);
    const float base = base_of(st.m);
    for (int j = threadIdx.x; j < p.V; j += kRowThreads) {
      const float d = at(j) - base, e = __expf(d);
      st.s += e;
      st.t += e * held(d);
    }
    st.s = block_sum(st.s, red);
    st.t = block_sum(st.t, red);
    if (threadIdx.x == 0) terms = row_terms(p, row, st, has ? at(a) : 0.f, has, sums);
    __syncthreads();
    if (p.dl) {
      const RowTerms r = terms;
      T* o = static_cast<T*>(p.dl) + row * p.lddl;
      for (int j = threadIdx.x; j < p.V; j += kRowThreads) {
        const float x = at(j), d = x - base;
        float g = __expf(d) * fmaf(r.a1, held(d), r.a0);
        if (j == a) g += r.hot;
        if (!r.kept || (k && !k[j])) g = 0.f;
        round_to(g, o[j]);
      }
    }
    __syncthreads();
  }
  if (p.part && threadIdx.x == 0) {
    for (int i = 0; i < kTerms; ++i) p.part[(int64_t)blockIdx.x * kTerms + i] = sums[i];
  }
}

// d_stats from the blocks' sums: a warp for each of them, in a fixed order.
__global__ void __launch_bounds__(kTerms * kWarp)
action_stats_kernel(const double* __restrict__ part, int blocks, float* __restrict__ stats) {
  pdl_wait();
  const int i = threadIdx.x / kWarp, lane = threadIdx.x % kWarp;
  double v = 0.0;
  for (int b = lane; b < blocks; b += kWarp) v += part[(int64_t)b * kTerms + i];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (lane == 0) stats[i] = (float)v;
}

template <typename T>
cudaError_t run_rows(const ActionArgs& p, float* stats, cudaStream_t st) {
  const int blocks = (int)std::min<int64_t>(p.M, kMaxBlocks);
  cudaError_t e = launch_pdl(action_rows_kernel<T>, dim3((unsigned)blocks), dim3(kRowThreads), 0, st, p);
  if (e != cudaSuccess || !stats) return e;
  return launch_pdl(action_stats_kernel, dim3(1), dim3(kTerms * kWarp), 0, st, (const double*)p.part, blocks,
                    stats);
}
cudaError_t run_any(int32_t dtype, const ActionArgs& p, float* stats, cudaStream_t st) {
  return dtype == PPO_DTYPE_F32 ? run_rows<float>(p, stats, st) : run_rows<__nv_bfloat16>(p, stats, st);
}

bool on(const void* p, int bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

// Sizes, pitches and alignment of the logits, mask and row vectors.
ppo_status rows_ok(int32_t dtype, const void* l, int64_t ld, int64_t M, int64_t V, const uint8_t* mask,
                   int64_t ldm, std::initializer_list<const void*> rows) {
  if (!l || !dtype_ok(dtype) || !extent_ok(M, ld, V) || (mask && !extent_ok(M, ldm, V)))
    return PPO_ERR_INVALID;
  if (V > PPO_MAX_ACTIONS || M >= (1ll << 31)) return PPO_ERR_UNSUPPORTED;
  if (!on(l, esize(dtype))) return PPO_ERR_ALIGN;
  for (const void* r : rows)
    if (!on(r, 4)) return PPO_ERR_ALIGN;
  return PPO_OK;
}
constexpr size_t kActionWork = (size_t)kMaxBlocks * kTerms * sizeof(double);

}  // namespace
}  // namespace ppo

using namespace ppo;

extern "C" {

ppo_status ppo_action_logp(int32_t dtype, const void* logits, int64_t ld, int64_t M, int64_t V,
                           const uint8_t* mask, int64_t ldm, const int32_t* action, float* logp,
                           float* entropy, cudaStream_t st) {
  if (logp && !action) return PPO_ERR_INVALID;
  const ppo_status s = rows_ok(dtype, logits, ld, M, V, mask, ldm, {action, logp, entropy});
  if (s != PPO_OK) return s;
  if (ops::num_sms() == 0) return PPO_ERR_CUDA;
  if (!logp && !entropy) return PPO_OK;
  ActionArgs p{};
  p.l = logits;
  p.ld = ld;
  p.M = M;
  p.V = (int)V;
  p.mask = mask;
  p.ldm = ldm;
  p.action = action;
  p.logp = logp;
  p.entropy = entropy;
  return ops::status_of(run_any(dtype, p, nullptr, st));
}

ppo_status ppo_action_loss_workspace_bytes(size_t* bytes) {
  if (!bytes) return PPO_ERR_INVALID;
  *bytes = kActionWork;
  return PPO_OK;
}

ppo_status ppo_action_loss_grad(int32_t dtype, const void* logits, int64_t ld, int64_t M, int64_t V,
                                const uint8_t* mask, int64_t ldm, const int32_t* action,
                                const float* logp_old, const float* adv, const float* logp_ref,
                                const float* weight, float scale, float clip_low, float clip_high,
                                float kl_coef, float ent_coef, void* dlogits, int64_t lddl, float* logp,
                                float* entropy, float* stats, void* work, size_t work_bytes,
                                cudaStream_t st) {
  if (!action || !logp_old || !adv || !dlogits) return PPO_ERR_INVALID;
  const ppo_status s = rows_ok(dtype, logits, ld, M, V, mask, ldm,
                               {action, logp_old, adv, logp_ref, weight, logp, entropy, stats});
  if (s != PPO_OK) return s;
  if (!ops::extent_ok(M, lddl, V) || (dlogits == logits && lddl != ld) || !(clip_low >= 0.f) ||
      !(clip_high >= 0.f))
    return PPO_ERR_INVALID;
  if (!on(dlogits, ops::esize(dtype))) return PPO_ERR_ALIGN;
  if (stats && (!work || work_bytes < kActionWork)) return PPO_ERR_INVALID;
  if (stats && !ops::al16(work)) return PPO_ERR_ALIGN;
  if (ops::num_sms() == 0) return PPO_ERR_CUDA;
  ActionArgs p{};
  p.l = logits;
  p.ld = ld;
  p.M = M;
  p.V = (int)V;
  p.mask = mask;
  p.ldm = ldm;
  p.action = action;
  p.old = logp_old;
  p.adv = adv;
  p.ref = logp_ref;
  p.weight = weight;
  p.scale = scale;
  p.lo = 1.f - clip_low;
  p.hi = 1.f + clip_high;
  p.kl = kl_coef;
  p.ent = ent_coef;
  p.dl = dlogits;
  p.lddl = lddl;
  p.logp = logp;
  p.entropy = entropy;
  p.part = stats ? static_cast<double*>(work) : nullptr;
  return ops::status_of(run_any(dtype, p, stats, st));
}

}  // extern "C"
