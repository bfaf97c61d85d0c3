// lnorm.cu -- layer norm over the rows of a matrix: forward, and backward with
// the reduction of gamma's and beta's gradients.
//
// Per row of D elements: mean and variance (from the deviations, so that a
// large mean costs no digits), y = (x - mean) rstd gamma + beta; backward
//   q = dy gamma, dx = rstd (q - mean(q) - xh mean(q xh)) + dres,
//   dgamma = sum_rows dy xh, dbeta = sum_rows dy.
// Both are bound by memory: 2 and 3 (4 with dres) row lengths per row.  A row
// is therefore read once and kept in registers (at most 16 elements a thread, 8
// where rows are not 16-byte aligned) between the reductions and the result; a
// row that fits a warp so belongs to 1..32 of its lanes (short rows share a
// warp), a longer one to a block of up to 512 threads.  Every warp (block) walks over many
// rows with the next row's loads in flight, and keeps its columns of gamma,
// beta and their gradient sums in registers meanwhile: the parameters are read
// once per warp instead of once per row.  Rows beyond 8,192 elements (4,096 unaligned)
// take the kernels that read the row once per reduction.
// The parameter gradients leave each block as one partial row; a second kernel
// adds the partial rows in a fixed order, so results do not depend on timing.
#include <algorithm>

#include "ops.cuh"

namespace ppo {
namespace {

using namespace ops;

constexpr int kWarpRowThreads = 256;   // block of the rows-per-warp kernels
constexpr int kMaxBlock = 512;
// elements of a row that a thread keeps: with the next row's loads in flight,
// twice as many single loads would spill at a block's 128 registers a thread
__host__ __device__ constexpr int max_kept(int vec) { return vec == 1 ? 8 : 16; }
constexpr int kLongThreads = 512;

struct LnArgs {
  const void *x, *dy, *res;
  void* out;                  // y or dx
  int64_t ldx, lddy, ldres, ldo;
  int64_t M;
  int D;
  const float *gamma, *beta;
  float* stats;               // forward: written (nullable); backward: read
  float eps;
  float* part;                // backward: [blocks][2][D] (nullable)
  int lanes;                  // rows-per-warp kernels: lanes of a row (power of two)
};

__device__ __forceinline__ float group_sum(float v, int lanes) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (o < lanes) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sum over the row's threads: lanes of a warp, or the block (N values at once;
// `red` has room for one set per warp and is free again at the next sync).
template <bool BLOCK, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], int lanes, float* red) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = group_sum(v[i], lanes);
  if constexpr (BLOCK) {
    const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp, nw = blockDim.x / kWarp;
    if (lane == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) red[i * 32 + warp] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = group_sum(lane < nw ? red[i * 32 + lane] : 0.f, 32);
    __syncthreads();
  }
}

// What a thread holds of a row: NV vectors of V elements, vector j at column
// (j * threads_of_row + rank) * V.
template <typename T, int V, int NV>
struct RowLoader {
  Raw<T, V> r[NV];
  __device__ __forceinline__ void load(const void* base, int64_t ld, int64_t row, bool ok, int rank,
                                       int tpr, int D) {
    const T* p = static_cast<const T*>(base) + row * ld;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * tpr + rank) * V;
      r[j] = Raw<T, V>{};
      // (plain loads: the result may be written in place)
      if (ok && c < D) r[j] = *reinterpret_cast<const Raw<T, V>*>(p + c);
    }
  }
};

// BLOCK: a block per row; else `lanes` lanes per row, kWarpRowThreads / lanes
// rows a block.  VECTOR loads need D, the pitches and the base aligned to V.
template <typename T, int V, int NV, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? kMaxBlock : kWarpRowThreads)
ln_fwd_kernel(const LnArgs a) {
  __shared__ float red[BLOCK ? 32 : 1];
  const int tpr = BLOCK ? (int)blockDim.x : a.lanes;
  const int rank = BLOCK ? (int)threadIdx.x : (int)(threadIdx.x & (a.lanes - 1));
  const int rpb = BLOCK ? 1 : kWarpRowThreads / a.lanes;
  const int lanes = BLOCK ? 32 : a.lanes;
  const int64_t step = (int64_t)gridDim.x * rpb;
  int64_t row = (int64_t)blockIdx.x * rpb + (BLOCK ? 0 : (int)threadIdx.x / a.lanes);
  float ga[NV][V], be[NV][V];
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (j * tpr + rank) * V + i;
      ga[j][i] = c < a.D && a.gamma ? __ldg(a.gamma + c) : 1.f;
      be[j][i] = c < a.D && a.beta ? __ldg(a.beta + c) : 0.f;
    }
  const float inv = 1.f / (float)a.D;
  RowLoader<T, V, NV> cur, nxt;
  // every thread of a block makes the same number of rounds (the sums use
  // whole warps); rows past the end are computed on zeros and not stored
  int64_t rounds = ((a.M - (int64_t)blockIdx.x * rpb) + step - 1) / step;
  cur.load(a.x, a.ldx, row, row < a.M, rank, tpr, a.D);
  for (; rounds > 0; --rounds, row += step) {
    nxt.load(a.x, a.ldx, row + step, row + step < a.M, rank, tpr, a.D);
    float x[NV][V];
    float s[1] = {0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      to_f32<T, V>(cur.r[j], x[j]);
#pragma unroll
      for (int i = 0; i < V; ++i) s[0] += x[j][i];
    }
    row_sum<BLOCK>(s, lanes, red);
    const float mean = s[0] * inv;
    float q[1] = {0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const bool in = (j * tpr + rank) * V < a.D;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        x[j][i] -= mean;
        q[0] += in ? x[j][i] * x[j][i] : 0.f;
      }
    }
    row_sum<BLOCK>(q, lanes, red);
    const float rstd = rsqrtf(q[0] * inv + a.eps);
    if (row < a.M) {
      T* y = static_cast<T*>(a.out) + row * a.ldo;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = (j * tpr + rank) * V;
        float o[V];
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] = x[j][i] * rstd * ga[j][i] + be[j][i];
        if (c < a.D) *reinterpret_cast<Raw<T, V>*>(y + c) = from_f32<T, V>(o);
      }
      if (a.stats && rank == 0)
        *reinterpret_cast<float2*>(a.stats + 2 * row) = make_float2(mean, rstd);
    }
    cur = nxt;
  }
}

template <typename T, int V, int NV, bool BLOCK, bool RES>
__global__ void __launch_bounds__(BLOCK ? kMaxBlock : kWarpRowThreads)
ln_bwd_kernel(const LnArgs a) {
  __shared__ float red[BLOCK ? 64 : 1];
  // the parameter gradients of a block's warps, 512 columns at most
  __shared__ float acc[BLOCK ? 1 : kWarpRowThreads / kWarp][BLOCK ? 1 : 2][BLOCK ? 1 : 512];
  const int tpr = BLOCK ? (int)blockDim.x : a.lanes;
  const int rank = BLOCK ? (int)threadIdx.x : (int)(threadIdx.x & (a.lanes - 1));
  const int rpb = BLOCK ? 1 : kWarpRowThreads / a.lanes;
  const int lanes = BLOCK ? 32 : a.lanes;
  const int64_t step = (int64_t)gridDim.x * rpb;
  int64_t row = (int64_t)blockIdx.x * rpb + (BLOCK ? 0 : (int)threadIdx.x / a.lanes);
  float ga[NV][V], dg[NV][V], db[NV][V];
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (j * tpr + rank) * V + i;
      ga[j][i] = c < a.D && a.gamma ? __ldg(a.gamma + c) : 1.f;
      dg[j][i] = db[j][i] = 0.f;
    }
  const float inv = 1.f / (float)a.D;
  RowLoader<T, V, NV> cx, cy, cr, nx, ny, nr;
  auto stat = [&](int64_t r) {
    return r < a.M ? __ldg(reinterpret_cast<const float2*>(a.stats + 2 * r)) : make_float2(0.f, 0.f);
  };
  auto fetch = [&](RowLoader<T, V, NV>& x, RowLoader<T, V, NV>& y, RowLoader<T, V, NV>& r,
                   int64_t at) {
    x.load(a.x, a.ldx, at, at < a.M, rank, tpr, a.D);
    y.load(a.dy, a.lddy, at, at < a.M, rank, tpr, a.D);
    if constexpr (RES) r.load(a.res, a.ldres, at, at < a.M, rank, tpr, a.D);
  };
  int64_t rounds = ((a.M - (int64_t)blockIdx.x * rpb) + step - 1) / step;
  fetch(cx, cy, cr, row);
  float2 st = stat(row), nst;
  for (; rounds > 0; --rounds, row += step) {
    fetch(nx, ny, nr, row + step);
    nst = stat(row + step);
    float xh[NV][V], q[NV][V];
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const bool in = (j * tpr + rank) * V < a.D;
      to_f32<T, V>(cx.r[j], xh[j]);
      to_f32<T, V>(cy.r[j], q[j]);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        xh[j][i] = in ? (xh[j][i] - st.x) * st.y : 0.f;
        dg[j][i] += q[j][i] * xh[j][i];
        db[j][i] += q[j][i];
        q[j][i] *= ga[j][i];
        s[0] += q[j][i];
        s[1] += q[j][i] * xh[j][i];
      }
    }
    row_sum<BLOCK>(s, lanes, red);
    const float m1 = s[0] * inv, m2 = s[1] * inv;
    if (row < a.M) {
      T* o = static_cast<T*>(a.out) + row * a.ldo;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = (j * tpr + rank) * V;
        float d[V], rr[V];
        if constexpr (RES) to_f32<T, V>(cr.r[j], rr);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          d[i] = st.y * (q[j][i] - m1 - xh[j][i] * m2);
          if constexpr (RES) d[i] += rr[i];
        }
        if (c < a.D) *reinterpret_cast<Raw<T, V>*>(o + c) = from_f32<T, V>(d);
      }
    }
    cx = nx;
    cy = ny;
    if constexpr (RES) cr = nr;
    st = nst;
  }
  if (!a.part) return;
  float* part = a.part + (int64_t)blockIdx.x * 2 * a.D;
  if constexpr (BLOCK) {
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = (j * tpr + rank) * V + i;
        if (c < a.D) {
          part[c] = dg[j][i];
          part[a.D + c] = db[j][i];
        }
      }
  } else {
    const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        // lanes that hold the same columns of the warp's rows
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
          if (o >= a.lanes) {
            dg[j][i] += __shfl_xor_sync(0xffffffffu, dg[j][i], o);
            db[j][i] += __shfl_xor_sync(0xffffffffu, db[j][i], o);
          }
        const int c = (j * tpr + rank) * V + i;
        if (lane < a.lanes && c < a.D) {
          acc[warp][0][c] = dg[j][i];
          acc[warp][1][c] = db[j][i];
        }
      }
    __syncthreads();
    for (int e = threadIdx.x; e < 2 * a.D; e += kWarpRowThreads) {
      const int k = e >= a.D, c = e - k * a.D;
      float t = 0.f;
#pragma unroll
      for (int w = 0; w < kWarpRowThreads / kWarp; ++w) t += acc[w][k][c];
      part[e] = t;
    }
  }
}

// Rows too long to keep: the row is read once per reduction and once for the
// result; the parameter gradients accumulate in the block's own partial row.
template <typename T>
__global__ void __launch_bounds__(kLongThreads) ln_fwd_long_kernel(const LnArgs a) {
  __shared__ float red[32];
  const float inv = 1.f / (float)a.D;
  for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + row * a.ldx;
    T* y = static_cast<T*>(a.out) + row * a.ldo;
    float s[1] = {0.f};
    for (int c = threadIdx.x; c < a.D; c += kLongThreads) s[0] += (float)x[c];
    row_sum<true>(s, 32, red);
    const float mean = s[0] * inv;
    float q[1] = {0.f};
    for (int c = threadIdx.x; c < a.D; c += kLongThreads) {
      const float d = (float)x[c] - mean;
      q[0] += d * d;
    }
    row_sum<true>(q, 32, red);
    const float rstd = rsqrtf(q[0] * inv + a.eps);
    for (int c = threadIdx.x; c < a.D; c += kLongThreads) {
      const float g = a.gamma ? __ldg(a.gamma + c) : 1.f, b = a.beta ? __ldg(a.beta + c) : 0.f;
      round_to(((float)x[c] - mean) * rstd * g + b, y[c]);
    }
    if (a.stats && threadIdx.x == 0)
      *reinterpret_cast<float2*>(a.stats + 2 * row) = make_float2(mean, rstd);
  }
}

template <typename T>
__global__ void __launch_bounds__(kLongThreads) ln_bwd_long_kernel(const LnArgs a) {
  __shared__ float red[64];
  const float inv = 1.f / (float)a.D;
  float* part = a.part ? a.part + (int64_t)blockIdx.x * 2 * a.D : nullptr;
  for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + row * a.ldx;
    const T* dy = static_cast<const T*>(a.dy) + row * a.lddy;
    const T* res = a.res ? static_cast<const T*>(a.res) + row * a.ldres : nullptr;
    T* o = static_cast<T*>(a.out) + row * a.ldo;
    const float2 st = *reinterpret_cast<const float2*>(a.stats + 2 * row);
    float s[2] = {0.f, 0.f};
    for (int c = threadIdx.x; c < a.D; c += kLongThreads) {
      const float xh = ((float)x[c] - st.x) * st.y, d = (float)dy[c];
      const float q = d * (a.gamma ? __ldg(a.gamma + c) : 1.f);
      s[0] += q;
      s[1] += q * xh;
      if (part) {   // column c of the partial row belongs to this thread alone
        const bool first = row == blockIdx.x;
        part[c] = (first ? 0.f : part[c]) + d * xh;
        part[a.D + c] = (first ? 0.f : part[a.D + c]) + d;
      }
    }
    row_sum<true>(s, 32, red);
    const float m1 = s[0] * inv, m2 = s[1] * inv;
    for (int c = threadIdx.x; c < a.D; c += kLongThreads) {
      const float xh = ((float)x[c] - st.x) * st.y;
      const float q = (float)dy[c] * (a.gamma ? __ldg(a.gamma + c) : 1.f);
      float d = st.y * (q - m1 - xh * m2);
      if (res) d += (float)res[c];
      round_to(d, o[c]);
    }
  }
}

// Sum of the partial rows, column by column in a fixed order: a block takes 32
// columns of the 2 D, its 8 warps every eighth row.
constexpr int kFinThreads = 256;
__global__ void __launch_bounds__(kFinThreads)
ln_param_grad_kernel(const float* __restrict__ part, int nparts, int D, float* __restrict__ dgamma,
                     float* __restrict__ dbeta) {
  __shared__ float s[kFinThreads / kWarp][kWarp];
  pdl_wait();
  const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp;
  const int c = blockIdx.x * kWarp + lane;
  float t = 0.f;
  if (c < 2 * D) {
#pragma unroll 8
    for (int r = warp; r < nparts; r += kFinThreads / kWarp)
      t += __ldcg(part + (int64_t)r * 2 * D + c);
  }
  s[warp][lane] = t;
  __syncthreads();
  if (warp == 0 && c < 2 * D) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kFinThreads / kWarp; ++w) v += s[w][lane];
    if (c < D) {
      if (dgamma) dgamma[c] = v;
    } else if (dbeta) {
      dbeta[c - D] = v;
    }
  }
}

// ---- plan ---------------------------------------------------------------------
constexpr int kGridCap = 1216;   // partial rows at most: 8 blocks on each of 152 SMs

// The widest vector whose alignment the row length and every pitch keep
int vec_of(int32_t dtype, int64_t D, std::initializer_list<int64_t> lds) {
  const int v = 16 / esize(dtype);
  if (D % v) return 1;
  for (int64_t l : lds)
    if (l % v) return 1;
  return v;
}

struct Plan {
  int vec, nv, lanes, threads;   // lanes: 0 for a block per row; threads: 0 for the long kernels
  int grid;
};

Plan plan_of(int64_t M, int64_t D, int vec, int sms, bool backward) {
  Plan p{};
  p.vec = vec;
  if (D > (int64_t)kMaxBlock * max_kept(vec)) {
    p.grid = (int)std::min<int64_t>(M, 2 * sms);
    return p;
  }
  int64_t per_sm;
  if (D <= (int64_t)kWarp * max_kept(vec)) {
    // fewest elements a thread with which the row fits a warp, so that a short
    // row keeps its lanes busy
    p.nv = vec == 1 ? 4 : 1;
    while (p.nv * vec * kWarp < D) p.nv *= 2;
    p.lanes = 1;
    while (p.lanes * p.nv * vec < D) p.lanes *= 2;
    p.threads = kWarpRowThreads;
    per_sm = backward ? 3 : 6;
  } else {
    p.nv = max_kept(vec) / vec;
    const int64_t per = (int64_t)p.nv * vec;
    p.threads = (int)(((D + per - 1) / per + kWarp - 1) / kWarp) * kWarp;
    per_sm = std::max<int64_t>(1, std::min<int64_t>(8, (backward ? 768 : 1536) / p.threads));
  }
  const int64_t rpb = p.lanes ? kWarpRowThreads / p.lanes : 1;
  p.grid = (int)std::min<int64_t>({(M + rpb - 1) / rpb, per_sm * sms, (int64_t)kGridCap});
  return p;
}

template <typename T, int V, int NV>
cudaError_t go(const LnArgs& a, const Plan& p, bool backward, cudaStream_t st) {
  const dim3 g(p.grid), b(p.threads);
  if (p.lanes) {
    if (!backward) ln_fwd_kernel<T, V, NV, false><<<g, b, 0, st>>>(a);
    else if (a.res) ln_bwd_kernel<T, V, NV, false, true><<<g, b, 0, st>>>(a);
    else ln_bwd_kernel<T, V, NV, false, false><<<g, b, 0, st>>>(a);
  } else if constexpr (V * NV == max_kept(V)) {   // (the one count that blocks use)
    if (!backward) ln_fwd_kernel<T, V, NV, true><<<g, b, 0, st>>>(a);
    else if (a.res) ln_bwd_kernel<T, V, NV, true, true><<<g, b, 0, st>>>(a);
    else ln_bwd_kernel<T, V, NV, true, false><<<g, b, 0, st>>>(a);
  } else {
    return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

template <typename T>
cudaError_t dispatch(const LnArgs& a, const Plan& p, bool backward, cudaStream_t st) {
  if (!p.threads) {
    if (backward) ln_bwd_long_kernel<T><<<p.grid, kLongThreads, 0, st>>>(a);
    else ln_fwd_long_kernel<T><<<p.grid, kLongThreads, 0, st>>>(a);
    return cudaGetLastError();
  }
  constexpr int V = 16 / (int)sizeof(T);
  if (p.vec == V) {
    if (p.nv == 1) return go<T, V, 1>(a, p, backward, st);
    if (p.nv == 2) return go<T, V, 2>(a, p, backward, st);
    if constexpr (V == 4)
      if (p.nv == 4) return go<T, V, 4>(a, p, backward, st);
    return cudaErrorInvalidValue;
  }
  if (p.nv == 4) return go<T, 1, 4>(a, p, backward, st);
  if (p.nv == 8) return go<T, 1, 8>(a, p, backward, st);
  return cudaErrorInvalidValue;
}

}  // namespace
}  // namespace ppo

using ppo::ops::al16;

extern "C" {

ppo_status ppo_layernorm_forward(int32_t dtype, const void* x, int64_t ldx, int64_t M, int64_t D,
                                 const float* gamma, const float* beta, float eps, void* y,
                                 int64_t ldy, float* stats, cudaStream_t st) {
  using namespace ppo;
  if (!ops::dtype_ok(dtype) || !x || !y) return PPO_ERR_INVALID;
  if (!ops::extent_ok(M, ldx, D) || !ops::extent_ok(M, ldy, D)) return PPO_ERR_INVALID;
  if (!(eps >= 0.f) || D >= (1ll << 30) || (x == y && ldx != ldy)) return PPO_ERR_INVALID;
  for (const void* p : {(const void*)x, (const void*)y, (const void*)gamma, (const void*)beta,
                        (const void*)stats})
    if (!al16(p)) return PPO_ERR_ALIGN;
  const int sms = ops::num_sms();
  if (sms < 1) return PPO_ERR_CUDA;
  LnArgs a{};
  a.x = x;
  a.out = y;
  a.ldx = ldx;
  a.ldo = ldy;
  a.M = M;
  a.D = (int)D;
  a.gamma = gamma;
  a.beta = beta;
  a.eps = eps;
  a.stats = stats;
  const Plan p = plan_of(M, D, vec_of(dtype, D, {ldx, ldy}), sms, false);
  a.lanes = p.lanes;
  const cudaError_t e = dtype == PPO_DTYPE_F32 ? dispatch<float>(a, p, false, st)
                                               : dispatch<__nv_bfloat16>(a, p, false, st);
  return e == cudaSuccess ? PPO_OK : PPO_ERR_CUDA;
}

ppo_status ppo_layernorm_backward_workspace_bytes(int64_t M, int64_t D, size_t* bytes) {
  if (!bytes || M < 1 || D < 1 || D >= (1ll << 30)) return PPO_ERR_INVALID;
  // one partial row (gamma's and beta's gradient) per block
  *bytes = (size_t)std::min<int64_t>(M, ppo::kGridCap) * 2 * (size_t)D * sizeof(float);
  return PPO_OK;
}

ppo_status ppo_layernorm_backward(int32_t dtype, const void* dy, int64_t lddy, const void* x,
                                  int64_t ldx, int64_t M, int64_t D, const float* gamma,
                                  const float* stats, const void* dres, int64_t lddres, void* dx,
                                  int64_t lddx, float* dgamma, float* dbeta, void* work,
                                  size_t work_bytes, cudaStream_t st) {
  using namespace ppo;
  if (!ops::dtype_ok(dtype) || !dy || !x || !stats || !dx) return PPO_ERR_INVALID;
  if (!ops::extent_ok(M, ldx, D) || !ops::extent_ok(M, lddy, D) || !ops::extent_ok(M, lddx, D) ||
      (dres && !ops::extent_ok(M, lddres, D)) || D >= (1ll << 30))
    return PPO_ERR_INVALID;
  if ((dx == dy && lddx != lddy) || (dx == dres && lddx != lddres)) return PPO_ERR_INVALID;
  const bool params = dgamma || dbeta;
  size_t need = 0;
  if (ppo_layernorm_backward_workspace_bytes(M, D, &need) != PPO_OK) return PPO_ERR_INVALID;
  if (params && (!work || work_bytes < need)) return PPO_ERR_INVALID;
  for (const void* p : {dy, x, (const void*)gamma, (const void*)stats, dres, (const void*)dx,
                        (const void*)dgamma, (const void*)dbeta, (const void*)work})
    if (!al16(p)) return PPO_ERR_ALIGN;
  const int sms = ops::num_sms();
  if (sms < 1) return PPO_ERR_CUDA;
  LnArgs a{};
  a.x = x;
  a.dy = dy;
  a.res = dres;
  a.out = dx;
  a.ldx = ldx;
  a.lddy = lddy;
  a.ldres = lddres;
  a.ldo = lddx;
  a.M = M;
  a.D = (int)D;
  a.gamma = gamma;
  a.stats = const_cast<float*>(stats);
  a.part = params ? static_cast<float*>(work) : nullptr;
  const Plan p =
      plan_of(M, D, vec_of(dtype, D, {ldx, lddy, lddx, dres ? lddres : ldx}), sms, true);
  a.lanes = p.lanes;
  cudaError_t e = dtype == PPO_DTYPE_F32 ? dispatch<float>(a, p, true, st)
                                         : dispatch<__nv_bfloat16>(a, p, true, st);
  if (e == cudaSuccess && params)
    e = launch_pdl(ln_param_grad_kernel, dim3((unsigned)((2 * D + kWarp - 1) / kWarp)),
                   dim3(kFinThreads), 0, st, (const float*)a.part, p.grid, (int)D, dgamma, dbeta);
  return e == cudaSuccess ? PPO_OK : PPO_ERR_CUDA;
}

}  // extern "C"
