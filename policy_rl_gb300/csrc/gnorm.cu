// gnorm.cu -- the 2-norm over many tensors, and the tensors scaled by
// min(1, max_norm / (norm + 1e-6)).
//
// The table of tensors travels in the kernel's arguments, so that a call needs no
// copy to the device and can be captured.  A tensor is cut into chunks; the blocks
// walk over all chunks of the table by the grid's stride.  Squares are summed in
// fp32 by piece and in 64 bits across pieces; pieces whose squares would
// overflow or lose digits are summed scaled by a power of two (the three ranges
// of Blue 1978, "A portable Fortran program to find the Euclidean norm of a
// vector").  Every block leaves one partial sum, and the scaling kernel adds them
// in a fixed order, so results do not depend on timing.
#include <algorithm>
#include <vector>

#include "ops.cuh"

namespace ppo {
namespace {

using namespace ops;

constexpr int kThreads = 256;
constexpr int kChunk = 4096;           // elements of a chunk
constexpr int kTable = 640;            // tensors of a launch (its arguments: 25 KB)
constexpr int kMaxBlocks = 1216;

struct Entry {
  const void* in;
  void* out;
  int64_t count;
  int64_t first;                       // chunks before this tensor << 1 | bf16
};
struct Table {
  int n;
  int64_t chunks;
  Entry e[kTable];
};

// Sum of squares of a chunk's pieces, in 64 bits whatever its size.
__device__ __forceinline__ double squares(const float (&f)[8]) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) s = fmaf(f[i], f[i], s);
  // below 2^-100 squares lose digits, above 2^120 a sum may overflow: once more, scaled
  if (s < 0x1p120f && (s > 0x1p-100f || s == 0.f)) {
    if (s != 0.f) return (double)s;
  }
  const float k = s > 1.f ? 0x1p-80f : 0x1p80f;
  float v = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) v = fmaf(f[i] * k, f[i] * k, v);
  if (s != s) return (double)s;
  return (double)v * (s > 1.f ? 0x1p160 : 0x1p-160);
}

__device__ __forceinline__ int find(const Table& t, int64_t chunk) {
  int lo = 0, hi = t.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if ((t.e[mid].first >> 1) <= chunk) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

template <typename T>
__device__ __forceinline__ double chunk_squares(const Entry& e, int64_t at, int n) {
  const T* p = static_cast<const T*>(e.in) + at;
  double sum = 0.0;
  for (int i = threadIdx.x; i < n; i += 8 * kThreads) {
    float f[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = i + k * kThreads < n ? (float)p[i + k * kThreads] : 0.f;
    sum += squares(f);
  }
  return sum;
}

__global__ void __launch_bounds__(kThreads)
sumsq_kernel(const __grid_constant__ Table t, double* __restrict__ part) {
  __shared__ double ws[kThreads / kWarp];
  pdl_wait();
  double s = 0.0;
  for (int64_t c = blockIdx.x; c < t.chunks; c += gridDim.x) {
    const Entry& e = t.e[find(t, c)];
    const int64_t at = (c - (e.first >> 1)) * kChunk;
    const int n = (int)min((int64_t)kChunk, e.count - at);
    s += e.first & 1 ? chunk_squares<__nv_bfloat16>(e, at, n) : chunk_squares<float>(e, at, n);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (threadIdx.x % kWarp == 0) ws[threadIdx.x / kWarp] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    double v = 0.0;
    for (int w = 0; w < kThreads / kWarp; ++w) v += ws[w];
    part[blockIdx.x] = v;
  }
}

// The norm from all partial sums, the same in every block.
__device__ __forceinline__ float norm_of(const double* part, int parts) {
  __shared__ double ws[kThreads / kWarp];
  double s = 0.0;
  for (int i = threadIdx.x; i < parts; i += kThreads) s += part[i];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (threadIdx.x % kWarp == 0) ws[threadIdx.x / kWarp] = s;
  __syncthreads();
  s = 0.0;
  for (int w = 0; w < kThreads / kWarp; ++w) s += ws[w];
  __syncthreads();
  return (float)sqrt(s);
}

__global__ void __launch_bounds__(kThreads)
norm_kernel(const double* __restrict__ part, int parts, float* __restrict__ norm) {
  pdl_wait();
  const float v = norm_of(part, parts);
  if (threadIdx.x == 0) *norm = v;
}

template <typename T>
__device__ __forceinline__ void chunk_scale(const Entry& e, int64_t at, int n, float f) {
  const T* p = static_cast<const T*>(e.in) + at;
  T* o = static_cast<T*>(e.out) + at;
  for (int i = threadIdx.x; i < n; i += kThreads) round_to((float)p[i] * f, o[i]);
}

__global__ void __launch_bounds__(kThreads)
scale_kernel(const __grid_constant__ Table t, const double* __restrict__ part, int parts, float max_norm,
             int in_place, float* __restrict__ norm) {
  pdl_wait();
  const float v = norm_of(part, parts);
  if (blockIdx.x == 0 && threadIdx.x == 0 && norm) *norm = v;
  const float q = max_norm / (v + 1e-6f);
  const float f = max_norm > 0.f && !(q >= 1.f) ? q : 1.f;
  if (in_place && f == 1.f) return;
  for (int64_t c = blockIdx.x; c < t.chunks; c += gridDim.x) {
    const Entry& e = t.e[find(t, c)];
    const int64_t at = (c - (e.first >> 1)) * kChunk;
    const int n = (int)min((int64_t)kChunk, e.count - at);
    if (e.first & 1) chunk_scale<__nv_bfloat16>(e, at, n, f);
    else chunk_scale<float>(e, at, n, f);
  }
}

// Tables of at most kTable tensors that hold something, one after another.
template <typename F>
cudaError_t each_table(const ppo_tensor* in, const ppo_tensor* out, int64_t n, F launch) {
  Table t;
  t.n = 0;
  t.chunks = 0;
  for (int64_t k = 0; k < n; ++k) {
    if (in[k].count == 0) continue;
    if (t.n == kTable) {
      const cudaError_t e = launch(t);
      if (e != cudaSuccess) return e;
      t.n = 0;
      t.chunks = 0;
    }
    t.e[t.n++] = Entry{in[k].d_data, out ? out[k].d_data : in[k].d_data, in[k].count,
                       t.chunks << 1 | (in[k].dtype == PPO_DTYPE_BF16)};
    t.chunks += (in[k].count + kChunk - 1) / kChunk;
  }
  return t.n ? launch(t) : cudaSuccess;
}
int blocks_of(const Table& t) { return (int)std::min<int64_t>(t.chunks, kMaxBlocks); }

// Partial sums of all tensors; how many there are.
cudaError_t sum_squares(const ppo_tensor* in, int64_t n, double* part, int* parts, cudaStream_t st) {
  *parts = 0;
  return each_table(in, nullptr, n, [&](const Table& t) {
    const int blocks = blocks_of(t);
    double* p = part + *parts;
    *parts += blocks;
    return launch_pdl(sumsq_kernel, dim3((unsigned)blocks), dim3(kThreads), 0, st, t, p);
  });
}

ppo_status tensors_ok(const ppo_tensor* t, int64_t n) {
  for (int64_t k = 0; k < n; ++k) {
    if (t[k].count < 0 || t[k].count > (1ll << 48) || !dtype_ok(t[k].dtype) || t[k].reserved != 0 ||
        (t[k].count > 0 && !t[k].d_data))
      return PPO_ERR_INVALID;
    if (reinterpret_cast<uintptr_t>(t[k].d_data) % esize(t[k].dtype)) return PPO_ERR_ALIGN;
  }
  return PPO_OK;
}
// Whether the written tensors overlap one another, or an input other than their own.
struct Range {
  uintptr_t from, to;
};
bool overlaps(const ppo_tensor* in, const ppo_tensor* out, int64_t n) {
  const ppo_tensor* w = out ? out : in;
  std::vector<Range> r;
  r.reserve((size_t)n);
  auto range = [](const ppo_tensor& t) {
    const uintptr_t p = reinterpret_cast<uintptr_t>(t.d_data);
    return Range{p, p + (uintptr_t)t.count * esize(t.dtype)};
  };
  bool sorted = true;
  for (int64_t k = 0; k < n; ++k)
    if (w[k].count > 0) {
      r.push_back(range(w[k]));
      if (r.size() > 1 && r[r.size() - 2].from > r.back().from) sorted = false;
    }
  if (!sorted) std::sort(r.begin(), r.end(), [](const Range& a, const Range& b) { return a.from < b.from; });
  for (size_t k = 1; k < r.size(); ++k)
    if (r[k].from < r[k - 1].to) return true;
  if (!out) return false;
  for (int64_t k = 0; k < n; ++k) {
    if (in[k].count == 0) continue;
    const Range a = range(in[k]);
    // the first written range that ends behind a's start
    auto it = std::lower_bound(r.begin(), r.end(), a.from,
                               [](const Range& x, uintptr_t v) { return x.to <= v; });
    for (; it != r.end() && it->from < a.to; ++it)
      if (it->from != a.from || out[k].d_data != in[k].d_data) return true;
  }
  return false;
}

size_t norm_bytes(int64_t n) { return (size_t)((n + kTable - 1) / kTable) * kMaxBlocks * sizeof(double); }

ppo_status call_ok(const ppo_tensor* in, int64_t n, const void* work, size_t work_bytes) {
  if (n < 0 || n >= (1ll << 20) || (n > 0 && !in)) return PPO_ERR_INVALID;
  const ppo_status s = tensors_ok(in, n);
  if (s != PPO_OK) return s;
  if (!work || work_bytes < norm_bytes(n < 1 ? 1 : n)) return PPO_ERR_INVALID;
  if (!al16(work)) return PPO_ERR_ALIGN;
  return PPO_OK;
}

}  // namespace
}  // namespace ppo

using namespace ppo;

extern "C" {

ppo_status ppo_grad_norm_workspace_bytes(int64_t n, size_t* bytes) {
  if (!bytes || n < 0 || n >= (1ll << 20)) return PPO_ERR_INVALID;
  *bytes = norm_bytes(n < 1 ? 1 : n);
  return PPO_OK;
}

ppo_status ppo_grad_norm(const ppo_tensor* tensors, int64_t n, float* norm, void* work, size_t work_bytes,
                         cudaStream_t st) {
  if (!norm) return PPO_ERR_INVALID;
  const ppo_status s = call_ok(tensors, n, work, work_bytes);
  if (s != PPO_OK) return s;
  if (reinterpret_cast<uintptr_t>(norm) % 4) return PPO_ERR_ALIGN;
  if (ops::num_sms() == 0) return PPO_ERR_CUDA;
  double* part = static_cast<double*>(work);
  int parts = 0;
  cudaError_t e = sum_squares(tensors, n, part, &parts, st);
  if (e == cudaSuccess)
    e = launch_pdl(norm_kernel, dim3(1), dim3(kThreads), 0, st, (const double*)part, parts, norm);
  return ops::status_of(e);
}

ppo_status ppo_clip_grad_norm(const ppo_tensor* tensors, const ppo_tensor* out, int64_t n, float max_norm,
                              float* norm, void* work, size_t work_bytes, cudaStream_t st) {
  if (!norm || max_norm != max_norm) return PPO_ERR_INVALID;
  ppo_status s = call_ok(tensors, n, work, work_bytes);
  if (s == PPO_OK && out) s = tensors_ok(out, n);
  if (s != PPO_OK) return s;
  if (reinterpret_cast<uintptr_t>(norm) % 4) return PPO_ERR_ALIGN;
  if (out)
    for (int64_t k = 0; k < n; ++k)
      if (out[k].count != tensors[k].count || out[k].dtype != tensors[k].dtype) return PPO_ERR_INVALID;
  if (overlaps(tensors, out, n)) return PPO_ERR_INVALID;
  if (ops::num_sms() == 0) return PPO_ERR_CUDA;
  double* part = static_cast<double*>(work);
  int parts = 0;
  cudaError_t e = sum_squares(tensors, n, part, &parts, st);
  bool first = true;
  if (e == cudaSuccess)
    e = each_table(tensors, out, n, [&](const Table& t) {
      float* at = first ? norm : nullptr;
      first = false;
      return launch_pdl(scale_kernel, dim3((unsigned)blocks_of(t)), dim3(kThreads), 0, st, t,
                        (const double*)part, parts, max_norm, out ? 0 : 1, at);
    });
  if (e == cudaSuccess && first)       // nothing to scale
    e = launch_pdl(norm_kernel, dim3(1), dim3(kThreads), 0, st, (const double*)part, parts, norm);
  return ops::status_of(e);
}

}  // extern "C"
