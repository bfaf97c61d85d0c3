// gnorm.cu -- the 2-norm over many tensors, and the tensors scaled by
// min(1, max_norm / (norm + 1e-6)).
//
// The table of tensors travels in the kernel's arguments, so that a call needs no
// copy to the device and can be captured.  A tensor is cut into chunks of aligned 16-byte
// pieces (its first and last may hold elements that are not its own); a block walks over a
// run of the table's chunks, the next chunk's pieces on their way while one is worked on.
// Squares are summed in fp32 over a thread's pieces of a chunk and with compensation (Kahan)
// across them; where they would overflow or lose digits, scaled by a power of two
// (the ranges of Blue 1978, "A portable Fortran program to find the Euclidean norm
// of a vector") and then in 64 bits.  64 bits throughout would be simpler, but a warp's
// FP64 instruction takes 15 clocks of an SM: the reductions of 1,024 threads 10 us.
// Every block leaves one partial sum, and the scaling kernel adds them in a fixed
// order, with compensation too, so results do not depend on timing.  It walks the runs from their other
// ends, so that it finds the last chunks in L2.  Both are bound by memory.
// Measured: 500,000,000 elements in 300 tensors, bf16 and fp32 (1.42 GB), 659 us for norm
// and clip, which move 4.27 GB: 96 % of the copy rate (element by element 1,256, pieces
// without the chunk ahead 713; four blocks an SM spill and take 6 % longer).  100,000
// floats 7.3 us in a graph, 12.7 in one launch of one cluster.  A tensor whose output lies on
// another place of 16 bytes is stored by element: 100,000,000 elements 95 us in bf16 and 189 in
// fp32, 314 and 271 so.
#include <algorithm>
#include <vector>

#include "ops.cuh"

namespace ppo {
namespace {

using namespace ops;

constexpr int kThreads = 256;
constexpr int kPieces = 4;             // pieces of a thread
constexpr int kChunk = kThreads * kPieces * 16;      // bytes
constexpr int kBlocksPerSm = 3, kMaxBlocks = 152 * kBlocksPerSm;
constexpr int kSmallTable = 32, kTable = 640;        // tensors of a launch (its arguments: 1 or 20 KB)

struct Entry {
  const void* in;
  void* out;
  int64_t count;
  int64_t first;                       // chunks before this tensor << 1 | bf16
};
template <int N>
struct Table {
  int n;
  int64_t chunks;
  Entry e[N];
};

template <typename T>
struct Pieces {
  static constexpr int E = 16 / (int)sizeof(T);
};

// Sum of squares of a thread's pieces, up to 32 elements, scaled by k before they are squared.
template <typename T>
__device__ __forceinline__ float piece_sum(const uint4 (&x)[kPieces], float k) {
  constexpr int E = Pieces<T>::E;
  float s[kPieces];
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    float f[E];
    to_f32<T, E>(x[i], f);
    s[i] = 0.f;
#pragma unroll
    for (int j = 0; j < E; ++j) {
      const float v = f[j] * k;
      s[i] = fmaf(v, v, s[i]);
    }
  }
#pragma unroll
  for (int n = kPieces / 2; n > 0; n /= 2)
#pragma unroll
    for (int i = 0; i < n; ++i) s[i] += s[i + n];
  return s[0];
}
// A sum of squares: s in fp32 (compensated by c) of what lies in fp32's middle range, and
// `odd` in 64 bits of what does not.
struct Sum {
  double odd;
  float s, c;
};
__device__ __forceinline__ void add_plain(Sum& a, float v) {
  const float y = v - a.c, t = a.s + y;
  a.c = (t - a.s) - y;
  a.s = t;
}
template <typename T>
__device__ __forceinline__ void add_squares(Sum& a, const uint4 (&x)[kPieces]) {
  const float v = piece_sum<T>(x, 1.f);
  // (what is summed in fp32 stays in its range, however many tensors: 2^60 such sums)
  if (v == 0.f || (v > 0x1p-100f && v < 0x1p64f)) {
    add_plain(a, v);
    if (v != 0.f) return;
    // (0, or too small to be squared)
  }
  // below, squares lose digits; above, their sum may overflow (NaN comes through)
  if (v > 1.f) a.odd += (double)piece_sum<T>(x, 0x1p-80f) * 0x1p160;
  else if (const float w = piece_sum<T>(x, 0x1p80f); w != 0.f) a.odd += (double)w * 0x1p-160;
}
__device__ __forceinline__ bool plain(const Sum& a) { return a.odd == 0.0; }      // (false for NaN)
// The sum of a warp's, in all of its lanes.
__device__ __forceinline__ Sum warp_total(Sum a) {
  if (!__all_sync(0xffffffffu, plain(a))) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a.odd += __shfl_xor_sync(0xffffffffu, a.odd, o);
  }
  a.s = warp_sum(a.s);
  a.c = 0.f;
  return a;
}
// The sum of a block's, in all of its threads.
__device__ __forceinline__ Sum block_total(Sum a) {
  __shared__ Sum ws[kThreads / kWarp];
  a = warp_total(a);
  if (threadIdx.x % kWarp == 0) ws[threadIdx.x / kWarp] = a;
  __syncthreads();
  if (threadIdx.x < kWarp) {
    a = threadIdx.x < kThreads / kWarp ? ws[threadIdx.x] : Sum{0.0, 0.f, 0.f};
    a = warp_total(a);
    __syncwarp();
    if (threadIdx.x == 0) ws[0] = a;
  }
  __syncthreads();
  return ws[0];
}
__device__ __forceinline__ float root(const Sum& a) {
  return plain(a) ? sqrtf(a.s) : (float)sqrt(a.odd + (double)a.s);
}

// A block's walk over its run of chunks, forwards or backwards.
template <int N>
struct Walk {
  const Table<N>& t;
  int64_t c, end;          // the chunk; the one after the last
  int step, i;             // 1 or -1; its tensor
  __device__ __forceinline__ Walk(const Table<N>& table, int dir) : t(table), step(dir) {
    const int64_t c0 = t.chunks * blockIdx.x / gridDim.x, c1 = t.chunks * (blockIdx.x + 1) / gridDim.x;
    c = dir > 0 ? c0 : c1 - 1;
    end = dir > 0 ? c1 : c0 - 1;
    int lo = 0, hi = t.n - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if ((t.e[mid].first >> 1) <= c) lo = mid;
      else hi = mid - 1;
    }
    i = lo;
  }
  __device__ __forceinline__ bool there() const { return c != end; }
  __device__ __forceinline__ void advance() {
    c += step;
    if (step > 0) {
      while (i + 1 < t.n && (t.e[i + 1].first >> 1) <= c) ++i;
    } else {
      while (i > 0 && (t.e[i].first >> 1) > c) --i;
    }
  }
};
// This thread's pieces of a chunk, in bytes: piece k lies at `at` + k kStep; the tensor is
// [from, to).  Bytes of a piece that are not the tensor's count as 0 and are not stored.
constexpr int kStep = kThreads * 16;
struct Place {
  const char *at, *from, *to;
  char* out;               // where `from` goes
  bool bf16;
  __device__ __forceinline__ Place() {}
  template <int N>
  __device__ __forceinline__ explicit Place(const Walk<N>& w) {
    const Entry& e = w.t.e[w.i];
    bf16 = e.first & 1;
    from = static_cast<const char*>(e.in);
    to = from + e.count * (bf16 ? 2 : 4);
    out = static_cast<char*>(e.out);
    at = from - (reinterpret_cast<uintptr_t>(from) & 15) + (w.c - (e.first >> 1)) * kChunk + threadIdx.x * 16;
  }
  __device__ __forceinline__ bool whole(int k) const { return at + k * kStep >= from && at + k * kStep + 16 <= to; }
  __device__ __forceinline__ void load(uint4 (&x)[kPieces]) const {
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
      if (whole(k)) x[k] = *reinterpret_cast<const uint4*>(at + k * kStep);
      else x[k] = load_some(at + k * kStep, from, to);
    }
  }
  // (elements are aligned: two bytes of one are in the tensor together)
  static __device__ __noinline__ uint4 load_some(const char* a, const char* from, const char* to) {
    uint32_t w[4] = {};
    for (int i = 0; i < 8; ++i)
      if (a + 2 * i >= from && a + 2 * i < to)
        w[i / 2] |= (uint32_t)*reinterpret_cast<const uint16_t*>(a + 2 * i) << (16 * (i & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  static __device__ __noinline__ void store_some(char* o, uint4 v, const char* a, const char* from, const char* to,
                                                 int es) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    for (int i = 0; i < 16 / es; ++i) {
      if (a + es * i < from || a + es * i >= to) continue;
      if (es == 4) *reinterpret_cast<uint32_t*>(o + 4 * i) = w[i];
      else *reinterpret_cast<uint16_t*>(o + 2 * i) = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
    }
  }
  template <typename T>
  __device__ __forceinline__ void scale(const uint4 (&x)[kPieces], float f) const {
    constexpr int E = Pieces<T>::E;
    const bool same = ((reinterpret_cast<uintptr_t>(out) ^ reinterpret_cast<uintptr_t>(from)) & 15) == 0;
    char* o = out + (at - from);
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
      float v[E];
      to_f32<T, E>(x[k], v);
#pragma unroll
      for (int i = 0; i < E; ++i) v[i] *= f;
      const uint4 r = from_f32<T, E>(v);
      if (same && whole(k)) __stcs(reinterpret_cast<uint4*>(o + k * kStep), r);
      else store_some(o + k * kStep, r, at + k * kStep, from, to, (int)sizeof(T));
    }
  }
};

__device__ __forceinline__ float factor(float norm, float max_norm) {
  const float q = max_norm / (norm + 1e-6f);
  return max_norm > 0.f && !(q >= 1.f) ? q : 1.f;
}

template <int N>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
sumsq_kernel(const __grid_constant__ Table<N> t, Sum* __restrict__ part) {
  pdl_wait();
  Sum a{};
  Walk<N> w(t, 1);
  uint4 x[kPieces], ahead[kPieces];
  Place here(w), next;
  here.load(x);
  while (w.there()) {
    w.advance();
    if (w.there()) {
      next = Place(w);
      next.load(ahead);
    }
    if (here.bf16) add_squares<__nv_bfloat16>(a, x);
    else add_squares<float>(a, x);
#pragma unroll
    for (int k = 0; k < kPieces; ++k) x[k] = ahead[k];
    here = next;
  }
  a = block_total(a);
  if (threadIdx.x == 0) part[blockIdx.x] = a;
}

// The sum of all partial sums, the same in every block.
__device__ __forceinline__ Sum total_of(const Sum* part, int parts) {
  Sum a{};
  for (int i = threadIdx.x; i < parts; i += kThreads) {
    const Sum b = part[i];
    if (!plain(b)) a.odd += b.odd;
    add_plain(a, b.s);
  }
  return block_total(a);
}
__device__ __forceinline__ float norm_of(const Sum* part, int parts) { return root(total_of(part, parts)); }

// The partial sums of several tables become one, the first: the scaling kernels of all tables
// read no other.
__global__ void __launch_bounds__(kThreads) total_kernel(Sum* part, int parts) {
  pdl_wait();
  const Sum a = total_of(part, parts);      // (all threads have read theirs)
  if (threadIdx.x == 0) part[0] = a;
}

__global__ void __launch_bounds__(kThreads)
norm_kernel(const Sum* __restrict__ part, int parts, float* __restrict__ norm) {
  pdl_wait();
  const float v = norm_of(part, parts);
  if (threadIdx.x == 0) *norm = v;
}

template <int N>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
scale_kernel(const __grid_constant__ Table<N> t, const Sum* __restrict__ part, int parts, float max_norm,
             int in_place, float* __restrict__ norm) {
  pdl_wait();
  const float v = norm_of(part, parts);
  if (blockIdx.x == 0 && threadIdx.x == 0 && norm) *norm = v;
  const float f = factor(v, max_norm);
  if (in_place && f == 1.f) return;
  Walk<N> w(t, -1);
  uint4 x[kPieces], ahead[kPieces];
  Place here(w), next;
  here.load(x);
  while (w.there()) {
    w.advance();
    if (w.there()) {
      next = Place(w);
      next.load(ahead);
    }
    if (here.bf16) here.scale<__nv_bfloat16>(x, f);
    else here.scale<float>(x, f);
#pragma unroll
    for (int k = 0; k < kPieces; ++k) x[k] = ahead[k];
    here = next;
  }
}

int64_t chunks_of(const ppo_tensor& t) {
  const int64_t off = (int64_t)(reinterpret_cast<uintptr_t>(t.d_data) & 15);
  return (off + t.count * esize(t.dtype) + kChunk - 1) / kChunk;
}
template <int N>
void put(Table<N>& t, const ppo_tensor& in, void* out) {
  t.e[t.n++] = Entry{in.d_data, out, in.count, t.chunks << 1 | (in.dtype == PPO_DTYPE_BF16)};
  t.chunks += chunks_of(in);
}
// Tables of at most kTable tensors that hold something, one after another.
template <int N, typename F>
cudaError_t each_table(const ppo_tensor* in, const ppo_tensor* out, int64_t n, F launch) {
  Table<N> t;
  t.n = 0;
  t.chunks = 0;
  for (int64_t k = 0; k < n; ++k) {
    if (in[k].count == 0) continue;
    if (t.n == N) {
      const cudaError_t e = launch(t);
      if (e != cudaSuccess) return e;
      t.n = 0;
      t.chunks = 0;
    }
    put(t, in[k], out ? out[k].d_data : in[k].d_data);
  }
  return t.n ? launch(t) : cudaSuccess;
}
template <int N>
int blocks_of(const Table<N>& t) { return (int)std::min<int64_t>(t.chunks, kMaxBlocks); }

// scale 0: the norm alone
template <int N>
cudaError_t run_table(const ppo_tensor* in, const ppo_tensor* out, int64_t n, int scale, float max_norm, float* norm,
                      Sum* part, cudaStream_t st) {
  const int in_place = out ? 0 : 1;
  int parts = 0;
  cudaError_t e = each_table<N>(in, nullptr, n, [&](const Table<N>& t) {
    const int blocks = blocks_of(t);
    Sum* p = part + parts;
    parts += blocks;
    return launch_pdl(sumsq_kernel<N>, dim3((unsigned)blocks), dim3(kThreads), 0, st, t, p);
  });
  // From three tables on: each block would add up all tables' partial sums (10,000 tensors of 1,000
  // floats, clipped, 421 us, 247 so; 1,300 42.9 and 40.4; but below the limit, with nothing to
  // write, 700 of two tables 14.6 and 15.0)
  if (e == cudaSuccess && scale && parts > 2 * kMaxBlocks) {
    e = launch_pdl(total_kernel, dim3(1), dim3(kThreads), 0, st, part, parts);
    parts = 1;
  }
  bool wanted = true;      // the norm is still to be written
  if (e == cudaSuccess && scale)
    e = each_table<N>(in, out, n, [&](const Table<N>& t) {
      float* at = wanted ? norm : nullptr;
      wanted = false;
      return launch_pdl(scale_kernel<N>, dim3((unsigned)blocks_of(t)), dim3(kThreads), 0, st, t, (const Sum*)part,
                        parts, max_norm, in_place, at);
    });
  if (e == cudaSuccess && wanted)
    e = launch_pdl(norm_kernel, dim3(1), dim3(kThreads), 0, st, (const Sum*)part, parts, norm);
  return e;
}
cudaError_t run_tables(const ppo_tensor* in, const ppo_tensor* out, int64_t n, int scale, float max_norm, float* norm,
                       Sum* part, cudaStream_t st) {
  return n <= kSmallTable ? run_table<kSmallTable>(in, out, n, scale, max_norm, norm, part, st)
                          : run_table<kTable>(in, out, n, scale, max_norm, norm, part, st);
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

size_t norm_bytes(int64_t n) { return (size_t)((n + kTable - 1) / kTable) * kMaxBlocks * sizeof(Sum); }

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
  return ops::status_of(run_tables(tensors, nullptr, n, 0, 0.f, norm, static_cast<Sum*>(work), st));
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
  return ops::status_of(run_tables(tensors, out, n, 1, max_norm, norm, static_cast<Sum*>(work), st));
}

}  // extern "C"
