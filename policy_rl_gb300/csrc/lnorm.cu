// lnorm.cu -- layer norm over the rows of a matrix: forward, and backward with
// the reduction of gamma's and beta's gradients.
//
// Per row of D elements: mean and variance (from the deviations, so that a
// large mean costs no digits), y = (x - mean) rstd gamma + beta; backward
//   q = dy gamma, dx = rstd (q - mean(q) - xh mean(q xh)) + dres,
//   dgamma = sum_rows dy xh, dbeta = sum_rows dy.
// Both are bound by memory: 2 and 3 (4 with dres) row lengths per row.  A row
// is therefore read once and kept in registers (16 or 32 elements a thread)
// between the reductions and the result; a row that fits a warp so belongs to
// 1..32 of its lanes (short rows share a warp), a longer one to a block of up to
// 512 threads.  Every warp (block) walks over many rows and keeps its columns of
// gamma, beta and their gradient sums in registers meanwhile: the parameters are
// read once per warp instead of once per row.  The rows ahead are fetched into
// the thread's own places of a ring in shared memory by 16-byte copies that need
// neither registers nor barriers.
// Rows off 16-byte boundaries (1,397 floats) are read in aligned pieces all the
// same: rows that start equally far from a boundary are dealt to the same block,
// so that a thread's columns, shifted by that distance, stay its own.  Only
// matrices whose pitches disagree go element by element.  Rows that 512 threads
// cannot keep (8,192 elements; 16,384 forward in bf16; 4,096 element by element)
// take the kernels that read the row once per reduction.
// Measured (of the copy rate): 262,144 x 512 bf16 forward 88 us (90 %), backward
// with dres 174 us (91 %); 48,000 x 1,397 fp32 92 us (86 %) and 146 us (81 %).
// Near that the instructions of a row are the other limit (75 and 80 % of the
// issue slots before the arithmetic was packed).
// The parameter gradients leave each block as one partial row; a second kernel
// adds the partial rows in a fixed order, so results do not depend on timing.
#include <algorithm>
#include <type_traits>

#include "ops.cuh"
#include "tc_ptx.cuh"

namespace ppo {
namespace {

using namespace ops;

constexpr int kWarpRowThreads = 256;   // block of the rows-per-warp kernels
constexpr int64_t kTall = 16384;       // rows from which they are many
constexpr int kMaxBlock = 512;
constexpr int kMaxWarps = kMaxBlock / kWarp;
// elements of a row that a thread of a block keeps: what its 128 registers hold
// beside the parameters (32,768 x 4,096 bf16 forward: 120 us with 16, 99 with 32)
__host__ __device__ constexpr int max_kept(int vec, bool backward) {
  return vec == 1 ? 8 : vec == 8 && !backward ? 32 : 16;
}
// a warp keeps twice as many before a row goes to a block and its barriers
// (131,072 x 1,024 bf16: forward 121 us with blocks of two warps, 89 with warps)
__host__ __device__ constexpr int max_kept_warp(int vec) { return vec == 1 ? 8 : 32; }
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
  int classes;                // rows r, r + classes, .. start equally far from a boundary
};

__device__ __forceinline__ float group_sum(float v, int lanes) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (o < lanes) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sum over the row's threads: lanes of a warp, or the block (N values at once).
// Successive sums of a block alternate between two sets of `red`, so that one
// barrier each is enough: a set is written again only after the next sum's.
template <bool BLOCK, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], int lanes, float* red, int& set) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = group_sum(v[i], lanes);
  if constexpr (BLOCK) {
    const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp, nw = blockDim.x / kWarp;
    float* r = red + set * (N * kMaxWarps);
    set ^= 1;
    if (lane == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) r[i * kMaxWarps + warp] = v[i];
    __syncthreads();
    const int from = lane & (kMaxWarps - 1);   // (both halves of the warp)
#pragma unroll
    for (int i = 0; i < N; ++i)
      v[i] = group_sum(from < nw ? r[i * kMaxWarps + from] : 0.f, kMaxWarps);
  }
}

// A piece's elements: in pairs, P of a piece, for the packed fp32 instructions
// (each half rounded as the scalar one would), or one by one.
template <int V, int P>
using Pair = std::conditional_t<P == V, float, float2>;
__device__ __forceinline__ float mul(float a, float b) { return a * b; }
__device__ __forceinline__ float2 mul(float2 a, float2 b) { return ptx::fmul2(a, b); }
__device__ __forceinline__ float fma(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ float2 fma(float2 a, float2 b, float2 c) { return ptx::ffma2(a, b, c); }
__device__ __forceinline__ void set(float& o, float x) { o = x; }
__device__ __forceinline__ void set(float2& o, float x) { o = make_float2(x, x); }
template <typename E>
__device__ __forceinline__ E all(float x) {
  E o;
  set(o, x);
  return o;
}
template <typename E>
__device__ __forceinline__ E add(E a, E b) { return fma(a, all<E>(1.f), b); }
__device__ __forceinline__ float total(float a) { return a; }
__device__ __forceinline__ float total(float2 a) { return a.x + a.y; }
template <int V, int P>
__device__ __forceinline__ void to_pairs(const float (&f)[V], Pair<V, P> (&o)[P]) {
  if constexpr (P == V) {
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = f[i];
  } else {
#pragma unroll
    for (int i = 0; i < P; ++i) o[i] = make_float2(f[2 * i], f[2 * i + 1]);
  }
}
template <int V, int P>
__device__ __forceinline__ void from_pairs(const Pair<V, P> (&p)[P], float (&f)[V]) {
  if constexpr (P == V) {
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = p[i];
  } else {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      f[2 * i] = p[i].x;
      f[2 * i + 1] = p[i].y;
    }
  }
}

// A thread's columns: NV pieces of V, piece j at column at[j] (below 0 where the
// row starts inside it), of which the elements of mask[j] exist.
template <int V, int NV>
struct Columns {
  int at[NV];
  unsigned mask[NV];
  static constexpr unsigned kFull = (1u << V) - 1;
  __device__ __forceinline__ Columns(int rank, int tpr, int shift, int D) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      at[j] = (j * tpr + rank) * V - shift;
      mask[j] = 0;
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (at[j] + i >= 0 && at[j] + i < D) mask[j] |= 1u << i;
    }
  }
};

// Rows on their way: IN matrices, DEEP rows, each thread's pieces at places of
// its own.  (V == 1: elements are loaded when they are needed.)
// (as deep as 512 threads of an SM find room for)
__host__ __device__ constexpr int ring_depth(int inputs, int size) {
  return inputs == 1 ? 5 : inputs * size == 12 ? 2 : 3;
}
template <typename T, int V, int NV, int IN, int THREADS>      // THREADS 0: blockDim.x
struct Ring {
  static constexpr bool kFetch = sizeof(T) * V == 16;
  static constexpr int kDeep = ring_depth(IN, (int)sizeof(T));
  uint4* mine;
  __device__ __forceinline__ int threads() const { return THREADS ? THREADS : (int)blockDim.x; }
  __device__ __forceinline__ uint4* place(int slot, int m, int j) const {
    return mine + ((slot * IN + m) * NV + j) * threads();
  }
  __device__ __forceinline__ void fetch(int slot, int m, const void* base, int64_t ld, int64_t row,
                                        const LnArgs& a, const Columns<V, NV>& c) const {
    const T* p = static_cast<const T*>(base) + row * ld;
    // (a piece may reach into the next rows, but not past the matrix)
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (c.mask[j]) {
        int n = 16;
        if (row + V >= a.M)
          n = (int)min((int64_t)V, (a.M - 1 - row) * ld + a.D - c.at[j]) * (int)sizeof(T);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(ptx::smem_u32(place(slot, m, j))),
                     "l"(p + c.at[j]), "r"(n)
                     : "memory");
      }
  }
  template <int P>
  __device__ __forceinline__ void get(int slot, int m, const void* base, int64_t ld, int64_t row,
                                      const Columns<V, NV>& c, Pair<V, P> (&o)[NV][P]) const {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float f[V];
      if constexpr (kFetch) {
        to_f32<T, V>(*place(slot, m, j), f);
        if (c.mask[j] != c.kFull) {
#pragma unroll
          for (int i = 0; i < V; ++i) f[i] = (c.mask[j] >> i) & 1u ? f[i] : 0.f;
        }
      } else {
        const T* p = static_cast<const T*>(base) + row * ld + c.at[j];
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = (c.mask[j] >> i) & 1u ? (float)p[i] : 0.f;
      }
      to_pairs<V, P>(f, o[j]);
    }
  }
};
template <typename T, int V, int NV, int P>
__device__ __forceinline__ void put_row(void* base, int64_t ld, int64_t row,
                                        const Columns<V, NV>& c, const Pair<V, P> (&q)[NV][P]) {
  T* p = static_cast<T*>(base) + row * ld;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    float f[V];
    from_pairs<V, P>(q[j], f);
    if (c.mask[j] == c.kFull) {
      *reinterpret_cast<Raw<T, V>*>(p + c.at[j]) = from_f32<T, V>(f);
    } else if (c.mask[j]) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if ((c.mask[j] >> i) & 1u) round_to(f[i], p[c.at[j] + i]);
    }
  }
}
__device__ __forceinline__ void ring_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int DEEP>
__device__ __forceinline__ void ring_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(DEEP - 2) : "memory");
}

// blocks of rows-per-warp kernels on an SM, by the elements a thread keeps
__host__ __device__ constexpr int fwd_blocks(int kept) { return kept > 16 ? 2 : 3; }
__host__ __device__ constexpr int bwd_blocks(int kept) { return kept > 16 ? 1 : 2; }

// A thread's walk: rows of its block's class, `step` apart.
struct RowWalk {
  int64_t row, step, rounds;
  int rank, tpr, lanes, shift;
};
template <typename T, int V, bool BLOCK>
__device__ __forceinline__ RowWalk row_walk(const LnArgs& a) {
  RowWalk w;
  w.tpr = BLOCK ? (int)blockDim.x : a.lanes;
  w.rank = BLOCK ? (int)threadIdx.x : (int)(threadIdx.x & (a.lanes - 1));
  w.lanes = BLOCK ? 32 : a.lanes;
  const int rpb = BLOCK ? 1 : kWarpRowThreads / a.lanes;
  const int cls = (int)(blockIdx.x % a.classes), b = (int)(blockIdx.x / a.classes);
  const int nb = (int)(gridDim.x / a.classes);
  w.shift = (int)((int64_t)cls * a.ldx % V);
  const int64_t mine = (a.M - cls + a.classes - 1) / a.classes;   // rows of the class
  const int64_t first = (int64_t)b * rpb;
  w.step = (int64_t)nb * rpb * a.classes;
  // every thread of a block makes the same number of rounds (the sums use whole
  // warps); rows past the end are computed on what the ring holds and not stored
  w.rounds = mine > first ? (mine - first + (int64_t)nb * rpb - 1) / ((int64_t)nb * rpb) : 0;
  w.row = cls + (first + (BLOCK ? 0 : (int)threadIdx.x / a.lanes)) * a.classes;
  return w;
}

// BLOCK: a block per row; else `lanes` lanes per row, kWarpRowThreads / lanes
// rows a block.
template <typename T, int V, int NV, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? kMaxBlock : kWarpRowThreads, BLOCK ? 1 : fwd_blocks(V * NV))
ln_fwd_kernel(const LnArgs a) {
  __shared__ float red[BLOCK ? 2 * kMaxWarps : 1];
  int set = 0;
  extern __shared__ uint4 ring_mem[];
  RowWalk w = row_walk<T, V, BLOCK>(a);
  const Columns<V, NV> c(w.rank, w.tpr, w.shift, a.D);
  using R = Ring<T, V, NV, 1, 0>;
  // packed: 32,768 x 4,096 bf16 93 us, 99 one by one; 48,000 x 1,397 fp32 91 and
  // 95; but bf16 rows of a warp 97 and 89 (262,144 x 512)
  constexpr int P = V > 1 && (BLOCK || sizeof(T) == 4) ? V / 2 : V;
  using E = Pair<V, P>;
  const R ring{ring_mem + threadIdx.x};
  E ga[NV][P], be[NV][P];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    float g[V], b[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const bool in = (c.mask[j] >> i) & 1u;
      g[i] = in && a.gamma ? __ldg(a.gamma + c.at[j] + i) : 1.f;
      b[i] = in && a.beta ? __ldg(a.beta + c.at[j] + i) : 0.f;
    }
    to_pairs<V, P>(g, ga[j]);
    to_pairs<V, P>(b, be[j]);
  }
  const float inv = 1.f / (float)a.D;
  auto fetch = [&](int slot, int64_t row) {
    if constexpr (R::kFetch) {
      if (row < a.M) ring.fetch(slot, 0, a.x, a.ldx, row, a, c);
      ring_commit();
    }
  };
  for (int i = 0; i < R::kDeep - 1; ++i) fetch(i, w.row + i * w.step);
  int slot = 0;
  for (; w.rounds > 0; --w.rounds, w.row += w.step) {
    if constexpr (R::kFetch) ring_wait<R::kDeep>();
    // the slot that was read a round ago takes the farthest row
    fetch(slot == 0 ? R::kDeep - 1 : slot - 1, w.row + (R::kDeep - 1) * w.step);
    E x[NV][P] = {};
    if (w.row < a.M) ring.template get<P>(slot, 0, a.x, a.ldx, w.row, c, x);
    slot = slot == R::kDeep - 1 ? 0 : slot + 1;
    E sum = all<E>(0.f);
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < P; ++i) sum = add<E>(x[j][i], sum);
    float s[1] = {total(sum)};
    row_sum<BLOCK>(s, w.lanes, red, set);
    const float mean = s[0] * inv;
    sum = all<E>(0.f);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
      for (int i = 0; i < P; ++i) x[j][i] = add<E>(x[j][i], all<E>(-mean));
      if (c.mask[j] != c.kFull) {
        float f[V];
        from_pairs<V, P>(x[j], f);
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = (c.mask[j] >> i) & 1u ? f[i] : 0.f;
        to_pairs<V, P>(f, x[j]);
      }
#pragma unroll
      for (int i = 0; i < P; ++i) sum = fma(x[j][i], x[j][i], sum);
    }
    float q[1] = {total(sum)};
    row_sum<BLOCK>(q, w.lanes, red, set);
    // (rsqrtf: 2 units in the last place; 48,000 x 1,397 fp32 is off by 2.5e-7 against 64
    // bits, elementary fp32 operations by 1.8e-7)
    const float rstd = rsqrtf(q[0] * inv + a.eps);
    if (w.row < a.M) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < P; ++i)
          x[j][i] = fma(mul(x[j][i], all<E>(rstd)), ga[j][i], be[j][i]);
      put_row<T, V, NV, P>(a.out, a.ldo, w.row, c, x);
      if (a.stats && w.rank == 0)
        *reinterpret_cast<float2*>(a.stats + 2 * w.row) = make_float2(mean, rstd);
    }
  }
}

template <typename T, int V, int NV, bool BLOCK, bool RES>
__global__ void __launch_bounds__(BLOCK ? kMaxBlock : kWarpRowThreads, BLOCK ? 1 : bwd_blocks(V * NV))
ln_bwd_kernel(const LnArgs a) {
  __shared__ float red[BLOCK ? 4 * kMaxWarps : 1];
  int set = 0;
  extern __shared__ uint4 ring_mem[];
  RowWalk w = row_walk<T, V, BLOCK>(a);
  const Columns<V, NV> c(w.rank, w.tpr, w.shift, a.D);
  using R = Ring<T, V, NV, RES ? 3 : 2, BLOCK ? 0 : kWarpRowThreads>;
  // packed: 262,144 x 512 bf16 173 us, 184 one by one; 48,000 x 1,397 fp32 146 and
  // 147; but bf16 rows of a block 230 and 205 (32,768 x 4,096)
  constexpr int P = V > 1 && (!BLOCK || sizeof(T) == 4) ? V / 2 : V;
  using E = Pair<V, P>;
  const R ring{ring_mem + threadIdx.x};
  E ga[NV][P], dg[NV][P], db[NV][P];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    float g[V];
#pragma unroll
    for (int i = 0; i < V; ++i)
      g[i] = ((c.mask[j] >> i) & 1u) && a.gamma ? __ldg(a.gamma + c.at[j] + i) : 1.f;
    to_pairs<V, P>(g, ga[j]);
#pragma unroll
    for (int i = 0; i < P; ++i) dg[j][i] = db[j][i] = all<E>(0.f);
  }
  const float inv = 1.f / (float)a.D;
  auto stat = [&](int64_t r) {
    return r < a.M ? __ldg(reinterpret_cast<const float2*>(a.stats + 2 * r)) : make_float2(0.f, 0.f);
  };
  auto fetch = [&](int slot, int64_t row) {
    if constexpr (R::kFetch) {
      if (row < a.M) {
        ring.fetch(slot, 0, a.x, a.ldx, row, a, c);
        ring.fetch(slot, 1, a.dy, a.lddy, row, a, c);
        if constexpr (RES) ring.fetch(slot, 2, a.res, a.ldres, row, a, c);
      }
      ring_commit();
    }
  };
  for (int i = 0; i < R::kDeep - 1; ++i) fetch(i, w.row + i * w.step);
  float2 st = stat(w.row), nst;
  int slot = 0;
  for (; w.rounds > 0; --w.rounds, w.row += w.step) {
    nst = stat(w.row + w.step);
    if constexpr (R::kFetch) ring_wait<R::kDeep>();
    fetch(slot == 0 ? R::kDeep - 1 : slot - 1, w.row + (R::kDeep - 1) * w.step);
    E xh[NV][P] = {}, q[NV][P] = {};
    if (w.row < a.M) {
      ring.template get<P>(slot, 0, a.x, a.ldx, w.row, c, xh);
      ring.template get<P>(slot, 1, a.dy, a.lddy, w.row, c, q);
    }
    E s0 = all<E>(0.f), s1 = all<E>(0.f);
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < P; ++i) {
        // (where no element is, q = 0 and xh reaches nothing that is stored)
        xh[j][i] = mul(add<E>(xh[j][i], all<E>(-st.x)), all<E>(st.y));
        dg[j][i] = fma(q[j][i], xh[j][i], dg[j][i]);
        db[j][i] = add<E>(q[j][i], db[j][i]);
        q[j][i] = mul(q[j][i], ga[j][i]);
        s0 = add<E>(q[j][i], s0);
        s1 = fma(q[j][i], xh[j][i], s1);
      }
    float s[2] = {total(s0), total(s1)};
    row_sum<BLOCK>(s, w.lanes, red, set);
    const float m1 = s[0] * inv, m2 = s[1] * inv;
    if (w.row < a.M) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < P; ++i)
          q[j][i] = mul(fma(xh[j][i], all<E>(-m2), add<E>(q[j][i], all<E>(-m1))), all<E>(st.y));
      if constexpr (RES) {
        ring.template get<P>(slot, 2, a.res, a.ldres, w.row, c, xh);
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int i = 0; i < P; ++i) q[j][i] = add<E>(q[j][i], xh[j][i]);
      }
      put_row<T, V, NV, P>(a.out, a.ldo, w.row, c, q);
    }
    slot = slot == R::kDeep - 1 ? 0 : slot + 1;
    st = nst;
  }
  if (!a.part) return;
  float* part = a.part + (int64_t)blockIdx.x * 2 * a.D;
  if constexpr (BLOCK) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float g[V], b[V];
      from_pairs<V, P>(dg[j], g);
      from_pairs<V, P>(db[j], b);
#pragma unroll
      for (int i = 0; i < V; ++i)
        if ((c.mask[j] >> i) & 1u) {
          part[c.at[j] + i] = g[i];
          part[a.D + c.at[j] + i] = b[i];
        }
    }
  } else {
    // the warps' sums meet in the ring's place: [warp][2][D], D <= 1,024
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();
    float* acc = reinterpret_cast<float*>(ring_mem);
    const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float g[V], b[V];
      from_pairs<V, P>(dg[j], g);
      from_pairs<V, P>(db[j], b);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        // lanes that hold the same columns of the warp's rows
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
          if (o >= a.lanes) {
            g[i] += __shfl_xor_sync(0xffffffffu, g[i], o);
            b[i] += __shfl_xor_sync(0xffffffffu, b[i], o);
          }
        if (lane < a.lanes && ((c.mask[j] >> i) & 1u)) {
          acc[(2 * warp) * a.D + c.at[j] + i] = g[i];
          acc[(2 * warp + 1) * a.D + c.at[j] + i] = b[i];
        }
      }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < 2 * a.D; e += kWarpRowThreads) {
      float t = 0.f;
#pragma unroll
      for (int k = 0; k < kWarpRowThreads / kWarp; ++k) t += acc[2 * k * a.D + e];
      part[e] = t;
    }
  }
}

// Rows too long to keep: the row is read once per reduction and once for the
// result; the parameter gradients accumulate in the block's own partial row.
template <typename T>
__global__ void __launch_bounds__(kLongThreads) ln_fwd_long_kernel(const LnArgs a) {
  __shared__ float red[2 * kMaxWarps];
  int set = 0;
  const float inv = 1.f / (float)a.D;
  for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + row * a.ldx;
    T* y = static_cast<T*>(a.out) + row * a.ldo;
    float s[1] = {0.f};
    for (int c = threadIdx.x; c < a.D; c += kLongThreads) s[0] += (float)x[c];
    row_sum<true>(s, 32, red, set);
    const float mean = s[0] * inv;
    float q[1] = {0.f};
    for (int c = threadIdx.x; c < a.D; c += kLongThreads) {
      const float d = (float)x[c] - mean;
      q[0] += d * d;
    }
    row_sum<true>(q, 32, red, set);
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
  __shared__ float red[4 * kMaxWarps];
  int set = 0;
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
    row_sum<true>(s, 32, red, set);
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

// Elements of a piece: 16 bytes where every matrix's rows start equally far from
// a boundary, else one; and how many rows on they do so again.
int vec_of(int32_t dtype, std::initializer_list<int64_t> lds) {
  const int v = 16 / esize(dtype);
  for (int64_t l : lds)
    if (l % v != *lds.begin() % v) return 1;
  return v;
}
int classes_of(int vec, int64_t ld) {
  int c = 1;
  while (c * ld % vec) c *= 2;
  return c;
}

struct Plan {
  int vec, nv, lanes, threads;   // lanes: 0 for a block per row; threads: 0 for the long kernels
  int grid, classes;
  size_t smem;
};

Plan plan_of(int64_t M, int64_t D, int vec, int64_t ld, int sms, bool backward, bool res) {
  Plan p{};
  p.vec = vec;
  p.classes = classes_of(vec, ld);
  if (p.classes > M) p.classes = 1, p.vec = vec = 1;   // too few rows to deal out
  const int64_t span = D + (p.classes > 1 ? vec - 1 : 0);   // shifted columns
  if (span > (int64_t)kMaxBlock * max_kept(vec, backward)) {
    p.classes = 1;
    p.grid = (int)std::min<int64_t>(M, 2 * sms);
    return p;
  }
  int64_t per_sm;
  const int inputs = !backward ? 1 : res ? 3 : 2;
  if (span <= (int64_t)kWarp * max_kept_warp(vec)) {
    // fewest elements a thread with which the row fits a warp, so that a short
    // row keeps its lanes busy
    // (many rows: rather many elements a thread, so that a warp's reductions
    // serve more rows; 262,144 x 512 bf16 forward 99 us with 16 elements, 89 with
    // 32; 1,000,000 x 64 58 us with 8, 48 with 16, 54 with 32)
    p.nv = vec == 1 ? 4 : M < kTall ? 1 : (backward || vec == 4 || span <= 128 ? 16 : 32) / vec;
    while (p.nv * vec * kWarp < span) p.nv *= 2;
    p.lanes = 1;
    while (p.lanes * p.nv * vec < span) p.lanes *= 2;
    p.threads = kWarpRowThreads;
    per_sm = backward ? bwd_blocks(p.nv * vec) : fwd_blocks(p.nv * vec);
  } else {
    p.nv = max_kept(vec, backward) / vec;
    const int64_t per = (int64_t)p.nv * vec;
    p.threads = (int)(((span + per - 1) / per + kWarp - 1) / kWarp) * kWarp;
    per_sm = std::max<int64_t>(1, std::min<int64_t>(8, 512 / p.threads));
  }
  if (vec > 1) p.smem = (size_t)ring_depth(inputs, 16 / vec) * inputs * p.nv * 16 * p.threads;
  if (backward && p.lanes)   // room for the warps' parameter gradients
    p.smem = std::max(p.smem, (size_t)(kWarpRowThreads / kWarp) * 2 * D * sizeof(float));
  const int64_t rpb = p.lanes ? kWarpRowThreads / p.lanes : 1;
  const int64_t rows = (M + p.classes - 1) / p.classes;   // of a class
  const int64_t most = std::min<int64_t>(per_sm * sms, kGridCap) / p.classes;
  p.grid = (int)(std::min((rows + rpb - 1) / rpb, std::max<int64_t>(1, most)) * p.classes);
  return p;
}

// Dynamic shared memory that the plans of a kernel ask for at most: its ring in the
// largest block and, backward with rows per warp, the warps' parameter gradients.
template <typename T, int V, int NV, bool BLOCK, int IN, bool BACK>
constexpr int most_smem() {
  const int ring = V > 1 ? ring_depth(IN, (int)sizeof(T)) * IN * NV * 16 *
                               (BLOCK ? kMaxBlock : kWarpRowThreads)
                         : 0;
  const int sums = BACK && !BLOCK ? kWarpRowThreads / kWarp * 2 * (kWarp * V * NV) * (int)sizeof(float) : 0;
  return std::max(ring, sums);
}
// One launch.  A kernel that may need it is allowed its largest size once per host
// thread and device, whatever this call's size: static shared memory counts
// towards the 48 KB that need no allowance, and a call must not take back what
// another thread's launch relies on.
template <auto KERNEL, int MOST>
cudaError_t launch(const LnArgs& a, const Plan& p, cudaStream_t st) {
  static_assert(MOST + 4 * kMaxWarps * 4 <= 232448, "shared memory per CTA");
  if (p.smem > (size_t)MOST) return cudaErrorInvalidValue;
  if constexpr (MOST > 40 * 1024) {
    static thread_local int prepared = -1;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && prepared != dev)
      e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, MOST);
    if (e != cudaSuccess) return e;
    prepared = dev;
  }
  KERNEL<<<p.grid, p.threads, p.smem, st>>>(a);
  return cudaGetLastError();
}

template <typename T, int V, int NV>
cudaError_t go(const LnArgs& a, const Plan& p, bool backward, cudaStream_t st) {
  if (p.lanes) {
    if (!backward)
      return launch<ln_fwd_kernel<T, V, NV, false>, most_smem<T, V, NV, false, 1, false>()>(a, p, st);
    return a.res ? launch<ln_bwd_kernel<T, V, NV, false, true>, most_smem<T, V, NV, false, 3, true>()>(a, p, st)
                 : launch<ln_bwd_kernel<T, V, NV, false, false>, most_smem<T, V, NV, false, 2, true>()>(a, p, st);
  }
  // (blocks use one count of elements each way)
  if constexpr (V * NV == max_kept(V, false))
    if (!backward)
      return launch<ln_fwd_kernel<T, V, NV, true>, most_smem<T, V, NV, true, 1, false>()>(a, p, st);
  if constexpr (V * NV == max_kept(V, true))
    if (backward)
      return a.res ? launch<ln_bwd_kernel<T, V, NV, true, true>, most_smem<T, V, NV, true, 3, true>()>(a, p, st)
                   : launch<ln_bwd_kernel<T, V, NV, true, false>, most_smem<T, V, NV, true, 2, true>()>(a, p, st);
  return cudaErrorInvalidValue;
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
    if (p.nv == 4) return go<T, V, 4>(a, p, backward, st);
    if constexpr (V == 4)
      if (p.nv == 8) return go<T, V, 8>(a, p, backward, st);
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
  const Plan p = plan_of(M, D, vec_of(dtype, {ldx, ldy}), ldx, sms, false, false);
  a.lanes = p.lanes;
  a.classes = p.classes;
  const cudaError_t e = dtype == PPO_DTYPE_F32 ? dispatch<float>(a, p, false, st)
                                               : dispatch<__nv_bfloat16>(a, p, false, st);
  return ops::status_of(e);
}

ppo_status ppo_layernorm_backward_workspace_bytes(int64_t M, int64_t D, size_t* bytes) {
  if (!bytes || M < 1 || D < 1 || D >= (1ll << 30)) return PPO_ERR_INVALID;
  // one partial row (gamma's and beta's gradient) per block: a row's, rounded up
  // to the at most 8 classes of rows
  *bytes = (size_t)std::min<int64_t>(M + 8, ppo::kGridCap) * 2 * (size_t)D * sizeof(float);
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
  const Plan p = plan_of(M, D, vec_of(dtype, {ldx, lddy, lddx, dres ? lddres : ldx}), ldx, sms,
                         true, dres != nullptr);
  a.lanes = p.lanes;
  a.classes = p.classes;
  cudaError_t e = dtype == PPO_DTYPE_F32 ? dispatch<float>(a, p, true, st)
                                         : dispatch<__nv_bfloat16>(a, p, true, st);
  if (e == cudaSuccess && params)
    e = launch_pdl(ln_param_grad_kernel, dim3((unsigned)((2 * D + kWarp - 1) / kWarp)),
                   dim3(kFinThreads), 0, st, (const float*)a.part, p.grid, (int)D, dgamma, dbeta);
  return ops::status_of(e);
}

}  // extern "C"
