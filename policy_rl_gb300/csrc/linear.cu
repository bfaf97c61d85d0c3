// linear.cu -- matrix products with bias, activation and residual: entry
// points, the products on the CUDA cores, and what every product shares (the
// epilogue of split products, column sums).
//
//   forward          y  = act(x W^T + b) + res          [M][N], sum over K
//   backward data    dx = (dz W) act'(pre_in) + res     [M][K], sum over N
//   backward weight  dW = dz^T x, db = sum_rows dz      [N][K], sum over M
//
// Each is out(i, j) = sum_r A(i, r) B(j, r) with A and B read through a row
// and a reduction stride; bf16 products run on the tensor cores (linear_tc.cu),
// and so do large fp32 ones, as products of three bf16 planes that together
// hold fp32's digits; smaller fp32 products run here on the CUDA cores, and so
// do forward products of a few rows of either type.  A product with too few
// output tiles for the GPU's SMs is cut along the sum; the partial products are
// added in order by finish_kernel, which then applies the epilogue, so that
// results do not depend on timing.
#include "linear.h"

#include <algorithm>

#include "lin_again.cuh"
#include "ops.cuh"
#include "tc_ptx.cuh"

namespace ppo {
namespace lin {
namespace {

using namespace ops;

// ---- epilogue -------------------------------------------------------------------
// n (<= 4) consecutive elements of a row, in one piece where rows allow it
template <typename T>
__device__ __forceinline__ void get4(const void* p, int64_t at, int n, bool vec, float (&f)[4]) {
  const T* q = static_cast<const T*>(p) + at;
  if (vec && n == 4) {
    to_f32<T, 4>(*reinterpret_cast<const Raw<T, 4>*>(q), f);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = i < n ? (float)q[i] : 0.f;
  }
}
template <typename T>
__device__ __forceinline__ void put4(void* p, int64_t at, int n, bool vec, const float (&f)[4]) {
  T* q = static_cast<T*>(p) + at;
  if (vec && n == 4) {
    *reinterpret_cast<Raw<T, 4>*>(q) = from_f32<T, 4>(f);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) round_to(f[i], q[i]);
  }
}

// What the epilogue of n (<= 4) output elements of row i from column j on reads;
// vec: pieces of four elements are aligned in every matrix.  Read ahead of the
// sums that it is applied to (nothing here comes from the product's kernel).
struct Beside {
  float bias[4], res[4], pre[4], out[4];
};
template <typename T>
__device__ __forceinline__ void beside4(const Epilogue& e, Beside& x, int64_t i, int64_t j, int n,
                                        bool vec) {
  if (e.mode == kWeight) {
    if (e.accumulate) get4<float>(e.out, i * e.ldo + j, n, vec, x.out);
    return;
  }
  if (e.mode == kForward) {
    if (e.bias) get4<float>(e.bias, j, n, j % 4 == 0, x.bias);
  } else if (e.act != PPO_ACT_NONE) {
    get4<T>(e.pre, i * e.ldpre + j, n, vec, x.pre);
  }
  if (e.res) get4<T>(e.res, i * e.ldres + j, n, vec, x.res);
}
// The elements from their finished sums.
template <typename T>
__device__ __forceinline__ void finish4(const Epilogue& e, const Beside& x, float (&v)[4], int64_t i,
                                        int64_t j, int n, bool vec) {
  if (e.mode == kWeight) {
    if (e.accumulate) {
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] += x.out[q];
    }
    put4<float>(e.out, i * e.ldo + j, n, vec, v);
    return;
  }
  if (e.mode == kForward) {
    if (e.bias) {
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] += x.bias[q];
    }
    if (e.pre) put4<T>(e.pre, i * e.ldpre + j, n, vec, v);
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = act_value<false>(e.act, v[q]);
  } else if (e.act != PPO_ACT_NONE) {
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] *= act_slope<false>(e.act, x.pre[q]);
  }
  if (e.res) {
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] += x.res[q];
  }
  put4<T>(e.out, i * e.ldo + j, n, vec, v);
}

// Every eighth row's share of a column sum, from row w on.
__device__ __noinline__ float sum_again(const float* a, int64_t step, int64_t R, int w) {
  constexpr int U = 8, S = 8;
  float v = 0.f;
  int64_t r = w;
  for (; r + (U - 1) * S < R; r += U * S) {
    float x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) x[u] = __ldg(a + (r + u * S) * step);
#pragma unroll
    for (int u = 0; u < U; ++u) v += x[u];
  }
  for (; r < R; r += S) v += __ldg(a + r * step);
  return v;
}

// out = epilogue of the sum of the partial products, in split order, four columns
// a thread; what the epilogue adds is on its way before the wait for the product's
// kernel.  4,999 x 512 fp32 with residual and pre, three parts (61 MB), takes 20 us,
// 45 % of the copy rate: what its threads wait for is their loads.  PLANES: of a product
// of planes.
constexpr int kFinishThreads = 256;
// This thread's pieces, one after another: f(row, column, columns that exist, piece).
template <typename F>
__device__ __forceinline__ void finish_pieces(int64_t I, int64_t J, int64_t ldp, F f) {
  const int64_t per = ldp / 4, n4 = I * per;
  for (int64_t k = (int64_t)blockIdx.x * kFinishThreads + threadIdx.x; k < n4;
       k += (int64_t)gridDim.x * kFinishThreads) {
    // (a 64-bit division costs as much as the rest)
    const int64_t i = n4 < (1ll << 32) ? (int64_t)((uint32_t)k / (uint32_t)per) : k / per;
    const int64_t j = 4 * (k - i * per);
    const int cols = (int)min((int64_t)4, J - j);
    if (cols > 0) f(i, j, cols, k);
  }
}
// piece k of the partial products, summed; 0 in the columns that do not exist, whose
// places hold anything
__device__ __forceinline__ void add_parts(const float* part, int splits, int64_t n, int64_t k, int cols,
                                          float (&v)[4]) {
#pragma unroll 4
  for (int s = 0; s < splits; ++s) {
    const float4 t = __ldcg(reinterpret_cast<const float4*>(part + s * n) + k);
    v[0] += t.x;
    v[1] += t.y;
    v[2] += t.z;
    v[3] += t.w;
  }
#pragma unroll
  for (int q = 1; q < 4; ++q) v[q] = q < cols ? v[q] : 0.f;
}
__device__ __forceinline__ bool finite4(const float (&v)[4]) {
  return isfinite(v[0]) && isfinite(v[1]) && isfinite(v[2]) && isfinite(v[3]);
}
// The pieces that the kernel has left out.  (A pass of its own: with the call in the
// kernel's loop that loop spilled, and a data gradient of 48,000 x 256 -> 1,397 took
// 394 us, 351 before.)
__device__ __noinline__ void finish_again(const Again* __restrict__ p, const Epilogue& e, int vec) {
  const int64_t J = p->g.J, ldp = part_pitch(J);
  finish_pieces(p->g.I, J, ldp, [&](int64_t i, int64_t j, int cols, int64_t k) {
    float v[4] = {};
    add_parts(p->part, p->splits, p->pitch, k, cols, v);
    if (finite4(v)) return;
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (q < cols && !isfinite(v[q])) v[q] = dot_again(p, i, j + q, 4 * k + q);
    Beside x;
    beside4<float>(e, x, i, j, cols, vec);
    finish4<float>(e, x, v, i, j, cols, vec);
  });
}
template <typename T, bool PLANES>
__global__ void __launch_bounds__(kFinishThreads, 4)
finish_kernel(const float* __restrict__ part, int splits, int64_t I, int64_t J, int64_t ldp,
              const __grid_constant__ Epilogue e, int vec, const __grid_constant__ Again again) {
  bool waited = false, left = false;
  finish_pieces(I, J, ldp, [&](int64_t i, int64_t j, int cols, int64_t k) {
    Beside x;
    beside4<T>(e, x, i, j, cols, vec);
    if (!waited) pdl_wait();      // for the partial products
    waited = true;
    float v[4] = {};
    add_parts(part, splits, I * ldp, k, cols, v);
    if (PLANES && !finite4(v)) left = true;
    else finish4<T>(e, x, v, i, j, cols, vec);
  });
  if (!waited) pdl_wait();
  if (PLANES && left) finish_again(&again, e, vec);
}

// ---- a few rows ------------------------------------------------------------------------
// The forward product of few rows: bound by reading W once, and for small W by
// the launch (one row of 512 -> 2,048 bf16: 2.3 us in a graph, 6.7 on the tensor
// cores).  A group of wk
// warps (1, 2 or 4, along the sum) takes CPW columns, every lane 16 bytes of
// each W row at a time and the same piece of MR rows of x, which stay in L1; the
// lanes' sums are then folded so that each of MR * CPW lanes holds one.  No
// tensor maps, no partial products in memory, no copies of rows off 16-byte
// boundaries: those are read element by element.
constexpr int kFewGroup = 8, kFewThreads = 256;
template <typename T, int MR>
__global__ void __launch_bounds__(kFewThreads)
few_rows_kernel(const Product g, const Epilogue e, int vec, int wk) {
  constexpr int CPW = MR >= 4 ? 2 : 1, A = MR * CPW, E = 16 / (int)sizeof(T);
  constexpr int U = MR >= 4 ? 2 : 4;     // pieces of a W row in flight
  __shared__ float sums[kFewThreads / kWarp][A];
  pdl_wait();
  const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp;
  const int per = kFewThreads / kWarp / wk;      // groups of a block
  const int64_t j0 = ((int64_t)blockIdx.x * per + warp / wk) * CPW;
  const int64_t i0 = (int64_t)blockIdx.y * MR;
  const int rows = (int)min((int64_t)MR, g.I - i0);
  // the output that this lane will hold, and whether it does
  int mine = 0;
#pragma unroll
  for (int n = A, off = 16; n > 1; n >>= 1, off >>= 1) mine += lane & off ? n / 2 : 0;
  const int64_t j = j0 + mine % CPW;
  const bool holds = (lane & (kWarp / A - 1)) == 0 && mine / CPW < rows && j < g.J && warp % wk == 0;
  Beside beside;
  if (holds) beside4<T>(e, beside, i0 + mine / CPW, j, 1, false);
  // rows and columns past the last one repeat it, so that no load is conditional
  const T *x[MR], *w[CPW];
#pragma unroll
  for (int m = 0; m < MR; ++m) x[m] = static_cast<const T*>(g.A) + (i0 + min(m, rows - 1)) * g.sai;
#pragma unroll
  for (int c = 0; c < CPW; ++c)
    w[c] = static_cast<const T*>(g.B) + min(j0 + c, g.J - 1) * g.sbj;
  float2 pair[A];      // sums of even and odd elements
#pragma unroll
  for (int i = 0; i < A; ++i) pair[i] = make_float2(0.f, 0.f);
  int64_t k = 0;
  if (vec) {
    const int64_t whole = g.R / E * E;
    const int64_t step = (int64_t)wk * kWarp * E;
    k = ((int64_t)(warp % wk) * kWarp + lane) * E;
    for (; k < whole; k += U * step) {
      Raw<T, E> rw[U][CPW];
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int c = 0; c < CPW; ++c)
          rw[u][c] = k + u * step < whole ? __ldg(reinterpret_cast<const Raw<T, E>*>(w[c] + k + u * step))
                                          : Raw<T, E>{};
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (k + u * step >= whole) break;
        Raw<T, E> rx[MR];
#pragma unroll
        for (int m = 0; m < MR; ++m) rx[m] = __ldg(reinterpret_cast<const Raw<T, E>*>(x[m] + k + u * step));
        float fw[CPW][E];
#pragma unroll
        for (int c = 0; c < CPW; ++c) to_f32<T, E>(rw[u][c], fw[c]);
#pragma unroll
        for (int m = 0; m < MR; ++m) {
          float fx[E];
          to_f32<T, E>(rx[m], fx);
#pragma unroll
          for (int c = 0; c < CPW; ++c)
#pragma unroll
            for (int i = 0; i < E; i += 2)
              pair[m * CPW + c] = ptx::ffma2(make_float2(fx[i], fx[i + 1]),
                                             make_float2(fw[c][i], fw[c][i + 1]), pair[m * CPW + c]);
        }
      }
    }
    k = whole;
  }
  float acc[A];
#pragma unroll
  for (int i = 0; i < A; ++i) acc[i] = pair[i].x + pair[i].y;
#pragma unroll 4
  for (k += (int64_t)(warp % wk) * kWarp + lane; k < g.R; k += (int64_t)wk * kWarp) {
    float f[CPW];
#pragma unroll
    for (int c = 0; c < CPW; ++c) f[c] = (float)w[c][k];
#pragma unroll
    for (int m = 0; m < MR; ++m)
#pragma unroll
      for (int c = 0; c < CPW; ++c) acc[m * CPW + c] = fmaf((float)x[m][k], f[c], acc[m * CPW + c]);
  }
  // lanes fold their sums: each keeps half of them and takes the other lane's
  // share, until one is left
#pragma unroll
  for (int n = A, off = 16; off >= 1; off >>= 1) {
    if (n > 1) {
      n >>= 1;
      const bool up = lane & off;
#pragma unroll
      for (int i = 0; i < n; ++i) {
        const float give = up ? acc[i] : acc[i + n], keep = up ? acc[i + n] : acc[i];
        acc[i] = keep + __shfl_xor_sync(0xffffffffu, give, off);
      }
    } else {
      acc[0] += __shfl_xor_sync(0xffffffffu, acc[0], off);
    }
  }
  float v[4] = {acc[0], 0.f, 0.f, 0.f};
  if (wk > 1) {
    if ((lane & (kWarp / A - 1)) == 0) sums[warp][mine] = acc[0];
    __syncthreads();
    if (holds) {
      v[0] = 0.f;
      for (int i = 0; i < wk; ++i) v[0] += sums[warp + i][mine];
    }
  }
  if (holds) finish4<T>(e, beside, v, i0 + mine / CPW, j, 1, false);
}

// Whether a forward product takes few_rows_kernel, by how often it reads W's
// elements: two rows always do; a group of up to four rows costs half a group
// of eight, and rows read element by element would have to be copied otherwise.
// (Measured in a graph, bf16, 8 rows: 1,024 x 1,024 4.3 us and 8.5 on the tensor
// cores, 2,048 x 2,048 7.1 and 7.5, 4,096 x 4,096 30 and 14; one row of the last
// 10.4 and 14.4.  fp32, 8 rows: 46 us at 4,096 x 4,096, 91 in 64 x 64 tiles.)
template <typename T>
bool takes_few_rows(const Product& g) {
  constexpr int E = 16 / (int)sizeof(T);
  if (g.I <= 2 || (sizeof(T) == 4 && g.I <= kFewGroup)) return true;
  // Many rows of few columns: a block for every eight of them costs more than tiles
  // do (here / there, bf16, K = 64: 2,048 rows 3.7 / 6.8 us of one column and 3.7 /
  // 4.3 of eight, 4,096 6.6 / 6.8 and 6.6 / 4.2, 100,000 118 / 29; fp32, one column:
  // 4,096 rows 5.4 / 7.7 and 8,192 9.4 / 7.9 at K = 64, 16,384 19 / 26 and 50,000
  // 75 / 66 at 256).  It also keeps the groups of rows below a grid's 65,535.
  if (g.I > (sizeof(T) == 4 ? std::max<int64_t>(2048, 64 * g.R) : 2048)) return false;
  const bool vec = g.sai % E == 0 && g.sbj % E == 0;
  const int64_t groups2 = g.I <= 4 ? 1 : 2 * ((g.I + kFewGroup - 1) / kFewGroup);   // halves
  return groups2 * g.J * g.R <= (vec ? 1ll << 22 : 1ll << 23);
}

template <typename T>
cudaError_t few_rows(const Product& g, const Epilogue& e, cudaStream_t st) {
  constexpr int E = 16 / (int)sizeof(T);
  const int vec = g.sai % E == 0 && g.sbj % E == 0;
  auto go = [&](auto kernel, int cpw) {
    // warps along the sum until there are 4,096 (one row of 1,024 -> 8,192 bf16
    // 6.9 us with one, 14 with four; 2,048 -> 512 3.5 and 2.5)
    int wk = 1;
    while (wk < 4 && g.J / cpw * wk < 4096 && g.R >= 4 * wk * kWarp * E) wk *= 2;
    const int64_t cols = (int64_t)(kFewThreads / kWarp / wk) * cpw;
    return launch_pdl(kernel, dim3((unsigned)((g.J + cols - 1) / cols),
                                   (unsigned)((g.I + kFewGroup - 1) / kFewGroup)),
                      dim3(kFewThreads), 0, st, g, e, vec, wk);
  };
  if (g.I <= 1) return go(few_rows_kernel<T, 1>, 1);
  if (g.I <= 2) return go(few_rows_kernel<T, 2>, 1);
  if (g.I <= 4) return go(few_rows_kernel<T, 4>, 2);
  return go(few_rows_kernel<T, kFewGroup>, 2);
}

// ---- fp32 products ----------------------------------------------------------------
// 64 x 64 output tiles, 16 of the sum at a time, 4 x 4 outputs a thread; the
// next k-tile's loads are in flight while this one is multiplied.  What is left to
// these kernels is bound by launches and latency (256 x 256 -> 256: 7.8 us
// forward; 512 x 512 -> 512 took 19 and 14 by planes).
constexpr int kTile = 64, kStep = 16, kSimtThreads = 256;
constexpr int kPer = kTile * kStep / kSimtThreads;

// AR (BR): the reduction index is the contiguous one of A (B)
template <bool AR, bool BR>
__global__ void __launch_bounds__(kSimtThreads)
simt_kernel(const Product g, const Epilogue e, int vec, float* __restrict__ part, int64_t r_per_split,
            unsigned tiles_j) {
  __shared__ float As[kStep][kTile + 4], Bs[kStep][kTile + 4];
  const unsigned ti = blockIdx.x / tiles_j;
  const int64_t i0 = (int64_t)ti * kTile, j0 = (int64_t)(blockIdx.x - ti * tiles_j) * kTile;
  const int64_t r0 = (int64_t)blockIdx.z * r_per_split, r1 = min(g.R, r0 + r_per_split);
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  const float* A = static_cast<const float*>(g.A);
  const float* B = static_cast<const float*>(g.B);
  float ra[kPer], rb[kPer];
  auto fetch = [&](int64_t rb0) {
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      const int idx = threadIdx.x + q * kSimtThreads;
      const int ka = AR ? idx % kStep : idx / kTile, ia = AR ? idx / kStep : idx % kTile;
      const int kb = BR ? idx % kStep : idx / kTile, jb = BR ? idx / kStep : idx % kTile;
      ra[q] = rb0 + ka < r1 && i0 + ia < g.I ? A[(i0 + ia) * g.sai + (rb0 + ka) * g.sar] : 0.f;
      rb[q] = rb0 + kb < r1 && j0 + jb < g.J ? B[(j0 + jb) * g.sbj + (rb0 + kb) * g.sbr] : 0.f;
    }
  };
  float acc[4][4] = {};
  fetch(r0);
  for (int64_t r = r0; r < r1; r += kStep) {
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      const int idx = threadIdx.x + q * kSimtThreads;
      As[AR ? idx % kStep : idx / kTile][AR ? idx / kStep : idx % kTile] = ra[q];
      Bs[BR ? idx % kStep : idx / kTile][BR ? idx / kStep : idx % kTile] = rb[q];
    }
    __syncthreads();
    if (r + kStep < r1) fetch(r + kStep);
#pragma unroll
    for (int k = 0; k < kStep; ++k) {
      const float4 a4 = *reinterpret_cast<const float4*>(&As[k][ty * 4]);
      const float4 b4 = *reinterpret_cast<const float4*>(&Bs[k][tx * 4]);
      const float a[4] = {a4.x, a4.y, a4.z, a4.w}, b[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
    }
    __syncthreads();
  }
  const int64_t ldp = part_pitch(g.J), oj = j0 + tx * 4;
  if (oj >= g.J) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t oi = i0 + ty * 4 + i;
    if (oi >= g.I) return;
    if (part)
      *reinterpret_cast<float4*>(part + (blockIdx.z * g.I + oi) * ldp + oj) =
          make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
    else {
      Beside x;
      beside4<float>(e, x, oi, oj, (int)min((int64_t)4, g.J - oj), vec);
      finish4<float>(e, x, acc[i], oi, oj, (int)min((int64_t)4, g.J - oj), vec);
    }
  }
}

// ---- column sums --------------------------------------------------------------------
// db: a block sums kSumCols columns over a chunk of rows, its warps taking
// every eighth row; the chunks are added by finish_kernel.  (Of small fp32
// products alone: elsewhere the product's own stages are summed.)
constexpr int kSumThreads = 256, kSumCols = 32;
__global__ void __launch_bounds__(kSumThreads)
colsum_kernel(const float* a, int64_t ld, int64_t rows, int64_t cols, int64_t rows_per_chunk,
              float* __restrict__ part) {
  __shared__ float s[kSumThreads / kWarp][kWarp];
  const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp;
  const int64_t c = (int64_t)blockIdx.x * kSumCols + lane;
  const int64_t r0 = (int64_t)blockIdx.y * rows_per_chunk, r1 = min(rows, r0 + rows_per_chunk);
  float t = 0.f;
  if (c < cols) {
#pragma unroll 8
    for (int64_t r = r0 + warp; r < r1; r += kSumThreads / kWarp) t += a[r * ld + c];
  }
  s[warp][lane] = t;
  __syncthreads();
  if (warp == 0 && c < cols) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kSumThreads / kWarp; ++w) v += s[w][lane];
    part[blockIdx.y * part_pitch(cols) + c] = v;
  }
}

// ---- plan ---------------------------------------------------------------------------
constexpr int kSms = 152;               // the plans are made for a whole GB300
constexpr int64_t kMinSplitR = 128;     // of the sum per split at least
constexpr int64_t kMaxSplits = 64;

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

int64_t simt_splits(int64_t I, int64_t J, int64_t R) {
  const int64_t tiles = cdiv(I, kTile) * cdiv(J, kTile);
  return std::max<int64_t>(1, std::min({(2 * kSms) / tiles, cdiv(R, kMinSplitR), kMaxSplits}));
}
int64_t sum_chunks(int64_t M, int64_t N) {
  return std::max<int64_t>(1, std::min({cdiv(4 * kSms, cdiv(N, kSumCols)), cdiv(M, 64), (int64_t)256}));
}
size_t split_bytes(int64_t I, int64_t J, int64_t R) {
  const int64_t s = simt_splits(I, J, R);
  return s > 1 ? (size_t)(s * I * part_pitch(J)) * 4 : 0;
}

// Whether pieces of four elements are aligned in all matrices of an epilogue
// (bases are on 16 bytes).
int fours(const Epilogue& e) {
  return e.ldo % 4 == 0 && (!e.res || e.ldres % 4 == 0) && (!e.pre || e.ldpre % 4 == 0);
}

template <typename T, bool PLANES = false>
cudaError_t launch_finish(const float* part, int64_t splits, int64_t I, int64_t J, int64_t ldp,
                          const Epilogue& e, cudaStream_t st, const Product& g = {},
                          int64_t r_per_split = 0) {
  const int64_t blocks = std::min<int64_t>(cdiv(I * ldp / 4, kFinishThreads), 16 * kSms);
  return launch_pdl(finish_kernel<T, PLANES>, dim3((unsigned)blocks), dim3(kFinishThreads), 0, st, part,
                    (int)splits, I, J, ldp, e, fours(e), Again{g, part, I * ldp, (int)splits, r_per_split});
}

cudaError_t simt_product(const Product& g, const Epilogue& e, float* part, cudaStream_t st) {
  const int64_t splits = simt_splits(g.I, g.J, g.R);
  const int64_t per = cdiv(cdiv(g.R, splits), kStep) * kStep;
  const int64_t used = cdiv(g.R, per);
  const int64_t tiles_j = cdiv(g.J, kTile), tiles = cdiv(g.I, kTile) * tiles_j;
  const dim3 grid((unsigned)tiles, 1, (unsigned)used);
  float* pp = used > 1 ? part : nullptr;
  const bool ar = g.sar == 1, br = g.sbr == 1;
  const int vec = fours(e);
  const unsigned tj = (unsigned)tiles_j;
  if (ar && br) simt_kernel<true, true><<<grid, kSimtThreads, 0, st>>>(g, e, vec, pp, per, tj);
  else if (ar) simt_kernel<true, false><<<grid, kSimtThreads, 0, st>>>(g, e, vec, pp, per, tj);
  else simt_kernel<false, false><<<grid, kSimtThreads, 0, st>>>(g, e, vec, pp, per, tj);
  const cudaError_t err = cudaGetLastError();
  if (err != cudaSuccess || used == 1) return err;
  return launch_finish<float>(pp, used, g.I, g.J, part_pitch(g.J), e, st);
}

// ---- bf16 operands on 16-byte rows ---------------------------------------------------
// TMA reads rows that start on 16-byte boundaries: others are copied once, with
// a pitch rounded up to 8 elements.  (One row starts on the base's boundary, whatever
// the pitch: callers give its length as well as its distance to a next row.)
}  // namespace
int64_t pitch8(int64_t cols) { return (cols + 7) / 8 * 8; }
size_t packed_bytes(int64_t rows, int64_t cols, int64_t ld) {
  if (ld <= 0) ld = cols;
  return ld % 8 && rows > 1 ? (size_t)(rows * pitch8(cols) * 2 + 255) / 256 * 256 : 0;
}
namespace {
constexpr int kPackThreads = 256;
__device__ __forceinline__ void copy_rows(const Copy& m, int block) {
  const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(m.src);
  const int64_t per = m.pitch / 8, n = m.rows * per, total = (m.rows - 1) * m.ld + m.cols;
  for (int64_t k = (int64_t)block * kPackThreads + threadIdx.x; k < n;
       k += (int64_t)m.blocks * kPackThreads) {
    const int64_t r = n < (1ll << 32) ? (int64_t)((uint32_t)k / (uint32_t)per) : k / per;
    const int64_t c = (k - r * per) * 8;
    m.dst[k] = load8_any(src, r * m.ld + c, total, (int)min((int64_t)8, m.cols - c));
  }
}
__global__ void __launch_bounds__(kPackThreads) pack_rows_kernel(const Copy a, const Copy b) {
  pdl_wait();
  pdl_trigger();
  if ((int)blockIdx.x < a.blocks) copy_rows(a, blockIdx.x);
  else copy_rows(b, blockIdx.x - a.blocks);
}
}  // namespace
Copy on_16_bytes(const void*& a, int64_t& ld, int64_t rows, int64_t cols, char*& work) {
  if (ld % 8 == 0) return Copy{};
  const int64_t pitch = pitch8(cols);
  if (rows == 1) {
    ld = pitch;
    return Copy{};
  }
  const Copy c{a, ld, rows, cols, pitch, rows, reinterpret_cast<uint4*>(work),
               (int)std::min<int64_t>(cdiv(rows * (pitch / 8), kPackThreads), 16 * kSms)};
  a = work;
  ld = pitch;
  work += (rows * pitch * 2 + 255) / 256 * 256;
  return c;
}
cudaError_t pack(const Copy& a, const Copy& b, cudaStream_t st) {
  if (a.blocks + b.blocks == 0) return cudaSuccess;
  return launch_pdl(pack_rows_kernel, dim3((unsigned)(a.blocks + b.blocks)), dim3(kPackThreads), 0, st, a, b);
}
namespace {

// ---- fp32 operands as three bf16 planes ------------------------------------------------
// x = x1 + x2 + x3 with bf16 x1 (x rounded), x2 (the rest rounded), x3: 24 bits
// together.  Of the nine products of two such operands the six of 2^-16 and more
// are kept; what is left out is below fp32's own rounding.  Six products at the
// tensor cores' rate are four times the CUDA cores' fp32 one.  The split is bound
// by memory: 4,999 x 1,397 (28 MB read, 42 written) 12 us.
int64_t plane_rows(int64_t rows) { return (rows + 63) / 64 * 64; }
size_t planes_bytes(int64_t rows, int64_t cols) {
  return (size_t)(3 * plane_rows(rows) * pitch8(cols)) * 2;
}
__device__ __forceinline__ void split_rows(const Copy& m, int block) {
  const float* src = static_cast<const float*>(m.src);
  const int64_t per = m.pitch / 8, n = m.rows_pad * per;
  const bool vec = m.ld % 4 == 0;
  for (int64_t k = (int64_t)block * kPackThreads + threadIdx.x; k < n;
       k += (int64_t)m.blocks * kPackThreads) {
    const int64_t r = n < (1ll << 32) ? (int64_t)((uint32_t)k / (uint32_t)per) : k / per;
    const int64_t c = (k - r * per) * 8;
    float f[8] = {}, p1[8], p2[8], p3[8];
    if (r < m.rows) {
      const float* q = src + r * m.ld + c;
      if (vec && c + 8 <= m.cols) {
        const float4 x = reinterpret_cast<const float4*>(q)[0], y = reinterpret_cast<const float4*>(q)[1];
        f[0] = x.x; f[1] = x.y; f[2] = x.z; f[3] = x.w;
        f[4] = y.x; f[5] = y.y; f[6] = y.z; f[7] = y.w;
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (c + i < m.cols) f[i] = q[i];
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      p1[i] = (float)__float2bfloat16_rn(f[i]);
      const float rest = f[i] - p1[i];      // exact
      p2[i] = (float)__float2bfloat16_rn(rest);
      p3[i] = rest - p2[i];
    }
    m.dst[k] = from_f32<__nv_bfloat16, 8>(p1);
    m.dst[n + k] = from_f32<__nv_bfloat16, 8>(p2);
    m.dst[2 * n + k] = from_f32<__nv_bfloat16, 8>(p3);
  }
}
__global__ void __launch_bounds__(kPackThreads) split_planes_kernel(const Copy a, const Copy b) {
  pdl_wait();
  pdl_trigger();
  if ((int)blockIdx.x < a.blocks) split_rows(a, blockIdx.x);
  else split_rows(b, blockIdx.x - a.blocks);
}
// Fewer multiplications than this take the CUDA cores, one or two launches
// instead of three (1,024 x 256 -> 256, 6.7e7 of them: 14.6 us forward, 12.5 and
// 18.9 the gradients; 12.1, 11.9 and 12.7 by planes; 256 x 256 -> 256 7.8, 12.5 and
// 16.9; 8.6, 13.0 and 11.7 by planes; 4,999 x 1,397 -> 512 230 to 460 and 67 to 77).
}  // namespace
bool takes_planes(int mode, int64_t M, int64_t N, int64_t K) {
  return M * N * K >= (mode == kWeight ? 1ll << 25 : 1ll << 26);
}
namespace {

}  // namespace
size_t tc_part_bytes(int64_t I, int64_t J, int64_t R, bool must_split, int terms) {
  const TcPlan p = tc_plan(I, J, R, must_split, terms);
  return p.splits > 1 || must_split ? (size_t)p.splits * I * part_pitch(J) * 4 : 0;
}
namespace {

// dW from its partial products, four columns a thread, and db from the partial
// column sums (the blocks after the first `wblocks`), all in a fixed order.
// PLANES: of a product of planes.
template <bool PLANES>
__global__ void __launch_bounds__(kFinishThreads)
finish_weight_kernel(const float* __restrict__ part, int splits, int64_t I, int64_t J, int64_t ldp,
                     float* __restrict__ dw, const float* __restrict__ sums, int64_t sum_rows,
                     float* __restrict__ db, int accumulate, int wblocks,
                     const __grid_constant__ Again again) {
  pdl_wait();
  if ((int)blockIdx.x < wblocks) {
    const int64_t n4 = I * ldp / 4, n = I * ldp;
    for (int64_t k = (int64_t)blockIdx.x * kFinishThreads + threadIdx.x; k < n4;
         k += (int64_t)wblocks * kFinishThreads) {
      const int64_t i = 4 * k / ldp, j = 4 * k - i * ldp;
      if (j >= J) continue;      // the partial rows' padding (J % 8 <= 4), which dW's rows lack
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int s = 0; s < splits; ++s) {
        const float4 x = __ldcg(reinterpret_cast<const float4*>(part + s * n) + k);
        v.x += x.x;
        v.y += x.y;
        v.z += x.z;
        v.w += x.w;
      }
      float* o = dw + i * J + j;
      float vv[4] = {v.x, v.y, v.z, v.w};
      if (PLANES && !(isfinite(v.x) && isfinite(v.y) && isfinite(v.z) && isfinite(v.w))) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (j + q < J && !isfinite(vv[q])) vv[q] = dot_again(&again, i, j + q, 4 * k + q);
      }
      if (J % 4 == 0 && !accumulate) {
        *reinterpret_cast<float4*>(o) = make_float4(vv[0], vv[1], vv[2], vv[3]);
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (j + q < J) o[q] = accumulate ? o[q] + vv[q] : vv[q];
      }
    }
    return;
  }
  __shared__ float part_sum[kFinishThreads / kWarp][kWarp];
  const int lane = threadIdx.x % kWarp, w = threadIdx.x / kWarp;
  const int64_t c = (int64_t)(blockIdx.x - wblocks) * kWarp + lane;
  float t = 0.f;
  if (c < I) {
#pragma unroll 4
    for (int64_t r = w; r < sum_rows; r += kFinishThreads / kWarp) t += __ldcg(sums + r * I + c);
  }
  part_sum[w][lane] = t;
  __syncthreads();
  float v = 0.f;
#pragma unroll
  for (int q = 0; q < kFinishThreads / kWarp; ++q) v += part_sum[q][lane];
  if (PLANES) {
    // (the warps share a second look)
    const bool mine = c < I && !isfinite(v);
    if (__syncthreads_or(mine)) {
      const Product& g = again.g;
      part_sum[w][lane] =
          mine ? sum_again(static_cast<const float*>(g.A) + c * g.sai, g.sar, g.R, w) : 0.f;
      __syncthreads();
      if (mine) {
        v = 0.f;
#pragma unroll
        for (int q = 0; q < kFinishThreads / kWarp; ++q) v += part_sum[q][lane];
      }
    }
  }
  if (w == 0 && c < I) db[c] = accumulate ? db[c] + v : v;
}

// (part nullptr: dW is there already)
template <bool PLANES>
cudaError_t launch_finish_weight(const float* part, int splits, const Product& g, const Epilogue& e,
                                 const float* sums, int64_t sum_rows, float* db, cudaStream_t st,
                                 int64_t r_per_split = 0) {
  const int64_t ldp = part_pitch(g.J);
  const int wb = part ? (int)std::min<int64_t>(cdiv(g.I * ldp / 4, kFinishThreads), 8 * kSms) : 0;
  const int sb = db ? (int)cdiv(g.I, kWarp) : 0;
  return launch_pdl(finish_weight_kernel<PLANES>, dim3((unsigned)(wb + sb)), dim3(kFinishThreads), 0, st,
                    part, splits, g.I, g.J, ldp, static_cast<float*>(e.out), sums, sum_rows, db,
                    e.accumulate, wb, Again{g, part, g.I * ldp, splits, r_per_split});
}
size_t sum_bytes(int64_t I, int64_t J, int64_t R, const TcPlan& plan) {
  const Product g{nullptr, 0, 0, nullptr, 0, 0, I, J, R};
  return (size_t)(tc_sum_rows(g, plan) * I * 4 + 255) / 256 * 256;
}

// A bf16 result straight from the accumulator has the drift of its truncations,
// 7.6e-8 of the sum's size a 16-deep step.  Sums past 2^16 (3e-4 there, a sixth of
// bf16's half unit; measured 1.5e-3 at 2^18 and 6.3e-3 at 2^20) are therefore taken
// out by windows and finished from partial products like split ones (2,048 x
// 2^18 -> 2,048: 1,173 us from the accumulator, 1,356 so).
bool long_sum(int64_t R) { return R > 1ll << 16; }

cudaError_t tc_run(const Product& g, const Epilogue& e, char* work, int* err, cudaStream_t st) {
  const TcPlan plan = tc_plan(g.I, g.J, g.R, long_sum(g.R));
  float* part = plan.splits > 1 || long_sum(g.R) ? reinterpret_cast<float*>(work) : nullptr;
  const cudaError_t x = tc_product(g, e, plan, part, nullptr, err, num_sms(), st);
  if (x != cudaSuccess || !part) return x;
  return launch_finish<__nv_bfloat16>(part, plan.splits, g.I, g.J, part_pitch(g.J), e, st);
}

// The sums of an fp32 product, by planes, as partial products (and db's partial
// column sums).  A lies as rows of `ca` elements (its own row or the sum's index), so does B.
cudaError_t planes_product(const Product& g, const Epilogue& e, char* work, int* err, cudaStream_t st,
                           bool with_sums, float** sums, PartialSums* out) {
  const bool amn = g.sai == 1 && e.mode == kWeight, bmn = e.mode != kForward;
  Product t = g;
  auto split = [&](const void*& a, int64_t ld, int64_t rows, int64_t cols, int64_t& pitch) {
    pitch = pitch8(cols);
    const int64_t pad = plane_rows(rows);
    const Copy c{a, ld, rows, cols, pitch, pad, reinterpret_cast<uint4*>(work),
                 (int)std::min<int64_t>(cdiv(pad * (pitch / 8), kPackThreads), 16 * kSms)};
    a = work;
    work += (planes_bytes(rows, cols) + 255) / 256 * 256;
    return c;
  };
  const Copy ca = amn ? split(t.A, g.sar, g.R, g.I, t.sar) : split(t.A, g.sai, g.I, g.R, t.sai);
  const Copy cb = bmn ? split(t.B, g.sbr, g.R, g.J, t.sbr) : split(t.B, g.sbj, g.J, g.R, t.sbj);
  cudaError_t x = launch_pdl(split_planes_kernel, dim3((unsigned)(ca.blocks + cb.blocks)), dim3(kPackThreads),
                             0, st, ca, cb);
  if (x != cudaSuccess) return x;
  const TcPlan plan = tc_plan(g.I, g.J, g.R, true, kTerms);
  *sums = with_sums ? reinterpret_cast<float*>(work) : nullptr;
  if (with_sums) work += sum_bytes(g.I, g.J, g.R, plan);
  float* part = reinterpret_cast<float*>(work);
  const int64_t ldp = part_pitch(g.J);
  *out = PartialSums{part, plan.splits, g.I * ldp, ldp, (int64_t)plan.kt_per_split / kTerms * kSumStep};
  return tc_product(t, e, plan, part, *sums, err, num_sms(), st, plane_rows(amn ? g.R : g.I),
                    plane_rows(bmn ? g.R : g.J));
}
// out = epilogue of an fp32 product, by planes.
cudaError_t planes_run(const Product& g, const Epilogue& e, float* db, char* work, int* err,
                       cudaStream_t st) {
  float* sums;
  PartialSums s;
  const cudaError_t x = planes_product(g, e, work, err, st, db != nullptr, &sums, &s);
  if (x != cudaSuccess) return x;
  if (e.mode == kWeight)
    return launch_finish_weight<true>(s.part, s.splits, g, e, sums,
                                      tc_sum_rows(g, tc_plan(g.I, g.J, g.R, true, kTerms)), db, st, s.r_per_split);
  return launch_finish<float, true>(s.part, s.splits, g.I, g.J, s.ldp, e, st, g, s.r_per_split);
}
}  // namespace
cudaError_t planes_sums(const Product& g, int mode, char* work, int* err, cudaStream_t st, PartialSums* out) {
  Epilogue e{};
  e.mode = mode;
  e.act = PPO_ACT_NONE;
  float* sums;
  return planes_product(g, e, work, err, st, false, &sums, out);
}
size_t planes_need(int64_t ra, int64_t ca, int64_t rb, int64_t cb, int64_t I, int64_t J, int64_t R) {
  return planes_bytes(ra, ca) + planes_bytes(rb, cb) + 512 + tc_part_bytes(I, J, R, true, kTerms) +
         sum_bytes(I, J, R, tc_plan(I, J, R, true, kTerms));
}

namespace {
// A gradient that is added to, or whose rows TMA cannot store, is finished from
// partial products even where the sum is not split.
bool must_finish(int64_t J, int accumulate) { return accumulate || J % 4; }
size_t tc_sum_bytes(int64_t N, int64_t K, int64_t M, bool must) {
  return sum_bytes(N, K, M, tc_plan(N, K, M, must));
}
cudaError_t tc_run_weight(const Product& g, const Epilogue& e, float* db, char* work, int* err,
                          cudaStream_t st) {
  const bool must = must_finish(g.J, e.accumulate);
  const TcPlan plan = tc_plan(g.I, g.J, g.R, must);
  const int64_t rows = tc_sum_rows(g, plan);
  float* sums = db ? reinterpret_cast<float*>(work) : nullptr;
  float* part = plan.splits > 1 || must
                    ? reinterpret_cast<float*>(work + tc_sum_bytes(g.I, g.J, g.R, must))
                    : nullptr;
  const cudaError_t x = tc_product(g, e, plan, part, sums, err, num_sms(), st);
  if (x != cudaSuccess || (!part && !db)) return x;
  return launch_finish_weight<false>(part, plan.splits, g, e, sums, rows, db, st);
}

cudaError_t column_sums(const float* dz, int64_t ld, int64_t M, int64_t N, float* db,
                        int accumulate, float* part, cudaStream_t st) {
  const int64_t chunks = sum_chunks(M, N), per = cdiv(M, chunks), used = cdiv(M, per);
  const dim3 grid((unsigned)cdiv(N, kSumCols), (unsigned)used);
  colsum_kernel<<<grid, kSumThreads, 0, st>>>(dz, ld, M, N, per, part);
  const cudaError_t err = cudaGetLastError();
  if (err != cudaSuccess) return err;
  Epilogue e{};
  e.mode = kWeight;
  e.out = db;
  e.ldo = N;
  e.accumulate = accumulate;
  return launch_finish<float>(part, used, 1, N, part_pitch(N), e, st);
}

// The fp32 product on the units that suit its size (db: kWeight alone, nullable).
cudaError_t run_f32(const Product& g, const Epilogue& e, int64_t M, int64_t N, int64_t K, float* db,
                    void* work, float* part, cudaStream_t st) {
  if (takes_planes(e.mode, M, N, K))
    return planes_run(g, e, db, reinterpret_cast<char*>(part), static_cast<int*>(work), st);
  const cudaError_t x = simt_product(g, e, part, st);
  if (x != cudaSuccess || !db) return x;
  return column_sums(static_cast<const float*>(g.A), g.sar, M, N, db, e.accumulate, part, st);
}

}  // namespace
bool sizes_ok(int64_t M, int64_t N, int64_t K) {
  // 32-bit TMA coordinates, of three planes too, and tile counts
  constexpr int64_t top = 1ll << 29;
  return M >= 1 && N >= 1 && K >= 1 && M < top && N < top && K < top && M <= (1ll << 40) / N &&
         M <= (1ll << 40) / K && N <= (1ll << 40) / K;
}

}  // namespace lin
}  // namespace ppo

using namespace ppo;
using ppo::ops::al16;

namespace {

constexpr size_t kCtrl = 256;   // the error word and its padding

ppo_status checked(std::initializer_list<const void*> ptrs, const void* work, size_t work_bytes,
                   size_t need) {
  for (const void* p : ptrs)
    if (!al16(p)) return PPO_ERR_ALIGN;
  if (!work || work_bytes < need) return PPO_ERR_INVALID;
  if (!al16(work)) return PPO_ERR_ALIGN;
  return ops::num_sms() > 0 ? PPO_OK : PPO_ERR_CUDA;
}
using ops::status_of;
// Workspace of one direction: the copies of its two operands (pitches lda,
// ldb) and the partial products or column sums behind them.
size_t need(int32_t dtype, int mode, int64_t M, int64_t N, int64_t K, int64_t lda, int64_t ldb) {
  if (dtype == PPO_DTYPE_F32) {
    const size_t sums = mode == lin::kWeight ? (size_t)(lin::sum_chunks(M, N) * lin::part_pitch(N)) * 4 : 0;
    size_t part = mode == lin::kForward ? lin::split_bytes(M, N, K)
                  : mode == lin::kData  ? lin::split_bytes(M, K, N)
                                        : lin::split_bytes(N, K, M);
    if (lin::takes_planes(mode, M, N, K))
      part = std::max(part, mode == lin::kForward ? lin::planes_need(M, K, N, K, M, N, K)
                            : mode == lin::kData  ? lin::planes_need(M, N, N, K, M, K, N)
                                                  : lin::planes_need(M, N, M, K, N, K, M));
    return kCtrl + std::max(part, sums);
  }
  switch (mode) {
    case lin::kForward:
      return kCtrl + lin::packed_bytes(M, K, lda) + lin::packed_bytes(N, K, ldb) +
             lin::tc_part_bytes(M, N, K, lin::long_sum(K));
    case lin::kData:
      return kCtrl + lin::packed_bytes(M, N, lda) + lin::packed_bytes(N, K, ldb) +
             lin::tc_part_bytes(M, K, N, lin::long_sum(N));
  }
  return kCtrl + lin::packed_bytes(M, N, lda) + lin::packed_bytes(M, K, ldb) +
         std::max(lin::tc_sum_bytes(N, K, M, false) + lin::tc_part_bytes(N, K, M, false),
                  lin::tc_sum_bytes(N, K, M, true) + lin::tc_part_bytes(N, K, M, true));
}
float* parts(void* work) { return reinterpret_cast<float*>(static_cast<char*>(work) + kCtrl); }

}  // namespace

extern "C" {

ppo_status ppo_linear_workspace_bytes(int32_t dtype, int64_t M, int64_t N, int64_t K, int64_t ldx,
                                      int64_t ldw, int64_t ldz, size_t* bytes) {
  if (!bytes || !ops::dtype_ok(dtype) || !lin::sizes_ok(M, N, K)) return PPO_ERR_INVALID;
  *bytes = std::max({need(dtype, lin::kForward, M, N, K, ldx, ldw),
                     need(dtype, lin::kData, M, N, K, ldz, ldw),
                     need(dtype, lin::kWeight, M, N, K, ldz, ldx)});
  return PPO_OK;
}

ppo_status ppo_linear_forward(int32_t dtype, const void* x, int64_t ldx, const void* w, int64_t ldw,
                              const float* bias, int32_t act, const void* res, int64_t ldres,
                              int64_t M, int64_t N, int64_t K, void* y, int64_t ldy, void* pre,
                              int64_t ldpre, void* work, size_t work_bytes, cudaStream_t st) {
  if (!x || !w || !y || !ops::act_ok(act)) return PPO_ERR_INVALID;
  if (!ops::dtype_ok(dtype) || !lin::sizes_ok(M, N, K) || !ops::extent_ok(M, ldx, K) || !ops::extent_ok(N, ldw, K) || !ops::extent_ok(M, ldy, N) ||
      (res && !ops::extent_ok(M, ldres, N)) || (pre && !ops::extent_ok(M, ldpre, N)) ||
      (y == res && ldy != ldres))
    return PPO_ERR_INVALID;
  const ppo_status s = checked({x, w, bias, res, y, pre}, work, work_bytes,
                               need(dtype, lin::kForward, M, N, K, ldx, ldw));
  if (s != PPO_OK) return s;
  lin::Epilogue e{};
  e.mode = lin::kForward;
  e.act = act;
  e.bias = bias;
  e.res = res;
  e.ldres = ldres;
  e.pre = pre;
  e.ldpre = ldpre;
  e.out = y;
  e.ldo = ldy;
  const lin::Product g{x, ldx, 1, w, ldw, 1, M, N, K};
  if (dtype == PPO_DTYPE_F32)
    return status_of(lin::takes_few_rows<float>(g) ? lin::few_rows<float>(g, e, st)
                                                   : lin::run_f32(g, e, M, N, K, nullptr, work, parts(work), st));
  if (lin::takes_few_rows<__nv_bfloat16>(g)) return status_of(lin::few_rows<__nv_bfloat16>(g, e, st));
  char* free = reinterpret_cast<char*>(parts(work));
  const lin::Copy ca = lin::on_16_bytes(x, ldx, M, K, free), cb = lin::on_16_bytes(w, ldw, N, K, free);
  cudaError_t err = lin::pack(ca, cb, st);
  if (err == cudaSuccess)
    err = lin::tc_run({x, ldx, 1, w, ldw, 1, M, N, K}, e, free, static_cast<int*>(work), st);
  return status_of(err);
}

ppo_status ppo_linear_backward_data(int32_t dtype, const void* dz, int64_t lddz, const void* w,
                                    int64_t ldw, const void* pre_in, int64_t ldpre, int32_t act,
                                    const void* res, int64_t ldres, int64_t M, int64_t N,
                                    int64_t K, void* dx, int64_t lddx, void* work,
                                    size_t work_bytes, cudaStream_t st) {
  if (!dz || !w || !dx || !ops::act_ok(act) || (act != PPO_ACT_NONE && !pre_in))
    return PPO_ERR_INVALID;
  if (!ops::dtype_ok(dtype) || !lin::sizes_ok(M, N, K) || !ops::extent_ok(M, lddz, N) || !ops::extent_ok(N, ldw, K) || !ops::extent_ok(M, lddx, K) ||
      (res && !ops::extent_ok(M, ldres, K)) ||
      (act != PPO_ACT_NONE && !ops::extent_ok(M, ldpre, K)) || (dx == res && lddx != ldres))
    return PPO_ERR_INVALID;
  const ppo_status s = checked({dz, w, pre_in, res, dx}, work, work_bytes,
                               need(dtype, lin::kData, M, N, K, lddz, ldw));
  if (s != PPO_OK) return s;
  lin::Epilogue e{};
  e.mode = lin::kData;
  e.act = act;
  e.pre = const_cast<void*>(pre_in);
  e.ldpre = ldpre;
  e.res = res;
  e.ldres = ldres;
  e.out = dx;
  e.ldo = lddx;
  if (dtype == PPO_DTYPE_F32)
    return status_of(
        lin::run_f32({dz, lddz, 1, w, 1, ldw, M, K, N}, e, M, N, K, nullptr, work, parts(work), st));
  char* free = reinterpret_cast<char*>(parts(work));
  const lin::Copy ca = lin::on_16_bytes(dz, lddz, M, N, free), cb = lin::on_16_bytes(w, ldw, N, K, free);
  cudaError_t err = lin::pack(ca, cb, st);
  if (err == cudaSuccess)
    err = lin::tc_run({dz, lddz, 1, w, 1, ldw, M, K, N}, e, free, static_cast<int*>(work), st);
  return status_of(err);
}

ppo_status ppo_linear_backward_weight(int32_t dtype, const void* dz, int64_t lddz, const void* x,
                                      int64_t ldx, int64_t M, int64_t N, int64_t K, float* dw,
                                      float* db, int32_t accumulate, void* work,
                                      size_t work_bytes, cudaStream_t st) {
  if (!dz || !x || !dw) return PPO_ERR_INVALID;
  if (!ops::dtype_ok(dtype) || !lin::sizes_ok(M, N, K) || !ops::extent_ok(M, lddz, N) || !ops::extent_ok(M, ldx, K))
    return PPO_ERR_INVALID;
  const ppo_status s = checked({dz, x, dw, db}, work, work_bytes,
                               need(dtype, lin::kWeight, M, N, K, lddz, ldx));
  if (s != PPO_OK) return s;
  lin::Epilogue e{};
  e.mode = lin::kWeight;
  e.out = dw;
  e.ldo = K;
  e.accumulate = accumulate != 0;
  if (dtype == PPO_DTYPE_F32)
    return status_of(
        lin::run_f32({dz, 1, lddz, x, 1, ldx, N, K, M}, e, M, N, K, db, work, parts(work), st));
  char* free = reinterpret_cast<char*>(parts(work));
  const lin::Copy ca = lin::on_16_bytes(dz, lddz, M, N, free), cb = lin::on_16_bytes(x, ldx, M, K, free);
  cudaError_t err = lin::pack(ca, cb, st);
  if (err == cudaSuccess)
    err = lin::tc_run_weight({dz, 1, lddz, x, 1, ldx, N, K, M}, e, db, free,
                             static_cast<int*>(work), st);
  return status_of(err);
}

ppo_status ppo_work_status(void* work, cudaStream_t st) {
  if (!work) return PPO_ERR_INVALID;
  if (!al16(work)) return PPO_ERR_ALIGN;
  int32_t word = 0;
  cudaError_t e = cudaMemcpyAsync(&word, work, sizeof(word), cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e != cudaSuccess || word == 0) return status_of(e);
  e = cudaMemsetAsync(work, 0, sizeof(word), st);
  return e == cudaSuccess ? PPO_ERR_TIMEOUT : status_of(e);
}

}  // extern "C"
