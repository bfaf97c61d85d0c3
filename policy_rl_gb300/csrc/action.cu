// action.cu -- the policy over any number of actions: log-probability and
// entropy of a row of logits, and the clipped policy loss with its gradient.
//
// Of a row's logits l over the allowed actions, with m = max l, in powers of two
// (k = log2 e, u = l k - m k):
//   s = sum 2^u,  t = sum 2^u u,   logp_j = (u_j - log2 s) / k,   H = (log2 s - t / s) / k,
// and with c and W the row's slope and weight (row_terms below) the gradient is
//   W (c (1[j = a] - p_j) + ent p_j (logp_j + H))
//     = 2^(u_j) (A1 u_j + A0) + 1[j = a] W c,
//   A1 = W ent / (k s),   A0 = W (ent (H - log2 s / k) - c) / s.
// u is one fused multiply-add: m k is rounded once for the row, the same in every
// use, so that its rounding cancels between 2^u, s and t.
//
// What bounds it: memory, the row read once and the gradient written once, and of bf16
// rows as much the 16 instructions of an element, two exponentials among them.  A row
// therefore stays in registers between its statistics and its gradient, 64 elements a
// thread, two blocks of 512 threads an SM; the next row comes meanwhile by copies
// into shared memory.  Registers are what it is made of: 20 bytes of spills less in the
// kernel of 8,192 x 32,768 were worth 14 % (hence masks and clusters at compile time, a
// row's own numbers one to a lane, joined statistics read twice).
// Measured in a graph (of the copy rate): 8,192 x 32,768 bf16 182 us (87 %), with a mask 280
// (71 %), 8,192 x 16,384 fp32 162 (98 %), 1,001 x 50,257 bf16 56 (53 %: one block an SM, rows
// off 16-byte boundaries, seven rounds of 152 rows), with a mask 77, 65,536 x 18 fp32 with
// a mask 8.1 (one round of rows, their terms, the sums), one row of 131,072 bf16 6.4 (forward
// 4.6).  Forward alone 8,192 x 32,768 bf16 102 (78 %), with a mask 191 (62 %), 8,192 x 16,384
// fp32 85 (93 %), 65,536 x 18 fp32 with a mask 4.2.  A gradient whose rows lie on other places of
// 16 bytes than the logits' is stored by element: 8,192 x 32,768 bf16 from a pitch of 32,768 to
// one of 32,769 883 us, to one of 32,776 178.
// Left: the row kept in shared memory and more threads (8,192 x 32,768 217 to 252), a cluster's
// statistics by copies that count on barriers of their own (4,096 x 131,072 635).  The mask's
// L2 lines are fetched ahead (1,001 x 50,257 98 without), its bytes are not: in shared memory
// they cost spills in a kernel that served rows with and without a mask, and have not been
// tried since the two have kernels of their own.
#include <algorithm>
#include <cfloat>
#include <math_constants.h>

#include "ops.cuh"
#include "tc_ptx.cuh"

namespace ppo {
namespace {

using namespace ops;

constexpr int kRowThreads = 128;     // block of the kernels that give a row to lanes of a warp
constexpr int kMaxBlocks = 1216;     // blocks of a call: rows are walked by their stride
constexpr int kTerms = 8;            // sums of d_stats
constexpr int kMaxCluster = 8;

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
  float* part;                       // [kTerms][blocks]
};

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kLow = -1e30f;       // what stands for -inf in a row's pieces

// A row's statistics: maximum, sum of 2^u, sum of 2^u u.
struct Stat {
  float m, s, t;
};

// What a row's gradient needs beyond its logits.
struct RowTerms {
  float a0, a1, hot;       // gradient: 2^u (a1 u + a0), + hot at the action
  bool kept;
};
// A row's own numbers, fetched ahead of its statistics (the same in all its threads).
struct RowInput {
  int a;                   // its action, -1: none
  float x, u;              // the action's logit, -inf where it is not allowed, and its u
  float old, adv, ref, w;
};
// s.x: a sum, s.y: its compensation (none beside an infinity)
__device__ __forceinline__ float2 add_kahan(float2 s, float x) {
  const float y = x - s.y, t = s.x + y, r = (t - s.x) - y;
  return make_float2(t, fabsf(t) < CUDART_INF_F ? r : 0.f);
}
// Two such sums as one, the rounding kept (the exact sum of two numbers of Knuth 1969, "The Art of
// Computer Programming" 2)
__device__ __forceinline__ float2 join_kahan(float2 a, float2 b) {
  const float t = a.x + b.x, z = t - a.x, r = (a.x - (t - z)) + (b.x - z);
  return make_float2(t, fabsf(t) < CUDART_INF_F ? (a.y + b.y) - r : 0.f);
}
// The sum of `n` lanes' next to one another, in each of them.
__device__ __forceinline__ float2 lanes_kahan(float2 s, int n) {
#pragma unroll
  for (int o = n / 2; o > 0; o >>= 1)
    s = join_kahan(s, make_float2(__shfl_xor_sync(0xffffffffu, s.x, o), __shfl_xor_sync(0xffffffffu, s.y, o)));
  return s;
}
// A thread's sums over rows, in shared memory (only a row's first thread has any),
// compensated (Kahan): an add costs four fp32 operations, where one in 64 bits would
// hold the FP64 units for 15 clocks.
struct RowSums {
  float2* at;              // [kTerms], `step` apart: sum and compensation
  int step;
  __device__ __forceinline__ void add(int i, float x) { at[i * step] = add_kahan(at[i * step], x); }
};

// Every thread of a row takes its terms; `lead` writes what the row gives and adds it up.
__device__ __forceinline__ RowTerms row_terms(const ActionArgs& p, int64_t row, const Stat& st, const RowInput& in,
                                              bool lead, RowSums sums) {
  RowTerms r{0.f, 0.f, 0.f, false};
  const bool has = in.a >= 0;
  const float logs = logf(st.s);
  const float H = st.s == 0.f ? 0.f : logs - st.t / st.s * kLn2;
  // (u ends at kLow, where p is 0 long since; a finite logit's logp does not)
  const bool none = in.x == -CUDART_INF_F;
  const float far = in.x - st.m, d = far < 0.5f * kLow ? fmaxf(far, -FLT_MAX) : in.u * kLn2;
  const float lp = has ? (none ? in.x : d - logs) : 0.f;
  if (lead) {
    if (p.logp) p.logp[row] = lp;
    if (p.entropy) p.entropy[row] = H;
  }
  if (!p.dl) return r;
  if (!has || none) {
    if (lead && p.part) sums.add(7, 1.f);
    return r;
  }
  if (in.w == 0.f) return r;
  const float u = lp - in.old, ratio = expf(u);
  // (an advantage of 0 makes 0 of any ratio, of one past fp32's range too)
  const float by = in.adv == 0.f && u < CUDART_INF_F ? 1.f : ratio;
  const float s1 = by * in.adv, s2 = fminf(fmaxf(by, p.lo), p.hi) * in.adv;
  // (s1 alone is NaN where the ratio is, or is e^inf beside an advantage of 0)
  const float pg = s1 <= s2 ? -s1 : s1 != s1 ? s1 : -s2;
  float c = s1 <= s2 ? -s1 : s1 != s1 ? s1 : 0.f, kl = 0.f;
  if (p.ref) {
    const float y = in.ref - lp, em = expm1f(y);
    kl = em - y;
    // (a coefficient of 0 leaves out what fp32 may not hold: from y = 89 on)
    if (p.kl != 0.f) c -= p.kl * em;
  }
  const float W = p.scale * in.w;
  if (lead && p.part) {
    sums.add(0, W * (pg + (p.kl != 0.f ? p.kl * kl : 0.f) - p.ent * H));
    sums.add(1, W * pg);
    sums.add(2, W * kl);
    sums.add(3, W * H);
    sums.add(4, ratio < p.lo || ratio > p.hi ? W : 0.f);
    sums.add(5, W * (expm1f(u) - u));
    sums.add(6, W);
  }
  r.kept = true;
  r.hot = W * c;
  const float k = W / st.s;
  r.a1 = k * p.ent * kLn2;
  r.a0 = k * (p.ent * (H - logs) - c);
  return r;
}

// ---- pieces of 16 bytes ------------------------------------------------------------------
// A row is handled as the aligned 16-byte pieces that hold it; its first and last
// piece may hold elements that are not its own, which count as -inf.
template <typename T>
struct Piece {
  static constexpr int E = 16 / (int)sizeof(T);
  static constexpr uint32_t kNone = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;     // -inf
  uint32_t w[4];
  __device__ __forceinline__ void none() {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = kNone;
  }
  // element i becomes -inf
  __device__ __forceinline__ void drop(int i) {
    if constexpr (sizeof(T) == 2) w[i / 2] = i & 1 ? (w[i / 2] & 0xffffu) | 0xff800000u : (w[i / 2] & 0xffff0000u) | 0xff80u;
    else w[i] = kNone;
  }
  __device__ __forceinline__ float2 pair(int i) const {      // elements 2 i, 2 i + 1
    if constexpr (sizeof(T) == 2) return make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    else return make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
  }
  __device__ __forceinline__ void put(int i, float2 v) {
    if constexpr (sizeof(T) == 2) w[i] = pack_bf16x2(v.x, v.y);
    else {
      w[2 * i] = __float_as_uint(v.x);
      w[2 * i + 1] = __float_as_uint(v.y);
    }
  }
  __device__ __forceinline__ float max() const {
    if constexpr (sizeof(T) == 2) {
      auto h = [&](int i) { return *reinterpret_cast<const __nv_bfloat162*>(&w[i]); };
      const __nv_bfloat162 m = __hmax2(__hmax2(h(0), h(1)), __hmax2(h(2), h(3)));
      return fmaxf(__low2float(m), __high2float(m));
    } else {
      auto f = [&](int i) { return __uint_as_float(w[i]); };
      return fmaxf(fmaxf(f(0), f(1)), fmaxf(f(2), f(3)));
    }
  }
};
// 16 bytes into shared memory without registers; a thread waits for its own copies alone
__device__ __forceinline__ void fetch16(uint32_t dst, const void* p) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(p) : "memory");
}
__device__ __forceinline__ void fetched() { asm volatile("cp.async.wait_all;" ::: "memory"); }
__device__ __forceinline__ void store16(void* p, const uint32_t (&w)[4]) {
  asm volatile("st.global.v4.b32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
               : "memory");
}

// PRMT with a sign selector (8 + byte): that byte's top bit, eight times
__device__ __forceinline__ uint32_t spread(uint32_t v, uint32_t selector) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %1, %2;" : "=r"(r) : "r"(v), "r"(selector));
  return r;
}
// The mask bytes of a piece, four of them a word: E bytes from `sh` on in the two words
// of E bytes at a.
template <int E>
__device__ __forceinline__ void mask_words(const uint8_t* a, int sh, uint32_t (&v)[E / 4]) {
  using Word = typename RawOf<E>::type;       // 4 or 8 bytes
  uint32_t b[E / 4 + 1 + (E == 8)] = {};
  const Word w0 = *reinterpret_cast<const Word*>(a);
  memcpy(b, &w0, E);
  if (sh) {
    const Word w1 = *reinterpret_cast<const Word*>(a + E);
    memcpy(b + E / 4, &w1, E);
  }
  if constexpr (E == 8) {
    if (sh & 4) {
      b[0] = b[1];
      b[1] = b[2];
      b[2] = b[3];
    }
  }
#pragma unroll
  for (int i = 0; i < E / 4; ++i) v[i] = __funnelshift_r(b[i], b[i + 1], 8 * (sh & 3));
}
// The same one by one, for the mask's first and last: 0 where the row has none.
template <int E>
__device__ __forceinline__ void mask_bytes(const uint8_t* row, int j, int V, uint32_t (&v)[E / 4]) {
#pragma unroll
  for (int i = 0; i < E / 4; ++i) {
    v[i] = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int e = j + 4 * i + k;
      if (e >= 0 && e < V && row[e]) v[i] |= 1u << (8 * k);
    }
  }
}
// Elements of a piece whose mask bytes are 0 become -inf.
template <typename T>
__device__ __forceinline__ void cover(Piece<T>& x, const uint32_t (&v)[Piece<T>::E / 4]) {
#pragma unroll
  for (int i = 0; i < Piece<T>::E / 4; ++i) {
    // the top bit of each byte that is not 0, spread over the element by PRMT's sign mode
    const uint32_t nz = ((v[i] & 0x7f7f7f7fu) + 0x7f7f7f7fu) | v[i];
    if constexpr (sizeof(T) == 2) {
      const uint32_t m0 = spread(nz, 0x9988), m1 = spread(nz, 0xbbaa);
      x.w[2 * i] = (x.w[2 * i] & m0) | (Piece<T>::kNone & ~m0);
      x.w[2 * i + 1] = (x.w[2 * i + 1] & m1) | (Piece<T>::kNone & ~m1);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t m = spread(nz, 0x8888 + 0x1111 * k);
        x.w[k] = (x.w[k] & m) | (Piece<T>::kNone & ~m);
      }
    }
  }
}

// ---- reductions over a row's threads ---------------------------------------------------
template <int G>
__device__ __forceinline__ float lanes_max(float v) {
  if constexpr (G == kWarp) {
    // in the order of integers; no NaN comes here
    const int b = __float_as_int(v), o = __reduce_max_sync(0xffffffffu, b >= 0 ? b : b ^ 0x7fffffff);
    return __int_as_float(o >= 0 ? o : o ^ 0x7fffffff);
  } else {
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
  }
}
template <int G>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float max_nan(float a, float b) {      // NaN where one is
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// u and 2^u of a pair, base = m k
__device__ __forceinline__ float2 exp_pair(float2 x, float base, float2& u) {
  u = ptx::ffma2(x, make_float2(kLog2e, kLog2e), make_float2(-base, -base));
  float2 e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(u.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(u.y));
  return e;
}

// Pieces are made safe for 2^u u and 2^u (a1 u + a0), which would be NaN at u = -inf:
// nothing below kLow is left in them.  In a warp whose maximum m is ordinary that
// is all.  Past that m k's rounding would be felt, and the logits become their
// distances from m: exact ones in fp32; in bf16, where neighbours are 2^8 apart from
// 2^15 on, 0 at the maximum and kLow elsewhere (2^u is 1 and 0).
template <typename T>
__device__ __forceinline__ bool is_wild(float m) { return !(fabsf(m) < (sizeof(T) == 2 ? 32768.f : 65536.f)); }
template <typename T>
__device__ __forceinline__ void make_safe(Piece<T>& x) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 2) {
      constexpr uint32_t low = 0xf149f149u;      // -9.95e29, twice
      asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(x.w[i]) : "r"(low));
    } else {
      x.w[i] = __float_as_uint(max_nan(__uint_as_float(x.w[i]), kLow));
    }
  }
}
// a logit's distance from m (infinite m: NaN at +inf as the formula gives it, kLow at -inf)
template <typename T>
__device__ __forceinline__ float distance(float x, float m) {
  if (m == -CUDART_INF_F) return x != x ? x : kLow;
  if constexpr (sizeof(T) == 2) return x == m ? m - m : x != x ? x : kLow;
  else return max_nan(x - m, kLow);
}
template <typename T>
__device__ __forceinline__ void make_safe_wild(Piece<T>& x, float m) {
#pragma unroll
  for (int i = 0; i < Piece<T>::E / 2; ++i) {
    const float2 v = x.pair(i);
    x.put(i, make_float2(distance<T>(v.x, m), distance<T>(v.y, m)));
  }
}
// m k, rounded wherever it is used: fused into a sum it would keep what the other uses drop, by
// which a warp's sums and its gradients would differ (0.3 % at m = 60,000)
__device__ __forceinline__ float scaled(float m) { return __fmul_rn(m, kLog2e); }
// What that rounding drops of m k: distances from m, which are exact, are brought by it to what
// the others count from, since both kinds meet in a row whose warps lie on either side of the
// border.  (Not in bf16, where 2^u is 1 or 0 there; past 2^17 logits of the other kind are
// so far off that their 2^u is 0.)
template <typename T>
__device__ __forceinline__ float dropped(float m) {
  return sizeof(T) == 4 && fabsf(m) < 131072.f ? fmaf(m, kLog2e, -scaled(m)) : 0.f;
}
// what to take from a logit's k-fold (a wild warp's: from its distance's) for u, in a row
// whose maximum is m and a warp whose own is m0
template <typename T>
__device__ __forceinline__ float base_for(float m, float m0) {
  return is_wild<T>(m0) ? scaled(fminf(m - m0, -kLow)) - dropped<T>(m) : scaled(fminf(m, -kLow));
}
// the same of a warp's own maximum
template <typename T>
__device__ __forceinline__ float own_base(float m0) {
  return is_wild<T>(m0) ? -dropped<T>(m0) : scaled(m0);
}

__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void put_remote(uint32_t addr, uint32_t rank, float a, float b, float c) {
  asm volatile(
      "{\n\t.reg .b32 r;\n\tmapa.shared::cluster.u32 r, %0, %1;\n\t"
      "st.shared::cluster.v4.f32 [r], {%2, %3, %4, %4};\n\t}" ::"r"(addr),
      "r"(rank), "f"(a), "f"(b), "f"(c)
      : "memory");
}

// What the threads of a block's row take from its first warp.
struct RowShared {
  RowTerms r;
  float m, u;
};

// A row belongs to G threads (lanes of a warp, a block, or all blocks of a cluster),
// each of which keeps up to GR of its 16-byte pieces in registers between the
// statistics and the gradient, so that the row is read once.  ON16: all rows, of
// the gradient too, start on 16-byte boundaries.  MASK: there may be a mask.  CLUSTER:
// more than one block a row.  (Each of them at run time costs registers that the row needs.)
template <typename T, int G, int GR, bool ON16, bool MASK, bool CLUSTER>
__global__ void __launch_bounds__(G <= kWarp ? kRowThreads : G, G <= kWarp ? 8 : GR > 8 || G == 1024 ? 1 : 1024 / G)
action_kernel(const ActionArgs p) {
  using P = Piece<T>;
  constexpr int E = P::E, ES = (int)sizeof(T);
  constexpr bool kLanes = G <= kWarp;
  constexpr int R = kLanes ? kRowThreads / G : 1;       // rows of a block at a time
  constexpr int NW = kLanes ? 1 : G / kWarp;
  constexpr int L = kLanes ? G : kWarp;
  __shared__ float4 entry[2][kLanes ? 1 : (CLUSTER ? kMaxCluster : 1) * NW];
  __shared__ RowShared shared;
  __shared__ float2 sum[kTerms][R];
  const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp;
  const int t = kLanes ? threadIdx.x % G : threadIdx.x;
  const uint32_t cn = CLUSTER ? cluster_size() : 1, cr = CLUSTER ? cluster_rank() : 0;
  const int64_t stride = (int64_t)(gridDim.x / cn) * R;
  const RowSums sums{&sum[0][kLanes ? threadIdx.x / G : 0], R};
  if (t == 0) {
    for (int i = 0; i < kTerms; ++i) sums.at[i * R] = make_float2(0.f, 0.f);
  }
  const uint8_t* mend = MASK && p.mask ? p.mask + (p.M - 1) * p.ldm + p.V : nullptr;
  const char* lfrom = static_cast<const char*>(p.l);
  const char* lto = lfrom + ((p.M - 1) * p.ld + p.V) * (int64_t)ES;
  if (cn > 1) {        // the other blocks' shared memory is there
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  }
  pdl_wait();
  // a block of a cluster takes a run of the row's pieces
  const int most = (p.V + E - 1) / E + (ON16 ? 0 : 1);
  const int chunk = kLanes ? most : (most + (int)cn - 1) / (int)cn, q0 = (int)cr * chunk + t;
  // where a row's pieces lie
  struct Place {
    const char* la;        // the row
    const char* lp;        // its first piece
    int off, nq;           // elements of another row in that; the end of the block's pieces
    int from, to;          // the pieces that lie wholly in the matrix (ON16: in the row)
    int last;              // the row's last piece
  };
  auto place = [&](int64_t row) {
    Place w;
    w.la = lfrom + row * p.ld * (int64_t)ES;
    w.off = ON16 ? 0 : (int)(reinterpret_cast<uintptr_t>(w.la) & 15) / ES;
    w.lp = w.la - w.off * ES;
    const int n = (w.off + p.V + E - 1) / E;
    w.last = n - 1;
    w.nq = kLanes ? n : min(n, ((int)cr + 1) * chunk);
    w.from = ON16 || w.lp >= lfrom ? 0 : 1;
    w.to = ON16 ? p.V / E : w.lp + (int64_t)n * 16 <= lto ? n : n - 1;
    return w;
  };
  auto row_of = [&](int64_t row0) { return min(kLanes ? row0 + threadIdx.x / G : row0, p.M - 1); };
  auto action_of = [&](int64_t row) {
    const int a = p.action ? p.action[row] : -1;
    return a < p.V ? a : -1;
  };
  // A row's pieces on their way to this thread's places in shared memory, while the
  // row before it is worked on.
  extern __shared__ uint4 ahead[];
  const uint32_t slot = ptx::smem_u32(&ahead[threadIdx.x]);
  constexpr int kSlots = kLanes ? kRowThreads : G;
  auto fetch = [&](const Place& w) {
    const int to = min(w.nq, w.to);
#pragma unroll
    for (int k = 0; k < GR; ++k) {
      const int q = q0 + k * G;
      if (q < to && (ON16 || q >= w.from)) fetch16(slot + k * kSlots * 16, w.lp + (int64_t)q * 16);
    }
  };
  const int64_t first = (int64_t)(blockIdx.x / cn) * R;
  int next_a = -1;
  if (first < p.M) {
    fetch(place(row_of(first)));
    next_a = action_of(row_of(first));
  }
  uint32_t par = 0;
  for (int64_t row0 = first; row0 < p.M; row0 += stride, par ^= 1) {
    const int64_t row = row_of(row0);
    const bool active = !kLanes || row0 + threadIdx.x / G < p.M;
    const Place at = place(row);
    const char* la = at.la;
    const int off = at.off, nq = at.nq;
    const uint8_t* mrow = MASK && p.mask ? p.mask + row * p.ldm : nullptr;
    // (no branch waits for these)
    RowInput in{next_a, 0.f, 0.f, 0.f, 0.f, 0.f, 1.f};
    float one_of = 0.f;      // blocks: a lane of the first warp holds one of the row's numbers
    if (!kLanes && warp == 0) {
      const float* from = lane == 1 ? p.old : lane == 2 ? p.adv : lane == 3 ? p.ref : lane == 4 ? p.weight : nullptr;
      if (lane == 0) {
        const int a = max(next_a, 0);
        one_of = (float)reinterpret_cast<const T*>(la)[a];
        if (mrow) one_of = mrow[a] ? one_of : -CUDART_INF_F;
      } else if (from) {
        one_of = from[row];
      } else if (lane == 4) {
        one_of = 1.f;
      }
    }
    if (kLanes) {
      const int a = max(in.a, 0);
      in.x = (float)reinterpret_cast<const T*>(la)[a];
      if (mrow) in.x = mrow[a] ? in.x : -CUDART_INF_F;
      if (p.dl) {
        in.old = p.old[row];
        in.adv = p.adv[row];
        if (p.ref) in.ref = p.ref[row];
        if (p.weight) in.w = p.weight[row];
      }
    }
    P x[GR];
    fetched();
#pragma unroll
    for (int k = 0; k < GR; ++k) {
      const int q = q0 + k * G;
      x[k].none();
      if (q < min(nq, at.to) && (ON16 || q >= at.from)) {
        const uint4 v = ahead[k * kSlots + threadIdx.x];
        x[k].w[0] = v.x;
        x[k].w[1] = v.y;
        x[k].w[2] = v.z;
        x[k].w[3] = v.w;
      } else if (q < nq) {
        const T* o = reinterpret_cast<const T*>(la);
#pragma unroll
        for (int i = 0; i < E; ++i) {
          const int j = q * E + i - off;
          if (j >= 0 && j < p.V) {
            if constexpr (ES == 2) {
              const uint32_t b = __bfloat16_as_ushort(o[j]);
              x[k].w[i / 2] = i & 1 ? (x[k].w[i / 2] & 0xffffu) | b << 16 : (x[k].w[i / 2] & 0xffff0000u) | b;
            } else {
              x[k].w[i] = __float_as_uint(o[j]);
            }
          }
        }
      }
    }
    if (MASK && mrow) {
      // the aligned words that hold the row's bytes, two for each piece: all lie in the mask,
      // or those of the first two and last two pieces may not
      const uint8_t* mb = mrow - off;
      const int sh = (int)(reinterpret_cast<uintptr_t>(mb) & (E - 1));
      mb -= sh;
      const bool all = mb >= p.mask && mb + (int64_t)(at.last + 2) * E <= mend;
#pragma unroll
      for (int k = 0; k < GR; ++k) {
        const int q = q0 + k * G;
        if (q >= nq) break;
        uint32_t v[E / 4];
        if (all || (q > 1 && q + 1 < at.last)) mask_words<E>(mb + q * E, sh, v);
        else mask_bytes<E>(mrow, q * E - off, p.V, v);
        cover(x[k], v);
      }
    }
    if constexpr (!ON16) {
#pragma unroll
      for (int k = 0; k < GR; ++k) {
        const int q = q0 + k * G;
        if (q == 0 || q == at.last) {
#pragma unroll
          for (int i = 0; i < E; ++i) {
            const int j = q * E + i - off;
            if (j < 0 || j >= p.V) x[k].drop(i);
          }
        }
      }
    }
    // statistics
    Stat st{-CUDART_INF_F, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < GR; ++k) st.m = fmaxf(st.m, x[k].max());
    // (the pieces are in registers)
    if (row0 + stride < p.M) {
      const int64_t next = row_of(row0 + stride);
      fetch(place(next));
      next_a = action_of(next);
      if (MASK && !kLanes && mrow && threadIdx.x == 0) {
        // this block's run of the next row's mask towards L2, in whole 16 bytes
        const uint8_t* m = p.mask + next * p.ldm;
        const uintptr_t a = (reinterpret_cast<uintptr_t>(m) + (int)cr * chunk * E + 15) & ~(uintptr_t)15;
        const uintptr_t z = (reinterpret_cast<uintptr_t>(m) + min(p.V, ((int)cr + 1) * chunk * E)) & ~(uintptr_t)15;
        if (a < z) ptx::bulk_prefetch_l2(reinterpret_cast<const void*>(a), (uint32_t)(z - a));
      }
    }
    st.m = lanes_max<L>(st.m);
    const float m0 = st.m;
    const bool wild = is_wild<T>(m0);
    float own = scaled(m0);      // own_base, of a wild warp after this
    if (wild) {
      own = own_base<T>(m0);
#pragma unroll
      for (int k = 0; k < GR; ++k) make_safe_wild(x[k], m0);
    } else {
#pragma unroll
      for (int k = 0; k < GR; ++k) make_safe(x[k]);
    }
    float2 s2 = make_float2(0.f, 0.f), t2 = make_float2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < GR; ++k) {
      if (q0 - t + k * G >= nq) break;       // (the same in all the row's threads)
#pragma unroll
      for (int i = 0; i < E / 2; ++i) {
        float2 u;
        const float2 e = exp_pair(x[k].pair(i), own, u);
        s2 = ptx::ffma2(e, make_float2(1.f, 1.f), s2);
        t2 = ptx::ffma2(e, u, t2);
      }
    }
    st.s = lanes_sum<L>(s2.x + s2.y);
    st.t = lanes_sum<L>(t2.x + t2.y);
    // the action's u as the row's pieces have it
    auto action_u = [&]() {
      const bool far = is_wild<T>(st.m);
      return fmaf(max_nan(far ? in.x - st.m : in.x, kLow), kLog2e, -own_base<T>(st.m));
    };
    RowTerms r;
    if constexpr (kLanes) {
      in.u = action_u();
      r = row_terms(p, row, st, in, t == 0 && active, sums);
    } else {
      // every warp's statistics to every block of the row; the first warp of each joins
      // them and finds the row's terms for its block
      if (lane < (int)cn) put_remote(ptx::smem_u32(&entry[par][cr * NW + warp]), lane, st.m, st.s, st.t);
      if (cn > 1) {
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
      } else {
        __syncthreads();
      }
      if (warp == 0) {
        // (read twice rather than kept: the row fills this warp's registers too)
        const int n = (int)cn * NW;
        float m = -CUDART_INF_F;
        for (int i = lane; i < n; i += kWarp) m = fmaxf(m, entry[par][i].x);
        st.m = lanes_max<kWarp>(m);
        float s = 0.f, w = 0.f;
        for (int i = lane; i < n; i += kWarp) {
          // A warp's sums, counted from its own maximum, by what its logits' u is off the
          // row's: as the gradient will have it.  (Nothing allowed there: they are 0, or NaN.)
          const float4 v = entry[par][i];
          const float d = v.x == -CUDART_INF_F ? 0.f : max_nan(own_base<T>(v.x) - base_for<T>(st.m, v.x), kLow);
          float f;
          asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(f) : "f"(d));
          s += f * v.y;
          w += f * fmaf(v.y, d, v.z);
        }
        st.s = lanes_sum<kWarp>(s);
        st.t = lanes_sum<kWarp>(w);
        in.x = __shfl_sync(0xffffffffu, one_of, 0);
        in.old = __shfl_sync(0xffffffffu, one_of, 1);
        in.adv = __shfl_sync(0xffffffffu, one_of, 2);
        in.ref = __shfl_sync(0xffffffffu, one_of, 3);
        in.w = __shfl_sync(0xffffffffu, one_of, 4);
        in.u = action_u();
        r = row_terms(p, row, st, in, lane == 0 && cr == 0, sums);
        if (lane == 0) shared = RowShared{r, st.m, in.u};
      }
      if (!p.dl) continue;       // (entry has two sets in turn)
      __syncthreads();
      r = shared.r;
      st.m = shared.m;
      in.u = shared.u;
    }
    if (!p.dl || !active) continue;
    // the gradient, over the logits' registers
    char* oa = static_cast<char*>(p.dl) + row * p.lddl * (int64_t)ES;
    T* o = reinterpret_cast<T*>(oa);
    const bool same = ON16 || (reinterpret_cast<uintptr_t>(oa) & 15) == (reinterpret_cast<uintptr_t>(la) & 15);
    // the pieces that are the row's alone
    const int whole0 = ON16 || off == 0 ? 0 : 1, whole1 = (off + p.V) / E;
    char* op = oa - off * ES;
    const float base = base_for<T>(st.m, m0);
    // sums that are not finite: what the mask covers is 0 all the same
    const bool odd = !r.kept || !(fabsf(r.a0) < CUDART_INF_F && fabsf(r.a1) < 1e7f);
#pragma unroll
    for (int k = 0; k < GR; ++k) {
      const int q = q0 + k * G;
      if (q >= nq) break;
      P g;
#pragma unroll
      for (int i = 0; i < E / 2; ++i) {
        float2 u;
        const float2 e = exp_pair(x[k].pair(i), base, u);
        g.put(i, ptx::fmul2(e, ptx::ffma2(u, make_float2(r.a1, r.a1), make_float2(r.a0, r.a0))));
      }
      if (odd) {
#pragma unroll
        for (int i = 0; i < E / 2; ++i) {
          const float2 l = x[k].pair(i);
          float2 v = g.pair(i);
          v.x = !r.kept || l.x <= 0.9f * kLow ? 0.f : v.x;
          v.y = !r.kept || l.y <= 0.9f * kLow ? 0.f : v.y;
          g.put(i, v);
        }
      }
      if (same && q < whole1 && (ON16 || q >= whole0)) {
        store16(op + (int64_t)q * 16, g.w);
      } else {
#pragma unroll
        for (int i = 0; i < E; ++i) {
          const int j = q * E - off + i;
          if (j < 0 || j >= p.V) continue;
          if constexpr (ES == 2) o[j] = __ushort_as_bfloat16((uint16_t)(g.w[i / 2] >> (16 * (i & 1))));
          else o[j] = __uint_as_float(g.w[i]);
        }
      }
    }
    // the action's own element, stored again by the thread that has stored its piece
    if (r.kept) {
      const int q = (in.a + off) / E;
      if (q < nq && q >= q0 && (q - q0) % G == 0) {
        float e;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(in.u));
        round_to(fmaf(e, fmaf(in.u, r.a1, r.a0), r.hot), o[in.a]);
      }
    }
  }
  if (!p.part) return;
  // the block's sums, in a fixed order: 16 threads to each of the terms (one thread that adds up to
  // 64 of them loses 10 x 2^-24 of equal ones)
  __syncthreads();
  if constexpr (kLanes) {
    constexpr int S = kRowThreads / kTerms;
    const int term = threadIdx.x / S, w0 = threadIdx.x % S;
    float2 v = make_float2(0.f, 0.f);
#pragma unroll
    for (int w = 0; w < R; w += S)
      if (w + w0 < R) v = join_kahan(v, sum[term][w + w0]);
    v = lanes_kahan(v, S);
    if (w0 == 0) p.part[(int64_t)term * gridDim.x + blockIdx.x] = v.x - v.y;
  } else if (threadIdx.x < kTerms) {
    const float2 v = sum[threadIdx.x][0];
    p.part[(int64_t)threadIdx.x * gridDim.x + blockIdx.x] = v.x - v.y;
  }
}

// d_stats from the blocks' sums, in a fixed order: four warps for each of them, all loads at once.
constexpr int kStatThreads = 128;
__global__ void __launch_bounds__(kTerms * kStatThreads)
action_stats_kernel(const float* __restrict__ part, int blocks, float* __restrict__ stats) {
  constexpr int kPer = (kMaxBlocks + kStatThreads - 1) / kStatThreads, kWarps = kStatThreads / kWarp;
  __shared__ float2 ws[kTerms][kWarps];
  pdl_wait();
  const int i = threadIdx.x / kStatThreads, t = threadIdx.x % kStatThreads;
  float x[kPer];
#pragma unroll
  for (int u = 0; u < kPer; ++u) x[u] = t + u * kStatThreads < blocks ? part[(int64_t)i * blocks + t + u * kStatThreads] : 0.f;
  float2 s = make_float2(0.f, 0.f);
#pragma unroll
  for (int u = 0; u < kPer; ++u) s = add_kahan(s, x[u]);
  s = lanes_kahan(s, kWarp);
  if (t % kWarp == 0) ws[i][t / kWarp] = s;
  __syncthreads();
  if (threadIdx.x >= kTerms * kWarps) return;
  s = lanes_kahan(ws[threadIdx.x / kWarps][threadIdx.x % kWarps], kWarps);
  if (threadIdx.x % kWarps == 0) stats[threadIdx.x / kWarps] = s.x - s.y;
}

// ---- launch ------------------------------------------------------------------------------
constexpr int kSms = 152;

template <typename T, int G, int GR, bool ON16, bool MASK, bool CLUSTER>
cudaError_t launch(const ActionArgs& p, int cn, float* stats, cudaStream_t st) {
  constexpr int R = G <= kWarp ? kRowThreads / G : 1, threads = G <= kWarp ? kRowThreads : G;
  // two blocks of 512 threads an SM, or as many threads in smaller ones
  constexpr int top = G <= kWarp ? kMaxBlocks : kSms * (GR > 8 ? 1 : 1024 / G);
  // a block's run of a row's pieces, as the kernel counts it: no plan leaves any of them out
  const int most = (p.V + Piece<T>::E - 1) / Piece<T>::E + (ON16 ? 0 : 1);
  if ((most + cn - 1) / cn > G * GR) return cudaErrorInvalidValue;
  const int64_t want = (p.M + R - 1) / R;
  const int blocks = (int)std::min<int64_t>(want, top / cn) * cn;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = threads * GR * 16;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cn;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cn > 1 ? 2 : 1;
  cudaError_t e;
  if constexpr (threads * GR * 16 > 48 * 1024) {
    static thread_local int prepared = -1;   // the device whose shared-memory opt-in is made
    int dev = 0;
    e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (prepared != dev) {
      e = cudaFuncSetAttribute(action_kernel<T, G, GR, ON16, MASK, CLUSTER>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               threads * GR * 16);
      if (e != cudaSuccess) return e;
      prepared = dev;
    }
  }
  e = cudaLaunchKernelEx(&cfg, action_kernel<T, G, GR, ON16, MASK, CLUSTER>, p);
  if (e != cudaSuccess || !stats) return e;
  return launch_pdl(action_stats_kernel, dim3(1), dim3(kTerms * kStatThreads), 0, st, (const float*)p.part, blocks, stats);
}
template <typename T, int G, int GR>
cudaError_t go(const ActionArgs& p, int cn, float* stats, cudaStream_t st) {
  constexpr int E = Piece<T>::E;
  auto on16 = [](const void* m, int64_t ld) { return al16(m) && ld % E == 0; };
  const bool whole = on16(p.l, p.ld) && on16(p.dl, p.dl ? p.lddl : 0);
  if constexpr (G >= 512) {
    if (cn > 1)
      return whole && !p.mask ? launch<T, G, GR, true, false, true>(p, cn, stats, st)
             : whole          ? launch<T, G, GR, true, true, true>(p, cn, stats, st)
             : !p.mask        ? launch<T, G, GR, false, false, true>(p, cn, stats, st)
                              : launch<T, G, GR, false, true, true>(p, cn, stats, st);
  }
  if constexpr (G > kWarp && GR <= 8) {
    if (!p.mask)
      return whole ? launch<T, G, GR, true, false, false>(p, 1, stats, st)
                   : launch<T, G, GR, false, false, false>(p, 1, stats, st);
  }
  if constexpr (GR <= 8)
    return whole ? launch<T, G, GR, true, true, false>(p, 1, stats, st)
                 : launch<T, G, GR, false, true, false>(p, 1, stats, st);
  return cudaErrorInvalidValue;      // (such rows take a cluster)
}

template <typename T>
cudaError_t run_rows(const ActionArgs& p, float* stats, cudaStream_t st) {
  constexpr int E = Piece<T>::E;
  // pieces of a row at most (the kernel for any rows counts one more than its longest has)
  const bool on16 = al16(p.l) && p.ld % E == 0 && al16(p.dl) && p.lddl % E == 0;
  const int64_t nq = (p.V + E - 1) / E + (on16 ? 0 : 1);
  // (many rows: fewer threads for each, so that a row's terms cost fewer warps.  65,536 x
  // 18 fp32 with a mask 13.4 us with four lanes, 10.3 with two; 4,096 x 18 4.2 and 4.7)
  if (nq <= 8 && p.M >= 16384) return go<T, 2, 4>(p, 1, stats, st);
  // Rows enough that fewer threads for each still fill the GPU (ten warps an SM): eight pieces
  // a thread.  (30,000 x 300 bf16 32 us with a warp a row, 18 with eight lanes; 100,000 x 100 29 and
  // 21; 8,000 x 700 14.6 and 11.9 with 16; but 2,000 x 700 6.9 and 9.3)
  if (nq > 8 && nq <= 128) {
    const int lanes = nq <= 16 ? 2 : nq <= 32 ? 4 : nq <= 64 ? 8 : 16;
    if (p.M * lanes >= 320 * kSms) {
      if (lanes == 2) return go<T, 2, 8>(p, 1, stats, st);
      if (lanes == 4) return go<T, 4, 8>(p, 1, stats, st);
      if (lanes == 8) return go<T, 8, 8>(p, 1, stats, st);
      return go<T, 16, 8>(p, 1, stats, st);
    }
  }
  if (nq <= 4) return go<T, 4, 1>(p, 1, stats, st);
  if (nq <= 8) return go<T, 4, 2>(p, 1, stats, st);
  if (nq <= 16) return go<T, 8, 2>(p, 1, stats, st);
  if (nq <= 32) return go<T, 8, 4>(p, 1, stats, st);
  if (nq <= 64) return go<T, 32, 2>(p, 1, stats, st);
  if (nq <= 128) return go<T, 32, 4>(p, 1, stats, st);
  if (nq <= 256) return go<T, 32, 8>(p, 1, stats, st);
  if (nq <= 512) return go<T, 128, 4>(p, 1, stats, st);
  // (a longest fp32 row off 16 bytes has a piece more than eight blocks of 8,192)
  if constexpr (sizeof(T) == 4) {
    if (nq > kMaxCluster * 8192)
      return p.mask ? launch<T, 1024, 9, false, true, true>(p, kMaxCluster, stats, st)
                    : launch<T, 1024, 9, false, false, true>(p, kMaxCluster, stats, st);
  }
  // few rows: more blocks for each, down to two pieces a thread
  const bool few = p.M < kSms;
  if (nq <= 1024 && !few) return go<T, 128, 8>(p, 1, stats, st);
  if (nq <= 2048 && !few) return go<T, 256, 8>(p, 1, stats, st);
  // Long rows, many of them: blocks of 1,024 threads, alone or in clusters of as few as hold
  // one.  (1,001 x 50,257 bf16 56 us with one and 66 with two of 512, 4,000 x 32,000 fp32 162
  // and 185, 4,096 x 131,072 434 with two and 672 with four of 512; but 8,192 x 32,768 255
  // with one of 1,024 and 183 with one of 512, which leave room for two rows an SM)
  if (nq > 4096 && !few) return go<T, 1024, 8>(p, nq <= 8192 ? 1 : nq <= 16384 ? 2 : nq <= 32768 ? 4 : 8, stats, st);
  int cn = 1;
  while (cn < kMaxCluster && (nq > 4096 * cn || (p.M * cn * 2 <= kSms && nq > 1024 * cn))) cn *= 2;
  return nq <= 4096 * cn ? go<T, 512, 8>(p, cn, stats, st) : go<T, 512, 16>(p, cn, stats, st);
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
constexpr size_t kActionWork = (size_t)kMaxBlocks * kTerms * sizeof(float);

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
  p.part = stats ? static_cast<float*>(work) : nullptr;
  return ops::status_of(run_any(dtype, p, stats, st));
}

}  // extern "C"
