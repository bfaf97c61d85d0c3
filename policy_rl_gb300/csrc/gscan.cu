// gscan.cu -- the gated linear recurrence of a MinGRU layer over T steps, and
// its backward pass.
//
//   z = sigmoid(pz),  a = 1 - z,  b = z ph,   h_t = a_t h_{t-1} + b_t,
// h_{t-1} taken as 0 where the state was cleared.  A step is the affine map
// (a, b); maps of consecutive steps compose, (a1, b1) then (a2, b2) is
// (a1 a2, a2 b1 + b2), so a channel's steps can be cut into blocks that are
// reduced to one map each, joined, and run again from their entering state.
// The backward recurrence g_t = dh_t + u_t, u_{t-1} = a_t g_t (0 where the
// state was cleared) has the same form from the other end, with the same a.
//
// Bound by memory (6 bytes per channel and step forward, 10 backward, in
// bf16), so an input is read from DRAM once: warps fetch their steps into
// shared memory two tiles ahead, reduce L steps of 32 channels (pairs) to maps
// in registers, and run the steps after the maps of the block's warps
// (consecutive steps of the same channels) were joined in shared memory.  A
// block of WT warps so covers a tile of L * WT steps and walks over tiles.
// The forward pass leaves the state that enters every 128th step for the
// backward pass, which walks the same tiles from the end and recomputes the
// states in between.  Three shapes of work:
//   - many channels, forward: a warp alone walks its channels, nothing to join;
//   - enough channels for every SM: a block walks along its channels' tiles;
//   - few channels and a long sequence ("split"): one launch reduces every tile
//     to its maps, a second joins them along the sequence, a third runs all
//     tiles at once from their entering states.  This reads the gates (and ph
//     or dh) twice, and leaves no tile waiting for another.  The maps lie in
//     rows of the output that the third launch overwrites.
// Measured, forward and backward, bf16: 128 x 2,048 x 256 72 us (5.6 TB/s) and
// 146 us (4.6 TB/s: limited by the instructions of the walk back, two blocks of
// 128 registers a thread on an SM); 65,537 x 1 x 1,024 151 and 214 us, of which
// the maps take 55, the join 14, the run 78 and 142.  Forward without a carry, in
// which a split pass keeps its tiles' entering states, it is walked by 16 blocks:
// 1,157 us.  A few hundred groups of channels are walked too, a block each, which
// leaves SMs idle and tiles one after another: 1,023 x 37 x 129 fp32 30 and 44 us (0.8
// and 1.3 TB/s).
// Compositions happen in an order fixed by the sizes: results are
// deterministic.  A cleared state is dropped by a select, never multiplied by
// 0, so that infinities and NaN do not cross it.  Within an episode an infinite
// state stays infinite or becomes NaN (where the product of a block's 1 - z has
// left fp32's range).
#include <algorithm>
#include <type_traits>

#include "ops.cuh"
#include "tc_ptx.cuh"

namespace ppo {
namespace {

using namespace ops;

// Rows (t * N + n) and row pitches in bytes fit 32 bits, so that an address is one
// wide multiplication.
struct ScanArgs {
  const void *p, *dh;
  uint32_t ldp, lddh, ldo; // bytes
  const float *done, *done0, *h0, *dhT;
  int T, N, H;
  int64_t C;               // N * H channels
  void* out;               // h, or dp
  float *last;             // hT, or dh0 (nullable)
  float* carry;            // [ceil(T / 128)][C]: written (nullable), or read
  int groups;              // of channels, one block each
  int whole;               // a warp's channels always belong to one environment
  unsigned div_m;          // c / H = c * div_m >> div_s for c < 2^31
  int div_s;
  int wide;                // rows are read in 16-byte pieces
  int split;               // tiles start from stored entering states (see above)
};

// V channels at once; pairs go through the packed fp32 instructions (each half
// rounded as the scalar instruction would).
template <int V>
__device__ __forceinline__ void vfma(const float (&a)[V], const float (&b)[V], const float (&c)[V],
                                     float (&o)[V]) {
  if constexpr (V == 2) {
    const float2 r = ptx::ffma2(make_float2(a[0], a[1]), make_float2(b[0], b[1]),
                                make_float2(c[0], c[1]));
    o[0] = r.x;
    o[1] = r.y;
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) o[v] = fmaf(a[v], b[v], c[v]);
  }
}
template <int V>
__device__ __forceinline__ void vmul(const float (&a)[V], const float (&b)[V], float (&o)[V]) {
  if constexpr (V == 2) {
    const float2 r = ptx::fmul2(make_float2(a[0], a[1]), make_float2(b[0], b[1]));
    o[0] = r.x;
    o[1] = r.y;
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) o[v] = a[v] * b[v];
  }
}
template <int V>
__device__ __forceinline__ void vset(float (&o)[V], float x) {
#pragma unroll
  for (int v = 0; v < V; ++v) o[v] = x;
}
template <int V>
__device__ __forceinline__ void one_minus(const float (&z)[V], float (&a)[V]) {
  float m[V], one[V];
  vset<V>(m, -1.f);
  vset<V>(one, 1.f);
  vfma<V>(z, m, one, a);
}
// z = 1 / (1 + 2^(-x log2 e)): the power is inf below -88, its reciprocal 0.  Both
// types use the hardware's power and reciprocal, 2^-22 and 2^-23 of their values,
// with |x| 2^-24 from the rounded product: z is off by less than 1e-6 of itself for
// |x| < 10, where 1 - z in fp32 is off by as much as 6e-8 whatever z's error.
template <int V>
__device__ __forceinline__ void sigmoid(const float (&x)[V], float (&z)[V]) {
  float k[V], one[V], e[V];
  vset<V>(k, -1.4426950408889634f);
  vset<V>(one, 1.f);
  vmul<V>(x, k, e);
#pragma unroll
  for (int v = 0; v < V; ++v) asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e[v]) : "f"(e[v]));
  vfma<V>(e, one, one, e);
#pragma unroll
  for (int v = 0; v < V; ++v) asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(z[v]) : "f"(e[v]));
}

// The affine map of a block of steps.  a < 0 stands for "the state was cleared
// inside": what enters does not matter (products of 1 - z are never negative).
__device__ __forceinline__ float apply(float a, float b, float h) {
  return a < 0.f ? b : fmaf(a, h, b);
}
__device__ __forceinline__ float joined(float a1, float a2) {
  return a1 < 0.f || a2 < 0.f ? -1.f : a1 * a2;
}

// Keeps a row step out of the compiler's reach, so that it does not carry its
// multiples from tile to tile in registers (measured with 16 steps: 128
// registers and 500 to 1,200 bytes of spills a thread).
__device__ __forceinline__ int64_t opaque(int64_t v) {
  asm volatile("" : "+l"(v));
  return v;
}
// Where the state entering a step is cleared (steps outside [0, T): nowhere).
__device__ __forceinline__ float reset_flag(const ScanArgs& s, int t, int n) {
  if (t < 0 || t >= s.T) return 0.f;
  if (t == 0) return s.done0 ? __ldg(s.done0 + n) : 0.f;
  return s.done ? __ldg(s.done + ((unsigned)(t - 1) * (unsigned)s.N + (unsigned)n)) : 0.f;
}
// element j of row t * N + n of a matrix of pitch ld bytes
template <typename T>
__device__ __forceinline__ T* element(const ScanArgs& s, const void* base, uint32_t ld, int t, int n,
                                      int j) {
  const uint32_t row = (uint32_t)t * (uint32_t)s.N + (uint32_t)n;
  return reinterpret_cast<T*>(reinterpret_cast<char*>(const_cast<void*>(base)) + (uint64_t)row * ld) +
         j;
}
// rows of one step, in bytes
__device__ __forceinline__ int64_t step_of(const ScanArgs& s, uint32_t ld) {
  return opaque((int64_t)((uint64_t)(uint32_t)s.N * ld));
}

// A channel's environment and its place within it.
struct Channel {
  int n, j;
};
__device__ __forceinline__ Channel channel(const ScanArgs& s, unsigned c) {
  const unsigned n = (unsigned)((uint64_t)c * s.div_m >> s.div_s);
  return {(int)n, (int)(c - n * (unsigned)s.H)};
}
// A lane's channels: V consecutive ones of one environment.
struct Place {
  unsigned c;
  int n, j;
  bool ok, two;   // two: the warp's channels belong to environment n0 or n0 and n1
  int n0, n1;
};
template <int V>
__device__ __forceinline__ Place place_of(const ScanArgs& s, int group, int lane) {
  Place p;
  const unsigned first = (unsigned)group * kWarp * V, C = (unsigned)s.C;
  p.c = first + lane * V;
  p.ok = p.c < C;
  const Channel x0 = channel(s, first < C ? first : 0);
  p.n0 = p.n1 = p.n = x0.n;
  p.two = true;
  p.j = x0.j + lane * V;
  if (s.whole) return p;
  const Channel x = channel(s, p.ok ? p.c : 0);
  const unsigned lastc = first + kWarp * V <= C ? first + kWarp * V - 1 : C - 1;
  p.n1 = first < C ? channel(s, lastc).n : x0.n;
  p.two = p.n1 - p.n0 <= 1;
  if (p.ok) p.n = x.n;   // lanes past the end read flags of n0
  p.j = x.j;
  return p;
}

// Bit i: the state entering step t0 + i is cleared.  Where the warp's channels
// belong to two environments at most, lanes i and L + i have loaded their flags
// of step i beforehand (1,023 x 37 x 129 fp32, where a quarter of the warps
// straddles two: 30 and 44 us; 46 and 60 with every lane's flags loaded here).
template <int L>
__device__ __forceinline__ float load_flag(const ScanArgs& s, int t0, const Place& pl, int lane) {
  if (L == 1 || !pl.two || lane >= 2 * L) return 0.f;
  return lane < L ? reset_flag(s, t0 + lane, pl.n0) : reset_flag(s, t0 + lane - L, pl.n1);
}
template <int L>
__device__ __forceinline__ uint32_t reset_mask(const ScanArgs& s, float mine, int t0,
                                               const Place& pl) {
  static_assert(2 * L <= kWarp, "a lane for each step and environment");
  if (L > 1 && pl.two) {
    const uint32_t all = __ballot_sync(0xffffffffu, mine != 0.f);
    return (pl.n == pl.n0 ? all : all >> L) & ((1u << L) - 1);
  }
  uint32_t m = 0;
  if (pl.ok) {
#pragma unroll
    for (int i = 0; i < L; ++i) m |= reset_flag(s, t0 + i, pl.n) != 0.f ? 1u << i : 0u;
  }
  return m;
}

// The steps of a thread's block of L in [t0, T): their count.
template <int L>
__device__ __forceinline__ int steps_in(int t0, int T) { return min(max(T - t0, 0), L); }

// One input's L steps of a warp: 2-byte elements in registers ..
template <typename T, int V, int L>
struct RegColumn {
  Raw<T, V> r[L];
  __device__ __forceinline__ void load(const ScanArgs& s, const void* base, uint32_t ld, int off,
                                       int t0, int n, const Place& pl, int) {
    const int64_t step = step_of(s, ld);
    const char* p = element<const char>(s, base, ld, t0, pl.n, (pl.j + off) * (int)sizeof(T));
#pragma unroll
    for (int i = 0; i < L; ++i) {
      r[i] = pl.ok && i < n ? __ldg(reinterpret_cast<const Raw<T, V>*>(p)) : Raw<T, V>{};
      p += step;
    }
  }
  __device__ __forceinline__ void get(int i, int, float (&f)[V]) const { to_f32<T, V>(r[i], f); }
};
// .. others in the warp's [L][32] words of shared memory, filled asynchronously
// two tiles ahead (steps past n keep what was there): in 16-byte pieces, eight
// of a row, where the rows are so aligned, else word by word.
template <typename T, int V, int L>
struct SharedColumn {
  uint32_t* w;
  __device__ __forceinline__ void load(const ScanArgs& s, const void* base, uint32_t ld, int off,
                                       int t0, int n, const Place& pl, int lane) const {
    const int64_t step = step_of(s, ld);
    if (s.wide) {
      const int r0 = lane >> 3, back = (lane & 7) * (16 / (int)sizeof(T)) - lane * V;
      const unsigned c = pl.c + back;      // the piece's first channel
      const bool ok = c < (unsigned)s.C;
      Channel x{pl.n, pl.j + back};
      if (!s.whole) x = channel(s, ok ? c : 0);
      const char* p = element<const char>(s, base, ld, t0 + r0, x.n, (x.j + off) * (int)sizeof(T));
      uint32_t dst = ptx::smem_u32(w) + r0 * 128 + (lane & 7) * 16;
#pragma unroll
      for (int i = 0; i < L; i += 4) {
        if (ok && r0 + i < n)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + i * 128), "l"(p)
                       : "memory");
        p += 4 * step;
      }
    } else {
      const char* p = element<const char>(s, base, ld, t0, pl.n, (pl.j + off) * (int)sizeof(T));
      const uint32_t dst = ptx::smem_u32(w) + lane * 4;
#pragma unroll
      for (int i = 0; i < L; ++i) {
        if (pl.ok && i < n)
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst + i * 128), "l"(p)
                       : "memory");
        p += step;
      }
    }
  }
  __device__ __forceinline__ void get(int i, int lane, float (&f)[V]) const {
    static_assert(sizeof(Raw<T, V>) == 4, "one word");
    const uint32_t x = w[i * kWarp + lane];
    Raw<T, V> r;
    memcpy(&r, &x, 4);
    to_f32<T, V>(r, f);
  }
};
template <typename T, int V> constexpr bool kFetch = sizeof(T) * V == 4;
constexpr int kStages = 2;   // tiles on their way
__device__ __forceinline__ void fetch_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int STAGES>
__device__ __forceinline__ void fetch_wait() {   // all but the newest STAGES - 1 groups
  asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 1) : "memory");
}
// what lane i has read of step i's flag, kept with the tile it belongs to
template <int N>
struct Flags {
  float f[N];
  __device__ __forceinline__ float get(int k) const {
    float v = f[0];
#pragma unroll
    for (int i = 1; i < N; ++i) v = k == i ? f[i] : v;
    return v;
  }
  __device__ __forceinline__ void set(int k, float v) {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = k == i ? v : f[i];
  }
};

// ---- steps in registers ----------------------------------------------------------
// PLAIN: all L steps exist and none clears a state.
template <int V, int L, bool PLAIN, typename Col>
__device__ __forceinline__ void block_map(const float (&z)[L][V], const Col& rh, int n,
                                          uint32_t clear, int lane, float (&ma)[V],
                                          float (&mb)[V]) {
  vset<V>(ma, 1.f);
  vset<V>(mb, 0.f);
#pragma unroll
  for (int i = 0; i < L; ++i) {
    float c[V], a[V], b[V];
    rh.get(i, lane, c);
    if (PLAIN || i < n) {
      one_minus<V>(z[i], a);
      vmul<V>(z[i], c, b);
      if (!PLAIN && ((clear >> i) & 1u)) vset<V>(mb, 0.f);
      vfma<V>(a, mb, b, mb);
      vmul<V>(ma, a, ma);
    }
  }
  if (!PLAIN && clear) vset<V>(ma, -1.f);
}

// The steps themselves, from the entering state h to the last one.
template <typename T, int V, int L, bool PLAIN, typename Col>
__device__ __forceinline__ void run_steps(const float (&z)[L][V], const Col& rh, int n,
                                          uint32_t clear, int lane, bool ok, float (&h)[V], T* o,
                                          int64_t ostep) {
#pragma unroll
  for (int i = 0; i < L; ++i) {
    float c[V], a[V], b[V];
    rh.get(i, lane, c);
    if (PLAIN || i < n) {
      one_minus<V>(z[i], a);
      vmul<V>(z[i], c, b);
      if (!PLAIN && ((clear >> i) & 1u)) vset<V>(h, 0.f);
      vfma<V>(a, h, b, h);
      if (ok) *reinterpret_cast<Raw<T, V>*>(o) = from_f32<T, V>(h);
    }
    o = reinterpret_cast<T*>(reinterpret_cast<char*>(o) + ostep);
  }
}

// What n steps pass back from their own dh, in reverse order (and, with MAP,
// the factor of what reaches them from later steps).
template <int V, int L, bool PLAIN, bool MAP, typename Col>
__device__ __forceinline__ void block_back(const float (&z)[L][V], const Col& rg, int n,
                                           uint32_t clear, int lane, float (&ma)[V],
                                           float (&g)[V]) {
  vset<V>(g, 0.f);
  if (MAP) vset<V>(ma, 1.f);
  float one[V];
  vset<V>(one, 1.f);
#pragma unroll
  for (int i = L - 1; i >= 0; --i) {
    float d[V], a[V];
    rg.get(i, lane, d);
    if (PLAIN || i < n) {
      one_minus<V>(z[i], a);
      vfma<V>(d, one, g, g);
      vmul<V>(a, g, g);
      if (MAP) vmul<V>(ma, a, ma);
      if (!PLAIN && ((clear >> i) & 1u)) vset<V>(g, 0.f);
    }
  }
  if (MAP && !PLAIN && clear) vset<V>(ma, -1.f);
}

// The steps from the last to the first, given the state h entering the first
// and u, what reaches the last state from later steps.
template <typename T, int V, int L, bool PLAIN, typename Col>
__device__ __forceinline__ void run_back(const float (&z)[L][V], const Col& rh, const Col& rg,
                                         int n, uint32_t clear, int lane, bool ok, float (&h)[V],
                                         float (&u)[V], T* o, int64_t ostep, int H) {
  float w[L][V];   // dpz / g of each step
  float one[V], minus[V];
  vset<V>(one, 1.f);
  vset<V>(minus, -1.f);
#pragma unroll
  for (int i = 0; i < L; ++i) {
    float c[V], a[V], k[V];
    rh.get(i, lane, c);
    if (!PLAIN && ((clear >> i) & 1u)) vset<V>(h, 0.f);
    one_minus<V>(z[i], a);
    vmul<V>(z[i], a, k);
    vfma<V>(h, minus, c, w[i]);
    vmul<V>(w[i], k, w[i]);
    vmul<V>(z[i], c, k);
    vfma<V>(a, h, k, h);
  }
  o = reinterpret_cast<T*>(reinterpret_cast<char*>(o) + (L - 1) * ostep);
#pragma unroll
  for (int i = L - 1; i >= 0; --i) {
    float d[V], dz[V], dc[V], a[V];
    rg.get(i, lane, d);
    if (PLAIN || i < n) {
      vfma<V>(d, one, u, d);
      vmul<V>(d, z[i], dc);
      vmul<V>(d, w[i], dz);
      one_minus<V>(z[i], a);
      vmul<V>(a, d, u);
      if (!PLAIN && ((clear >> i) & 1u)) vset<V>(u, 0.f);
      if (ok) {
        *reinterpret_cast<Raw<T, V>*>(o) = from_f32<T, V>(dz);
        *reinterpret_cast<Raw<T, V>*>(o + H) = from_f32<T, V>(dc);
      }
    }
    o = reinterpret_cast<T*>(reinterpret_cast<char*>(o) - ostep);
  }
}

// ---- maps kept in the output's rows (split) -----------------------------------------
// Value k (0, 1, 2) of a tile and channel: fp32 outputs hold it in the tile's
// row k, bf16 outputs its upper and lower halves in rows 2k and 2k + 1.  (dp
// uses its pz columns.)
template <typename T>
__device__ __forceinline__ T* below(T* row, int64_t step, int k) {
  return reinterpret_cast<T*>(reinterpret_cast<char*>(row) + k * step);
}
template <typename T>
__device__ __forceinline__ void put_value(T* row, int64_t step, int k, float v) {
  if constexpr (sizeof(T) == 4) {
    *below(row, step, k) = v;
  } else {
    const uint32_t u = __float_as_uint(v);
    *below(row, step, 2 * k) = __ushort_as_bfloat16((uint16_t)(u >> 16));
    *below(row, step, 2 * k + 1) = __ushort_as_bfloat16((uint16_t)u);
  }
}
template <typename T>
__device__ __forceinline__ float get_value(T* row, int64_t step, int k) {
  if constexpr (sizeof(T) == 4) {
    return *below(row, step, k);
  } else {
    const uint32_t hi = __bfloat16_as_ushort(*below(row, step, 2 * k));
    return __uint_as_float(hi << 16 | __bfloat16_as_ushort(*below(row, step, 2 * k + 1)));
  }
}
// rows that values 0..k need
template <typename T>
__host__ __device__ constexpr int value_rows(int k) { return sizeof(T) == 4 ? k + 1 : 2 * k + 2; }

// ---- the kernels ----------------------------------------------------------------------
// A block's walk over (group of channels, tile) pairs, tiles fastest.
struct Walk {
  int group, tile;
};

enum Phase : int { kWhole = 0, kMaps = 1 };

// Threads of an SM that the registers of L steps leave room for (65,537 x 1 x
// 1,024 bf16: forward 95 us with 512, 79 with 768; its maps 64 and 56; backward
// 142 with 512, 249 with 768, which spills).
__host__ __device__ constexpr int threads_per_sm(int L, int phase, bool backward) {
  return L <= 8 ? 1024 : phase == kMaps ? 768 : backward ? 512 : 768;
}

// WT warps along time, WC along channels.  PHASE kMaps writes each tile's map
// and runs nothing.
template <typename T, int V, int L, int WT, int WC, int PHASE>
__global__ void __launch_bounds__(WT* WC* kWarp, L > 1 ? threads_per_sm(L, PHASE, false) / (WT * WC * kWarp) : 1)
scan_fwd_kernel(const ScanArgs s) {
  constexpr int CH = WC * kWarp * V, NT = WT * WC * kWarp;
  __shared__ float sa[WT > 1 ? WT : 1][WT > 1 ? CH : 1], sb[WT > 1 ? WT : 1][WT > 1 ? CH : 1];
  constexpr bool FETCH = L > 1 && kFetch<T, V>;
  extern __shared__ __align__(128) uint32_t ring[];   // FETCH: [kStages][pz, ph][warp][L][32]
  const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp;
  const int wt = warp % WT, wc = warp / WT;
  const int tiles = (s.T + L * WT - 1) / (L * WT), groups = s.groups;
  // units: the pairs of a block, dealt out round by round; unsplit, a group's
  // tiles stay with one block
  const int first = s.split ? blockIdx.x / groups : 0;
  using Col = std::conditional_t<FETCH, SharedColumn<T, V, L>, RegColumn<T, V, L>>;
  auto column = [&](int stage, int k) {
    if constexpr (FETCH) return Col{ring + ((stage * 2 + k) * (WT * WC) + warp) * (L * kWarp)};
    else return Col{};
  };
  auto place = [&](int group) { return place_of<V>(s, group * WC + wc, lane); };
  auto load = [&](const Place& pl, int tile, Col& cz, Col& ch, float& flag) {
    const int t0 = (tile * WT + wt) * L;
    const int n = steps_in<L>(t0, s.T);
    cz.load(s, s.p, s.ldp, 0, t0, n, pl, lane);
    ch.load(s, s.p, s.ldp, s.H, t0, n, pl, lane);
    flag = load_flag<L>(s, t0, pl, lane);
  };
  const int stride = s.split ? gridDim.x / groups : 1;   // tiles from one to the next
  Walk at{(int)(s.split ? blockIdx.x % groups : blockIdx.x), first}, ahead = at;
  auto more = [&](const Walk& w) { return s.split ? w.tile < tiles : w.group < groups; };
  auto advance = [&](Walk& w) {
    w.tile += stride;
    if (!s.split && w.tile >= tiles) {
      w.tile = 0;
      w.group += gridDim.x;
    }
  };
  // the maps are made from the last tile on, so that the run that follows finds
  // the first ones' inputs in L2
  auto tile_of = [&](const Walk& w) { return PHASE == kMaps ? tiles - 1 - w.tile : w.tile; };
  Flags<kStages> flags{};
  if constexpr (FETCH) {
#pragma unroll
    for (int i = 0; i < kStages; ++i) {
      Col cz = column(i, 0), ch = column(i, 1);
      if (more(ahead)) {
        load(place(ahead.group), tile_of(ahead), cz, ch, flags.f[i]);
        advance(ahead);
      }
      fetch_commit();
    }
  }
  // the running state: each thread's own (WT == 1), or that of the channel
  // thread x joins (block channel x, below CH)
  float h[V];
  float hj[(CH + NT - 1) / NT];
  int stage = 0;
  while (more(at)) {
    const Place pl = place(at.group);
    const int tile = tile_of(at);
    const int t0 = (tile * WT + wt) * L;
    const int n = steps_in<L>(t0, s.T);
    const int64_t ostep = step_of(s, s.ldo);
    T* out = element<T>(s, s.out, s.ldo, t0, pl.n, pl.j);
    if constexpr (PHASE == kWhole) {
      if (tile == 0 || s.split) {
        // (split, not h0 itself, which the last tile's block may be replacing)
        const float* from = s.split ? s.carry + (int64_t)tile * s.C : s.h0;
        if constexpr (WT == 1) {
#pragma unroll
          for (int v = 0; v < V; ++v) h[v] = pl.ok && from ? from[pl.c + v] : 0.f;
        } else {
#pragma unroll
          for (int k = 0; k < (CH + NT - 1) / NT; ++k) {
            const int x = threadIdx.x + k * NT;
            const unsigned c = (unsigned)at.group * CH + x;
            hj[k] = x < CH && c < s.C && from ? from[c] : 0.f;
          }
        }
      }
    }
    Col cz = column(stage, 0), rh = column(stage, 1);
    float flag;
    if constexpr (FETCH) {
      fetch_wait<kStages>();
      __syncwarp();   // pieces that other lanes fetched
      flag = flags.get(stage);
    } else {
      load(pl, tile, cz, rh, flag);
    }
    float z[L][V];
#pragma unroll
    for (int i = 0; i < L; ++i) {
      cz.get(i, lane, z[i]);
      sigmoid<V>(z[i], z[i]);
    }
    const uint32_t clear = reset_mask<L>(s, flag, t0, pl);
    const bool plain = __all_sync(0xffffffffu, n == L && clear == 0);
    float hin[V];   // the state entering this thread's steps
    if constexpr (WT > 1) {
      float ma[V], mb[V];
      if (plain) block_map<V, L, true>(z, rh, n, clear, lane, ma, mb);
      else block_map<V, L, false>(z, rh, n, clear, lane, ma, mb);
      const int x0 = (wc * kWarp + lane) * V;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        sa[wt][x0 + v] = ma[v];
        sb[wt][x0 + v] = mb[v];
      }
      __syncthreads();
      // a channel's thread replaces each block's map by the state entering it
#pragma unroll
      for (int k = 0; k < (CH + NT - 1) / NT; ++k) {
        const int x = threadIdx.x + k * NT;
        if (x < CH) {
          if constexpr (PHASE == kWhole) {
#pragma unroll
            for (int w = 0; w < WT; ++w) {
              const float a = sa[w][x], b = sb[w][x];
              sb[w][x] = hj[k];
              hj[k] = apply(a, b, hj[k]);
            }
          } else {
            float a = 1.f, b = 0.f;
#pragma unroll
            for (int w = 0; w < WT; ++w) {
              b = apply(sa[w][x], sb[w][x], b);
              a = joined(a, sa[w][x]);
            }
            const unsigned c = (unsigned)at.group * CH + x;
            if (c < s.C && tile < tiles - 1) {   // (the last one's is not needed)
              const Channel e = channel(s, c);
              T* row = element<T>(s, s.out, s.ldo, tile * (L * WT), e.n, e.j);
              put_value<T>(row, ostep, 0, a);
              put_value<T>(row, ostep, 1, b);
            }
          }
        }
      }
      __syncthreads();
#pragma unroll
      for (int v = 0; v < V; ++v) hin[v] = sb[wt][x0 + v];
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) hin[v] = h[v];
    }
    if constexpr (PHASE == kWhole) {
      if (s.carry && !s.split && pl.ok && n > 0 && t0 % PPO_SCAN_BLOCK == 0) {
#pragma unroll
        for (int v = 0; v < V; ++v)
          s.carry[(int64_t)(t0 / PPO_SCAN_BLOCK) * s.C + pl.c + v] = clear & 1u ? 0.f : hin[v];
      }
      if (plain) run_steps<T, V, L, true>(z, rh, n, clear, lane, pl.ok, hin, out, ostep);
      else run_steps<T, V, L, false>(z, rh, n, clear, lane, pl.ok, hin, out, ostep);
      // the thread of the last step has the last state
      if (s.last && pl.ok && n > 0 && t0 + n == s.T) {
#pragma unroll
        for (int v = 0; v < V; ++v) s.last[pl.c + v] = hin[v];
      }
      if constexpr (WT == 1) {
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = hin[v];
      }
    }
    if constexpr (FETCH) {
      __syncwarp();   // the warp has read its words: they may be refilled
      if (more(ahead)) {
        float f;
        load(place(ahead.group), tile_of(ahead), cz, rh, f);
        flags.set(stage, f);
        advance(ahead);
      }
      fetch_commit();
      stage = stage == kStages - 1 ? 0 : stage + 1;
    }
    advance(at);
  }
}

// A tile of fewer than PPO_SCAN_BLOCK steps has to hold the whole sequence.
template <typename T, int V, int L, int WT, int WC, int PHASE>
__global__ void __launch_bounds__(WT* WC* kWarp, L > 1 ? threads_per_sm(L, PHASE, true) / (WT * WC * kWarp) : 1)
scan_bwd_kernel(const ScanArgs s) {
  constexpr int CH = WC * kWarp * V, NT = WT * WC * kWarp;
  // maps of the blocks of steps (factor, state), and what they pass back
  __shared__ float sa[WT > 1 ? WT : 1][WT > 1 ? CH : 1], sb[WT > 1 ? WT : 1][WT > 1 ? CH : 1],
      sg[WT > 1 ? WT : 1][WT > 1 ? CH : 1];
  constexpr bool FETCH = L > 1 && kFetch<T, V>;
  constexpr int IN = PHASE == kMaps ? 2 : 3;
  extern __shared__ __align__(128) uint32_t ring[];   // FETCH: [kStages][pz, dh (, ph)][warp][L][32]
  const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp;
  const int wt = warp % WT, wc = warp / WT;
  const int tiles = (s.T + L * WT - 1) / (L * WT), groups = s.groups;
  using Col = std::conditional_t<FETCH, SharedColumn<T, V, L>, RegColumn<T, V, L>>;
  auto column = [&](int stage, int k) {
    if constexpr (FETCH) return Col{ring + ((stage * IN + k) * (WT * WC) + warp) * (L * kWarp)};
    else return Col{};
  };
  auto place = [&](int group) { return place_of<V>(s, group * WC + wc, lane); };
  auto load = [&](const Place& pl, int tile, Col& cz, Col& cd, Col& ch, float& flag) {
    const int t0 = (tile * WT + wt) * L;
    const int n = steps_in<L>(t0, s.T);
    cz.load(s, s.p, s.ldp, 0, t0, n, pl, lane);
    cd.load(s, s.dh, s.lddh, 0, t0, n, pl, lane);
    if constexpr (PHASE == kWhole) ch.load(s, s.p, s.ldp, s.H, t0, n, pl, lane);
    flag = load_flag<L>(s, t0, pl, lane);
  };
  // tiles run from the last to the first
  const int stride = s.split ? gridDim.x / groups : 1;
  Walk at{(int)(s.split ? blockIdx.x % groups : blockIdx.x),
          tiles - 1 - (int)(s.split ? blockIdx.x / groups : 0)},
      ahead = at;
  auto more = [&](const Walk& w) { return s.split ? w.tile >= 0 : w.group < groups; };
  auto advance = [&](Walk& w) {
    w.tile -= stride;
    if (!s.split && w.tile < 0) {
      w.tile = tiles - 1;
      w.group += gridDim.x;
    }
  };
  // (the maps from the first tile on: the run finds the last ones in L2)
  auto tile_of = [&](const Walk& w) { return PHASE == kMaps ? tiles - 1 - w.tile : w.tile; };
  Flags<kStages> flags{};
  if constexpr (FETCH) {
#pragma unroll
    for (int i = 0; i < kStages; ++i) {
      Col a = column(i, 0), b = column(i, 1), c = column(i, IN - 1);
      if (more(ahead)) {
        load(place(ahead.group), tile_of(ahead), a, b, c, flags.f[i]);
        advance(ahead);
      }
      fetch_commit();
    }
  }
  float u[V];
  float uj[(CH + NT - 1) / NT], hj[(CH + NT - 1) / NT];
  int stage = 0;
  while (more(at)) {
    const Place pl = place(at.group);
    const int tile = tile_of(at);
    const int t0 = (tile * WT + wt) * L;
    const int n = steps_in<L>(t0, s.T);
    const int64_t ostep = step_of(s, s.ldo);
    T* out = element<T>(s, s.out, s.ldo, t0, pl.n, pl.j);
    float hin[V], uin[V];   // the state entering this thread's steps, what reaches the last of them
    if constexpr (PHASE == kWhole) {
      const float* from = s.carry + ((int64_t)tile * L * WT / PPO_SCAN_BLOCK) * s.C;
      if constexpr (WT == 1) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
          hin[v] = pl.ok ? __ldg(from + pl.c + v) : 0.f;
          if (tile == tiles - 1) u[v] = pl.ok && s.dhT ? s.dhT[pl.c + v] : 0.f;
        }
      } else {
#pragma unroll
        for (int k = 0; k < (CH + NT - 1) / NT; ++k) {
          const int x = threadIdx.x + k * NT;
          const unsigned c = (unsigned)at.group * CH + x;
          const bool in = x < CH && c < s.C;
          hj[k] = in ? __ldg(from + c) : 0.f;
          if (tile == tiles - 1) {
            uj[k] = in && s.dhT ? s.dhT[c] : 0.f;
          } else if (s.split && in) {
            const Channel e = channel(s, c);
            uj[k] = get_value<T>(element<T>(s, s.out, s.ldo, tile * (L * WT), e.n, e.j), ostep, 2);
          }
        }
      }
    }
    Col cz = column(stage, 0), rg = column(stage, 1), rh = column(stage, IN - 1);
    float flag;
    if constexpr (FETCH) {
      fetch_wait<kStages>();
      __syncwarp();
      flag = flags.get(stage);
    } else {
      load(pl, tile, cz, rg, rh, flag);
    }
    float z[L][V];
#pragma unroll
    for (int i = 0; i < L; ++i) {
      cz.get(i, lane, z[i]);
      sigmoid<V>(z[i], z[i]);
    }
    const uint32_t clear = reset_mask<L>(s, flag, t0, pl);
    const bool plain = __all_sync(0xffffffffu, n == L && clear == 0);
    if constexpr (WT > 1) {
      const int x0 = (wc * kWarp + lane) * V;
      float ma[V], mb[V], g[V];
      if constexpr (PHASE == kWhole) {
        if (plain) {
          block_map<V, L, true>(z, rh, n, clear, lane, ma, mb);
          block_back<V, L, true, false>(z, rg, n, clear, lane, ma, g);
        } else {
          block_map<V, L, false>(z, rh, n, clear, lane, ma, mb);
          block_back<V, L, false, false>(z, rg, n, clear, lane, ma, g);
        }
#pragma unroll
        for (int v = 0; v < V; ++v) sb[wt][x0 + v] = mb[v];
      } else {
        if (plain) block_back<V, L, true, true>(z, rg, n, clear, lane, ma, g);
        else block_back<V, L, false, true>(z, rg, n, clear, lane, ma, g);
      }
#pragma unroll
      for (int v = 0; v < V; ++v) {
        sa[wt][x0 + v] = ma[v];
        sg[wt][x0 + v] = g[v];
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < (CH + NT - 1) / NT; ++k) {
        const int x = threadIdx.x + k * NT;
        if (x < CH) {
          if constexpr (PHASE == kWhole) {
#pragma unroll
            for (int w = 0; w < WT; ++w) {
              const float b = sb[w][x];
              sb[w][x] = hj[k];
              hj[k] = apply(sa[w][x], b, hj[k]);
            }
#pragma unroll
            for (int w = WT - 1; w >= 0; --w) {
              const float b = sg[w][x];
              sg[w][x] = uj[k];
              uj[k] = apply(sa[w][x], b, uj[k]);
            }
          } else {
            float a = 1.f, b = 0.f;
#pragma unroll
            for (int w = WT - 1; w >= 0; --w) {
              b = apply(sa[w][x], sg[w][x], b);
              a = joined(a, sa[w][x]);
            }
            const unsigned c = (unsigned)at.group * CH + x;
            // (a last tile too short for them is joined from its steps)
            if (c < s.C && s.T - tile * (L * WT) >= value_rows<T>(1)) {
              const Channel e = channel(s, c);
              T* row = element<T>(s, s.out, s.ldo, tile * (L * WT), e.n, e.j);
              put_value<T>(row, ostep, 0, a);
              put_value<T>(row, ostep, 1, b);
            }
          }
        }
      }
      __syncthreads();
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if constexpr (PHASE == kWhole) hin[v] = sb[wt][x0 + v];
        uin[v] = sg[wt][x0 + v];
      }
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) uin[v] = u[v];
    }
    if constexpr (PHASE == kWhole) {
      if (plain) run_back<T, V, L, true>(z, rh, rg, n, clear, lane, pl.ok, hin, uin, out, ostep, s.H);
      else run_back<T, V, L, false>(z, rh, rg, n, clear, lane, pl.ok, hin, uin, out, ostep, s.H);
      if (s.last && pl.ok && t0 == 0) {   // the thread of the first step
#pragma unroll
        for (int v = 0; v < V; ++v) s.last[pl.c + v] = uin[v];
      }
      if constexpr (WT == 1) {
#pragma unroll
        for (int v = 0; v < V; ++v) u[v] = uin[v];
      }
    }
    if constexpr (FETCH) {
      __syncwarp();
      if (more(ahead)) {
        float f;
        load(place(ahead.group), tile_of(ahead), cz, rg, rh, f);
        flags.set(stage, f);
        advance(ahead);
      }
      fetch_commit();
      stage = stage == kStages - 1 ? 0 : stage + 1;
    }
    advance(at);
  }
}

// Joins the tiles' maps along the sequence: a block takes 32 channels, its
// warps consecutive runs of kRun tiles, round after round.  Forward it leaves
// the state entering each tile in carry; backward, what reaches each tile's last
// state from later tiles as value 2 of the tile.
constexpr int kRun = 8, kJoinWarps = 32;
template <typename T, bool BACK>
__global__ void __launch_bounds__(kJoinWarps* kWarp) scan_join_kernel(const ScanArgs s) {
  __shared__ float sa[kJoinWarps][kWarp], sb[kJoinWarps][kWarp];
  pdl_wait();
  const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp;
  const int64_t c = (int64_t)blockIdx.x * kWarp + lane;
  const bool ok = c < s.C;
  const Channel e = channel(s, ok ? (unsigned)c : 0);
  const int n = e.n, j = e.j;
  const int tiles = (s.T + PPO_SCAN_BLOCK - 1) / PPO_SCAN_BLOCK;
  const int need = value_rows<T>(1);
  auto rows_of = [&](int tile) { return element<T>(s, s.out, s.ldo, tile * PPO_SCAN_BLOCK, n, j); };
  // maps 0 .. tiles - 2 forward (what enters tile 0 is h0); tiles - 1 .. 1 backward
  const int maps = tiles - 1;
  float x = 0.f;
  if (ok) {
    if (!BACK) {
      x = s.h0 ? s.h0[c] : 0.f;
      if (warp == 0) s.carry[c] = reset_flag(s, 0, n) != 0.f ? 0.f : x;
    } else {
      x = s.dhT ? s.dhT[c] : 0.f;
    }
  }
  for (int m0 = 0; m0 < maps; m0 += kJoinWarps * kRun) {
    float a[kRun], b[kRun];
    float ta = 1.f, tb = 0.f;
    const int64_t ostep = step_of(s, s.ldo);
    uint32_t cut = 0;   // forward: the state entering the tile after map i is cleared
    if (!BACK && ok) {
#pragma unroll
      for (int i = 0; i < kRun; ++i)
        cut |= reset_flag(s, (m0 + warp * kRun + i + 1) * PPO_SCAN_BLOCK, n) != 0.f ? 1u << i : 0u;
    }
    // all of a run's loads at once (off the end: the last map's, not used)
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
      const int m = min(m0 + warp * kRun + i, maps - 1);
      // (a last tile too short to hold its map: the one before it, not used)
      const int tile = BACK ? tiles - 1 - m - (s.T - (tiles - 1 - m) * PPO_SCAN_BLOCK < need) : m;
      T* row = rows_of(tile);
      a[i] = get_value<T>(row, ostep, 0);
      b[i] = get_value<T>(row, ostep, 1);
    }
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
      if (!ok || m0 + warp * kRun + i >= maps) {
        a[i] = 1.f;
        b[i] = 0.f;
      }
    }
    if (BACK && m0 + warp == 0 && ok && s.T - (tiles - 1) * PPO_SCAN_BLOCK < need) {
      // the short last tile: from its steps
      a[0] = 1.f;
      b[0] = 0.f;
      for (int t = s.T - 1; t >= (tiles - 1) * PPO_SCAN_BLOCK; --t) {
        const float pz = (float)*element<const T>(s, s.p, s.ldp, t, n, j);
        const float d = (float)*element<const T>(s, s.dh, s.lddh, t, n, j);
        float z[1], q[1] = {pz};
        sigmoid<1>(q, z);
        const bool gone = reset_flag(s, t, n) != 0.f;
        b[0] = gone ? 0.f : (1.f - z[0]) * (d + b[0]);
        a[0] = gone ? -1.f : joined(a[0], 1.f - z[0]);
      }
    }
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
      tb = apply(a[i], b[i], tb);
      ta = joined(ta, a[i]);
    }
    __syncthreads();
    sa[warp][lane] = ta;
    sb[warp][lane] = tb;
    __syncthreads();
    float y = x;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) {
      if (w == warp) y = x;
      x = apply(sa[w][lane], sb[w][lane], x);
    }
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
      const int m = m0 + warp * kRun + i;
      y = apply(a[i], b[i], y);
      if (ok && m < maps) {
        const int tile = BACK ? tiles - 2 - m : m + 1;
        if (BACK) put_value<T>(rows_of(tile), ostep, 2, y);
        else s.carry[(int64_t)tile * s.C + c] = (cut >> i) & 1u ? 0.f : y;
      }
    }
  }
}

// ---- plan -------------------------------------------------------------------------
// Steps of a warp's block (with 8, forward 76 us and backward 156 us instead of
// 72 and 146 at 128 x 2,048 x 256 bf16; 191 and 243 instead of 157 and 220 at
// 65,537 x 1 x 1,024); 8 blocks are a tile of PPO_SCAN_BLOCK.
constexpr int kSteps = 16;
constexpr int kTileWarps = PPO_SCAN_BLOCK / kSteps;
constexpr int kSms = 152;
// Channels from which a forward warp walks alone (862 steps of 304 x 512 bf16
// 151 us so, 167 in blocks; of 152 x 512, below the bound, 214 and 182).
constexpr int64_t kWalkChannels = kSms * 1024;
// "split" takes at most this many groups of channels (2,000 steps of 64 groups:
// 29 and 42 us split, 39 and 58 walked; of 256 groups 125 and 153 split, 57 and
// 83 walked) and at least this many tiles (600 steps of 64 groups, five tiles:
// 21 and 22 us split, 13 and 18 walked).
constexpr int kSplitGroups = 96, kSplitTiles = 8;

template <typename T, int V, int L, int WT, int WC, int PHASE>
cudaError_t launch(ScanArgs s, bool backward, cudaStream_t st) {
  constexpr int per = kWarp * V * WC, threads = WT * WC * kWarp;
  if (s.C > (1ll << 31) - per) return cudaErrorInvalidValue;
  s.groups = (int)((s.C + per - 1) / per);
  s.whole = s.H % (kWarp * V) == 0;
  const auto kernel = backward ? scan_bwd_kernel<T, V, L, WT, WC, PHASE>
                               : scan_fwd_kernel<T, V, L, WT, WC, PHASE>;
  const int inputs = backward && PHASE == kWhole ? 3 : 2;
  const size_t ring = L > 1 && kFetch<T, V> ? (size_t)kStages * inputs * L * threads * 4 : 0;
  if (ring) {
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)ring);
    if (e != cudaSuccess) return e;
  }
  // with fetched columns the blocks that fit an SM together stay on it and walk
  const int64_t resident = (int64_t)kSms * std::max(1, threads_per_sm(L, PHASE, backward) / threads);
  int64_t grid = ring ? std::min<int64_t>(s.groups, resident) : s.groups;
  if (s.split) {
    const int64_t tiles = (s.T + L * WT - 1) / (L * WT);
    grid = s.groups * std::min(tiles, std::max<int64_t>(1, resident / s.groups));
  }
  if (grid > (1ll << 30)) return cudaErrorInvalidValue;
  kernel<<<(unsigned)grid, threads, ring, st>>>(s);
  return cudaGetLastError();
}

// Few channels and a long sequence.  Forward it needs the carry to leave the
// entering states in, so that a call without one is walked (see above).
template <int V>
bool splits(const ScanArgs& s, bool backward) {
  // (the first tile's block may replace dhT while the last one's reads it)
  if (backward && s.last && s.last == s.dhT) return false;
  const int64_t groups = (s.C + kWarp * V - 1) / (kWarp * V);
  return s.carry && groups <= kSplitGroups && s.T >= kSplitTiles * PPO_SCAN_BLOCK;
}

template <typename T, int V>
cudaError_t dispatch(ScanArgs s, bool backward, cudaStream_t st) {
  // one step: a thread per channel (pair), nothing to join
  if (s.T == 1) return launch<T, V, 1, 1, 4, kWhole>(s, backward, st);
  if (s.T <= kSteps / 2) return launch<T, V, kSteps / 2, 1, 8, kWhole>(s, backward, st);
  // enough channels to fill the GPU: forward, a warp walks its channels alone
  if (s.T <= kSteps || (!backward && s.C >= kWalkChannels))
    return launch<T, V, kSteps, 1, 8, kWhole>(s, backward, st);
  // short sequences: as many warps along time as there are blocks of steps, the
  // others take more channels
  if (s.T <= 2 * kSteps) return launch<T, V, kSteps, 2, 4, kWhole>(s, backward, st);
  if (s.T <= 4 * kSteps) return launch<T, V, kSteps, 4, 2, kWhole>(s, backward, st);
  if (splits<V>(s, backward)) {
    s.split = 1;
    cudaError_t e = launch<T, V, kSteps, kTileWarps, 1, kMaps>(s, backward, st);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)((s.C + kWarp - 1) / kWarp)), block(kJoinWarps * kWarp);
    e = backward ? launch_pdl(scan_join_kernel<T, true>, grid, block, 0, st, s)
                 : launch_pdl(scan_join_kernel<T, false>, grid, block, 0, st, s);
    if (e != cudaSuccess) return e;
  }
  return launch<T, V, kSteps, kTileWarps, 1, kWhole>(s, backward, st);
}

ppo_status run(int32_t dtype, ScanArgs s, bool backward, bool pairs, bool wide, cudaStream_t st) {
  s.wide = wide;
  // ceil(log2 H) + 31 bits: exact for every c of 31 bits
  s.div_s = 31;
  while ((1ll << (s.div_s - 31)) < s.H) ++s.div_s;
  s.div_m = (unsigned)((1ull << s.div_s) / (uint64_t)s.H + 1);
  cudaError_t e;
  if (dtype == PPO_DTYPE_F32) e = dispatch<float, 1>(s, backward, st);
  else if (pairs) e = dispatch<__nv_bfloat16, 2>(s, backward, st);
  else e = dispatch<__nv_bfloat16, 1>(s, backward, st);
  return status_of(e);
}

bool aligned(std::initializer_list<const void*> ptrs, int bytes) {
  for (const void* q : ptrs)
    if (reinterpret_cast<uintptr_t>(q) % bytes) return false;
  return true;
}

bool sizes_ok(int64_t T, int64_t N, int64_t H) {
  constexpr int64_t top = 1ll << 31;
  return T >= 1 && N >= 1 && H >= 1 && H < (1ll << 28) && N < top && T < top - 4096 && T * N < top &&
         N * H < top - 4096;
}

}  // namespace
}  // namespace ppo

extern "C" {

ppo_status ppo_gated_scan_forward(int32_t dtype, const void* p, int64_t ldp, const float* done,
                                  const float* done0, const float* h0, int64_t T, int64_t N,
                                  int64_t H, void* h, int64_t ldh, float* hT, float* carry,
                                  cudaStream_t st) {
  using namespace ppo;
  if (!ops::dtype_ok(dtype) || !p || !h || !sizes_ok(T, N, H)) return PPO_ERR_INVALID;
  if (!ops::extent_ok(T * N, ldp, 2 * H) || !ops::extent_ok(T * N, ldh, H) ||
      ldp >= (1ll << 30) || ldh >= (1ll << 30))
    return PPO_ERR_INVALID;
  if (!aligned({p, h}, ops::esize(dtype)) || !aligned({done, done0, h0, hT, carry}, 4))
    return PPO_ERR_ALIGN;
  ScanArgs s{};
  s.p = p;
  s.ldp = (uint32_t)(ldp * ops::esize(dtype));
  s.done = done;
  s.done0 = done0;
  s.h0 = h0;
  s.T = (int)T;
  s.N = (int)N;
  s.H = (int)H;
  s.C = N * H;
  s.out = h;
  s.ldo = (uint32_t)(ldh * ops::esize(dtype));
  s.last = hT;
  s.carry = carry;
  const int piece = 16 / ops::esize(dtype);
  return run(dtype, s, false, H % 2 == 0 && ldp % 2 == 0 && ldh % 2 == 0 && aligned({p, h}, 4),
             H % piece == 0 && ldp % piece == 0 && aligned({p}, 16), st);
}

ppo_status ppo_gated_scan_backward(int32_t dtype, const void* dh, int64_t lddh, const void* p,
                                   int64_t ldp, const float* done, const float* done0,
                                   const float* carry, const float* dhT, int64_t T, int64_t N,
                                   int64_t H, void* dp, int64_t lddp, float* dh0,
                                   cudaStream_t st) {
  using namespace ppo;
  if (!ops::dtype_ok(dtype) || !dh || !p || !carry || !dp || !sizes_ok(T, N, H))
    return PPO_ERR_INVALID;
  if (!ops::extent_ok(T * N, ldp, 2 * H) || !ops::extent_ok(T * N, lddp, 2 * H) ||
      !ops::extent_ok(T * N, lddh, H) || ldp >= (1ll << 30) || lddp >= (1ll << 30) ||
      lddh >= (1ll << 30))
    return PPO_ERR_INVALID;
  if (!aligned({dh, p, dp}, ops::esize(dtype)) || !aligned({done, done0, carry, dhT, dh0}, 4))
    return PPO_ERR_ALIGN;
  ScanArgs s{};
  s.p = p;
  s.ldp = (uint32_t)(ldp * ops::esize(dtype));
  s.dh = dh;
  s.lddh = (uint32_t)(lddh * ops::esize(dtype));
  s.done = done;
  s.done0 = done0;
  s.dhT = dhT;
  s.T = (int)T;
  s.N = (int)N;
  s.H = (int)H;
  s.C = N * H;
  s.out = dp;
  s.ldo = (uint32_t)(lddp * ops::esize(dtype));
  s.last = dh0;
  s.carry = const_cast<float*>(carry);
  const int piece = 16 / ops::esize(dtype);
  return run(dtype, s, true, H % 2 == 0 && ldp % 2 == 0 && lddh % 2 == 0 && lddp % 2 == 0 && aligned({dh, p, dp}, 4),
             H % piece == 0 && ldp % piece == 0 && lddh % piece == 0 && aligned({p, dh}, 16), st);
}

}  // extern "C"
