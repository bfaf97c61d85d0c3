// gscan.cu -- the gated linear recurrence of a MinGRU layer over T steps, and
// its backward pass.
//
//   z = sigmoid(pz),  a = 1 - z,  b = z ph,   h_t = a_t h_{t-1} + b_t,
// h_{t-1} taken as 0 where the state was cleared.  A step is the affine map
// (a, b); maps of consecutive steps compose, (a1, b1) then (a2, b2) is
// (a1 a2, a2 b1 + b2), so a channel's steps can be cut into blocks that are
// reduced to one map each, joined, and run again from their entering state.
// The backward recurrence g_t = dh_t + u_t, u_{t-1} = a_t g_t (0 where the
// state was cleared) has the same form from the other end.
//
// Bound by memory (6 bytes per channel and step forward, 10 backward, in
// bf16), so every pre-activation is read once: a thread keeps kSteps steps of
// its channels in registers, reduces them, meets the other warps of its
// block (consecutive steps of the same channels) in shared memory and runs the
// steps again from registers.  A block of WT warps so covers a tile of
// kSteps * WT steps and walks along the time axis tile by tile; with few
// channels, a cluster of CS blocks takes CS consecutive tiles at a time and
// joins them through distributed shared memory.  The forward pass leaves the
// state that enters every 128th step for the backward pass, which walks the
// same tiles from the end and recomputes the states in between.
// Compositions happen in an order fixed by the sizes: results are
// deterministic.  A cleared state is dropped by a select, never multiplied by
// 0, so that infinities and NaN do not cross it.
#include <cooperative_groups.h>

#include <algorithm>

#include "ops.cuh"

namespace ppo {
namespace {

using namespace ops;
namespace cg = cooperative_groups;

struct ScanArgs {
  const void *p, *dh;
  int64_t ldp, lddh;
  const float *done, *done0, *h0, *dhT;
  int64_t T, N, H, C;      // C = N * H channels
  void* out;               // h, or dp
  int64_t ldo;
  float *last;             // hT, or dh0 (nullable)
  float* carry;            // [ceil(T / 128)][C]: written (nullable), or read
};

__device__ __forceinline__ float sigmoid(float x) {
  // 1 / (1 + e^-x): e^-x overflows to inf below -88, whose reciprocal is 0
  return __fdividef(1.f, 1.f + __expf(-x));
}

// The affine map of a block of steps.  a < 0 stands for "the state was cleared
// inside": what enters does not matter (products of 1 - z are never negative).
struct Map {
  float a, b;
};
__device__ __forceinline__ float apply(const Map& m, float h) {
  return m.a < 0.f ? m.b : fmaf(m.a, h, m.b);
}

// Bit i: the state entering step t0 + i is cleared (steps beyond T: clear no
// state).  `same`: all lanes of the warp belong to one environment.
template <int L>
__device__ __forceinline__ uint32_t reset_mask(const ScanArgs& s, int64_t t0, int64_t n, bool ok,
                                               bool same, int lane) {
  auto flag = [&](int64_t t) {
    if (t < 0 || t >= s.T) return false;
    if (t == 0) return s.done0 && __ldg(s.done0 + n) != 0.f;
    return s.done && __ldg(s.done + (t - 1) * s.N + n) != 0.f;
  };
  if (L > 1 && same) return __ballot_sync(0xffffffffu, lane < L && flag(t0 + lane)) & ((1ull << L) - 1);
  uint32_t m = 0;
  if (ok) {
#pragma unroll
    for (int i = 0; i < L; ++i) m |= flag(t0 + i) ? 1u << i : 0u;
  }
  return m;
}

// A thread's place: V consecutive channels of one environment, L steps.
struct Place {
  int64_t c, n, j;
  bool ok, same;
};
template <int V>
__device__ __forceinline__ Place place_of(const ScanArgs& s, int64_t group, int lane) {
  Place p;
  const int64_t first = group * kWarp * V;
  p.c = first + lane * V;
  p.ok = p.c < s.C;
  p.n = p.ok ? p.c / s.H : 0;
  p.j = p.ok ? p.c - p.n * s.H : 0;
  const int64_t lastc = min(first + kWarp * V, s.C) - 1;
  p.same = first < s.C && first / s.H == lastc / s.H;
  // lanes past the end share the warp's environment where all others do
  if (p.same) p.n = first / s.H;
  return p;
}

// ---- forward --------------------------------------------------------------------
// WT warps along time, WC along channels; CS blocks of a cluster along time.
template <typename T, int V, int L, int WT, int WC, bool CLUSTER>
__global__ void __launch_bounds__(WT* WC* kWarp)
scan_fwd_kernel(const ScanArgs s) {
  __shared__ Map maps[2][WC][WT][V][kWarp];
  __shared__ Map total[2][WC][V][kWarp];
  const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp;
  const int wt = warp % WT, wc = warp / WT;
  int rank = 0, cs = 1;
  if constexpr (CLUSTER) {
    rank = (int)cg::this_cluster().block_rank();
    cs = (int)cg::this_cluster().num_blocks();
  }
  const Place pl = place_of<V>(s, (int64_t)(blockIdx.x / cs) * WC + wc, lane);
  const int64_t tiles = (s.T + L * WT - 1) / (L * WT);
  const T* pz = static_cast<const T*>(s.p) + pl.n * s.ldp + pl.j;
  const T* ph = pz + s.H;
  const int64_t pstep = s.N * s.ldp;
  T* out = static_cast<T*>(s.out) + pl.n * s.ldo + pl.j;
  float h[V];
#pragma unroll
  for (int v = 0; v < V; ++v) h[v] = pl.ok && s.h0 ? s.h0[pl.c + v] : 0.f;
  int buf = 0;
  for (int64_t base = 0; base < tiles; base += cs, buf ^= 1) {
    const int64_t t0 = ((base + rank) * WT + wt) * L;
    Raw<T, V> rz[L], rh[L];
#pragma unroll
    for (int i = 0; i < L; ++i) {
      const bool in = pl.ok && t0 + i < s.T;
      rz[i] = in ? __ldg(reinterpret_cast<const Raw<T, V>*>(pz + (t0 + i) * pstep)) : Raw<T, V>{};
      rh[i] = in ? __ldg(reinterpret_cast<const Raw<T, V>*>(ph + (t0 + i) * pstep)) : Raw<T, V>{};
    }
    const uint32_t clear = reset_mask<L>(s, t0, pl.n, pl.ok, pl.same, lane);
    float z[L][V];
    Map m[V];
#pragma unroll
    for (int v = 0; v < V; ++v) m[v] = Map{1.f, 0.f};
#pragma unroll
    for (int i = 0; i < L; ++i) {
      const bool in = t0 + i < s.T;
      float x[V], c[V];
      to_f32<T, V>(rz[i], x);
      to_f32<T, V>(rh[i], c);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        z[i][v] = sigmoid(x[v]);
        if (in) {
          const float a = 1.f - z[i][v], b = z[i][v] * c[v];
          m[v].b = (clear >> i) & 1u ? b : fmaf(a, m[v].b, b);
          m[v].a *= a;
        }
      }
    }
    if constexpr (WT > 1) {
#pragma unroll
      for (int v = 0; v < V; ++v)
        maps[buf][wc][wt][v][lane] = Map{clear ? -1.f : m[v].a, m[v].b};
      __syncthreads();
    }
    // hin: the state entering this thread's steps; h moves past the tiles
    float hin[V];
    if constexpr (CLUSTER) {
      if (wt == 0) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
          Map t{1.f, 0.f};
#pragma unroll
          for (int w = 0; w < WT; ++w) {
            const Map k = maps[buf][wc][w][v][lane];
            t.b = k.a < 0.f ? k.b : fmaf(k.a, t.b, k.b);
            t.a = k.a < 0.f || t.a < 0.f ? -1.f : t.a * k.a;
          }
          total[buf][wc][v][lane] = t;
        }
      }
      cg::this_cluster().sync();
#pragma unroll
      for (int v = 0; v < V; ++v) {
        for (int r = 0; r < cs; ++r) {
          if (r == rank) hin[v] = h[v];
          const Map* remote = cg::this_cluster().map_shared_rank(&total[buf][wc][v][lane], r);
          h[v] = apply(*remote, h[v]);
        }
#pragma unroll
        for (int w = 0; w < WT; ++w)
          if (w < wt) hin[v] = apply(maps[buf][wc][w][v][lane], hin[v]);
      }
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if constexpr (WT > 1) {
#pragma unroll
          for (int w = 0; w < WT; ++w) {
            if (w == wt) hin[v] = h[v];
            h[v] = apply(maps[buf][wc][w][v][lane], h[v]);
          }
        } else {
          hin[v] = h[v];
        }
      }
    }
    if (s.carry && pl.ok && t0 % PPO_SCAN_BLOCK == 0 && t0 < s.T) {
#pragma unroll
      for (int v = 0; v < V; ++v)
        s.carry[(t0 / PPO_SCAN_BLOCK) * s.C + pl.c + v] = clear & 1u ? 0.f : hin[v];
    }
#pragma unroll
    for (int i = 0; i < L; ++i) {
      float c[V];
      to_f32<T, V>(rh[i], c);
      if (t0 + i < s.T) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float b = z[i][v] * c[v];
          hin[v] = (clear >> i) & 1u ? b : fmaf(1.f - z[i][v], hin[v], b);
        }
        if (pl.ok)
          *reinterpret_cast<Raw<T, V>*>(out + (t0 + i) * s.N * s.ldo) = from_f32<T, V>(hin);
      }
    }
    if constexpr (WT == 1) {
#pragma unroll
      for (int v = 0; v < V; ++v) h[v] = hin[v];
    }
  }
  if (s.last && wt == 0 && rank == 0 && pl.ok) {
#pragma unroll
    for (int v = 0; v < V; ++v) s.last[pl.c + v] = h[v];
  }
  if constexpr (CLUSTER) cg::this_cluster().sync();   // no block leaves while its maps are read
}

// ---- backward ---------------------------------------------------------------------
template <typename T, int V, int L, int WT, int WC, bool CLUSTER>
__global__ void __launch_bounds__(WT* WC* kWarp)
scan_bwd_kernel(const ScanArgs s) {
  // fwd maps of the blocks of steps, and the maps of what they pass back
  // (same a; the states of a tile start from the stored carry)
  __shared__ Map maps[2][WC][WT][V][kWarp];
  __shared__ float back[2][WC][WT][V][kWarp];
  __shared__ Map total[2][WC][V][kWarp];
  static_assert(PPO_SCAN_BLOCK % (L * WT) == 0, "tiles start at stored states or inside a block");
  const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp;
  const int wt = warp % WT, wc = warp / WT;
  int rank = 0, cs = 1;
  if constexpr (CLUSTER) {
    rank = (int)cg::this_cluster().block_rank();
    cs = (int)cg::this_cluster().num_blocks();
  }
  const Place pl = place_of<V>(s, (int64_t)(blockIdx.x / cs) * WC + wc, lane);
  const int64_t tiles = (s.T + L * WT - 1) / (L * WT);
  const T* pz = static_cast<const T*>(s.p) + pl.n * s.ldp + pl.j;
  const T* ph = pz + s.H;
  const T* gh = static_cast<const T*>(s.dh) + pl.n * s.lddh + pl.j;
  const int64_t pstep = s.N * s.ldp, gstep = s.N * s.lddh, ostep = s.N * s.ldo;
  T* oz = static_cast<T*>(s.out) + pl.n * s.ldo + pl.j;
  T* oh = oz + s.H;
  float u[V];
#pragma unroll
  for (int v = 0; v < V; ++v) u[v] = pl.ok && s.dhT ? s.dhT[pl.c + v] : 0.f;
  int buf = 0;
  const int64_t rounds = (tiles + cs - 1) / cs;
  for (int64_t r0 = rounds - 1; r0 >= 0; --r0, buf ^= 1) {
    const int64_t t0 = ((r0 * cs + rank) * WT + wt) * L;
    Raw<T, V> rz[L], rh[L], rg[L];
#pragma unroll
    for (int i = 0; i < L; ++i) {
      const bool in = pl.ok && t0 + i < s.T;
      rz[i] = in ? __ldg(reinterpret_cast<const Raw<T, V>*>(pz + (t0 + i) * pstep)) : Raw<T, V>{};
      rh[i] = in ? __ldg(reinterpret_cast<const Raw<T, V>*>(ph + (t0 + i) * pstep)) : Raw<T, V>{};
      rg[i] = in ? __ldg(reinterpret_cast<const Raw<T, V>*>(gh + (t0 + i) * gstep)) : Raw<T, V>{};
    }
    const int64_t tile0 = (r0 * cs + rank) * WT * L;
    float hin[V];
#pragma unroll
    for (int v = 0; v < V; ++v)
      hin[v] = pl.ok && tile0 < s.T ? __ldg(s.carry + (tile0 / PPO_SCAN_BLOCK) * s.C + pl.c + v) : 0.f;
    const uint32_t clear = reset_mask<L>(s, t0, pl.n, pl.ok, pl.same, lane);
    float z[L][V];
    Map m[V];
    float g[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      m[v] = Map{1.f, 0.f};
      g[v] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < L; ++i) {
      float x[V], c[V];
      to_f32<T, V>(rz[i], x);
      to_f32<T, V>(rh[i], c);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        z[i][v] = sigmoid(x[v]);
        if (t0 + i < s.T) {
          const float a = 1.f - z[i][v], b = z[i][v] * c[v];
          m[v].b = (clear >> i) & 1u ? b : fmaf(a, m[v].b, b);
          m[v].a *= a;
        }
      }
    }
    if constexpr (WT > 1) {
#pragma unroll
      for (int i = L - 1; i >= 0; --i) {
        float d[V];
        to_f32<T, V>(rg[i], d);
        if (t0 + i < s.T) {
#pragma unroll
          for (int v = 0; v < V; ++v)
            g[v] = (clear >> i) & 1u ? 0.f : (1.f - z[i][v]) * (d[v] + g[v]);
        }
      }
#pragma unroll
      for (int v = 0; v < V; ++v) {
        maps[buf][wc][wt][v][lane] = Map{clear ? -1.f : m[v].a, m[v].b};
        back[buf][wc][wt][v][lane] = g[v];
      }
      __syncthreads();
      // the state entering this thread's steps, from the tile's
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int w = 0; w < WT - 1; ++w)
          if (w < wt) hin[v] = apply(maps[buf][wc][w][v][lane], hin[v]);
    }
    // uin: what reaches this thread's last state from later steps
    float uin[V];
    auto pass_back = [&](int w, int v, float x) {
      const float a = maps[buf][wc][w][v][lane].a, b = back[buf][wc][w][v][lane];
      return a < 0.f ? b : fmaf(a, x, b);
    };
    if constexpr (CLUSTER) {
      if (wt == 0) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
          Map t{1.f, 0.f};
#pragma unroll
          for (int w = WT - 1; w >= 0; --w) {
            const float a = maps[buf][wc][w][v][lane].a;
            t.b = pass_back(w, v, t.b);
            t.a = a < 0.f || t.a < 0.f ? -1.f : t.a * a;
          }
          total[buf][wc][v][lane] = t;
        }
      }
      cg::this_cluster().sync();
#pragma unroll
      for (int v = 0; v < V; ++v) {
        for (int r = cs - 1; r >= 0; --r) {
          if (r == rank) uin[v] = u[v];
          const Map* remote = cg::this_cluster().map_shared_rank(&total[buf][wc][v][lane], r);
          u[v] = apply(*remote, u[v]);
        }
#pragma unroll
        for (int w = WT - 1; w > 0; --w)
          if (w > wt) uin[v] = pass_back(w, v, uin[v]);
      }
    } else if constexpr (WT > 1) {
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int w = WT - 1; w >= 0; --w) {
          if (w == wt) uin[v] = u[v];
          u[v] = pass_back(w, v, u[v]);
        }
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) uin[v] = u[v];
    }
    // the states entering the steps, then the steps from the last to the first
    float hp[L][V];
#pragma unroll
    for (int i = 0; i < L; ++i) {
      float c[V];
      to_f32<T, V>(rh[i], c);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if ((clear >> i) & 1u) hin[v] = 0.f;
        hp[i][v] = hin[v];
        hin[v] = fmaf(1.f - z[i][v], hin[v], z[i][v] * c[v]);
      }
    }
#pragma unroll
    for (int i = L - 1; i >= 0; --i) {
      float c[V], d[V], dz[V], dc[V];
      to_f32<T, V>(rh[i], c);
      to_f32<T, V>(rg[i], d);
      if (t0 + i < s.T) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float gg = d[v] + uin[v], a = 1.f - z[i][v];
          dc[v] = gg * z[i][v];
          dz[v] = dc[v] * (c[v] - hp[i][v]) * a;
          uin[v] = (clear >> i) & 1u ? 0.f : a * gg;
        }
        if (pl.ok) {
          *reinterpret_cast<Raw<T, V>*>(oz + (t0 + i) * ostep) = from_f32<T, V>(dz);
          *reinterpret_cast<Raw<T, V>*>(oh + (t0 + i) * ostep) = from_f32<T, V>(dc);
        }
      }
    }
    if constexpr (WT == 1) {
#pragma unroll
      for (int v = 0; v < V; ++v) u[v] = uin[v];
    }
  }
  if (s.last && wt == 0 && rank == 0 && pl.ok) {
#pragma unroll
    for (int v = 0; v < V; ++v) s.last[pl.c + v] = u[v];
  }
  if constexpr (CLUSTER) cg::this_cluster().sync();
}

// ---- plan -------------------------------------------------------------------------
template <typename T, int V, int L, int WT, int WC>
cudaError_t launch(const ScanArgs& s, bool backward, cudaStream_t st) {
  const int64_t groups = (s.C + (int64_t)kWarp * V * WC - 1) / ((int64_t)kWarp * V * WC);
  if (groups > (1ll << 30)) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)groups), block(WT * WC * kWarp);
  if (backward) scan_bwd_kernel<T, V, L, WT, WC, false><<<grid, block, 0, st>>>(s);
  else scan_fwd_kernel<T, V, L, WT, WC, false><<<grid, block, 0, st>>>(s);
  return cudaGetLastError();
}

template <typename T, int V>
cudaError_t dispatch(const ScanArgs& s, bool backward, cudaStream_t st) {
  if (s.T == 1) return launch<T, V, 1, 1, 4>(s, backward, st);
  return launch<T, V, 16, 8, 1>(s, backward, st);
}

ppo_status run(int32_t dtype, const ScanArgs& s, bool backward, bool pairs, cudaStream_t st) {
  cudaError_t e;
  if (dtype == PPO_DTYPE_F32) e = dispatch<float, 1>(s, backward, st);
  else if (pairs) e = dispatch<__nv_bfloat16, 2>(s, backward, st);
  else e = dispatch<__nv_bfloat16, 1>(s, backward, st);
  return e == cudaSuccess ? PPO_OK : PPO_ERR_CUDA;
}

bool aligned(std::initializer_list<const void*> ptrs, int bytes) {
  for (const void* q : ptrs)
    if (reinterpret_cast<uintptr_t>(q) % bytes) return false;
  return true;
}

bool sizes_ok(int64_t T, int64_t N, int64_t H) {
  return T >= 1 && N >= 1 && H >= 1 && H < (1ll << 30) && N < (1ll << 31) && T < (1ll << 31) &&
         N * H < (1ll << 34);
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
  if (!ops::extent_ok(T * N, ldp, 2 * H) || !ops::extent_ok(T * N, ldh, H)) return PPO_ERR_INVALID;
  if (!aligned({p, h}, ops::esize(dtype)) || !aligned({done, done0, h0, hT, carry}, 4))
    return PPO_ERR_ALIGN;
  ScanArgs s{};
  s.p = p;
  s.ldp = ldp;
  s.done = done;
  s.done0 = done0;
  s.h0 = h0;
  s.T = T;
  s.N = N;
  s.H = H;
  s.C = N * H;
  s.out = h;
  s.ldo = ldh;
  s.last = hT;
  s.carry = carry;
  return run(dtype, s, false, H % 2 == 0 && ldp % 2 == 0 && ldh % 2 == 0 && aligned({p, h}, 4), st);
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
      !ops::extent_ok(T * N, lddh, H))
    return PPO_ERR_INVALID;
  if (!aligned({dh, p, dp}, ops::esize(dtype)) || !aligned({done, done0, carry, dhT, dh0}, 4))
    return PPO_ERR_ALIGN;
  ScanArgs s{};
  s.p = p;
  s.ldp = ldp;
  s.dh = dh;
  s.lddh = lddh;
  s.done = done;
  s.done0 = done0;
  s.dhT = dhT;
  s.T = T;
  s.N = N;
  s.H = H;
  s.C = N * H;
  s.out = dp;
  s.ldo = lddp;
  s.last = dh0;
  s.carry = const_cast<float*>(carry);
  return run(dtype, s, true, H % 2 == 0 && ldp % 2 == 0 && lddh % 2 == 0 && lddp % 2 == 0 && aligned({dh, p, dp}, 4),
             st);
}

}  // extern "C"
