// glinear_tc.cu -- gated linear layers in bf16 on the tensor cores (tcgen05): the
// product and the gate in one kernel, operands streamed by TMA.
//
// Forward: a tile's B operand is made of two runs of W's rows, the gate's and the
// other projection's of the same columns, so that both sums of an output lie in
// one accumulator, side by side, and the epilogue has them at once: bias,
// pre-activations out, activation, product, y out.  Backward: a tile of d = dz W2;
// the epilogue reads the two pre-activations of each element and writes
// d u act'(g), d act(g) and act(g) u.
//
// As in linear_tc.cu a CTA, or a pair of CTAs, walks over tiles: warp 0 loads, warp
// 1 issues the MMAs into one of two accumulators, 16 warps (8 for single CTAs)
// drain the other one.  An epilogue warp has three boxes of 16 rows x 64 columns
// in shared memory: forward those of y, gate and up on their way out; backward gate
// and up come in by TMA, are overwritten by their gradients and leave with y.
//
// What bounds it: 32,768 x 512 -> 2,048 (in a graph), forward without pre 89 us, by the
// multiplications 73 and by the operands that an SM takes in 78; with pre 109: the
// epilogue, which waits for its stores to leave the boxes; backward 105 and with y 121, by
// its 570 and 705 MB 84 and 104.  Long sums: 8,192 x 4,096 -> 4,096 forward 330 (291 by the
// multiplications), backward 200 (146).
//
// Every wait on an mbarrier is bounded; on expiry the kernel sets the error
// word, stops issuing, drains what is in flight and frees its TMEM.
#include <algorithm>

#include "gemm.h"
#include "glinear.h"
#include "lin_tile.cuh"

namespace ppo {
namespace glin {
namespace {

using namespace lin;

constexpr int kFirstEpi = 4;           // warps 0..3: producer, MMA, two idle
constexpr int kBox = 2048;             // 16 rows x 128 bytes, 128-byte swizzle

template <int CG, bool BACK>
struct Cfg {
  static constexpr int BN = CG == 2 ? 256 : 128;       // columns of an accumulator
  static constexpr int GC = BACK ? BN : BN / 2;        // gated columns of a tile
  static constexpr int A_BYTES = BM * BK * 2;
  static constexpr int B_ROWS = BN / CG;
  static constexpr int B_BYTES = B_ROWS * BK * 2;
  static constexpr int STAGE = A_BYTES + B_BYTES;
  static constexpr int S = 4;
  static constexpr int EW = CG == 2 ? 16 : 8;
  static constexpr int THREADS = (kFirstEpi + EW) * kWarp;
  static constexpr int BOXES = EW * 3 * kBox;
  static constexpr int TMEM = 2 * BN;
  static constexpr int CTRL = 512;
  static constexpr size_t SMEM = 1024 + (size_t)S * STAGE + BOXES + CTRL;
  static_assert(SMEM <= 232448, "shared memory per CTA");
};

struct TcArgs {
  int I, J;                      // rows, gated columns
  int tiles_i, tiles_j, k_tiles, units;
  int act;
  const float* bias;             // [2 J] (nullable)
  int bias2;                     // pairs of either half are aligned
  // the two halves side by side (forward: pre out, nullable; backward: dp out), and y (nullable backward)
  void* both;
  int64_t ldboth;
  void* y;
  int64_t ldy;
  const void* in;                // backward: pre
  int64_t ldin;
  int tma_both, tma_y, tma_in;   // they move by TMA
  int* err;
};

// 16 TMEM lanes x 32 columns, laid out as tmem_ld_16x64's first four groups of columns
__device__ __forceinline__ void tmem_ld_16x32(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait16(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}

// act(g) of pairs
template <int ACT>
__device__ __forceinline__ void act_all(float2 (&v)[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] = act_pair<ACT>(v[k]);
}
__device__ __forceinline__ void act_all(int act, float2 (&v)[8]) {
  switch (act) {
    case PPO_ACT_TANH: act_all<PPO_ACT_TANH>(v); break;
    case PPO_ACT_RELU: act_all<PPO_ACT_RELU>(v); break;
    case PPO_ACT_SILU: act_all<PPO_ACT_SILU>(v); break;
    case PPO_ACT_GELU: act_all<PPO_ACT_GELU>(v); break;
    default: break;
  }
}
// act(x) and act'(x) of a pair
template <int ACT>
__device__ __forceinline__ void value_and_slope(float2 x, float2& a, float2& s) {
  if constexpr (ACT == PPO_ACT_SILU || ACT == PPO_ACT_GELU) {
    float2 q, e, x2;
    gate_pair<ACT>(x, q, e, x2);
    a = fmul2(x, q);
    float2 t = ffma2(q, both(-1.f), both(1.f));
    if constexpr (ACT == PPO_ACT_GELU)
      t = fmul2(t, ffma2(make_float2(fminf(x2.x, ops::kGeluTop), fminf(x2.y, ops::kGeluTop)),
                         both(3.f * ops::kGeluU * ops::kGeluA), both(ops::kGeluU)));
    s = ffma2(a, t, q);
  } else {
    a = act_pair<ACT>(x);
    s = slope_pair<ACT>(x);
  }
}
// d (in place of it) and the pre-activations of eight pairs become d act(g) u's
// gradients; y[k] = act(g) u.
template <int ACT>
__device__ __forceinline__ void grad_all(const float2 (&d)[8], uint32_t (&g)[8], uint32_t (&u)[8],
                                         uint32_t (&y)[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float2 up = unpack_bf16x2(u[k]);
    float2 a, s;
    value_and_slope<ACT>(unpack_bf16x2(g[k]), a, s);
    // (d u may overflow where the slope is 0)
    const float2 v = fmul2(a, up), dg = fmul2(fmul2(d[k], s), up), du = fmul2(d[k], a);
    g[k] = pack_bf16x2(dg.x, dg.y);
    u[k] = pack_bf16x2(du.x, du.y);
    y[k] = pack_bf16x2(v.x, v.y);
  }
}
__device__ __forceinline__ void grad_all(int act, const float2 (&d)[8], uint32_t (&g)[8], uint32_t (&u)[8],
                                         uint32_t (&y)[8]) {
  switch (act) {
    case PPO_ACT_TANH: grad_all<PPO_ACT_TANH>(d, g, u, y); break;
    case PPO_ACT_RELU: grad_all<PPO_ACT_RELU>(d, g, u, y); break;
    case PPO_ACT_SILU: grad_all<PPO_ACT_SILU>(d, g, u, y); break;
    case PPO_ACT_GELU: grad_all<PPO_ACT_GELU>(d, g, u, y); break;
    default: grad_all<PPO_ACT_NONE>(d, g, u, y); break;
  }
}

// tmB: W (forward) or W2; tmG, tmU, tmY: boxes out; tmP, tmQ: gate and up in (backward)
template <int CG, bool BACK, int SETS>
__global__ void __launch_bounds__(Cfg<CG, BACK>::THREADS, 1)
glin_tc_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
               const __grid_constant__ CUtensorMap tmG, const __grid_constant__ CUtensorMap tmU,
               const __grid_constant__ CUtensorMap tmY, const __grid_constant__ CUtensorMap tmP,
               const __grid_constant__ CUtensorMap tmQ, const TcArgs p) {
  using C = Cfg<CG, BACK>;
  constexpr int S = C::S;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  uint8_t* boxes = gbase + (size_t)S * C::STAGE;
  uint8_t* ctrl = boxes + C::BOXES;
  // full[S] empty[S] tfull[2] tempty[2] drain box[EW]
  uint64_t* bars = reinterpret_cast<uint64_t*>(ctrl);
  auto full = [&](int s) { return smem_u32(&bars[s]); };
  auto empty = [&](int s) { return smem_u32(&bars[S + s]); };
  auto tfull = [&](int a) { return smem_u32(&bars[2 * S + a]); };
  auto tempty = [&](int a) { return smem_u32(&bars[2 * S + 2 + a]); };
  const uint32_t drain = smem_u32(&bars[2 * S + 4]);
  auto box_bar = [&](int w) { return smem_u32(&bars[2 * S + 5 + w]); };
  constexpr int kBars = 2 * S + 5 + C::EW;
  static_assert(kBars * 8 + 16 <= C::CTRL, "control block");
  uint32_t* tslot = reinterpret_cast<uint32_t*>(&bars[kBars]);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tslot + 1);
  volatile uint32_t* cnt = reinterpret_cast<volatile uint32_t*>(tslot + 2);   // issued, consumed

  const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp;
  const uint32_t rank = CG == 2 ? lin::cluster_rank() : 0u;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull(a), 1);
      mbar_init(tempty(a), CG * C::EW / SETS);
    }
    mbar_init(drain, 1);
    for (int w = 0; w < C::EW; ++w) mbar_init(box_bar(w), 1);
    *abort_flag = 0;
    cnt[0] = cnt[1] = 0;
    fence_mbar_init();
  }
  if (warp == 1) alloc<CG>(smem_u32(tslot), C::TMEM);
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tmA);
    prefetch_tmap(&tmB);
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync();   // the pair's barriers exist
  tc_fence_after();
  const uint32_t tmem = *tslot;
  const Guard g{abort_flag, p.err, kWaitNs};
  const int group = blockIdx.x / CG, groups = gridDim.x / CG;
  pdl_wait();
  pdl_trigger();
  auto sA = [&](int s) { return base + (uint32_t)(s * C::STAGE); };
  auto sB = [&](int s) { return base + (uint32_t)(s * C::STAGE + C::A_BYTES); };
  // tiles in their order, column tiles first, without a division for each
  struct Tile {
    int i, j;
  };
  const int dr = groups / p.tiles_j, dc = groups - dr * p.tiles_j;
  auto after = [&](Tile x) {
    x.i += dr;
    x.j += dc;
    if (x.j >= p.tiles_j) {
      x.j -= p.tiles_j;
      ++x.i;
    }
    return x;
  };
  const Tile first{group / p.tiles_j, group % p.tiles_j};

  // 16 epilogue warps leave 96 registers a thread: their four warpgroups take
  // some from the first one (64 + 4 x 104 = 5 x 96, the launch's registers)
  constexpr bool kShift = C::EW == 16;
  if (warp < kFirstEpi) {
    if constexpr (kShift) regs_dec<64>();
    if (warp == 0 && lane == 0) {
      uint32_t it = 0, ph = 0;
      int s = 0;
      bool ok = true;
      Tile x = first;
      for (int n = group; n < p.units && ok; n += groups, x = after(x)) {
        const int i0 = (x.i * CG + (int)rank) * BM;
        for (int kt = 0; kt < p.k_tiles; ++kt) {
          if (!wait_bar(empty(s), ph ^ 1, g)) { ok = false; break; }
          if (rank == 0) mbar_arrive_expect_tx(full(s), CG * C::STAGE);
          const uint32_t bar = CG == 2 ? map_rank(full(s), 0) : full(s);
          load_2d<CG>(sA(s), &tmA, kt * BK, i0, bar);
          if constexpr (BACK) {
            const int j0 = x.j * C::GC + (int)rank * C::B_ROWS;
#pragma unroll
            for (int b = 0; b < C::B_ROWS / 64; ++b)
              load_2d<CG>(sB(s) + b * 8192, &tmB, j0 + 64 * b, kt * BK, bar);
          } else if constexpr (CG == 2) {
            // the accumulator's first half is this CTA's or the other's rows of W
            load_2d<CG>(sB(s), &tmB, kt * BK, (rank ? p.J : 0) + x.j * C::GC, bar);
          } else {
            load_2d<CG>(sB(s), &tmB, kt * BK, x.j * C::GC, bar);
            load_2d<CG>(sB(s) + C::B_BYTES / 2, &tmB, kt * BK, p.J + x.j * C::GC, bar);
          }
          cnt[0] = ++it;
          if (++s == S) { s = 0; ph ^= 1; }
        }
      }
      // every stage released: no commit is still to arrive here when the CTA leaves
      if (ok)
        for (int j = 0; j < S; ++j) {
          if (!wait_bar(empty(s), ph ^ 1, g)) break;
          if (++s == S) { s = 0; ph ^= 1; }
        }
    } else if (warp == 1 && lane == 0 && rank == 0) {
      constexpr uint32_t idesc = idesc_bf16(CG * BM, C::BN, false, BACK);
      uint32_t it = 0, ph = 0, n = 0;
      int s = 0;
      bool ok = true;
      for (int t = group; t < p.units && ok; t += groups, ++n) {
        const int acc = n & 1;
        if (!wait_bar(tempty(acc), ((n >> 1) & 1) ^ 1, g)) break;
        tc_fence_after();
        const uint32_t d = tmem + (uint32_t)(acc * C::BN);
        for (int kt = 0; kt < p.k_tiles; ++kt) {
          if (!wait_bar(full(s), ph, g)) { ok = false; break; }
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < BK / 16; ++kk) {
            const uint64_t da = sdesc_sw128(sA(s) + kk * 32, 16, 1024);
            const uint64_t db = BACK ? sdesc_sw128(sB(s) + kk * 2048, 8192, 1024)
                                     : sdesc_sw128(sB(s) + kk * 32, 16, 1024);
            mma<CG>(d, da, db, idesc, (kt != 0 || kk != 0) ? 1u : 0u);
          }
          commit<CG>(empty(s));
          cnt[1] = ++it;
          if (++s == S) { s = 0; ph ^= 1; }
        }
        if (ok) commit<CG>(tfull(acc));
      }
    }
  } else {
    if constexpr (kShift) regs_inc<104>();
    const int q = warp & 3, we = warp - kFirstEpi;
    // One set of warps reads every accumulator, or two sets one each.  64 columns of a tile
    // a warp, 16 rows of them at a time.
    constexpr int PARTS = C::GC / 64, TURNS = BACK ? 2 : SETS;
    static_assert(C::EW / SETS * TURNS == 8 * PARTS, "warps of a tile");
    const int set = SETS == 2 ? we / (C::EW / 2) : 0, ws = we - set * (C::EW / SETS);
    const int part = ws / 4 % PARTS, half = TURNS == 2 ? 0 : ws / 4 / PARTS;
    uint8_t* const bg = boxes + we * 3 * kBox;
    uint8_t* const bu = bg + kBox;
    uint8_t* const by = bu + kBox;
    const int I = p.I, J = p.J;
    auto row_of = [&](Tile x) { return (x.i * CG + (int)rank) * BM + q * 32 + 16 * half; };
    auto col_of = [&](Tile x) { return x.j * C::GC + part * 64; };
    uint32_t n = 0;      // accumulators read
    auto acc_of = [&](uint32_t k) { return SETS == 2 ? set : (int)(k & 1); };
    auto phase_of = [&](uint32_t k) { return (SETS == 2 ? k : k >> 1) & 1; };
    // the accumulator's columns are read: the MMAs may overwrite them
    auto release = [&]() {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (CG == 2) arrive_cluster(map_rank(tempty(acc_of(n)), 0));
        else mbar_arrive(tempty(acc_of(n)));
      }
    };
    // 16 rows of a box to where they belong (by TMA: after a fence).  A TMA store ends on
    // 16 bytes, not on the matrix's last column: a box that reaches past a width that is
    // no multiple of 8 is stored by hand, or it would overwrite what follows the row.
    auto leave = [&](uint8_t* box, const CUtensorMap* tm, bool tma, void* out, int64_t ld, int first_col, int row,
                     int col) {
      if (tma && (col + 64 <= J || (J & 7) == 0)) {
        if (lane == 0) tma_store_2d(tm, smem_u32(box), col, row);
      } else {
        box_store_slow(box, lane, out, ld, row, first_col + col, I, first_col + J, 16);
        fence_proxy_async_smem();      // (read by all lanes before TMA writes it again)
        __syncwarp();
      }
    };
    // this set's tiles
    const int u0 = group + set * groups, step = SETS * groups;
    auto next = [&](Tile y) { return SETS == 2 ? after(after(y)) : after(y); };
    Tile x = set ? after(first) : first;
    bool ok = true;
    if constexpr (!BACK) {
      for (int t = u0; t < p.units; t += step, x = next(x), ++n) {
        if (!wait_bar(tfull(acc_of(n)), phase_of(n), g)) break;
        tc_fence_after();
        const uint32_t at = tmem + (uint32_t)(acc_of(n) * C::BN + part * 64) + ((uint32_t)(q * 32 + 16 * half) << 16);
        const int col = col_of(x);
#pragma unroll 1
        for (int hr = 0; hr < TURNS; ++hr) {
          const int row = row_of(x) + 16 * hr;
          const bool there = row < I && col < J;
#pragma unroll
          for (int c = 0; c < 2; ++c) {      // 32 columns at a time
            uint32_t rg[16], ru[16];
            tmem_ld_16x32(at + (uint32_t)(32 * c) + ((uint32_t)(16 * hr) << 16), rg);
            tmem_ld_16x32(at + (uint32_t)(C::GC + 32 * c) + ((uint32_t)(16 * hr) << 16), ru);
            float2 b0[4], b1[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int c8 = col + 32 * c + 8 * i + 2 * (lane & 3);
              b0[i] = b1[i] = make_float2(0.f, 0.f);
              if (p.bias && there) {
                if (p.bias2 && col + 64 <= J) {
                  b0[i] = __ldg(reinterpret_cast<const float2*>(p.bias + c8));
                  b1[i] = __ldg(reinterpret_cast<const float2*>(p.bias + J + c8));
                } else {
                  b0[i] = bias_slow(p.bias, c8, J);
                  b1[i] = bias_slow(p.bias + J, c8, J);
                }
              }
            }
            tmem_wait16(rg);
            tmem_wait16(ru);
            if (hr == TURNS - 1 && c == 1) release();
            if (!there) continue;
            float2 vg[8], vu[8];      // [2 i + b]: column group i, row lane / 4 + 8 b
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              vg[k] = ffma2(make_float2(__uint_as_float(rg[2 * k]), __uint_as_float(rg[2 * k + 1])), both(1.f), b0[k / 2]);
              vu[k] = ffma2(make_float2(__uint_as_float(ru[2 * k]), __uint_as_float(ru[2 * k + 1])), both(1.f), b1[k / 2]);
            }
            auto pack = [&](const float2 (&v)[8], uint32_t (&w)[8]) {
#pragma unroll
              for (int k = 0; k < 8; ++k) w[k] = pack_bf16x2(v[k].x, v[k].y);
            };
            auto put = [&](uint8_t* box, const uint32_t (&w)[8]) {
              quad_put(box, lane, 4 * c, w);
              quad_put(box, lane, 4 * c + 2, w + 4);
            };
            uint32_t wg[8], wu[8], wy[8];
            pack(vg, wg);
            pack(vu, wu);
            act_all(p.act, vg);
#pragma unroll
            for (int k = 0; k < 8; ++k) vg[k] = fmul2(vg[k], vu[k]);
            pack(vg, wy);
            if (c == 0) {      // (the boxes: the last stores have read them)
              if (lane == 0) bulk_wait_read0();
              __syncwarp();
            }
            if (p.both) {
              put(bg, wg);
              put(bu, wu);
            }
            put(by, wy);
          }
          if (there) {
            fence_proxy_async_smem();
            __syncwarp();
            if (p.both) {
              leave(bg, &tmG, p.tma_both, p.both, p.ldboth, 0, row, col);
              leave(bu, &tmU, p.tma_both, p.both, p.ldboth, J, row, col);
            }
            leave(by, &tmY, p.tma_y, p.y, p.ldy, 0, row, col);
            if (lane == 0) bulk_commit();
          }
        }
      }
    } else {
      // A tile is two turns of 16 rows.  Turns that are off the matrix have no boxes; the
      // next one's pre-activations are sent when this one's results have left them.  (Not
      // fetched to L2 earlier, nor into a second pair of boxes; the latter costs two stages
      // of operands.  32,768 x 512 -> 2,048: 121 us; lines fetched a tile ahead 149 and two
      // ahead 164; second boxes 138, and 152 with both.)
      uint32_t sent = 0, in = 0;
      Tile sx = x;             // the turn to be sent for next
      int su = u0, sh = 0;
      auto send_next = [&]() {
        while (su < p.units) {
          const int row = row_of(sx) + 16 * sh, col = col_of(sx);
          if (++sh == 2) {
            sh = 0;
            su += step;
            sx = next(sx);
          }
          if (row >= I || col >= J) continue;
          if (lane == 0) {
            mbar_arrive_expect_tx(box_bar(we), 2 * kBox);
            tma_load_2d(smem_u32(bg), &tmP, col, row, box_bar(we));
            tma_load_2d(smem_u32(bu), &tmQ, col, row, box_bar(we));
          }
          ++sent;
          return;
        }
      };
      // a turn's pre-activations towards L2, half a row a lane (where they come by hand)
      auto ahead = [&](Tile y, int turn) {
        const int row = row_of(y) + 16 * turn + (lane & 15), col = col_of(y);
        if (row >= I || col >= J) return;
        const __nv_bfloat16* r = static_cast<const __nv_bfloat16*>(p.in) + (int64_t)row * p.ldin + col + (lane & 16 ? J : 0);
        prefetch_l2(r);
        prefetch_l2(r + min(63, J - 1 - col));
      };
      if (p.tma_in) send_next();
      for (int t = u0; t < p.units && ok; t += step, x = next(x), ++n) {
        if (!wait_bar(tfull(acc_of(n)), phase_of(n), g)) break;
        tc_fence_after();
        const uint32_t at = tmem + (uint32_t)(acc_of(n) * C::BN + part * 64) + ((uint32_t)(q * 32) << 16);
        const int col = col_of(x);
#pragma unroll 1
        for (int hr = 0; hr < 2; ++hr) {
          const int row = row_of(x) + 16 * hr;
          const bool there = row < I && col < J;
          if (there) {
            if (p.tma_in) {
              ok = wait_bar(box_bar(we), in & 1, g);
            } else {
              if (lane == 0) bulk_wait_read0();
              __syncwarp();
              box_load_slow(bg, lane, p.in, p.ldin, row, col, I, J, 16);
              box_load_slow(bu, lane, p.in, p.ldin, row, J + col, I, 2 * (int64_t)J, 16);
              ahead(hr == 0 ? x : next(x), hr ^ 1);
              __syncwarp();
            }
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            if (p.tma_in) ++in;
          }
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t rd[16];
            tmem_ld_16x32(at + (uint32_t)(32 * c) + ((uint32_t)(16 * hr) << 16), rd);
            uint32_t wg[8], wu[8], wy[8];
            if (there) {
#pragma unroll
              for (int i = 0; i < 4; i += 2) {
                quad_get(bg, lane, 4 * c + i, wg + 2 * i);
                quad_get(bu, lane, 4 * c + i, wu + 2 * i);
              }
            }
            tmem_wait16(rd);
            if (hr == 1 && c == 1) release();
            if (!there) continue;
            float2 d[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
              d[k] = make_float2(__uint_as_float(rd[2 * k]), __uint_as_float(rd[2 * k + 1]));
            grad_all(p.act, d, wg, wu, wy);
            __syncwarp();   // all have read these columns
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
              quad_put(bg, lane, 4 * c + i, wg + 2 * i);
              quad_put(bu, lane, 4 * c + i, wu + 2 * i);
              if (p.y) quad_put(by, lane, 4 * c + i, wy + 2 * i);
            }
          }
          if (there) {
            fence_proxy_async_smem();
            __syncwarp();
            leave(bg, &tmG, p.tma_both, p.both, p.ldboth, 0, row, col);
            leave(bu, &tmU, p.tma_both, p.both, p.ldboth, J, row, col);
            if (p.y) leave(by, &tmY, p.tma_y, p.y, p.ldy, 0, row, col);
            if (lane == 0) bulk_commit();
          }
          if (lane == 0) bulk_wait_read0();
          if (p.tma_in && sent == in) send_next();
          __syncwarp();
        }
      }
      // boxes that were sent for but not used (after an abort)
      if (p.tma_in && lane == 0 && *abort_flag && sent != in) drain_wait(box_bar(we), in & 1, 1000000ull);
    }
    if (lane == 0) bulk_wait0();   // this warp's stores are complete before the CTA exits
  }

  __syncthreads();
  if (rank == 0 && *abort_flag) {
    // loads issued by this CTA (and, with it, the other one) but never
    // consumed, and outstanding MMAs
    if (threadIdx.x == 0) {
      const uint32_t issued = cnt[0], consumed = cnt[1];
      for (uint32_t it = consumed; it < issued; ++it)
        drain_wait(full(it % S), (it / S) & 1, kWaitNs);
    }
    if (warp == 1 && lane == 0) {
      if constexpr (CG == 1) {
        tc_commit(drain);
      } else {
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(drain)
            : "memory");
      }
      drain_wait(drain, 0, kWaitNs);
    }
    __syncthreads();
  }
  if (rank == 1 && *abort_flag) {
    // the odd CTA's loads complete on the other CTA's barriers: let them land
    const uint64_t t0 = globaltimer();
    while (globaltimer() - t0 < 1000000ull) {
    }
  }
  if constexpr (CG == 2) cluster_sync();   // neither CTA leaves while the other still uses it
  if (warp == 1) {
    tc_fence_after();
    dealloc<CG>(tmem, C::TMEM);
  }
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

template <int CG, bool BACK, int SETS>
cudaError_t launch(const Product& m, const Gate& gate, int* err, int sms, cudaStream_t st) {
  using C = Cfg<CG, BACK>;
  const int64_t I = gate.M, J = gate.N;
  TcArgs p{};
  p.I = (int)I;
  p.J = (int)J;
  p.tiles_i = (int)cdiv(I, CG * BM);
  p.tiles_j = (int)cdiv(J, C::GC);
  p.k_tiles = (int)cdiv(m.R, BK);
  p.units = p.tiles_i * p.tiles_j;
  p.act = gate.act;
  p.bias = gate.bias;
  p.bias2 = J % 2 == 0;
  p.both = BACK ? gate.dp : gate.pre;
  p.ldboth = BACK ? gate.lddp : gate.ldpre;
  p.y = gate.y;
  p.ldy = gate.ldy;
  p.in = gate.pre_in;
  p.ldin = gate.ldin;
  p.err = err;
  auto al = [](const void* q, int64_t ld) { return q && ops::al16(q) && ld % 8 == 0; };
  p.tma_both = al(p.both, p.ldboth) && J % 8 == 0;      // (the second half starts at column J)
  p.tma_y = al(p.y, p.ldy);
  p.tma_in = BACK && al(p.in, p.ldin) && J % 8 == 0;
  CUtensorMap ta, tb;
  cudaError_t e = tc_make_tmap(&ta, m.A, m.R, I, m.sai, BK, BM);
  if (e != cudaSuccess) return e;
  if (BACK) e = tc_make_tmap(&tb, m.B, J, m.R, m.sbr, 64, BK);
  else e = tc_make_tmap(&tb, m.B, m.R, 2 * J, m.sbj, BK, C::GC);
  if (e != cudaSuccess) return e;
  CUtensorMap tg = ta, tu = ta, ty = ta, tp = ta, tq = ta;
  auto box = [&](CUtensorMap* t, const void* at, int64_t ld) {
    if (e == cudaSuccess) e = tc_make_tmap(t, at, J, I, ld, 64, 16);
  };
  auto second = [&](const void* at) { return static_cast<const __nv_bfloat16*>(at) + J; };
  if (p.tma_both) {
    box(&tg, p.both, p.ldboth);
    box(&tu, second(p.both), p.ldboth);
  }
  if (p.tma_y) box(&ty, p.y, p.ldy);
  if (p.tma_in) {
    box(&tp, p.in, p.ldin);
    box(&tq, second(p.in), p.ldin);
  }
  if (e != cudaSuccess) return e;
  const auto kernel = glin_tc_kernel<CG, BACK, SETS>;
  static thread_local int prepared = -1;   // the device whose shared-memory opt-in is made
  int dev = 0;
  e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (prepared != dev) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM);
    if (e != cudaSuccess) return e;
    prepared = dev;
  }
  const int64_t groups = std::min<int64_t>(p.units, sms / CG);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(groups * CG));
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CG;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CG == 2 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, ta, tb, tg, tu, ty, tp, tq, p);
}

}  // namespace

int fused_pairs(bool back, int64_t M, int64_t N, int64_t R) {
  constexpr int kSms = 152;
  const int64_t kt = cdiv(R, BK);
  // sums that long drift in the accumulator, and are taken out piece by piece elsewhere
  if (R > 1ll << 16 || cdiv(M, BM) * cdiv(N, 64) > (1ll << 30)) return 0;
  int best = 0;
  double cost = 0;
  for (int cg = 1; cg <= 2; ++cg) {
    const int gc = (cg == 2 ? 256 : 128) / (back ? 1 : 2);
    const int64_t rounds = cdiv(cdiv(M, cg * BM) * cdiv(N, gc), kSms / cg);
    const double c = rounds * (kt * (cg == 2 ? 0.30 : 0.20) + 2.0);
    if (best == 0 || c < cost) {
      best = cg;
      cost = c;
    }
  }
  // partial products: a launch more, and the sums written and read once more
  const int64_t J = back ? N : 2 * N;
  const lin::TcPlan plan = lin::tc_plan(M, J, R, true);
  const int64_t units = cdiv(M, plan.cg * BM) * cdiv(J, plan.cg == 2 ? 256 : 128) * plan.splits;
  const double split = cdiv(units, kSms / plan.cg) * (plan.kt_per_split * (plan.cg == 2 ? 0.30 : 0.20) + 2.0) + 3.0 +
                       (double)(plan.splits + 1) * M * J * 8 / 5e6;
  return cost <= split ? best : 0;
}

cudaError_t fused_forward(const Product& m, const Gate& g, int pairs, int* err, int sms, cudaStream_t st) {
  // Two sets of epilogue warps where pre goes out too and there are tiles enough: while one
  // waits (for TMEM, a fence, its stores) the other computes.  32,768 x 512 -> 2,048 with
  // pre 121 us with one set and 109 with two, without 89 and 90; 2,048 x 512 -> 2,048 14.2 and 14.8.
  // (of rows that TMA cannot store, one: 10,007 x 1,397 -> 1,001 82 us and 96.)
  if (pairs == 2 && g.pre && ops::al16(g.pre) && g.ldpre % 8 == 0 && g.N % 8 == 0 && cdiv(g.M, 2 * BM) * cdiv(g.N, 128) >= 4 * (sms / 2))
    return launch<2, false, 2>(m, g, err, sms, st);
  return pairs == 2 ? launch<2, false, 1>(m, g, err, sms, st) : launch<1, false, 1>(m, g, err, sms, st);
}
cudaError_t fused_backward(const Product& m, const Gate& g, int pairs, int* err, int sms, cudaStream_t st) {
  return pairs == 2 ? launch<2, true, 1>(m, g, err, sms, st) : launch<1, true, 1>(m, g, err, sms, st);
}

}  // namespace glin
}  // namespace ppo
