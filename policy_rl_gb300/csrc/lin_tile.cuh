// lin_tile.cuh -- pieces of the tensor-core products with fused epilogues
// (linear_tc.cu, glinear_tc.cu): CTA pairs, boxes of results in shared memory, reads
// of accumulators as 8 x 8 matrices, packed activations.
#pragma once

#include "linear.h"
#include "ops.cuh"
#include "tc_tile.cuh"

namespace ppo {
namespace lin {
namespace {

using namespace ptx;
using ppo::tc::Guard;
using ppo::tc::drain_wait;
using ppo::tc::wait_bar;

constexpr uint64_t kWaitNs = 2000000000ull;
constexpr int BM = 128, BK = kSumStep;

__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Relaxed: what it tells the other CTA is that this warp's TMEM loads have
// completed (they have, before it is issued); no memory is handed over.
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// TMA load whose completion counts on the even CTA's barrier
template <int CG>
__device__ __forceinline__ void load_2d(uint32_t dst, const void* tmap, int x, int y, uint32_t bar) {
  if constexpr (CG == 1) {
    tma_load_2d(dst, tmap, x, y, bar);
  } else {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"((uint64_t)tmap), "r"(x), "r"(y), "r"(bar)
        : "memory");
  }
}
template <int CG>
__device__ __forceinline__ void alloc(uint32_t slot, uint32_t ncols) {
  if constexpr (CG == 1) {
    tmem_alloc(slot, ncols);
  } else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot),
                 "r"(ncols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
}
template <int CG>
__device__ __forceinline__ void dealloc(uint32_t taddr, uint32_t ncols) {
  if constexpr (CG == 1) {
    tmem_dealloc(taddr, ncols);
  } else {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols)
                 : "memory");
  }
}
// arrives on `bar` (of both CTAs of a pair) when this thread's MMAs are done
template <int CG>
__device__ __forceinline__ void commit(uint32_t bar) {
  if constexpr (CG == 1) {
    tc_commit(bar);
  } else {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
        " [%0], %1;" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
  }
}
template <int CG>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                    uint32_t accumulate) {
  if constexpr (CG == 1) {
    tc_mma_bf16(d, a, b, idesc, accumulate);
  } else {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
  }
}

// Piece c (16 bytes) of row r of a box.
__device__ __forceinline__ uint8_t* box_piece(uint8_t* box, int r, int c) {
  return box + r * 128 + ((c ^ (r & 7)) << 4);
}
// Boxes that TMA cannot move (rows off 16-byte boundaries).  Loads: lane l of a
// warp takes the 16-byte piece l % 8 of rows l / 8, l / 8 + 4, ..  (Not inlined:
// rare, and the code would only be in the way.)
__device__ __noinline__ void box_load_slow(uint8_t* box, int lane, const void* base, int64_t ld,
                                           int64_t row0, int64_t col0, int64_t I, int64_t J,
                                           int rows) {
  const int64_t col = col0 + (lane & 7) * 8, total = (I - 1) * ld + J;
  const int n = (int)max((int64_t)0, min((int64_t)8, J - col));
  for (int r = lane >> 3; r < rows; r += 4)
    *reinterpret_cast<uint4*>(box_piece(box, r, lane & 7)) =
        ops::load8_any(static_cast<const __nv_bfloat16*>(base), (row0 + r) * ld + col, total,
                       row0 + r < I ? n : 0);
}
// Stores: a row at a time, in aligned pairs.  A row that starts on an odd element
// is stored one element further on, its first and last elements alone (30,000 x
// 33 -> 4,001 with gelu and pre: 303 us; 864 element by element; 115 for 40 ->
// 4,000, whose boxes TMA moves).
__device__ __noinline__ void box_store_slow(uint8_t* box, int lane, void* base, int64_t ld,
                                            int64_t row0, int64_t col0, int64_t I, int64_t J,
                                            int rows) {
  const int n = (int)min((int64_t)64, J - col0), last = (int)min((int64_t)rows, I - row0);
  for (int r = 0; r < last; ++r) {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(box_piece(box, r, lane >> 2) + (lane & 3) * 4);
    const uint32_t next = __shfl_down_sync(0xffffffffu, w, 1);
    __nv_bfloat16* p = static_cast<__nv_bfloat16*>(base) + (row0 + r) * ld + col0;
    const int odd = (int)(reinterpret_cast<uintptr_t>(p) >> 1) & 1;
    const int c = 2 * lane + odd;      // this lane's pair: elements c and c + 1
    const uint32_t v = odd ? __funnelshift_r(w, next, 16) : w;
    if (c + 1 < n) *reinterpret_cast<uint32_t*>(p + c) = v;
    else if (c < n) p[c] = __ushort_as_bfloat16((uint16_t)v);
    if (odd && lane == 0) p[0] = __ushort_as_bfloat16((uint16_t)w);
  }
}

// 16 TMEM lanes x 64 fp32 columns: thread t gets, of every group i of 8 columns,
// columns 2 (t % 4) and + 1 of rows t / 4 (r[4 i], r[4 i + 1]) and t / 4 + 8
// (r[4 i + 2], r[4 i + 3]) -- the layout of 8 x 8 matrices of stmatrix, and one
// in which a thread meets 16 of the 64 columns, so that it needs 16 biases (in
// rows of 64 columns a thread, the broadcast loads of 64 cost 12 % of the
// forward product: shared memory and L1 are busy with the operands).
__device__ __forceinline__ void tmem_ld_16x64(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
  tmem_wait_ld(r);
}
// Four 8 x 8 matrices: rows 0..7 and 8..15 of column groups i and i + 1 of half
// a box (16 rows of 128 bytes).
__device__ __forceinline__ uint32_t quad_addr(uint8_t* half, int lane, int i) {
  const int m = lane >> 3;
  return smem_u32(box_piece(half, (m & 1) * 8 + (lane & 7), i + (m >> 1)));
}
__device__ __forceinline__ void quad_put(uint8_t* half, int lane, int i, const uint32_t* w) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(
                   quad_addr(half, lane, i)),
               "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
               : "memory");
}
__device__ __forceinline__ void quad_get(uint8_t* half, int lane, int i, uint32_t* w) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
               : "r"(quad_addr(half, lane, i))
               : "memory");
}
template <int N>
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
// bias[c], bias[c + 1], zeros past J
__device__ __noinline__ float2 bias_slow(const float* b, int64_t c, int64_t J) {
  return make_float2(c < J ? b[c] : 0.f, c + 1 < J ? b[c + 1] : 0.f);
}

// Activations of a pair of values, the multiplications and additions packed.
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 ex2_pair(float2 u) {
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(u.x) : "f"(u.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(u.y) : "f"(u.y));
  return u;
}
__device__ __forceinline__ float2 rcp_pair(float2 u) {
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(u.x) : "f"(u.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(u.y) : "f"(u.y));
  return u;
}
constexpr float kLog2e = 1.4426950408889634f;
// q = sigmoid(u), u = x (silu) or 2 sqrt(2/pi) (x + 0.044715 x^3) (gelu); e = 2^(-u log2 e)
template <int ACT>
__device__ __forceinline__ void gate_pair(float2 x, float2& q, float2& e, float2& x2) {
  float2 u;
  if constexpr (ACT == PPO_ACT_GELU) {
    x2 = fmul2(x, x);
    u = fmul2(x, ffma2(x2, both(-kLog2e * ops::kGeluU * ops::kGeluA), both(-kLog2e * ops::kGeluU)));
  } else {
    u = fmul2(x, both(-kLog2e));
  }
  e = ex2_pair(u);
  q = rcp_pair(ffma2(e, both(1.f), both(1.f)));
}
template <int ACT>
__device__ __forceinline__ float2 act_pair(float2 x) {
  if constexpr (ACT == PPO_ACT_SILU || ACT == PPO_ACT_GELU) {
    float2 q, e, x2;
    gate_pair<ACT>(x, q, e, x2);
    return fmul2(x, q);
  }
  return make_float2(ops::act_value<true>(ACT, x.x), ops::act_value<true>(ACT, x.y));
}
template <int ACT>
__device__ __forceinline__ float2 slope_pair(float2 x) {
  if constexpr (ACT == PPO_ACT_SILU || ACT == PPO_ACT_GELU) {
    // q + x q (1 - q) u'
    float2 q, e, x2;
    gate_pair<ACT>(x, q, e, x2);
    float2 t = ffma2(q, both(-1.f), both(1.f));
    if constexpr (ACT == PPO_ACT_GELU)
      t = fmul2(t, ffma2(make_float2(fminf(x2.x, ops::kGeluTop), fminf(x2.y, ops::kGeluTop)),
                         both(3.f * ops::kGeluU * ops::kGeluA), both(ops::kGeluU)));
    return ffma2(fmul2(x, q), t, q);
  }
  return make_float2(ops::act_slope<true>(ACT, x.x), ops::act_slope<true>(ACT, x.y));
}
template <int ACT>
__device__ __forceinline__ void act_chunk(float2 (&v)[16]) {
#pragma unroll
  for (int k = 0; k < 16; ++k) v[k] = act_pair<ACT>(v[k]);
}
__device__ __forceinline__ void act_chunk(int act, float2 (&v)[16]) {
  switch (act) {
    case PPO_ACT_TANH: act_chunk<PPO_ACT_TANH>(v); break;
    case PPO_ACT_RELU: act_chunk<PPO_ACT_RELU>(v); break;
    case PPO_ACT_SILU: act_chunk<PPO_ACT_SILU>(v); break;
    case PPO_ACT_GELU: act_chunk<PPO_ACT_GELU>(v); break;
    default: break;
  }
}
template <int ACT>
__device__ __forceinline__ void slope_chunk(const uint32_t (&aux)[16], float2 (&v)[16]) {
#pragma unroll
  for (int k = 0; k < 16; ++k) v[k] = fmul2(v[k], slope_pair<ACT>(unpack_bf16x2(aux[k])));
}
__device__ __forceinline__ void slope_chunk(int act, const uint32_t (&aux)[16], float2 (&v)[16]) {
  switch (act) {
    case PPO_ACT_TANH: slope_chunk<PPO_ACT_TANH>(aux, v); break;
    case PPO_ACT_RELU: slope_chunk<PPO_ACT_RELU>(aux, v); break;
    case PPO_ACT_SILU: slope_chunk<PPO_ACT_SILU>(aux, v); break;
    case PPO_ACT_GELU: slope_chunk<PPO_ACT_GELU>(aux, v); break;
    default: break;
  }
}
__device__ __forceinline__ void store_32b(void* p, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
__device__ __forceinline__ void prefetch_l2(const void* p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}
template <int N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

}  // namespace
}  // namespace lin
}  // namespace ppo
