// ops.cuh -- what the context-free operators (layer norm, gated scan, linear)
// share: argument checks, the device's SM count, element loads and the
// activations.
#pragma once

#include "common.cuh"

namespace ppo {
namespace ops {

inline bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool dtype_ok(int32_t d) { return d == PPO_DTYPE_F32 || d == PPO_DTYPE_BF16; }
inline int esize(int32_t d) { return d == PPO_DTYPE_F32 ? 4 : 2; }
// a matrix of `rows` rows, pitch ld, whose byte offsets fit in 63 bits
inline bool extent_ok(int64_t rows, int64_t ld, int64_t row) {
  return rows >= 1 && row >= 1 && ld >= row && ld < (1ll << 40) && rows < (1ll << 40) &&
         rows <= (1ll << 59) / ld;
}

// A call's status.  The runtime remembers the error of a refused launch or query:
// it is dropped here, or the next call's launch check would report it.
inline ppo_status status_of(cudaError_t e) {
  if (e == cudaSuccess) return PPO_OK;
  cudaGetLastError();
  return PPO_ERR_CUDA;
}

// SM count of the current device (0 without a device); one query per device
inline int num_sms() {
  static int cached[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  const bool slot = dev >= 0 && dev < 64;
  if (slot && cached[dev] > 0) return cached[dev];
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  if (slot) cached[dev] = n;
  return n;
}

// V elements of type T as one load or store of their size
template <int BYTES> struct RawOf;
template <> struct RawOf<2> { using type = uint16_t; };
template <> struct RawOf<4> { using type = uint32_t; };
template <> struct RawOf<8> { using type = uint2; };
template <> struct RawOf<16> { using type = uint4; };
template <typename T, int V> using Raw = typename RawOf<(int)sizeof(T) * V>::type;

template <typename T, int V>
__device__ __forceinline__ void to_f32(const Raw<T, V>& r, float (&f)[V]) {
  T v[V];
  static_assert(sizeof(v) == sizeof(r), "element vector");
  memcpy(v, &r, sizeof(r));
#pragma unroll
  for (int i = 0; i < V; ++i) f[i] = (float)v[i];
}
__device__ __forceinline__ void round_to(float f, float& o) { o = f; }
__device__ __forceinline__ void round_to(float f, __nv_bfloat16& o) { o = __float2bfloat16_rn(f); }
template <typename T, int V>
__device__ __forceinline__ Raw<T, V> from_f32(const float (&f)[V]) {
  T v[V];
#pragma unroll
  for (int i = 0; i < V; ++i) round_to(f[i], v[i]);
  Raw<T, V> r;
  memcpy(&r, v, sizeof(r));
  return r;
}

// Elements e .. e + n - 1 (n <= 8) of `base` (on 16 bytes), wherever e lies, zeros
// after them: the one or two aligned 16-byte pieces that hold them, shifted.
// Nothing past the first `total` elements is read.
__device__ __forceinline__ uint4 load8_any(const __nv_bfloat16* base, int64_t e, int64_t total, int n) {
  if (n <= 0) return make_uint4(0, 0, 0, 0);
  const int64_t a = e & ~7ll;
  const int sh = (int)(e & 7);
  const bool more = sh + n > 8;
  uint32_t w[8] = {};
  if (a + (more ? 16 : 8) <= total) {
    const uint4 x = *reinterpret_cast<const uint4*>(base + a);
    w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
    if (more) {
      const uint4 y = *reinterpret_cast<const uint4*>(base + a + 8);
      w[4] = y.x; w[5] = y.y; w[6] = y.z; w[7] = y.w;
    }
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = sh & 4 ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = sh & 2 ? w[i + 1] : w[i];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = sh & 1 ? __funnelshift_r(w[i], w[i + 1], 16) : w[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) w[i >> 1] |= (uint32_t)__bfloat16_as_ushort(base[e + i]) << (16 * (i & 1));
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = 2 * i + 2 <= n ? w[i] : 2 * i < n ? w[i] & 0xffffu : 0u;
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Activations and their derivatives at the pre-activation x (codes of
// ppo_activation).  x sigmoid(u) has no cancellation where it is small, unlike
// 0.5 x (1 + tanh(u / 2)).  __expf is off by 2 + 1.2 |x| units in the last place
// and __fdividef by 2: a sigmoid by 1e-6 of itself for |x| < 10, in fp32 results too.
__device__ __forceinline__ float sigmoid_f(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }
constexpr float kGeluU = 1.5957691216057308f;   // 2 sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;
// From x^2 = 256 on gelu's slope is 0 or 1 to fp32's digits: the polynomial beside
// q (1 - q) = 0 stays finite there.  (x q comes first, so that -x is not multiplied
// by it either; a NaN comes through q.)
constexpr float kGeluTop = 256.f;

// FAST: tanh by the hardware approximation (error 2^-11 of its value), for results
// that are rounded to bf16 (2^-9) next.  Products that are split or of a few rows take
// tanhf: a layer's bf16 results may differ by one rounding between a rollout and an
// acting step.
template <bool FAST>
__device__ __forceinline__ float act_value(int act, float x) {
  switch (act) {
    case PPO_ACT_TANH: return FAST ? tanh_fast(x) : tanhf(x);
    case PPO_ACT_RELU: return x > 0.f ? x : (x != x ? x : 0.f);
    case PPO_ACT_SILU: return x * sigmoid_f(x);
    case PPO_ACT_GELU: return x * sigmoid_f(kGeluU * (x + kGeluA * x * x * x));
  }
  return x;
}
template <bool FAST>
__device__ __forceinline__ float act_slope(int act, float x) {
  switch (act) {
    case PPO_ACT_TANH: {
      // 1 - tanh^2 = 4 s (1 - s), s = sigmoid(2 x): no cancellation at large |x|
      const float e = __expf(-2.f * fabsf(x)), r = __fdividef(1.f, 1.f + e);
      return 4.f * e * r * r;
    }
    case PPO_ACT_RELU: return x > 0.f ? 1.f : 0.f;
    case PPO_ACT_SILU: {
      const float q = sigmoid_f(x);
      return q * (1.f + x * (1.f - q));
    }
    case PPO_ACT_GELU: {
      const float q = sigmoid_f(kGeluU * (x + kGeluA * x * x * x));
      return q + x * q * (1.f - q) * kGeluU * (1.f + 3.f * kGeluA * fminf(x * x, kGeluTop));
    }
  }
  return 1.f;
}
inline bool act_ok(int32_t a) { return a >= PPO_ACT_NONE && a <= PPO_ACT_GELU; }

}  // namespace ops
}  // namespace ppo
