// lin_again.cuh -- the second look at sums of products of planes (linear.cu,
// glinear.cu).
#pragma once

#include "linear.h"

namespace ppo {
namespace lin {
namespace {

// Of a product of planes: where the sum of an element's parts is not finite, each part
// that is not either is computed again, straight from the fp32 operands.  (The planes of
// an infinity, or of what rounds to one in bf16, do not add up: their products hold NaN
// where the product may not.)  Eight steps' loads are in flight: an infinity among
// 1,000,000 rows of a weight gradient takes 18 ms, 2 s a step at a time over the
// whole sum.  A part that has become NaN ends early.
struct Again {
  Product g;              // the fp32 operands
  const float* part;
  int64_t pitch;          // of the parts
  int splits;
  int64_t r_per_split;
};
__device__ __noinline__ float dot_again(const Again* __restrict__ p, int64_t i, int64_t j, int64_t at) {
  constexpr int U = 8;
  const int64_t sar = p->g.sar, sbr = p->g.sbr;
  float sum = 0.f;
  for (int s = 0; s < p->splits; ++s) {
    float v = __ldcg(p->part + s * p->pitch + at);
    if (!isfinite(v)) {
      v = 0.f;
      const int64_t r0 = s * p->r_per_split;
      const float* a = static_cast<const float*>(p->g.A) + i * p->g.sai + r0 * sar;
      const float* b = static_cast<const float*>(p->g.B) + j * p->g.sbj + r0 * sbr;
      int64_t n = min(p->g.R - r0, p->r_per_split);
      for (; n >= U && v == v; n -= U) {
        float x[U], y[U];
#pragma unroll
        for (int u = 0; u < U; ++u, a += sar, b += sbr) {
          x[u] = __ldg(a);
          y[u] = __ldg(b);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) v = fmaf(x[u], y[u], v);
      }
      for (; n > 0 && v == v; --n, a += sar, b += sbr) v = fmaf(__ldg(a), __ldg(b), v);
    }
    sum += v;
  }
  return sum;
}

}  // namespace
}  // namespace lin
}  // namespace ppo
