// glinear.h -- internal interface of the gated linear layers.
#pragma once

#include "linear.h"

namespace ppo {
namespace glin {

// What the sums of element (i, j) of the gated width go into.
struct Gate {
  int act;
  const float* bias;       // [2N] (nullable)
  const void* pre_in;      // backward: [M][2N]
  int64_t ldin;
  void* pre;               // forward: [M][2N] (nullable)
  int64_t ldpre;
  void* dp;                // backward: [M][2N]
  int64_t lddp;
  void* y;                 // [M][N] (backward: nullable)
  int64_t ldy;
  int64_t M, N;
  lin::PartialSums s;
};

// bf16 in one kernel (glinear_tc.cu), operands on 16-byte rows: A is x [M][R] or dz,
// B W [2N][R] (forward) or W2 [R][N] (backward).
// CTAs of a tile (1 or 2) that suit a product best, 0 where partial products do.
int fused_pairs(bool back, int64_t M, int64_t N, int64_t R);
cudaError_t fused_forward(const lin::Product& m, const Gate& g, int pairs, int* err, int sms, cudaStream_t st);
cudaError_t fused_backward(const lin::Product& m, const Gate& g, int pairs, int* err, int sms, cudaStream_t st);
// bf16 forward of up to 64 rows (glinear_skinny.cu): CTAs that share a sum, 0 where it does
// not apply.
int skinny_ctas(int64_t M, int64_t N, int64_t R);
cudaError_t skinny_forward(const lin::Product& m, const Gate& g, int ctas, int* err, cudaStream_t st);

}  // namespace glin
}  // namespace ppo
