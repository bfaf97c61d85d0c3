// linear.h -- internal interface of the matrix products with fused epilogues.
#pragma once

#include "common.cuh"

namespace ppo {
namespace lin {

// out(i, j) = sum_r A(i, r) B(j, r), i < I, j < J, r < R, with
// A(i, r) = A[i * sai + r * sar] and B(j, r) = B[j * sbj + r * sbr].
struct Product {
  const void* A;
  int64_t sai, sar;
  const void* B;
  int64_t sbj, sbr;
  int64_t I, J, R;
};

enum Mode : int { kForward = 0, kData = 1, kWeight = 2 };

// What happens to a finished sum v at (i, j):
//   kForward  v + bias[j] -> pre (nullable), act(v) + res -> out
//   kData     v act'(pre[i][j]) + res -> out
//   kWeight   v (+ out) -> out, fp32
struct Epilogue {
  int mode, act, accumulate;
  const float* bias;
  const void* res;
  int64_t ldres;
  void* pre;
  int64_t ldpre;
  void* out;
  int64_t ldo;
};

// ---- tensor-core products (bf16, linear_tc.cu) ------------------------------------
// A product whose rows (A(i, .), B(j, .), or for the weight gradient A(., r),
// B(., r)) start on 16-byte boundaries.
struct TcPlan {
  int cg;              // CTAs of an output tile: 1 (128 x 128) or 2 (256 x 256)
  int kt_per_split;    // 64-deep steps of the sum per split
  int splits;
};
TcPlan tc_plan(int64_t I, int64_t J, int64_t R, bool must_split);
bool tc_fits(const Product& g);
// Rows of partial column sums that the weight gradient's kernel leaves.
int64_t tc_sum_rows(const Product& g, const TcPlan& plan);
// part: [splits][I][J rounded up to 4] for split products (the epilogue is
// then finish_kernel's), else nullptr; db_part (kWeight, nullable):
// [tc_sum_rows][I], sums over r of A
cudaError_t tc_product(const Product& g, const Epilogue& e, const TcPlan& plan, float* part,
                       float* db_part, int* err, int sms, cudaStream_t st);

}  // namespace lin

// fp32 [splits][rows][cols] with row pitch ld (a multiple of 4) as 32-column x
// 32-row x 1-split boxes, 128-byte swizzle (gemm_tc.cu)
cudaError_t tc_make_tmap_f32(CUtensorMap* m, float* base, int64_t cols, int64_t rows,
                             int64_t splits, int64_t ld);
}  // namespace ppo
