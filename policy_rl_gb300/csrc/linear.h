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
constexpr int kSumStep = 64;
struct TcPlan {
  int cg;              // CTAs of an output tile: 1 (128 x 128) or 2 (256 x 256)
  int kt_per_split;    // 64-deep steps of the sum per split
  int splits;
};
// terms: products of bf16 planes that make one product (fp32 operands: kTerms)
constexpr int kTerms = 6;
TcPlan tc_plan(int64_t I, int64_t J, int64_t R, bool must_split, int terms = 1);
// Row pitch of partial products: rows start on 32-byte boundaries.
__host__ __device__ constexpr int64_t part_pitch(int64_t J) { return (J + 7) / 8 * 8; }
// Rows of partial column sums that the weight gradient's kernel leaves.
int64_t tc_sum_rows(const Product& g, const TcPlan& plan);
// part: [splits][I][part_pitch(J)] for split products (the epilogue is
// then finish_kernel's), else nullptr; db_part (kWeight, nullable):
// [tc_sum_rows][I], sums over r of A.  plane_a, plane_b: the operands are three
// planes of that many rows each (a multiple of 64, zeros past the operand's),
// one below the other, whose sum is the fp32 operand; part is then required.
cudaError_t tc_product(const Product& g, const Epilogue& e, const TcPlan& plan, float* part,
                       float* db_part, int* err, int sms, cudaStream_t st, int64_t plane_a = 0,
                       int64_t plane_b = 0);

// ---- what other products share (linear.cu) ------------------------------------------
// A matrix that is copied, and the blocks that do it.  A product's two operands
// take one launch (2,000 x 130 -> 250 forward: 15 us, 21 with a launch each).
struct Copy {
  const void* src;
  int64_t ld, rows, cols, pitch, rows_pad;
  uint4* dst;
  int blocks;
};
int64_t pitch8(int64_t cols);
// Workspace of a bf16 operand's copy onto 16-byte rows (0 where it needs none).
size_t packed_bytes(int64_t rows, int64_t cols, int64_t ld);
// the operand itself, or its copy in the workspace (advanced past it)
Copy on_16_bytes(const void*& a, int64_t& ld, int64_t rows, int64_t cols, char*& work);
cudaError_t pack(const Copy& a, const Copy& b, cudaStream_t st);
// Bytes of a product's partial products (0 where its tiles are finished at once).
size_t tc_part_bytes(int64_t I, int64_t J, int64_t R, bool must_split, int terms = 1);
bool sizes_ok(int64_t M, int64_t N, int64_t K);
// Sums of a product in `splits` parts, `stride` apart, of rows of pitch ldp, each of
// r_per_split terms.
struct PartialSums {
  const float* part;
  int splits;
  int64_t stride, ldp, r_per_split;
};
// Whether an fp32 product is taken by planes; its sums so (forward and data gradient), and
// the workspace for operands of ra x ca and rb x cb.
bool takes_planes(int mode, int64_t M, int64_t N, int64_t K);
cudaError_t planes_sums(const Product& g, int mode, char* work, int* err, cudaStream_t st, PartialSums* out);
size_t planes_need(int64_t ra, int64_t ca, int64_t rb, int64_t cb, int64_t I, int64_t J, int64_t R);

}  // namespace lin
}  // namespace ppo
