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

}  // namespace lin
}  // namespace ppo
