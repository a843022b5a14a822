// Layer norm: parameters of the launchers in norm.hip.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace ttt {

struct NormParams {
  const void *x, *gy;               // [n][ld] rows of `groups` groups of `width` columns
  int64_t ldx, ldgy;
  const float *gamma, *beta;        // [width]; null: 1, 0
  float eps;
  int64_t n;
  int groups, width;
  void *y;                          // the output, or the gradient of x
  int64_t ldy;
  float *ggamma, *gbeta;            // [width], each may be null
  float *part;                      // [norm_grid][2][width]
};

constexpr int kNormMaxWidth = 8192;
int norm_grid(int64_t vectors, int width);      // vectors: rows x groups
hipError_t launch_norm(const NormParams &p, bool bf16, hipStream_t s);
hipError_t launch_norm_backward(const NormParams &p, bool bf16, hipStream_t s);

}  // namespace ttt
