// Gated residual tail of a block: parameters of the launchers in residual.hip.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace ttt {

struct ResidualParams {
  const void *x, *o, *z;            // [n][ld] rows of `channels`; z may be null (no gate)
  int64_t ldx, ldo, ldz;
  const float *gamma, *alpha, *gamma_next;   // [channels]; null: 1 (gamma_next null: no h)
  float eps;
  int64_t n;
  int channels, norm;               // norm: width of the groups that o is normalised over
  void *y, *h;
  int64_t ldy, ldh;
  // backward (x unused, y is the forward's output)
  const void *gy, *gh;
  int64_t ldgy, ldgh;
  void *gx, *go, *gz;
  int64_t ldgx, ldgo, ldgz;
  float *ggamma, *galpha, *ggamma_next;      // [channels], each may be null
  float *part;                      // [residual_grid][2][channels]
};

constexpr int kResidualMaxChannels = 8192;
int residual_grid(int64_t n, int channels);
hipError_t launch_residual(const ResidualParams &p, bool bf16, hipStream_t s);
hipError_t launch_residual_backward(const ResidualParams &p, bool bf16, hipStream_t s);

}  // namespace ttt
