// AdamW over many tensors: parameters of the launcher in adamw.hip.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "ttt.h"

namespace ttt {

constexpr int kAdamwBlock = 256;    // elements that share a scale of 8-bit states
constexpr int kAdamwTensors = 48;   // tensors of one launch: their table is a kernel argument (3.4 of at most 4 KB)

// What one step has for all elements.  From a device step or rate these are computed by a kernel of their own.
struct AdamwFactors {
  float keep, c1, c2, pad;          // 1 - lr decay, lr / (1 - beta1^step), 1 / sqrt(1 - beta2^step)
};

struct AdamwParams {
  ttt_adamw_tensor t[kAdamwTensors];
  int first[kAdamwTensors + 1];     // the first work item of each
  int count;
  float beta1, beta2, rest1, rest2, eps;
  AdamwFactors f;
  const AdamwFactors *f_device;     // null: f
  const float *grad_scale;          // device, may be null
};

AdamwFactors adamw_factors(double lr, double beta1, double beta2, double decay, int64_t step);
hipError_t launch_adamw_factors(AdamwFactors *out, const int64_t *step_device, int64_t step, const float *lr_device, double lr,
                                double beta1, double beta2, double decay, hipStream_t s);
int64_t adamw_items(int64_t n);     // work items of a tensor of n elements
hipError_t launch_adamw(const AdamwParams &p, bool bits8, bool bf16, hipStream_t s);

}  // namespace ttt
