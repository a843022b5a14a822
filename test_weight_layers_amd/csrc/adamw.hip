// One AdamW step over many tensors, one pass over each of their arrays:
//   m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2,  w = w (1 - lr decay) - lr / (1 - b1^t) m / (sqrt(v) / sqrt(1 - b2^t) + eps)
// A lane has 8 consecutive elements.  8-bit states: blocks of 256 elements, 32 lanes, share a scale s, the largest
// |m| or sqrt(v); an element is s c |c| / 127^2 (m) or, its root, s c^2 / 255^2 (v), c to the nearest: the codes are
// finer where values are small.  The arithmetic is fp32 without contraction, each step rounded as it is written, so
// that a code is the formula's also where a value lies next to the border of two.
// Bound by memory: bf16 with fp32 masters and 8-bit states, 16 bytes an element read and written, 151 million elements in
// three launches 495 us (4.9 TB/s, a copy's rate); fp32 with 32-bit states, 7.1 million elements 32 us (28 bytes each; part
// of it stays in the last level of cache from call to call).  Up to 48 tensors go in a launch, as its argument.
#include <cmath>

#include "adamw.h"
#include "common.h"

namespace ttt {
namespace {

constexpr int kItem = 2048;         // elements of a work item: 256 lanes of 8

// 8 elements, `n` of which exist, in one access where the array allows it.
template <typename T> __device__ __forceinline__ f32x8 get8(const void *p, int64_t at, int n, bool wide) {
  const T *b = static_cast<const T *>(p) + at;
  f32x8 v;
  if (wide && n == 8) {
    const typename FragOf<T>::type x = ld8(b);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (float)x[i];
    return v;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = i < n ? (float)b[i] : 0.0f;
  return v;
}
template <typename T> __device__ __forceinline__ void put8(void *p, int64_t at, int n, bool wide, f32x8 v) {
  T *b = static_cast<T *>(p) + at;
  if (wide && n == 8) {
    typename FragOf<T>::type x;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = (T)v[i];
    *reinterpret_cast<typename FragOf<T>::type *>(b) = x;
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) b[i] = (T)v[i];
}
// 8 codes.
__device__ __forceinline__ uint2 get_codes(const void *p, int64_t at, int n, bool wide) {
  const unsigned char *b = static_cast<const unsigned char *>(p) + at;
  if (wide && n == 8) return *reinterpret_cast<const uint2 *>(b);
  uint2 r{0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) (i < 4 ? r.x : r.y) |= (unsigned)b[i] << (8 * (i & 3));
  return r;
}
__device__ __forceinline__ void put_codes(void *p, int64_t at, int n, bool wide, uint2 c) {
  unsigned char *b = static_cast<unsigned char *>(p) + at;
  if (wide && n == 8) {
    *reinterpret_cast<uint2 *>(b) = c;
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) b[i] = (unsigned char)((i < 4 ? c.x : c.y) >> (8 * (i & 3)));
}
__device__ __forceinline__ float largest32(float x) {
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const float y = __shfl_xor(x, m);
    x = x > y || !(x == x) ? x : y;     // a NaN stays
  }
  return x;
}

template <typename T, bool BITS8> __global__ __launch_bounds__(256) void adamw_kernel(AdamwParams p) {
#pragma clang fp contract(off)
  int k = 0;
  for (int s = 32; s > 0; s >>= 1)
    if (k + s < p.count && p.first[k + s] <= (int)blockIdx.x) k += s;
  const ttt_adamw_tensor &t = p.t[k];
  const int64_t at = (int64_t)((int)blockIdx.x - p.first[k]) * kItem + threadIdx.x * 8;
  const int64_t left = t.n - at;
  const int n = left < 0 ? 0 : (left < 8 ? (int)left : 8);
  const uintptr_t all = (uintptr_t)t.param | (uintptr_t)t.grad | (uintptr_t)t.master |
                        (BITS8 ? ((uintptr_t)t.exp_avg | (uintptr_t)t.exp_avg_sq) << 1 : (uintptr_t)t.exp_avg | (uintptr_t)t.exp_avg_sq);
  const bool wide = (all & 15) == 0;
  const AdamwFactors f = p.f_device ? *p.f_device : p.f;
  const float gs = p.grad_scale ? *p.grad_scale : 1.0f;
  f32x8 g = get8<T>(t.grad, at, n, wide);
  f32x8 w = t.master ? get8<float>(t.master, at, n, wide) : get8<T>(t.param, at, n, wide);
  f32x8 m, v;
  const int64_t blk = at / kAdamwBlock;
  if constexpr (BITS8) {
    const uint2 cm = get_codes(t.exp_avg, at, n, wide), cv = get_codes(t.exp_avg_sq, at, n, wide);
    const float sm = n > 0 ? t.exp_avg_scale[blk] : 0.0f, sv = n > 0 ? t.exp_avg_sq_scale[blk] : 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int a = (int)(signed char)((i < 4 ? cm.x : cm.y) >> (8 * (i & 3))), b = ((i < 4 ? cv.x : cv.y) >> (8 * (i & 3))) & 255;
      m[i] = (float)(a * (a < 0 ? -a : a)) * (1.0f / 16129.0f) * sm;
      const float r = (float)(b * b) * (1.0f / 65025.0f) * sv;
      v[i] = r * r;
    }
  } else {
    m = get8<float>(t.exp_avg, at, n, wide), v = get8<float>(t.exp_avg_sq, at, n, wide);
  }
  f32x8 root;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float gi = p.grad_scale ? g[i] * gs : g[i];
    m[i] = m[i] * p.beta1 + gi * p.rest1;
    v[i] = v[i] * p.beta2 + (gi * gi) * p.rest2;
    root[i] = sqrtf(v[i]);
    w[i] = w[i] * f.keep - (m[i] * f.c1) / (root[i] * f.c2 + p.eps);
  }
  if (t.master) put8<float>(t.master, at, n, wide, w);
  put8<T>(t.param, at, n, wide, w);
  if constexpr (BITS8) {
    float sm = 0.0f, sv = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = i < n ? fabsf(m[i]) : 0.0f, b = i < n ? root[i] : 0.0f;
      sm = sm > a || !(sm == sm) ? sm : a, sv = sv > b || !(sv == sv) ? sv : b;
    }
    sm = largest32(sm), sv = largest32(sv);
    // (below 2^-126 a reciprocal may be infinite: such a block becomes zero)
    const float rm = sm >= 1.17549435e-38f ? 1.0f / sm : 0.0f, rv = sv >= 1.17549435e-38f ? 1.0f / sv : 0.0f;
    uint2 cm{0, 0}, cv{0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = rintf(sqrtf(fabsf(m[i]) * rm) * 127.0f), b = rintf(sqrtf(root[i] * rv) * 255.0f);
      // (a NaN or an infinity makes the scale one, and with it the block: of the code of a NaN nothing depends)
      const int x = (int)fminf(a, 127.0f), y = (int)fminf(b, 255.0f);
      (i < 4 ? cm.x : cm.y) |= (unsigned)((m[i] < 0.0f ? -x : x) & 255) << (8 * (i & 3));
      (i < 4 ? cv.x : cv.y) |= (unsigned)y << (8 * (i & 3));
    }
    put_codes(t.exp_avg, at, n, wide, cm);
    put_codes(t.exp_avg_sq, at, n, wide, cv);
    if (n > 0 && (threadIdx.x & 31) == 0) t.exp_avg_scale[blk] = sm, t.exp_avg_sq_scale[blk] = sv;
  } else {
    put8<float>(t.exp_avg, at, n, wide, m);
    put8<float>(t.exp_avg_sq, at, n, wide, v);
  }
}

__global__ void adamw_factors_kernel(AdamwFactors *out, const int64_t *step_device, int64_t step, const float *lr_device, double lr,
                                     double beta1, double beta2, double decay) {
#pragma clang fp contract(off)
  const double t = (double)(step_device ? *step_device : step), a = lr_device ? (double)*lr_device : lr;
  *out = AdamwFactors{(float)(1.0 - a * decay), (float)(a / (1.0 - pow(beta1, t))), (float)(1.0 / sqrt(1.0 - pow(beta2, t))), 0.0f};
}

}  // namespace

AdamwFactors adamw_factors(double lr, double beta1, double beta2, double decay, int64_t step) {
  const double t = (double)step;
  return AdamwFactors{(float)(1.0 - lr * decay), (float)(lr / (1.0 - std::pow(beta1, t))),
                      (float)(1.0 / std::sqrt(1.0 - std::pow(beta2, t))), 0.0f};
}

hipError_t launch_adamw_factors(AdamwFactors *out, const int64_t *step_device, int64_t step, const float *lr_device, double lr,
                                double beta1, double beta2, double decay, hipStream_t s) {
  hipLaunchKernelGGL(adamw_factors_kernel, dim3(1), dim3(1), 0, s, out, step_device, step, lr_device, lr, beta1, beta2, decay);
  return hipGetLastError();
}

int64_t adamw_items(int64_t n) { return (n + kItem - 1) / kItem; }

hipError_t launch_adamw(const AdamwParams &p, bool bits8, bool bf16, hipStream_t s) {
  const dim3 grid(p.first[p.count]), block(256);
  if (bf16) {
    if (bits8) hipLaunchKernelGGL((adamw_kernel<__bf16, true>), grid, block, 0, s, p);
    else hipLaunchKernelGGL((adamw_kernel<__bf16, false>), grid, block, 0, s, p);
  } else {
    if (bits8) hipLaunchKernelGGL((adamw_kernel<float, true>), grid, block, 0, s, p);
    else hipLaunchKernelGGL((adamw_kernel<float, false>), grid, block, 0, s, p);
  }
  return hipGetLastError();
}

}  // namespace ttt
