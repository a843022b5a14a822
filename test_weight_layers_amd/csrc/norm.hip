// Layer norm and its gradient, one pass over the rows each:
//   y = gamma xn + beta,  xn = (x - mean) r,  r = 1 / sqrt(var + eps), over `width` columns
//   t = gy gamma,  gx = r (t - mean(t) - xn mean(t xn));  ggamma = sum gy xn,  gbeta = sum gy
// A vector (a row, or one group of its columns) stays in registers, 8 elements a lane and piece.  The mean is taken
// first and the squares of what is left of it then, whose own mean, what rounding left of the first, is taken off
// again: no digits are lost where the mean is large beside the deviation.  Everything is fp32, rounded at the stores.
// The sums over rows stay in registers over a workgroup's vectors; one partial a workgroup, then a second kernel adds
// them in a fixed order.
// Bound by memory, so that lanes are given to a vector until each has 16 bytes or more of it: 8 lanes for 64 columns, 64 for
// up to 1024, whole workgroups from there.  bf16, 137,400 rows of 16 groups of 64: 124 us (4.5 TB/s), the gradient of 43,968
// rows of 1024 50 us (5.4 TB/s) and 6 for the sums; fp32, 8192 rows of 768: 20 and 5.  A copy moves 4.9 TB/s.
#include "common.h"
#include "norm.h"

namespace ttt {
namespace {

__device__ __forceinline__ f32x8 splat8(float x) { return f32x8{x, x, x, x, x, x, x, x}; }
template <typename V> __device__ __forceinline__ f32x8 widen(const V v) {
  f32x8 r;
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = (float)v[i];
  return r;
}
// Elements c .. c + 7 of a vector of `width`: zeros behind its end, which are not read.
template <typename T> __device__ __forceinline__ typename FragOf<T>::type load8(const T *p, int c, int width) {
  if (c + 8 <= width) return ld8(p + c);
  typename FragOf<T>::type v = zero8<T>();
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (c + i < width) v[i] = p[c + i];
  return v;
}
__device__ __forceinline__ void put8(__bf16 *p, f32x8 v) {
  bf16x8 r;
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = (__bf16)v[i];
  *reinterpret_cast<bf16x8 *>(p) = r;
}
__device__ __forceinline__ void put8(float *p, f32x8 v) {
  *reinterpret_cast<f32x4 *>(p) = f32x4{v[0], v[1], v[2], v[3]};
  *reinterpret_cast<f32x4 *>(p + 4) = f32x4{v[4], v[5], v[6], v[7]};
}
template <typename T> __device__ __forceinline__ void store8(T *p, int c, int width, f32x8 v) {
  if (c + 8 <= width) {
    put8(p + c, v);
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (c + i < width) p[c + i] = from_f32<T>(v[i]);
}

constexpr int threads_of(int lpr) { return lpr > 256 ? lpr : 256; }

// Two sums over the LPR lanes of a vector.
template <int LPR> __device__ __forceinline__ float2 lane_sums(float a, float b, float2 *s_row) {
#pragma unroll
  for (int m = 1; m < (LPR < 64 ? LPR : 64); m <<= 1) a += __shfl_xor(a, m), b += __shfl_xor(b, m);
  if constexpr (LPR >= 256) {
    __syncthreads();
    if ((threadIdx.x & 63) == 0) s_row[threadIdx.x >> 6] = float2{a, b};
    __syncthreads();
    a = b = 0.0f;
#pragma unroll
    for (int i = 0; i < LPR / 64; ++i) a += s_row[i].x, b += s_row[i].y;
  }
  return float2{a, b};
}

// Takes the mean off x (zero behind the vector's end) and returns 1 / sqrt(var + eps).
template <int LPR, int NV> __device__ __forceinline__ float centre(f32x8 (&x)[NV], int lane, int width, float inv, float eps, float2 *s_row) {
  float a = 0.0f;
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) a += x[j][i];
  const float mean = lane_sums<LPR>(a, 0.0f, s_row).x * inv;
  a = 0.0f;
  float b = 0.0f;
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[j][i] = (j * LPR + lane) * 8 + i < width ? x[j][i] - mean : 0.0f;
      a += x[j][i], b += x[j][i] * x[j][i];
    }
  const float2 s = lane_sums<LPR>(a, b, s_row);
  const float rest = s.x * inv;
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if ((j * LPR + lane) * 8 + i < width) x[j][i] -= rest;
  return 1.0f / sqrtf(fmaxf(s.y * inv - rest * rest, 0.0f) + eps);
}

template <typename T, int LPR, int NV> __global__ __launch_bounds__(threads_of(LPR)) void norm_kernel(NormParams p) {
  constexpr int NTH = threads_of(LPR), RPB = NTH / LPR;      // vectors a workgroup has at once
  __shared__ float2 s_row[NTH / 64];
  const int lane = threadIdx.x % LPR;
  f32x8 ga[NV], be[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * LPR + lane) * 8;
    ga[j] = p.gamma ? load8(p.gamma, c, p.width) : splat8(1.0f);
    be[j] = p.beta ? load8(p.beta, c, p.width) : splat8(0.0f);
  }
  const float inv = 1.0f / (float)p.width;
  const int64_t total = p.n * p.groups;
  for (int64_t v0 = (int64_t)blockIdx.x * RPB; v0 < total; v0 += (int64_t)gridDim.x * RPB) {
    const int64_t v = v0 + threadIdx.x / LPR;
    const bool live = v < total;
    const int64_t row = live ? v / p.groups : 0, at = live ? v % p.groups * p.width : 0;
    f32x8 x[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j)
      x[j] = widen(load8(static_cast<const T *>(p.x) + row * p.ldx + at, (j * LPR + lane) * 8, p.width));
    const float r = centre<LPR, NV>(x, lane, p.width, inv, p.eps, s_row);
    if (live)
#pragma unroll
      for (int j = 0; j < NV; ++j)
        store8(static_cast<T *>(p.y) + row * p.ldy + at, (j * LPR + lane) * 8, p.width, x[j] * r * ga[j] + be[j]);
  }
}

template <typename T, int LPR, int NV> __global__ __launch_bounds__(threads_of(LPR)) void norm_backward_kernel(NormParams p) {
  constexpr int NTH = threads_of(LPR), RPB = NTH / LPR;
  __shared__ float2 s_row[NTH / 64];
  __shared__ __attribute__((aligned(16))) float s_acc[NTH * NV * 8];
  const int lane = threadIdx.x % LPR;
  f32x8 ga[NV], ag[NV], ab[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    ga[j] = p.gamma ? load8(p.gamma, (j * LPR + lane) * 8, p.width) : splat8(1.0f);
    ag[j] = ab[j] = splat8(0.0f);
  }
  const float inv = 1.0f / (float)p.width;
  const int64_t total = p.n * p.groups;
  for (int64_t v0 = (int64_t)blockIdx.x * RPB; v0 < total; v0 += (int64_t)gridDim.x * RPB) {
    const int64_t v = v0 + threadIdx.x / LPR;
    const bool live = v < total;
    const int64_t row = live ? v / p.groups : 0, at = live ? v % p.groups * p.width : 0;
    f32x8 x[NV], t[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * LPR + lane) * 8;
      x[j] = widen(load8(static_cast<const T *>(p.x) + row * p.ldx + at, c, p.width));
      t[j] = widen(load8(static_cast<const T *>(p.gy) + row * p.ldgy + at, c, p.width));
    }
    const float r = centre<LPR, NV>(x, lane, p.width, inv, p.eps, s_row);
    float a = 0.0f, b = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      x[j] *= r;
      if (live) ag[j] += t[j] * x[j], ab[j] += t[j];
      t[j] *= ga[j];
#pragma unroll
      for (int i = 0; i < 8; ++i) a += t[j][i], b += t[j][i] * x[j][i];
    }
    const float2 s = lane_sums<LPR>(a, b, s_row);
    if (live)
#pragma unroll
      for (int j = 0; j < NV; ++j)
        store8(static_cast<T *>(p.y) + row * p.ldy + at, (j * LPR + lane) * 8, p.width, (t[j] - s.x * inv - x[j] * (s.y * inv)) * r);
  }
  // one partial a workgroup: its slots added in order
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NV; ++j)
      put8(s_acc + (threadIdx.x / LPR) * (LPR * NV * 8) + (j * LPR + lane) * 8, k ? ab[j] : ag[j]);
    __syncthreads();
    for (int c = threadIdx.x; c < p.width; c += NTH) {
      float s = 0.0f;
#pragma unroll
      for (int r = 0; r < RPB; ++r) s += s_acc[r * (LPR * NV * 8) + c];
      p.part[((int64_t)blockIdx.x * 2 + k) * p.width + c] = s;
    }
  }
}

// The workgroups' partials, in order: 16 columns x 64 interleaved sums a workgroup.
__global__ __launch_bounds__(1024) void norm_sum_kernel(NormParams p, int parts) {
  __shared__ float s[64][17];
  const int c = blockIdx.x * 16 + (threadIdx.x & 15), k = blockIdx.y, q = threadIdx.x >> 4;
  float v = 0.0f;
  if (c < p.width)
#pragma unroll 8
    for (int i = q; i < parts; i += 64) v += p.part[((int64_t)i * 2 + k) * p.width + c];
  s[q][threadIdx.x & 15] = v;
  __syncthreads();
  float *out = k ? p.gbeta : p.ggamma;
  if (q == 0 && c < p.width && out) {
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 64; ++i) sum += s[i][threadIdx.x & 15];
    out[c] = sum;
  }
}

struct Shape { int lpr, nv; };
Shape shape_of(int width) {
  const int v = (width + 7) / 8;
  if (v <= 8) return {8, 1};
  if (v <= 16) return {16, 1};
  if (v <= 32) return {32, 1};
  if (v <= 64) return {64, 1};
  if (v <= 128) return {64, 2};
  if (v <= 256) return {256, 1};
  if (v <= 512) return {256, 2};
  return {512, 2};
}

template <typename T, int LPR, int NV> hipError_t go(const NormParams &p, bool backward, hipStream_t s) {
  const int grid = norm_grid(p.n * p.groups, p.width);
  if (!backward) {
    hipLaunchKernelGGL((norm_kernel<T, LPR, NV>), dim3(grid), dim3(threads_of(LPR)), 0, s, p);
    return hipGetLastError();
  }
  hipLaunchKernelGGL((norm_backward_kernel<T, LPR, NV>), dim3(grid), dim3(threads_of(LPR)), 0, s, p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !(p.ggamma || p.gbeta)) return e;
  hipLaunchKernelGGL(norm_sum_kernel, dim3((p.width + 15) / 16, 2), dim3(1024), 0, s, p, grid);
  return hipGetLastError();
}

template <typename T> hipError_t pick(const NormParams &p, bool backward, hipStream_t s) {
  const Shape h = shape_of(p.width);
  switch (h.lpr * 10 + h.nv) {
    case 81: return go<T, 8, 1>(p, backward, s);
    case 161: return go<T, 16, 1>(p, backward, s);
    case 321: return go<T, 32, 1>(p, backward, s);
    case 641: return go<T, 64, 1>(p, backward, s);
    case 642: return go<T, 64, 2>(p, backward, s);
    case 2561: return go<T, 256, 1>(p, backward, s);
    case 2562: return go<T, 256, 2>(p, backward, s);
    default: return go<T, 512, 2>(p, backward, s);
  }
}

}  // namespace

int norm_grid(int64_t vectors, int width) {
  const int lpr = shape_of(width).lpr;
  const int64_t rpb = threads_of(lpr) / lpr, want = (vectors + rpb - 1) / rpb;
  return (int)(want < 1 ? 1 : (want < 1024 ? want : 1024));
}
hipError_t launch_norm(const NormParams &p, bool bf16, hipStream_t s) {
  if (p.n == 0) return hipSuccess;
  return bf16 ? pick<__bf16>(p, false, s) : pick<float>(p, false, s);
}
hipError_t launch_norm_backward(const NormParams &p, bool bf16, hipStream_t s) {
  return bf16 ? pick<__bf16>(p, true, s) : pick<float>(p, true, s);
}

}  // namespace ttt
