// Gated residual tail of a block and its gradient, one pass over the rows each:
//   u = gamma o / rms_group(o),  y = x + alpha u SiLU(z),  h = gamma_next y / rms(y)
// rms(a) = sqrt(mean(a^2) + eps), over groups of `norm` channels for o (a head, or the row).
// Bound by memory: a row stays in registers between its two reductions (8 channels a lane and
// vector), every tensor is read or written once.  Sums of squares, the gates and y up to h are
// fp32; y and h are rounded once, at their stores.  Measured, bf16: 137400 rows of 1024 1.41 GB in 268 us
// (5.2 TB/s; a copy reaches 5.1), the gradient of 43968 rows 0.72 GB in 155 us (4.6 TB/s); fp32, 8192
// rows of 768 without z 151 MB in 32 us and 5 more for the sums over rows; 1374 rows 8 us, a launch.
//
// Gradient (gy, gh given; y is the stored output; r = 1 / rms):
//   t = gh gamma_next,  yn = y r2,   gx = gy + r2 (t - yn mean(t yn))
//   on = o r1,  q = gx SiLU(z) alpha gamma,  go = r1 (q - on mean_group(q on))
//   gz = gx alpha gamma on SiLU'(z)
//   S = sum over rows of gx SiLU(z) on:  ggamma = alpha S,  galpha = gamma S;   ggamma_next = sum gh yn
// The sums over rows stay in registers over a workgroup's rows, then one partial a workgroup is
// added in a fixed order by a second kernel: no atomics, the same bits every time.
#include "common.h"
#include "residual.h"

namespace ttt {
namespace {

template <typename V> __device__ __forceinline__ f32x8 widen(const V v) {
  f32x8 r;
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = (float)v[i];
  return r;
}
template <typename T> __device__ __forceinline__ f32x8 load8(const T *p) { return widen(ld8(p)); }
__device__ __forceinline__ void store8(__bf16 *p, f32x8 v) {
  bf16x8 r;
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = (__bf16)v[i];
  *reinterpret_cast<bf16x8 *>(p) = r;
}
__device__ __forceinline__ void store8(float *p, f32x8 v) {
  *reinterpret_cast<f32x4 *>(p) = f32x4{v[0], v[1], v[2], v[3]};
  *reinterpret_cast<f32x4 *>(p + 4) = f32x4{v[4], v[5], v[6], v[7]};
}
__device__ __forceinline__ float dot8(f32x8 a, f32x8 b) {
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) s += a[i] * b[i];
  return s;
}
__device__ __forceinline__ f32x8 splat8(float x) { return f32x8{x, x, x, x, x, x, x, x}; }

// 1 / (1 + e^-z) and what it lacks of 1, both as exact as fp32 has them: e^-|z| = 2^p (1 + r ln 2), p + r = -|z| log2 e
// in two floats (with p alone it is 3.7e-6 off at |z| = 80; 137400 rows of 1024 in 268 us for 260).  e^-128 is 0
// beside 1 and in fp32.
__device__ __forceinline__ float2 sigmoid(float z) {
  const float a = fmaxf(-fabsf(z), -128.0f), p = a * 1.4426950408889634f;
  const float r = __builtin_fmaf(a, 1.9259630e-8f, __builtin_fmaf(a, 1.4426950408889634f, -p));
  const float e2 = __builtin_amdgcn_exp2f(p), e = __builtin_fmaf(e2, r * 0.6931471805599453f, e2);
  const float large = __builtin_amdgcn_rcpf(1.0f + e), small = e * large;
  return z < 0.0f ? float2{small, large} : float2{large, small};
}

// Threads of a workgroup: 256, or one row's lanes.
constexpr int threads_of(int lpr) { return lpr > 256 ? lpr : 256; }

// Sums over the LPR lanes of a row (from 256 on: the workgroup), and over groups of `norm` channels.
// The forms of a group: the row; a power of two of lanes (shuffles); of whole waves (and their sums through
// LDS); any other width (LDS, in two levels: one after another the squares of 512 vectors were added with the same
// rounding each time, 7.6e-6 of the sum at worst).
enum GroupMode { kGroupRow, kGroupLanes, kGroupWaves, kGroupAny };
template <int LPR, int NV> struct RowSums {
  float *s_row;       // [threads / 64]
  float *s_vec;       // [threads * NV]
  int groups8, mode;  // norm / 8
  __device__ float row(float v) const {
#pragma unroll
    for (int m = 1; m < (LPR < 64 ? LPR : 64); m <<= 1) v += __shfl_xor(v, m);
    if constexpr (LPR >= 256) {
      __syncthreads();
      if ((threadIdx.x & 63) == 0) s_row[threadIdx.x >> 6] = v;
      __syncthreads();
      v = 0.0f;
#pragma unroll
      for (int i = 0; i < LPR / 64; ++i) v += s_row[i];
    }
    return v;
  }
  // v[j]: this lane's sum over its j-th vector; out: the sum over that vector's group
  __device__ void group(float (&v)[NV]) const {
    if (mode == kGroupRow) {
      float s = 0.0f;
#pragma unroll
      for (int j = 0; j < NV; ++j) s += v[j];
      s = row(s);
#pragma unroll
      for (int j = 0; j < NV; ++j) v[j] = s;
    } else if (mode == kGroupLanes) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
        for (int m = 1; m < groups8; m <<= 1) v[j] += __shfl_xor(v[j], m);
    } else if (mode == kGroupWaves) {           // rows of a workgroup, whose waves a group divides
      if constexpr (LPR >= 256) {
        const int wave = threadIdx.x >> 6, n = groups8 >> 6;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int m = 1; m < 64; m <<= 1) v[j] += __shfl_xor(v[j], m);
        __syncthreads();
        if ((threadIdx.x & 63) == 0)
#pragma unroll
          for (int j = 0; j < NV; ++j) s_vec[j * (LPR / 64) + wave] = v[j];
        __syncthreads();
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          const float *s = s_vec + j * (LPR / 64) + wave / n * n;
          v[j] = 0.0f;
          for (int i = 0; i < n; ++i) v[j] += s[i];
        }
      }
    } else {
      const int lane = threadIdx.x % LPR;
      float *mine = s_vec + threadIdx.x / LPR * (LPR * NV);
      const int part = (int)ceilf(sqrtf((float)groups8));       // vectors of a part of a group
      __syncthreads();
#pragma unroll
      for (int j = 0; j < NV; ++j) mine[j * LPR + lane] = v[j];
      __syncthreads();
      // the first vector of a part takes its sum
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int i0 = j * LPR + lane, at = i0 % groups8, left = groups8 - at;
        v[j] = 0.0f;
        if (at % part == 0)
          for (int i = 0; i < (left < part ? left : part) && i0 + i < LPR * NV; ++i) v[j] += mine[i0 + i];
      }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < NV; ++j) mine[j * LPR + lane] = v[j];
      __syncthreads();
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int i0 = (j * LPR + lane) / groups8 * groups8;
        v[j] = 0.0f;
        for (int i = i0; i < i0 + groups8 && i < LPR * NV; i += part) v[j] += mine[i];
      }
    }
  }
};

// How the groups lie on the lanes (a power of two of at most 64 lanes never crosses a wave; one of more is a
// part of a workgroup's row, at most one vector a lane).
int group_mode(int channels, int norm) {
  if (norm == channels) return kGroupRow;
  const int g8 = norm / 8;
  if (g8 & (g8 - 1)) return kGroupAny;
  return g8 <= 64 ? kGroupLanes : kGroupWaves;
}

template <typename T, int LPR, int NV>
__global__ __launch_bounds__(threads_of(LPR)) void residual_kernel(ResidualParams p, int mode) {
  constexpr int NTH = threads_of(LPR), RPB = NTH / LPR;      // rows a workgroup has at once
  __shared__ float s_row[NTH / 64], s_vec[NTH * NV];
  const RowSums<LPR, NV> sums{s_row, s_vec, p.norm / 8, mode};
  const int lane = threadIdx.x % LPR;
  f32x8 ag[NV], gn[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * LPR + lane) * 8;
    ag[j] = gn[j] = splat8(c < p.channels ? 1.0f : 0.0f);
    if (c < p.channels) {
      if (p.gamma) ag[j] = load8(p.gamma + c);
      if (p.alpha) ag[j] *= load8(p.alpha + c);
      if (p.gamma_next) gn[j] = load8(p.gamma_next + c);
    }
  }
  const float inv_norm = 1.0f / (float)p.norm, inv_c = 1.0f / (float)p.channels;
  for (int64_t r0 = (int64_t)blockIdx.x * RPB; r0 < p.n; r0 += (int64_t)gridDim.x * RPB) {
    const int64_t row = r0 + threadIdx.x / LPR;
    const bool live = row < p.n;
    f32x8 o[NV], x[NV], z[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * LPR + lane) * 8;
      const bool in = live && c < p.channels;
      o[j] = in ? load8(static_cast<const T *>(p.o) + row * p.ldo + c) : splat8(0.0f);
      x[j] = in ? load8(static_cast<const T *>(p.x) + row * p.ldx + c) : splat8(0.0f);
      if (p.z) z[j] = in ? load8(static_cast<const T *>(p.z) + row * p.ldz + c) : splat8(0.0f);
    }
    float ss[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) ss[j] = dot8(o[j], o[j]);
    sums.group(ss);
    float sy = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * LPR + lane) * 8;
      const float r = 1.0f / sqrtf(ss[j] * inv_norm + p.eps);
      f32x8 u = o[j] * ag[j] * r;
      if (p.z)
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] *= z[j][i] * sigmoid(z[j][i]).x;
      x[j] += u;
      if (c < p.channels) sy += dot8(x[j], x[j]);
      if (live && c < p.channels) store8(static_cast<T *>(p.y) + row * p.ldy + c, x[j]);
    }
    if (p.h) {
      const float r = 1.0f / sqrtf(sums.row(sy) * inv_c + p.eps);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = (j * LPR + lane) * 8;
        if (live && c < p.channels) store8(static_cast<T *>(p.h) + row * p.ldh + c, x[j] * gn[j] * r);
      }
    }
  }
}

template <typename T, int LPR, int NV>
__global__ __launch_bounds__(threads_of(LPR)) void residual_backward_kernel(ResidualParams p, int mode) {
  constexpr int NTH = threads_of(LPR), RPB = NTH / LPR;
  __shared__ float s_row[NTH / 64], s_vec[NTH * NV];
  __shared__ __attribute__((aligned(16))) float s_acc[NTH * NV * 8];
  const RowSums<LPR, NV> sums{s_row, s_vec, p.norm / 8, mode};
  const int lane = threadIdx.x % LPR;
  f32x8 ag[NV], gn[NV], acc[NV], accn[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * LPR + lane) * 8;
    ag[j] = gn[j] = splat8(c < p.channels ? 1.0f : 0.0f);
    acc[j] = accn[j] = splat8(0.0f);
    if (c < p.channels) {
      if (p.gamma) ag[j] = load8(p.gamma + c);
      if (p.alpha) ag[j] *= load8(p.alpha + c);
      if (p.gamma_next) gn[j] = load8(p.gamma_next + c);
    }
  }
  const float inv_norm = 1.0f / (float)p.norm, inv_c = 1.0f / (float)p.channels;
  // bf16: the next row's tensors are loaded while this one is worked on (44k rows of 1024: 148 against
  // 235 us); fp32 rows would take the registers of a second wave a SIMD (8k rows of 768: 46 against 32)
  constexpr bool kAhead = sizeof(T) == 2;
  typedef typename FragOf<T>::type Raw;
  Raw n_gy[NV], n_gh[NV], n_y[NV], n_o[NV], n_z[NV];
  const auto fetch = [&](int64_t r0) {
    const int64_t row = r0 + threadIdx.x / LPR;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * LPR + lane) * 8;
      const bool in = row < p.n && c < p.channels;
      n_gy[j] = in && p.gy ? ld8(static_cast<const T *>(p.gy) + row * p.ldgy + c) : zero8<T>();
      n_gh[j] = in && p.gh ? ld8(static_cast<const T *>(p.gh) + row * p.ldgh + c) : zero8<T>();
      n_y[j] = in && p.gh ? ld8(static_cast<const T *>(p.y) + row * p.ldy + c) : zero8<T>();
      n_o[j] = in ? ld8(static_cast<const T *>(p.o) + row * p.ldo + c) : zero8<T>();
      n_z[j] = in && p.z ? ld8(static_cast<const T *>(p.z) + row * p.ldz + c) : zero8<T>();
    }
  };
  if (kAhead) fetch((int64_t)blockIdx.x * RPB);
  for (int64_t r0 = (int64_t)blockIdx.x * RPB; r0 < p.n; r0 += (int64_t)gridDim.x * RPB) {
    const int64_t row = r0 + threadIdx.x / LPR;
    const bool live = row < p.n;
    f32x8 gx[NV], o[NV], z[NV], y[NV], gh[NV];
    if (!kAhead) fetch(r0);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      gx[j] = widen(n_gy[j]), gh[j] = widen(n_gh[j]), y[j] = widen(n_y[j]), o[j] = widen(n_o[j]), z[j] = widen(n_z[j]);
    }
    if (kAhead) fetch(r0 + (int64_t)gridDim.x * RPB);
    if (p.gh) {
      float sy = 0.0f, sty = 0.0f;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        sy += dot8(y[j], y[j]);
        sty += dot8(y[j], gh[j] * gn[j]);
      }
      sy = sums.row(sy);
      sty = sums.row(sty);
      const float r2 = live ? 1.0f / sqrtf(sy * inv_c + p.eps) : 0.0f;
      const float m = sty * inv_c * r2 * r2;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        accn[j] += gh[j] * y[j] * r2;
        gx[j] += (gh[j] * gn[j] - y[j] * m) * r2;
      }
    }
    float ss[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) ss[j] = dot8(o[j], o[j]);
    sums.group(ss);
    f32x8 q[NV];
    float sq[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * LPR + lane) * 8;
      const bool in = live && c < p.channels;
      const float r1 = 1.0f / sqrtf(ss[j] * inv_norm + p.eps);
      ss[j] = in ? r1 : 0.0f;
      o[j] *= ss[j];
      if (in) store8(static_cast<T *>(p.gx) + row * p.ldgx + c, gx[j]);
      q[j] = gx[j];
      if (p.z) {
        f32x8 dz;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float zi = z[j][i];
          const float2 sg = sigmoid(zi);
          dz[i] = gx[j][i] * ag[j][i] * o[j][i] * (sg.x * (1.0f + zi * sg.y));
          q[j][i] *= zi * sg.x;
        }
        if (in) store8(static_cast<T *>(p.gz) + row * p.ldgz + c, dz);
      }
      if (in) acc[j] += q[j] * o[j];
      q[j] *= ag[j];
      sq[j] = dot8(q[j], o[j]);
    }
    sums.group(sq);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * LPR + lane) * 8;
      if (live && c < p.channels)
        store8(static_cast<T *>(p.go) + row * p.ldgo + c, (q[j] - o[j] * (sq[j] * inv_norm)) * ss[j]);
    }
  }
  // one partial a workgroup: its row slots added in order
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NV; ++j)
      store8(s_acc + (threadIdx.x / LPR) * (LPR * NV * 8) + (j * LPR + lane) * 8, k ? accn[j] : acc[j]);
    __syncthreads();
    for (int c = threadIdx.x; c < p.channels; c += NTH) {
      float s = 0.0f;
#pragma unroll
      for (int r = 0; r < RPB; ++r) s += s_acc[r * (LPR * NV * 8) + c];
      p.part[((int64_t)blockIdx.x * 2 + k) * p.channels + c] = s;
    }
  }
}

// The workgroups' partials, in order: 16 channels x 64 interleaved sums a workgroup.
__global__ __launch_bounds__(1024) void residual_sum_kernel(ResidualParams p, int parts) {
  __shared__ float s[64][17];
  const int c = blockIdx.x * 16 + (threadIdx.x & 15), k = blockIdx.y, q = threadIdx.x >> 4;
  float v = 0.0f;
  if (c < p.channels)
#pragma unroll 8
    for (int i = q; i < parts; i += 64) v += p.part[((int64_t)i * 2 + k) * p.channels + c];
  s[q][threadIdx.x & 15] = v;
  __syncthreads();
  if (q == 0 && c < p.channels) {
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 64; ++i) sum += s[i][threadIdx.x & 15];
    if (k == 1) {
      if (p.ggamma_next) p.ggamma_next[c] = sum;
    } else {
      if (p.ggamma) p.ggamma[c] = p.alpha ? p.alpha[c] * sum : sum;
      if (p.galpha) p.galpha[c] = p.gamma ? p.gamma[c] * sum : sum;
    }
  }
}

struct Shape { int lpr, nv; };
// One wave (or a part of it) a row up to 1024 channels, then a workgroup a row; two vectors a lane at
// most (four leave one wave a SIMD).
Shape shape_of(int channels) {
  const int v = (channels + 7) / 8;
  if (v <= 8) return {8, 1};
  if (v <= 16) return {16, 1};
  if (v <= 32) return {32, 1};
  if (v <= 64) return {64, 1};
  if (v <= 128) return {64, 2};
  if (v <= 256) return {256, 1};
  if (v <= 512) return {256, 2};
  return {512, 2};
}

template <typename T, int LPR, int NV>
hipError_t go(const ResidualParams &p, bool backward, hipStream_t s) {
  const int mode = group_mode(p.channels, p.norm), grid = residual_grid(p.n, p.channels);
  if (!backward) {
    hipLaunchKernelGGL((residual_kernel<T, LPR, NV>), dim3(grid), dim3(threads_of(LPR)), 0, s, p, mode);
    return hipGetLastError();
  }
  hipLaunchKernelGGL((residual_backward_kernel<T, LPR, NV>), dim3(grid), dim3(threads_of(LPR)), 0, s, p, mode);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !(p.ggamma || p.galpha || p.ggamma_next)) return e;
  hipLaunchKernelGGL(residual_sum_kernel, dim3((p.channels + 15) / 16, 2), dim3(1024), 0, s, p, grid);
  return hipGetLastError();
}

template <typename T> hipError_t pick(const ResidualParams &p, bool backward, hipStream_t s) {
  const Shape h = shape_of(p.channels);
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

// Four workgroups a CU loop over the rows (fewer for few rows).
int residual_grid(int64_t n, int channels) {
  const int lpr = shape_of(channels).lpr;
  const int64_t rpb = threads_of(lpr) / lpr, want = (n + rpb - 1) / rpb;
  return (int)(want < 1 ? 1 : (want < 1024 ? want : 1024));
}
hipError_t launch_residual(const ResidualParams &p, bool bf16, hipStream_t s) {
  if (p.n == 0) return hipSuccess;
  return bf16 ? pick<__bf16>(p, false, s) : pick<float>(p, false, s);
}
hipError_t launch_residual_backward(const ResidualParams &p, bool bf16, hipStream_t s) {
  return bf16 ? pick<__bf16>(p, true, s) : pick<float>(p, true, s);
}

}  // namespace ttt
