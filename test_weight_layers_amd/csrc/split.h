// Operands of the delta-rule kernels.  Tokens enter the matrix cores as they are (bf16, or
// fp32 on fp32 MFMA).  What is computed on the way (states, U, T, ...) is fp32; beside bf16
// tokens it enters as two bf16 parts, x = h + l with l = bf16(x - h): 17 significant bits,
// so a product keeps about 4e-6 relative where one bf16 part would leave 2e-3 in the fp32
// states.  Dropped in a product of two split operands: l * l, at most 2^-18 of the product.
//
// A split matrix in memory is one [rows][cols] plane a part, or one fp32 plane.
#pragma once
#include "common.h"
#include "delta.h"

namespace ttt {

struct Split8 {
  bf16x8 p[kParts];
};

__device__ __forceinline__ f32x4 mm(bf16x8 a, bf16x8 b, f32x4 c) { return mma(a, b, c); }
__device__ __forceinline__ f32x4 mm(bf16x8 a, const Split8 &b, f32x4 c) {
#pragma unroll
  for (int i = kParts - 1; i >= 0; --i) c = mma(a, b.p[i], c);
  return c;
}
__device__ __forceinline__ f32x4 mm(const Split8 &a, bf16x8 b, f32x4 c) {
#pragma unroll
  for (int i = kParts - 1; i >= 0; --i) c = mma(a.p[i], b, c);
  return c;
}
__device__ __forceinline__ f32x4 mm(const Split8 &a, const Split8 &b, f32x4 c) {
#pragma unroll
  for (int d = kParts - 1; d >= 0; --d)         // the small products first
#pragma unroll
    for (int i = 0; i <= d; ++i) c = mma(a.p[i], b.p[d - i], c);
  return c;
}
__device__ __forceinline__ f32x4 mm(f32x8 a, f32x8 b, f32x4 c) { return mma(a, b, c); }

// The products of one operand with every part of the other, each added to a sum of its own: products
// that follow one another then do not wait for one another.
template <typename T> struct Sums {
  static constexpr int N = sizeof(T) == 2 ? kParts : 1;
  f32x4 v[N];
  __device__ __forceinline__ Sums() {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = f32x4{0, 0, 0, 0};
  }
  __device__ __forceinline__ void add(bf16x8 a, const Split8 &b) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = mma(a, b.p[i], v[i]);
  }
  __device__ __forceinline__ void add(f32x8 a, f32x8 b) { v[0] = mma(a, b, v[0]); }
  __device__ __forceinline__ f32x4 sum() const {
    f32x4 s = v[N - 1];
#pragma unroll
    for (int i = N - 2; i >= 0; --i) s += v[i];
    return s;
  }
};

// Split matrices beside T tokens: `plane` is the byte distance from one part's plane to the next.
template <typename T> struct Sp;
template <> struct Sp<__bf16> {
  typedef Split8 Frag;
  static constexpr int kBytes = 2;          // of one element in one plane
  static constexpr int kPlanes = kParts;
  static constexpr int kPad = 8;            // row padding (elements) of LDS tiles: 16 bytes
  static __device__ __forceinline__ Frag ld(const char *base, int64_t plane, int64_t e) {
    Frag f;
#pragma unroll
    for (int i = 0; i < kParts; ++i) f.p[i] = ld8(reinterpret_cast<const __bf16 *>(base + i * plane) + e);
    return f;
  }
  static __device__ __forceinline__ void st4(char *base, int64_t plane, int64_t e, f32x4 v) {
#pragma unroll
    for (int i = 0; i < kParts; ++i) {
      bf16x4 h;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        h[r] = (__bf16)v[r];
        v[r] -= (float)h[r];
      }
      *reinterpret_cast<bf16x4 *>(reinterpret_cast<__bf16 *>(base + i * plane) + e) = h;
    }
  }
  static __device__ __forceinline__ void st1(char *base, int64_t plane, int64_t e, float v) {
#pragma unroll
    for (int i = 0; i < kParts; ++i) {
      const __bf16 h = (__bf16)v;
      reinterpret_cast<__bf16 *>(base + i * plane)[e] = h;
      v -= (float)h;
    }
  }
  // eight consecutive elements
  static __device__ __forceinline__ void st8(char *base, int64_t plane, int64_t e, const float *x) {
    float v[8];
#pragma unroll
    for (int r = 0; r < 8; ++r) v[r] = x[r];
#pragma unroll
    for (int i = 0; i < kParts; ++i) {
      bf16x8 h;
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        h[r] = (__bf16)v[r];
        v[r] -= (float)h[r];
      }
      *reinterpret_cast<bf16x8 *>(reinterpret_cast<__bf16 *>(base + i * plane) + e) = h;
    }
  }
  static __device__ __forceinline__ float at(const Frag &f, int k) {
    float v = 0.0f;
#pragma unroll
    for (int i = kParts - 1; i >= 0; --i) v += (float)f.p[i][k];
    return v;
  }
};
template <> struct Sp<float> {
  typedef f32x8 Frag;
  static constexpr int kBytes = 4;
  static constexpr int kPlanes = 1;
  static constexpr int kPad = 4;
  static __device__ __forceinline__ Frag ld(const char *base, int64_t, int64_t e) {
    return ld8(reinterpret_cast<const float *>(base) + e);
  }
  static __device__ __forceinline__ void st4(char *base, int64_t, int64_t e, f32x4 v) {
    *reinterpret_cast<f32x4 *>(reinterpret_cast<float *>(base) + e) = v;
  }
  static __device__ __forceinline__ void st1(char *base, int64_t, int64_t e, float v) {
    reinterpret_cast<float *>(base)[e] = v;
  }
  static __device__ __forceinline__ void st8(char *base, int64_t, int64_t e, const float *x) {
    float *o = reinterpret_cast<float *>(base) + e;
    *reinterpret_cast<f32x4 *>(o) = f32x4{x[0], x[1], x[2], x[3]};
    *reinterpret_cast<f32x4 *>(o + 4) = f32x4{x[4], x[5], x[6], x[7]};
  }
  static __device__ __forceinline__ float at(const Frag &f, int i) { return f[i]; }
};

// Bytes of a split matrix of n elements in memory.
template <typename T> __device__ __forceinline__ int64_t split_bytes(int64_t n) {
  return n * (Sp<T>::kBytes * Sp<T>::kPlanes);
}

// Launch-order block id -> work item, so that consecutive items (which read the same tokens and
// chunk terms) run on one XCD: workgroups go round the 8 XCDs.
__device__ __forceinline__ int xcd_item() {
  const int n = gridDim.x, b = blockIdx.x;
  return n % 8 == 0 ? (b & 7) * (n >> 3) + (b >> 3) : b;
}

// A split matrix in LDS: R rows of Ccols elements, rows padded by 16 bytes (a ds_read_b128 of
// 16 rows at one column then meets 16 distinct bank groups for every Ccols that is a multiple of 64).
template <typename T, int R, int Ccols> struct SpTile {
  static constexpr int kPitch = Ccols + Sp<T>::kPad;
  static constexpr int kPlane = R * kPitch * Sp<T>::kBytes;
  static constexpr int kSize = Sp<T>::kPlanes * kPlane;
  char b[kSize];
  __device__ __forceinline__ typename Sp<T>::Frag ld(int r, int c) const { return Sp<T>::ld(b, kPlane, r * kPitch + c); }
  __device__ __forceinline__ void st4(int r, int c, f32x4 v) { Sp<T>::st4(b, kPlane, r * kPitch + c, v); }
  __device__ __forceinline__ void st1(int r, int c, float v) { Sp<T>::st1(b, kPlane, r * kPitch + c, v); }
  // Lane (g, li)'s rows r0 + 4 g .. + 3 of column c0 + li, copied to element e of a split matrix in memory.
  __device__ __forceinline__ void copy_t4(int r0, int c0, char *dst, int64_t plane, int64_t e) const {
    const int l = threadIdx.x & 63, g = l >> 4, li = l & 15;
    if constexpr (sizeof(T) == 2) {
      const int o = ((r0 + 4 * g + (li >> 2)) * kPitch + c0 + 4 * (li & 3)) * 2;
#pragma unroll
      for (int i = 0; i < Sp<T>::kPlanes; ++i)
        *reinterpret_cast<bf16x4 *>(dst + i * plane + e * 2) =
            lds_read_tr16(reinterpret_cast<const unsigned char *>(b) + i * kPlane + o);
    } else {
      f32x4 v;
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] = reinterpret_cast<const float *>(b)[(r0 + 4 * g + r) * kPitch + c0 + li];
      *reinterpret_cast<f32x4 *>(dst + e * 4) = v;
    }
  }
};

// Operands in memory are kept in the order in which lanes take them: a matrix of rows x k is cut in
// 16 x 32 fragments, the `nk` fragments of 16 rows one after another, each 64 lanes x 8 elements
// (lane = 16 (k / 8 % 4) + row % 16).  One load then is 1 KB on end for a wave; with the rows as
// they are it touches 16 rows, one lookup a lane (measured: 60 against 16 cycles a load).
__device__ __forceinline__ int frag_of(int rt, int kt, int nk) { return ((rt * nk + kt) * 64 + (threadIdx.x & 63)) * 8; }
__device__ __forceinline__ int64_t frag_at(int row, int k, int nk) {
  return ((int64_t)((row >> 4) * nk + (k >> 5)) * 64 + ((k >> 3) & 3) * 16 + (row & 15)) * 8 + (k & 7);
}

// Workgroup barrier that waits for this wave's LDS traffic only: loads from memory stay in flight.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(15 | (7 << 4) | (3 << 14));      // lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

__device__ __forceinline__ f32x4 zero4() { return f32x4{0, 0, 0, 0}; }

// e^x for a difference of cumulative log decays held in 64 bits.
__device__ __forceinline__ float exp_of(double x) { return __builtin_amdgcn_exp2f((float)(x * 1.4426950408889634)); }

}  // namespace ttt
