// Operands of the delta-rule kernels.  Tokens enter the matrix cores as they are (bf16, or
// fp32 on fp32 MFMA).  What is computed on the way (states, U, T, ...) is fp32; beside bf16
// tokens it enters as two bf16 parts, x = h + l with l = bf16(x - h): 17 significant bits,
// so a product keeps about 4e-6 relative where one bf16 part would leave 2e-3 in the fp32
// states.  Dropped in a product of two split operands: l * l, at most 2^-18 of the product.
//
// A split matrix takes 4 bytes an element for either token type: bf16 planes h and l, each
// [rows][cols], or one fp32 plane.
#pragma once
#include "common.h"

namespace ttt {

struct Split8 {
  bf16x8 h, l;
};

__device__ __forceinline__ f32x4 mm(bf16x8 a, bf16x8 b, f32x4 c) { return mma(a, b, c); }
__device__ __forceinline__ f32x4 mm(bf16x8 a, Split8 b, f32x4 c) { return mma(a, b.h, mma(a, b.l, c)); }
__device__ __forceinline__ f32x4 mm(Split8 a, bf16x8 b, f32x4 c) { return mma(a.h, b, mma(a.l, b, c)); }
__device__ __forceinline__ f32x4 mm(Split8 a, Split8 b, f32x4 c) {
  return mma(a.h, b.h, mma(a.h, b.l, mma(a.l, b.h, c)));
}
__device__ __forceinline__ f32x4 mm(f32x8 a, f32x8 b, f32x4 c) { return mma(a, b, c); }

// Split matrices of T tokens: `plane` is the byte distance from the h plane to the l plane.
template <typename T> struct Sp;
template <> struct Sp<__bf16> {
  typedef Split8 Frag;
  static constexpr int kBytes = 2;          // of one element in one plane
  static constexpr int kPad = 8;            // row padding (elements) of LDS tiles: 16 bytes
  static __device__ __forceinline__ Frag ld(const char *base, int64_t plane, int64_t e) {
    return Split8{ld8(reinterpret_cast<const __bf16 *>(base) + e), ld8(reinterpret_cast<const __bf16 *>(base + plane) + e)};
  }
  static __device__ __forceinline__ void st4(char *base, int64_t plane, int64_t e, f32x4 v) {
    bf16x4 h, l;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      h[i] = (__bf16)v[i];
      l[i] = (__bf16)(v[i] - (float)h[i]);
    }
    *reinterpret_cast<bf16x4 *>(reinterpret_cast<__bf16 *>(base) + e) = h;
    *reinterpret_cast<bf16x4 *>(reinterpret_cast<__bf16 *>(base + plane) + e) = l;
  }
  static __device__ __forceinline__ void st1(char *base, int64_t plane, int64_t e, float v) {
    const __bf16 h = (__bf16)v;
    reinterpret_cast<__bf16 *>(base)[e] = h;
    reinterpret_cast<__bf16 *>(base + plane)[e] = (__bf16)(v - (float)h);
  }
  static __device__ __forceinline__ float at(const Frag &f, int i) { return (float)f.h[i] + (float)f.l[i]; }
};
template <> struct Sp<float> {
  typedef f32x8 Frag;
  static constexpr int kBytes = 4;
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
  static __device__ __forceinline__ float at(const Frag &f, int i) { return f[i]; }
};

// A split matrix in LDS: R rows of Ccols elements, rows padded by 16 bytes (a ds_read_b128 of
// 16 rows at one column then meets 16 distinct bank groups for every Ccols that is a multiple of 64).
template <typename T, int R, int Ccols> struct SpTile {
  static constexpr int kPitch = Ccols + Sp<T>::kPad;
  static constexpr int kPlane = R * kPitch * Sp<T>::kBytes;
  static constexpr int kSize = sizeof(T) == 2 ? 2 * kPlane : kPlane;
  char b[kSize];
  __device__ __forceinline__ typename Sp<T>::Frag ld(int r, int c) const { return Sp<T>::ld(b, kPlane, r * kPitch + c); }
  __device__ __forceinline__ void st4(int r, int c, f32x4 v) { Sp<T>::st4(b, kPlane, r * kPitch + c, v); }
  __device__ __forceinline__ void st1(int r, int c, float v) { Sp<T>::st1(b, kPlane, r * kPitch + c, v); }
};

__device__ __forceinline__ f32x4 zero4() { return f32x4{0, 0, 0, 0}; }

// e^x for a difference of cumulative log decays held in 64 bits.
__device__ __forceinline__ float exp_of(double x) { return __builtin_amdgcn_exp2f((float)(x * 1.4426950408889634)); }

}  // namespace ttt
