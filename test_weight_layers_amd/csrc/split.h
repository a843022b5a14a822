// Operands of the delta-rule kernels.
//
// Sums and states are fp32; products run on bf16 MFMA, on operands written as sums of bf16 parts,
// x = p0 + p1 + p2, p0 = bf16(x), p1 = bf16(x - p0), .. (8 bits of significand each).  bf16 tokens
// are one part, exactly.  fp32 tokens, and what is computed on the way (states, U, T, A, ..), are three
// parts, 24 bits: a result before its rounding then is as good as from fp32 products, at 2.7 times the
// rate of fp32 MFMA (six products of 16 clocks against one of 256 for 32 reduction elements).  Two parts
// (17 bits) of what only reaches bf16 outputs leave these as far from 64 bits, but round a few of them to the
// other neighbour (outputs 1.3e-4 off the 64-bit ones rounded, with three 1.1e-5 to 3.1e-5).
// A product of two operands takes the part pairs (i, j) with i + j below the larger part count.
// Measured beside bf16 tokens with two parts everywhere: fp32 states 4.0e-6 off and gradients of
// the rates 6.9e-6, with three 1.1e-7 and 3.1e-7 (fp32 arithmetic: 2.2e-7 and 4.0e-7).
#pragma once
#include "common.h"
#include "delta.h"

namespace ttt {

template <int P> struct Split {
  bf16x8 p[P];
};
// Parts of T tokens.
template <typename T> constexpr int kTok = sizeof(T) == 2 ? 1 : 3;
constexpr int kFull = kDeltaParts;

template <int A, int B> __device__ __forceinline__ f32x4 mm(const Split<A> &a, const Split<B> &b, f32x4 c) {
  constexpr int N = A > B ? A : B;
#pragma unroll
  for (int d = N - 1; d >= 0; --d)                // the small products first
#pragma unroll
    for (int i = 0; i <= d; ++i)
      if (i < A && d - i < B) c = mma(a.p[i], b.p[d - i], c);
  return c;
}
// The same into one sum for every d: products that follow one another then do not wait for one another.
template <int N> struct Sums {
  f32x4 v[N];
  __device__ __forceinline__ Sums() {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = f32x4{0, 0, 0, 0};
  }
  template <int A, int B> __device__ __forceinline__ void add(const Split<A> &a, const Split<B> &b) {
#pragma unroll
    for (int d = N - 1; d >= 0; --d)
#pragma unroll
      for (int i = 0; i <= d; ++i)
        if (i < A && d - i < B) v[d] = mma(a.p[i], b.p[d - i], v[d]);
  }
  __device__ __forceinline__ f32x4 sum() const {
    f32x4 s = v[N - 1];
#pragma unroll
    for (int i = N - 2; i >= 0; --i) s += v[i];
    return s;
  }
};

template <int P> __device__ __forceinline__ Split<P> split_of(const f32x8 x) {
  Split<P> s;
  f32x8 v = x;
#pragma unroll
  for (int i = 0; i < P; ++i)
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      s.p[i][r] = (__bf16)v[r];
      if (i + 1 < P) v[r] -= (float)s.p[i][r];
    }
  return s;
}
// Eight tokens' elements as an operand.
__device__ __forceinline__ Split<1> token_of(const bf16x8 x) { return Split<1>{{x}}; }
__device__ __forceinline__ Split<3> token_of(const f32x8 x) { return split_of<3>(x); }
template <int P> __device__ __forceinline__ float at(const Split<P> &f, int k) {
  float v = 0.0f;
#pragma unroll
  for (int i = P - 1; i >= 0; --i) v += (float)f.p[i][k];
  return v;
}

// Split matrices in memory: one plane a part, `plane` bytes apart, in fragment order.
//
// Operands are kept in the order in which lanes take them: a matrix of rows x k is cut in 16 x 32
// fragments, the `nk` fragments of 16 rows one after another, each 64 lanes x 8 elements
// (lane = 16 (k / 8 % 4) + row % 16).  One load then is 1 KB on end for a wave; with the rows as
// they are it touches 16 rows, one lookup a lane (measured: 60 against 16 clocks a load).
__device__ __forceinline__ int frag_of(int rt, int kt, int nk) { return ((rt * nk + kt) * 64 + (threadIdx.x & 63)) * 8; }
__device__ __forceinline__ int64_t frag_at(int row, int k, int nk) {
  return ((int64_t)((row >> 4) * nk + (k >> 5)) * 64 + ((k >> 3) & 3) * 16 + (row & 15)) * 8 + (k & 7);
}
// Fragment f of a split (or fp32) matrix.  `base` and f are the same for the whole wave, so that the address
// is a scalar base and the lane's 32-bit offset.
template <int P> __device__ __forceinline__ Split<P> load_frag(const char *base, int64_t plane, int f) {
  const unsigned lane = (threadIdx.x & 63) * 16;
  const char *b = base + (int64_t)f * 1024;
  Split<P> s;
#pragma unroll
  for (int i = 0; i < P; ++i) s.p[i] = *reinterpret_cast<const bf16x8 *>(b + i * plane + lane);
  return s;
}
__device__ __forceinline__ f32x8 load_frag(const float *base, int f) {
  const unsigned lane = (threadIdx.x & 63) * 32;
  return ld8(reinterpret_cast<const float *>(reinterpret_cast<const char *>(base + (int64_t)f * 512) + lane));
}
template <int P> __device__ __forceinline__ Split<P> load_split(const char *base, int64_t plane, int64_t e) {
  Split<P> f;
#pragma unroll
  for (int i = 0; i < P; ++i) f.p[i] = ld8(reinterpret_cast<const __bf16 *>(base + i * plane) + e);
  return f;
}
template <int P> __device__ __forceinline__ void store_split(char *base, int64_t plane, int64_t e, const Split<P> &f) {
#pragma unroll
  for (int i = 0; i < P; ++i) *reinterpret_cast<bf16x8 *>(reinterpret_cast<__bf16 *>(base + i * plane) + e) = f.p[i];
}

// The wave's index in its workgroup, known to be the same for all its lanes.
__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

// Launch-order block id -> work item, so that consecutive items (which read the same tokens and
// chunk terms) run on one XCD: workgroups go round the 8 XCDs.
__device__ __forceinline__ int xcd_item(int id, int n) { return n % 8 == 0 ? (id & 7) * (n >> 3) + (id >> 3) : id; }

// A split matrix in LDS: P parts of R rows of Ccols elements (a multiple of 64).  A ds_read_b128 is served 16
// lanes at a time, which are not 16 lanes on end: eight rows of one 16-byte column and the other eight of the
// column beside it (rows padded by 16 bytes then meet one bank twice: half of the LDS cycles were
// conflicts).  The 16-byte units of a row therefore stand in an order of the row's, by xor: those of 128 bytes
// in tiles of 64 columns, two rows to the 64 banks; those of 64 bytes in wider tiles, whose rows are padded
// by 64 bytes, so that four rows turn round the banks and the column's multiple of 32 elements stays an
// immediate offset (0 2 3 1 for the row's bits 2 and 3).
template <int P, int R, int Ccols> struct SplitTile {
  static constexpr int kPitch = Ccols * 2 + (Ccols > 64 ? 64 : 0), kPlane = R * kPitch;
  // byte offset of element (r, c) in a part
  static __device__ __forceinline__ int at_byte(int r, int c) {
    if (Ccols == 64) return r * kPitch + ((c * 2) ^ ((r >> 1 & 7) << 4));
    const int x = (r >> 1 & 2) ^ (r & 8 ? 3 : 0);
    return r * kPitch + (c >> 5) * 64 + (((c >> 3 & 3) ^ x) << 4) + (c & 7) * 2;
  }
  char b[P * kPlane];
  template <int Q = P> __device__ __forceinline__ Split<Q> ld(int r, int c) const {     // its first Q parts
    return load_split<Q>(b, kPlane, at_byte(r, c) / 2);
  }
  __device__ __forceinline__ void st4(int r, int c, f32x4 v) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      bf16x4 h;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        h[x] = (__bf16)v[x];
        v[x] -= (float)h[x];
      }
      *reinterpret_cast<bf16x4 *>(b + i * kPlane + at_byte(r, c)) = h;
    }
  }
  __device__ __forceinline__ f32x4 at4(int r, int c) const {
    f32x4 v = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int i = P - 1; i >= 0; --i) {
      const bf16x4 h = *reinterpret_cast<const bf16x4 *>(b + i * kPlane + at_byte(r, c));
#pragma unroll
      for (int x = 0; x < 4; ++x) v[x] += (float)h[x];
    }
    return v;
  }
  // four elements to element e of a split matrix in memory
  __device__ __forceinline__ void copy4(int r, int c, char *dst, int64_t plane, int64_t e) const {
#pragma unroll
    for (int i = 0; i < P; ++i)
      *reinterpret_cast<bf16x4 *>(dst + i * plane + e * 2) = *reinterpret_cast<const bf16x4 *>(b + i * kPlane + at_byte(r, c));
  }
  // Lane (g, li)'s rows r0 + 4 g .. + 3 of column c0 + li: to element e of a split matrix in memory, or
  // (their sum, which is the fp32 value for three parts) to fp32 memory.
  __device__ __forceinline__ bf16x4 t4(int part, int r0, int c0) const {
    const int l = threadIdx.x & 63, g = l >> 4, li = l & 15;
    const int o = at_byte(r0 + 4 * g + (li >> 2), c0 + 4 * (li & 3));
    return lds_read_tr16(reinterpret_cast<const unsigned char *>(b) + part * kPlane + o);
  }
  // Lane (g, li)'s eight rows r0 + 8 g .. + 7 of column c0 + li: an operand of the transposed matrix.
  __device__ __forceinline__ Split<P> ld_t(int r0, int c0) const {
    const int l = threadIdx.x & 63, g = l >> 4, li = l & 15;
    const int r = r0 + 8 * g + (li >> 2), c = c0 + 4 * (li & 3);
    const unsigned char *lo = reinterpret_cast<const unsigned char *>(b) + at_byte(r, c);
    const unsigned char *hi = reinterpret_cast<const unsigned char *>(b) + at_byte(r + 4, c);
    Split<P> f;
#pragma unroll
    for (int i = 0; i < P; ++i) f.p[i] = cat8(lds_read_tr16(lo + i * kPlane), lds_read_tr16(hi + i * kPlane));
    return f;
  }
  __device__ __forceinline__ void copy_t4(int r0, int c0, char *dst, int64_t plane, int64_t e) const {
#pragma unroll
    for (int i = 0; i < P; ++i) *reinterpret_cast<bf16x4 *>(dst + i * plane + e * 2) = t4(i, r0, c0);
  }
  __device__ __forceinline__ void copy_t4(int r0, int c0, float *dst) const {
    f32x4 v = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int i = P - 1; i >= 0; --i) {
      const bf16x4 h = t4(i, r0, c0);
#pragma unroll
      for (int x = 0; x < 4; ++x) v[x] += (float)h[x];
    }
    *reinterpret_cast<f32x4 *>(dst) = v;
  }
};

// One lane's column of four rows (t4 .. t4 + 3) of a chunk's token rows, `left` of which exist: a base
// that is the same for the wave and a 32-bit byte offset (64 rows span less than 2 GiB).
template <typename T> struct Rows4 {
  unsigned off, col, step;
  __device__ __forceinline__ Rows4(int t4, int li, int64_t ld) {
    step = (unsigned)(ld * sizeof(T));
    col = li * sizeof(T);
    off = (unsigned)t4 * step + col;
  }
  // rows past the chunk repeat its first
  __device__ __forceinline__ void load(const T *base, int t4, int left, T (&v)[4]) const {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const char *b = reinterpret_cast<const char *>(base) + (int64_t)(r < left ? r : 0) * step;
      v[r] = *reinterpret_cast<const T *>(b + (t4 + r < left ? off : col));
    }
  }
  __device__ __forceinline__ void store(T *base, int t4, int left, const f32x4 v) const {
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (t4 + r < left) *reinterpret_cast<T *>(reinterpret_cast<char *>(base) + (int64_t)r * step + off) = from_f32<T>(v[r]);
  }
};

// The sum over the 16 lanes of a lane group, in every one of them (row rotations, no LDS).
__device__ __forceinline__ float sum16(float v) {
#define TTT_ROR_ADD(N) \
  v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x120 + N, 0xf, 0xf, false))
  TTT_ROR_ADD(8);
  TTT_ROR_ADD(4);
  TTT_ROR_ADD(2);
  TTT_ROR_ADD(1);
#undef TTT_ROR_ADD
  return v;
}

// Workgroup barrier that waits for this wave's LDS traffic only: loads from memory stay in flight.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(15 | (7 << 4) | (3 << 14));      // lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

__device__ __forceinline__ f32x4 zero4() { return f32x4{0, 0, 0, 0}; }

// The state that `count` segments before one leave it, into s[0]: what the first leaves, u_of(0), then
// times M plus U of each other, (u_of(0) m_of(1) + u_of(1)) m_of(2) + ..  Eight waves, a 16 x 16 tile each at
// a time; u_of: this lane's row, m_of: split dk x dk, rows = columns of the product.
template <int DK, typename U, typename M>
__device__ __forceinline__ void join_segments(SplitTile<kFull, kDeltaSlice, DK> (&s)[2], int count, const U &u_of, const M &m_of) {
  constexpr int NK = DK / 32, NW = (DK / 16 + 7) / 8;
  const int wave = wave_id(), l = threadIdx.x & 63, g = l >> 4, li = l & 15;
  for (int j = 0; j < count; ++j) {
    const SplitTile<kFull, kDeltaSlice, DK> &W = s[(count - j) & 1];
    const char *m = m_of(j > 0 ? j : 1);
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      const int tile = wave * NW + i;
      if (tile >= DK / 16) break;
      f32x4 x = *reinterpret_cast<const f32x4 *>(u_of(j) + 16 * tile);
      if (j > 0) {
        Sums<kFull> d;
#pragma unroll 4
        for (int k = 0; k < NK; ++k) d.add(load_frag<kFull>(m, (int64_t)DK * DK * 2, tile * NK + k), W.ld(li, 32 * k + 8 * g));
        x += d.sum();
      }
      s[(count - 1 - j) & 1].st4(li, 16 * tile + 4 * g, x);
    }
    lds_barrier();
  }
}

// Cumulative log decays are summed in 64 bits and kept as two floats, in base 2: their differences, small
// beside them, then are exact to 2^-23, without 64-bit arithmetic for every pair of tokens.
__device__ __forceinline__ float2 log_of(double gam) {
  const double x = gam * 1.4426950408889634;
  const float h = (float)x;
  return float2{h, (float)(x - (double)h)};
}
// e^(gamma_a - gamma_b)
__device__ __forceinline__ float exp_of(float2 a, float2 b) { return __builtin_amdgcn_exp2f((a.x - b.x) + (a.y - b.y)); }
__device__ __forceinline__ float exp_of(double x) { return __builtin_amdgcn_exp2f((float)(x * 1.4426950408889634)); }

}  // namespace ttt
