// Newton-Schulz orthogonalisation of a batch of matrices of any size:
//   X = G / (|G|_F + eps) (transposed while G has more rows than columns), then `steps` times
//   A = X X^T,  B = a I + b A + c A A,  X <- B X.
//
// All products run on fp16 MFMA with fp32 accumulation, on operands of two fp16 parts,
// x = h + l, l = fp16(x - h): 22 bits, products h*h + h*l + l*h.  Every matrix here has a spectral
// norm below 3.9 (X 1.2, A 1.5, B 3.45): stored times 2^14 its elements stay in fp16's range, and an element
// above 2^-17 keeps its low part out of the subnormal numbers; what smaller ones lose is below 2^-38.
// (X is that small throughout only where |G| is below 1e-10, where 1e-7 beside it leaves X near zero.)
// One part would not do: the steps multiply what is lost along small singular directions by up to 3.4445
// each, 485 in five, and even one part in only the last two steps of bf16 matrices, where that is 3.4 and the
// result has 8 bits, left it 1.57e-3 off the 64-bit result rounded (4 x 4096 x 1024), with two 7.7e-5 (fp32
// arithmetic 1.3e-4).
// bf16 matrices enter the first step exactly in one part, times a power of two, with the rest of 1 / |G|
// applied to A and X.
// Measured off the definition in 64 bits, 2 x 1300 x 1200 fp32: 1.2e-6 (fp32 arithmetic 3.2e-6, three bf16
// parts and six products 3.0e-6 at 1.6 times the time); 4 x 4096 x 1024 bf16: 1.66e-3, the rounding of the
// result alone.
// The parts are written as planes by the kernel that computes a matrix, so that the main loop
// copies tiles from memory straight into LDS.  Every product is C[i][j] = sum_k P[i][k] Q[j][k]
// of row panels: X X^T, A A (A is symmetric) and B X from the stored X^T; A and B are
// symmetric, so only their tiles on and below the diagonal are computed.  Bound by the matrix cores
// where matrices are large: 4 x 4096 x 1024 bf16, five steps, 279 GFLOP (805 with the parts, tiles above the
// diagonal left out) in 895 us, 900 TFLOP/s (B X about 1000, A 640 and B 510, whose 144 tiles leave 112 of the
// CUs out); small ones by their 17 launches: 12 x 512 x 256 fp32 119 us.
// Sizes are padded with zeros to whole tiles.
#include <type_traits>

#include "common.h"
#include "dma.h"
#include "orth.h"

namespace ttt {
namespace {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ f32x4 mma(const f16x8 a, const f16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// Called on a value before it is split in h and l.  Folded into the conversions, the arithmetic before gives an h
// rounded once (v_fma_mix) for the one of its two uses and twice (v_mul, v_cvt) for the other: where they differ,
// one value in some thousands, l is taken from another h than the one stored, and 2^-11 is lost.
__device__ __forceinline__ void settle(f32x4 &v) { asm("" : "+v"(v)); }

constexpr int KS = 32;              // reduction elements a stage
constexpr float kUnit = 16384.0f;   // a stored element for 1

// Split matrix: one plane a part.  A plane is cut in fragments of 16 rows x 32 columns, 1 KB each in
// the order in which lanes take them (lane = 16 (column / 8 % 4) + row % 16, eight columns a lane),
// the nrt fragments of 32 columns one after another: a stage's panel is one piece of memory.  (With
// plain rows a copy of 16 rows meets one channel of the L2 where the row length is a power of two:
// 93 against 91 us for the symmetric products of four 1024 x 4096 matrices, 64 x 64 tiles of 512-wide
// ones 13.7 against 11.9.)
struct Mat {
  char *p;
  int64_t plane, bs;                // bytes from plane to plane, from matrix to matrix
  int nrt;                          // fragments of rows
};
__device__ __forceinline__ int64_t frag_byte(const Mat &m, int rt, int kt) { return ((int64_t)kt * m.nrt + rt) * 1024; }

// Eight values as one lane's piece of a fragment, in `parts` parts.
__device__ __forceinline__ void put8(char *p, int64_t plane, int parts, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (i >= parts) break;
    f16x8 h;
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      h[r] = (_Float16)v[r];
      v[r] -= (float)h[r];
    }
    *reinterpret_cast<f16x8 *>(p + i * plane) = h;
  }
}
// Elements (row, col .. col + 3), col % 4 == 0, of a matrix of P parts.
template <int P> __device__ __forceinline__ f32x4 get4(const Mat &m, int64_t base, int row, int col) {
  const char *p = m.p + base + frag_byte(m, row >> 4, col >> 5) + (((col >> 3) & 3) * 16 + (row & 15)) * 16 + (col & 7) * 2;
  f32x4 v = f32x4{0, 0, 0, 0};
#pragma unroll
  for (int i = P - 1; i >= 0; --i) {
    const f16x4 h = *reinterpret_cast<const f16x4 *>(p + i * m.plane);
#pragma unroll
    for (int r = 0; r < 4; ++r) v[r] += (float)h[r];
  }
  return v;
}

// Partial sums of squares, in 64 bits: block x of matrix y, V elements (a 16-byte piece, or one) a load.
template <typename T, int V>
__global__ __launch_bounds__(256) void orth_norm_kernel(OrthParams p, double *part) {
  __shared__ double red[4];
  const T *g = static_cast<const T *>(p.g) + (int64_t)blockIdx.y * p.bsg;
  // thread e, e + step, ..: row and piece move by a fixed amount, with a carry
  const unsigned step = gridDim.x * 256, e0 = blockIdx.x * 256 + threadIdx.x, np = p.plan.cols / V;
  const unsigned dr = step / np, dc = step % np, rows = p.plan.rows;
  unsigned r = e0 / np, c = e0 % np;
  double s = 0.0;
  while (r < rows) {
    float x[4][V];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const T *at = g + (int64_t)r * p.ldg + c * V;
#pragma unroll
      for (int k = 0; k < V; ++k) x[i][k] = 0.0f;
      if (r < rows) {
        if constexpr (V == 1) {
          x[i][0] = to_f32(*at);
        } else {
          typedef T piece __attribute__((ext_vector_type(V)));
          const piece v = *reinterpret_cast<const piece *>(at);
#pragma unroll
          for (int k = 0; k < V; ++k) x[i][k] = (float)v[k];
        }
      }
      r += dr, c += dc;
      if (c >= np) c -= np, ++r;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int k = 0; k < V; ++k) s += (double)x[i][k] * (double)x[i][k];
  }
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) s += __shfl_xor(s, m);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) part[(int64_t)blockIdx.y * gridDim.x + blockIdx.x] = (red[0] + red[1]) + (red[2] + red[3]);
}

// 1 / (|G| + eps) of matrix b, by every wave (the partials in one fixed order).
__device__ __forceinline__ double orth_scale(const OrthParams &p, const double *part, int b) {
  double s = 0.0;
  for (int i = threadIdx.x & 63; i < p.plan.norm_blocks; i += 64) s += part[(int64_t)b * p.plan.norm_blocks + i];
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) s += __shfl_xor(s, m);
  return 1.0 / (sqrt(s) + (double)p.eps);
}

// X and X^T of the first step: G scaled, split and padded.  64 x 64 tiles of [rows][cols].  bf16
// matrices are scaled by the power of two below 1 / |G|, exactly; the factor left over goes to rest[b].
template <typename T>
__global__ __launch_bounds__(256) void orth_load_kernel(OrthParams p, const double *part, float *rest, Mat x, Mat xt) {
  __shared__ float tile[64][65];
  const OrthPlan &q = p.plan;
  const int b = blockIdx.z;
  const int r0 = blockIdx.y * 64, c0 = blockIdx.x * 64, tx = threadIdx.x & 63, w = threadIdx.x >> 6;
  const T *g = static_cast<const T *>(p.g) + b * p.bsg;
  float in[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int r = r0 + w + 4 * i, c = c0 + tx;
    in[i] = r < q.rows && c < q.cols ? to_f32(g[(int64_t)r * p.ldg + c]) : 0.0f;
  }
  double scale = orth_scale(p, part, b);
  const bool exact = sizeof(T) == 2 && !q.narrow;
  if (exact) {
    int e;
    const double f = frexp(scale, &e);                        // scale = f 2^e, f in [1/2, 1)
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) rest[b] = (float)(2.0 * f);
    scale = ldexp(1.0, e - 1);
    if (!(f == f)) scale = f;                                 // NaN stays NaN
  }
  scale *= (double)kUnit;
#pragma unroll
  for (int i = 0; i < 16; ++i) tile[w + 4 * i][tx] = (float)((double)in[i] * scale);
  __syncthreads();
  const Mat &m = q.tall ? xt : x, &mt = q.tall ? x : xt;      // G's own layout, and its transpose
  const int gr = tx >> 4, li = tx & 15, parts = exact ? 1 : 2;
#pragma unroll
  for (int k = 0; k < 2; ++k) {                               // wave w: fragment rows w
    float v[8], u[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      v[e] = tile[16 * w + li][32 * k + 8 * gr + e];
      u[e] = tile[32 * k + 8 * gr + e][16 * w + li];
    }
    put8(m.p + b * m.bs + frag_byte(m, r0 / 16 + w, c0 / 32 + k) + tx * 16, m.plane, parts, v);
    put8(mt.p + b * mt.bs + frag_byte(mt, c0 / 16 + w, r0 / 32 + k) + tx * 16, mt.plane, parts, u);
  }
}

// What a product's tile becomes.
enum Kind { kGram, kPoly, kNext, kLast };   // A;  B = a I + b A + c A A;  X and X^T;  the result
struct Product {
  Mat P, Q;                         // C = P Q^T
  Mat c, ct;                        // results: [i][j] and [j][i] (the same matrix where C is symmetric)
  const float *rest;                // [matrix] factor of each X in it (1 in kNext, 2 in kGram), or null
  int K, ti, tj;                    // reduction length, tiles along i and j
  int tiles;                        // tiles a matrix
};

// A workgroup's tile: TM x TN by WR x WC waves, a ring of NST stages of KS reduction elements.
// Both operands pass through LDS once a stage; a wave's fragment reads against its MFMAs fall
// with the wave tile, which sets the sizes (reads and copies share the LDS with 128 bytes a clock,
// 16 clocks an MFMA and SIMD): 256 x 256 where such tiles fill the card, 128 x 128 where those do,
// else 64 x 64.  Two waves share a SIMD (of one workgroup, or of two 64 x 64 ones on a CU), so that one's
// reads fall on the other's products; reading a stage ahead into registers instead, with a wave a SIMD,
// was slower (112 against 84 us for the symmetric products of four 1024 x 4096 matrices).
template <int TM_, int TN_, int WR_, int WC_, int NST_> struct Geo {
  static constexpr int TM = TM_, TN = TN_, WR = WR_, WC = WC_, NST = NST_, kThreads = WR * WC * 64;
  static constexpr int WM = TM / WR, WN = TN / WC, FM = WM / 16, FN = WN / 16;
};
// N: parts of both operands together (2, 3 or 4): the deeper ring where a stage is smaller
template <int TILE, int N> struct GeoOf;
template <int N> struct GeoOf<64, N> { typedef Geo<64, 64, 2, 2, N == 4 ? 5 : 6> type; };
template <int N> struct GeoOf<128, N> { typedef Geo<128, 128, 4, 2, N == 4 ? 4 : N == 3 ? 3 : 5> type; };
template <int N> struct GeoOf<256, N> { typedef Geo<256, 256, 4, 2, N == 2 ? 4 : 2> type; };

template <typename T, typename G, int PA, int PB, int KIND>
__global__ __launch_bounds__(G::kThreads, G::kThreads / 256) void orth_product_kernel(OrthParams p, Product q) {
  constexpr int kRows = G::TM * PA + G::TN * PB, kStage = kRows * 64, kWaves = G::kThreads / 64;
  constexpr int PPW = kRows / 16 / kWaves;        // copies of 16 rows a wave and stage
  constexpr int kPitch = G::WN * 2 + 16;          // epilogue: a row of a wave's tile of one part
  constexpr int kEpi = kWaves * G::WM * kPitch;
  static_assert(kRows / 16 % kWaves == 0, "a stage splits evenly over the waves");
  __shared__ __attribute__((aligned(16))) unsigned char s[G::NST * kStage > kEpi ? G::NST * kStage : kEpi];
  const int t = threadIdx.x, w = __builtin_amdgcn_readfirstlane(t >> 6), l = t & 63, g = l >> 4, li = l & 15;
  // consecutive tiles (which share panels) on one XCD: workgroups go round the 8 XCDs
  const int n = gridDim.x, id = n % 8 == 0 ? (blockIdx.x & 7) * (n >> 3) + (blockIdx.x >> 3) : blockIdx.x;
  const int b = id / q.tiles;
  int e = id % q.tiles, bi, bj;
  if (KIND == kGram || KIND == kPoly) {           // on and below the diagonal
    bi = 0;
    while (e > bi) e -= ++bi;
    bj = e;
  } else {
    bi = e % q.ti, bj = e / q.ti;
  }
  // A stage holds, part by part, the fragments of the P panel, then those of the Q panel.
  const char *src[PPW];
  int64_t step_bytes[2] = {(int64_t)q.P.nrt * 1024, (int64_t)q.Q.nrt * 1024};
#pragma unroll
  for (int x = 0; x < PPW; ++x) {
    const int f = w * PPW + x;                    // fragment of the stage
    const bool second = f >= G::TM / 16 * PA;
    const int r = second ? f - G::TM / 16 * PA : f, nf = second ? G::TN / 16 : G::TM / 16;
    const Mat &m = second ? q.Q : q.P;
    src[x] = m.p + b * m.bs + r / nf * m.plane + frag_byte(m, (second ? bj : bi) * nf + r % nf, 0) + l * 16;
  }
  const int nk = q.K / KS;
  const auto copy = [&](int x, int kc) {
    const bool second = w * PPW + x >= G::TM / 16 * PA;
    copy16_to_lds_untracked(src[x] + kc * step_bytes[second], s + kc % G::NST * kStage + (w * PPW + x) * 1024);
  };
  f32x4 acc[G::FM][G::FN];
#pragma unroll
  for (int i = 0; i < G::FM; ++i)
#pragma unroll
    for (int j = 0; j < G::FN; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
  // The products of low parts in sums of their own, where registers allow it: a large sum then is rounded
  // once a stage, not three times (2 x 36 x 1216 fp32: 3.2e-6 -> 2.2e-6 off, 2 x 1300 x 1200 2.1e-6 -> 1.2e-6).
  // Tiles of 256, whose sums take half of the registers, go without: 4 x 4096 x 1024 fp32 1.4e-6 off and 2 x 2000 x
  // 3900 1.8e-6, where fp32 arithmetic is 3.7e-6 and 4.4e-6.
  constexpr bool kLow = PA == 2 && PB == 2 && G::TM <= 128;
  f32x4 low[kLow ? G::FM : 1][kLow ? G::FN : 1];
#pragma unroll
  for (auto &row : low)
#pragma unroll
    for (auto &v : row) v = f32x4{0, 0, 0, 0};
  const int wi = (w / G::WC) * G::WM, wj = (w % G::WC) * G::WN;
#pragma unroll
  for (int k = 0; k < G::NST - 1; ++k)
    if (k < nk)
#pragma unroll
      for (int x = 0; x < PPW; ++x) copy(x, k);
  const auto read = [&](const unsigned char *st, int row) {     // the fragment of a stage's row
    return *reinterpret_cast<const f16x8 *>(st + row * 64 + l * 16);
  };
  // products with the fragments of one column tile, the small ones first
  constexpr int ND = PA > PB ? PA : PB;
  const auto products = [&](int j, const f16x8 (&fa)[G::FM][PA], const f16x8 (&fb)[PB]) {
#pragma unroll
    for (int d = ND - 1; d >= 0; --d)
#pragma unroll
      for (int x = 0; x <= d; ++x)
        if (x < PA && d - x < PB)
#pragma unroll
          for (int i = 0; i < G::FM; ++i) {
            f32x4 &sum = kLow && d > 0 ? low[kLow ? i : 0][kLow ? j : 0] : acc[i][j];
            sum = mma(fb[d - x], fa[i][x], sum);
          }
  };
  for (int kc = 0; kc < nk; ++kc) {
    // this wave's copies of stage kc have arrived (those of the NST - 2 stages after it may be in flight)
    if (kc + G::NST - 2 < nk) wait_vmcnt<(G::NST - 2) * PPW>(); else wait_vmcnt<0>();
    bare_barrier();                             // everyone's have, and the stage before is free
    const unsigned char *st = s + kc % G::NST * kStage;
    const bool more = kc + G::NST - 1 < nk;
    f16x8 fa[G::FM][PA], fb[2][PB];
    const auto read_b = [&](int j, f16x8 (&f)[PB]) {
#pragma unroll
      for (int x = 0; x < PB; ++x) f[x] = read(st, G::TM * PA + x * G::TN + wj + 16 * j);
    };
#pragma unroll
    for (int x = 0; x < PA; ++x)
#pragma unroll
      for (int i = 0; i < G::FM; ++i) fa[i][x] = read(st, x * G::TM + wi + 16 * i);
    read_b(0, fb[0]);
#pragma unroll
    for (int j = 0; j < G::FN; ++j) {
      if (j + 1 < G::FN) read_b(j + 1, fb[(j + 1) & 1]);
      // the next stage's copies, spread over the products
#pragma unroll
      for (int x = 0; x < PPW; ++x)
        if (x * G::FN / PPW == j && more) copy(x, kc + G::NST - 1);
      products(j, fa, fb[j & 1]);
    }
  }
  __syncthreads();                                // the ring is free
  if constexpr (kLow)
#pragma unroll
    for (int i = 0; i < G::FM; ++i)
#pragma unroll
      for (int j = 0; j < G::FN; ++j) acc[i][j] += low[i][j];
  // lane (g, li) holds C[16 i + li][16 j + 4 g + r], r = 0 .. 3, of the wave's tile
  const int r0 = bi * G::TM + wi, c0 = bj * G::TN + wj;
  if constexpr (KIND == kPoly) {
#pragma unroll
    for (int i = 0; i < G::FM; ++i)
#pragma unroll
      for (int j = 0; j < G::FN; ++j) {
        const int row = r0 + 16 * i + li, col = c0 + 16 * j + 4 * g;
        const f32x4 a = get4<PA>(q.P, b * q.P.bs, row, col);
#pragma unroll
        for (int r = 0; r < 4; ++r)
          acc[i][j][r] = (p.c / kUnit) * acc[i][j][r] + (p.b * a[r] + (row == col + r ? p.a * kUnit : 0.0f));
      }
  } else {
    // back to one kUnit (the result: none)
    float f = KIND == kLast ? 1.0f / (kUnit * kUnit) : 1.0f / kUnit;
    if (q.rest) f *= KIND == kGram ? q.rest[b] * q.rest[b] : q.rest[b];
#pragma unroll
    for (int i = 0; i < G::FM; ++i)
#pragma unroll
      for (int j = 0; j < G::FN; ++j) acc[i][j] *= f;
  }
  if constexpr (KIND == kLast) {
    T *out = static_cast<T *>(p.out) + b * p.bso;
#pragma unroll
    for (int i = 0; i < G::FM; ++i)
#pragma unroll
      for (int j = 0; j < G::FN; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = r0 + 16 * i + li, col = c0 + 16 * j + 4 * g + r;
          if (row >= p.plan.r || col >= p.plan.c) continue;
          const int64_t o = p.plan.tall ? (int64_t)col * p.ldo + row : (int64_t)row * p.ldo + col;
          out[o] = from_f32<T>(acc[i][j][r]);
        }
    return;
  }
  // Parts, one at a time, through the wave's own piece of LDS: whole rows of C out of it as they
  // are, and of C^T by transposing reads.
#pragma unroll
  for (int i = 0; i < G::FM; ++i)
#pragma unroll
    for (int j = 0; j < G::FN; ++j) settle(acc[i][j]);
  unsigned char *mine = s + w * (G::WM * kPitch);
  const bool both = KIND == kNext || bi != bj;
#pragma unroll
  for (int x = 0; x < 2; ++x) {
#pragma unroll
    for (int i = 0; i < G::FM; ++i)
#pragma unroll
      for (int j = 0; j < G::FN; ++j) {
        f16x4 h;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          h[r] = (_Float16)acc[i][j][r];
          acc[i][j][r] -= (float)h[r];
        }
        *reinterpret_cast<f16x4 *>(mine + (16 * i + li) * kPitch + (16 * j + 4 * g) * 2) = h;
      }
    char *c = q.c.p + b * q.c.bs + x * q.c.plane + l * 16;
#pragma unroll
    for (int i = 0; i < G::FM; ++i)
#pragma unroll
      for (int k = 0; k < G::WN / 32; ++k)        // columns 32 k + 8 g .. + 7 of row 16 i + li
        *reinterpret_cast<u32x4 *>(c + frag_byte(q.c, r0 / 16 + i, c0 / 32 + k)) =
            *reinterpret_cast<const u32x4 *>(mine + (16 * i + li) * kPitch + (32 * k + 8 * g) * 2);
    if (both) {
      char *ct = q.ct.p + b * q.ct.bs + x * q.ct.plane + l * 16;
#pragma unroll
      for (int i = 0; i < G::WM / 32; ++i)
#pragma unroll
        for (int j = 0; j < G::FN; ++j) {         // rows 32 i + 8 g .. + 7 of column 16 j + li
          const unsigned char *a = mine + (32 * i + 8 * g + (li >> 2)) * kPitch + (16 * j + 4 * (li & 3)) * 2;
          *reinterpret_cast<bf16x8 *>(ct + frag_byte(q.ct, c0 / 16 + j, r0 / 32 + i)) =
              cat8(lds_read_tr16(a), lds_read_tr16(a + 4 * kPitch));
        }
    }
  }
}

// ------------------------------------------------------------------ at most 64 rows
// A whole step in one launch, a workgroup per 64 columns: A is the sum of what the tiles gave (in tile order),
// B = a I + b A + c A A, this tile's B X, and its part of the next A.  A and B are 64 x 64 and computed by every
// workgroup; they take three parts (22 bits are what would be off: where b A and a I cancel, 1 x 1400 x 50 fp32
// 2.3e-6 with two, 1.3e-6 with three, fp32 arithmetic 1.4e-6).  Bound by latency: the sum, four products and their
// exchanges; 2 x 36 x 1216 fp32 61 us in 8 launches, as large matrices are done 101 in 17.
// Matrices in LDS in fragments too: [part][column / 32][row / 16], 1 KB each.
template <typename T>
__global__ __launch_bounds__(256) void orth_narrow_kernel(OrthParams p, Mat x, Mat xt, const float *in, float *out, bool first,
                                                          bool last) {
  __shared__ __attribute__((aligned(16))) unsigned char s_m[3 * 8 * 1024], s_x[2 * 8 * 1024];
  const OrthPlan &q = p.plan;
  const int nt = q.cp / 64, b = blockIdx.x / nt, tile = blockIdx.x % nt, t = threadIdx.x;
  const int w = __builtin_amdgcn_readfirstlane(t >> 6), l = t & 63, g = l >> 4, li = l & 15;
  const int rt0 = (w >> 1) * 2, ct0 = (w & 1) * 2;      // this wave's 32 x 32 of every product, in fragments
  // element (row, col .. col + 3) of a part
  const auto at = [&](unsigned char *m, int part, int row, int col) {
    return m + (part * 8 + (col >> 5) * 4 + (row >> 4)) * 1024 + ((col >> 3 & 3) * 16 + (row & 15)) * 16 + (col & 7) * 2;
  };
  // lane (g, li) has C[16 i + li][16 j + 4 g + r] of its wave's tiles
  const auto put = [&](unsigned char *m, int parts, const f32x4 (&c)[2][2]) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        f32x4 v = c[i][j];
        settle(v);
#pragma unroll
        for (int k = 0; k < 3; ++k) {
          if (k >= parts) break;
          f16x4 h;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            h[r] = (_Float16)v[r];
            v[r] -= (float)h[r];
          }
          *reinterpret_cast<f16x4 *>(at(m, k, 16 * (rt0 + i) + li, 16 * (ct0 + j) + 4 * g)) = h;
        }
      }
  };
  const auto frag = [&](const unsigned char *m, int part, int rt, int kt) {
    return *reinterpret_cast<const f16x8 *>(m + (part * 8 + kt * 4 + rt) * 1024 + l * 16);
  };
  // C = P Q^T over 64, P of PP parts in LDS, Q of PQ from `qf`(part, fragment row, kt)
  const auto product = [&](auto pp, auto pq, const unsigned char *P, auto qf, f32x4 (&c)[2][2]) {
    constexpr int PP = decltype(pp)::value, PQ = decltype(pq)::value, N = PP > PQ ? PP : PQ;
    f32x4 low[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) c[i][j] = low[i][j] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int kt = 0; kt < 2; ++kt) {
      f16x8 fa[2][PP], fb[2][PQ];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int k = 0; k < PP; ++k) fa[i][k] = frag(P, k, rt0 + i, kt);
#pragma unroll
        for (int k = 0; k < PQ; ++k) fb[i][k] = qf(k, ct0 + i, kt);
      }
#pragma unroll
      for (int d = N - 1; d >= 0; --d)
#pragma unroll
        for (int k = 0; k <= d; ++k)
          if (k < PP && d - k < PQ)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                f32x4 &sum = d > 0 ? low[i][j] : c[i][j];
                sum = mma(fb[j][d - k], fa[i][k], sum);
              }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) c[i][j] += low[i][j];
  };
  typedef std::integral_constant<int, 2> Two;
  typedef std::integral_constant<int, 3> Three;
  f32x4 c[2][2];
  if (first) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {                       // X's fragments as they are
      const int f = w + 4 * e, part = f >> 3, kt = f >> 2 & 1, rt = f & 3;
      *reinterpret_cast<u32x4 *>(s_x + f * 1024 + l * 16) =
          *reinterpret_cast<const u32x4 *>(x.p + b * x.bs + part * x.plane + frag_byte(x, rt, 2 * tile + kt) + l * 16);
    }
  } else {
    f32x4 a[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) a[i][j] = f32x4{0, 0, 0, 0};
    const float *src = in + (int64_t)b * nt * 4096 + t * 4;
#pragma unroll 4
    for (int k = 0; k < nt; ++k)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) a[i][j] += *reinterpret_cast<const f32x4 *>(src + (int64_t)k * 4096 + (2 * i + j) * 1024);
    put(s_m, 3, a);
    __syncthreads();
    product(Three{}, Three{}, s_m, [&](int k, int rt, int kt) { return frag(s_m, k, rt, kt); }, c);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          c[i][j][r] = (p.c / kUnit) * c[i][j][r] +
                       (p.b * a[i][j][r] + (16 * (rt0 + i) + li == 16 * (ct0 + j) + 4 * g + r ? p.a * kUnit : 0.0f));
    __syncthreads();
    put(s_m, 3, c);
    __syncthreads();
    product(Three{}, Two{}, s_m, [&](int k, int rt, int kt) {
      return *reinterpret_cast<const f16x8 *>(xt.p + b * xt.bs + k * xt.plane + frag_byte(xt, 4 * tile + rt, kt) + l * 16);
    }, c);
    const float f = last ? 1.0f / (kUnit * kUnit) : 1.0f / kUnit;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) c[i][j] *= f;
    if (last) {
      T *o = static_cast<T *>(p.out) + b * p.bso;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int row = 16 * (rt0 + i) + li, col = 64 * tile + 16 * (ct0 + j) + 4 * g + r;
            if (row < q.r && col < q.c) o[q.tall ? (int64_t)col * p.ldo + row : (int64_t)row * p.ldo + col] = from_f32<T>(c[i][j][r]);
          }
      return;
    }
    put(s_x, 2, c);
  }
  __syncthreads();
  if (!first) {         // X^T of the tile, in place: only this workgroup reads it, and has
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int f = w + 4 * e, part = f >> 3, kt = f >> 2 & 1, rt = f & 3;
      const int row = 32 * kt + 8 * g + (li >> 2), col = 16 * rt + 4 * (li & 3);
      *reinterpret_cast<bf16x8 *>(xt.p + b * xt.bs + part * xt.plane + frag_byte(xt, 4 * tile + rt, kt) + l * 16) =
          cat8(lds_read_tr16(at(s_x, part, row, col)), lds_read_tr16(at(s_x, part, row + 4, col)));
    }
  }
  product(Two{}, Two{}, s_x, [&](int k, int rt, int kt) { return frag(s_x, k, rt, kt); }, c);
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
      *reinterpret_cast<f32x4 *>(out + ((int64_t)b * nt + tile) * 4096 + (2 * i + j) * 1024 + t * 4) = c[i][j] * (1.0f / kUnit);
}

// G as it is (steps = 0): only scaled.
template <typename T>
__global__ __launch_bounds__(256) void orth_scale_kernel(OrthParams p, const double *part) {
  const OrthPlan &q = p.plan;
  const int b = blockIdx.y;
  const double scale = orth_scale(p, part, b);
  const int64_t total = (int64_t)q.rows * q.cols;
  for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < total; e += (int64_t)gridDim.x * 256) {
    const int64_t r = e / q.cols, c = e % q.cols;
    static_cast<T *>(p.out)[b * p.bso + r * p.ldo + c] =
        from_f32<T>((float)((double)to_f32(static_cast<const T *>(p.g)[b * p.bsg + r * p.ldg + c]) * scale));
  }
}

template <typename T, int PA, int PB, int KIND, int TILE>
void product_of(const OrthParams &p, Product q, int rows, int cols, hipStream_t s) {
  typedef typename GeoOf<TILE, PA + PB>::type G;
  const bool sym = KIND == kGram || KIND == kPoly;
  q.ti = rows / G::TM, q.tj = cols / G::TN;
  q.tiles = sym ? q.ti * (q.ti + 1) / 2 : q.ti * q.tj;
  hipLaunchKernelGGL((orth_product_kernel<T, G, PA, PB, KIND>), dim3((unsigned)(p.plan.batch * q.tiles)),
                     dim3(G::kThreads), 0, s, p, q);
}
template <typename T, int PA, int PB, int KIND>
void product(const OrthParams &p, const Product &q, int rows, int cols, hipStream_t s) {
  // symmetric results: square tiles of at most 128, so that half of them stay away
  const int tile = KIND == kGram || KIND == kPoly ? p.plan.tile_sym : p.plan.tile;
  if constexpr (KIND == kNext || KIND == kLast) {
    if (tile == 256) return product_of<T, PA, PB, KIND, 256>(p, q, rows, cols, s);
  }
  if (tile == 128) return product_of<T, PA, PB, KIND, 128>(p, q, rows, cols, s);
  product_of<T, PA, PB, KIND, 64>(p, q, rows, cols, s);
}

template <typename T> hipError_t run_orth(const OrthParams &p, hipStream_t s) {
  const OrthPlan &q = p.plan;
  double *part = reinterpret_cast<double *>(p.ws + q.off_norm);
  float *rest = reinterpret_cast<float *>(p.ws + q.off_rest);
  constexpr int V = 16 / (int)sizeof(T);
  constexpr bool kBf16 = sizeof(T) == 2;
  if ((uintptr_t)p.g % 16 == 0 && q.cols % V == 0 && p.ldg % V == 0 && p.bsg % V == 0)
    hipLaunchKernelGGL((orth_norm_kernel<T, V>), dim3(q.norm_blocks, q.batch), dim3(256), 0, s, p, part);
  else
    hipLaunchKernelGGL((orth_norm_kernel<T, 1>), dim3(q.norm_blocks, q.batch), dim3(256), 0, s, p, part);
  if (p.steps == 0) {
    hipLaunchKernelGGL(orth_scale_kernel<T>, dim3(q.norm_blocks, q.batch), dim3(256), 0, s, p, part);
    return hipGetLastError();
  }
  const int64_t xb = (int64_t)q.rp * q.cp * 2, ab = (int64_t)q.rp * q.rp * 2;
  Mat x[2], xt[2];
  for (int i = 0; i < 2; ++i) {
    x[i] = Mat{p.ws + q.off_x[i], xb, 2 * xb, q.rp / 16};
    xt[i] = Mat{p.ws + q.off_xt[i], xb, 2 * xb, q.cp / 16};
  }
  const Mat A{p.ws + q.off_a, ab, 2 * ab, q.rp / 16}, B{p.ws + q.off_b, ab, 2 * ab, q.rp / 16};
  const int pr = q.tall ? q.cp : q.rp, pc = q.tall ? q.rp : q.cp;       // padded sizes of G
  hipLaunchKernelGGL(orth_load_kernel<T>, dim3(pc / 64, pr / 64, q.batch), dim3(256), 0, s, p, part, rest, x[0], xt[0]);
  if (q.narrow) {       // the sums over tiles take the room of the other X and X^T
    float *sums[2] = {reinterpret_cast<float *>(p.ws + q.off_x[1]), reinterpret_cast<float *>(p.ws + q.off_xt[1])};
    const dim3 grid((unsigned)((int64_t)q.batch * (q.cp / 64)));
    for (int i = 0; i <= p.steps; ++i)
      hipLaunchKernelGGL((orth_narrow_kernel<T>), grid, dim3(256), 0, s, p, x[0], xt[0], sums[~i & 1], sums[i & 1], i == 0,
                         i == p.steps);
    return hipGetLastError();
  }
  for (int i = 0; i < p.steps; ++i) {
    const int cur = i & 1;
    const bool one = kBf16 && i == 0;                         // X is one part, exactly
    const float *f = one ? rest : nullptr;
    const Product gram{x[cur], x[cur], A, A, f, q.cp}, poly{A, A, B, B, nullptr, q.rp};
    const Product next{B, xt[cur], x[cur ^ 1], xt[cur ^ 1], f, q.rp};
    if (one) product<float, 1, 1, kGram>(p, gram, q.rp, q.rp, s); else product<float, 2, 2, kGram>(p, gram, q.rp, q.rp, s);
    product<float, 2, 2, kPoly>(p, poly, q.rp, q.rp, s);
    if (i + 1 < p.steps) {
      if (one) product<float, 2, 1, kNext>(p, next, q.rp, q.cp, s); else product<float, 2, 2, kNext>(p, next, q.rp, q.cp, s);
    } else {
      if (one) product<T, 2, 1, kLast>(p, next, q.rp, q.cp, s); else product<T, 2, 2, kLast>(p, next, q.rp, q.cp, s);
    }
  }
  return hipGetLastError();
}

}  // namespace

OrthPlan plan_orth(int rows, int cols, int batch, bool bf16) {
  OrthPlan q{};
  q.rows = rows, q.cols = cols, q.batch = batch, q.bf16 = bf16;
  q.tall = rows > cols;
  q.r = q.tall ? cols : rows, q.c = q.tall ? rows : cols;
  // The largest tile that still fills the card and is not mostly padding: the products' work, rows^2 x columns in
  // whole tiles, may be a third above that in tiles of 64, which is what a larger tile's rate makes up for.  bf16,
  // with that limit and without: 64 x 128 x 1024 201 and 408 us, 200 x 100 x 120 153 and 478, 64 x 300 x 1024 734 and
  // 1137, 40 x 300 x 1400 640 and 1008; 8 x 768 x 2048 616 in tiles of 256 and 697 of 64, 2 x 1300 x 5100 (1.31 times
  // the work) 1165 and 1273.
  const auto up = [](int64_t x, int t) { return (x + t - 1) / t * t; };
  const auto tiles = [&](int t) { return batch * (up(q.r, t) / t) * (up(q.c, t) / t); };
  const auto work = [&](int t) { return up(q.r, t) * up(q.r, t) * up(q.c, t); };
  const auto fits = [&](int t) { return 3 * work(t) <= 4 * work(64); };
  q.tile = tiles(256) >= 200 && fits(256) ? 256 : (tiles(128) >= 200 && fits(128) ? 128 : 64);
  const int64_t nr = up(q.r, 128) / 128;
  q.tile_sym = batch * (nr * (nr + 1) / 2) >= 100 && fits(128) ? 128 : 64;
  // one tile of rows, and few enough of columns that every workgroup sums all of theirs: a launch a step (1 x 64 x
  // 8192 fp32 139 us; as larger matrices are done, 1 x 64 x 8200 362)
  q.narrow = q.r <= 64 && q.c <= 8192;
  if (q.narrow) q.tile = q.tile_sym = 64;
  const int pad = q.tile > q.tile_sym ? q.tile : q.tile_sym;
  q.rp = (q.r + pad - 1) / pad * pad, q.cp = (q.c + pad - 1) / pad * pad;
  const int64_t elems = (int64_t)rows * cols, blocks = (elems + 4095) / 4096;
  q.norm_blocks = (int)(blocks < 1 ? 1 : (blocks > 256 ? 256 : blocks));
  const auto al = [](size_t x) { return (x + 255) & ~size_t(255); };
  const size_t xb = (size_t)q.rp * q.cp * 4 * batch, ab = (size_t)q.rp * q.rp * 4 * batch;
  size_t o = 0;
  q.off_norm = o, o = al(o + (size_t)batch * q.norm_blocks * 8);
  q.off_rest = o, o = al(o + (size_t)batch * 4);
  for (int i = 0; i < 2; ++i) {
    q.off_x[i] = o, o = al(o + xb);
    q.off_xt[i] = o, o = al(o + xb);
  }
  q.off_a = o, o = al(o + ab);
  q.off_b = o, o = al(o + ab);
  q.total = o;
  return q;
}

hipError_t launch_orth(const OrthParams &p, hipStream_t s) {
  return p.plan.bf16 ? run_orth<__bf16>(p, s) : run_orth<float>(p, s);
}

}  // namespace ttt
