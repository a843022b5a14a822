// Newton-Schulz orthogonalisation of a batch of matrices of any size:
//   X = G / (|G|_F + eps) (transposed while G has more rows than columns), then `steps` times
//   A = X X^T,  B = a I + b A + c A A,  X <- B X.
//
// All products run on bf16 MFMA with fp32 accumulation, on operands split into bf16 parts:
// two for bf16 matrices (17 bits: products h*h + h*l + l*h), three for fp32 ones (24 bits, six
// products, 2.5 times the rate of fp32 MFMA).  One part would not do: the five steps multiply
// what is lost in the small singular directions by up to 3.4445^5 = 485.
// The parts are written as planes by the kernel that computes a matrix, so that the main loop
// copies tiles from memory straight into LDS.  Every product is C[i][j] = sum_k P[i][k] Q[j][k]
// of row panels: X X^T, A A (A is symmetric) and B X from the stored X^T; A and B are
// symmetric, so only their tiles on and below the diagonal are computed.
// Sizes are padded with zeros to whole tiles.
#include "common.h"
#include "orth.h"

namespace ttt {
namespace {

constexpr int KS = 32;              // reduction elements a stage: 64-byte rows in LDS

struct Mat {                        // split matrix: `parts` planes of [rows][ld], one after another
  char *p;
  int64_t plane, bs;                // bytes from plane to plane, from matrix to matrix
  int ld;
};

template <int P> __device__ __forceinline__ void put4(char *p, int64_t plane, int64_t e, f32x4 v) {
#pragma unroll
  for (int i = 0; i < P; ++i) {
    bf16x4 h;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      h[r] = (__bf16)v[r];
      v[r] -= (float)h[r];
    }
    *reinterpret_cast<bf16x4 *>(reinterpret_cast<__bf16 *>(p + i * plane) + e) = h;
  }
}
template <int P> __device__ __forceinline__ f32x4 get4(const char *p, int64_t plane, int64_t e) {
  f32x4 v = f32x4{0, 0, 0, 0};
#pragma unroll
  for (int i = P - 1; i >= 0; --i) {
    const bf16x4 h = *reinterpret_cast<const bf16x4 *>(reinterpret_cast<const __bf16 *>(p + i * plane) + e);
#pragma unroll
    for (int r = 0; r < 4; ++r) v[r] += (float)h[r];
  }
  return v;
}

// Partial sums of squares, in 64 bits: block x of matrix y.
template <typename T>
__global__ __launch_bounds__(256) void orth_norm_kernel(OrthParams p, double *part) {
  __shared__ double red[4];
  const T *g = static_cast<const T *>(p.g) + (int64_t)blockIdx.y * p.bsg;
  // thread e, e + step, ..: row and column move by a fixed amount, with a carry
  const int64_t step = (int64_t)gridDim.x * 256, e0 = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int cols = p.plan.cols, dr = (int)(step / cols), dc = (int)(step % cols);
  int64_t r = e0 / cols;
  int c = (int)(e0 % cols);
  double s = 0.0;
  while (r < p.plan.rows) {
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i] = r < p.plan.rows ? to_f32(g[r * p.ldg + c]) : 0.0f;
      r += dr, c += dc;
      if (c >= cols) c -= cols, ++r;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) s += (double)x[i] * (double)x[i];
  }
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) s += __shfl_xor(s, m);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) part[(int64_t)blockIdx.y * gridDim.x + blockIdx.x] = (red[0] + red[1]) + (red[2] + red[3]);
}

// 1 / (|G| + eps) of matrix b, by every wave (the partials in one fixed order).
__device__ __forceinline__ float orth_scale(const OrthParams &p, const double *part, int b) {
  double s = 0.0;
  for (int i = threadIdx.x & 63; i < p.plan.norm_blocks; i += 64) s += part[(int64_t)b * p.plan.norm_blocks + i];
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) s += __shfl_xor(s, m);
  return (float)(1.0 / (sqrt(s) + (double)p.eps));
}

// X and X^T of the first step: G scaled, split and padded.  64 x 64 tiles of [rows][cols].
template <typename T, int P>
__global__ __launch_bounds__(256) void orth_load_kernel(OrthParams p, const double *part, Mat x, Mat xt) {
  __shared__ float tile[64][65];
  const OrthPlan &q = p.plan;
  const int b = blockIdx.z;
  const float scale = orth_scale(p, part, b);
  const int r0 = blockIdx.y * 64, c0 = blockIdx.x * 64, tx = (threadIdx.x & 15) * 4, ty = threadIdx.x >> 4;
  const T *g = static_cast<const T *>(p.g) + b * p.bsg;
  const Mat &m = q.tall ? xt : x, &mt = q.tall ? x : xt;      // G's own layout, and its transpose
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = r0 + ty + 16 * i;
    f32x4 v;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int c = c0 + tx + e;
      v[e] = r < q.rows && c < q.cols ? to_f32(g[(int64_t)r * p.ldg + c]) * scale : 0.0f;
      tile[ty + 16 * i][tx + e] = v[e];
    }
    put4<P>(m.p + b * m.bs, m.plane, (int64_t)r * m.ld + c0 + tx, v);
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f32x4 v;
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = tile[tx + e][ty + 16 * i];
    put4<P>(mt.p + b * mt.bs, mt.plane, (int64_t)(c0 + ty + 16 * i) * mt.ld + r0 + tx, v);
  }
}

// What a product's tile becomes.
enum Kind { kGram, kPoly, kNext, kLast };   // A;  B = a I + b A + c A A;  X and X^T;  the result
struct Product {
  Mat P, Q;                         // C = P Q^T
  Mat c, ct;                        // results: [i][j] and [j][i] (the same matrix where C is symmetric)
  int K, ti, tj;                    // reduction length, tiles along i and j
  int tiles;                        // tiles a matrix
};

// A workgroup's tile: TM x TN by WR x WC waves, a ring of NST stages of KS reduction elements.
// Both operands pass through LDS once a stage; a wave's fragment reads against its MFMAs fall
// with the wave tile, which sets the sizes (reads and copies share the LDS with 128 bytes a clock,
// 16 clocks an MFMA and SIMD): 256 x 256 where such tiles fill the card, 128 x 128 where those do,
// else 64 x 64.
template <int TM_, int TN_, int WR_, int WC_, int NST_> struct Geo {
  static constexpr int TM = TM_, TN = TN_, WR = WR_, WC = WC_, NST = NST_, kThreads = WR * WC * 64;
  static constexpr int WM = TM / WR, WN = TN / WC, FM = WM / 16, FN = WN / 16;
};
template <int TILE, int P> struct GeoOf;
template <int P> struct GeoOf<64, P> { typedef Geo<64, 64, 2, 2, P == 2 ? 4 : 3> type; };
template <int P> struct GeoOf<128, P> { typedef Geo<128, 128, 2, 2, P == 2 ? 4 : 3> type; };
template <> struct GeoOf<256, 2> { typedef Geo<256, 256, 4, 2, 2> type; };
template <> struct GeoOf<256, 3> { typedef Geo<256, 128, 4, 2, 2> type; };

template <typename T, typename G, int P, int KIND>
__global__ __launch_bounds__(G::kThreads, G::kThreads / 256) void orth_product_kernel(OrthParams p, Product q) {
  constexpr int kRows = (G::TM + G::TN) * P, kStage = kRows * 64, kWaves = G::kThreads / 64;
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
  const char *pp = q.P.p + b * q.P.bs + (int64_t)bi * G::TM * q.P.ld * 2;
  const char *pq = q.Q.p + b * q.Q.bs + (int64_t)bj * G::TN * q.Q.ld * 2;
  // A stage holds, part by part, the rows of the P panel, then those of the Q panel.  A copy is 16
  // rows of 64 bytes: lane = 4 * row + position, and the piece at position a is chunk a ^ swz_64(row).
  const int cr = l >> 2, cc = ((l & 3) ^ swz_64(cr)) * 16;
  const char *src[PPW];
#pragma unroll
  for (int x = 0; x < PPW; ++x) {
    const int row = (w * PPW + x) * 16;           // of the stage
    const bool second = row >= G::TM * P;
    const int r = second ? row - G::TM * P : row, rows = second ? G::TN : G::TM;
    const Mat &m = second ? q.Q : q.P;
    src[x] = (second ? pq : pp) + (r / rows) * m.plane + (int64_t)(r % rows + cr) * m.ld * 2 + cc;
  }
  const int nk = q.K / KS;
  const auto copy = [&](int x, int kc) {
    copy16_to_lds_untracked(src[x] + kc * (KS * 2), s + kc % G::NST * kStage + (w * PPW + x) * 1024);
  };
  f32x4 acc[G::FM][G::FN];
#pragma unroll
  for (int i = 0; i < G::FM; ++i)
#pragma unroll
    for (int j = 0; j < G::FN; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
  const int wi = (w / G::WC) * G::WM, wj = (w % G::WC) * G::WN;
  const int fo = li * 64 + ((g ^ swz_64(li)) * 16);
#pragma unroll
  for (int k = 0; k < G::NST - 1; ++k)
    if (k < nk)
#pragma unroll
      for (int x = 0; x < PPW; ++x) copy(x, k);
  for (int kc = 0; kc < nk; ++kc) {
    // this wave's copies of stage kc have arrived (those of the NST - 2 stages after it may be in flight)
    if (kc + G::NST - 2 < nk) wait_vmcnt<(G::NST - 2) * PPW>(); else wait_vmcnt<0>();
    bare_barrier();                               // everyone's have, and the stage before is free
    const unsigned char *st = s + kc % G::NST * kStage;
    const bool more = kc + G::NST - 1 < nk;
    bf16x8 fa[G::FM][P], fb[2][P];
    const auto read_b = [&](int j, bf16x8 (&f)[P]) {
#pragma unroll
      for (int x = 0; x < P; ++x)
        f[x] = *reinterpret_cast<const bf16x8 *>(st + ((G::TM * P + x * G::TN + wj + 16 * j) * 64 + fo));
    };
#pragma unroll
    for (int i = 0; i < G::FM; ++i)
#pragma unroll
      for (int x = 0; x < P; ++x) fa[i][x] = *reinterpret_cast<const bf16x8 *>(st + ((x * G::TM + wi + 16 * i) * 64 + fo));
    read_b(0, fb[0]);
#pragma unroll
    for (int j = 0; j < G::FN; ++j) {
      if (j + 1 < G::FN) read_b(j + 1, fb[(j + 1) & 1]);
      // the next stage's copies, spread over the products
#pragma unroll
      for (int x = 0; x < PPW; ++x)
        if (x * G::FN / PPW == j && more) copy(x, kc + G::NST - 1);
#pragma unroll
      for (int d = P - 1; d >= 0; --d)            // the small products first
#pragma unroll
        for (int x = 0; x <= d; ++x)
#pragma unroll
          for (int i = 0; i < G::FM; ++i) acc[i][j] = mma(fb[j & 1][d - x], fa[i][x], acc[i][j]);
    }
  }
  __syncthreads();                                // the ring is free
  // lane (g, li) holds C[16 i + li][16 j + 4 g + r], r = 0 .. 3, of the wave's tile
  const int r0 = bi * G::TM + wi, c0 = bj * G::TN + wj;
  if constexpr (KIND == kPoly) {
    const char *pa = q.P.p + b * q.P.bs;
#pragma unroll
    for (int i = 0; i < G::FM; ++i)
#pragma unroll
      for (int j = 0; j < G::FN; ++j) {
        const int row = r0 + 16 * i + li, col = c0 + 16 * j + 4 * g;
        const f32x4 a = get4<P>(pa, q.P.plane, (int64_t)row * q.P.ld + col);
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[i][j][r] = p.c * acc[i][j][r] + (p.b * a[r] + (row == col + r ? p.a : 0.0f));
      }
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
  unsigned char *mine = s + w * (G::WM * kPitch);
  const bool both = KIND == kNext || bi != bj;
#pragma unroll
  for (int x = 0; x < P; ++x) {
#pragma unroll
    for (int i = 0; i < G::FM; ++i)
#pragma unroll
      for (int j = 0; j < G::FN; ++j) {
        bf16x4 h;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          h[r] = (__bf16)acc[i][j][r];
          acc[i][j][r] -= (float)h[r];
        }
        *reinterpret_cast<bf16x4 *>(mine + (16 * i + li) * kPitch + (16 * j + 4 * g) * 2) = h;
      }
    constexpr int RC = G::WN / 8;                 // 16-byte pieces of a row
    __bf16 *c = reinterpret_cast<__bf16 *>(q.c.p + b * q.c.bs + x * q.c.plane);
#pragma unroll
    for (int y = 0; y < G::WM * RC / 64; ++y) {
      const int u = l + 64 * y, r = u / RC, k = u % RC;
      *reinterpret_cast<u32x4 *>(c + (int64_t)(r0 + r) * q.c.ld + c0 + 8 * k) =
          *reinterpret_cast<const u32x4 *>(mine + r * kPitch + 16 * k);
    }
    if (both) {
      __bf16 *ct = reinterpret_cast<__bf16 *>(q.ct.p + b * q.ct.bs + x * q.ct.plane);
#pragma unroll
      for (int i = 0; i < G::WM / 32; ++i)
#pragma unroll
        for (int j = 0; j < G::FN; ++j) {         // rows 32 i + 8 g .. + 7 of column 16 j + li
          const unsigned char *a = mine + (32 * i + 8 * g + (li >> 2)) * kPitch + (16 * j + 4 * (li & 3)) * 2;
          *reinterpret_cast<bf16x8 *>(ct + (int64_t)(c0 + 16 * j + li) * q.ct.ld + r0 + 32 * i + 8 * g) =
              cat8(lds_read_tr16(a), lds_read_tr16(a + 4 * kPitch));
        }
    }
  }
}

// G as it is (steps = 0): only scaled.
template <typename T>
__global__ __launch_bounds__(256) void orth_scale_kernel(OrthParams p, const double *part) {
  const OrthPlan &q = p.plan;
  const int b = blockIdx.y;
  const float scale = orth_scale(p, part, b);
  const int64_t total = (int64_t)q.rows * q.cols;
  for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < total; e += (int64_t)gridDim.x * 256) {
    const int64_t r = e / q.cols, c = e % q.cols;
    static_cast<T *>(p.out)[b * p.bso + r * p.ldo + c] =
        from_f32<T>(to_f32(static_cast<const T *>(p.g)[b * p.bsg + r * p.ldg + c]) * scale);
  }
}

template <typename T, int P, int KIND, int TILE> void product_of(const OrthParams &p, Product q, int rows, int cols, hipStream_t s) {
  typedef typename GeoOf<TILE, P>::type G;
  const bool sym = KIND == kGram || KIND == kPoly;
  q.ti = rows / G::TM, q.tj = cols / G::TN;
  q.tiles = sym ? q.ti * (q.ti + 1) / 2 : q.ti * q.tj;
  hipLaunchKernelGGL((orth_product_kernel<T, G, P, KIND>), dim3((unsigned)(p.plan.batch * q.tiles)), dim3(G::kThreads), 0, s, p, q);
}
template <typename T, int P, int KIND> void product(const OrthParams &p, const Product &q, int rows, int cols, hipStream_t s) {
  // symmetric results: square tiles of at most 128, so that half of them stay away
  const int tile = KIND == kGram || KIND == kPoly ? p.plan.tile_sym : p.plan.tile;
  if constexpr (KIND == kNext || KIND == kLast) {
    if (tile == 256) return product_of<T, P, KIND, 256>(p, q, rows, cols, s);
  }
  if (tile == 128) return product_of<T, P, KIND, 128>(p, q, rows, cols, s);
  product_of<T, P, KIND, 64>(p, q, rows, cols, s);
}

template <typename T, int P> hipError_t steps_of(const OrthParams &p, hipStream_t s) {
  const OrthPlan &q = p.plan;
  const int64_t xb = (int64_t)q.rp * q.cp * 2, ab = (int64_t)q.rp * q.rp * 2;
  Mat x[2], xt[2];
  for (int i = 0; i < 2; ++i) {
    x[i] = Mat{p.ws + q.off_x[i], xb, xb * P, q.cp};
    xt[i] = Mat{p.ws + q.off_xt[i], xb, xb * P, q.rp};
  }
  const Mat A{p.ws + q.off_a, ab, ab * P, q.rp}, B{p.ws + q.off_b, ab, ab * P, q.rp};
  const double *part = reinterpret_cast<const double *>(p.ws + q.off_norm);
  const int pr = q.tall ? q.cp : q.rp, pc = q.tall ? q.rp : q.cp;       // padded sizes of G
  hipLaunchKernelGGL((orth_load_kernel<T, P>), dim3(pc / 64, pr / 64, q.batch), dim3(256), 0, s, p, part, x[0], xt[0]);
  for (int i = 0; i < p.steps; ++i) {
    const int cur = i & 1;
    product<T, P, kGram>(p, Product{x[cur], x[cur], A, A, q.cp}, q.rp, q.rp, s);
    product<T, P, kPoly>(p, Product{A, A, B, B, q.rp}, q.rp, q.rp, s);
    const Product nx{B, xt[cur], x[cur ^ 1], xt[cur ^ 1], q.rp};
    if (i + 1 < p.steps)
      product<T, P, kNext>(p, nx, q.rp, q.cp, s);
    else
      product<T, P, kLast>(p, nx, q.rp, q.cp, s);
  }
  return hipGetLastError();
}

template <typename T, int P> hipError_t run_orth(const OrthParams &p, hipStream_t s) {
  const OrthPlan &q = p.plan;
  double *part = reinterpret_cast<double *>(p.ws + q.off_norm);
  hipLaunchKernelGGL(orth_norm_kernel<T>, dim3(q.norm_blocks, q.batch), dim3(256), 0, s, p, part);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (p.steps == 0) {
    hipLaunchKernelGGL(orth_scale_kernel<T>, dim3(q.norm_blocks, q.batch), dim3(256), 0, s, p, part);
    return hipGetLastError();
  }
  return steps_of<T, P>(p, s);
}

}  // namespace

OrthPlan plan_orth(int rows, int cols, int batch, bool bf16) {
  OrthPlan q{};
  q.rows = rows, q.cols = cols, q.batch = batch, q.bf16 = bf16;
  q.tall = rows > cols;
  q.r = q.tall ? cols : rows, q.c = q.tall ? rows : cols;
  q.parts = bf16 ? 2 : 3;
  const auto tiles = [&](int tm, int tn) { return (int64_t)batch * ((q.r + tm - 1) / tm) * ((q.c + tn - 1) / tn); };
  const int tn = bf16 ? 256 : 128;
  q.tile = tiles(256, tn) >= 200 ? 256 : (tiles(128, 128) >= 200 ? 128 : 64);
  const int64_t nr = (q.r + 127) / 128;
  q.tile_sym = batch * (nr * (nr + 1) / 2) >= 100 ? 128 : 64;
  const int pad = q.tile > q.tile_sym ? q.tile : q.tile_sym;
  q.rp = (q.r + pad - 1) / pad * pad, q.cp = (q.c + pad - 1) / pad * pad;
  const int64_t elems = (int64_t)rows * cols, blocks = (elems + 4095) / 4096;
  q.norm_blocks = (int)(blocks < 1 ? 1 : (blocks > 256 ? 256 : blocks));
  const auto al = [](size_t x) { return (x + 255) & ~size_t(255); };
  const size_t xb = (size_t)q.rp * q.cp * 2 * q.parts * batch, ab = (size_t)q.rp * q.rp * 2 * q.parts * batch;
  size_t o = 0;
  q.off_norm = o, o = al(o + (size_t)batch * q.norm_blocks * 8);
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
  return p.plan.bf16 ? run_orth<__bf16, 2>(p, s) : run_orth<float, 3>(p, s);
}

}  // namespace ttt
