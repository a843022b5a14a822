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

template <int P> __device__ __forceinline__ void put1(char *p, int64_t plane, int64_t e, float v) {
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const __bf16 h = (__bf16)v;
    reinterpret_cast<__bf16 *>(p + i * plane)[e] = h;
    v -= (float)h;
  }
}
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
  const int64_t total = (int64_t)p.plan.rows * p.plan.cols;
  double s = 0.0;
  for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < total; e += (int64_t)gridDim.x * 256) {
    const double x = (double)to_f32(g[e / p.plan.cols * p.ldg + e % p.plan.cols]);
    s += x * x;
  }
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) s += __shfl_xor(s, m);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) part[(int64_t)blockIdx.y * gridDim.x + blockIdx.x] = (red[0] + red[1]) + (red[2] + red[3]);
}

// X and X^T of the first step: G scaled, split and padded.  32 x 32 tiles of [rows][cols].
template <typename T, int P>
__global__ __launch_bounds__(256) void orth_load_kernel(OrthParams p, const double *part, Mat x, Mat xt) {
  __shared__ float tile[32][33];
  __shared__ float s_scale;
  const OrthPlan &q = p.plan;
  const int b = blockIdx.z;
  if (threadIdx.x == 0) {
    double s = 0.0;
    for (int i = 0; i < q.norm_blocks; ++i) s += part[(int64_t)b * q.norm_blocks + i];
    s_scale = (float)(1.0 / (sqrt(s) + (double)p.eps));
  }
  __syncthreads();
  const int r0 = blockIdx.y * 32, c0 = blockIdx.x * 32, tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const T *g = static_cast<const T *>(p.g) + b * p.bsg;
  const float scale = s_scale;
  Mat &m = q.tall ? xt : x, &mt = q.tall ? x : xt;      // G's own layout, and its transpose
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = r0 + ty + 8 * i, c = c0 + tx;
    const float v = r < q.rows && c < q.cols ? to_f32(g[(int64_t)r * p.ldg + c]) * scale : 0.0f;
    tile[ty + 8 * i][tx] = v;
    put1<P>(m.p + b * m.bs, m.plane, (int64_t)r * m.ld + c, v);
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i)
    put1<P>(mt.p + b * mt.bs, mt.plane, (int64_t)(c0 + ty + 8 * i) * mt.ld + r0 + tx, tile[tx][ty + 8 * i]);
}

// What a product's tile becomes.
enum Kind { kGram, kPoly, kNext, kLast };   // A;  B = a I + b A + c A A;  X and X^T;  the result
struct Product {
  Mat P, Q;                         // C = P Q^T
  Mat c, ct;                        // results: [i][j] and [j][i] (the same matrix where C is symmetric)
  int K, ti, tj;                    // reduction length, tiles along i and j
  int tiles;                        // tiles a matrix
};

template <typename T, int TILE, int P, int KIND>
__global__ __launch_bounds__(256) void orth_product_kernel(OrthParams p, Product q) {
  constexpr int W = TILE / 32;                    // 16-wide tiles a wave and direction
  constexpr int kPanel = TILE * KS * 2;           // bytes of one plane of one panel in a stage
  __shared__ __attribute__((aligned(16))) unsigned char s[2][2][P][kPanel];
  const int t = threadIdx.x, w = t >> 6, l = t & 63, g = l >> 4, li = l & 15;
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
  const char *pp = q.P.p + b * q.P.bs + (int64_t)bi * TILE * q.P.ld * 2;
  const char *pq = q.Q.p + b * q.Q.bs + (int64_t)bj * TILE * q.Q.ld * 2;
  // a wave's copy: 16 rows of 64 bytes; lane = 4 * row + position, the piece at position a is chunk a ^ swz_64(row)
  const int cr = l >> 2, cc = ((l & 3) ^ swz_64(cr)) * 16;
  auto stage = [&](int k, int buf) {
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
      for (int x = 0; x < TILE / 64; ++x) {
        const int r = (w + 4 * x) * 16;
        copy16_to_lds(pp + i * q.P.plane + (int64_t)(r + cr) * q.P.ld * 2 + k * 2 + cc, &s[buf][0][i][r * 64]);
        copy16_to_lds(pq + i * q.Q.plane + (int64_t)(r + cr) * q.Q.ld * 2 + k * 2 + cc, &s[buf][1][i][r * 64]);
      }
  };
  f32x4 acc[W][W];
#pragma unroll
  for (int i = 0; i < W; ++i)
#pragma unroll
    for (int j = 0; j < W; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
  const int wi = (w >> 1) * (TILE / 2), wj = (w & 1) * (TILE / 2);
  const int fo = li * 64 + ((g ^ swz_64(li)) * 16);
  stage(0, 0);
  int buf = 0;
  for (int k = 0; k < q.K; k += KS, buf ^= 1) {
    __syncthreads();                              // this stage has arrived, the other buffer is free
    if (k + KS < q.K) stage(k + KS, buf ^ 1);
    bf16x8 fa[W][P], fb[W][P];
#pragma unroll
    for (int i = 0; i < W; ++i)
#pragma unroll
      for (int x = 0; x < P; ++x) {
        fa[i][x] = *reinterpret_cast<const bf16x8 *>(&s[buf][0][x][(wi + 16 * i) * 64 + fo]);
        fb[i][x] = *reinterpret_cast<const bf16x8 *>(&s[buf][1][x][(wj + 16 * i) * 64 + fo]);
      }
#pragma unroll
    for (int d = P - 1; d >= 0; --d)              // the small products first
#pragma unroll
      for (int x = 0; x <= d; ++x)
#pragma unroll
        for (int i = 0; i < W; ++i)
#pragma unroll
          for (int j = 0; j < W; ++j) acc[i][j] = mma(fa[i][x], fb[j][d - x], acc[i][j]);
  }
  const int r0 = bi * TILE + wi + 4 * g, c0 = bj * TILE + wj + li;
#pragma unroll
  for (int i = 0; i < W; ++i)
#pragma unroll
    for (int j = 0; j < W; ++j) {
      f32x4 v = acc[i][j];
      const int row = r0 + 16 * i, col = c0 + 16 * j;     // rows row .. row + 3, column col
      if (KIND == kPoly) {
        const f32x4 a = get4<P>(q.P.p + b * q.P.bs, q.P.plane, (int64_t)col * q.P.ld + row);
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] = p.c * v[r] + (p.b * a[r] + (row + r == col ? p.a : 0.0f));
      }
      if (KIND == kLast) {
        T *out = static_cast<T *>(p.out) + b * p.bso;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          if (row + r >= p.plan.r || col >= p.plan.c) continue;
          const int64_t o = p.plan.tall ? (int64_t)col * p.ldo + row + r : (int64_t)(row + r) * p.ldo + col;
          out[o] = from_f32<T>(v[r]);
        }
        continue;
      }
      put4<P>(q.ct.p + b * q.ct.bs, q.ct.plane, (int64_t)col * q.ct.ld + row, v);
      if (KIND == kNext || bi != bj)
#pragma unroll
        for (int r = 0; r < 4; ++r) put1<P>(q.c.p + b * q.c.bs, q.c.plane, (int64_t)(row + r) * q.c.ld + col, v[r]);
    }
}

// G as it is (steps = 0): only scaled.
template <typename T>
__global__ __launch_bounds__(256) void orth_scale_kernel(OrthParams p, const double *part) {
  const OrthPlan &q = p.plan;
  const int b = blockIdx.y;
  double s = 0.0;
  for (int i = 0; i < q.norm_blocks; ++i) s += part[(int64_t)b * q.norm_blocks + i];
  const float scale = (float)(1.0 / (sqrt(s) + (double)p.eps));
  const int64_t total = (int64_t)q.rows * q.cols;
  for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < total; e += (int64_t)gridDim.x * 256) {
    const int64_t r = e / q.cols, c = e % q.cols;
    static_cast<T *>(p.out)[b * p.bso + r * p.ldo + c] =
        from_f32<T>(to_f32(static_cast<const T *>(p.g)[b * p.bsg + r * p.ldg + c]) * scale);
  }
}

template <typename T, int TILE, int P> hipError_t steps_of(const OrthParams &p, hipStream_t s) {
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
  hipLaunchKernelGGL((orth_load_kernel<T, P>), dim3(pc / 32, pr / 32, q.batch), dim3(256), 0, s, p, part, x[0], xt[0]);
  const int nr = q.rp / TILE, ncol = q.cp / TILE;
  const unsigned sym = (unsigned)(q.batch * (nr * (nr + 1) / 2)), all = (unsigned)(q.batch * nr * ncol);
  for (int i = 0; i < p.steps; ++i) {
    const int cur = i & 1;
    hipLaunchKernelGGL((orth_product_kernel<T, TILE, P, kGram>), dim3(sym), dim3(256), 0, s, p,
                       Product{x[cur], x[cur], A, A, q.cp, nr, nr, nr * (nr + 1) / 2});
    hipLaunchKernelGGL((orth_product_kernel<T, TILE, P, kPoly>), dim3(sym), dim3(256), 0, s, p,
                       Product{A, A, B, B, q.rp, nr, nr, nr * (nr + 1) / 2});
    const Product nx{B, xt[cur], x[cur ^ 1], xt[cur ^ 1], q.rp, nr, ncol, nr * ncol};
    if (i + 1 < p.steps)
      hipLaunchKernelGGL((orth_product_kernel<T, TILE, P, kNext>), dim3(all), dim3(256), 0, s, p, nx);
    else
      hipLaunchKernelGGL((orth_product_kernel<T, TILE, P, kLast>), dim3(all), dim3(256), 0, s, p, nx);
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
  return q.tile == 128 ? steps_of<T, 128, P>(p, s) : steps_of<T, 64, P>(p, s);
}

}  // namespace

OrthPlan plan_orth(int rows, int cols, int batch, bool bf16) {
  OrthPlan q{};
  q.rows = rows, q.cols = cols, q.batch = batch, q.bf16 = bf16;
  q.tall = rows > cols;
  q.r = q.tall ? cols : rows, q.c = q.tall ? rows : cols;
  q.parts = bf16 ? 2 : 3;
  // 128-wide tiles halve the operand traffic of 64-wide ones, which fill the card at smaller sizes
  const int64_t big = (int64_t)batch * ((q.r + 127) / 128) * ((q.c + 127) / 128);
  q.tile = big >= 256 ? 128 : 64;
  q.rp = (q.r + q.tile - 1) / q.tile * q.tile, q.cp = (q.c + q.tile - 1) / q.tile * q.tile;
  const int64_t elems = (int64_t)rows * cols, blocks = (elems + 4095) / 4096;
  q.norm_blocks = (int)(blocks < 1 ? 1 : (blocks > 64 ? 64 : blocks));
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
