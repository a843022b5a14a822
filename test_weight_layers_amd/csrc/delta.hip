// Gated delta rule: the fast-weight layer f_W(x) = W x, one step of size beta_t per token on
// 1/2 |W k_t - v_t|^2 after the decay a_t = e^(g_t):
//   e_t = v_t - a_t W k_t,   W <- a_t W + beta_t e_t k_t^T,   o_t = scale W q_t.
//
// Chunked form (64 tokens; gamma_i = g_1 + .. + g_i inside the chunk, D_ij = e^(gamma_i - gamma_j)
// for j <= i, W0 the state before the chunk):
//   L_ij = beta_i D_ij k_i.k_j (j < i),  T = (I + L)^-1,  A_ij = scale D_ij q_i.k_j (j <= i)
//   R = beta o (V - e^gamma o (K W0^T)),  U = T R
//   O = scale e^gamma o (Q W0^T) + A U
//   W = e^gamma_last W0 + (e^(gamma_last - gamma) o U)^T K
// Two kernels: T and A of every chunk at once (chunk), then the states in order of the chunks, split
// over heads and 16-column slices of dv, which do not depend on one another (states, delta_state.h).  Every wave lays
// the packed sequences out in chunks for itself; for more than 63 of them a first kernel does (plan).
#include "delta_state.h"

namespace ttt {
namespace {

// ------------------------------------------------------------------ plan
// Tables of the sequences and chunks, for more sequences than a wave has lanes.
__global__ __launch_bounds__(256) void delta_plan_kernel(DeltaParams p) {
  __shared__ int s_a[256], s_b[256];
  const int t = threadIdx.x;
  const auto off = [&](int i) { return delta_offset(p, i); };
  int carry_max = off(0), carry_chunks = 0;
  for (int b0 = 0; b0 < p.nseq; b0 += 256) {
    const int b = b0 + t;
    // inclusive running maximum of the end offsets
    s_a[t] = b < p.nseq ? off(b + 1) : 0;
    __syncthreads();
    for (int d = 1; d < 256; d <<= 1) {
      const int x = t >= d ? s_a[t - d] : 0;
      __syncthreads();
      s_a[t] = s_a[t] > x ? s_a[t] : x;
      __syncthreads();
    }
    const int end = s_a[t] > carry_max ? s_a[t] : carry_max;
    const int prev = t > 0 ? s_a[t - 1] : carry_max;
    const int start = prev > carry_max ? prev : carry_max;
    const int len = b < p.nseq ? end - start : 0;
    const int nc = (len + C - 1) / C;
    s_b[t] = nc;
    __syncthreads();
    for (int d = 1; d < 256; d <<= 1) {
      const int x = t >= d ? s_b[t - d] : 0;
      __syncthreads();
      s_b[t] += x;
      __syncthreads();
    }
    if (b < p.nseq) p.seqs[b] = DeltaSeq{start, len, carry_chunks + s_b[t] - nc, 0};
    carry_max = s_a[255] > carry_max ? s_a[255] : carry_max;
    carry_chunks += s_b[255];
    __syncthreads();
  }
  if (t == 0) *p.used = carry_max;
  __threadfence_block();
  __syncthreads();
  for (int c = t; c < p.nchunk; c += 256) {
    if (c >= carry_chunks) {
      p.chunks[c] = DeltaChunk{0, 0, 0, 0};
      continue;
    }
    int lo = 0, hi = p.nseq - 1;      // the last sequence whose chunk0 <= c (empty ones share it with their successor)
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (p.seqs[mid].chunk0 <= c) lo = mid; else hi = mid - 1;
    }
    const DeltaSeq sq = p.seqs[lo];
    const int r = (c - sq.chunk0) * C;
    p.chunks[c] = DeltaChunk{sq.start + r, sq.len - r < C ? sq.len - r : C, lo, 0};
  }
}

// Zeros in the rows before the first sequence and behind the last: rows [n][ld] of `width`.
template <typename T>
__device__ void zero_rows(const DeltaParams &p, int2 used, void *rows, int64_t ld, int width, int block, int blocks) {
  const int total = used.x + (p.n - used.y);
  for (int64_t i = (int64_t)block * 256 + threadIdx.x; i < (int64_t)total * width; i += (int64_t)blocks * 256) {
    const int64_t r = i / width, row = r < used.x ? r : used.y + (r - used.x);
    static_cast<T *>(rows)[row * ld + i % width] = from_f32<T>(0.0f);
  }
}
constexpr int kZeroBlocks = 64;     // workgroups of the chunk kernel's launch that write those zeros

// ------------------------------------------------------------------ chunk terms
// One workgroup per chunk and head: e^gamma, T = (I + L)^-1 by block substitution in fp32 and A,
// and (once per key head) the tokens and their transposes in fragment order.
// Substitution, not products of powers of L: those grow without bound where keys repeat.
// 687 chunks of 4 heads of 256, bf16: 99 us for 588 MB, 5.9 TB/s, a copy reaches 5.1; 22 chunks 14.9 us,
// the latency of the loads and the substitution.
template <typename T, int DK, bool BWD>
__global__ __launch_bounds__(256, sizeof(T) == 2 ? 2 : 1) void delta_chunk_kernel(DeltaParams p) {
  constexpr int kPitch = DK + 16 / (int)sizeof(T), NK = DK / 32, kA = C + 4, TP = kTok<T>;
  constexpr int kTokBytes = C * kPitch * (int)sizeof(T), kABytes = C * kA * 4;
  __shared__ __attribute__((aligned(16))) unsigned char s_raw[kTokBytes > kABytes ? kTokBytes : kABytes];
  __shared__ float2 s_gam[C];
  __shared__ float s_beta[C];
  __shared__ __attribute__((aligned(16))) float s_l[C][kA], s_t[C][kA], s_x[32][36];
  T *s_tok = reinterpret_cast<T *>(s_raw);              // [64][kPitch]
  float *s_a = reinterpret_cast<float *>(s_raw);        // [64][kA], after the tokens
  const int items = p.nchunk * p.heads;
  if ((int)blockIdx.x >= items) {                       // rows of no sequence
    const int blk = blockIdx.x - items;
    const int2 used = rows_of(p);
    if (!BWD) {
      zero_rows<T>(p, used, p.o, p.ldo, p.heads * p.dv, blk, kZeroBlocks);
      return;
    }
    zero_rows<T>(p, used, p.gq, p.ldgq, p.key_heads * DK, blk, kZeroBlocks);
    zero_rows<T>(p, used, p.gk, p.ldgk, p.key_heads * DK, blk, kZeroBlocks);
    zero_rows<T>(p, used, p.gv, p.ldgv, p.heads * p.dv, blk, kZeroBlocks);
    for (int h = blk; h < p.heads; h += kZeroBlocks) {
      zero_rows<float>(p, used, p.gbeta + h * p.gbeta_hs, 1, 1, 0, 1);
      if (p.gdecay) zero_rows<float>(p, used, p.gdecay + h * p.gdecay_hs, 1, 1, 0, 1);
    }
    return;
  }
  const int item = xcd_item(blockIdx.x, items), h = item % p.heads, c = item / p.heads;
  const DeltaChunk ck = chunk_of(p, c);
  if (ck.len == 0) return;
  const int t = threadIdx.x, w = t >> 6, l = t & 63, g = l >> 4, li = l & 15;
  const int grp = p.heads / p.key_heads, kh = h / grp;
  const bool writer = h % grp == 0;                     // of the key head's operands
  const int64_t ch = (int64_t)c * p.heads + h;
  const int64_t tokens = ((int64_t)c * p.key_heads + kh) * (DK * C * 2 * TP);
  constexpr int64_t tplane = DK * C * 2;
  constexpr int V = 16 / (int)sizeof(T), NP = C * DK / V / 256;      // 16-byte pieces: elements, and a thread's
  const auto fetch = [&](const void *src, int64_t ld, u32x4 (&x)[NP]) {
    const T *b = static_cast<const T *>(src) + (int64_t)ck.tok0 * ld + kh * DK;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int e = t + 256 * i, r = e / (DK / V), col = e % (DK / V) * V;
      x[i] = u32x4{0, 0, 0, 0};                         // rows past the chunk are zero
      if (r < ck.len) x[i] = *reinterpret_cast<const u32x4 *>(b + r * ld + col);
    }
  };
  const auto stage = [&](const u32x4 (&x)[NP]) {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int e = t + 256 * i, r = e / (DK / V), col = e % (DK / V) * V;
      *reinterpret_cast<u32x4 *>(s_tok + r * kPitch + col) = x[i];
    }
  };
  u32x4 xq[NP], xk[NP];
  fetch(p.q, p.ldq, xq);
  fetch(p.k, p.ldk, xk);
  float rate = 0.0f, be = 0.0f;
  if (t < ck.len) {
    if (p.decay) rate = p.decay[h * p.decay_hs + ck.tok0 + t];
    be = p.beta[h * p.beta_hs + ck.tok0 + t];
  }
  // the first wave, which has the least of the products, sums the decays after them
  const auto rates = [&] {
    double gam = rate < -200.0f ? -200.0 : (double)rate;        // e^-200 is 0 in fp32; -inf would leave inf - inf
#pragma unroll
    for (int d = 1; d < C; d <<= 1) {
      const double x = __shfl_up(gam, d);
      if (t >= d) gam += x;
    }
    const float2 lg = log_of(gam);
    s_gam[t] = lg;
    s_beta[t] = be;
    p.be[ch * C + t] = be;
    if (BWD) p.gam[ch * C + t] = lg;
    p.eg[ch * C + t] = exp_of(gam);
    p.el[ch * C + t] = exp_of(__shfl(gam, 63) - gam);
  };
  // the transposed operand: row = column of the tokens, k = token
  const auto write_transposed = [&](char *dst) {
#pragma unroll
    for (int i = 0; i < DK / 64; ++i) {
      const int rt = w * (DK / 64) + i;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int k0 = 32 * x + 8 * g;
        typename FragOf<T>::type f;
        if constexpr (sizeof(T) == 2) {
          const unsigned char *b = s_raw + ((k0 + (li >> 2)) * kPitch + 16 * rt + 4 * (li & 3)) * 2;
          f = cat8(lds_read_tr16(b), lds_read_tr16(b + 4 * kPitch * 2));
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] = s_tok[(k0 + e) * kPitch + 16 * rt + li];
        }
        store_split(dst + tokens, tplane, frag_of(rt, x, 2), token_of(f));
      }
    }
  };
  stage(xq);
  __syncthreads();
  Split<TP> qa[NK];                                     // wave w has rows 16 w .. 16 w + 15
#pragma unroll
  for (int i = 0; i < NK; ++i) {
    qa[i] = token_of(ld8(s_tok + (16 * w + li) * kPitch + 32 * i + 8 * g));
    if (writer) store_split(p.qp + tokens, tplane, frag_of(w, i, NK), qa[i]);
  }
  if (BWD && writer) write_transposed(p.qt);
  __syncthreads();
  stage(xk);
  __syncthreads();
  f32x4 kk[4], qk[4];                                   // K K^T and Q K^T, four column tiles
#pragma unroll
  for (int j = 0; j < 4; ++j) kk[j] = qk[j] = zero4();
#pragma unroll
  for (int i = 0; i < NK; ++i) {
    const Split<TP> ka = token_of(ld8(s_tok + (16 * w + li) * kPitch + 32 * i + 8 * g));
    if (writer) store_split(p.kp + tokens, tplane, frag_of(w, i, NK), ka);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j > w) continue;                              // above the diagonal
      const Split<TP> kb = token_of(ld8(s_tok + (16 * j + li) * kPitch + 32 * i + 8 * g));
      kk[j] = mm(ka, kb, kk[j]);
      qk[j] = mm(qa[i], kb, qk[j]);
    }
  }
  if (t < C) rates();
  if (writer) write_transposed(p.kt);
  __syncthreads();
  float2 gr[4], gcol[4];                                // (read ahead of the stores, which may be to the same LDS for all
  float br[4];                                          // that the compiler knows)
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    gr[r] = s_gam[16 * w + 4 * g + r];
    gcol[r] = s_gam[16 * r + li];
    br[r] = s_beta[16 * w + 4 * g + r];
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int col = 16 * j + li;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = 16 * w + 4 * g + r;
      s_t[row][col] = 0.0f;
      if (j > w) {                                      // above the diagonal; L there is not read
        s_a[row * kA + col] = 0.0f;
        continue;
      }
      const bool in = row < ck.len && col <= row;
      const float d = exp_of(gr[r], gcol[j]);           // (below the diagonal; elsewhere not used)
      s_l[row][col] = in && col < row ? br[r] * d * kk[j][r] : 0.0f;
      s_a[row * kA + col] = in ? p.scale * d * qk[j][r] : 0.0f;
    }
  }
  __syncthreads();
  // T = (I + L)^-1.  Diagonal 16 x 16 blocks: wave w has block w, one column a lane (four lanes alike).
  {
    float x[16];
    const int o = 16 * w;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      f32x4 row[4];
#pragma unroll
      for (int m = 0; m < (i + 3) / 4; ++m) row[m] = *reinterpret_cast<const f32x4 *>(&s_l[o + i][o + 4 * m]);
      float v = i == li ? 1.0f : 0.0f, u = 0.0f;        // two sums: half the chain
#pragma unroll
      for (int m = 0; m < i; ++m) {
        if (m & 1) u -= row[m >> 2][m & 3] * x[m];
        else v -= row[m >> 2][m & 3] * x[m];
      }
      x[i] = u + v;
    }
    if (g == 0)
#pragma unroll
      for (int i = 0; i < 16; ++i) s_t[o + i][o + li] = x[i];
  }
  __syncthreads();
  // Blocks below the diagonal: T21 = -T22 (L21 T11), first 16 wide (two pairs, waves 0 and 1), then
  // 32 wide (four 16 x 16 tiles, one a wave), on fp32 MFMA.
  const auto tile = [&](const float *a, int lda, const float *b, int ldb, int k) {      // 16 x 16, k = 16 or 32
    f32x4 s = zero4();
    const int n = k / 4;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n)      // reduction elements n g .. n g + n - 1 of lane group g
        s = __builtin_amdgcn_mfma_f32_16x16x4f32(a[li * lda + n * g + i], b[(n * g + i) * ldb + li], s, 0, 0, 0);
    return s;
  };
  if (w < 2) {
    const int o = 32 * w;
    const f32x4 s = tile(&s_l[o + 16][o], kA, &s_t[o][o], kA, 16);
#pragma unroll
    for (int r = 0; r < 4; ++r) s_x[16 * w + 4 * g + r][li] = s[r];
  }
  __syncthreads();
  if (w < 2) {
    const int o = 32 * w;
    const f32x4 s = tile(&s_t[o + 16][o + 16], kA, &s_x[16 * w][0], 36, 16);
#pragma unroll
    for (int r = 0; r < 4; ++r) s_t[o + 16 + 4 * g + r][o + li] = -s[r];
  }
  __syncthreads();
  const int ti = 16 * (w >> 1), tj = 16 * (w & 1);
  {
    const f32x4 s = tile(&s_l[32 + ti][0], kA, &s_t[0][tj], kA, 32);
#pragma unroll
    for (int r = 0; r < 4; ++r) s_x[ti + 4 * g + r][tj + li] = s[r];
  }
  __syncthreads();
  {
    const f32x4 s = tile(&s_t[32 + ti][32], kA, &s_x[0][tj], 36, 32);
#pragma unroll
    for (int r = 0; r < 4; ++r) s_t[32 + ti + 4 * g + r][tj + li] = -s[r];
  }
  __syncthreads();
  const int64_t mat = ch * kSquare, plane = C * C * 2;
#pragma unroll
  for (int q = 0; q < 2; ++q) {                         // fragment w + 4 q: rows 16 rt, k 32 kt
    const int f = w + 4 * q, row = 16 * (f >> 1) + li, k0 = 32 * (f & 1) + 8 * g, e = f * 512 + l * 8;
    store_split(p.tm + mat, plane, e, split_of<kFull>(ld8(&s_t[row][k0])));
    if (BWD) {
      f32x8 x, y;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[i] = s_t[k0 + i][row];
        y[i] = s_a[(k0 + i) * kA + row];
      }
      store_split(p.tt + mat, plane, e, split_of<kFull>(x));
      store_split(p.am + mat, plane, e, split_of<kFull>(y));
    } else {
      store_split(p.am + mat, plane, e, split_of<kFull>(ld8(s_a + row * kA + k0)));
    }
  }
  if (BWD) {
    const int row = 16 * w + li, nk = p.dv / 32;
    const T *go = static_cast<const T *>(p.go) + (int64_t)(ck.tok0 + (row < ck.len ? row : 0)) * p.ldgo + h * p.dv + 8 * g;
    char *o = p.gop + ch * C * p.dv * 2 * TP;
    for (int i = 0; i < nk; ++i) {
      auto v = ld8(go + 32 * i);
      if (row >= ck.len) v = zero8<T>();
      store_split(o, (int64_t)C * p.dv * 2, frag_of(w, i, nk), token_of(v));
    }
  }
}

// ------------------------------------------------------------------ states
template <typename T, int DK, int PART>
__global__ __launch_bounds__(512, sizeof(T) == 2 ? 4 : 2) void delta_state_kernel(DeltaParams p) {
  __shared__ __attribute__((aligned(16))) StateLds<T, DK, false> lds;
  delta_states<T, DK, false, PART>(p, lds, blockIdx.x, gridDim.x);
}

// ------------------------------------------------------------------ one token
// The recurrent form for one token of each row's sequence: one read and one write of the state.
//   o = scale (a W q + beta e (k.q)),  W <- a W + beta e k^T,  e = v - a W k
// 16 lanes hold one dv row of W; rows that name the same state are applied in row order by the
// workgroups of the first of them, found among all slots by each (4.2e12 looks a second: 17% of a call of
// 16,384 rows of 8 heads of 128, 3.9 ms).  Bound by memory: 300 rows of 8 heads of 128 x 128 move 316 MB in
// 70 us (4.5 TB/s; 49 while the 157 MB of states stay in the 256 MB cache), one row of 4 heads of
// 256 x 256 takes the 6.3 us of a launch and two memory latencies.
template <typename T, int DK>
__global__ __launch_bounds__(256) void delta_step_kernel(DeltaStepParams p) {
  constexpr int V4 = DK / 64;           // float4 a lane and dv row
  constexpr int NR = 4;                 // dv rows of a 16-lane group
  __shared__ int s_hit;
  const int t = threadIdx.x, li = t & 15, grp = t >> 4;
  const int blocks = p.dv / 64;
  const int db = blockIdx.x % blocks, h = blockIdx.x / blocks % p.heads, row0 = blockIdx.x / blocks / p.heads;
  const int kh = h / (p.heads / p.key_heads);
  const int slot = p.slots ? p.slots[row0] : row0;
  const bool valid = slot >= 0 && slot < p.nslots;
  if (!valid) {
    if (p.zero_unused && t < 64) static_cast<T *>(p.o)[(int64_t)row0 * p.ldo + h * p.dv + db * 64 + t] = from_f32<T>(0.0f);
    return;
  }
  int rows_left = 0;
  if (p.slots) {
    if (t == 0) s_hit = 0;
    __syncthreads();
    int hit = 0;
    for (int i = t; i < p.n; i += 256)
      if (p.slots[i] == slot && i != row0) hit |= i < row0 ? 1 : 2;
    if (hit) atomicOr(&s_hit, hit);
    __syncthreads();
    if (s_hit & 1) return;              // an earlier row's workgroups apply this one too
    rows_left = s_hit;
  }
  f32x4 st[NR][V4];
  float *W = p.w + (((int64_t)slot * p.heads + h) * p.dv + db * 64 + grp * NR) * DK + li * 4;
#pragma unroll
  for (int i = 0; i < NR; ++i)
#pragma unroll
    for (int j = 0; j < V4; ++j) st[i][j] = *reinterpret_cast<const f32x4 *>(W + i * DK + j * 64);
  for (int row = row0;;) {
    const T *K = static_cast<const T *>(p.k) + (int64_t)row * p.ldk + kh * DK + li * 4;
    const T *Q = static_cast<const T *>(p.q) + (int64_t)row * p.ldq + kh * DK + li * 4;
    const float a = p.decay ? __builtin_amdgcn_exp2f(p.decay[h * p.decay_hs + row] * 1.4426950408889634f) : 1.0f;
    const float be = p.beta[h * p.beta_hs + row];
    f32x4 kf[V4], qf[V4];
    float kq = 0.0f;
#pragma unroll
    for (int j = 0; j < V4; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        kf[j][e] = to_f32(K[j * 64 + e]);
        qf[j][e] = to_f32(Q[j * 64 + e]);
        kq += kf[j][e] * qf[j][e];
      }
    float wk[NR], wq[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      wk[i] = wq[i] = 0.0f;
#pragma unroll
      for (int j = 0; j < V4; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          wk[i] += st[i][j][e] * kf[j][e];
          wq[i] += st[i][j][e] * qf[j][e];
        }
    }
#pragma unroll
    for (int m = 1; m < 16; m <<= 1) {
      kq += __shfl_xor(kq, m);
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        wk[i] += __shfl_xor(wk[i], m);
        wq[i] += __shfl_xor(wq[i], m);
      }
    }
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      const int d = h * p.dv + db * 64 + grp * NR + i;
      const float v = to_f32(static_cast<const T *>(p.v)[(int64_t)row * p.ldv + d]);
      const float be_e = be * (v - a * wk[i]);
      if (li == i) static_cast<T *>(p.o)[(int64_t)row * p.ldo + d] = from_f32<T>(p.scale * (a * wq[i] + be_e * kq));
#pragma unroll
      for (int j = 0; j < V4; ++j) st[i][j] = st[i][j] * a + kf[j] * be_e;
    }
    if (!rows_left) break;
    do ++row; while (row < p.n && p.slots[row] != slot);
    if (row >= p.n) break;
  }
#pragma unroll
  for (int i = 0; i < NR; ++i)
#pragma unroll
    for (int j = 0; j < V4; ++j) *reinterpret_cast<f32x4 *>(W + i * DK + j * 64) = st[i][j];
}

template <typename T, int DK>
hipError_t step_impl(const DeltaStepParams &p, hipStream_t s) {
  hipLaunchKernelGGL((delta_step_kernel<T, DK>), dim3((unsigned)((int64_t)p.n * p.heads * (p.dv / 64))), dim3(256), 0, s, p);
  return hipGetLastError();
}

template <typename T, int DK>
hipError_t chunk_impl(const DeltaParams &p, bool backward, hipStream_t s) {
  const bool zero = p.cu && p.n > 0 && (backward || p.zero_unused);     // without offsets every row has a sequence
  const dim3 grid((unsigned)((int64_t)p.nchunk * p.heads) + (zero ? kZeroBlocks : 0));
  if (backward)
    hipLaunchKernelGGL((delta_chunk_kernel<T, DK, true>), grid, dim3(256), 0, s, p);
  else
    hipLaunchKernelGGL((delta_chunk_kernel<T, DK, false>), grid, dim3(256), 0, s, p);
  return hipGetLastError();
}

template <typename T, int DK>
hipError_t states_impl(const DeltaParams &p, hipStream_t s) {
  if (p.segs < 3) {
    hipLaunchKernelGGL((delta_state_kernel<T, DK, kWhole>), dim3(state_wgs(p, kWhole)), dim3(512), 0, s, p);
    return hipGetLastError();
  }
  hipLaunchKernelGGL((delta_state_kernel<T, DK, kFirst>), dim3(state_wgs(p, kFirst)), dim3(512), 0, s, p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((delta_state_kernel<T, DK, kSecond>), dim3(state_wgs(p, kSecond)), dim3(512), 0, s, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_delta_plan(const DeltaParams &p, hipStream_t s) {
  if (p.cu == nullptr || p.nseq <= kDeltaLaneSeqs) return hipSuccess;
  hipLaunchKernelGGL(delta_plan_kernel, dim3(1), dim3(256), 0, s, p);
  return hipGetLastError();
}
hipError_t launch_delta_chunk(const DeltaParams &p, bool bf16, bool backward, hipStream_t s) {
  if (p.nchunk == 0) return hipSuccess;
  return TTT_DELTA_BY_DK(chunk_impl, p, p, backward, s);
}
hipError_t launch_delta_forward(const DeltaParams &p, bool bf16, hipStream_t s) {
  hipError_t e = launch_delta_plan(p, s);
  if (e == hipSuccess) e = launch_delta_chunk(p, bf16, false, s);
  if (e == hipSuccess) e = TTT_DELTA_BY_DK(states_impl, p, p, s);
  return e;
}
hipError_t launch_delta_step(const DeltaStepParams &p, bool bf16, hipStream_t s) {
  if (p.n == 0) return hipSuccess;
  return TTT_DELTA_BY_DK(step_impl, p, p, s);
}

}  // namespace ttt
