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
// over heads and 16-column slices of dv, which do not depend on one another (states).  Every wave lays
// the packed sequences out in chunks for itself; for more than 63 of them a first kernel does (plan).
#include <type_traits>

#include "delta.h"
#include "delta_layout.h"
#include "split.h"

namespace ttt {
namespace {

constexpr int C = kDeltaChunk;
constexpr int SL = kDeltaSlice;

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
constexpr int64_t kSquare = C * C * 2 * kFull;      // bytes of a split 64 x 64 matrix
constexpr int kZeroBlocks = 64;     // workgroups of the chunk kernel's launch that write those zeros

// ------------------------------------------------------------------ chunk terms
// One workgroup per chunk and head: e^gamma, T = (I + L)^-1 by block substitution in fp32 and A,
// and (once per key head) the tokens and their transposes in fragment order.
// Substitution, not products of powers of L: those grow without bound where keys repeat.
// 687 chunks of 4 heads of 256, bf16: 108 us for 565 MB, 5.2 TB/s, what a copy reaches; 22 chunks 16.5 us,
// the latency of the loads and the substitution.
template <typename T, int DK, bool BWD>
__global__ __launch_bounds__(256, sizeof(T) == 2 ? 2 : 1) void delta_chunk_kernel(DeltaParams p) {
  constexpr int kPitch = DK + 16 / (int)sizeof(T), NK = DK / 32, kA = C + 4, TP = kTok<T>;
  constexpr int kTokBytes = C * kPitch * (int)sizeof(T), kABytes = C * kA * 4;
  __shared__ __attribute__((aligned(16))) unsigned char s_raw[kTokBytes > kABytes ? kTokBytes : kABytes];
  __shared__ double s_gam[C];
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
  const int item = xcd_item(items), h = item % p.heads, c = item / p.heads;
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
  if (t < C) {
    const bool ok = t < ck.len;
    double gam = 0.0;
    if (ok && p.decay) {
      const float x = p.decay[h * p.decay_hs + ck.tok0 + t];
      gam = x < -200.0f ? -200.0 : (double)x;           // e^-200 is 0 in fp32; -inf would leave inf - inf
    }
    for (int d = 1; d < C; d <<= 1) {
      const double x = __shfl_up(gam, d);
      if (t >= d) gam += x;
    }
    s_gam[t] = gam;
    const float be = ok ? p.beta[h * p.beta_hs + ck.tok0 + t] : 0.0f;
    s_beta[t] = be;
    p.be[ch * C + t] = be;
    if (BWD) p.gam[ch * C + t] = gam;
    p.eg[ch * C + t] = exp_of(gam);
    p.el[ch * C + t] = exp_of(__shfl(gam, 63) - gam);
  }
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
  if (writer) write_transposed(p.kt);
  __syncthreads();
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int col = 16 * j + li;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = 16 * w + 4 * g + r;
      const float d = exp_of(row >= col ? s_gam[row] - s_gam[col] : 0.0);
      const bool in = row < ck.len && col <= row;
      s_l[row][col] = in && col < row ? s_beta[row] * d * kk[j][r] : 0.0f;
      s_a[row * kA + col] = in ? p.scale * d * qk[j][r] : 0.0f;
      s_t[row][col] = 0.0f;
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
      store_split(p.am + mat, plane, e, split_of<kOut<T>>(ld8(s_a + row * kA + k0)));
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
// One workgroup per sequence, head and 16-column slice of dv, over the chunks in order.  Its first
// four waves have the rows of the chunk (wave w rows 16 w ..), the last four the state: lane
// (g, li) of wave w holds W[dv = li][dk = w DK/4 + 16 i + 4 g + r] in fp32 accumulators.  A chunk
// is three steps, each ended by an exchange through LDS:
//   rows: P = K W0^T, R        rows: U = T R        state: W += (el o U)^T K;  rows: O = Q W0^T, A U
// so two waves share a SIMD and one works while the other waits or loads.  Tokens and chunk terms
// go from memory straight into operand registers (each is used once), the next chunk's as soon
// as this chunk's have been used, Q into the registers that K leaves, A into those of T.  Bound by the
// order of the chunks: 2.45 us each, heads of 256, of which the matrix cores work 0.5 and the operands,
// 138 KB, take 0.9 at the 64 bytes a clock of a CU; the rest is the three exchanges, one after another.
// BWD writes the states and U that the gradient needs, in place of the outputs.
//
// Where sequences are long and few, the chunks of one are cut in segments that run at once (the state is
// linear in the one before): W after a segment = W before it times M + U, U the state that the segment
// alone leaves and M the one that a unit matrix becomes in it with v = 0.
//   kFirst: the first segment, outputs and all; U and M of the others but the last, of which M is
//           dk / 16 more slices of rows
//   kSecond: the others, each from its own starting state, (W_1 M_1 + U_1) M_2 + U_2 ..
// 687 chunks of 4 heads of 256: 1680 us whole, 534 + 398 in five segments (448 and 256 workgroups; a CU's
// two then take 3.9 us a chunk).
template <typename T, int DK, bool BWD, int PART>
__global__ __launch_bounds__(512, sizeof(T) == 2 ? 4 : 2) void delta_state_kernel(DeltaParams p) {
  constexpr int NT = DK / 64, NK = DK / 32, TP = kTok<T>, UP = BWD ? kFull : kOut<T>;
  __shared__ __attribute__((aligned(16))) SplitTile<kFull, SL, DK> s_w[2];
  __shared__ __attribute__((aligned(16))) SplitTile<kFull, SL, C> s_r, s_ul;
  __shared__ __attribute__((aligned(16))) SplitTile<UP, SL, C> s_u;
  constexpr int64_t tokens = DK * C * 2 * TP, tplane = DK * C * 2;      // bytes of a chunk's tokens and a part
  const int slices = p.dv / SL, item = xcd_item(gridDim.x);
  const int wave = wave_id(), w = wave & 3, l = threadIdx.x & 63, g = l >> 4, li = l & 15;
  int bh, sl, seg = 0;
  bool unit = false;                    // rows of M
  if constexpr (PART == kFirst) {
    const int each = slices + DK / SL, all = slices + (p.segs - 2) * each;
    bh = item / all, sl = item % all;
    if (sl >= slices) {
      sl -= slices;
      seg = 1 + sl / each, sl %= each;
      unit = sl >= slices;
      if (unit) sl -= slices;
    }
  } else if constexpr (PART == kSecond) {
    const int all = (p.segs - 1) * slices;
    bh = item / all, sl = item % slices;
    seg = 1 + item % all / slices;
  } else {
    bh = item / slices, sl = item % slices;
  }
  const int h = bh % p.heads, b = bh / p.heads;
  const int kh = h / (p.heads / p.key_heads);
  const DeltaSeq sq = seq_of(p, b);
  const int chunks = (sq.len + C - 1) / C;
  int c_first = 0, c_end = chunks;
  if constexpr (PART != kWhole) {
    const int per = (chunks + p.segs - 1) / p.segs;
    c_first = seg * per, c_end = c_first + per < chunks ? c_first + per : chunks;
    if (seg > 0 && (c_first >= c_end || (PART == kFirst && c_end == chunks))) return;   // empty, or the last
  }
  const int64_t ch0 = (int64_t)sq.chunk0 * p.heads + h, ck0 = (int64_t)sq.chunk0 * p.key_heads + kh;
  const int64_t plane = C * C * 2;
  constexpr int64_t mplane = DK * DK * 2;
  // U (this lane's row) and M of segment j
  const auto u_of = [&](int j) {
    return p.seg_u + (((int64_t)(b * (p.segs - 1) + j) * p.heads + h) * p.dv + sl * SL + li) * DK + 4 * g;
  };
  const auto m_of = [&](int j) {
    return p.seg_m + ((int64_t)(b * (p.segs - 2) + j - 1) * p.heads + h) * (mplane * kFull * (BWD ? 2 : 1));
  };
  if constexpr (PART == kSecond) join_segments<DK>(s_w, seg, u_of, m_of);
  if (wave < 4) {
    const int t4 = 16 * w + 4 * g;      // this lane's four rows of every 64 x 16 product
    const int vcol = h * p.dv + (unit ? 0 : sl * SL);
    const Rows4<T> v_rows(t4, li, p.ldv), o_rows(t4, li, BWD ? 0 : p.ldo);
    const auto rows = [&](auto live) {
      constexpr bool OUT = decltype(live)::value && !BWD, RECORD = decltype(live)::value && BWD;
      Split<TP> kf[NK], qf[OUT ? NK : 1];
      Split<kFull> tf[2];
      Split<kOut<T>> af[2];
      T v[4];
      f32x4 eg, el, be;
      const auto load_token = [&](const char *tok, int c, int i) {
        return load_frag<TP>(tok + (ck0 + (int64_t)c * p.key_heads) * tokens, tplane, w * NK + i);
      };
      const auto load_values = [&](int c) {
        const int64_t o = (ch0 + (int64_t)c * p.heads) * C + t4;
        eg = *reinterpret_cast<const f32x4 *>(p.eg + o);
        el = *reinterpret_cast<const f32x4 *>(p.el + o);
        be = *reinterpret_cast<const f32x4 *>(p.be + o);
        v_rows.load(static_cast<const T *>(p.v) + ((int64_t)sq.start + c * C) * p.ldv + vcol, t4, sq.len - c * C, v);
      };
      const auto load_square = [&](const char *m, int c, auto &f) {
#pragma unroll
        // (the second half is zero for the first two waves, whose products leave it out; loads under a
        // condition would make every later wait one for all loads)
        for (int i = 0; i < 2; ++i)
          f[i] = load_frag<sizeof(f[0]) / 16>(m + (ch0 + (int64_t)c * p.heads) * kSquare, plane, w * 2 + i);
      };
      if (c_first < c_end) {
#pragma unroll
        for (int i = 0; i < NK; ++i) kf[i] = load_token(p.kp, c_first, i);
        load_values(c_first);
        load_square(p.tm, c_first, tf);
      }
      lds_barrier();
      for (int c = c_first; c < c_end; ++c) {
        const int len = sq.len - c * C < C ? sq.len - c * C : C, nx = c + 1 < c_end ? c + 1 : c;
        const SplitTile<kFull, SL, DK> &W0 = s_w[BWD ? 0 : (c - c_first) & 1];
        Sums<kFull> pa;
#pragma unroll
        for (int i = 0; i < NK; ++i) {
          pa.add(kf[i], W0.ld(li, 32 * i + 8 * g));
          if constexpr (OUT) qf[i] = load_token(p.qp, c, i);    // into the registers that K leaves
          else kf[i] = load_token(p.kp, nx, i);
        }
        f32x4 rr = pa.sum();
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float vr = unit ? 0.0f : to_f32(v[r]);
          rr[r] = t4 + r < len ? be[r] * (vr - eg[r] * rr[r]) : 0.0f;
        }
        const f32x4 eg_now = eg, el_now = el;
        s_r.st4(li, t4, rr);
        lds_barrier();
        load_values(nx);
        Sums<kFull> tr;
        tr.add(tf[0], s_r.ld(li, 8 * g));
        if (w >= 2) tr.add(tf[1], s_r.ld(li, 32 + 8 * g));
        const f32x4 u = tr.sum();
        s_ul.st4(li, t4, u * el_now);
        if (OUT || RECORD) s_u.st4(li, t4, u);
        if constexpr (OUT) load_square(p.am, c, af);
        else load_square(p.tm, nx, tf);
        lds_barrier();
        if constexpr (RECORD)
          s_u.copy_t4(0, 16 * w, p.u + (ch0 + (int64_t)c * p.heads) * (C * p.dv * 2 * kFull), (int64_t)C * p.dv * 2,
                      frag_at(16 * w + li, sl * SL + 4 * g, p.dv / 32));
        if constexpr (OUT) {
          Sums<kOut<T>> qa[2];
#pragma unroll
          for (int i = 0; i < NK; ++i) {
            qa[i & 1].add(qf[i], W0.template ld<kOut<T>>(li, 32 * i + 8 * g));
            kf[i] = load_token(p.kp, nx, i);
          }
          Sums<kOut<T>> au;
          au.add(af[0], s_u.template ld<kOut<T>>(li, 8 * g));
          if (w >= 2) au.add(af[1], s_u.template ld<kOut<T>>(li, 32 + 8 * g));
          const f32x4 o = (qa[0].sum() + qa[1].sum()) * eg_now * p.scale + au.sum();
          load_square(p.tm, nx, tf);
          o_rows.store(static_cast<T *>(p.o) + ((int64_t)sq.start + c * C) * p.ldo + h * p.dv + sl * SL, t4, len, o);
        }
        lds_barrier();
      }
    };
    if (PART != kFirst || seg == 0) rows(std::true_type{});
    else rows(std::false_type{});
  } else {
    const int64_t wrow = ((int64_t)bh * p.dv + sl * SL + li) * DK + w * (DK / 4) + 4 * g;
    f32x4 st[NT];
    Split<TP> ktf[NT][2];
    float ec = 0.0f;
    const auto load_transposed = [&](int c, int i, int x) {
      return load_frag<TP>(p.kt + (ck0 + (int64_t)c * p.key_heads) * tokens, tplane, (w * NT + i) * 2 + x);
    };
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int col = (w * NT + i) * 16 + 4 * g;
      if constexpr (PART == kSecond) {
        st[i] = s_w[0].at4(li, col);
      } else {
        if (PART == kFirst && seg > 0) {
#pragma unroll
          for (int r = 0; r < 4; ++r) st[i][r] = unit && col + r == sl * SL + li ? 1.0f : 0.0f;
        } else {
          st[i] = *reinterpret_cast<const f32x4 *>(p.w + wrow + 16 * i);
        }
        s_w[0].st4(li, col, st[i]);
      }
    }
    const auto chain = [&](auto live) {
      if (c_first < c_end) {
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int x = 0; x < 2; ++x) ktf[i][x] = load_transposed(c_first, i, x);
        ec = p.eg[(ch0 + (int64_t)c_first * p.heads) * C + C - 1];
      }
      lds_barrier();
      for (int c = c_first; c < c_end; ++c) {
        const int nx = c + 1 < c_end ? c + 1 : c;
        if constexpr (decltype(live)::value && BWD) {    // the state before the chunk, dk x dv
          float *o = p.w0t + (ch0 + (int64_t)c * p.heads) * (DK * p.dv);
#pragma unroll
          for (int i = 0; i < NT; ++i)
            s_w[0].copy_t4(0, (w * NT + i) * 16, o + frag_at((w * NT + i) * 16 + li, sl * SL + 4 * g, p.dv / 32));
        }
        lds_barrier();
        lds_barrier();
        SplitTile<kFull, SL, DK> &W1 = s_w[BWD ? 0 : ~(c - c_first) & 1];
        const Split<kFull> u0 = s_ul.ld(li, 8 * g), u1 = s_ul.ld(li, 32 + 8 * g);
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          Sums<kFull> d;
          d.add(ktf[i][0], u0);
          d.add(ktf[i][1], u1);
          st[i] = st[i] * ec + d.sum();
          W1.st4(li, (w * NT + i) * 16 + 4 * g, st[i]);
        }
        lds_barrier();
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int x = 0; x < 2; ++x) ktf[i][x] = load_transposed(nx, i, x);
        ec = p.eg[(ch0 + (int64_t)nx * p.heads) * C + C - 1];
      }
    };
    if (!BWD || PART != kFirst || seg == 0) chain(std::true_type{});
    else chain(std::false_type{});
    if (PART == kFirst && unit) {       // M^T: rows dk, k = the rows that this slice has; M for the gradient
      const SplitTile<kFull, SL, DK> &W = s_w[BWD ? 0 : (c_end - c_first) & 1];
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const int col = (w * NT + i) * 16;
        W.copy_t4(0, col, m_of(seg), mplane, frag_at(col + li, sl * SL + 4 * g, NK));
        if (BWD) W.copy4(li, col + 4 * g, m_of(seg) + kFull * mplane, mplane, frag_at(sl * SL + li, col + 4 * g, NK));
      }
    } else if ((PART == kFirst && c_end < chunks) || (!BWD && c_end == chunks)) {
      float *o = PART == kFirst && c_end < chunks ? u_of(seg) + w * (DK / 4) : p.w_out + wrow;
#pragma unroll
      for (int i = 0; i < NT; ++i) *reinterpret_cast<f32x4 *>(o + 16 * i) = st[i];
    }
  }
}

// ------------------------------------------------------------------ one token
// The recurrent form for one token of each row's sequence: one read and one write of the state.
//   o = scale (a W q + beta e (k.q)),  W <- a W + beta e k^T,  e = v - a W k
// 16 lanes hold one dv row of W; rows that name the same state are applied in row order by the
// workgroups of the first of them.  Bound by memory: 300 rows of 8 heads of 128 x 128 move 316 MB in
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

template <typename T, int DK, bool BWD>
hipError_t states_of(const DeltaParams &p, hipStream_t s) {
  const int bh = p.nseq * p.heads, slices = p.dv / SL;
  if (p.segs < 3) {
    hipLaunchKernelGGL((delta_state_kernel<T, DK, BWD, kWhole>), dim3(bh * slices), dim3(512), 0, s, p);
    return hipGetLastError();
  }
  hipLaunchKernelGGL((delta_state_kernel<T, DK, BWD, kFirst>), dim3(bh * (slices + (p.segs - 2) * (slices + DK / SL))),
                     dim3(512), 0, s, p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((delta_state_kernel<T, DK, BWD, kSecond>), dim3(bh * (p.segs - 1) * slices), dim3(512), 0, s, p);
  return hipGetLastError();
}
template <typename T, int DK>
hipError_t states_impl(const DeltaParams &p, bool backward, hipStream_t s) {
  return backward ? states_of<T, DK, true>(p, s) : states_of<T, DK, false>(p, s);
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
hipError_t launch_delta_states(const DeltaParams &p, bool bf16, bool backward, hipStream_t s) {
  return TTT_DELTA_BY_DK(states_impl, p, p, backward, s);
}
hipError_t launch_delta_forward(const DeltaParams &p, bool bf16, hipStream_t s) {
  hipError_t e = launch_delta_plan(p, s);
  if (e == hipSuccess) e = launch_delta_chunk(p, bf16, false, s);
  if (e == hipSuccess) e = launch_delta_states(p, bf16, false, s);
  return e;
}
hipError_t launch_delta_step(const DeltaStepParams &p, bool bf16, hipStream_t s) {
  if (p.n == 0) return hipSuccess;
  return TTT_DELTA_BY_DK(step_impl, p, p, s);
}

}  // namespace ttt
