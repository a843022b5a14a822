// Windowed attention over packed sequences: one pass over the keys with a running maximum and sum.
//   s_ij = scale q_i k_j over the keys that i sees,  o_i = sum_j e^(s_ij - lse_i) v_j,  lse_i = ln sum_j e^s_ij
// See attn_tile.h for the orientation of the products and attention.h for the parameters.
// Bound by the products (4 d operations a visible pair) and the exponentials: at d = 64 a pair costs as long in e^x and the
// sums as in the matrix cores, so that two to four waves a SIMD have to overlap the two.  MI355X, bf16, 8192 x 8192, no mask:
// 8 heads of 64 211 us (650 TFLOP/s; 48 heads 853), 8 of 128 279 (985), 4 of 256 445 (617: one workgroup a CU, bound by LDS
// reads as much as by products); fp32, 8 heads of 64 1060 us and of 128 2038 (130 and 135 of 137 TFLOP/s of a large product),
// 4 of 256 2818 (98: tiles of 64 rows in four waves, one a SIMD, which nothing overlaps).
// bf16 probabilities are rounded once more, to the operands of the second product: half a step each, 2^-8 of a term at most and
// independent of v.  Outputs are 2.3e-3 off 64 bits, of which their own rounding is 1.7e-3; two operands for one would make
// three products of two.  Sums of probabilities and of outputs are fp32.
// What was tried and did not pay: three LDS stages, touching tiles ahead for L2, wave priorities (4% at d = 256 alone), eight
// waves that take turns at products and exponentials (25% slower: a barrier makes both halves as long as the longer).
#include <algorithm>

#include "attn_tile.h"

namespace ttt {
namespace {

constexpr int kZeroBlocks = 32;     // workgroups that fill rows of no sequence

// Query tile `item` of all heads; false: there is none.  Without a window late tiles see the most keys: the late half first,
// then the early half from its first tile on, so that a CU that takes one of each has as much to do as the others.
__device__ __forceinline__ bool forward_tile(const AttnParams &p, int item, AttnSeq *s, int *tile, int *seq, int *h) {
  *h = quotient(item, p.per_qtiles);
  const int order = item - *h * p.qtiles, half = (p.qtiles + 1) / 2;
  return tile_of<false>(p, order < half ? p.qtiles - 1 - order : order - half, s, tile, seq);
}

// Four waves of NC x 16 queries each; BK keys at a time through two LDS buffers.  KG = 2: eight waves, the second four with
// the same queries and every other tile of keys, joined at the end: where there are few query tiles a SIMD then has two
// waves that wait in turn.
template <typename T, int D, int NC, int BK, int KG, int OCC>
__global__ __launch_bounds__(256 * KG, OCC) void attn_forward_kernel(AttnParams p) {
  typedef AttnTile<T, D> Tile;
  typedef typename FragOf<T>::type Frag;
  constexpr int NK = D / 32, ND = D / 16, NU = BK / 16, kTile = BK * Tile::kRow, QR = 64 * NC;
  constexpr int kPitch = D + 4;                       // floats of a query's row of the second four waves' sums
  __shared__ __attribute__((aligned(1024))) unsigned char s_kv[KG][2][2][kTile];
  static_assert(KG == 1 || QR * kPitch * 4 <= (int)sizeof(s_kv), "");
  const int cut = (p.qtiles * p.heads - p.whole) * p.splits, items = p.whole + cut;
  if ((int)blockIdx.x >= items) {
    if (threadIdx.x >= 256) return;
    const int blk = blockIdx.x - items;
    const int2 used = used_rows<false>(p);
    if (p.zero_unused) zero_unused_rows<T>(used, p.nq, p.o, p.ldo, p.heads * D, blk, kZeroBlocks);
    if (p.lse)
      for (int h = 0; h < p.heads; ++h)
        for (int64_t i = blk * 256 + threadIdx.x; i < used.x + (int64_t)(p.nq - used.y); i += kZeroBlocks * 256)
          p.lse[(int64_t)h * p.nq + (i < used.x ? i : used.y + (i - used.x))] = -__builtin_inff();
    return;
  }
  const bool in_parts = (int)blockIdx.x >= p.whole;
  const int id = in_parts ? attn_item(blockIdx.x - p.whole, cut) : attn_item(blockIdx.x, p.whole);
  const int one = in_parts ? quotient(id, p.per_splits) : id, split = in_parts ? id - one * p.splits : 0;
  AttnSeq s;
  int tile, seq, h;
  if (!forward_tile(p, in_parts ? p.whole + one : one, &s, &tile, &seq, &h)) return;
  const int kh = quotient(h, p.group);
  const int wave8 = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wave = wave8 & 3, kg = wave8 >> 2;
  const int l = threadIdx.x & 63, g = l >> 4, li = l & 15;
  const int t0 = tile * QR, row0 = t0 + wave * 16 * NC;
  const T *kb = static_cast<const T *>(p.k) + (int64_t)s.ks * p.ldk + kh * D;
  const T *vb = static_cast<const T *>(p.v) + (int64_t)s.ks * p.ldv + kh * D;

  Frag q[NC][NK];
  own_rows<T, D, NC>(q, static_cast<const T *>(p.q) + (int64_t)s.qs * p.ldq + h * D, p.ldq, row0, s.ql);
  int lo[NC], hi[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int i = row0 + 16 * c + li;
    const int2 r = i < s.ql ? seen_keys(p, s, i) : int2{0, 0};
    lo[c] = r.x, hi[c] = r.y;
  }
  // the workgroup's keys: sinks [0, se) and the window [k0, k1); this wave's: from its first and last row
  const int last = t0 + QR < s.ql ? t0 + QR : s.ql, wlast = row0 + 16 * NC < s.ql ? row0 + 16 * NC : s.ql;
  const int k0 = seen_keys(p, s, t0).x, k1 = seen_keys(p, s, last - 1).y, se = p.sinks < k0 ? p.sinks : k0;
  const int2 wa = row0 < s.ql ? seen_keys(p, s, row0) : int2{0, 0}, wb = row0 < s.ql ? seen_keys(p, s, wlast - 1) : int2{0, 0};
  const int ns = tiles_of(se, BK), nt = ns + tiles_of(k1 - k0, BK);
  const int share = in_parts ? quotient(nt + p.splits - 1, p.per_splits) : nt, first = split * share;
  const int end = first + share < nt ? first + share : nt;
  const typename Tile::Lane lane = Tile::lane();
  const typename Tile::template Copy<BK> copy_k(p.ldk), copy_v(p.ldv);
  const KeyWalk<T, BK> start(first + kg, ns, se, k0, k1, kb, vb, p.ldk, p.ldv);
  const auto fetch = [&](const KeyWalk<T, BK> &w, int stage) {
    copy_k.fetch(w.k, w.end() - w.j, s_kv[kg][stage][0]);
    copy_v.fetch(w.v, w.end() - w.j, s_kv[kg][stage][1]);
  };

  const float c2 = p.scale * kLog2e;
  f32x4 o[ND][NC];
  float m[NC], sum[NC];
  bool huge = false;
  // A second pass where the first left an infinity or a NaN: a value of v that is not finite reaches, as a zero times it,
  // rows that do not see its key.  In tiles that are not seen whole it is then added to those that see it and removed.
  for (int careful = 0; careful < 2; ++careful) {
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      m[c] = -__builtin_inff(), sum[c] = 0.0f;
#pragma unroll
      for (int d = 0; d < ND; ++d) o[d][c] = zero_f4();
    }
    __syncthreads();
    KeyWalk<T, BK> ahead = start;
    if (first + kg < end) fetch(ahead, 0);
    // (with KG = 2 the second four waves' last tile may be none: they go along for the barriers)
    for (int t = first, stage = 0; t < end; t += KG, stage ^= 1) {
      const bool there = KG == 1 || t + kg < end;
      const int2 r{ahead.j, ahead.end()};
#pragma unroll
      for (int i = 0; i < KG; ++i) ahead.next();
      landed();                                       // this tile is there, and nobody reads the one before it any more
      if (t + KG + kg < end) fetch(ahead, stage ^ 1);
      const bool full = r.y - r.x == BK && wa.y >= r.y && (wb.x <= r.x || r.y <= p.sinks);
      const bool none = !there || !(r.x < wb.y && (r.y > wa.x || r.x < p.sinks));
      unsigned char *vt = s_kv[kg][stage][1];
      const int ka = Tile::offset(s_kv[kg][stage][0]), va = Tile::offset(vt);
      Frag pr[NU / 2][NC];
      if (!none) {
        f32x4 sc[NU][NC];
#pragma unroll
        for (int u = 0; u < NU; ++u) {
#pragma unroll
          for (int c = 0; c < NC; ++c) sc[u][c] = zero_f4();
#pragma unroll
          for (int k = 0; k < NK; ++k) {
            const Frag a = Tile::rows(ka, lane, 16 * u, k);
#pragma unroll
            for (int c = 0; c < NC; ++c) sc[u][c] = mma(a, q[c][k], sc[u][c]);
          }
        }
        if (!full) {
          rarely();
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            const int e = hi[c] < r.y ? hi[c] : r.y;
#pragma unroll
            for (int u = 0; u < NU; ++u)
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                const int j = r.x + 16 * u + 4 * g + x;
                sc[u][c][x] = ((j < e) & ((j >= lo[c]) | (j < p.sinks))) ? sc[u][c][x] : -__builtin_inff();
              }
          }
        }
        float mx[NC];
        bool up = false;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          mx[c] = -__builtin_inff();
#pragma unroll
          for (int u = 0; u < NU; ++u)
#pragma unroll
            for (int x = 0; x < 4; ++x) mx[c] = fmaxf(mx[c], sc[u][c][x]);
          up |= (mx[c] - m[c]) * c2 > 8.0f;
        }
        // the sums are kept relative to m, which follows a column's maximum only where that grew by more than 2^8: P
        // stays below 2^8, which costs no digits
        if (__any(up)) {
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            mx[c] = column_max(mx[c]);
            const float to = (mx[c] - m[c]) * c2 > 8.0f ? mx[c] : m[c], a = to == m[c] ? 1.0f : __builtin_amdgcn_exp2f((m[c] - to) * c2);
            m[c] = to, sum[c] *= a;
            huge |= fabsf(to) * c2 > kHuge && to > -__builtin_inff();
#pragma unroll
            for (int d = 0; d < ND; ++d) o[d][c] *= a;
          }
          huge = __any(huge);
        }
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          const float top = m[c] == -__builtin_inff() ? 0.0f : m[c];
          float base = -top * c2;
          if (huge) {
            rarely();                                 // in some column: there the maximum is taken off first
            const bool off = fabsf(base) > kHuge;
            base = off ? 0.0f : base;
#pragma unroll
            for (int u = 0; u < NU; ++u)
#pragma unroll
              for (int x = 0; x < 4; ++x) sc[u][c][x] -= off ? top : 0.0f;
          }
#pragma unroll
          for (int u = 0; u < NU; ++u)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              sc[u][c][x] = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[u][c][x], c2, base));
              sum[c] += sc[u][c][x];
            }
#pragma unroll
          for (int u = 0; u < NU; u += 2) pr[u / 2][c] = pack44<T>(sc[u][c], sc[u + 1][c]);      // (rounded: see above)
        }
      }
      if (careful) {
        const bool whole = r.y - r.x == BK && seen_keys(p, s, t0).y >= r.y && (seen_keys(p, s, last - 1).x <= r.x || r.y <= p.sinks);
        if (!whole && !none)
          for (int x = 0; x < BK; ++x) {
            const int j = r.x + x;
#pragma unroll
            for (int d = 0; d < ND; ++d)
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                const float f = to_f32(*reinterpret_cast<const T *>(vt + Tile::elem(x, 16 * d + 4 * g + y)));
                if (fabsf(f) < __builtin_inff()) continue;
#pragma unroll
                for (int c = 0; c < NC; ++c)
                  if (j < r.y && j < hi[c] && (j >= lo[c] || j < p.sinks)) o[d][c][y] += f;
              }
          }
        __syncthreads();
        if (!whole && there) Tile::settle(vt, 0, BK);
        __syncthreads();
      }
      if (!none) {
#pragma unroll
        for (int u = 0; u < NU / 2; ++u)
#pragma unroll
          for (int d = 0; d < ND; ++d) {
            const Frag a = Tile::cols(va, lane, 32 * u, d);
#pragma unroll
            for (int c = 0; c < NC; ++c) o[d][c] = mma(a, pr[u][c], o[d][c]);
          }
      }
    }
    bool odd = false;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int x = 0; x < 4; ++x) odd |= !(fabsf(o[d][c][x]) < __builtin_inff());
    if (!__syncthreads_or(odd)) break;
  }
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    sum[c] += __shfl_xor(sum[c], 16);
    sum[c] += __shfl_xor(sum[c], 32);
  }
  if constexpr (KG == 2) {                            // (nobody reads the tiles behind the barrier above)
    float *so = reinterpret_cast<float *>(s_kv) + (wave * 16 * NC + li) * kPitch;       // a query's sums, then its m and sum
    if (kg == 1)
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        float *to = so + 16 * c * kPitch;
#pragma unroll
        for (int d = 0; d < ND; ++d) *reinterpret_cast<f32x4 *>(to + 16 * d + 4 * g) = o[d][c];
        if (g == 0) to[D] = m[c], to[D + 1] = sum[c];
      }
    __syncthreads();
    if (kg == 1) return;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const float *from = so + 16 * c * kPitch;
      const float m2 = from[D], top = fmaxf(m[c], m2);
      const float a = m[c] == top ? 1.0f : __builtin_amdgcn_exp2f((m[c] - top) * c2);
      const float b = m2 == top ? 1.0f : __builtin_amdgcn_exp2f((m2 - top) * c2);
      m[c] = top, sum[c] = sum[c] * a + from[D + 1] * b;
#pragma unroll
      for (int d = 0; d < ND; ++d) o[d][c] = o[d][c] * a + *reinterpret_cast<const f32x4 *>(from + 16 * d + 4 * g) * b;
    }
  }
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int i = row0 + 16 * c + li;
    if (i >= s.ql) continue;
    const bool empty = hi[c] == lo[c] && (p.sinks == 0 || lo[c] == 0);
    const int64_t row = s.qs + i;
    if (in_parts) {
      const int64_t at = (int64_t)id * QR + (i - t0);
#pragma unroll
      for (int d = 0; d < ND; ++d) store4(p.part_o + at * D + 16 * d + 4 * g, o[d][c]);
      if (g == 0) p.part_ml[at] = float2{m[c], empty ? -1.0f : sum[c]};
      continue;
    }
    const float inv = empty ? 0.0f : 1.0f / sum[c];
    T *out = static_cast<T *>(p.o) + row * p.ldo + h * D + 4 * g;
#pragma unroll
    for (int d = 0; d < ND; ++d) store4(out + 16 * d, o[d][c] * inv);
    if (p.lse && g == 0)
      p.lse[(int64_t)h * p.nq + row] = empty ? -__builtin_inff() : (m[c] * c2 + __builtin_amdgcn_logf(sum[c])) * kLn2;
  }
}

// Joins the ranges of keys, in their order: a query tile by blockIdx.x, 1024 / D of its rows by blockIdx.y, D / 4 lanes a row.
template <typename T, int D> __global__ __launch_bounds__(256) void attn_join_kernel(AttnParams p) {
  constexpr int L = D / 4;
  const int c = threadIdx.x % L, r = blockIdx.y * (256 / L) + threadIdx.x / L;
  AttnSeq s;
  int tile, seq, h;
  if (!forward_tile(p, p.whole + blockIdx.x, &s, &tile, &seq, &h)) return;
  const int i = tile * p.qrows + r;
  if (i >= s.ql) return;
  const int64_t row = s.qs + i, first = (int64_t)blockIdx.x * p.splits * p.qrows + r;
  const float c2 = p.scale * kLog2e;
  float m = -__builtin_inff(), sum = 0.0f;
  for (int x = 0; x < p.splits; ++x) m = fmaxf(m, p.part_ml[first + x * p.qrows].x);
  f32x4 o = zero_f4();
  bool empty = false;
#pragma unroll 4
  for (int x = 0; x < p.splits; ++x) {
    const float2 ml = p.part_ml[first + x * p.qrows];
    empty |= ml.y < 0.0f;
    const float w = ml.x == m ? 1.0f : __builtin_amdgcn_exp2f((ml.x - m) * c2);
    sum += ml.y * w;
    o += *reinterpret_cast<const f32x4 *>(p.part_o + (first + x * p.qrows) * D + 4 * c) * w;
  }
  const float inv = empty ? 0.0f : 1.0f / sum;
  store4(static_cast<T *>(p.o) + row * p.ldo + h * D + 4 * c, o * inv);
  if (p.lse && c == 0) p.lse[(int64_t)h * p.nq + row] = empty ? -__builtin_inff() : (m * c2 + __builtin_amdgcn_logf(sum)) * kLn2;
}

// More sequences than a wave has lanes: one workgroup writes the table.
__global__ __launch_bounds__(1024) void attn_plan_kernel(AttnParams p) {
  __shared__ int s_a[1024], s_b[1024];
  const int t = threadIdx.x;
  int mq = 0, mk = 0, cq = 0, ck = 0;           // maxima and tile counts of all before
  // an inclusive scan of two values over the workgroup
  const auto scan = [&](int &a, int &b, bool sum) {
    for (int d = 1; d < 1024; d <<= 1) {
      __syncthreads();
      s_a[t] = a, s_b[t] = b;
      __syncthreads();
      if (t < d) continue;
      const int x = s_a[t - d], y = s_b[t - d];
      a = sum ? a + x : (x > a ? x : a), b = sum ? b + y : (y > b ? y : b);
    }
    __syncthreads();
    s_a[t] = a, s_b[t] = b;
    __syncthreads();
  };
  // sequences in groups of 1023: the last lane has the next group's first offset
  for (int b0 = 0; b0 <= p.nseq; b0 += 1023) {
    const int i = b0 + t;
    int q = i <= p.nseq ? attn_offset(p.cu_q, i, p.nq) : 0, k = i <= p.nseq ? attn_offset(p.cu_k, i, p.nk) : 0;
    q = q > mq ? q : mq, k = k > mk ? k : mk;
    scan(q, k, false);
    const bool own = t < 1023 && i < p.nseq;
    const int ql = own ? s_a[t + 1] - q : 0, kl = own ? s_b[t + 1] - k : 0;
    mq = s_a[1023], mk = s_b[1023];
    int tq = tiles_of(ql, p.qrows), tk = tiles_of(kl, p.krows);
    const int wq = tq, wk = tk;
    scan(tq, tk, true);
    if (t < 1023 && i <= p.nseq) p.seqs[i] = AttnSeq{q, ql, k, kl, cq + tq - wq, ck + tk - wk};
    cq += s_a[1023], ck += s_b[1023];
    __syncthreads();
  }
}

template <typename T, int D, int NC, int BK, int KG, int OCC> hipError_t go(const AttnParams &p, hipStream_t s) {
  const int tiles = p.qtiles * p.heads - p.whole;     // in ranges
  hipLaunchKernelGGL((attn_forward_kernel<T, D, NC, BK, KG, OCC>), dim3(p.whole + tiles * p.splits + (p.cu_q ? kZeroBlocks : 0)),
                     dim3(256 * KG), 0, s, p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || tiles == 0) return e;
  hipLaunchKernelGGL((attn_join_kernel<T, D>), dim3(tiles, p.qrows * D / 1024), dim3(256), 0, s, p);
  return hipGetLastError();
}

}  // namespace

int attn_query_rows(int d, bool bf16, bool small) { return small || (!bf16 && d == 256) ? 64 : 128; }

// Ranges that the keys of a query tile are cut in, for all tiles or, where these are alike, for those behind the last full
// round of workgroups on 256 CUs: what takes least by the time of a tile on a CU alone (measured, as is how many such a CU
// does at once), the rounds of equal workgroups, or of unequal ones the longest and what all keep the CUs busy with, and what
// the ranges' sums cost (at 3 TB/s, with a launch of 4 us).  Of 35 shapes of both types and all d, 100 to 8192 rows, the times
// are 2% over the best number of ranges' in the mean and 29% at most.  10992 queries, 8 heads of 128, 9618 keys each: 688
// workgroups in rounds of 512, all in two ranges 574 us, the last 176 so 538; fp32, 2 heads of 256 on 1, 1974 tokens in 5
// sequences: 209 us in one range, 97 in four.
AttnCut attn_cut(const AttnWork &w, int d, int rows, bool bf16) {
  const bool small = rows == 64;
  const int per_cu = bf16 ? (d == 64 && !small ? 3 : d == 256 ? 1 : 2) : d == 64 ? 2 : 1;
  // us of a tile and 32 keys, and tiles at once
  double alone, at_once;
  if (bf16) {
    alone = small ? (d == 64 ? 0.29 : d == 128 ? 0.45 : 0.84) : d == 64 ? 0.8 : d == 128 ? 0.9 : 1.76;
    at_once = small ? (d == 64 ? 1.4 : d == 128 ? 1.6 : 1.0) : d == 64 ? 2.5 : d == 128 ? 1.6 : 1.0;
  } else {
    alone = small ? (d == 64 ? 1.16 : d == 128 ? 2.2 : 5.1) : d == 64 ? 2.4 : 4.4;
    at_once = d == 64 ? 1.18 : d == 128 && !small ? 1.1 : 1.0;
  }
  const int64_t slots = 256 * per_cu, full = w.even ? w.busy / slots * slots : 0;
  const double longest = w.keys / 32.0 * alone, mean = w.mean_keys / 32.0 * alone, round = per_cu / at_once;
  const auto time = [&](int64_t whole, int s) {
    const int64_t n = (w.busy - whole) * s;
    const double one = longest / s;
    double t = (double)(whole / slots) * round * longest;
    if (w.even)
      t += (double)(n / slots) * round * one + (n % slots ? std::max(1.0, (double)((n % slots + 255) / 256) / at_once) * one : 0.0);
    else
      t += n <= 256 ? one : std::max(one * std::max(1.0, std::min<double>(per_cu, (double)((n + 255) / 256)) / at_once),
                                     (double)w.busy * mean / (256 * at_once) + one / 2);
    return s == 1 ? t : t + 4.0 + 0.1 * s + (double)n * rows * d * 8 / 3e6;
  };
  AttnCut best{w.tiles, 1};
  double least = time(0, 1);
  for (const int64_t whole : {int64_t(0), full})
    for (int s = 2; whole < w.busy && s <= 64 && w.keys / s >= 32; ++s) {
      const double t = time(whole, s);
      if (t < 0.97 * least) least = t, best = AttnCut{whole, s};
    }
  return best;
}

hipError_t launch_attention_plan(const AttnParams &p, hipStream_t s) {
  if (p.cu_q == nullptr || p.nseq <= kAttnLaneSeqs) return hipSuccess;
  hipLaunchKernelGGL(attn_plan_kernel, dim3(1), dim3(1024), 0, s, p);
  return hipGetLastError();
}

hipError_t launch_attention(const AttnParams &p, bool bf16, hipStream_t s) {
  if (p.nq == 0) return hipSuccess;
  const hipError_t e = launch_attention_plan(p, s);
  if (e != hipSuccess) return e;
  const bool small = p.qrows == 64;
  if (bf16) {
    if (p.d == 64) return small ? go<__bf16, 64, 1, 64, 2, 4>(p, s) : go<__bf16, 64, 2, 64, 1, 3>(p, s);
    if (p.d == 128) return small ? go<__bf16, 128, 1, 32, 2, 2>(p, s) : go<__bf16, 128, 2, 64, 1, 2>(p, s);
    return small ? go<__bf16, 256, 1, 32, 2, 2>(p, s) : go<__bf16, 256, 2, 32, 1, 2>(p, s);
  }
  if (p.d == 64) return small ? go<float, 64, 1, 32, 2, 3>(p, s) : go<float, 64, 2, 32, 1, 3>(p, s);
  if (p.d == 128) return small ? go<float, 128, 1, 32, 2, 2>(p, s) : go<float, 128, 2, 32, 1, 2>(p, s);
  return go<float, 256, 1, 32, 1, 1>(p, s);
}

}  // namespace ttt
