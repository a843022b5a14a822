// Gradient of windowed attention, from the forward's lse and output:
//   delta_i = sum_d do_id o_id,  P_ij = e^(s_ij - lse_i),  dS_ij = P_ij (do_i v_j - delta_i)
//   dq_i = scale sum_j dS_ij k_j,   dk_j = scale sum_i dS_ij q_i,   dv_j = sum_i P_ij do_i
// Every workgroup has its own rows' gradients in registers: dk and dv of a key tile, where the heads that share a key head
// follow one another in one sum, or dq of a query tile.  The scores are computed twice (7 products a pair instead of 5): in
// one pass the other side's gradients would be added by atomics, in no fixed order.  Both kinds go in one launch, so that
// the second fills the CUs that the first leaves idle, at its end and where it has few tiles (8192 x 8192 causal, 8 heads of
// 64: 405 -> 280 us; 8 x 1024 tokens, 12 heads of 64 on 4, window 512: 123 -> 92).
// Bound by the products, 7 of 2 d operations a visible pair where the formula has 5.  8192 x 8192 without a mask, bf16: 8 heads
// of 64 560 us, 8 of 128 1070, 4 of 256 1750 (860, 900 and 550 TFLOP/s of the 7; a large product reaches 1216); fp32: 3570,
// 7280 and 8800 us (135, 132 and 109 of 137).
// bf16 P and dS are rounded once, to the operands of the products that add them up (2^-8 of a term at most): gradients are 2.5e-3
// off 64 bits, of which their own rounding is 1.7e-3.  All sums are fp32.
#include <algorithm>
#include <cmath>

#include "attn_tile.h"

namespace ttt {
namespace {

constexpr int kZeroBlocks = 64;

// delta, D / 8 lanes a row and head; the workgroups behind write the zeros of rows of no sequence.
template <typename T, int D> __global__ __launch_bounds__(256) void attn_delta_kernel(AttnParams p, int blocks) {
  constexpr int L = D / 8;
  const int2 used = used_rows<false>(p);
  if ((int)blockIdx.x >= blocks) {
    const int blk = blockIdx.x - blocks;
    const int2 keys = used_rows<true>(p);
    zero_unused_rows<T>(used, p.nq, p.gq, p.ldgq, p.heads * D, blk, kZeroBlocks);
    zero_unused_rows<T>(keys, p.nk, p.gk, p.ldgk, p.key_heads * D, blk, kZeroBlocks);
    zero_unused_rows<T>(keys, p.nk, p.gv, p.ldgv, p.key_heads * D, blk, kZeroBlocks);
    return;
  }
  const int64_t at = (int64_t)blockIdx.x * (256 / L) + threadIdx.x / L;
  if (at >= (int64_t)p.nq * p.heads) return;
  const int h = (int)(at % p.heads), c = threadIdx.x % L;
  const int64_t row = at / p.heads;
  if (row < used.x || row >= used.y) return;
  const auto a = ld8(static_cast<const T *>(p.go) + row * p.ldgo + h * D + 8 * c);
  const auto b = ld8(static_cast<const T *>(p.o) + row * p.ldo + h * D + 8 * c);
  float v = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) v += (float)a[i] * (float)b[i];
#pragma unroll
  for (int m = 1; m < L; m <<= 1) v += __shfl_xor(v, m);
  if (c == 0) p.delta[(int64_t)h * p.nq + row] = v;
}

// Four waves.  The first `keys` workgroups: dk and dv of NCK x 16 keys a wave, of one key head; BQ queries of one head at a time.
// Those behind: dq of NCQ x 16 queries a wave; BK keys at a time.  32 of either go through the registers at once.
template <typename T, int D, int NCQ, int BK, int NCK, int BQ, int OCC>
__global__ __launch_bounds__(256, OCC) void attn_grads_kernel(AttnParams p, int keys) {
  typedef AttnTile<T, D> Tile;
  typedef typename FragOf<T>::type Frag;
  constexpr int NK = D / 32, ND = D / 16, kTile = (BQ > BK ? BQ : BK) * Tile::kRow;
  __shared__ __attribute__((aligned(1024))) unsigned char s_a[2][kTile], s_b[2][kTile];
  __shared__ __attribute__((aligned(256))) float s_lse[2][64], s_del[2][64];
  if ((int)blockIdx.x < keys) {
    const int block = blockIdx.x, blocks = keys;
    constexpr int KR = 64 * NCK;
    const int window_items = p.ktiles * p.key_heads * p.parts, grp = (int)p.group.d;
    const bool sink_item = block >= window_items;
    AttnSeq s;
    int tile, seq, kh, part, parts;
    if (!sink_item) {
      const int item = attn_item(block, window_items), rest = quotient(item, p.per_parts);
      part = item - rest * p.parts, parts = p.parts, kh = quotient(rest, p.per_ktiles);
      if (!tile_of<true>(p, rest - kh * p.ktiles, &s, &tile, &seq)) return;
    } else {
      const int item = attn_item(block - window_items, blocks - window_items), rest = quotient(item, p.per_sink_parts);
      const int one = quotient(rest, p.per_key_heads);
      part = item - rest * p.sink_parts, parts = p.sink_parts, kh = rest - one * p.key_heads;
      seq = quotient(one, p.per_sink_tiles), tile = one - seq * p.sink_tiles;
      s = seq_of(p, seq);
      if (tile * KR >= s.kl) return;
    }
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = threadIdx.x & 63, g = l >> 4, li = l & 15;
    const int t0 = tile * KR, row0 = t0 + wave * 16 * NCK;
    const int last = (t0 + KR < s.kl ? t0 + KR : s.kl) - 1, wlast = (row0 + 16 * NCK < s.kl ? row0 + 16 * NCK : s.kl) - 1;
    Frag k[NCK][NK], v[NCK][NK];
    own_rows<T, D, NCK>(k, static_cast<const T *>(p.k) + (int64_t)s.ks * p.ldk + kh * D, p.ldk, row0, s.kl);
    own_rows<T, D, NCK>(v, static_cast<const T *>(p.v) + (int64_t)s.ks * p.ldv + kh * D, p.ldv, row0, s.kl);
    // The queries that see key j: [x, y) in their window and, for a sink, all behind.
    const bool with_sinks = (sink_item || p.sink_parts == 0) && t0 < p.sinks;
    int lo[NCK], hi[NCK];
#pragma unroll
    for (int c = 0; c < NCK; ++c) {
      const int j = row0 + 16 * c + li;
      const int2 r = j < s.kl ? seeing_queries(p, s, j) : int2{0, 0};
      lo[c] = r.x, hi[c] = r.y;
    }
    const int2 ta = seeing_queries(p, s, t0), tb = seeing_queries(p, s, last);
    const int2 wa = row0 < s.kl ? seeing_queries(p, s, row0) : int2{0, 0}, wb = row0 < s.kl ? seeing_queries(p, s, wlast) : int2{0, 0};
    // a head's tiles: na over the window [ta.x, tb.y), nb over what is behind the first key's window [ta.y, ql)
    const int na = sink_item ? 0 : tiles_of(tb.y - ta.x, BQ), nb = with_sinks ? tiles_of(s.ql - ta.y, BQ) : 0, per = na + nb;
    const int total = per * grp, share = quotient(total + parts - 1, sink_item ? p.per_sink_parts : p.per_parts);
    const int first = part * share, end = first + share < total ? first + share : total;
    const typename Tile::Lane lane = Tile::lane();
    const typename Tile::template Copy<BQ> copy_q(p.ldq), copy_o(p.ldgo);
    struct Walk {                                       // over the heads' tiles
      int x, i, e;                                      // tile of the head, its rows [i, min(i + BQ, e))
      const T *q, *o;                                   // its first rows
      const float *lse, *del;
      __device__ __forceinline__ int end() const { return i + BQ < e ? i + BQ : e; }
    };
    const auto at = [&](int h, int x) {
      Walk w;
      w.x = x, w.i = x < na ? ta.x + x * BQ : ta.y + (x - na) * BQ, w.e = x < na ? tb.y : s.ql;
      const int64_t row = s.qs + w.i;
      w.q = static_cast<const T *>(p.q) + row * p.ldq + (kh * grp + h) * D;
      w.o = static_cast<const T *>(p.go) + row * p.ldgo + (kh * grp + h) * D;
      w.lse = p.lse + (int64_t)(kh * grp + h) * p.nq + row, w.del = p.delta + (int64_t)(kh * grp + h) * p.nq + row;
      return w;
    };
    const int64_t step_q = BQ * p.ldq, step_o = BQ * p.ldgo;
    const int h0 = per > 0 ? first / per : 0, x0 = first - h0 * per;
    const auto fetch = [&](const Walk &w, int stage) {
      const int n = w.end() - w.i;
      copy_q.fetch(w.q, n, s_a[stage]);
      copy_o.fetch(w.o, n, s_b[stage]);
      if (wave < 2)                                     // 64 values each (zeros behind the last)
        copy_to_lds_untracked<4>(untracked_view(wave ? w.del : w.lse, n * 4), l * 4,
                                 reinterpret_cast<unsigned char *>(wave ? s_del[stage] : s_lse[stage]));
    };
    const float c2 = p.scale * kLog2e;
    f32x4 dk[ND][NCK], dv[ND][NCK];
    for (int careful = 0; careful < 2; ++careful) {     // as in the forward, for q and do that are not finite
#pragma unroll
      for (int c = 0; c < NCK; ++c)
#pragma unroll
        for (int d = 0; d < ND; ++d) dk[d][c] = dv[d][c] = zero_f4();
      __syncthreads();
      int h = h0;
      Walk ahead = at(h, x0);
      if (first < end) fetch(ahead, first & 1);
      for (int t = first; t < end; ++t) {
        const int2 r{ahead.i, ahead.end()};
        const bool window = ahead.x < na;
        if (++ahead.x == na || ahead.x == per) {
          if (ahead.x == per) ++h, ahead.x = 0;
          ahead = at(h, ahead.x);
        } else {
          ahead.i += BQ, ahead.q += step_q, ahead.o += step_o, ahead.lse += BQ, ahead.del += BQ;
        }
        landed();
        if (t + 1 < end) fetch(ahead, (t + 1) & 1);
        // this wave's keys are seen by queries from .. to: by all of them [a, b), by any [x, y)
        int all_x, all_y, any_x, any_y;
        if (window) {
          all_x = wb.x, all_y = wa.y, any_x = wa.x, any_y = wb.y;
        } else {
          all_x = wlast < p.sinks ? wb.y : s.ql, all_y = s.ql, any_x = wa.y, any_y = row0 < p.sinks && row0 < s.kl ? s.ql : 0;
        }
        const bool full = r.y - r.x == BQ && all_x <= r.x && all_y >= r.y, none = row0 >= s.kl || !(any_x < r.y && any_y > r.x);
        unsigned char *qt = s_a[t & 1], *ot = s_b[t & 1];
        const int qa = Tile::offset(qt), oa = Tile::offset(ot);
        const float *lse = s_lse[t & 1], *del = s_del[t & 1];
#pragma unroll
        for (int x0 = 0; x0 < BQ; x0 += 32) {
          Frag pr[NCK], ds[NCK];
          if (!none) {
            f32x4 sc[2][NCK], dp[2][NCK];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
#pragma unroll
              for (int c = 0; c < NCK; ++c) sc[u][c] = dp[u][c] = zero_f4();
#pragma unroll
              for (int x = 0; x < NK; ++x) {
                const Frag a = Tile::rows(qa, lane, x0 + 16 * u, x), b = Tile::rows(oa, lane, x0 + 16 * u, x);
#pragma unroll
                for (int c = 0; c < NCK; ++c) {
                  sc[u][c] = mma(a, k[c][x], sc[u][c]);
                  dp[u][c] = mma(b, v[c][x], dp[u][c]);
                }
                if (D == 256 && x % 2 == 1) __builtin_amdgcn_sched_barrier(0);
              }
              const f32x4 l4 = *reinterpret_cast<const f32x4 *>(lse + x0 + 16 * u + 4 * g) * kLog2e;
              const f32x4 d4 = *reinterpret_cast<const f32x4 *>(del + x0 + 16 * u + 4 * g);
#pragma unroll
              for (int c = 0; c < NCK; ++c)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                  sc[u][c][x] = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[u][c][x], c2, -l4[x]));
                  dp[u][c][x] = sc[u][c][x] * (dp[u][c][x] - d4[x]);
                }
            }
            if (!full) {                                // the queries [first, e) see column c
              rarely();
#pragma unroll
              for (int c = 0; c < NCK; ++c) {
                const int j = row0 + 16 * c + li;
                const int first = window ? lo[c] : ((j < p.sinks) & (j < s.kl)) ? hi[c] : s.ql, e = window ? (hi[c] < r.y ? hi[c] : r.y) : r.y;
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                  for (int x = 0; x < 4; ++x) {
                    const int i = r.x + x0 + 16 * u + 4 * g + x;
                    const bool sees = (i >= first) & (i < e);
                    sc[u][c][x] = sees ? sc[u][c][x] : 0.0f, dp[u][c][x] = sees ? dp[u][c][x] : 0.0f;
                  }
              }
            }
#pragma unroll
            for (int c = 0; c < NCK; ++c) pr[c] = pack44<T>(sc[0][c], sc[1][c]), ds[c] = pack44<T>(dp[0][c], dp[1][c]);
          }
          if (careful && !(r.y - r.x == BQ && (window ? tb.x <= r.x && ta.y >= r.y : last < p.sinks && tb.y <= r.x))) {
            if (!none)
              for (int x = x0; x < x0 + 32; ++x) {
                const int i = r.x + x;
#pragma unroll
                for (int d = 0; d < ND; ++d)
#pragma unroll
                  for (int y = 0; y < 4; ++y) {
                    const float f = to_f32(*reinterpret_cast<const T *>(ot + Tile::elem(x, 16 * d + 4 * g + y)));
                    if (fabsf(f) < __builtin_inff()) continue;
#pragma unroll
                    for (int c = 0; c < NCK; ++c) {
                      const int j = row0 + 16 * c + li;
                      if (i < r.y && (window ? i >= lo[c] && i < hi[c] : i >= hi[c] && j < p.sinks && j < s.kl)) dv[d][c][y] += f;
                    }
                  }
              }
            __syncthreads();
            Tile::settle(qt, x0, 32);
            Tile::settle(ot, x0, 32);
            __syncthreads();
          }
          if (!none) {
#pragma unroll
            for (int d = 0; d < ND; ++d) {
              const Frag a = Tile::cols(oa, lane, x0, d), b = Tile::cols(qa, lane, x0, d);
#pragma unroll
              for (int c = 0; c < NCK; ++c) {
                dv[d][c] = mma(a, pr[c], dv[d][c]);
                dk[d][c] = mma(b, ds[c], dk[d][c]);
              }
              // (wide heads: operands that are all read ahead would take the registers of the second wave)
              if (D == 256 && d % 2 == 1) __builtin_amdgcn_sched_barrier(0);
            }
          }
        }
      }
      bool odd = false;
#pragma unroll
      for (int c = 0; c < NCK; ++c)
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
          for (int x = 0; x < 4; ++x) odd |= !(fabsf(dk[d][c][x]) + fabsf(dv[d][c][x]) < __builtin_inff());
      if (!__syncthreads_or(odd)) break;
    }
    const bool apart = p.sink_parts > 0 && tile < p.sink_tiles;       // this tile's sinks are other items' work
#pragma unroll
    for (int c = 0; c < NCK; ++c) {
      const int j = row0 + 16 * c + li;
      if (j >= s.kl) continue;
      const int64_t row = s.ks + j;
      if (!sink_item && p.parts == 1 && !apart) {
        T *ok = static_cast<T *>(p.gk) + row * p.ldgk + kh * D + 4 * g, *ov = static_cast<T *>(p.gv) + row * p.ldgv + kh * D + 4 * g;
#pragma unroll
        for (int d = 0; d < ND; ++d) store4(ok + 16 * d, dk[d][c] * p.scale), store4(ov + 16 * d, dv[d][c]);
        continue;
      }
      if (sink_item && j >= p.sinks) continue;
      float *out;
      if (sink_item || p.parts == 1)
        out = p.spart + (((((int64_t)seq * p.sink_tiles + tile) * p.key_heads + kh) * (1 + p.sink_parts) + (sink_item ? 1 + part : 0)) * KR +
                         (j - t0)) * 2 * D;
      else
        out = p.part + (((int64_t)part * p.nk + row) * p.key_heads + kh) * 2 * D;
#pragma unroll
      for (int d = 0; d < ND; ++d)
        store4(out + 16 * d + 4 * g, dk[d][c] * p.scale), store4(out + D + 16 * d + 4 * g, dv[d][c]);
    }
  } else {
    constexpr int QR = 64 * NCQ;
    const int item = attn_item(blockIdx.x - keys, p.qtiles * p.heads * p.qparts);
    const int rest = p.qparts > 1 ? quotient(item, p.per_qparts) : item, part = item - rest * p.qparts;
    const int h = quotient(rest, p.per_qtiles), kh = quotient(h, p.group);
    AttnSeq s;
    int tile, seq;
    if (!tile_of<false>(p, p.qtiles - 1 - (rest - h * p.qtiles), &s, &tile, &seq)) return;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = threadIdx.x & 63, g = l >> 4, li = l & 15;
    const int t0 = tile * QR, row0 = t0 + wave * 16 * NCQ;
    const T *kb = static_cast<const T *>(p.k) + (int64_t)s.ks * p.ldk + kh * D;
    const T *vb = static_cast<const T *>(p.v) + (int64_t)s.ks * p.ldv + kh * D;
    Frag q[NCQ][NK], go[NCQ][NK];
    own_rows<T, D, NCQ>(q, static_cast<const T *>(p.q) + (int64_t)s.qs * p.ldq + h * D, p.ldq, row0, s.ql);
    own_rows<T, D, NCQ>(go, static_cast<const T *>(p.go) + (int64_t)s.qs * p.ldgo + h * D, p.ldgo, row0, s.ql);
    int lo[NCQ], hi[NCQ];
    float lse[NCQ], delta[NCQ];
#pragma unroll
    for (int c = 0; c < NCQ; ++c) {
      const int i = row0 + 16 * c + li;
      const bool in = i < s.ql;
      const int2 r = in ? seen_keys(p, s, i) : int2{0, 0};
      lo[c] = r.x, hi[c] = r.y;
      const int64_t at = (int64_t)h * p.nq + s.qs + i;
      lse[c] = in ? p.lse[at] * -kLog2e : -__builtin_inff();
      delta[c] = in ? p.delta[at] : 0.0f;
    }
    const int last = t0 + QR < s.ql ? t0 + QR : s.ql, wlast = row0 + 16 * NCQ < s.ql ? row0 + 16 * NCQ : s.ql;
    const int k0 = seen_keys(p, s, t0).x, k1 = seen_keys(p, s, last - 1).y, se = p.sinks < k0 ? p.sinks : k0;
    const int2 wa = row0 < s.ql ? seen_keys(p, s, row0) : int2{0, 0}, wb = row0 < s.ql ? seen_keys(p, s, wlast - 1) : int2{0, 0};
    const int ns = tiles_of(se, BK), nt = ns + tiles_of(k1 - k0, BK);
    const int share = p.qparts > 1 ? quotient(nt + p.qparts - 1, p.per_qparts) : nt, first = part * share;
    const int count = first + share < nt ? share : nt - first;                // of its tiles (below 1: none)
    const typename Tile::Lane lane = Tile::lane();
    const typename Tile::template Copy<BK> copy_k(p.ldk), copy_v(p.ldv);
    const KeyWalk<T, BK> start(first, ns, se, k0, k1, kb, vb, p.ldk, p.ldv);
    const auto fetch = [&](const KeyWalk<T, BK> &w, int stage) {
      copy_k.fetch(w.k, w.end() - w.j, s_a[stage]);
      copy_v.fetch(w.v, w.end() - w.j, s_b[stage]);
    };
    const float c2 = p.scale * kLog2e;
    f32x4 dq[ND][NCQ];
    for (int careful = 0; careful < 2; ++careful) {     // as in the forward, for k that is not finite
#pragma unroll
      for (int c = 0; c < NCQ; ++c)
#pragma unroll
        for (int d = 0; d < ND; ++d) dq[d][c] = zero_f4();
      __syncthreads();
      KeyWalk<T, BK> ahead = start;
      if (count > 0) fetch(ahead, 0);
      for (int t = 0; t < count; ++t) {
        const int2 r{ahead.j, ahead.end()};
        ahead.next();
        landed();
        if (t + 1 < count) fetch(ahead, (t + 1) & 1);
        const bool full = r.y - r.x == BK && wa.y >= r.y && (wb.x <= r.x || r.y <= p.sinks);
        const bool none = !(r.x < wb.y && (r.y > wa.x || r.x < p.sinks));
        unsigned char *kt = s_a[t & 1];
        const int ka = Tile::offset(kt), va = Tile::offset(s_b[t & 1]);
#pragma unroll
        for (int x0 = 0; x0 < BK; x0 += 32) {
          Frag ds[NCQ];
          if (!none) {
            f32x4 sc[2][NCQ], dp[2][NCQ];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
#pragma unroll
              for (int c = 0; c < NCQ; ++c) sc[u][c] = dp[u][c] = zero_f4();
#pragma unroll
              for (int k = 0; k < NK; ++k) {
                const Frag a = Tile::rows(ka, lane, x0 + 16 * u, k), b = Tile::rows(va, lane, x0 + 16 * u, k);
#pragma unroll
                for (int c = 0; c < NCQ; ++c) {
                  sc[u][c] = mma(a, q[c][k], sc[u][c]);
                  dp[u][c] = mma(b, go[c][k], dp[u][c]);
                }
              }
            }
#pragma unroll
            for (int c = 0; c < NCQ; ++c) {
              const int e = hi[c] < r.y ? hi[c] : r.y;
#pragma unroll
              for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                  const float pr = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[u][c][x], c2, lse[c]));
                  sc[u][c][x] = pr * (dp[u][c][x] - delta[c]);
                }
              if (!full) {
                rarely();
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                  for (int x = 0; x < 4; ++x) {
                    const int j = r.x + x0 + 16 * u + 4 * g + x;
                    sc[u][c][x] = ((j < e) & ((j >= lo[c]) | (j < p.sinks))) ? sc[u][c][x] : 0.0f;
                  }
              }
              ds[c] = pack44<T>(sc[0][c], sc[1][c]);
            }
          }
          if (careful) {
            const bool whole = r.y - r.x == BK && seen_keys(p, s, t0).y >= r.y && (seen_keys(p, s, last - 1).x <= r.x || r.y <= p.sinks);
            if (!whole) {
              __syncthreads();
              Tile::settle(kt, x0, 32);
              __syncthreads();
            }
          }
          if (!none) {
#pragma unroll
            for (int d = 0; d < ND; ++d) {
              const Frag a = Tile::cols(ka, lane, x0, d);
#pragma unroll
              for (int c = 0; c < NCQ; ++c) dq[d][c] = mma(a, ds[c], dq[d][c]);
            }
          }
        }
      }
      bool odd = false;
#pragma unroll
      for (int c = 0; c < NCQ; ++c)
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
          for (int x = 0; x < 4; ++x) odd |= !(fabsf(dq[d][c][x]) < __builtin_inff());
      if (!__syncthreads_or(odd)) break;
    }
#pragma unroll
    for (int c = 0; c < NCQ; ++c) {
      const int i = row0 + 16 * c + li;
      if (i >= s.ql) continue;
      if (p.qparts > 1) {
        float *out = p.qpart + (((int64_t)part * p.nq + s.qs + i) * p.heads + h) * D + 4 * g;
#pragma unroll
        for (int d = 0; d < ND; ++d) store4(out + 16 * d, dq[d][c] * p.scale);
        continue;
      }
      T *out = static_cast<T *>(p.gq) + (int64_t)(s.qs + i) * p.ldgq + h * D + 4 * g;
#pragma unroll
      for (int d = 0; d < ND; ++d) store4(out + 16 * d, dq[d][c] * p.scale);
    }
  }
}

// The sums over ranges, in their order.  The first `keys` workgroups those of queries: a key tile (of sinks only, where the window
// is one range) and key head, 512 / D of its rows, D / 2 lanes a row; behind them those of keys: a query tile, 1024 / D of its
// rows, D / 4 lanes a row.
template <typename T, int D> __global__ __launch_bounds__(256) void attn_sum_kernel(AttnParams p, int keys) {
  if ((int)blockIdx.x >= keys) {
    constexpr int L = D / 4;
    const int b = blockIdx.x - keys, per = p.qrows * D / 1024, item = b >> __builtin_ctz(per), y = b & (per - 1);
    const int h = quotient(item, p.per_qtiles);
    AttnSeq s;
    int tile, seq;
    if (!tile_of<false>(p, p.qtiles - 1 - (item - h * p.qtiles), &s, &tile, &seq)) return;
    const int c = threadIdx.x % L * 4, r = y * (256 / L) + threadIdx.x / L;
    if (tile * p.qrows + r >= s.ql) return;
    const int64_t row = s.qs + tile * p.qrows + r, step = (int64_t)p.nq * p.heads * D;
    const float *a = p.qpart + (row * p.heads + h) * D + c;
    f32x4 v = zero_f4();
#pragma unroll 4
    for (int i = 0; i < p.qparts; ++i) v += *reinterpret_cast<const f32x4 *>(a + i * step);
    store4(static_cast<T *>(p.gq) + row * p.ldgq + h * D + c, v);
    return;
  }
  constexpr int L = D / 2;
  const int per = p.krows * D / 512, bx = blockIdx.x >> __builtin_ctz(per), by = blockIdx.x & (per - 1);      // (a power of two)
  AttnSeq s;
  int tile, seq;
  const int x = quotient(bx, p.per_key_heads), kh = bx - x * p.key_heads;
  if (p.parts > 1) {
    if (!tile_of<true>(p, x, &s, &tile, &seq)) return;
  } else {
    seq = quotient(x, p.per_sink_tiles), tile = x - seq * p.sink_tiles;
    s = seq_of(p, seq);
  }
  const int c = threadIdx.x % L * 4, r = by * (256 / L) + threadIdx.x / L;
  if (tile * p.krows + r >= s.kl) return;
  const int64_t row = s.ks + tile * p.krows + r;
  f32x4 v = zero_f4();
  const float *a = p.part + (row * p.key_heads + kh) * 2 * D + c;
  const int64_t step = (int64_t)p.nk * p.key_heads * 2 * D;
  if (p.parts > 1)
#pragma unroll 4
    for (int i = 0; i < p.parts; ++i) v += *reinterpret_cast<const f32x4 *>(a + i * step);
  if (p.sink_parts > 0 && tile < p.sink_tiles) {
    const float *b = p.spart + (((((int64_t)seq * p.sink_tiles + tile) * p.key_heads + kh) * (1 + p.sink_parts)) * p.krows + r) * 2 * D + c;
    const int64_t next = (int64_t)p.krows * 2 * D;
#pragma unroll 4
    for (int i = p.parts > 1 ? 1 : 0; i <= (tile * p.krows + r < p.sinks ? p.sink_parts : 0); ++i)
      v += *reinterpret_cast<const f32x4 *>(b + i * next);
  }
  if (c < D)
    store4(static_cast<T *>(p.gk) + row * p.ldgk + kh * D + c, v);
  else
    store4(static_cast<T *>(p.gv) + row * p.ldgv + kh * D + c - D, v);
}

template <typename T, int D, int NCQ, int BK, int NCK, int BQ, int OCC> hipError_t go(const AttnParams &p, hipStream_t s) {
  const int blocks = (int)(((int64_t)p.nq * p.heads + 2048 / D - 1) / (2048 / D));
  if (blocks > 0 || p.cu_q) {
    hipLaunchKernelGGL((attn_delta_kernel<T, D>), dim3(blocks + (p.cu_q ? kZeroBlocks : 0)), dim3(256), 0, s, p, blocks);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const int sinks = p.nseq * p.sink_tiles * p.key_heads, tiles = p.qtiles * p.heads;
  const int keys = p.ktiles * p.key_heads * p.parts + sinks * p.sink_parts, queries = tiles * p.qparts;
  if (queries + keys > 0) hipLaunchKernelGGL((attn_grads_kernel<T, D, NCQ, BK, NCK, BQ, OCC>), dim3(queries + keys), dim3(256), 0, s, p, keys);
  const hipError_t e = hipGetLastError();
  const int key_sums = (p.parts > 1 ? p.ktiles * p.key_heads : p.sink_parts > 0 ? sinks : 0) * (p.krows * D / 512);
  const int sums = key_sums + (p.qparts > 1 ? tiles * (p.qrows * D / 1024) : 0);
  if (e != hipSuccess || sums == 0) return e;
  hipLaunchKernelGGL((attn_sum_kernel<T, D>), dim3(sums), dim3(256), 0, s, p, key_sums);
  return hipGetLastError();
}

}  // namespace

// Ranges that the queries of a key tile (all heads of its key head) and the keys of a query tile are cut in, each a workgroup
// of its own whose sums are written and added (2.5 TB/s together, 6 us the launch): as many as bring the longest workgroup
// down to what all keep the 256 CUs busy with.  Times of 32 rows of the other axis for a tile of 64 of its own on a CU
// alone, and how many such a CU does at once, are measured; a larger tile takes less than in proportion and dq three
// quarters of dk and dv.  fp32, 2 heads of 256 on 1, 1974 tokens in 5 sequences: 755 us uncut, 298 with the queries cut, 221
// with both; bf16, 2 heads of 128 on 1, 2048 tokens, causal: 89 with the queries cut, 42 with both.  Where all take longer
// than the longest they even out by themselves (8192 tokens, 8 heads of 64: 527 us, 559 cut).
AttnGradCut attn_grad_cut(const AttnGradWork &w, int d, bool bf16, int qrows, int krows) {
  const double key = (bf16 ? (d == 64 ? 0.7 : d == 128 ? 1.1 : 2.1) : d == 64 ? 3.0 : d == 128 ? 4.7 : 9.3) * std::pow(krows / 64.0, 0.8) / 32;
  const double query = 0.75 * key * std::pow((double)qrows / krows, 0.8);
  const double at_once = bf16 ? (d == 64 ? 3.0 : d == 128 ? 2.0 : 1.2) : d == 64 ? 1.5 : d == 128 ? 1.3 : 1.15;
  const double mean = (w.key_items * w.mean_queries * key + w.query_items * w.mean_keys * query) / (256 * at_once);
  const double key_sum = w.key_tiles * (double)krows * 2 * d * 4 / 2.5e6, query_sum = w.query_tiles * (double)qrows * d * 4 / 2.5e6;
  static constexpr int kRanges[] = {1, 2, 3, 4, 5, 6, 8, 10, 12, 16, 20, 24, 32};
  AttnGradCut best{1, 1};
  if (std::max((double)w.queries * key, (double)w.keys * query) <= mean) return best;
  double least = 0.0;
  for (const int q : kRanges) {
    if (q > 1 && w.keys / q < 32) break;
    int before = 0;
    for (const int k : kRanges) {
      if (k > 1 && before >= w.query_steps) break;      // (more ranges than steps: some of nothing)
      before = k;
      const double longest = std::max((double)w.queries / k * key, (double)w.keys / q * query);
      const double t = (w.key_items * k + w.query_items * q > 256 ? std::max(longest, mean + longest / 2) : longest) +
                       (k > 1 || q > 1 ? 6.0 : 0.0) + (k > 1 ? k * key_sum : 0.0) + (q > 1 ? q * query_sum : 0.0);
      if (k * q == 1 || t < 0.97 * least) least = t, best = AttnGradCut{k, q};
    }
  }
  return best;
}

int attn_grad_query_rows(int d, bool bf16, bool small) { return small || (!bf16 && d >= 128) ? 64 : 128; }
int attn_grad_key_rows(int d, bool bf16, bool small) { return small || d >= 128 ? 64 : 128; }

hipError_t launch_attention_backward(const AttnParams &p, bool bf16, hipStream_t s) {
  const hipError_t e = launch_attention_plan(p, s);
  if (e != hipSuccess) return e;
  // Tiles of two columns of 16 rows a wave read LDS half as often, and where they leave few workgroups one column does (256:
  // 2048 tokens of 4 heads 214 us against 251, 8192 tokens 1939 against 1717).  The occupancies leave the vector registers in
  // place, but for 4 of bf16 256 in its tiles of 128 queries.  Scalar registers are short, as both kinds of work share a kernel
  // and its arguments: 82 to 146 of them are kept elsewhere (lanes of vector registers; bf16 128, and fp32 64 in tiles of 128,
  // have 68 bytes of scratch a lane).
  if (bf16) {
    if (p.d == 64) return p.krows == 64 ? go<__bf16, 64, 1, 64, 1, 64, 4>(p, s) : go<__bf16, 64, 2, 64, 2, 64, 2>(p, s);
    if (p.d == 128) return go<__bf16, 128, 2, 32, 1, 32, 2>(p, s);
    return p.qrows == 64 ? go<__bf16, 256, 1, 32, 1, 32, 1>(p, s) : go<__bf16, 256, 2, 32, 1, 32, 1>(p, s);
  }
  if (p.d == 64) return p.krows == 64 ? go<float, 64, 1, 32, 1, 32, 3>(p, s) : go<float, 64, 2, 32, 2, 32, 2>(p, s);
  return p.d == 128 ? go<float, 128, 1, 32, 1, 32, 2>(p, s) : go<float, 256, 1, 32, 1, 32, 1>(p, s);
}

}  // namespace ttt
