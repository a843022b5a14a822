// Gradient of the chunked gated delta rule (notation of delta.hip; G = gradient of the state
// after the chunk, go = gradient of O).  The forward's chunk terms, states and U are computed
// again, then, in reverse order of the chunks,
//   dU = A^T go + el o (K G^T),   dR = T^T dU,   dP = -beta eg o dR
//   G before the chunk = e^gamma_last G + scale (eg o go)^T Q + dP^T K
// and, for all chunks at once, with X = scale (go U^T) o D and Y = -beta o (dR U^T) o D (j < i),
//   dq = scale eg o (go W0) + X K
//   dk = -beta eg o (dR W0) + el o (U G) + X^T Q + (Y + Y^T) K
//   dv = beta o dR
//   dbeta_i = dR_i.(V - eg o P)_i + sum_j Y_ij k_i.k_j / beta_i
//   dgamma_i = q_i.(first term of dq)_i + k_i.(first of dk)_i - k_i.(second of dk)_i
//              + rowsum_i(M) - colsum_i(M),  M = X o Q K^T + Y o K K^T,
//   dgamma_last += e^gamma_last <W0, G> + sum_j k_j.(second of dk)_j,   dg_i = sum_{j >= i} dgamma_j
// (k_i.(dR W0)_i is dR_i.P_i, so P itself is not needed).
#include "delta_state.h"

namespace ttt {
namespace {

// ------------------------------------------------------------------ state gradients
// The reverse of the states kernel, with the same split, layout, waves and order of loads:
//   rows: K G^T, dU        rows: dR = T^T dU;  state: G <- e^gamma_last G + (scale eg o go)^T Q
//   state: G += dP^T K;  rows: the next chunk's go
// Segments of few long sequences (see there) run at once here too: G before a segment is G after it times
// M^T plus what the segment alone has.  kFirst: the last segment, and the others but the first from G = 0;
// kSecond: all but the last, over what the first launch wrote for their rows.
template <typename T, int DK, int PART> struct GradLds {
  SplitTile<kFull, SL, DK> g[PART == kSecond ? 2 : 1];
  SplitTile<kFull, SL, C> goe[2], du, dr, dp;
  SplitTile<kTok<T>, SL, C> go;
};
template <typename T, int DK, int PART>
__device__ __forceinline__ void delta_gstates(const DeltaParams &p, GradLds<T, DK, PART> &lds, int id, int count) {
  constexpr int NT = DK / 64, NK = DK / 32, TP = kTok<T>;
  auto &s_gs = lds.g;
  auto &s_goe = lds.goe;
  auto &s_du = lds.du, &s_dr = lds.dr, &s_dp = lds.dp;
  auto &s_go = lds.go;
  constexpr int64_t tokens = DK * C * 2 * TP, tplane = DK * C * 2;      // bytes of a chunk's tokens and a part
  const int slices = p.dv / SL, item = xcd_item(id, count);
  SplitTile<kFull, SL, DK> &s_g = s_gs[0];
  const int all = PART == kWhole ? slices : (p.segs - 1) * slices;
  const int sl = item % slices, bh = item / all, h = bh % p.heads, b = bh / p.heads;
  const int wave = wave_id(), w = wave & 3, l = threadIdx.x & 63, g = l >> 4, li = l & 15;
  const int kh = h / (p.heads / p.key_heads);
  const DeltaSeq sq = seq_of(p, b);
  const int chunks = (sq.len + C - 1) / C;
  int seg = item % all / slices, c_first = 0, c_end = chunks;
  bool live = true;                     // its gradients are the sequence's
  if constexpr (PART != kWhole) {
    const int per = (chunks + p.segs - 1) / p.segs, last = chunks > 0 ? (chunks - 1) / per : 0;
    if constexpr (PART == kFirst) {
      if (last > 0) ++seg;              // (the only segment is the first launch's)
      if (seg > last) return;
      live = seg == last;
    } else {
      if (seg >= last) return;
    }
    c_first = seg * per, c_end = c_first + per < chunks ? c_first + per : chunks;
    if constexpr (PART == kSecond)
      join_segments<DK>(
          s_gs, last - seg,
          [&](int j) { return p.seg_g + (((int64_t)(b * (p.segs - 1) + last - j - 1) * p.heads + h) * p.dv + sl * SL + li) * DK + 4 * g; },
          [&](int j) {
            // (no M is read for the first step; its index then is one that exists)
            return p.seg_m + ((int64_t)(b * (p.segs - 2) + (last - j > 0 ? last - j : 1) - 1) * p.heads + h) * (DK * DK * 4 * kFull) +
                   DK * DK * 2 * kFull;
          });
  }
  const int64_t ch0 = (int64_t)sq.chunk0 * p.heads + h, ck0 = (int64_t)sq.chunk0 * p.key_heads + kh;
  const int64_t plane = C * C * 2;
  if (wave < 4) {
    const int t4 = 16 * w + 4 * g;
    Split<TP> kf[NK];
    Split<kFull> tf[2], af[2];
    T gv[4];
    f32x4 be, eg, el;
    const Rows4<T> go_rows(t4, li, p.ldgo), gv_rows(t4, li, p.ldgv);
    const auto load_token = [&](int c, int i) {
      return load_frag<TP>(p.kp + (ck0 + (int64_t)c * p.key_heads) * tokens, tplane, w * NK + i);
    };
    const auto load_values = [&](int c) {
      const int64_t o = (ch0 + (int64_t)c * p.heads) * C + t4;
      eg = *reinterpret_cast<const f32x4 *>(p.eg + o);
      el = *reinterpret_cast<const f32x4 *>(p.el + o);
      be = *reinterpret_cast<const f32x4 *>(p.be + o);
      go_rows.load(static_cast<const T *>(p.go) + ((int64_t)sq.start + c * C) * p.ldgo + h * p.dv + sl * SL, t4,
                   sq.len - c * C, gv);
    };
    // the chunk's go, 0 past its end, to LDS (as it is, and as the state's update takes it)
    const auto store_go = [&](int c, int buf) {
      f32x4 go;
#pragma unroll
      for (int r = 0; r < 4; ++r) go[r] = c * C + t4 + r < sq.len ? to_f32(gv[r]) : 0.0f;
      s_go.st4(li, t4, go);
      s_goe[buf].st4(li, t4, go * eg * p.scale);
    };
    const auto load_square = [&](const char *m, int c, Split<kFull> (&f)[2]) {
#pragma unroll
      for (int i = 0; i < 2; ++i)       // (the first half is zero for the last two waves)
        f[i] = load_frag<kFull>(m + (ch0 + (int64_t)c * p.heads) * kSquare, plane, w * 2 + i);
    };
    if (c_first < c_end) {
#pragma unroll
      for (int i = 0; i < NK; ++i) kf[i] = load_token(c_end - 1, i);
      load_values(c_end - 1);
      load_square(p.am, c_end - 1, af);
      load_square(p.tt, c_end - 1, tf);
      store_go(c_end - 1, (c_end - 1) & 1);
    }
    lds_barrier();
    for (int c = c_end - 1; c >= c_first; --c) {
      const int nx = c > c_first ? c - 1 : c, left = sq.len - c * C;
      Sums<kFull> kg;
#pragma unroll
      for (int i = 0; i < NK; ++i) {
        kg.add(kf[i], s_g.ld(li, 32 * i + 8 * g));
        kf[i] = load_token(nx, i);
      }
      f32x4 du = kg.sum();
#pragma unroll
      for (int r = 0; r < 4; ++r) du[r] = t4 + r < left ? du[r] * el[r] : 0.0f;
      Sums<kFull> ag;
      if (w < 2) ag.add(af[0], s_go.ld(li, 8 * g));
      ag.add(af[1], s_go.ld(li, 32 + 8 * g));
      load_square(p.am, nx, af);
      s_du.st4(li, t4, du + ag.sum());
      lds_barrier();
      Sums<kFull> td;
      if (w < 2) td.add(tf[0], s_du.ld(li, 8 * g));
      td.add(tf[1], s_du.ld(li, 32 + 8 * g));
      const f32x4 dr = td.sum();
      load_square(p.tt, nx, tf);
      s_dp.st4(li, t4, dr * be * eg * -1.0f);
      s_dr.st4(li, t4, dr);
      const f32x4 dv = be * dr;
      load_values(nx);
      lds_barrier();
      gv_rows.store(static_cast<T *>(p.gv) + ((int64_t)sq.start + c * C) * p.ldgv + h * p.dv + sl * SL, t4, left, dv);
      s_dr.copy_t4(0, 16 * w, p.dr + (ch0 + (int64_t)c * p.heads) * (C * p.dv * 2 * kFull), (int64_t)C * p.dv * 2,
                   frag_at(16 * w + li, sl * SL + 4 * g, p.dv / 32));
      store_go(nx, ~c & 1);
      lds_barrier();
    }
  } else {
    const int64_t wrow = (((int64_t)b * p.heads + h) * p.dv + sl * SL + li) * DK + w * (DK / 4) + 4 * g;
    f32x4 st[NT];
    Split<TP> ktf[NT][2], qtf[NT][2];
    // fp32 tokens of 256: K^T follows Q^T through the same registers (held side by side they spill)
    constexpr bool kShare = TP == 3 && DK == 256;
    float ec = 0.0f;
    const auto load_transposed = [&](const char *m, int c, int i, int x) {
      return load_frag<TP>(m + (ck0 + (int64_t)c * p.key_heads) * tokens, tplane, (w * NT + i) * 2 + x);
    };
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int col = (w * NT + i) * 16 + 4 * g;
      if constexpr (PART == kSecond) {
        st[i] = s_g.at4(li, col);
      } else {
        st[i] = live && p.gw_out ? *reinterpret_cast<const f32x4 *>(p.gw_out + wrow + 16 * i) : zero4();
        s_g.st4(li, col, st[i]);
      }
    }
    if (c_first < c_end) {
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          qtf[i][x] = load_transposed(p.qt, c_end - 1, i, x);
          if (!kShare) ktf[i][x] = load_transposed(p.kt, c_end - 1, i, x);
        }
      ec = p.eg[(ch0 + (int64_t)(c_end - 1) * p.heads) * C + C - 1];
    }
    lds_barrier();
    for (int c = c_end - 1; c >= c_first; --c) {
      const int nx = c > c_first ? c - 1 : c;
      {                                 // the gradient after the chunk, dk x dv
        float *o = p.gwt + (ch0 + (int64_t)c * p.heads) * (DK * p.dv);
#pragma unroll
        for (int i = 0; i < NT; ++i)
          s_g.copy_t4(0, (w * NT + i) * 16, o + frag_at((w * NT + i) * 16 + li, sl * SL + 4 * g, p.dv / 32));
      }
      {
        const Split<kFull> g0 = s_goe[c & 1].ld(li, 8 * g), g1 = s_goe[c & 1].ld(li, 32 + 8 * g);
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          Sums<kFull> d;
          d.add(qtf[i][0], g0);
          d.add(qtf[i][1], g1);
          st[i] = st[i] * ec + d.sum();
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            if constexpr (kShare) ktf[i][x] = load_transposed(p.kt, c, i, x);
            else qtf[i][x] = load_transposed(p.qt, nx, i, x);
          }
        }
        ec = p.eg[(ch0 + (int64_t)nx * p.heads) * C + C - 1];
      }
      lds_barrier();
      lds_barrier();
      const Split<kFull> p0 = s_dp.ld(li, 8 * g), p1 = s_dp.ld(li, 32 + 8 * g);
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        Sums<kFull> d;
        d.add(ktf[i][0], p0);
        d.add(ktf[i][1], p1);
        st[i] += d.sum();
        s_g.st4(li, (w * NT + i) * 16 + 4 * g, st[i]);
      }
      lds_barrier();
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if constexpr (kShare) qtf[i][x] = load_transposed(p.qt, nx, i, x);
          else ktf[i][x] = load_transposed(p.kt, nx, i, x);
        }
    }
    float *o = p.gw + wrow;
    if (PART == kFirst && seg > 0)
      o = p.seg_g + (((int64_t)(b * (p.segs - 1) + seg - 1) * p.heads + h) * p.dv + sl * SL + li) * DK + w * (DK / 4) + 4 * g;
    if (PART != kSecond || seg == 0)
#pragma unroll
      for (int i = 0; i < NT; ++i) *reinterpret_cast<f32x4 *>(o + 16 * i) = st[i];
  }
}

// The states and their gradients do not depend on one another (but for M, which the first launch leaves to the
// second): one launch for both, the gradients' workgroups, which take longer, first.  8 sequences of 16
// chunks, 6 heads of 128: 110 us for 768 workgroups, two to a CU (132 one after the other); 6 ragged
// sequences, 4 heads of 64, fp32: 69 (86).  fp32 heads of 256 whole take all 256 registers and spill 2.
template <typename T, int DK, int PART>
__global__ __launch_bounds__(512, sizeof(T) == 2 && DK <= 128 ? 4 : 2) void delta_chain_kernel(DeltaParams p, int grads) {
  union Lds {
    StateLds<T, DK, true> states;
    GradLds<T, DK, PART> grads;
  };
  __shared__ __attribute__((aligned(16))) Lds lds;
  const int id = blockIdx.x;
  if (id < grads) delta_gstates<T, DK, PART>(p, lds.grads, id, grads);
  else delta_states<T, DK, true, PART>(p, lds.states, id - grads, gridDim.x - grads);
}

// ------------------------------------------------------------------ token gradients
// One workgroup of eight waves per chunk and head.  First the 64 x 64 matrices X and Y (wave w has
// row tile w % 4 and half of the column tiles), which pass through LDS and are read both ways round,
// then dq and dk: wave w has the rows of half w / 4 and every fourth 16-wide column tile.  Operands
// come from memory in fragment order; bound by their latency, so registers are kept few enough for
// four waves a SIMD (one wave of 4 x 2 tiles a SIMD took 175 us where this takes 123 for 128 chunks
// of 6 heads of 128; of that its 278 MB are 55 us at a copy's rate, the products 15 and the vector
// operations 30.  Two column tiles at once, two fifths fewer operand loads, took as long).
template <typename T, int DK>
__global__ __launch_bounds__(512, sizeof(T) == 2 ? 4 : 2) void delta_gtoken_kernel(DeltaParams p) {
  constexpr int NT = DK / 64, TP = kTok<T>;
  __shared__ __attribute__((aligned(16))) SplitTile<kFull, C, C> s_xt, s_yt;      // X^T, Y^T
  __shared__ __attribute__((aligned(16))) float s_row[3][4][C];      // partials of q.(go W0), k.(dR W0), k.(U G)
  __shared__ float s_rs[2][C], s_db[2][C], s_cs[4][C], s_red[4], s_be[C];
  __shared__ float2 s_gam[C];
  const int item = xcd_item(blockIdx.x, gridDim.x), h = item % p.heads, c = item / p.heads;
  const DeltaChunk ck = chunk_of(p, c);
  if (ck.len == 0) return;
  const int t = threadIdx.x, wave = wave_id(), w4 = wave & 3, half = wave >> 2, l = t & 63, g = l >> 4, li = l & 15;
  const int kh = h / (p.heads / p.key_heads);
  const int64_t ch = (int64_t)c * p.heads + h;
  const int last = ck.len - 1, nv = p.dv / 32;
  const int64_t to = ((int64_t)c * p.key_heads + kh) * (DK * C * 2 * TP);
  constexpr int64_t tplane = DK * C * 2;
  const char *K = p.kp + to, *Q = p.qp + to, *KT = p.kt + to, *QT = p.qt + to;
  const T *V = static_cast<const T *>(p.v) + (int64_t)ck.tok0 * p.ldv + h * p.dv;
  const int64_t up = (int64_t)C * p.dv * 2;
  const char *GO = p.gop + ch * up * TP, *U = p.u + ch * up * kFull, *DR = p.dr + ch * up * kFull;

  if (t < C) {
    s_gam[t] = p.gam[ch * C + t];
    s_be[t] = p.be[ch * C + t];
  }
  // ---- X, Y and the sums over them: row tile w4, column tiles 2 half, 2 half + 1
  {
    f32x4 kk[2], qk[2], da[2], dl[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) kk[j] = qk[j] = da[j] = dl[j] = zero4();
    const int ra = 16 * w4 + li, rac = ra < last ? ra : last;
#pragma unroll 2
    for (int i = 0; i < DK / 32; ++i) {
      const auto ka = load_frag<TP>(K, tplane, w4 * (DK / 32) + i), qa = load_frag<TP>(Q, tplane, w4 * (DK / 32) + i);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if (2 * half + j > w4) continue;                // above the diagonal
        const auto kb = load_frag<TP>(K, tplane, (2 * half + j) * (DK / 32) + i);
        kk[j] = mm(ka, kb, kk[j]);
        qk[j] = mm(qa, kb, qk[j]);
      }
    }
    float drv = 0.0f;                                   // dR_i . V_i
#pragma unroll 2
    for (int i = 0; i < nv; ++i) {
      const auto ga = load_frag<TP>(GO, up, w4 * nv + i);
      const auto ra_f = load_frag<kFull>(DR, up, w4 * nv + i);
      if (half == 0) {
        const auto va = ld8(V + (int64_t)rac * p.ldv + 32 * i + 8 * g);
#pragma unroll
        for (int e = 0; e < 8; ++e) drv += at(ra_f, e) * (float)va[e];
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if (2 * half + j > w4) continue;
        const auto ub = load_frag<kFull>(U, up, (2 * half + j) * nv + i);
        da[j] = mm(ga, ub, da[j]);
        dl[j] = mm(ra_f, ub, dl[j]);
      }
    }
    drv += __shfl_xor(drv, 16);
    drv += __shfl_xor(drv, 32);
    if (g == 0) s_db[half][ra] = drv;
    __syncthreads();                                    // s_gam, s_be
    f32x4 rs = zero4(), dbs = zero4();
    float2 gr[4];                                       // (read ahead of the stores to LDS)
    float br[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      gr[r] = s_gam[16 * w4 + 4 * g + r];
      br[r] = s_be[16 * w4 + 4 * g + r];
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int col = 16 * (2 * half + j) + li;
      f32x4 x, y;
      const float2 gc = s_gam[col];
      float cs = 0.0f;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 16 * w4 + 4 * g + r;
        const bool in = row < ck.len && col <= row;
        const float d = in ? exp_of(gr[r], gc) : 0.0f;
        x[r] = in ? p.scale * d * da[j][r] : 0.0f;
        const float dn = in && col < row ? -d * dl[j][r] : 0.0f;
        y[r] = br[r] * dn;
        const float qkr = in ? qk[j][r] : 0.0f, kkr = in ? kk[j][r] : 0.0f;
        const float m = x[r] * qkr + y[r] * kkr;
        rs[r] += m;
        cs += m;
        dbs[r] += dn * kkr;
      }
      s_xt.st4(col, 16 * w4 + 4 * g, x);
      s_yt.st4(col, 16 * w4 + 4 * g, y);
      cs += __shfl_xor(cs, 16);
      cs += __shfl_xor(cs, 32);
      if (g == 0) s_cs[w4][col] = cs;
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      rs[r] = sum16(rs[r]);
      dbs[r] = sum16(dbs[r]);
    }
    if (li == 0)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 16 * w4 + 4 * g + r;
        s_rs[half][row] = rs[r];
        s_db[half][row] += dbs[r];     // written above by a lane of this wave
      }
  }
  __syncthreads();

  // ---- dq, dk: rows 32 half .. + 31, column tiles w4, w4 + 4, ..
  float wg = 0.0f;                                      // <W0, G>, by the first half
  const float *W0 = p.w0t + ch * (DK * p.dv), *G = p.gwt + ch * (DK * p.dv);
#pragma unroll 1
  for (int i = 0; i < NT; ++i) {
    int zero = 0;                       // opaque: keeps what is the same for every tile out of registers between them
    asm volatile("" : "+v"(zero));
    const int rt = w4 + 4 * i;
    f32x4 aq[2], ar[2], au[2];
#pragma unroll
    for (int a = 0; a < 2; ++a) aq[a] = ar[a] = au[a] = zero4();
#pragma unroll 2
    for (int ks = 0; ks < nv; ++ks) {
      const f32x8 w8 = load_frag(W0, rt * nv + ks), g8 = load_frag(G, rt * nv + ks);
      if (half == 0)
#pragma unroll
        for (int e = 0; e < 8; ++e) wg += w8[e] * g8[e];
      const auto wf = split_of<kFull>(w8), gf = split_of<kFull>(g8);
#pragma unroll
      for (int a = 0; a < 2; ++a) {
        const int f = (2 * half + a) * nv + ks;
        aq[a] = mm(load_frag<TP>(GO, up, f), wf, aq[a]);
        ar[a] = mm(load_frag<kFull>(DR, up, f), wf, ar[a]);
        au[a] = mm(load_frag<kFull>(U, up, f), gf, au[a]);
      }
    }
    const auto k0 = load_frag<TP>(KT, tplane, rt * 2 + 0), k1 = load_frag<TP>(KT, tplane, rt * 2 + 1);
    const auto q0 = load_frag<TP>(QT, tplane, rt * 2 + 0), q1 = load_frag<TP>(QT, tplane, rt * 2 + 1);
    const int col = rt * 16 + li;
#pragma unroll
    for (int a = 0; a < 2; ++a) {
      f32x4 xq = zero4(), xk = zero4();
      const int r16 = 32 * half + 16 * a + zero, row = r16 + li;
      xq = mm(s_xt.ld_t(0, r16), k0, xq);
      xq = mm(s_xt.ld_t(32, r16), k1, xq);
      xk = mm(s_xt.ld(row, 8 * g), q0, xk);
      xk = mm(s_xt.ld(row, 32 + 8 * g), q1, xk);
      xk = mm(s_yt.ld_t(0, r16), k0, xk);
      xk = mm(s_yt.ld_t(32, r16), k1, xk);
      xk = mm(s_yt.ld(row, 8 * g), k0, xk);
      xk = mm(s_yt.ld(row, 32 + 8 * g), k1, xk);
      const int r0 = r16 + 4 * g;
      const f32x4 eg = *reinterpret_cast<const f32x4 *>(p.eg + ch * C + r0);
      const f32x4 el = *reinterpret_cast<const f32x4 *>(p.el + ch * C + r0);
      const f32x4 be = *reinterpret_cast<const f32x4 *>(p.be + ch * C + r0);
      f32x4 dots[3] = {zero4(), zero4(), zero4()};      // of q with aq, k with ar, k with au: this lane's column
      f32x4 kv = zero4(), qv = zero4();             // four tokens' elements
#pragma unroll
      for (int x = TP - 1; x >= 0; --x) {
        const int64_t e = frag_at(col, r0, 2) * 2 + x * tplane;
        const bf16x4 kx = *reinterpret_cast<const bf16x4 *>(KT + e), qx = *reinterpret_cast<const bf16x4 *>(QT + e);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          kv[r] += (float)kx[r];
          qv[r] += (float)qx[r];
        }
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        if (r0 + r >= ck.len) continue;
        const int64_t tk = ck.tok0 + r0 + r;
        const float dqi = p.scale * eg[r] * aq[a][r], dui = el[r] * au[a][r];
        dots[0][r] = qv[r] * dqi;
        dots[1][r] = kv[r] * ar[a][r];
        dots[2][r] = kv[r] * dui;
        const float dq = dqi + xq[r], dk = dui - be[r] * eg[r] * ar[a][r] + xk[r];
        if (p.gqp) {
          p.gqp[(tk * p.heads + h) * DK + col] = dq;
          p.gkp[(tk * p.heads + h) * DK + col] = dk;
        } else {
          static_cast<T *>(p.gq)[tk * p.ldgq + kh * DK + col] = from_f32<T>(dq);
          static_cast<T *>(p.gk)[tk * p.ldgk + kh * DK + col] = from_f32<T>(dk);
        }
      }
      // row sums over the tile's columns, added to this wave's (kept in registers over the tiles they would
      // spill, and every reload wait for the loads before it)
#pragma unroll
      for (int x = 0; x < 3; ++x) {
#pragma unroll
        for (int r = 0; r < 4; ++r) dots[x][r] = sum16(dots[x][r]);
        if (li == 0) {
          f32x4 *s = reinterpret_cast<f32x4 *>(&s_row[x][w4][r0]);
          *s = i == 0 ? dots[x] : *s + dots[x];
        }
      }
    }
  }
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) wg += __shfl_xor(wg, m);
  if (l == 0 && half == 0) s_red[w4] = wg;
  __syncthreads();
  if (t < C) {
    float s[3];
#pragma unroll
    for (int j = 0; j < 3; ++j) s[j] = s_row[j][0][t] + s_row[j][1][t] + s_row[j][2][t] + s_row[j][3][t];
    const bool ok = t < ck.len;
    const float eg = p.eg[ch * C + t], be = p.be[ch * C + t];
    float cs = 0.0f;
    for (int x = t >> 4; x < 4; ++x) cs += s_cs[x][t];          // row tiles on and below this column's
    if (ok) p.gbeta[h * p.gbeta_hs + ck.tok0 + t] = s_db[0][t] + s_db[1][t] - eg * s[1];
    // in 64 bits: the rows' terms cancel in part
    double d = ok ? (double)s[0] - (double)(be * eg * s[1]) - (double)s[2] +
                        ((double)s_rs[0][t] + (double)s_rs[1][t] - (double)cs) : 0.0;
    double us = ok ? (double)s[2] : 0.0;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) us += __shfl_xor(us, m);
    if (t == last)
      d += us + (double)(p.eg[ch * C + C - 1] * (s_red[0] + s_red[1] + s_red[2] + s_red[3]));
    // sum over the later tokens of the chunk
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
      const double x = __shfl_down(d, m);
      if (t + m < 64) d += x;
    }
    if (ok && p.gdecay) p.gdecay[h * p.gdecay_hs + ck.tok0 + t] = (float)d;
  }
}

// dq and dk of a key head: the sum over the heads that share it, in head order.
template <typename T>
__global__ __launch_bounds__(256) void delta_group_kernel(DeltaParams p) {
  const int grp = p.heads / p.key_heads, dk = p.dk;
  const int2 rows = rows_of(p);
  const int first = rows.x, used = rows.y;
  const int64_t per = (int64_t)p.key_heads * dk / 4;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < (int64_t)(used - first) * per; i += (int64_t)gridDim.x * 256) {
    const int64_t tk = first + i / per;
    const int e = (int)(i % per) * 4, kh = e / dk, d = e % dk;
    const float *a = p.gqp + (tk * p.heads + kh * grp) * dk + d, *b = p.gkp + (tk * p.heads + kh * grp) * dk + d;
    f32x4 x = zero4(), y = zero4();
    for (int j = 0; j < grp; ++j) {
      x += *reinterpret_cast<const f32x4 *>(a + j * dk);
      y += *reinterpret_cast<const f32x4 *>(b + j * dk);
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      static_cast<T *>(p.gq)[tk * p.ldgq + e + r] = from_f32<T>(x[r]);
      static_cast<T *>(p.gk)[tk * p.ldgk + e + r] = from_f32<T>(y[r]);
    }
  }
}

// Gradient of a rate that the heads share: the sum over heads, in order.
__global__ __launch_bounds__(256) void delta_sum_rates_kernel(DeltaParams p) {
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i >= p.n) return;
  float x = 0.0f, y = 0.0f;
  for (int h = 0; h < p.heads; ++h) {
    if (p.sum_beta) x += p.gbeta_part[(int64_t)h * p.n + i];
    if (p.sum_decay) y += p.gdecay_part[(int64_t)h * p.n + i];
  }
  if (p.sum_beta) p.gbeta_out[i] = x;
  if (p.sum_decay) p.gdecay_out[i] = y;
}

template <typename T, int DK>
hipError_t chain_impl(const DeltaParams &p, hipStream_t s) {
  const int wgs = p.nseq * p.heads * (p.dv / SL);
  if (p.segs < 3) {     // (without chunks only the gradients, which pass through)
    hipLaunchKernelGGL((delta_chain_kernel<T, DK, kWhole>), dim3(wgs + (p.nchunk > 0 ? state_wgs(p, kWhole) : 0)), dim3(512), 0, s,
                       p, wgs);
    return hipGetLastError();
  }
  const int grads = wgs * (p.segs - 1);
  hipLaunchKernelGGL((delta_chain_kernel<T, DK, kFirst>), dim3(grads + state_wgs(p, kFirst)), dim3(512), 0, s, p, grads);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((delta_chain_kernel<T, DK, kSecond>), dim3(grads + state_wgs(p, kSecond)), dim3(512), 0, s, p, grads);
  return hipGetLastError();
}
template <typename T, int DK>
hipError_t gtoken_impl(const DeltaParams &p, hipStream_t s) {
  hipLaunchKernelGGL((delta_gtoken_kernel<T, DK>), dim3((unsigned)((int64_t)p.nchunk * p.heads)), dim3(512), 0, s, p);
  return hipGetLastError();
}
template <typename T>
hipError_t group_impl(const DeltaParams &p, hipStream_t s) {
  hipLaunchKernelGGL(delta_group_kernel<T>, dim3(2048), dim3(256), 0, s, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_delta_backward(const DeltaParams &p, bool bf16, hipStream_t s) {
  hipError_t e = launch_delta_plan(p, s);
  if (e == hipSuccess) e = launch_delta_chunk(p, bf16, true, s);
  if (e == hipSuccess) e = TTT_DELTA_BY_DK(chain_impl, p, p, s);
  if (e == hipSuccess && p.nchunk > 0) e = TTT_DELTA_BY_DK(gtoken_impl, p, p, s);
  if (e == hipSuccess && p.nchunk > 0 && p.gqp) e = bf16 ? group_impl<__bf16>(p, s) : group_impl<float>(p, s);
  if (p.n == 0) return e;
  if (e == hipSuccess && (p.sum_beta || p.sum_decay)) {
    hipLaunchKernelGGL(delta_sum_rates_kernel, dim3((p.n + 255) / 256), dim3(256), 0, s, p);
    e = hipGetLastError();
  }
  return e;
}

}  // namespace ttt
