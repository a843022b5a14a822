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
#include "delta.h"
#include "split.h"

namespace ttt {
namespace {

constexpr int C = kDeltaChunk;
constexpr int SL = kDeltaSlice;

// ------------------------------------------------------------------ state gradients
// The reverse of the states kernel, with the same split and layout.
template <typename T, int DK>
__global__ __launch_bounds__(256, 1) void delta_gstate_kernel(DeltaParams p) {
  __shared__ __attribute__((aligned(16))) SpTile<T, SL, DK> s_g;
  __shared__ __attribute__((aligned(16))) SpTile<T, SL, C> s_go, s_goe, s_du, s_dp;
  constexpr int NT = DK / 64;
  const int slices = p.dv / SL;
  const int sl = blockIdx.x % slices, h = blockIdx.x / slices % p.heads, b = blockIdx.x / slices / p.heads;
  const int t = threadIdx.x, w = t >> 6, l = t & 63, g = l >> 4, li = l & 15;
  const int kh = h / (p.heads / p.key_heads);
  const DeltaSeq sq = p.seqs[b];
  const int64_t wrow = (((int64_t)b * p.heads + h) * p.dv + sl * SL + li) * DK + w * (DK / 4) + 4 * g;
  f32x4 st[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    st[i] = p.gw_out ? *reinterpret_cast<const f32x4 *>(p.gw_out + wrow + 16 * i) : zero4();
    s_g.st4(li, w * (DK / 4) + 16 * i + 4 * g, st[i]);
  }
  const int64_t plane = C * C * 2;
  const int t4 = 16 * w + 4 * g;
  for (int c0 = (sq.len - 1) / C * C; c0 >= 0 && sq.len > 0; c0 -= C) {
    const int len = sq.len - c0 < C ? sq.len - c0 : C;
    const int64_t c = sq.chunk0 + c0 / C, ch = c * p.heads + h;
    const int64_t tok0 = sq.start + c0;
    const f32x4 eg = *reinterpret_cast<const f32x4 *>(p.eg + ch * C + t4);
    const f32x4 el = *reinterpret_cast<const f32x4 *>(p.el + ch * C + t4);
    f32x4 go, be;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const bool ok = t4 + r < len;
      const int64_t tk = tok0 + (ok ? t4 + r : len - 1);
      const float x = to_f32(static_cast<const T *>(p.go)[tk * p.ldgo + h * p.dv + sl * SL + li]);
      go[r] = ok ? x : 0.0f;
      be[r] = ok ? p.beta[h * p.beta_hs + tk] : 0.0f;
    }
    s_go.st4(li, t4, go);
    s_goe.st4(li, t4, go * eg * p.scale);
    __syncthreads();
    const int row = 16 * w + li < len ? 16 * w + li : len - 1;
    const T *K = static_cast<const T *>(p.k) + (tok0 + row) * p.ldk + kh * DK + 8 * g;
    f32x4 du = zero4();
#pragma unroll
    for (int ks = 0; ks < DK; ks += 32) du = mm(ld8(K + ks), s_g.ld(li, ks + 8 * g), du);
#pragma unroll
    for (int r = 0; r < 4; ++r) du[r] = t4 + r < len ? du[r] * el[r] : 0.0f;
    const char *am = p.am + ch * (C * C * 4), *tt = p.tt + ch * (C * C * 4);
#pragma unroll
    for (int ks = 0; ks < C; ks += 32)
      if (ks + 32 > 16 * w) du = mm(Sp<T>::ld(am, plane, (16 * w + li) * C + ks + 8 * g), s_go.ld(li, ks + 8 * g), du);
    s_du.st4(li, t4, du);
    {                                   // the gradient after the chunk, [dk][dv]
      char *o = p.gwt + ch * ((int64_t)DK * p.dv * 4);
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          Sp<T>::st1(o, (int64_t)DK * p.dv * 2, (int64_t)(w * (DK / 4) + 16 * i + 4 * g + r) * p.dv + sl * SL + li,
                     st[i][r]);
    }
    __syncthreads();
    f32x4 dr = zero4();
#pragma unroll
    for (int ks = 0; ks < C; ks += 32)
      if (ks + 32 > 16 * w) dr = mm(Sp<T>::ld(tt, plane, (16 * w + li) * C + ks + 8 * g), s_du.ld(li, ks + 8 * g), dr);
    s_dp.st4(li, t4, dr * be * eg * -1.0f);
    {
      char *o = p.dr + ch * ((int64_t)C * p.dv * 4);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        Sp<T>::st1(o, (int64_t)C * p.dv * 2, (int64_t)(t4 + r) * p.dv + sl * SL + li, dr[r]);
        if (t4 + r < len)
          static_cast<T *>(p.gv)[(tok0 + t4 + r) * p.ldgv + h * p.dv + sl * SL + li] = from_f32<T>(be[r] * dr[r]);
      }
    }
    __syncthreads();
    const float ec = p.eg[ch * C + C - 1];
    const int64_t to = (c * p.key_heads + kh) * (DK * C) + (w * (DK / 4) + li) * C + 8 * g;
    const T *kt = static_cast<const T *>(p.kt) + to, *qt = static_cast<const T *>(p.qt) + to;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      st[i] = st[i] * ec;
#pragma unroll
      for (int ks = 0; ks < C; ks += 32) {
        st[i] = mm(ld8(kt + 16 * i * C + ks), s_dp.ld(li, ks + 8 * g), st[i]);
        st[i] = mm(ld8(qt + 16 * i * C + ks), s_goe.ld(li, ks + 8 * g), st[i]);
      }
      s_g.st4(li, w * (DK / 4) + 16 * i + 4 * g, st[i]);
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < NT; ++i) *reinterpret_cast<f32x4 *>(p.gw + wrow + 16 * i) = st[i];
}

// ------------------------------------------------------------------ token gradients
// One workgroup per chunk and head.  First the 64 x 64 matrices X and Y (wave w has rows 16 w ..),
// which pass through LDS as operands both ways round, then dq and dk, where wave w has dk / 4
// columns, one 16-wide tile at a time, so that each state fragment is read by one wave.
template <typename T, int DK>
__global__ __launch_bounds__(256, 1) void delta_gtoken_kernel(DeltaParams p) {
  __shared__ __attribute__((aligned(16))) SpTile<T, C, C> s_x, s_xt, s_y, s_yt;
  __shared__ float s_row[5][4][C];      // per-wave partials: q.(go W0), k.(dR W0), k.(U G), row / column sums of M
  __shared__ float s_db[C], s_red[4];
  typedef typename Sp<T>::Frag Frag;
  constexpr int NT = DK / 64;
  const int h = blockIdx.x % p.heads, c = blockIdx.x / p.heads;
  const DeltaChunk ck = p.chunks[c];
  if (ck.len == 0) return;
  const int t = threadIdx.x, w = t >> 6, l = t & 63, g = l >> 4, li = l & 15;
  const int grp = p.heads / p.key_heads, kh = h / grp;
  const int64_t ch = (int64_t)c * p.heads + h;
  const int last = ck.len - 1;
  const T *K = static_cast<const T *>(p.k) + (int64_t)ck.tok0 * p.ldk + kh * DK;
  const T *Q = static_cast<const T *>(p.q) + (int64_t)ck.tok0 * p.ldq + kh * DK;
  const T *V = static_cast<const T *>(p.v) + (int64_t)ck.tok0 * p.ldv + h * p.dv;
  const T *GO = static_cast<const T *>(p.go) + (int64_t)ck.tok0 * p.ldgo + h * p.dv;
  const int64_t uo = ch * ((int64_t)C * p.dv * 4), up = (int64_t)C * p.dv * 2;
  const char *U = p.u + uo, *DR = p.dr + uo;

  // ---- X, Y and the sums over them
  {
    f32x4 kk[4], qk[4], da[4], dl[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) kk[j] = qk[j] = da[j] = dl[j] = zero4();
    const int ra = 16 * w + li, rac = ra < last ? ra : last;
#pragma unroll 2
    for (int ks = 0; ks < DK; ks += 32) {
      const auto ka = ld8(K + (int64_t)rac * p.ldk + ks + 8 * g);
      const auto qa = ld8(Q + (int64_t)rac * p.ldq + ks + 8 * g);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (j > w) continue;
        const int rb = 16 * j + li < last ? 16 * j + li : last;
        const auto kb = ld8(K + (int64_t)rb * p.ldk + ks + 8 * g);
        kk[j] = mm(ka, kb, kk[j]);
        qk[j] = mm(qa, kb, qk[j]);
      }
    }
    float drv = 0.0f;                                   // dR_i . V_i
    for (int ks = 0; ks < p.dv; ks += 32) {
      const auto ga = ld8(GO + (int64_t)rac * p.ldgo + ks + 8 * g);
      const Frag ra_f = Sp<T>::ld(DR, up, (int64_t)ra * p.dv + ks + 8 * g);
      const auto va = ld8(V + (int64_t)rac * p.ldv + ks + 8 * g);
#pragma unroll
      for (int i = 0; i < 8; ++i) drv += Sp<T>::at(ra_f, i) * (float)va[i];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (j > w) continue;
        const Frag ub = Sp<T>::ld(U, up, (int64_t)(16 * j + li) * p.dv + ks + 8 * g);
        da[j] = mm(ga, ub, da[j]);
        dl[j] = mm(ra_f, ub, dl[j]);
      }
    }
    drv += __shfl_xor(drv, 16);
    drv += __shfl_xor(drv, 32);
    if (g == 0) s_db[ra] = drv;
    f32x4 rs = zero4(), dbs = zero4();
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int col = 16 * j + li;
      f32x4 x, y;
      float cs = 0.0f;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 16 * w + 4 * g + r;
        const bool in = row < ck.len && col <= row;
        const float d = in ? exp_of(p.gam[ch * C + row] - p.gam[ch * C + col]) : 0.0f;
        const float be = in ? p.beta[h * p.beta_hs + ck.tok0 + row] : 0.0f;
        x[r] = in ? p.scale * d * da[j][r] : 0.0f;
        const float dn = in && col < row ? -d * dl[j][r] : 0.0f;
        y[r] = be * dn;
        const float qkr = in ? qk[j][r] : 0.0f, kkr = in ? kk[j][r] : 0.0f;
        const float m = x[r] * qkr + y[r] * kkr;
        rs[r] += m;
        cs += m;
        dbs[r] += dn * kkr;
        s_x.st1(row, col, x[r]);
        s_y.st1(row, col, y[r]);
      }
      s_xt.st4(col, 16 * w + 4 * g, x);
      s_yt.st4(col, 16 * w + 4 * g, y);
      cs += __shfl_xor(cs, 16);
      cs += __shfl_xor(cs, 32);
      if (g == 0) s_row[4][w][col] = cs;
    }
#pragma unroll
    for (int m = 1; m < 16; m <<= 1)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        rs[r] += __shfl_xor(rs[r], m);
        dbs[r] += __shfl_xor(dbs[r], m);
      }
    if (li == 0)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 16 * w + 4 * g + r;
        s_row[3][0][row] = rs[r];
        s_db[row] += dbs[r];           // written above by a lane of this wave
      }
  }
  __syncthreads();

  // ---- dq, dk
  float dq_dot[4][4], dr_dot[4][4], du_dot[4][4];       // [row tile][r]: this lane's column of the row sums
#pragma unroll
  for (int a = 0; a < 4; ++a)
#pragma unroll
    for (int r = 0; r < 4; ++r) dq_dot[a][r] = dr_dot[a][r] = du_dot[a][r] = 0.0f;
  float wg = 0.0f;                                      // <W0, G>
  const int64_t so = ch * ((int64_t)DK * p.dv * 4), sp = (int64_t)DK * p.dv * 2;
  const int64_t to = ((int64_t)c * p.key_heads + kh) * (DK * C);
  const T *KT = static_cast<const T *>(p.kt) + to, *QT = static_cast<const T *>(p.qt) + to;
#pragma unroll 1
  for (int i = 0; i < NT; ++i) {
    const int d0 = w * (DK / 4) + 16 * i;
    int base = li;                      // opaque: keeps the LDS operands below out of registers between tiles
    asm volatile("" : "+v"(base));
    f32x4 aq[4], ar[4], au[4];
#pragma unroll
    for (int a = 0; a < 4; ++a) aq[a] = ar[a] = au[a] = zero4();
    for (int ks = 0; ks < p.dv; ks += 32) {
      const Frag wf = Sp<T>::ld(p.w0t + so, sp, (int64_t)(d0 + li) * p.dv + ks + 8 * g);
      const Frag gf = Sp<T>::ld(p.gwt + so, sp, (int64_t)(d0 + li) * p.dv + ks + 8 * g);
#pragma unroll
      for (int e = 0; e < 8; ++e) wg += Sp<T>::at(wf, e) * Sp<T>::at(gf, e);
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        const int row = 16 * a + li, rc = row < last ? row : last;
        aq[a] = mm(ld8(GO + (int64_t)rc * p.ldgo + ks + 8 * g), wf, aq[a]);
        ar[a] = mm(Sp<T>::ld(DR, up, (int64_t)row * p.dv + ks + 8 * g), wf, ar[a]);
        au[a] = mm(Sp<T>::ld(U, up, (int64_t)row * p.dv + ks + 8 * g), gf, au[a]);
      }
    }
    const auto k0 = ld8(KT + (d0 + li) * C + 8 * g), k1 = ld8(KT + (d0 + li) * C + 32 + 8 * g);
    const auto q0 = ld8(QT + (d0 + li) * C + 8 * g), q1 = ld8(QT + (d0 + li) * C + 32 + 8 * g);
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      f32x4 xq = zero4(), xk = zero4();
      const int row = 16 * a + base;
      xq = mm(s_x.ld(row, 8 * g), k0, xq);
      xq = mm(s_x.ld(row, 32 + 8 * g), k1, xq);
      xk = mm(s_xt.ld(row, 8 * g), q0, xk);
      xk = mm(s_xt.ld(row, 32 + 8 * g), q1, xk);
      xk = mm(s_y.ld(row, 8 * g), k0, xk);
      xk = mm(s_y.ld(row, 32 + 8 * g), k1, xk);
      xk = mm(s_yt.ld(row, 8 * g), k0, xk);
      xk = mm(s_yt.ld(row, 32 + 8 * g), k1, xk);
      const int r0 = 16 * a + 4 * g, col = d0 + li;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        if (r0 + r >= ck.len) continue;
        const int64_t tk = ck.tok0 + r0 + r;
        const float eg = p.eg[ch * C + r0 + r], el = p.el[ch * C + r0 + r], be = p.beta[h * p.beta_hs + tk];
        const float qv = to_f32(Q[(int64_t)(r0 + r) * p.ldq + col]), kv = to_f32(K[(int64_t)(r0 + r) * p.ldk + col]);
        const float dqi = p.scale * eg * aq[a][r], dui = el * au[a][r];
        dq_dot[a][r] += qv * dqi;
        dr_dot[a][r] += kv * ar[a][r];
        du_dot[a][r] += kv * dui;
        const float dq = dqi + xq[r], dk = dui - be * eg * ar[a][r] + xk[r];
        if (p.gqp) {
          p.gqp[(tk * p.heads + h) * DK + col] = dq;
          p.gkp[(tk * p.heads + h) * DK + col] = dk;
        } else {
          static_cast<T *>(p.gq)[tk * p.ldgq + kh * DK + col] = from_f32<T>(dq);
          static_cast<T *>(p.gk)[tk * p.ldgk + kh * DK + col] = from_f32<T>(dk);
        }
      }
    }
  }
#pragma unroll
  for (int a = 0; a < 4; ++a)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      float x = dq_dot[a][r], y = dr_dot[a][r], z = du_dot[a][r];
#pragma unroll
      for (int m = 1; m < 16; m <<= 1) {
        x += __shfl_xor(x, m);
        y += __shfl_xor(y, m);
        z += __shfl_xor(z, m);
      }
      if (li == 0) {
        const int row = 16 * a + 4 * g + r;
        s_row[0][w][row] = x;
        s_row[1][w][row] = y;
        s_row[2][w][row] = z;
      }
    }
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) wg += __shfl_xor(wg, m);
  if (l == 0) s_red[w] = wg;
  __syncthreads();
  if (t < C) {
    float s[3];
#pragma unroll
    for (int j = 0; j < 3; ++j) s[j] = s_row[j][0][t] + s_row[j][1][t] + s_row[j][2][t] + s_row[j][3][t];
    const bool ok = t < ck.len;
    const float eg = p.eg[ch * C + t], be = ok ? p.beta[h * p.beta_hs + ck.tok0 + t] : 0.0f;
    float cs = 0.0f;
    for (int x = t >> 4; x < 4; ++x) cs += s_row[4][x][t];      // rows of waves below this column's tile
    if (ok) p.gbeta[h * p.gbeta_hs + ck.tok0 + t] = s_db[t] - eg * s[1];
    // in 64 bits: the rows' terms cancel in part
    double d = ok ? (double)s[0] - (double)(be * eg * s[1]) - (double)s[2] + ((double)s_row[3][0][t] - (double)cs) : 0.0;
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
  const int first = p.seqs[0].start, used = *p.used;
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

// Rows of no sequence have no gradient: zeros in the rates' gradients there.
__global__ __launch_bounds__(256) void delta_zero_rates_kernel(DeltaParams p) {
  const int first = p.seqs[0].start, used = *p.used, total = first + (p.n - used);
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < (int64_t)total * p.heads; i += (int64_t)gridDim.x * 256) {
    const int r = (int)(i % total), h = (int)(i / total), row = r < first ? r : used + (r - first);
    p.gbeta[h * p.gbeta_hs + row] = 0.0f;
    if (p.gdecay) p.gdecay[h * p.gdecay_hs + row] = 0.0f;
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
hipError_t gstate_impl(const DeltaParams &p, hipStream_t s) {
  hipLaunchKernelGGL((delta_gstate_kernel<T, DK>), dim3((unsigned)((int64_t)p.nseq * p.heads * (p.dv / SL))), dim3(256), 0, s, p);
  return hipGetLastError();
}
template <typename T, int DK>
hipError_t gtoken_impl(const DeltaParams &p, hipStream_t s) {
  hipLaunchKernelGGL((delta_gtoken_kernel<T, DK>), dim3((unsigned)((int64_t)p.nchunk * p.heads)), dim3(256), 0, s, p);
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
  if (e == hipSuccess && p.nchunk > 0) e = launch_delta_states(p, bf16, true, s);
  if (e == hipSuccess) e = TTT_DELTA_BY_DK(gstate_impl, p, p, s);
  if (e == hipSuccess && p.nchunk > 0) e = TTT_DELTA_BY_DK(gtoken_impl, p, p, s);
  if (e == hipSuccess && p.nchunk > 0 && p.gqp) e = bf16 ? group_impl<__bf16>(p, s) : group_impl<float>(p, s);
  if (p.n == 0) return e;
  if (p.cu) {
    const int kw = p.key_heads * p.dk;
    if (e == hipSuccess) e = launch_delta_zero_rows(p, p.gq, p.ldgq, kw, bf16, s);
    if (e == hipSuccess) e = launch_delta_zero_rows(p, p.gk, p.ldgk, kw, bf16, s);
    if (e == hipSuccess) e = launch_delta_zero_rows(p, p.gv, p.ldgv, p.heads * p.dv, bf16, s);
    if (e == hipSuccess) {
      hipLaunchKernelGGL(delta_zero_rates_kernel, dim3(64), dim3(256), 0, s, p);
      e = hipGetLastError();
    }
  }
  if (e == hipSuccess && (p.sum_beta || p.sum_decay)) {
    hipLaunchKernelGGL(delta_sum_rates_kernel, dim3((p.n + 255) / 256), dim3(256), 0, s, p);
    e = hipGetLastError();
  }
  return e;
}

}  // namespace ttt
