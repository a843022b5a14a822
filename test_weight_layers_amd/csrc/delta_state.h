// Gated delta rule: the states in order of the chunks (notation of delta.hip), for the forward pass and, beside
// the states' gradients, for the backward one.
#pragma once
#include <type_traits>

#include "delta.h"
#include "delta_layout.h"
#include "split.h"

namespace ttt {
namespace {

constexpr int C = kDeltaChunk;
constexpr int SL = kDeltaSlice;
constexpr int64_t kSquare = C * C * 2 * kFull;      // bytes of a split 64 x 64 matrix

// One workgroup per sequence, head and 16-column slice of dv, over the chunks in order.  Its first
// four waves have the rows of the chunk (wave w rows 16 w ..), the last four the state: lane
// (g, li) of wave w holds W[dv = li][dk = w DK/4 + 16 i + 4 g + r] in fp32 accumulators.  A chunk
// is three steps, each ended by an exchange through LDS:
//   rows: P = K W0^T, R        rows: U = T R        state: W += (el o U)^T K;  rows: O = Q W0^T, A U
// so two waves share a SIMD and one works while the other waits or loads.  Tokens and chunk terms
// go from memory straight into operand registers (each is used once), the next chunk's as soon
// as this chunk's have been used, Q into the registers that K leaves, A into those of T.  Bound by the
// order of the chunks: 2.85 us each, heads of 256, of which the matrix cores work 0.6 and the operands,
// 146 KB, take 1.0 at the 64 bytes a clock of a CU; the rest is the three exchanges, one after another.
// BWD writes the states and U that the gradient needs, in place of the outputs.
//
// Where sequences are long and few, the chunks of one are cut in segments that run at once (the state is
// linear in the one before): W after a segment = W before it times M + U, U the state that the segment
// alone leaves and M the one that a unit matrix becomes in it with v = 0.
//   kFirst: the first segment, outputs and all; U and M of the others but the last, of which M is
//           dk / 16 more slices of rows
//   kSecond: the others, each from its own starting state, (W_1 M_1 + U_1) M_2 + U_2 ..
// 687 chunks of 4 heads of 256: 1955 us whole, 558 + 465 in five segments (448 and 256 workgroups; a CU's
// two then take 4.0 us a chunk).
// `id` of `count`: this workgroup among those that do this.
template <typename T, int DK, bool BWD> struct StateLds {
  SplitTile<kFull, SL, DK> w[2];
  SplitTile<kFull, SL, C> r, ul, u;
};
template <typename T, int DK, bool BWD, int PART>
__device__ __forceinline__ void delta_states(const DeltaParams &p, StateLds<T, DK, BWD> &lds, int id, int count) {
  constexpr int NT = DK / 64, NK = DK / 32, TP = kTok<T>;
  auto &s_w = lds.w;
  auto &s_r = lds.r, &s_ul = lds.ul, &s_u = lds.u;
  constexpr int64_t tokens = DK * C * 2 * TP, tplane = DK * C * 2;      // bytes of a chunk's tokens and a part
  const int slices = p.dv / SL, item = xcd_item(id, count);
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
      Split<kFull> tf[2], af[2];
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
      const auto load_square = [&](const char *m, int c, Split<kFull> (&f)[2]) {
#pragma unroll
        // (the second half is zero for the first two waves, whose products leave it out; loads under a
        // condition would make every later wait one for all loads)
        for (int i = 0; i < 2; ++i)
          f[i] = load_frag<kFull>(m + (ch0 + (int64_t)c * p.heads) * kSquare, plane, w * 2 + i);
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
          Sums<kFull> qa[2];
#pragma unroll
          for (int i = 0; i < NK; ++i) {
            qa[i & 1].add(qf[i], W0.ld(li, 32 * i + 8 * g));
            kf[i] = load_token(p.kp, nx, i);
          }
          Sums<kFull> au;
          au.add(af[0], s_u.ld(li, 8 * g));
          if (w >= 2) au.add(af[1], s_u.ld(li, 32 + 8 * g));
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

// Workgroups of it.
int state_wgs(const DeltaParams &p, int part) {
  const int bh = p.nseq * p.heads, slices = p.dv / SL;
  if (part == kWhole) return bh * slices;
  return part == kFirst ? bh * (slices + (p.segs - 2) * (slices + p.dk / SL)) : bh * (p.segs - 1) * slices;
}

}  // namespace
}  // namespace ttt
