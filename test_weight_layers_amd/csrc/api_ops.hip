// C entry points of the gated delta rule, the gated residual tail and the orthogonalisation
// (declared in include/ttt.h): argument checks and workspace layout.
#include <hip/hip_runtime.h>

#include <cmath>

#include "ttt.h"
#include "api_util.h"
#include "delta.h"
#include "orth.h"
#include "residual.h"

using namespace ttt;

namespace {

// A launch has at most 2^32 - 1 work-items in a direction: below 2^23 workgroups of 512.
constexpr int64_t kMaxGroups = (int64_t(1) << 23) - 1;
constexpr int64_t kMaxRows = 2147483647LL - 64;

// Rows [n][ld] of `width` elements of `es` bytes.
struct Rows {
  const void *p;
  int64_t ld, width;
  size_t es;
  const char *name;
};

int check_row(const Rows &r, int64_t n) {
  if (r.ld < r.width)
    return fail(TTT_EINVAL, "ld of %s (%lld) < its width (%lld)", r.name, (long long)r.ld, (long long)r.width);
  if (n == 0) return TTT_OK;
  if (!r.p) return fail(TTT_EINVAL, "%s is null", r.name);
  if (((uintptr_t)r.p) % 16 != 0 || (r.ld * (int64_t)r.es) % 16 != 0)
    return fail(TTT_EINVAL, "%s rows must be 16-byte aligned", r.name);
  return TTT_OK;
}

// The delta-rule kernels reach the 64 rows of a chunk by 32-bit offsets.
int check_chunk_row(const Rows &r, int64_t n) {
  const int st = check_row(r, n);
  if (st) return st;
  if (r.ld * (int64_t)r.es >= (int64_t(1) << 31) / kDeltaChunk)
    return fail(TTT_EUNSUPPORTED, "row stride of %s too large (64 rows must span < 2 GiB)", r.name);
  return TTT_OK;
}

// Whether two sets of n rows share bytes.  Column slices of one buffer (equal strides) do not
// where their columns are apart.
bool rows_overlap(const Rows &a, const Rows &b, int64_t n) {
  if (n == 0 || !a.p || !b.p) return false;
  const int64_t sa = a.ld * (int64_t)a.es, sb = b.ld * (int64_t)b.es;
  const int64_t wa = a.width * (int64_t)a.es, wb = b.width * (int64_t)b.es;
  if (!overlap(a.p, (size_t)((n - 1) * sa + wa), b.p, (size_t)((n - 1) * sb + wb))) return false;
  if (sa != sb || n == 1) return true;
  int64_t d = (int64_t)((intptr_t)b.p - (intptr_t)a.p) % sa;
  if (d < 0) d += sa;
  return d < wa || d + wb > sa;
}
bool rows_overlap_span(const Rows &a, int64_t n, const void *p, size_t bytes) {
  return n > 0 && a.p && p &&
         overlap(a.p, (size_t)(((n - 1) * a.ld + a.width) * (int64_t)a.es), p, bytes);
}

int check_dtype(int dtype) {
  if (dtype != TTT_F32 && dtype != TTT_BF16) return fail(TTT_EUNSUPPORTED, "unknown dtype %d", dtype);
  return TTT_OK;
}
int check_aligned(const void *p, const char *name) {
  if (p && ((uintptr_t)p) % 16 != 0) return fail(TTT_EINVAL, "%s must be 16-byte aligned", name);
  return TTT_OK;
}

// ------------------------------------------------------------------ gated delta rule
int check_delta_shape(int H, int Hk, int dk, int dv, int dtype) {
  if (H < 1 || Hk < 1) return fail(TTT_EINVAL, "heads and key_heads must be >= 1 (got %d, %d)", H, Hk);
  if (H % Hk != 0) return fail(TTT_EINVAL, "heads (%d) must be a multiple of key_heads (%d)", H, Hk);
  int st = check_dtype(dtype);
  if (st) return st;
  if (dk != 64 && dk != 128 && dk != 256) return fail(TTT_EUNSUPPORTED, "dk=%d is not 64, 128 or 256", dk);
  if (dv < 64 || dv > 1024 || dv % 64 != 0)
    return fail(TTT_EUNSUPPORTED, "dv=%d is not a multiple of 64 in [64, 1024]", dv);
  return TTT_OK;
}

struct DeltaPlan {
  int nchunk;
  size_t off_seqs, off_chunks, off_used, off_eg, off_el, off_be, off_gam, off_tm, off_am, off_tt, off_kp, off_qp, off_kt, off_qt;
  size_t off_gop, off_w0t, off_gwt, off_u, off_dr, off_gqp, off_gkp, off_gb, off_gd, off_su, off_sg, off_sm, total;
  int segs;
};

// Segments that the chunks of a sequence are cut in (1: none), from what the states of a chunk take where
// the order of the chunks bounds them (us), half as much again for their gradients (whose workgroups run
// beside the states'), how many workgroups run at once on 256 CUs of one or two each, and what a further
// segment (its start) and the second launch cost.  Whole calls without and with: 687 chunks x 4 heads of 256
// 2054 and 1051 us (5 segments), 313 x 2 heads of 128 518 and 122 (17), the gradient over 94 232 and 122; not
// taken for 9 sequences of 35 chunks x 2 heads of 128 (82, with 3 89).  (Without rounding per / s up the number
// never falls as rows are added, so that a workspace for more rows of as many sequences serves fewer.)
// The lengths are on the device, so the rule goes by the mean: a long sequence packed with enough short ones
// runs uncut, in the time of its own chunks.
int delta_segments(int H, int dk, int dv, int64_t nc, int64_t nseq, bool bf16, bool backward) {
  const int slices = dv / kDeltaSlice, size = dk == 64 ? 0 : dk == 128 ? 1 : 2;
  const int64_t wgs = nseq * H * slices, per = (nc + nseq - 1) / nseq;
  if (wgs > 256) return 1;
  constexpr double kChunkUs[2][3] = {{1.35, 1.55, 2.05}, {1.8, 2.6, 4.0}}, kJoinUs[3] = {1.0, 1.4, 4.0}, kBothUs[3] = {2, 4, 0};
  const auto rounds = [](int64_t x) {
    const int64_t r = x % 512;
    return (double)(x / 512) * 1.6 + (r == 0 ? 0.0 : r <= 256 ? 1.0 : 1.5);
  };
  int best = 1;
  const double chunk = kChunkUs[bf16 ? 0 : 1][size] * (backward ? 1.5 : 1.0);
  double least = chunk * (double)per * rounds(backward ? 2 * wgs : wgs);
  for (int s = 3; s <= 64 && s <= per; ++s) {
    const int64_t g = backward ? wgs * (s - 1) : 0;
    const double both = rounds(nseq * H * (slices + (int64_t)(s - 2) * (slices + dk / kDeltaSlice)) + g) + rounds(wgs * (s - 1) + g);
    const double t = chunk * (double)per / s * both + (kBothUs[size] + s * kJoinUs[size]) * (backward ? 2.0 : 1.0);
    if (t < least) least = t, best = s;
  }
  return best;
}

int plan_delta(int H, int Hk, int dk, int dv, int64_t n, int64_t nseq, int dtype, bool backward, DeltaPlan *out) {
  if (n < 0 || nseq < 1) return fail(TTT_EINVAL, "n must be >= 0 and sequences >= 1");
  if (n > kMaxRows) return fail(TTT_EUNSUPPORTED, "n=%lld exceeds %lld rows", (long long)n, (long long)kMaxRows);
  // a sequence of len rows has at most len / 64 + 1 chunks, an empty one none
  const int64_t nc = n / kDeltaChunk + (nseq < n ? nseq : n);
  if (nc * H > kMaxGroups || nseq * H * (dv / kDeltaSlice) * (backward ? 2 : 1) > kMaxGroups)
    return fail(TTT_EUNSUPPORTED, "too many chunks or sequences for %d heads in one call", H);
  DeltaPlan P{};
  P.nchunk = (int)nc;
  size_t o = 0;
  const auto take = [&](size_t bytes) {
    const size_t at = o;
    o = align256(o + bytes);
    return at;
  };
  const size_t cc = (size_t)nc * H, sb = 2 * kDeltaParts, tb = 2 * delta_token_parts(dtype == TTT_BF16);
  const size_t mat = (size_t)kDeltaChunk * kDeltaChunk * sb;
  const size_t tok = (size_t)nc * Hk * dk * kDeltaChunk * tb;
  P.off_seqs = take((size_t)nseq * sizeof(DeltaSeq));
  P.off_chunks = take((size_t)nc * sizeof(DeltaChunk));
  P.off_used = take(4);
  P.off_eg = take(cc * kDeltaChunk * 4);
  P.off_el = take(cc * kDeltaChunk * 4);
  P.off_tm = take(cc * mat);
  P.off_am = take(cc * mat);
  P.off_be = take(cc * kDeltaChunk * 4);
  P.off_kp = take(tok);
  P.off_qp = take(tok);
  P.off_kt = take(tok);
  P.segs = delta_segments(H, dk, dv, nc, nseq, dtype == TTT_BF16, backward);
  if (P.segs > 2) {
    P.off_su = take((size_t)nseq * (P.segs - 1) * H * dv * dk * 4);
    if (backward) P.off_sg = take((size_t)nseq * (P.segs - 1) * H * dv * dk * 4);
    P.off_sm = take((size_t)nseq * (P.segs - 2) * H * dk * dk * sb * (backward ? 2 : 1));
  }
  if (backward) {
    P.off_gop = take(cc * kDeltaChunk * dv * tb);
    P.off_gam = take(cc * kDeltaChunk * 8);
    P.off_tt = take(cc * mat);
    P.off_qt = take(tok);
    P.off_w0t = take(cc * dk * dv * 4);
    P.off_gwt = take(cc * dk * dv * 4);
    P.off_u = take(cc * kDeltaChunk * dv * sb);
    P.off_dr = take(cc * kDeltaChunk * dv * sb);
    if (H != Hk) {
      P.off_gqp = take((size_t)n * H * dk * 4);
      P.off_gkp = take((size_t)n * H * dk * 4);
    }
    P.off_gb = take((size_t)n * H * 4);       // gradients of shared rates, per head
    P.off_gd = take((size_t)n * H * 4);
  }
  P.total = o;
  *out = P;
  return TTT_OK;
}

// Checks and parameters that ttt_delta and ttt_delta_backward share.
int delta_params(int H, int Hk, int dk, int dv, const float *w, const Rows &q, const Rows &k, const Rows &v,
                 const float *beta, int64_t bhs, const float *decay, int64_t dhs, int64_t n, const int32_t *cu,
                 int nseq, float scale, int dtype, bool backward, void *ws, size_t ws_bytes, DeltaParams *p) {
  DeltaPlan P;
  int st = plan_delta(H, Hk, dk, dv, n, nseq, dtype, backward, &P);
  if (st) return st;
  if (!cu && nseq != 1) return fail(TTT_EINVAL, "sequences must be 1 without cu_seqlens (got %d)", nseq);
  if (!std::isfinite(scale)) return fail(TTT_EINVAL, "scale must be finite");
  if (!w) return fail(TTT_EINVAL, "w is null");
  if ((st = check_aligned(w, "w"))) return st;
  if ((st = check_chunk_row(q, n)) || (st = check_chunk_row(k, n)) || (st = check_chunk_row(v, n))) return st;
  if (n > 0 && !beta) return fail(TTT_EINVAL, "beta is null");
  if (bhs < 0 || dhs < 0) return fail(TTT_EINVAL, "head strides must be >= 0");
  if ((st = check_ws(ws, ws_bytes, P.total))) return st;
  char *b = static_cast<char *>(ws);
  *p = DeltaParams{};
  p->q = q.p, p->k = k.p, p->v = v.p, p->ldq = q.ld, p->ldk = k.ld, p->ldv = v.ld;
  p->beta = beta, p->decay = decay, p->beta_hs = bhs, p->decay_hs = dhs;
  p->w = w, p->cu = cu, p->n = (int)n, p->heads = H, p->key_heads = Hk, p->dk = dk, p->dv = dv, p->nseq = nseq;
  p->nchunk = P.nchunk, p->scale = scale;
  p->seqs = reinterpret_cast<DeltaSeq *>(b + P.off_seqs);
  p->chunks = reinterpret_cast<DeltaChunk *>(b + P.off_chunks);
  p->used = reinterpret_cast<int *>(b + P.off_used);
  p->eg = reinterpret_cast<float *>(b + P.off_eg);
  p->el = reinterpret_cast<float *>(b + P.off_el);
  p->tm = b + P.off_tm, p->am = b + P.off_am, p->kt = b + P.off_kt;
  p->be = reinterpret_cast<float *>(b + P.off_be);
  p->kp = b + P.off_kp, p->qp = b + P.off_qp;
  p->segs = P.segs;
  p->seg_u = reinterpret_cast<float *>(b + P.off_su), p->seg_g = reinterpret_cast<float *>(b + P.off_sg), p->seg_m = b + P.off_sm;
  if (backward) {
    p->gam = reinterpret_cast<float2 *>(b + P.off_gam);
    p->gop = b + P.off_gop;
    p->tt = b + P.off_tt, p->qt = b + P.off_qt, p->w0t = reinterpret_cast<float *>(b + P.off_w0t), p->gwt = reinterpret_cast<float *>(b + P.off_gwt);
    p->u = b + P.off_u, p->dr = b + P.off_dr;
    if (H != Hk) {
      p->gqp = reinterpret_cast<float *>(b + P.off_gqp);
      p->gkp = reinterpret_cast<float *>(b + P.off_gkp);
    }
    p->gbeta_part = reinterpret_cast<float *>(b + P.off_gb);
    p->gdecay_part = reinterpret_cast<float *>(b + P.off_gd);
  }
  return TTT_OK;
}

}  // namespace

extern "C" {

int ttt_delta_workspace_bytes(int32_t heads, int32_t key_heads, int32_t dk, int32_t dv, int64_t n, int32_t sequences,
                              int32_t dtype, int32_t backward, size_t *bytes) {
  int st = check_delta_shape(heads, key_heads, dk, dv, dtype);
  if (st) return st;
  if (!bytes) return fail(TTT_EINVAL, "bytes is null");
  DeltaPlan P;
  if ((st = plan_delta(heads, key_heads, dk, dv, n, sequences, dtype, backward != 0, &P))) return st;
  *bytes = P.total;
  return TTT_OK;
}

int ttt_delta(int32_t heads, int32_t key_heads, int32_t dk, int32_t dv, const float *w, float *w_out, const void *q,
              int64_t ld_q, const void *k, int64_t ld_k, const void *v, int64_t ld_v, const float *beta,
              int64_t beta_head_stride, const float *decay, int64_t decay_head_stride, void *o, int64_t ld_o,
              int64_t n, const int32_t *cu_seqlens, int32_t sequences, float scale, int32_t dtype, uint32_t flags,
              void *workspace, size_t workspace_bytes, void *stream) {
  int st = check_delta_shape(heads, key_heads, dk, dv, dtype);
  if (st) return st;
  if (flags & ~uint32_t(TTT_DELTA_ZERO_UNUSED)) return fail(TTT_EINVAL, "unknown flag bits 0x%x", flags);
  const size_t es = esize(dtype);
  const int64_t kw = (int64_t)key_heads * dk, vw = (int64_t)heads * dv;
  const Rows rq{q, ld_q, kw, es, "q"}, rk{k, ld_k, kw, es, "k"}, rv{v, ld_v, vw, es, "v"}, ro{o, ld_o, vw, es, "o"};
  DeltaParams p;
  if ((st = delta_params(heads, key_heads, dk, dv, w, rq, rk, rv, beta, beta_head_stride, decay, decay_head_stride, n,
                         cu_seqlens, sequences, scale, dtype, false, workspace, workspace_bytes, &p)))
    return st;
  if ((st = check_chunk_row(ro, n)) || (st = check_aligned(w_out, "w_out"))) return st;
  if (!w_out) return fail(TTT_EINVAL, "w_out is null");
  const size_t wb = (size_t)sequences * heads * dv * dk * 4;
  if (w != w_out && overlap(w, wb, w_out, wb)) return fail(TTT_EINVAL, "w_out must equal w or not overlap it");
  if (rows_overlap(ro, rq, n) || rows_overlap(ro, rk, n) || rows_overlap(ro, rv, n))
    return fail(TTT_EINVAL, "o must not overlap q, k or v");
  for (const Rows *r : {&rq, &rk, &rv, &ro})
    if (rows_overlap_span(*r, n, w_out, wb)) return fail(TTT_EINVAL, "w_out must not overlap %s", r->name);
  if (rows_overlap_span(ro, n, w, wb)) return fail(TTT_EINVAL, "o must not overlap w");
  p.w_out = w_out, p.o = o, p.ldo = ld_o, p.zero_unused = (flags & TTT_DELTA_ZERO_UNUSED) != 0;
  hipStream_t s = static_cast<hipStream_t>(stream);
  return run(TTT_K_DELTA, "delta", s, [&] { return launch_delta_forward(p, dtype == TTT_BF16, s); });
}

int ttt_delta_backward(int32_t heads, int32_t key_heads, int32_t dk, int32_t dv, const float *w, const void *q,
                       int64_t ld_q, const void *k, int64_t ld_k, const void *v, int64_t ld_v, const float *beta,
                       int64_t beta_head_stride, const float *decay, int64_t decay_head_stride, const void *grad_o,
                       int64_t ld_grad_o, const float *grad_w_out, void *grad_q, int64_t ld_grad_q, void *grad_k,
                       int64_t ld_grad_k, void *grad_v, int64_t ld_grad_v, float *grad_beta, float *grad_decay,
                       float *grad_w, int64_t n, const int32_t *cu_seqlens, int32_t sequences, float scale,
                       int32_t dtype, void *workspace, size_t workspace_bytes, void *stream) {
  int st = check_delta_shape(heads, key_heads, dk, dv, dtype);
  if (st) return st;
  const size_t es = esize(dtype);
  const int64_t kw = (int64_t)key_heads * dk, vw = (int64_t)heads * dv;
  const Rows in[4] = {{q, ld_q, kw, es, "q"}, {k, ld_k, kw, es, "k"}, {v, ld_v, vw, es, "v"}, {grad_o, ld_grad_o, vw, es, "grad_o"}};
  const Rows out[3] = {{grad_q, ld_grad_q, kw, es, "grad_q"}, {grad_k, ld_grad_k, kw, es, "grad_k"}, {grad_v, ld_grad_v, vw, es, "grad_v"}};
  DeltaParams p;
  if ((st = delta_params(heads, key_heads, dk, dv, w, in[0], in[1], in[2], beta, beta_head_stride, decay,
                         decay_head_stride, n, cu_seqlens, sequences, scale, dtype, true, workspace, workspace_bytes, &p)))
    return st;
  if ((st = check_chunk_row(in[3], n))) return st;
  for (const Rows &r : out)
    if ((st = check_chunk_row(r, n))) return st;
  if (!grad_w) return fail(TTT_EINVAL, "grad_w is null");
  if ((st = check_aligned(grad_w, "grad_w")) || (st = check_aligned(grad_w_out, "grad_w_out"))) return st;
  if (n > 0 && !grad_beta) return fail(TTT_EINVAL, "grad_beta is null");
  if (n > 0 && (decay != nullptr) != (grad_decay != nullptr))
    return fail(TTT_EINVAL, "grad_decay must be given exactly when decay is");
  const size_t wb = (size_t)sequences * heads * dv * dk * 4;
  if (overlap(grad_w, wb, w, wb) || (grad_w_out && overlap(grad_w, wb, grad_w_out, wb)))
    return fail(TTT_EINVAL, "grad_w must not overlap w or grad_w_out");
  for (int i = 0; i < 3; ++i) {
    for (const Rows &r : in)
      if (rows_overlap(out[i], r, n)) return fail(TTT_EINVAL, "%s must not overlap %s", out[i].name, r.name);
    for (int j = 0; j < i; ++j)
      if (rows_overlap(out[i], out[j], n)) return fail(TTT_EINVAL, "%s must not overlap %s", out[i].name, out[j].name);
    if (rows_overlap_span(out[i], n, grad_w, wb) || rows_overlap_span(out[i], n, w, wb))
      return fail(TTT_EINVAL, "%s must not overlap the states", out[i].name);
  }
  p.go = grad_o, p.ldgo = ld_grad_o, p.gw_out = grad_w_out;
  p.gq = grad_q, p.gk = grad_k, p.gv = grad_v, p.ldgq = ld_grad_q, p.ldgk = ld_grad_k, p.ldgv = ld_grad_v;
  p.gw = grad_w;
  // a rate that several heads share: per-head gradients in the workspace, summed at the end
  p.gbeta_out = grad_beta, p.gdecay_out = grad_decay;
  const bool sb = beta_head_stride == 0 && heads > 1, sd = decay && decay_head_stride == 0 && heads > 1;
  p.gbeta = sb ? p.gbeta_part : grad_beta, p.gbeta_hs = n;
  p.gdecay = !decay ? nullptr : (sd ? p.gdecay_part : grad_decay), p.gdecay_hs = n;
  p.sum_beta = sb, p.sum_decay = sd;
  hipStream_t s = static_cast<hipStream_t>(stream);
  return run(TTT_K_DELTA, "delta_backward", s, [&] { return launch_delta_backward(p, dtype == TTT_BF16, s); });
}

int ttt_delta_step(int32_t heads, int32_t key_heads, int32_t dk, int32_t dv, float *w, int32_t pool,
                   const int32_t *slots, const void *q, int64_t ld_q, const void *k, int64_t ld_k, const void *v,
                   int64_t ld_v, const float *beta, int64_t beta_head_stride, const float *decay,
                   int64_t decay_head_stride, void *o, int64_t ld_o, int64_t n, float scale, int32_t dtype,
                   uint32_t flags, void *stream) {
  int st = check_delta_shape(heads, key_heads, dk, dv, dtype);
  if (st) return st;
  if (flags & ~uint32_t(TTT_DELTA_ZERO_UNUSED)) return fail(TTT_EINVAL, "unknown flag bits 0x%x", flags);
  if (n < 0 || pool < 1) return fail(TTT_EINVAL, "n must be >= 0 and pool >= 1");
  if (n > kMaxRows || n * heads * (dv / 64) > kMaxGroups)
    return fail(TTT_EUNSUPPORTED, "too many rows (%lld) for %d heads in one call", (long long)n, heads);
  // every workgroup looks for rows of the same state among all slots: 2^42 looks take a second
  if (slots && n * n > (int64_t(1) << 42) / ((int64_t)heads * (dv / 64)))
    return fail(TTT_EUNSUPPORTED, "too many rows (%lld) with slots for %d heads in one call", (long long)n, heads);
  if (!slots && n > pool) return fail(TTT_EINVAL, "%lld rows without slots need as many states (pool %d)", (long long)n, pool);
  if (!std::isfinite(scale)) return fail(TTT_EINVAL, "scale must be finite");
  const size_t es = esize(dtype);
  const int64_t kw = (int64_t)key_heads * dk, vw = (int64_t)heads * dv;
  const Rows rq{q, ld_q, kw, es, "q"}, rk{k, ld_k, kw, es, "k"}, rv{v, ld_v, vw, es, "v"}, ro{o, ld_o, vw, es, "o"};
  for (const Rows *r : {&rq, &rk, &rv, &ro})
    if ((st = check_row(*r, n))) return st;
  if (!w) return fail(TTT_EINVAL, "w is null");
  if ((st = check_aligned(w, "w"))) return st;
  if (n > 0 && !beta) return fail(TTT_EINVAL, "beta is null");
  if (beta_head_stride < 0 || decay_head_stride < 0) return fail(TTT_EINVAL, "head strides must be >= 0");
  if (rows_overlap(ro, rq, n) || rows_overlap(ro, rk, n) || rows_overlap(ro, rv, n))
    return fail(TTT_EINVAL, "o must not overlap q, k or v");
  for (const Rows *r : {&rq, &rk, &rv, &ro})
    if (rows_overlap_span(*r, n, w, (size_t)pool * heads * dv * dk * 4))
      return fail(TTT_EINVAL, "w must not overlap %s", r->name);
  DeltaStepParams p{};
  p.q = q, p.k = k, p.v = v, p.ldq = ld_q, p.ldk = ld_k, p.ldv = ld_v;
  p.beta = beta, p.decay = decay, p.beta_hs = beta_head_stride, p.decay_hs = decay_head_stride;
  p.w = w, p.slots = slots, p.o = o, p.ldo = ld_o;
  p.n = (int)n, p.nslots = pool, p.heads = heads, p.key_heads = key_heads, p.dk = dk, p.dv = dv;
  p.scale = scale, p.zero_unused = (flags & TTT_DELTA_ZERO_UNUSED) != 0;
  hipStream_t s = static_cast<hipStream_t>(stream);
  return run(TTT_K_DELTA, "delta_step", s, [&] { return launch_delta_step(p, dtype == TTT_BF16, s); });
}

// ------------------------------------------------------------------ gated residual tail
static int check_residual(int channels, int norm, float eps, int64_t n, int dtype, const float *gamma,
                          const float *alpha, const float *gamma_next) {
  int st = check_dtype(dtype);
  if (st) return st;
  if (channels < 8 || channels % 8 != 0 || channels > kResidualMaxChannels)
    return fail(TTT_EUNSUPPORTED, "channels=%d is not a multiple of 8 in [8, %d]", channels, kResidualMaxChannels);
  if (norm < 8 || norm % 8 != 0 || channels % norm != 0)
    return fail(TTT_EUNSUPPORTED, "norm_width=%d must be a multiple of 8 that divides channels=%d", norm, channels);
  if (n < 0) return fail(TTT_EINVAL, "n must be >= 0");
  if (!(eps >= 0.0f) || !std::isfinite(eps)) return fail(TTT_EINVAL, "eps must be finite and >= 0");
  if ((st = check_aligned(gamma, "gamma")) || (st = check_aligned(alpha, "alpha")) ||
      (st = check_aligned(gamma_next, "gamma_next")))
    return st;
  return TTT_OK;
}

int ttt_gated_residual(int32_t channels, int32_t norm_width, const void *x, int64_t ld_x, const void *o, int64_t ld_o,
                       const void *z, int64_t ld_z, const float *gamma, const float *alpha, const float *gamma_next,
                       float eps, void *y, int64_t ld_y, void *h, int64_t ld_h, int64_t n, int32_t dtype,
                       void *stream) {
  int st = check_residual(channels, norm_width, eps, n, dtype, gamma, alpha, gamma_next);
  if (st) return st;
  if (n == 0) return TTT_OK;
  if ((gamma_next != nullptr) != (h != nullptr)) return fail(TTT_EINVAL, "h must be given exactly when gamma_next is");
  const size_t es = esize(dtype);
  const Rows in[3] = {{x, ld_x, channels, es, "x"}, {o, ld_o, channels, es, "o"}, {z, ld_z, channels, es, "z"}};
  const Rows out[2] = {{y, ld_y, channels, es, "y"}, {h, ld_h, channels, es, "h"}};
  if ((st = check_row(in[0], n)) || (st = check_row(in[1], n)) || (st = check_row(out[0], n))) return st;
  if (z && (st = check_row(in[2], n))) return st;
  if (h && (st = check_row(out[1], n))) return st;
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 3; ++j) {
      if (i == 0 && j == 0 && x == y && ld_x == ld_y) continue;      // in place
      if (rows_overlap(out[i], in[j], n)) return fail(TTT_EINVAL, "%s must not overlap %s", out[i].name, in[j].name);
    }
  if (rows_overlap(out[0], out[1], n)) return fail(TTT_EINVAL, "y must not overlap h");
  ResidualParams p{};
  p.x = x, p.o = o, p.z = z, p.ldx = ld_x, p.ldo = ld_o, p.ldz = ld_z;
  p.gamma = gamma, p.alpha = alpha, p.gamma_next = gamma_next, p.eps = eps, p.n = n;
  p.channels = channels, p.norm = norm_width, p.y = y, p.h = h, p.ldy = ld_y, p.ldh = ld_h;
  hipStream_t s = static_cast<hipStream_t>(stream);
  return run(TTT_K_RESIDUAL, "gated_residual", s, [&] { return launch_residual(p, dtype == TTT_BF16, s); });
}

int ttt_gated_residual_backward_workspace_bytes(int32_t channels, int64_t n, size_t *bytes) {
  if (!bytes) return fail(TTT_EINVAL, "bytes is null");
  const int st = check_residual(channels, channels, 0.0f, n, TTT_F32, nullptr, nullptr, nullptr);
  if (st) return st;
  *bytes = align256((size_t)residual_grid(n, channels) * 2 * channels * 4);
  return TTT_OK;
}

int ttt_gated_residual_backward(int32_t channels, int32_t norm_width, const void *grad_y, int64_t ld_grad_y,
                                const void *grad_h, int64_t ld_grad_h, const void *y, int64_t ld_y, const void *o,
                                int64_t ld_o, const void *z, int64_t ld_z, const float *gamma, const float *alpha,
                                const float *gamma_next, float eps, void *grad_x, int64_t ld_grad_x, void *grad_o,
                                int64_t ld_grad_o, void *grad_z, int64_t ld_grad_z, float *grad_gamma,
                                float *grad_alpha, float *grad_gamma_next, int64_t n, int32_t dtype, void *workspace,
                                size_t workspace_bytes, void *stream) {
  int st = check_residual(channels, norm_width, eps, n, dtype, gamma, alpha, gamma_next);
  if (st) return st;
  if (grad_h && !gamma_next) return fail(TTT_EINVAL, "grad_h needs gamma_next");
  if (n > 0 && (z != nullptr) != (grad_z != nullptr)) return fail(TTT_EINVAL, "grad_z must be given exactly when z is");
  const size_t es = esize(dtype);
  const Rows in[5] = {{grad_y, ld_grad_y, channels, es, "grad_y"}, {grad_h, ld_grad_h, channels, es, "grad_h"},
                      {y, ld_y, channels, es, "y"}, {o, ld_o, channels, es, "o"}, {z, ld_z, channels, es, "z"}};
  const Rows out[3] = {{grad_x, ld_grad_x, channels, es, "grad_x"}, {grad_o, ld_grad_o, channels, es, "grad_o"},
                       {grad_z, ld_grad_z, channels, es, "grad_z"}};
  if (grad_y && (st = check_row(in[0], n))) return st;
  if (grad_h && ((st = check_row(in[1], n)) || (st = check_row(in[2], n)))) return st;
  if ((st = check_row(in[3], n)) || (st = check_row(out[0], n)) || (st = check_row(out[1], n))) return st;
  if (z && ((st = check_row(in[4], n)) || (st = check_row(out[2], n)))) return st;
  for (int i = 0; i < 3; ++i) {
    for (int j = 0; j < 5; ++j) {
      if (i == 0 && j == 0 && grad_x == grad_y && ld_grad_x == ld_grad_y) continue;      // in place
      if (rows_overlap(out[i], in[j], n)) return fail(TTT_EINVAL, "%s must not overlap %s", out[i].name, in[j].name);
    }
    for (int j = 0; j < i; ++j)
      if (rows_overlap(out[i], out[j], n)) return fail(TTT_EINVAL, "%s must not overlap %s", out[i].name, out[j].name);
  }
  size_t need = 0;
  if ((st = ttt_gated_residual_backward_workspace_bytes(channels, n, &need))) return st;
  if ((st = check_ws(workspace, workspace_bytes, need))) return st;
  ResidualParams p{};
  p.o = o, p.z = z, p.ldo = ld_o, p.ldz = ld_z;
  p.gamma = gamma, p.alpha = alpha, p.gamma_next = gamma_next, p.eps = eps, p.n = n;
  p.channels = channels, p.norm = norm_width, p.y = const_cast<void *>(y), p.ldy = ld_y;
  p.gy = grad_y, p.gh = grad_h, p.ldgy = ld_grad_y, p.ldgh = ld_grad_h;
  p.gx = grad_x, p.go = grad_o, p.gz = grad_z, p.ldgx = ld_grad_x, p.ldgo = ld_grad_o, p.ldgz = ld_grad_z;
  p.ggamma = grad_gamma, p.galpha = grad_alpha, p.ggamma_next = grad_gamma_next;
  p.part = static_cast<float *>(workspace);
  hipStream_t s = static_cast<hipStream_t>(stream);
  return run(TTT_K_RESIDUAL, "gated_residual_backward", s,
             [&] { return launch_residual_backward(p, dtype == TTT_BF16, s); });
}

// ------------------------------------------------------------------ orthogonalisation
static int check_orth(int rows, int cols, int batch, int dtype) {
  int st = check_dtype(dtype);
  if (st) return st;
  if (rows < 1 || cols < 1 || batch < 0) return fail(TTT_EINVAL, "rows and cols must be >= 1, batch >= 0");
  if (rows > 65536 || cols > 65536 || batch > 65535)
    return fail(TTT_EUNSUPPORTED, "rows and cols must be <= 65536, batch <= 65535");
  const OrthPlan q = plan_orth(rows, cols, batch, dtype == TTT_BF16);
  if ((int64_t)batch * (q.rp / q.tile) * (q.cp / q.tile) > kMaxGroups)
    return fail(TTT_EUNSUPPORTED, "too many tiles in one call");
  return TTT_OK;
}

int ttt_orthogonalise_workspace_bytes(int32_t rows, int32_t cols, int32_t batch, int32_t dtype, size_t *bytes) {
  if (!bytes) return fail(TTT_EINVAL, "bytes is null");
  const int st = check_orth(rows, cols, batch, dtype);
  if (st) return st;
  *bytes = plan_orth(rows, cols, batch, dtype == TTT_BF16).total;
  return TTT_OK;
}

int ttt_orthogonalise(int32_t rows, int32_t cols, int32_t batch, const void *g, int64_t ld_g, int64_t bs_g, void *out,
                      int64_t ld_out, int64_t bs_out, int32_t steps, int32_t dtype, void *workspace,
                      size_t workspace_bytes, void *stream) {
  int st = check_orth(rows, cols, batch, dtype);
  if (st) return st;
  if (steps < 0) return fail(TTT_EINVAL, "steps must be >= 0");
  if (ld_g < cols || ld_out < cols || bs_g < 0 || bs_out < 0) return fail(TTT_EINVAL, "ld < cols or a negative stride");
  if (batch > 1 && bs_out < (int64_t)(rows - 1) * ld_out + cols)
    return fail(TTT_EINVAL, "matrices of out must not overlap");
  if (batch == 0) return TTT_OK;
  if (!g || !out) return fail(TTT_EINVAL, "g or out is null");
  const size_t es = esize(dtype);
  const auto span = [&](int64_t ld, int64_t bs) {
    return (size_t)(((int64_t)(batch - 1) * bs + (int64_t)(rows - 1) * ld + cols) * (int64_t)es);
  };
  if (overlap(g, span(ld_g, bs_g), out, span(ld_out, bs_out)) && !(g == out && ld_g == ld_out && (batch == 1 || bs_g == bs_out)))
    return fail(TTT_EINVAL, "out must be g with the same strides or not overlap it");
  OrthParams p{};
  p.plan = plan_orth(rows, cols, batch, dtype == TTT_BF16);
  if ((st = check_ws(workspace, workspace_bytes, p.plan.total))) return st;
  p.g = g, p.ldg = ld_g, p.bsg = bs_g, p.out = out, p.ldo = ld_out, p.bso = bs_out;
  p.a = 3.4445f, p.b = -4.7750f, p.c = 2.0315f, p.eps = 1e-7f, p.steps = steps;
  p.ws = static_cast<char *>(workspace);
  hipStream_t s = static_cast<hipStream_t>(stream);
  return run(TTT_K_ORTH, "orthogonalise", s, [&] { return launch_orth(p, s); });
}

}  // extern "C"
