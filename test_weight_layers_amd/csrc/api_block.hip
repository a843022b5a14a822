// C entry points of windowed attention, layer norm and AdamW (declared in include/ttt.h): argument checks, plans and
// workspace layout.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <vector>

#include "ttt.h"
#include "adamw.h"
#include "api_util.h"
#include "attention.h"
#include "norm.h"

using namespace ttt;

namespace {

// ------------------------------------------------------------------ windowed attention
struct AttnShape {
  int heads, key_heads, d;
  int64_t nq, nk;
  int nseq, block, before, after, sinks, dtype;
};

struct AttnPlan {
  int64_t whole;
  int qrows, krows, qtiles, ktiles, splits, parts, qparts, sink_parts, sink_tiles;
  size_t off_seqs, off_o, off_ml, off_delta, off_part, off_qpart, off_spart, total;
};

int check_attention_heads(int H, int Hk, int d, int dtype) {
  if (H < 1 || Hk < 1) return fail(TTT_EINVAL, "heads and key_heads must be >= 1 (got %d, %d)", H, Hk);
  if (H % Hk != 0) return fail(TTT_EINVAL, "heads (%d) must be a multiple of key_heads (%d)", H, Hk);
  const int st = check_dtype(dtype);
  if (st) return st;
  if (d != 64 && d != 128 && d != 256) return fail(TTT_EUNSUPPORTED, "d=%d is not 64, 128 or 256", d);
  return TTT_OK;
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

int plan_attention(const AttnShape &a, bool backward, AttnPlan *out) {
  const int st = check_attention_heads(a.heads, a.key_heads, a.d, a.dtype);
  if (st) return st;
  if (a.nq < 0 || a.nk < 0 || a.nseq < 1) return fail(TTT_EINVAL, "nq and nk must be >= 0 and sequences >= 1");
  if (a.nq > kAttnMaxRows || a.nk > kAttnMaxRows) return fail(TTT_EUNSUPPORTED, "more than %lld rows", (long long)kAttnMaxRows);
  if (a.block < 1 || a.sinks < 0) return fail(TTT_EINVAL, "block must be >= 1 and sinks >= 0");
  const bool bf16 = a.dtype == TTT_BF16;
  // a sequence of len rows has at most len / rows + 1 tiles, an empty one none
  const auto tiles = [&](int64_t n, int rows) { return a.nseq == 1 ? ceil_div(n, rows) : n / rows + std::min<int64_t>(a.nseq, n); };
  // keys that a query sees inside its window, at most, and those of a sequence, at the mean
  const int64_t lk = ceil_div(a.nk, a.nseq), lq = ceil_div(a.nq, a.nseq);
  // limited on one side only, a window's rows see unlike numbers of keys, about half of all in the mean
  const bool bounded = a.before >= 0 && a.after >= 0, limited = a.before >= 0 || a.after >= 0;
  const int64_t span = bounded ? std::min(((int64_t)a.before + a.after + 1) * a.block, int64_t(1) << 40) : 0;
  const int64_t window = bounded ? std::min(span, lk) : lk;
  // Tiles that have something to do, of sequences with `mean` such rows: of the side with fewer rows each sequence has a last
  // tile of its own (gradient of 120 queries on 8694 keys in 70 sequences, 16 heads of 128 on 2, fp32: 178 us with full tiles
  // counted and 135 so); where both sides are alike the models' times are of full tiles (2441 tokens in 8 sequences 58 and 77).
  const auto items = [&](int64_t n, int64_t mean, int rows, bool shorter) {
    return shorter ? std::min(tiles(n, rows), a.nseq * ceil_div(mean, rows)) : ceil_div(std::min(n, a.nseq * mean), rows);
  };
  AttnPlan P{};
  P.splits = P.parts = P.qparts = 1;
  size_t o = 0;
  const auto take = [&](size_t bytes) {
    const size_t at = o;
    o = align256(o + bytes);
    return at;
  };
  P.off_seqs = take(a.nseq > kAttnLaneSeqs ? ((size_t)a.nseq + 1) * sizeof(AttnSeq) : 0);
  const int grp = a.heads / a.key_heads;
  if (!backward) {
    const bool small = tiles(a.nq, attn_query_rows(a.d, bf16, false)) * a.heads < 512;
    P.qrows = attn_query_rows(a.d, bf16, small);
    P.krows = 64;
    const int64_t longest = a.nseq == 1 ? lk : std::min(a.nk, lk + lk / 2), wgs = tiles(a.nq, P.qrows) * a.heads;
    AttnWork w;
    // (fewer queries than keys in several sequences: about the mean length each, with a last tile of its own)
    w.tiles = wgs, w.busy = items(a.nq, lq, P.qrows, a.nq < a.nk) * a.heads, w.even = a.nseq == 1 && (bounded || !limited);
    w.keys = std::min(longest, (bounded ? span : longest) + P.qrows + a.sinks);
    w.mean_keys = std::min(lk, window + P.qrows + a.sinks) * (bounded || !limited ? 1.0 : 0.55);
    const AttnCut cut = attn_cut(w, a.d, P.qrows, bf16);
    P.whole = cut.whole, P.splits = cut.splits;
    const size_t rows = (size_t)(wgs - cut.whole) * cut.splits * P.qrows;
    P.off_o = take(rows * a.d * 4);
    P.off_ml = take(rows * 8);
  } else {
    // Tiles of 64 rows where tiles of 128 are few for 256 CUs, and for twice as many where a mask makes their work uneven
    // (bf16, 64: 8 x 1024 tokens of 12 heads, window 512: 77 us against 91; 8192 tokens of 8 heads, no mask: 589 against 540).
    const int64_t few = limited ? 1024 : 512;
    const bool small = a.d == 64 ? tiles(a.nk, 128) * a.key_heads < few : a.d == 256 && tiles(a.nq, 128) * a.heads < 256;
    P.qrows = attn_grad_query_rows(a.d, bf16, small);
    P.krows = attn_grad_key_rows(a.d, bf16, small);
    P.off_delta = take((size_t)a.heads * a.nq * 4);
    // Rows of a sequence, at the mean, that see or are seen at all: queries that stand further before the first key than the
    // window reaches do not, nor keys that are further behind the first query.  Each walk is bounded by the rows that it goes
    // over: with the larger of both for either, 64 queries on 8192 keys (8 heads of 128 on 2, bf16) had the queries cut in ten.
    const int64_t bq = a.after < 0 ? lq : std::min(lq, lk + ((int64_t)a.after + 1) * a.block);
    const int64_t bk = a.before < 0 ? lk : std::min(lk, lq + ((int64_t)a.before + 1) * a.block);
    // (lengths are on the device: the longest sequence is taken as twice the mean)
    const int64_t long_q = a.nseq == 1 ? bq : std::min(a.nq, 2 * bq), long_k = a.nseq == 1 ? bk : std::min(a.nk, 2 * bk);
    AttnGradWork w;
    w.key_tiles = ceil_div(a.nk, P.krows) * a.key_heads, w.query_tiles = ceil_div(a.nq, P.qrows) * a.heads;
    w.key_items = items(a.nk, bk, P.krows, a.nk < a.nq) * a.key_heads;
    w.query_items = items(a.nq, bq, P.qrows, a.nq < a.nk) * a.heads;
    w.queries = std::min(long_q, (bounded ? span : long_q) + P.krows) * grp, w.keys = std::min(long_k, (bounded ? span : long_k) + P.qrows);
    w.query_steps = ceil_div(a.sinks > 0 ? long_q : std::min(long_q, (bounded ? span : long_q) + P.krows), 32) * grp;
    // (a mask with one limit takes half of the square of the shorter side)
    const double part = bounded || !limited ? 1.0 : 1.0 - 0.4 * std::min(bq, bk) / std::max<int64_t>(1, std::max(bq, bk));
    w.mean_queries = std::min(bq, (bounded ? span : bq) + P.krows) * grp * part;
    w.mean_keys = std::min(bk, (bounded ? span : bk) + P.qrows) * part;
    const AttnGradCut cut = attn_grad_cut(w, a.d, bf16, P.qrows, P.krows);
    P.parts = cut.parts, P.qparts = cut.qparts;
    if (P.qparts > 1) P.off_qpart = take((size_t)P.qparts * a.nq * a.heads * a.d * 4);
    if (P.parts > 1) P.off_part = take((size_t)P.parts * a.nk * a.key_heads * 2 * a.d * 4);
    // Sinks, which all queries behind their window see: ranges of these of their own, where a sequence may be long beside
    // the window (lengths are on the device: taken as four times the mean), joined with the window's part by the sums' kernel.
    // Not where one range takes 64 MB already: so many sequences keep the CUs busy without.
    const int64_t sink_tiles = ceil_div(std::min<int64_t>(a.sinks, a.nk), P.krows);
    const int64_t most = int64_t(64) << 20;
    const double bytes = (double)a.nseq * (double)sink_tiles * a.key_heads * P.krows * 2.0 * a.d * 4.0;
    if (bytes > 0 && bytes <= (double)most && a.before >= 0 && a.nq > 2 * (window + P.krows)) {
      const int64_t one = (int64_t)bytes;
      P.sink_tiles = (int)sink_tiles;
      const int64_t behind = std::min(a.nq, 4 * lq) * grp / std::max<int64_t>(window * grp / 2, 512);
      P.sink_parts = (int)std::max<int64_t>(1, std::min<int64_t>({32, behind, most / one}));
      P.off_spart = take((size_t)one * (1 + P.sink_parts));
    }
  }
  const int64_t qt = tiles(a.nq, P.qrows), kt = tiles(a.nk, P.krows);
  const int64_t key_items = kt * a.key_heads * P.parts + (int64_t)a.nseq * P.sink_tiles * a.key_heads * P.sink_parts;
  if (qt * a.heads * P.splits * P.qparts + (backward ? key_items : 0) > kMaxGroups ||
      a.nq * a.heads / (1024 / a.d) > kMaxGroups)
    return fail(TTT_EUNSUPPORTED, "too many rows or sequences for %d heads in one call", a.heads);
  P.qtiles = (int)qt, P.ktiles = (int)kt;
  P.total = std::max<size_t>(o, 256);
  *out = P;
  return TTT_OK;
}

// Tiles of 64 rows are reached by 32-bit offsets.
int check_tile_row(const Rows &r, int64_t n) {
  const int st = check_row(r, n);
  if (st) return st;
  if (r.ld * (int64_t)r.es >= (int64_t(1) << 31) / 64)
    return fail(TTT_EUNSUPPORTED, "row stride of %s too large (64 rows must span < 2 GiB)", r.name);
  return TTT_OK;
}
int check_scale(float scale) {
  if (!std::isfinite(scale) || scale <= 0.0f) return fail(TTT_EINVAL, "scale must be finite and > 0");
  return TTT_OK;
}

// Checks and parameters that the forward and the gradient share.
int attention_params(const AttnShape &a, bool backward, const Rows &q, const Rows &k, const Rows &v, const int32_t *cu,
                     const int32_t *cu_k, float scale, void *ws, size_t ws_bytes, AttnParams *out) {
  AttnPlan P;
  int st = plan_attention(a, backward, &P);
  if (st || (st = check_scale(scale))) return st;
  if ((st = check_tile_row(q, a.nq)) || (st = check_tile_row(k, a.nk)) || (st = check_tile_row(v, a.nk))) return st;
  if (cu_k && !cu) return fail(TTT_EINVAL, "cu_seqlens_k needs cu_seqlens");
  if (!cu && a.nseq != 1) return fail(TTT_EINVAL, "cu_seqlens is needed for %d sequences", a.nseq);
  if (cu && !cu_k && a.nq != a.nk)
    return fail(TTT_EINVAL, "cu_seqlens_k is needed where k has other rows (%lld) than q (%lld)", (long long)a.nk, (long long)a.nq);
  if ((st = check_ws(ws, ws_bytes, P.total))) return st;
  AttnParams p{};
  char *b = static_cast<char *>(ws);
  p.q = q.p, p.k = k.p, p.v = v.p, p.ldq = q.ld, p.ldk = k.ld, p.ldv = v.ld;
  p.nq = (int)a.nq, p.nk = (int)a.nk, p.nseq = a.nseq, p.cu_q = cu, p.cu_k = cu_k ? cu_k : cu;
  p.heads = a.heads, p.key_heads = a.key_heads, p.d = a.d, p.sinks = a.sinks, p.scale = scale;
  // (positions lie within kAttnMaxRows of 0: a larger block is as large as 2^28)
  const int64_t block = std::min<int64_t>(a.block, kAttnMaxRows), most = int64_t(1) << 30;
  const auto span = [&](int64_t blocks) { return (int)std::min<int64_t>(blocks * block, most); };
  p.block = fast_div(block), p.group = fast_div(a.heads / a.key_heads);
  p.back = a.before < 0 ? (int)most : span(a.before), p.ahead = a.after < 0 ? (int)most : span((int64_t)a.after + 1);
  p.back_q = a.after < 0 ? (int)most : span(a.after), p.ahead_q = a.before < 0 ? (int)most : span((int64_t)a.before + 1);
  p.per_qtiles = fast_div(P.qtiles), p.per_ktiles = fast_div(P.ktiles), p.per_splits = fast_div(P.splits);
  p.per_parts = fast_div(P.parts), p.per_qparts = fast_div(P.qparts);
  p.per_sink_parts = fast_div(P.sink_parts), p.per_sink_tiles = fast_div(P.sink_tiles), p.per_key_heads = fast_div(a.key_heads);
  p.seqs = reinterpret_cast<AttnSeq *>(b + P.off_seqs);
  p.qrows = P.qrows, p.krows = P.krows, p.qtiles = P.qtiles, p.ktiles = P.ktiles;
  p.whole = (int)P.whole, p.splits = P.splits;
  p.part_o = reinterpret_cast<float *>(b + P.off_o), p.part_ml = reinterpret_cast<float2 *>(b + P.off_ml);
  p.delta = reinterpret_cast<float *>(b + P.off_delta);
  p.parts = P.parts, p.part = reinterpret_cast<float *>(b + P.off_part);
  p.qparts = P.qparts, p.qpart = reinterpret_cast<float *>(b + P.off_qpart);
  p.sink_parts = P.sink_parts, p.sink_tiles = P.sink_tiles, p.spart = reinterpret_cast<float *>(b + P.off_spart);
  *out = p;
  return TTT_OK;
}

// Ranges of 512 keys (a workgroup's start takes as long as 256), shorter where there are fewer workgroups than CUs, longer
// where there are over 2048: 16 tokens over 2048 keys, 8 heads of 256 on 4, bf16 57 us in ranges of 128 and 37 of 512.
int step_splits(int H, int Hk, int64_t n, int capacity) {
  const int64_t wgs = std::max<int64_t>(1, n * Hk * ceil_div(H / Hk, 16));
  const int64_t fill = std::min<int64_t>(256 / wgs, ceil_div(capacity, 128)), most = std::min<int64_t>(2048 / wgs, ceil_div(capacity, 512));
  return (int)std::max<int64_t>(1, std::min<int64_t>(std::max(fill, most), 64));
}
struct StepPlan {
  int splits;
  size_t off_ml, total;
};
int plan_step(int H, int Hk, int d, int64_t n, int capacity, int dtype, StepPlan *out) {
  const int st = check_attention_heads(H, Hk, d, dtype);
  if (st) return st;
  if (n < 0 || capacity < 1) return fail(TTT_EINVAL, "n must be >= 0 and capacity >= 1");
  StepPlan P;
  P.splits = step_splits(H, Hk, n, capacity);
  if (n > kMaxRows || n * Hk * ceil_div(H / Hk, 16) * P.splits > kMaxGroups || H > 65535)
    return fail(TTT_EUNSUPPORTED, "too many rows (%lld) for %d heads in one call", (long long)n, H);
  P.off_ml = align256((size_t)P.splits * n * H * d * 4);
  P.total = std::max<size_t>(256, P.off_ml + align256((size_t)P.splits * n * H * 8));
  *out = P;
  return TTT_OK;
}

}  // namespace

extern "C" {

int ttt_window_attention_workspace_bytes(int32_t heads, int32_t key_heads, int32_t d, int64_t nq, int64_t nk,
                                         int32_t sequences, int32_t block, int32_t before, int32_t after,
                                         int32_t sinks, int32_t dtype, int32_t backward, size_t *bytes) {
  if (!bytes) return fail(TTT_EINVAL, "bytes is null");
  AttnPlan P;
  const int st = plan_attention(AttnShape{heads, key_heads, d, nq, nk, sequences, block, before, after, sinks, dtype}, backward != 0, &P);
  if (st) return st;
  *bytes = P.total;
  return TTT_OK;
}

int ttt_window_attention(int32_t heads, int32_t key_heads, int32_t d, const void *q, int64_t ld_q, const void *k,
                         int64_t ld_k, const void *v, int64_t ld_v, void *o, int64_t ld_o, float *lse, int64_t nq,
                         int64_t nk, const int32_t *cu_seqlens, const int32_t *cu_seqlens_k, int32_t sequences,
                         int32_t block, int32_t before, int32_t after, int32_t sinks, float scale, int32_t dtype,
                         uint32_t flags, void *workspace, size_t workspace_bytes, void *stream) {
  const AttnShape a{heads, key_heads, d, nq, nk, sequences, block, before, after, sinks, dtype};
  int st = check_attention_heads(heads, key_heads, d, dtype);
  if (st) return st;
  if (flags & ~uint32_t(TTT_ATTENTION_ZERO_UNUSED)) return fail(TTT_EINVAL, "unknown flag bits 0x%x", flags);
  const size_t es = esize(dtype);
  const int64_t qw = (int64_t)heads * d, kw = (int64_t)key_heads * d;
  const Rows rq{q, ld_q, qw, es, "q"}, rk{k, ld_k, kw, es, "k"}, rv{v, ld_v, kw, es, "v"}, ro{o, ld_o, qw, es, "o"};
  AttnParams p;
  if ((st = attention_params(a, false, rq, rk, rv, cu_seqlens, cu_seqlens_k, scale, workspace, workspace_bytes, &p))) return st;
  if ((st = check_row(ro, nq))) return st;
  if (rows_overlap(ro, rq, nq)) return fail(TTT_EINVAL, "o must not overlap q");
  for (const Rows *r : {&rk, &rv})
    if (nq > 0 && nk > 0 && rows_overlap_span(*r, nk, o, (size_t)(((nq - 1) * ld_o + qw) * (int64_t)es)) &&
        rows_overlap(ro, *r, std::max(nq, nk)))
      return fail(TTT_EINVAL, "o must not overlap %s", r->name);
  p.o = o, p.ldo = ld_o, p.lse = lse, p.zero_unused = (flags & TTT_ATTENTION_ZERO_UNUSED) != 0;
  hipStream_t s = static_cast<hipStream_t>(stream);
  return run(TTT_K_ATTENTION, "window_attention", s, [&] { return launch_attention(p, dtype == TTT_BF16, s); });
}

int ttt_window_attention_backward(int32_t heads, int32_t key_heads, int32_t d, const void *q, int64_t ld_q,
                                  const void *k, int64_t ld_k, const void *v, int64_t ld_v, const void *o,
                                  int64_t ld_o, const float *lse, const void *grad_o, int64_t ld_grad_o,
                                  void *grad_q, int64_t ld_grad_q, void *grad_k, int64_t ld_grad_k, void *grad_v,
                                  int64_t ld_grad_v, int64_t nq, int64_t nk, const int32_t *cu_seqlens,
                                  const int32_t *cu_seqlens_k, int32_t sequences, int32_t block, int32_t before,
                                  int32_t after, int32_t sinks, float scale, int32_t dtype, void *workspace,
                                  size_t workspace_bytes, void *stream) {
  const AttnShape a{heads, key_heads, d, nq, nk, sequences, block, before, after, sinks, dtype};
  int st = check_attention_heads(heads, key_heads, d, dtype);
  if (st) return st;
  const size_t es = esize(dtype);
  const int64_t qw = (int64_t)heads * d, kw = (int64_t)key_heads * d;
  const Rows rq{q, ld_q, qw, es, "q"}, rk{k, ld_k, kw, es, "k"}, rv{v, ld_v, kw, es, "v"}, ro{o, ld_o, qw, es, "o"};
  const Rows rg{grad_o, ld_grad_o, qw, es, "grad_o"};
  const Rows out[3] = {{grad_q, ld_grad_q, qw, es, "grad_q"}, {grad_k, ld_grad_k, kw, es, "grad_k"}, {grad_v, ld_grad_v, kw, es, "grad_v"}};
  AttnParams p;
  if ((st = attention_params(a, true, rq, rk, rv, cu_seqlens, cu_seqlens_k, scale, workspace, workspace_bytes, &p))) return st;
  if ((st = check_tile_row(rg, nq)) || (st = check_row(ro, nq))) return st;
  if (nq > 0 && !lse) return fail(TTT_EINVAL, "lse is null");
  const int64_t rows[3] = {nq, nk, nk};
  for (int i = 0; i < 3; ++i) {
    if ((st = check_row(out[i], rows[i]))) return st;
    const struct { const Rows *r; int64_t n; } in[5] = {{&rq, nq}, {&rk, nk}, {&rv, nk}, {&ro, nq}, {&rg, nq}};
    for (const auto &x : in)
      if (rows[i] > 0 && x.n > 0 && rows_overlap(out[i], *x.r, std::max(rows[i], x.n)) &&
          rows_overlap_span(out[i], rows[i], x.r->p, (size_t)(((x.n - 1) * x.r->ld + x.r->width) * (int64_t)es)))
        return fail(TTT_EINVAL, "%s must not overlap %s", out[i].name, x.r->name);
    for (int j = 0; j < i; ++j)
      if (rows[i] > 0 && rows[j] > 0 && rows_overlap(out[i], out[j], std::max(rows[i], rows[j])) &&
          rows_overlap_span(out[i], rows[i], out[j].p, (size_t)(((rows[j] - 1) * out[j].ld + out[j].width) * (int64_t)es)))
        return fail(TTT_EINVAL, "%s must not overlap %s", out[i].name, out[j].name);
  }
  p.o = const_cast<void *>(o), p.ldo = ld_o, p.lse = const_cast<float *>(lse), p.go = grad_o, p.ldgo = ld_grad_o;
  p.gq = grad_q, p.gk = grad_k, p.gv = grad_v, p.ldgq = ld_grad_q, p.ldgk = ld_grad_k, p.ldgv = ld_grad_v;
  hipStream_t s = static_cast<hipStream_t>(stream);
  return run(TTT_K_ATTENTION, "window_attention_backward", s, [&] { return launch_attention_backward(p, dtype == TTT_BF16, s); });
}

int ttt_window_attention_step_workspace_bytes(int32_t heads, int32_t key_heads, int32_t d, int64_t n, int32_t capacity,
                                              int32_t dtype, size_t *bytes) {
  if (!bytes) return fail(TTT_EINVAL, "bytes is null");
  StepPlan P;
  const int st = plan_step(heads, key_heads, d, n, capacity, dtype, &P);
  if (st) return st;
  *bytes = P.total;
  return TTT_OK;
}

int ttt_window_attention_step(int32_t heads, int32_t key_heads, int32_t d, void *k_cache, void *v_cache, int64_t ld_cache,
                              int64_t pool_stride, int32_t pool, int32_t capacity, const int32_t *slots,
                              const int32_t *positions, const void *q, int64_t ld_q, const void *k, int64_t ld_k,
                              const void *v, int64_t ld_v, void *o, int64_t ld_o, int64_t n, int32_t block,
                              int32_t before, int32_t sinks, float scale, int32_t dtype, uint32_t flags,
                              void *workspace, size_t workspace_bytes, void *stream) {
  StepPlan P;
  int st = plan_step(heads, key_heads, d, n, capacity, dtype, &P);
  if (st || (st = check_scale(scale))) return st;
  if (flags & ~uint32_t(TTT_ATTENTION_ZERO_UNUSED)) return fail(TTT_EINVAL, "unknown flag bits 0x%x", flags);
  if (pool < 1) return fail(TTT_EINVAL, "pool must be >= 1");
  if (block < 1 || sinks < 0) return fail(TTT_EINVAL, "block must be >= 1 and sinks >= 0");
  if (capacity <= sinks) return fail(TTT_EINVAL, "capacity (%d) must be larger than sinks (%d)", capacity, sinks);
  if (!slots && n > pool) return fail(TTT_EINVAL, "%lld rows without slots need as many caches (pool %d)", (long long)n, pool);
  if (slots && n * n > (int64_t(1) << 42)) return fail(TTT_EUNSUPPORTED, "too many rows (%lld) with slots in one call", (long long)n);
  const size_t es = esize(dtype);
  const int64_t qw = (int64_t)heads * d, kw = (int64_t)key_heads * d;
  const Rows rq{q, ld_q, qw, es, "q"}, rk{k, ld_k, kw, es, "k"}, rv{v, ld_v, kw, es, "v"}, ro{o, ld_o, qw, es, "o"};
  for (const Rows *r : {&rq, &rk, &rv, &ro})
    if ((st = check_row(*r, n))) return st;
  const Rows kc{k_cache, ld_cache, kw, es, "k_cache"}, vc{v_cache, ld_cache, kw, es, "v_cache"};
  if ((st = check_row(kc, capacity)) || (st = check_row(vc, capacity))) return st;
  if (pool > 1 && (pool_stride < (capacity - 1) * ld_cache + kw || pool_stride * (int64_t)es % 16 != 0))
    return fail(TTT_EINVAL, "pool_stride (%lld) must hold a cache and be a multiple of 16 bytes", (long long)pool_stride);
  if (n > 0 && !positions) return fail(TTT_EINVAL, "positions is null");
  const size_t span = (size_t)(((int64_t)(pool - 1) * pool_stride + (int64_t)(capacity - 1) * ld_cache + kw) * (int64_t)es);
  if (rows_overlap(ro, rq, n) || rows_overlap(ro, rk, n) || rows_overlap(ro, rv, n)) return fail(TTT_EINVAL, "o must not overlap q, k or v");
  for (const Rows *r : {&rq, &rk, &rv, &ro})
    for (const Rows *c : {&kc, &vc})
      if (rows_overlap_span(*r, n, c->p, span)) return fail(TTT_EINVAL, "%s must not overlap %s", c->name, r->name);
  // (halves of one buffer's rows may be given: rows of both caches then lie between one another)
  if (overlap(k_cache, span, v_cache, span)) {
    const int64_t ls = ld_cache * (int64_t)es, wb = kw * (int64_t)es;
    const int64_t ps = pool > 1 ? pool_stride * (int64_t)es : INT64_MAX;
    int64_t x = (int64_t)((intptr_t)v_cache - (intptr_t)k_cache);
    x = x < 0 ? -x : x;
    const int64_t cache = (int64_t)(capacity - 1) * ls + wb, in_pool = x % ps, in_row = in_pool % ls;
    const bool inside = in_pool + cache <= ps;          // an entry of one lies in one entry of the other's stride
    const bool beside = inside && in_pool >= cache;     // one cache after the other in each entry
    const bool between = (inside || ps % ls == 0) && in_row >= wb && in_row + wb <= ls;   // column halves of the same rows
    if (!beside && !between) return fail(TTT_EINVAL, "k_cache must not overlap v_cache");
  }
  if ((st = check_ws(workspace, workspace_bytes, P.total))) return st;
  AttnStepParams p{};
  p.kc = k_cache, p.vc = v_cache, p.ldc = ld_cache, p.pool_stride = pool_stride, p.slots = slots, p.positions = positions;
  p.q = q, p.k = k, p.v = v, p.ldq = ld_q, p.ldk = ld_k, p.ldv = ld_v, p.o = o, p.ldo = ld_o;
  p.n = (int)n, p.pool = pool, p.capacity = capacity, p.heads = heads, p.key_heads = key_heads, p.d = d;
  p.block = block, p.before = before < 0 ? -1 : before, p.sinks = sinks, p.scale = scale;
  p.zero_unused = (flags & TTT_ATTENTION_ZERO_UNUSED) != 0;
  p.splits = P.splits, p.part_o = static_cast<float *>(workspace);
  p.part_ml = reinterpret_cast<float2 *>(static_cast<char *>(workspace) + P.off_ml);
  hipStream_t s = static_cast<hipStream_t>(stream);
  return run(TTT_K_ATTENTION, "window_attention_step", s, [&] { return launch_attention_step(p, dtype == TTT_BF16, s); });
}

// ------------------------------------------------------------------ layer norm
static int check_norm(int channels, int width, float eps, int64_t n, int dtype, const float *gamma, const float *beta) {
  int st = check_dtype(dtype);
  if (st) return st;
  if (width < 1 || width > kNormMaxWidth) return fail(TTT_EUNSUPPORTED, "norm_width=%d is not in [1, %d]", width, kNormMaxWidth);
  if (channels < width || channels % width != 0)
    return fail(TTT_EINVAL, "norm_width=%d must divide channels=%d", width, channels);
  if (channels > width && width % 8 != 0)
    return fail(TTT_EUNSUPPORTED, "norm_width=%d of several groups must be a multiple of 8", width);
  if (n < 0 || n > kMaxRows) return fail(TTT_EINVAL, "n must be in [0, %lld]", (long long)kMaxRows);
  if (!(eps >= 0.0f) || !std::isfinite(eps)) return fail(TTT_EINVAL, "eps must be finite and >= 0");
  if ((st = check_aligned(gamma, "gamma")) || (st = check_aligned(beta, "beta"))) return st;
  return TTT_OK;
}

int ttt_layer_norm(int32_t channels, int32_t norm_width, const void *x, int64_t ld_x, const float *gamma, const float *beta,
                   float eps, void *y, int64_t ld_y, int64_t n, int32_t dtype, void *stream) {
  int st = check_norm(channels, norm_width, eps, n, dtype, gamma, beta);
  if (st) return st;
  const size_t es = esize(dtype);
  const Rows in{x, ld_x, channels, es, "x"}, out{y, ld_y, channels, es, "y"};
  if ((st = check_row(in, n)) || (st = check_row(out, n))) return st;
  if (!(x == y && ld_x == ld_y) && rows_overlap(out, in, n)) return fail(TTT_EINVAL, "y must be x or not overlap it");
  NormParams p{};
  p.x = x, p.ldx = ld_x, p.gamma = gamma, p.beta = beta, p.eps = eps, p.n = n;
  p.groups = channels / norm_width, p.width = norm_width, p.y = y, p.ldy = ld_y;
  hipStream_t s = static_cast<hipStream_t>(stream);
  return run(TTT_K_NORM, "layer_norm", s, [&] { return launch_norm(p, dtype == TTT_BF16, s); });
}

int ttt_layer_norm_backward_workspace_bytes(int32_t channels, int32_t norm_width, int64_t n, size_t *bytes) {
  if (!bytes) return fail(TTT_EINVAL, "bytes is null");
  const int st = check_norm(channels, norm_width, 0.0f, n, TTT_F32, nullptr, nullptr);
  if (st) return st;
  *bytes = align256((size_t)norm_grid(n * (channels / norm_width), norm_width) * 2 * norm_width * 4);
  return TTT_OK;
}

int ttt_layer_norm_backward(int32_t channels, int32_t norm_width, const void *grad_y, int64_t ld_grad_y, const void *x,
                            int64_t ld_x, const float *gamma, float eps, void *grad_x, int64_t ld_grad_x,
                            float *grad_gamma, float *grad_beta, int64_t n, int32_t dtype, void *workspace,
                            size_t workspace_bytes, void *stream) {
  int st = check_norm(channels, norm_width, eps, n, dtype, gamma, nullptr);
  if (st) return st;
  const size_t es = esize(dtype);
  const Rows rx{x, ld_x, channels, es, "x"}, rg{grad_y, ld_grad_y, channels, es, "grad_y"}, out{grad_x, ld_grad_x, channels, es, "grad_x"};
  for (const Rows *r : {&rx, &rg, &out})
    if ((st = check_row(*r, n))) return st;
  if (rows_overlap(out, rx, n)) return fail(TTT_EINVAL, "grad_x must not overlap x");
  if (!(grad_x == grad_y && ld_grad_x == ld_grad_y) && rows_overlap(out, rg, n))
    return fail(TTT_EINVAL, "grad_x must be grad_y or not overlap it");
  size_t need = 0;
  if ((st = ttt_layer_norm_backward_workspace_bytes(channels, norm_width, n, &need))) return st;
  if ((st = check_ws(workspace, workspace_bytes, need))) return st;
  NormParams p{};
  p.x = x, p.ldx = ld_x, p.gy = grad_y, p.ldgy = ld_grad_y, p.gamma = gamma, p.eps = eps, p.n = n;
  p.groups = channels / norm_width, p.width = norm_width, p.y = grad_x, p.ldy = ld_grad_x;
  p.ggamma = grad_gamma, p.gbeta = grad_beta, p.part = static_cast<float *>(workspace);
  hipStream_t s = static_cast<hipStream_t>(stream);
  return run(TTT_K_NORM, "layer_norm_backward", s, [&] { return launch_norm_backward(p, dtype == TTT_BF16, s); });
}

// ------------------------------------------------------------------ AdamW
static int check_adamw(const ttt_adamw_tensor *t, int count, int bits, int dtype, bool grads) {
  const int st = check_dtype(dtype);
  if (st) return st;
  if (bits != 8 && bits != 32) return fail(TTT_EUNSUPPORTED, "bits=%d is not 8 or 32", bits);
  if (count < 0) return fail(TTT_EINVAL, "count must be >= 0");
  if (count > 0 && !t) return fail(TTT_EINVAL, "tensors is null");
  const size_t es = esize(dtype), ss = bits == 8 ? 1 : 4;
  const auto off = [](const void *p, size_t a) { return ((uintptr_t)p) % a != 0; };
  const ttt_adamw_tensor *like = nullptr;             // the first that has elements
  for (int i = 0; i < count; ++i) {
    if (t[i].n < 0 || t[i].n > (int64_t(1) << 34)) return fail(TTT_EINVAL, "tensor %d: n must be in [0, 2^34]", i);
    if (t[i].n == 0) continue;                        // (whose pointers may all be null)
    if (!like) like = t + i;
    if ((t[i].master != nullptr) != (like->master != nullptr))
      return fail(TTT_EINVAL, "tensor %d: master for all tensors or for none", i);
    if (!t[i].param || !t[i].exp_avg || !t[i].exp_avg_sq || (grads && !t[i].grad))
      return fail(TTT_EINVAL, "tensor %d: param, grad, exp_avg or exp_avg_sq is null", i);
    if (bits == 8 ? !t[i].exp_avg_scale || !t[i].exp_avg_sq_scale : t[i].exp_avg_scale || t[i].exp_avg_sq_scale)
      return fail(TTT_EINVAL, "tensor %d: scales are given exactly with 8-bit states", i);
    if (off(t[i].param, es) || off(t[i].grad, es) || off(t[i].exp_avg, ss) || off(t[i].exp_avg_sq, ss) || off(t[i].master, 4) ||
        off(t[i].exp_avg_scale, 4) || off(t[i].exp_avg_sq_scale, 4))
      return fail(TTT_EINVAL, "tensor %d: an array is not aligned to its elements", i);
  }
  return TTT_OK;
}

int ttt_adamw_check(const ttt_adamw_tensor *tensors, int32_t count, int32_t bits, int32_t dtype) {
  const int st = check_adamw(tensors, count, bits, dtype, false);
  if (st) return st;
  struct Span {
    uintptr_t a, b;
    bool written;
  };
  try {
    std::vector<Span> spans;
    const auto add = [&](const void *p, int64_t bytes, bool written) {
      if (p && bytes > 0) spans.push_back({(uintptr_t)p, (uintptr_t)p + (uintptr_t)bytes, written});
    };
    const int64_t es = (int64_t)esize(dtype), ss = bits == 8 ? 1 : 4;
    for (int i = 0; i < count; ++i) {
      const ttt_adamw_tensor &t = tensors[i];
      const int64_t blocks = ceil_div(t.n, kAdamwBlock);
      add(t.param, t.n * es, true), add(t.grad, t.n * es, false), add(t.exp_avg, t.n * ss, true), add(t.exp_avg_sq, t.n * ss, true);
      add(t.exp_avg_scale, blocks * 4, true), add(t.exp_avg_sq_scale, blocks * 4, true), add(t.master, t.n * 4, true);
    }
    std::sort(spans.begin(), spans.end(), [](const Span &x, const Span &y) { return x.a < y.a; });
    uintptr_t end = 0, end_written = 0;               // of what begins before
    for (const Span &x : spans) {
      if (x.a < end_written || (x.written && x.a < end)) return fail(TTT_EINVAL, "arrays that are written overlap others");
      end = std::max(end, x.b);
      if (x.written) end_written = std::max(end_written, x.b);
    }
  } catch (...) {
    return fail(TTT_EINVAL, "out of host memory");
  }
  return TTT_OK;
}

int ttt_adamw_step(const ttt_adamw_tensor *tensors, int32_t count, int64_t step, const int64_t *step_device, double lr,
                   const float *lr_device, double beta1, double beta2, double eps, double weight_decay,
                   const float *grad_scale, int32_t bits, int32_t dtype, void *workspace, size_t workspace_bytes, void *stream) {
  int st = check_adamw(tensors, count, bits, dtype, true);
  if (st) return st;
  if (!step_device && step < 1) return fail(TTT_EINVAL, "step must be >= 1");
  if (!lr_device && !(std::isfinite(lr) && lr >= 0.0)) return fail(TTT_EINVAL, "lr must be finite and >= 0");
  if (!(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0)) return fail(TTT_EINVAL, "beta1 and beta2 must be in [0, 1)");
  if (!(std::isfinite(eps) && eps >= 0.0) || !(std::isfinite(weight_decay) && weight_decay >= 0.0))
    return fail(TTT_EINVAL, "eps and weight_decay must be finite and >= 0");
  if (((uintptr_t)step_device) % 8 != 0 || ((uintptr_t)lr_device) % 4 != 0 || ((uintptr_t)grad_scale) % 4 != 0)
    return fail(TTT_EINVAL, "step_device, lr_device and grad_scale must be aligned to their types");
  const bool device = step_device || lr_device;
  if (device && (st = check_ws(workspace, workspace_bytes, sizeof(AdamwFactors)))) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  AdamwParams p{};
  p.beta1 = (float)beta1, p.beta2 = (float)beta2, p.rest1 = (float)(1.0 - beta1), p.rest2 = (float)(1.0 - beta2), p.eps = (float)eps;
  p.grad_scale = grad_scale;
  AdamwFactors *factors = static_cast<AdamwFactors *>(workspace);
  if (device)
    p.f_device = factors;
  else
    p.f = adamw_factors(lr, beta1, beta2, weight_decay, step);
  return run(TTT_K_ADAMW, "adamw_step", s, [&] {
    if (device) {
      const hipError_t e = launch_adamw_factors(factors, step_device, step, lr_device, lr, beta1, beta2, weight_decay, s);
      if (e != hipSuccess) return e;
    }
    int64_t items = 0;
    for (int i = 0; i < count; ++i) {
      if (tensors[i].n > 0) {
        // a tensor has at most 2^23 work items, a launch fewer than 2^24
        p.first[p.count] = (int)items;
        p.t[p.count++] = tensors[i];
        items += adamw_items(tensors[i].n);
      }
      const bool last = i + 1 == count;
      if (p.count > 0 && (last || p.count == kAdamwTensors || items > kMaxGroups)) {
        p.first[p.count] = (int)items;
        const hipError_t e = launch_adamw(p, bits == 8, dtype == TTT_BF16, s);
        if (e != hipSuccess) return e;
        p.count = 0, items = 0;
      }
    }
    return hipSuccess;
  });
}

}  // extern "C"
