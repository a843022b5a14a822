// Windowed attention: parameters of the launchers in attention.hip, attention_bwd.hip and attention_step.hip.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace ttt {

constexpr int kAttnLaneSeqs = 63;   // up to here every wave lays the sequences out for itself

constexpr int64_t kAttnMaxRows = int64_t(1) << 28;      // positions and spans then add in 32 bits

// a / d for 0 <= a < 2^31 without a division (m = (2^32 - 1) / d: the product is at most one short).  A kernel's start is
// fetched cold: 2700 instructions of it, most of them divisions, took 20 us.
struct FastDiv {
  uint32_t d, m;
};
inline FastDiv fast_div(int64_t d) {
  const uint32_t x = d < 1 ? 1u : (uint32_t)d;
  return FastDiv{x, 0xffffffffu / x};
}

// One packed sequence: its query and key rows, its first query and key tile.
struct AttnSeq {
  int qs, ql, ks, kl, qt0, kt0;
};

struct AttnParams {
  const void *q, *k, *v;            // rows [n][ld]: heads * d, key_heads * d columns
  int64_t ldq, ldk, ldv;
  void *o;
  int64_t ldo;
  float *lse;                       // [heads][nq]
  int nq, nk, nseq;
  const int *cu_q, *cu_k;           // [nseq + 1]; both null: one sequence of all rows
  int heads, key_heads, d;
  // Query p sees keys [first key of its block - back, that + ahead); key j is seen by queries [first position of its block
  // - back_q, that + ahead_q).  At most 2^30 each, which is more than all.
  FastDiv block, group;             // group: heads / key_heads
  int back, ahead, back_q, ahead_q, sinks;
  float scale;
  bool zero_unused;
  AttnSeq *seqs;                    // [nseq + 1], more than kAttnLaneSeqs sequences
  int qrows, krows;                 // rows of a query tile and of a key tile
  int qtiles, ktiles;               // at most so many
  FastDiv per_qtiles, per_ktiles, per_splits, per_parts, per_qparts, per_sink_parts, per_sink_tiles, per_key_heads;
  // forward: the query tiles of all heads from the `whole`th on have their keys in `splits` ranges, joined from these
  int whole, splits;
  float *part_o;                    // [tiles in ranges][splits][qrows][d]
  float2 *part_ml;                  // [tiles in ranges][splits][qrows]
  // backward
  const void *go;
  int64_t ldgo;
  void *gq, *gk, *gv;
  int64_t ldgq, ldgk, ldgv;
  float *delta;                     // [heads][nq]
  int qparts;                       // ranges of a query tile's keys
  float *qpart;                     // [qparts][nq][heads][d], qparts > 1
  int parts, sink_parts, sink_tiles;// ranges of a key tile's queries; of a sink tile's beyond the window; tiles of sinks
  float *part;                      // [parts][nk][key_heads][2][d], parts > 1
  float *spart;                     // [nseq][sink_tiles][key_heads][1 + sink_parts][krows][2][d]
};

struct AttnStepParams {
  void *kc, *vc;                    // [pool] caches of [capacity][ld] rows, `pool_stride` elements apart
  int64_t ldc, pool_stride;
  const int *slots, *positions;     // slots may be null (row i: cache i)
  const void *q, *k, *v;
  int64_t ldq, ldk, ldv;
  void *o;
  int64_t ldo;
  int n, pool, capacity, heads, key_heads, d;
  int block, before, sinks;         // before < 0: no limit
  float scale;
  bool zero_unused;
  int splits;
  float *part_o;                    // [splits][n][heads][d]
  float2 *part_ml;                  // [splits][n][heads]
};

// Rows of the tiles that the launchers use.
int attn_query_rows(int d, bool bf16, bool small);
struct AttnCut {
  int64_t whole;                    // query tiles of all heads that are not cut
  int splits;                       // ranges of keys of the others
};
struct AttnWork {
  int64_t tiles, busy;              // query tiles of all heads, at most and at least
  bool even;                        // they see about as many keys
  int64_t keys;                     // that the longest sees
  double mean_keys;
};
AttnCut attn_cut(const AttnWork &w, int d, int rows, bool bf16);
struct AttnGradWork {
  int64_t key_tiles, query_tiles;               // key tiles of all key heads, query tiles of all heads
  int64_t key_items, query_items;               // those of them that have something to do
  int64_t queries, keys;                        // that the longest of them walk over
  int64_t query_steps;                          // tiles of 32 of these queries, head by head
  double mean_queries, mean_keys;
};
struct AttnGradCut {
  int parts, qparts;                            // ranges of queries of a key tile, of keys of a query tile
};
AttnGradCut attn_grad_cut(const AttnGradWork &w, int d, bool bf16, int qrows, int krows);
int attn_grad_query_rows(int d, bool bf16, bool small);
int attn_grad_key_rows(int d, bool bf16, bool small);
hipError_t launch_attention(const AttnParams &p, bool bf16, hipStream_t s);
hipError_t launch_attention_backward(const AttnParams &p, bool bf16, hipStream_t s);
hipError_t launch_attention_step(const AttnStepParams &p, bool bf16, hipStream_t s);
// Lays out more than kAttnLaneSeqs sequences (p.seqs).
hipError_t launch_attention_plan(const AttnParams &p, hipStream_t s);

}  // namespace ttt
