// Gated delta rule: parameters shared by the launchers (delta.hip, delta_bwd.hip) and the
// C entry points.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace ttt {

// Tokens per chunk of the chunked form.
constexpr int kDeltaChunk = 64;
// Sequences that a wave lays out for itself.
constexpr int kDeltaLaneSeqs = 63;
// dv columns of the state that one workgroup of the sequential kernels holds.
constexpr int kDeltaSlice = 16;

// bf16 parts of a computed operand (see split.h), and of a token.
constexpr int kDeltaParts = 3;
constexpr int delta_token_parts(bool bf16) { return bf16 ? 1 : 3; }

// What a launch of the sequential kernels does: everything, or the first or second part of segments.
enum DeltaPart { kWhole, kFirst, kSecond };

struct DeltaSeq {      // one packed sequence: rows [start, start + len), its chunks from chunk0 on
  int start, len, chunk0, pad;
};
struct DeltaChunk {    // rows [tok0, tok0 + len) of sequence seq; len = 0: unused entry
  int tok0, len, seq, pad;
};

struct DeltaParams {
  const void *q, *k, *v;            // [n][ld] token rows; Hk, Hk and H heads
  int64_t ldq, ldk, ldv;
  const float *beta, *decay;        // [h * stride + i]; decay may be null (no decay)
  int64_t beta_hs, decay_hs;
  const float *w;                   // [nseq][H][dv][dk] starting states
  float *w_out;                     // final states (may be w)
  void *o;
  int64_t ldo;
  const int *cu;                    // [nseq + 1] row offsets (device) or null: one sequence of n rows
  int n, heads, key_heads, dk, dv, nseq;
  int nchunk;                       // upper bound of the number of chunks
  float scale;
  int zero_unused;                  // write zeros to rows that belong to no sequence
  // workspace (matrices in fragment order, split ones a plane a part: see split.h)
  DeltaSeq *seqs;                   // [nseq]
  DeltaChunk *chunks;               // [nchunk]
  int *used;                        // one past the last row of the last sequence
  float *eg, *el, *be;              // [nchunk][H][64]: e^gamma_i, e^(gamma_last - gamma_i), beta (0 past the chunk)
  float2 *gam;                      // gamma_i in base 2, two floats (backward)
  char *tm, *am;                    // [nchunk][H] split 64 x 64: T, A (forward) or A^T (backward)
  char *tt;                         // T^T (backward)
  char *kp, *qp;                    // [nchunk][Hk] split tokens 64 x dk, 0 past the chunk
  char *kt, *qt;                    // [nchunk][Hk] the same transposed, dk x 64 (qt: backward)
  int segs;                         // segments of a sequence that run at once; < 3: none
  float *seg_u, *seg_g;             // [nseq][segs - 1][H][dv][dk] what segments leave (see delta_state.h), and their gradients
  char *seg_m;                      // [nseq][segs - 2][H] split dk x dk: M^T, and M (backward)
  // backward
  const void *go;                   // gradient of o
  int64_t ldgo;
  const float *gw_out;              // gradient of w_out, or null (zero)
  void *gq, *gk, *gv;
  int64_t ldgq, ldgk, ldgv;
  float *gbeta, *gdecay;            // [h * stride + i]
  int64_t gbeta_hs, gdecay_hs;
  float *gbeta_part, *gdecay_part;  // [H][n] of shared rates (then gbeta / gdecay), summed into
  float *gbeta_out, *gdecay_out;    // [n]
  int sum_beta, sum_decay;
  float *gw;                        // gradient of w
  char *gop;                        // [nchunk][H] split gradient of o, 64 x dv
  float *w0t, *gwt;                 // [nchunk][H] fp32 dk x dv: state before the chunk, its gradient after
  char *u, *dr;                     // [nchunk][H] split 64 x dv: U and dR
  float *gqp, *gkp;                 // [n][H][dk] per-head partials (grouped key heads), or null
};

struct DeltaStepParams {
  const void *q, *k, *v;
  int64_t ldq, ldk, ldv;
  const float *beta, *decay;
  int64_t beta_hs, decay_hs;
  float *w;                         // [slots][H][dv][dk], updated in place
  const int *slots;                 // [n] or null: row i uses state i
  void *o;
  int64_t ldo;
  int n, nslots, heads, key_heads, dk, dv;
  float scale;
  int zero_unused;
};

// Kernel instance by token type and dk.
#define TTT_DELTA_BY_DK(FN, P, ...)                                                            \
  (bf16 ? ((P).dk == 64 ? FN<__bf16, 64>(__VA_ARGS__)                                          \
                        : (P).dk == 128 ? FN<__bf16, 128>(__VA_ARGS__) : FN<__bf16, 256>(__VA_ARGS__)) \
        : ((P).dk == 64 ? FN<float, 64>(__VA_ARGS__)                                           \
                        : (P).dk == 128 ? FN<float, 128>(__VA_ARGS__) : FN<float, 256>(__VA_ARGS__)))

hipError_t launch_delta_forward(const DeltaParams &p, bool bf16, hipStream_t s);
hipError_t launch_delta_backward(const DeltaParams &p, bool bf16, hipStream_t s);
hipError_t launch_delta_step(const DeltaStepParams &p, bool bf16, hipStream_t s);

// Forward pieces that the backward pass runs again.
hipError_t launch_delta_plan(const DeltaParams &p, hipStream_t s);
hipError_t launch_delta_chunk(const DeltaParams &p, bool bf16, bool backward, hipStream_t s);

}  // namespace ttt
