// Packed sequences cut in chunks, on the device: row offsets -> sequences and chunks.
//
// The running maximum of the clamped offsets makes any offsets into disjoint ranges inside
// [0, n): nothing is read or written outside the rows.  Up to 63 sequences every wave lays them
// out for itself (a scan over its lanes, about 0.2 us); more come from tables that a plan kernel
// writes (a launch, 4.4 us).
#pragma once
#include "delta.h"

namespace ttt {

__device__ __forceinline__ int delta_offset(const DeltaParams &p, int i) {
  const int x = p.cu[i];
  return x < 0 ? 0 : (x > p.n ? p.n : x);
}

// Lane i's sequence (start, len, chunk0); every lane of the wave calls this.
__device__ __forceinline__ DeltaSeq lane_seq(const DeltaParams &p) {
  const int l = threadIdx.x & 63;
  int m = l <= p.nseq ? delta_offset(p, l) : 0;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int x = __shfl_up(m, d);
    if (l >= d && x > m) m = x;
  }
  const int end = __shfl_down(m, 1);
  const int len = l < p.nseq ? end - m : 0, nc = (len + kDeltaChunk - 1) / kDeltaChunk;
  int c = nc;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int x = __shfl_up(c, d);
    if (l >= d) c += x;
  }
  return DeltaSeq{m, len, c - nc, 0};
}

__device__ __forceinline__ DeltaSeq seq_of(const DeltaParams &p, int b) {
  if (p.cu == nullptr) return DeltaSeq{0, p.n, 0, 0};
  if (p.nseq > kDeltaLaneSeqs) return p.seqs[b];
  const DeltaSeq s = lane_seq(p);
  return DeltaSeq{__builtin_amdgcn_readlane(s.start, b), __builtin_amdgcn_readlane(s.len, b),
                  __builtin_amdgcn_readlane(s.chunk0, b), 0};
}

__device__ __forceinline__ DeltaChunk chunk_of(const DeltaParams &p, int c) {
  if (p.cu != nullptr && p.nseq > kDeltaLaneSeqs) return p.chunks[c];
  DeltaSeq s{0, p.n, 0, 0};
  int b = 0;
  if (p.cu != nullptr) {
    s = lane_seq(p);
    const unsigned long long hit = __ballot(c >= s.chunk0 && c - s.chunk0 < (s.len + kDeltaChunk - 1) / kDeltaChunk);
    if (hit == 0) return DeltaChunk{0, 0, 0, 0};
    b = __builtin_ctzll(hit);
    s = DeltaSeq{__builtin_amdgcn_readlane(s.start, b), __builtin_amdgcn_readlane(s.len, b),
                 __builtin_amdgcn_readlane(s.chunk0, b), 0};
  }
  const int r = (c - s.chunk0) * kDeltaChunk, left = s.len - r;
  return DeltaChunk{s.start + r, left < 0 ? 0 : (left < kDeltaChunk ? left : kDeltaChunk), b, 0};
}

// The rows that belong to a sequence: [x, y).
__device__ __forceinline__ int2 rows_of(const DeltaParams &p) {
  if (p.cu == nullptr) return int2{0, p.n};
  if (p.nseq > kDeltaLaneSeqs) return int2{p.seqs[0].start, *p.used};
  const DeltaSeq s = lane_seq(p);
  return int2{__builtin_amdgcn_readlane(s.start, 0), __builtin_amdgcn_readlane(s.start, p.nseq)};
}

}  // namespace ttt
