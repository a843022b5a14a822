// What the attention kernels share: tiles of token rows in LDS, packed sequences, visible ranges.
//
// Orientation.  Every kernel holds 16-column tiles of its own rows (queries, or keys for the gradients of k and v) as
// the B operand of 16x16 products and walks over tiles of the other axis, which are the A operand:
//   S[x][c] = sum_d tile[x][d] own[c][d],     out^T[d][c] += sum_x tile[x][d] P[x][c].
// D of the first product gives lane (g, li) column li and rows 16 u + 4 g + r: two such tiles (u = 0, 1) are the eight
// reduction elements of group g that the B operand of the second takes, so P never leaves the lane.  The second
// product's A operand reads the same rows down their columns (ds_read_b64_tr_b16 for bf16).  Statistics of a column
// are a lane's own and its three partners' (lanes 16 apart).
#pragma once
#include "attention.h"
#include "common.h"
#include "dma.h"

namespace ttt {

// A tile of rows of D elements in LDS, in 16-byte units, unit c of row r at c ^ swz(r): eight rows at one unit (and the
// eight beside them at the next one) then meet 16 different units of the 64 banks, and so do eight rows at a pair of
// units, as the transposing read takes them.
template <typename T, int D> struct AttnTile {
  static constexpr int kRow = D * (int)sizeof(T), kUnits = kRow / 16;
  static __device__ __forceinline__ int swz(int r) { return kUnits == 8 ? (r & 6) : (r & 7) << 1; }
  static __device__ __forceinline__ int at(int r, int c) { return r * kRow + ((c ^ swz(r)) << 4); }
  static __device__ __forceinline__ int elem(int r, int e) {      // byte of element e of row r
    return at(r, e * (int)sizeof(T) >> 4) + (e * (int)sizeof(T) & 15);
  }

  // Where a lane reads.  The rows' part of an address is a multiple of kRow and a unit changes by xor, so that a lane has one
  // address for all operands by rows and one (fp32: four) for those by columns, and each read one xor: left to itself the
  // compiler keeps an address for every operand, 16 to 32 registers of the second wave of a SIMD.
  static constexpr int kCols = sizeof(T) == 2 ? 1 : 4;
  struct Lane {
    int row, col[kCols];
  };
  static __device__ __forceinline__ Lane lane() {
    const int l = threadIdx.x & 63, g = l >> 4, li = l & 15;
    Lane a;
    a.row = elem(li, 8 * g);
    if constexpr (sizeof(T) == 2) {
      a.col[0] = elem(4 * g + (li >> 2), 4 * (li & 3));
    } else {
#pragma unroll
      for (int i = 0; i < kCols; ++i) a.col[i] = elem(4 * g + i, li);
    }
    return a;
  }
  template <typename V> static __device__ __forceinline__ V lds(int at) {
    return *(const __attribute__((address_space(3))) V *)(uint32_t)at;
  }
  static __device__ __forceinline__ int offset(const unsigned char *t) {
    return (int)(uint32_t)(uintptr_t)(__attribute__((address_space(3))) const unsigned char *)t;
  }
  // elements 32 k + 8 g .. + 7 of row r0 + li (r0 a multiple of 16)
  static __device__ __forceinline__ typename FragOf<T>::type rows(int tile, const Lane &a, int r0, int k) {
    const int at = xor_here(tile + a.row, k * 32 * (int)sizeof(T)) + r0 * kRow;
    if constexpr (sizeof(T) == 2) {
      return lds<bf16x8>(at);
    } else {
      const f32x4 x = lds<f32x4>(at), y = lds<f32x4>(at + 16);
      return f32x8{x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
    }
  }
  // column 16 d + li of rows r0 + 4 g .. + 3 and r0 + 16 + 4 g .. + 3 (r0 a multiple of 16)
  static __device__ __forceinline__ typename FragOf<T>::type cols(int tile, const Lane &a, int r0, int d) {
    if constexpr (sizeof(T) == 2) {
      const int at = xor_here(tile + a.col[0], d * 32) + r0 * kRow;
      const i16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4 *)(uint32_t)at);
      const i16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4 *)(uint32_t)(at + 16 * kRow));
      return cat8(__builtin_bit_cast(bf16x4, x), __builtin_bit_cast(bf16x4, y));
    } else {
      f32x8 v;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int at = xor_here(tile + a.col[i], d * 64) + r0 * kRow;
        v[i] = lds<float>(at), v[4 + i] = lds<float>(at + 16 * kRow);
      }
      return v;
    }
  }
  // A thread's byte offsets in ROWS rows that it copies, `ld` elements apart: four waves (of a workgroup of four or eight), a KB
  // each at a time.
  template <int ROWS> struct Copy {
    static constexpr int kCopies = ROWS * kRow / 4096, kStep = 4096 / kRow;
    static_assert(kCopies > 0 && ROWS % kStep == 0, "");
    unsigned off[kCopies], step;
    __device__ __forceinline__ explicit Copy(int64_t ld) {
      step = (unsigned)(ld * (int64_t)sizeof(T));
      const int r = (threadIdx.x & 255) / kUnits, pos = threadIdx.x % kUnits;
#pragma unroll
      for (int i = 0; i < kCopies; ++i) off[i] = (unsigned)(r + i * kStep) * step + ((pos ^ swz(r + i * kStep)) << 4);
    }
    // Fetches the rows (the first `valid` exist, the others become zero) from memory.  The copies are asynchronous and not
    // counted by the compiler: landed() before the barrier behind which they are read.
    __device__ __forceinline__ void fetch(const T *src, int valid, unsigned char *t) const {
      const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) & 3;
      const BufferView view = untracked_view(src, valid > 0 ? (unsigned)(valid - 1) * step + kRow : 0);
#pragma unroll
      for (int i = 0; i < kCopies; ++i) copy_to_lds_untracked<16>(view, off[i], t + (i * 4 + wave) * 1024);
    }
  };
  // Zeros in place of what is not finite, rows r0 .. r0 + n - 1 (four waves).
  static __device__ void settle(unsigned char *t, int r0, int n) {
    for (int i = threadIdx.x & 255; i < n * D; i += 256) {
      T *x = reinterpret_cast<T *>(t + elem(r0 + i / D, i % D));
      const float f = to_f32(*x);
      if (!(fabsf(f) < __builtin_inff())) *x = from_f32<T>(0.0f);
    }
  }
};

// Stands in a branch that few tiles take: without it the compiler turns the masks into selects for every tile.
__device__ __forceinline__ void rarely() { asm volatile("s_nop 0"); }

// Waits for this wave's copies to LDS but the last LEFT, then for the other waves.
// (__syncthreads would wait for all of them.)
template <int LEFT = 0> __device__ __forceinline__ void landed() {
  wait_vmcnt_lds<LEFT>();
  bare_barrier();
}

template <typename T> __device__ __forceinline__ typename FragOf<T>::type pack44(const f32x4 a, const f32x4 b) {
  const float v[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
  return pack8<T>(v);
}
__device__ __forceinline__ void store4(__bf16 *p, f32x4 v) {
  bf16x4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = (__bf16)v[i];
  *reinterpret_cast<bf16x4 *>(p) = r;
}
__device__ __forceinline__ void store4(float *p, f32x4 v) { *reinterpret_cast<f32x4 *>(p) = v; }
__device__ __forceinline__ f32x4 zero_f4() { return f32x4{0, 0, 0, 0}; }

// Own rows as B operands: column li of tile c is row row0 + 16 c + li; rows outside [0, len) are zero.
template <typename T, int D, int NC>
__device__ __forceinline__ void own_rows(typename FragOf<T>::type (&f)[NC][D / 32], const T *src, int64_t ld, int row0, int len) {
  const int l = threadIdx.x & 63, g = l >> 4, li = l & 15;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int r = row0 + 16 * c + li;
    const T *b = src + (int64_t)r * ld + 8 * g;
#pragma unroll
    for (int k = 0; k < D / 32; ++k) f[c][k] = r < len ? ld8(b + 32 * k) : zero8<T>();
  }
}

__device__ __forceinline__ int quotient(int a, FastDiv by) {
  const uint32_t q = __umulhi((uint32_t)a, by.m);
  return (int)(q + ((uint32_t)a - q * by.d >= by.d ? 1u : 0u));
}

// ------------------------------------------------------------------ packed sequences
__device__ __forceinline__ int attn_offset(const int *cu, int i, int n) {
  const int x = cu[i];
  return x < 0 ? 0 : (x > n ? n : x);
}
// (rows: a power of two)
__device__ __forceinline__ int tiles_of(int len, int rows) { return (len + rows - 1) >> __builtin_ctz(rows); }

// Lane i's sequence (lane nseq: what follows the last); every lane of the wave calls this.  The running maximum of the
// clamped offsets makes any offsets into disjoint ranges of rows.
__device__ __forceinline__ AttnSeq lane_seq(const AttnParams &p) {
  const int l = threadIdx.x & 63;
  int mq = l <= p.nseq ? attn_offset(p.cu_q, l, p.nq) : 0, mk = l <= p.nseq ? attn_offset(p.cu_k, l, p.nk) : 0;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int x = __shfl_up(mq, d), y = __shfl_up(mk, d);
    if (l >= d) mq = x > mq ? x : mq, mk = y > mk ? y : mk;
  }
  const int eq = __shfl_down(mq, 1), ek = __shfl_down(mk, 1);
  const int ql = l < p.nseq ? eq - mq : 0, kl = l < p.nseq ? ek - mk : 0;
  const int tq = tiles_of(ql, p.qrows), tk = tiles_of(kl, p.krows);
  int cq = tq, ck = tk;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int x = __shfl_up(cq, d), y = __shfl_up(ck, d);
    if (l >= d) cq += x, ck += y;
  }
  return AttnSeq{mq, ql, mk, kl, cq - tq, ck - tk};
}
__device__ __forceinline__ AttnSeq read_seq(const AttnSeq &s, int b) {
  return AttnSeq{__builtin_amdgcn_readlane(s.qs, b),  __builtin_amdgcn_readlane(s.ql, b),  __builtin_amdgcn_readlane(s.ks, b),
                 __builtin_amdgcn_readlane(s.kl, b),  __builtin_amdgcn_readlane(s.qt0, b), __builtin_amdgcn_readlane(s.kt0, b)};
}
__device__ __forceinline__ AttnSeq only_seq(const AttnParams &p) {
  if (p.cu_q == nullptr) return AttnSeq{0, p.nq, 0, p.nk, 0, 0};
  const int qs = attn_offset(p.cu_q, 0, p.nq), qe = attn_offset(p.cu_q, 1, p.nq);
  const int ks = attn_offset(p.cu_k, 0, p.nk), ke = attn_offset(p.cu_k, 1, p.nk);
  return AttnSeq{qs, qe > qs ? qe - qs : 0, ks, ke > ks ? ke - ks : 0, 0, 0};
}
__device__ __forceinline__ AttnSeq seq_of(const AttnParams &p, int b) {
  if (p.nseq == 1) return only_seq(p);
  if (p.nseq > kAttnLaneSeqs) return p.seqs[b];
  return read_seq(lane_seq(p), b);
}
// The sequence of query (or key) tile c and the tile's place in it; false behind the last tile.
template <bool KEYS> __device__ __forceinline__ bool tile_of(const AttnParams &p, int c, AttnSeq *s, int *tile, int *seq) {
  const int rows = KEYS ? p.krows : p.qrows;
  int b = 0;
  if (p.nseq == 1) {
    *s = only_seq(p);
  } else if (p.nseq <= kAttnLaneSeqs) {
    const AttnSeq x = lane_seq(p);
    const int first = KEYS ? x.kt0 : x.qt0;
    const unsigned long long hit = __ballot(c >= first && c - first < tiles_of(KEYS ? x.kl : x.ql, rows));
    if (hit == 0) return false;
    b = __builtin_ctzll(hit);
    *s = read_seq(x, b);
  } else {
    int lo = 0, hi = p.nseq;        // the last sequence that begins at or before c (empty ones share it with their successor)
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if ((KEYS ? p.seqs[mid].kt0 : p.seqs[mid].qt0) <= c) lo = mid; else hi = mid - 1;
    }
    b = lo;
    *s = p.seqs[b];
  }
  *tile = c - (KEYS ? s->kt0 : s->qt0);
  *seq = b;
  return *tile < tiles_of(KEYS ? s->kl : s->ql, rows);
}
// The query (key) rows that belong to a sequence: [x, y).
template <bool KEYS> __device__ __forceinline__ int2 used_rows(const AttnParams &p) {
  const AttnSeq a = seq_of(p, 0), b = p.nseq == 1 ? a : seq_of(p, p.nseq - 1);
  return KEYS ? int2{a.ks, b.ks + b.kl} : int2{a.qs, b.qs + b.ql};
}

// ------------------------------------------------------------------ what a query sees
// Query i of a sequence stands at position i + kl - ql, in block floor(position / block).  It sees keys [lo, hi), and
// those below min(sinks, hi).
__device__ __forceinline__ int clamp_to(int x, int n) { return x < 0 ? 0 : (x > n ? n : x); }
__device__ __forceinline__ int2 seen_keys(const AttnParams &p, const AttnSeq &s, int i) {
  const int at = i + s.kl - s.ql, b = at >= 0 ? quotient(at, p.block) : -quotient(-(at + 1), p.block) - 1;
  const int first = b * (int)p.block.d;
  return int2{clamp_to(first - p.back, s.kl), clamp_to(first + p.ahead, s.kl)};
}
// The queries that see key j inside their window: [x, y).  Those behind y see it if it is a sink.
__device__ __forceinline__ int2 seeing_queries(const AttnParams &p, const AttnSeq &s, int j) {
  const int first = quotient(j, p.block) * (int)p.block.d - (s.kl - s.ql);
  return int2{clamp_to(first - p.back_q, s.ql), clamp_to(first + p.ahead_q, s.ql)};
}

// The largest of a column's four lanes (16 apart), in each of them.
__device__ __forceinline__ float column_max(float x) {
  x = fmaxf(x, __shfl_xor(x, 16));
  return fmaxf(x, __shfl_xor(x, 32));
}

// The keys of a query tile, BK at a time: sinks [0, se), then the window [k0, k1).
template <typename T, int BK> struct KeyWalk {
  int j, e, k0, k1;                   // the tile's first key, the end of its range, and the window
  const T *k, *v;                     // rows of key j
  int64_t dk, dv;                     // from a tile to the next, and to the window's first key
  const T *kw, *vw;
  // tile t; n_sinks: tiles of sinks
  __device__ __forceinline__ KeyWalk(int t, int n_sinks, int se, int k0_, int k1_, const T *kb, const T *vb, int64_t ldk, int64_t ldv) {
    k0 = k0_, k1 = k1_;
    const bool sink = t < n_sinks;
    j = sink ? t * BK : k0 + (t - n_sinks) * BK, e = sink ? se : k1;
    k = kb + (int64_t)j * ldk, v = vb + (int64_t)j * ldv;
    dk = BK * ldk, dv = BK * ldv;
    kw = kb + (int64_t)k0 * ldk, vw = vb + (int64_t)k0 * ldv;
  }
  __device__ __forceinline__ int end() const { return j + BK < e ? j + BK : e; }
  __device__ __forceinline__ void next() {
    j += BK, k += dk, v += dv;
    if (j >= e && e != k1) j = k0, e = k1, k = kw, v = vw;      // (sinks end before the window does)
  }
};

// Work items in launch order go round the 8 XCDs: consecutive items (tiles of one head) on one XCD.
__device__ __forceinline__ int attn_item(int id, int n) {
  const int per = n >> 3;
  return id < per * 8 ? (id & 7) * per + (id >> 3) : id;
}

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
// Exponents above this are taken as differences of scores before they are scaled: e^(s - m) in one multiply-add has the
// rounding of m log2(e), a common factor of a row, which is far from 1 where m is 2^24.
constexpr float kHuge = 65536.0f;

// Zeros in rows of no sequence, 256 threads of `blocks` workgroups.
template <typename T>
__device__ void zero_unused_rows(int2 used, int n, void *rows, int64_t ld, int width, int block, int blocks) {
  const int total = used.x + (n - used.y);
  for (int64_t i = (int64_t)block * 256 + threadIdx.x; i < (int64_t)total * width; i += (int64_t)blocks * 256) {
    const int64_t r = i / width, row = r < used.x ? r : used.y + (r - used.x);
    static_cast<T *>(rows)[row * ld + i % width] = from_f32<T>(0.0f);
  }
}

}  // namespace ttt
