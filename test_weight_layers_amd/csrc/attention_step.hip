// One token for each of n rows against a rolling cache: position x of a sequence stands at place x (x < sinks) or
// sinks + (x - sinks) mod (capacity - sinks) of its cache.  A row sees the visible positions that are still in its cache
// and its own token; the second kernel joins the ranges of keys and then writes the tokens, so that the rows of a call
// read the caches as they were before it.
// Bound by reading the visible keys and values once.  The heads of a key head are the columns of the products of
// attn_tile.h; keys go from memory to registers, 32 a wave, values through the wave's own part of LDS.
// The keys go in ranges of 512 (api_block.hip): 4096 keys of one token, 16 heads of 64, take 9 + 4 us (the launches; 3.5 us
// of bytes; fp32 11 + 4); 64 tokens over caches of 4096 rows, 16 heads of 128 on 4, 116 us (537 MB at 4.6 TB/s; a copy reaches
// 4.9; fp32 205 + 5, 1073 MB at 5.1), and 51 to 54 where a third is visible (185 MB; 66 in ranges of 256, which are bound by
// their start).  The waves wait for all their copies before a tile's values are used, the next tile's among them: what is read ahead is
// covered by one tile's scores and exponentials.  bf16 probabilities are rounded as operands, as in the forward.
#include "attn_tile.h"

namespace ttt {
namespace {

// A row's cache (-1: padding) and position.
__device__ __forceinline__ int2 step_row(const AttnStepParams &p, int row) {
  const int slot = p.slots ? p.slots[row] : row, pos = p.positions[row];
  return int2{slot < 0 || slot >= p.pool || pos < 0 ? -1 : slot, pos};
}
__device__ __forceinline__ int place_of(const AttnStepParams &p, int x) {
  return x < p.sinks ? x : p.sinks + (x - p.sinks) % (p.capacity - p.sinks);
}

template <typename T, int D> __global__ __launch_bounds__(256) void attn_step_kernel(AttnStepParams p) {
  typedef AttnTile<T, D> Tile;
  typedef typename FragOf<T>::type Frag;
  constexpr int NK = D / 32, ND = D / 16, kTile = 32 * Tile::kRow;
  constexpr bool kStage = sizeof(T) == 2;             // fp32 values go straight to registers
  __shared__ __attribute__((aligned(1024))) unsigned char s_raw[kStage ? 8 * kTile : 4 * 16 * D * 4];
  __shared__ float s_m[4][16], s_l[4][16];
  const int grp = p.heads / p.key_heads, hgs = (grp + 15) / 16;
  int item = blockIdx.x;
  const int split = item % p.splits;
  item /= p.splits;
  const int hg = item % hgs;
  item /= hgs;
  const int kh = item % p.key_heads, row = item / p.key_heads;
  const int2 at = step_row(p, row);
  if (at.x < 0) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = threadIdx.x & 63, g = l >> 4, li = l & 15;
  const int pos = at.y, ring = p.capacity - p.sinks;
  int64_t lo64 = p.before < 0 ? 0 : ((int64_t)(pos / p.block) - p.before) * p.block;
  if (pos >= p.capacity && lo64 < (int64_t)pos + 1 - ring) lo64 = (int64_t)pos + 1 - ring;
  const int lo = lo64 < 0 ? 0 : (int)lo64, se = p.sinks < lo ? p.sinks : lo;
  const int ns = tiles_of(se, 32), nt = ns + (int)(((int64_t)pos + 1 - lo + 31) / 32), lo_place = place_of(p, lo);
  const int first = (int)((int64_t)nt * split / p.splits), end = (int)((int64_t)nt * (split + 1) / p.splits);
  const int heads = grp - hg * 16 < 16 ? grp - hg * 16 : 16;
  const int64_t out = ((int64_t)split * p.n + row) * p.heads + kh * grp + hg * 16;
  if (first >= end) {                                 // a range without keys (the row is short): no sums, which nobody takes
    if ((int)threadIdx.x < heads) p.part_ml[out + threadIdx.x] = float2{-__builtin_inff(), 0.0f};
    return;
  }
  const T *kc = static_cast<const T *>(p.kc) + (int64_t)at.x * p.pool_stride + kh * D;
  const T *vc = static_cast<const T *>(p.vc) + (int64_t)at.x * p.pool_stride + kh * D;
  const T *kn = static_cast<const T *>(p.k) + (int64_t)row * p.ldk + kh * D;
  const T *vn = static_cast<const T *>(p.v) + (int64_t)row * p.ldv + kh * D;
  // keys of tile t: x of it from position (or sink) j on
  const auto keys = [&](int t, int &x) {
    const int j = t < ns ? t * 32 : (t - ns) * 32;
    const int64_t left = t < ns ? se - j : (int64_t)pos + 1 - lo - j;
    x = left < 32 ? (int)left : 32;
    return j;
  };
  // row r of tile t in the cache; the new token's (null: it is not in the cache) at the end and for rows behind it
  const auto place = [&](int t, int r) {
    int x;
    const int j = keys(t, x) + r;
    if (t < ns) return r < x ? j : -1;
    if (r >= x || j == pos - lo) return -1;
    const int64_t c = (int64_t)lo_place + j;
    return (int)(c < p.capacity ? c : c - ring);
  };

  const typename Tile::Lane lane = Tile::lane();
  Frag q[NK];
  const int hq = hg * 16 + li;
#pragma unroll
  for (int k = 0; k < NK; ++k)
    q[k] = hq < grp ? ld8(static_cast<const T *>(p.q) + (int64_t)row * p.ldq + (int64_t)(kh * grp + hq) * D + 32 * k + 8 * g) : zero8<T>();
  unsigned char *vt[2] = {s_raw + wave * 2 * kTile, s_raw + wave * 2 * kTile + kTile};
  Frag kf[2][NK];
  const auto fetch_k = [&](int t) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int c = place(t, 16 * u + li);
      const T *b = c < 0 ? kn : kc + (int64_t)c * p.ldc;
#pragma unroll
      for (int k = 0; k < NK; ++k) kf[u][k] = ld8(b + 32 * k + 8 * g);
    }
  };
  const auto fetch_v = [&](int t, int b) {
#pragma unroll
    for (int i = 0; i < kTile / 1024; ++i) {
      const int unit = i * 64 + l, r = unit / Tile::kUnits, x = unit % Tile::kUnits;
      const int c = place(t, r);
      const T *s = c < 0 ? vn : vc + (int64_t)c * p.ldc;
      copy16_to_lds(reinterpret_cast<const char *>(s) + ((x ^ Tile::swz(r)) << 4), vt[b] + i * 1024);
    }
  };
  const float c2 = p.scale * kLog2e;
  float m = -__builtin_inff(), sum = 0.0f;
  f32x4 o[ND];
#pragma unroll
  for (int d = 0; d < ND; ++d) o[d] = zero_f4();
  int t = first + wave, b = 0;
  if (t < end) {
    fetch_k(t);
    if (kStage) fetch_v(t, 0);
  }
  for (; t < end; t += 4, b ^= 1) {
    int n;
    keys(t, n);
    f32x4 sc[2] = {zero_f4(), zero_f4()};
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int k = 0; k < NK; ++k) sc[u] = mma(kf[u][k], q[k], sc[u]);
    Frag vf[kStage ? 1 : ND];
    if (!kStage) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int c = place(t, 16 * (e >> 2) + 4 * g + (e & 3));
        const T *s = c < 0 ? vn : vc + (int64_t)c * p.ldc;
#pragma unroll
        for (int d = 0; d < ND; ++d) vf[kStage ? 0 : d][e] = s[16 * d + li];
      }
    }
    if (t + 4 < end) {
      fetch_k(t + 4);
      if (kStage) fetch_v(t + 4, b ^ 1);
    }
    float mx = -__builtin_inff();
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        if (16 * u + 4 * g + x >= n) sc[u][x] = -__builtin_inff();
        mx = fmaxf(mx, sc[u][x]);
      }
    mx = fmaxf(mx, __shfl_xor(mx, 16));
    mx = fmaxf(mx, __shfl_xor(mx, 32));
    if (__any((mx - m) * c2 > 8.0f)) {                // as in the forward
      const float to = (mx - m) * c2 > 8.0f ? mx : m, a = to == m ? 1.0f : __builtin_amdgcn_exp2f((m - to) * c2);
      m = to, sum *= a;
#pragma unroll
      for (int d = 0; d < ND; ++d) o[d] *= a;
    }
    const float base = m == -__builtin_inff() ? 0.0f : m;
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        sc[u][x] = __builtin_amdgcn_exp2f((sc[u][x] - base) * c2);
        sum += sc[u][x];
      }
    const Frag pr = pack44<T>(sc[0], sc[1]);
    if (kStage) wait_all_memory();
#pragma unroll
    for (int d = 0; d < ND; ++d) {
      if constexpr (kStage)
        o[d] = mma(Tile::cols(Tile::offset(vt[b]), lane, 0, d), pr, o[d]);
      else
        o[d] = mma(vf[d], pr, o[d]);
    }
  }
  // the four waves, in their order
  sum += __shfl_xor(sum, 16);
  sum += __shfl_xor(sum, 32);
  if (g == 0) s_m[wave][li] = m, s_l[wave][li] = sum;
  __syncthreads();                                    // also: every wave has read its values
  float top = -__builtin_inff();
#pragma unroll
  for (int w = 0; w < 4; ++w) top = fmaxf(top, s_m[w][li]);
  const float a = m == top ? 1.0f : __builtin_amdgcn_exp2f((m - top) * c2);
  float *so = reinterpret_cast<float *>(s_raw);       // [4][16][D]
#pragma unroll
  for (int d = 0; d < ND; ++d) *reinterpret_cast<f32x4 *>(so + (wave * 16 + li) * D + 16 * d + 4 * g) = o[d] * a;
  __syncthreads();
  for (int i = threadIdx.x; i < heads * D / 4; i += 256) {
    f32x4 v = zero_f4();
#pragma unroll
    for (int w = 0; w < 4; ++w) v += *reinterpret_cast<const f32x4 *>(so + w * 16 * D + 4 * i);
    store4(p.part_o + out * D + 4 * i, v);
  }
  if (threadIdx.x < heads) {
    const int x = threadIdx.x;
    float M = -__builtin_inff(), L = 0.0f;
#pragma unroll
    for (int w = 0; w < 4; ++w) M = fmaxf(M, s_m[w][x]);
#pragma unroll
    for (int w = 0; w < 4; ++w) L += s_m[w][x] == M ? s_l[w][x] : s_l[w][x] * __builtin_amdgcn_exp2f((s_m[w][x] - M) * c2);
    p.part_ml[out + x] = float2{M, L};
  }
}

// Joins the ranges of keys and writes the tokens: a workgroup a row and head, D / 4 lanes an output and 1024 / D interleaved
// parts of the ranges, added in order.
template <typename T, int D> __global__ __launch_bounds__(256) void attn_step_join_kernel(AttnStepParams p) {
  constexpr int L = D / 4, G = 256 / L;
  __shared__ __attribute__((aligned(16))) float s_o[G][D];
  __shared__ float s_m[G], s_l[G];
  const int row = blockIdx.x, h = blockIdx.y, c = threadIdx.x % L, g = threadIdx.x / L;
  const int2 at = step_row(p, row);
  T *out = static_cast<T *>(p.o) + (int64_t)row * p.ldo + (int64_t)h * D + 4 * c;
  if (at.x < 0) {
    if (p.zero_unused && g == 0) store4(out, zero_f4());
    return;
  }
  const float c2 = p.scale * kLog2e;
  const int64_t first = (int64_t)row * p.heads + h, step = (int64_t)p.n * p.heads;
  float m = -__builtin_inff(), sum = 0.0f;
  f32x4 o = zero_f4();
  for (int i = g; i < p.splits; i += G) {
    const float2 ml = p.part_ml[first + i * step];
    const f32x4 sums = *reinterpret_cast<const f32x4 *>(p.part_o + (first + i * step) * D + 4 * c);
    const f32x4 x = ml.x == -__builtin_inff() && ml.y == 0.0f ? zero_f4() : sums;
    const float top = fmaxf(m, ml.x);
    const float a = m == top ? 1.0f : __builtin_amdgcn_exp2f((m - top) * c2), b = ml.x == top ? 1.0f : __builtin_amdgcn_exp2f((ml.x - top) * c2);
    m = top, sum = sum * a + ml.y * b, o = o * a + x * b;
  }
  *reinterpret_cast<f32x4 *>(&s_o[g][4 * c]) = o;
  if (c == 0) s_m[g] = m, s_l[g] = sum;
  __syncthreads();
  if (g == 0) {
    for (int i = 1; i < G; ++i) m = fmaxf(m, s_m[i]);
    sum = 0.0f, o = zero_f4();
    for (int i = 0; i < G; ++i) {
      const float a = s_m[i] == m ? 1.0f : __builtin_amdgcn_exp2f((s_m[i] - m) * c2);
      sum += s_l[i] * a;
      o += *reinterpret_cast<const f32x4 *>(&s_o[i][4 * c]) * a;
    }
    store4(out, o * (1.0f / sum));
  }
  if (h != 0) return;
  // of rows with the same place the last is written
  const int place = place_of(p, at.y);
  bool later = false;
  if (p.slots)
    for (int i = row + 1 + threadIdx.x; i < p.n; i += 256) {
      const int2 other = step_row(p, i);
      later |= other.x == at.x && place_of(p, other.y) == place;
    }
  if (__syncthreads_or(later)) return;
  constexpr int V = 16 / (int)sizeof(T);
  const int64_t to = (int64_t)at.x * p.pool_stride + (int64_t)place * p.ldc;
  for (int i = threadIdx.x; i < p.key_heads * D / V; i += 256) {
    const u32x4 a = *reinterpret_cast<const u32x4 *>(static_cast<const T *>(p.k) + (int64_t)row * p.ldk + i * V);
    const u32x4 b = *reinterpret_cast<const u32x4 *>(static_cast<const T *>(p.v) + (int64_t)row * p.ldv + i * V);
    *reinterpret_cast<u32x4 *>(static_cast<T *>(p.kc) + to + i * V) = a;
    *reinterpret_cast<u32x4 *>(static_cast<T *>(p.vc) + to + i * V) = b;
  }
}

template <typename T, int D> hipError_t go(const AttnStepParams &p, hipStream_t s) {
  const int grp = p.heads / p.key_heads;
  hipLaunchKernelGGL((attn_step_kernel<T, D>), dim3(p.n * p.key_heads * ((grp + 15) / 16) * p.splits), dim3(256), 0, s, p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((attn_step_join_kernel<T, D>), dim3(p.n, p.heads), dim3(256), 0, s, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_attention_step(const AttnStepParams &p, bool bf16, hipStream_t s) {
  if (p.n == 0) return hipSuccess;
  if (bf16) return p.d == 64 ? go<__bf16, 64>(p, s) : p.d == 128 ? go<__bf16, 128>(p, s) : go<__bf16, 256>(p, s);
  return p.d == 64 ? go<float, 64>(p, s) : p.d == 128 ? go<float, 128>(p, s) : go<float, 256>(p, s);
}

}  // namespace ttt
