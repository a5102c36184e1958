// pkv_chunk.cuh -- what the chunk-attention kernels share: the argument
// block, a row's visible keys, the score form, and the end of a part.
//
// Rows.  The queries of a sequence and the G query heads of a KV head are
// packed: row r of (sequence b, KV head) is query r / G', head r % G' of the
// G' heads packed together (all G, or the largest power of two dividing G for
// the tcgen05 kernel), so short chunks and grouped heads fill the same tiles
// and read each key once.
//
// Visible keys.  Causal, prefix, window and document masks together leave a
// row the one interval [lo, hi):
//   lo = max(0, p - window + 1, kv_start),   hi = max(p + 1, min(prefix, n)).
//
// Scores stay in log2 units: with sc = scale * log2(e)
//   plain    t = sc * (q . k)
//   capped   t = cap * log2(e) * tanh(scale / cap * (q . k))
//   biased   t -= slope * log2(e) * |p - j|.
#pragma once

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {

// The workspace begins with kChunkCnt counters that are zero between calls,
// whatever their shapes: two of the persistent kernel (next item, CTAs done),
// then from kChunkCntFirst one per unit of a split call (its finished parts).
// What follows them holds nothing from one call to the next.
constexpr int kChunkCnt = 65536;
constexpr int kChunkCntFirst = 16;

struct ChunkArgs {
  void *out;
  const void *q;
  const void *k_cache, *v_cache;
  const int32_t *tables, *cu_q, *lens;
  const float *slopes;           // [H] or null
  const int32_t *prefix;         // [B] or null
  const int32_t *starts;         // [total_q] or null
  int *err;
  int *ws_cnt;                   // merge counters
  float *ws_m, *ws_l, *ws_o;     // [total_q * H][max_parts] (, [D])
  long long num_blocks, total_q;
  int B, H, KVH, D, G, bs, max_blocks;
  int max_q, max_n;              // the host's bounds
  int window;
  int P, max_parts;              // keys per part, parts the workspace holds per row
  int chunks;                    // row chunks per (sequence, KV head): the grid's and the counters'
  float scale_log2;              // scale * log2(e), or with a cap: scale / cap
  float cap_log2;                // 0, or cap * log2(e)
};

struct ChunkSeq {
  int q0, qlen, n, prefix;       // qlen 0: nothing to do
};

// Sequence b's lengths after the device-side checks (reported by the caller
// with `report`): an impossible one has no queries here.
__device__ __forceinline__ ChunkSeq chunk_seq(const ChunkArgs &a, int b, bool report) {
  ChunkSeq s;
  s.q0 = __ldg(a.cu_q + b);
  s.qlen = __ldg(a.cu_q + b + 1) - s.q0;
  s.n = __ldg(a.lens + b);
  s.prefix = a.prefix ? min(max(__ldg(a.prefix + b), 0), max(s.n, 0)) : 0;
  const bool ok = s.qlen >= 0 && s.n >= s.qlen && (long long)s.n <= (long long)a.max_blocks * a.bs &&
                  s.q0 >= 0 && (long long)s.q0 + s.qlen <= a.total_q;
  if (!ok) {
    if (report) raise_flag(a.err, PKV_FLAG_QUERY_LEN);
    s.qlen = 0;
  } else if (s.qlen > a.max_q) {
    if (report) raise_flag(a.err, PKV_FLAG_QUERY_OVER_HINT);
    s.qlen = 0;
  } else if (s.n > a.max_n && s.qlen > 0) {
    if (report) raise_flag(a.err, PKV_FLAG_CONTEXT_OVER_HINT);
    s.qlen = 0;
  }
  return s;
}

// Visible keys [lo, hi) of query i of the sequence.
__device__ __forceinline__ void chunk_visible(const ChunkArgs &a, const ChunkSeq &s, int i, int &lo,
                                              int &hi) {
  const int p = s.n - s.qlen + i;
  hi = max(p + 1, s.prefix);
  lo = a.window > 0 ? max(0, p - a.window + 1) : 0;
  if (a.starts) lo = max(lo, __ldg(a.starts + s.q0 + i));
  if (lo >= hi) lo = hi = 0;
}

// tanh(x) = sign(x) (1 - e) / (1 + e), e = 2^(-2 log2(e) |x|), and below 1/4,
// where 1 - e cancels, its Taylor series through x^9 (next term 1.4e-9 of x
// at 1/4): within a few fp32 roundings everywhere.
__device__ __forceinline__ float chunk_tanh(float x) {
  const float y = fabsf(x);
  if (y < 0.25f) {
    const float z = x * x;
    float p = fmaf(z, 62.f / 2835.f, -17.f / 315.f);
    p = fmaf(z, p, 2.f / 15.f);
    p = fmaf(z, p, -1.f / 3.f);
    return fmaf(x * z, p, x);
  }
  const float e = exp2f(-2.f * kLog2e * y);
  return copysignf(__fdividef(1.f - e, 1.f + e), x);
}

// The row's score of a key in log2 units from the raw product q . k.
__device__ __forceinline__ float chunk_score(const ChunkArgs &a, float dot, float slope_log2, int p, int j) {
  float t = dot * a.scale_log2;
  if (a.cap_log2 > 0.f) t = a.cap_log2 * chunk_tanh(t);
  if (a.slopes) t = fmaf(-slope_log2, fabsf((float)(p - j)), t);
  return t;
}

}  // namespace pkv
