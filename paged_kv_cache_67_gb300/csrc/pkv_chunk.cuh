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

#include <type_traits>

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
  float scale_log2;              // scale * log2(e)
  float cap_log2;                // 0, or cap * log2(e)
  float cap_k[4], cap_small;     // chunk_cap_fit: the near series in the raw product, and its range there
  float cap_c[6], cap_mid;       // the middle one in scale / cap (q . k), times cap * log2(e); its range in the raw product
  float scale_y;                 // scale * log2(e), or with a cap: chunk_capped's 2 log2(e) scale / cap
  float cap_ratio;               // with a cap: scale / cap (before cap_k, whose wide constant loads it would shift,
                                 // it costs capped prompts 6 %: 180 us for 169)
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

// The capped score cap tanh(x), x = scale / cap (q . k), in log2 units, off by
// a few fp32 roundings of the score itself, however large the cap.  With
// e = 2^(-2 log2(e) |x|), tanh(x) = sign(x) (1 - e) / (1 + e); below 1/4,
// where 1 - e cancels, the plain score times the Taylor series of tanh(x) / x
// through x^8 (next term 1.4e-9 of 1 at 1/4), so that a cap far above the
// scores leaves them as they are, even where scale / cap is 0 in fp32.
constexpr float kCapNear = 0.25f;
__device__ __forceinline__ float chunk_cap_near(const ChunkArgs &a, float dot) {
  const float x = dot * a.cap_ratio, t = dot * a.scale_log2, z = x * x;
  float p = fmaf(z, 62.f / 2835.f, -17.f / 315.f);
  p = fmaf(z, p, 2.f / 15.f);
  p = fmaf(z, p, -1.f / 3.f);
  return fmaf(t * z, p, t);
}
__device__ __forceinline__ float chunk_cap(const ChunkArgs &a, float dot) {
  const float x = dot * a.cap_ratio, y = fabsf(x);
  if (y < kCapNear) return chunk_cap_near(a, dot);
  const float e = exp2f(-2.f * kLog2e * y);
  return copysignf(a.cap_log2 * __fdividef(1.f - e, 1.f + e), x);
}

// The row's score of a key in log2 units from the raw product q . k.
__device__ __forceinline__ float chunk_score(const ChunkArgs &a, float dot, float slope_log2, int p, int j) {
  float t = a.cap_log2 > 0.f ? chunk_cap(a, dot) : dot * a.scale_log2;
  if (a.slopes) t = fmaf(-slope_log2, fabsf((float)(p - j)), t);
  return t;
}

// How a 16-bit kernel caps its scores, a template parameter: no cap, a cap up
// to kCapShort, a larger one.
constexpr int kCapNone = 0, kCapUsual = 1, kCapLarge = 2;

// The capped score for caps up to kCapShort, with y = 2 log2(e) scale / cap
// (q . k):  cap tanh(x) = cap - 2 cap / (1 + 2^y).  Half of it cancels near 0:
// off by some 2^-23 of the cap, which moves a weight by 3e-5 at a cap of 256, a
// sixteenth of fp16's half step.  That grows with the cap (1.2 % of a weight at
// 1e5), so larger caps take chunk_cap (kCapLarge), at a price: 64 sequences of
// 512 to 4096 keys 114 us for 105, 8 drafts with a bias 165 for 135, four
// prompt chunks 257 for 169.
constexpr float kCapShort = 256.f * kLog2e;   // in log2 units, as cap_log2
__device__ __forceinline__ float chunk_capped(float y, float cap_log2) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + fast_exp2(y)));
  return fmaf(-2.f * cap_log2, r, cap_log2);
}

// tanh(x) = x P(x^2) on the FMA pipe: P fitted to tanh(x) / x by reweighted
// least squares (towards the least maximum), relative error 6e-7 for |x| <= 1/2
// with 4 terms and 7e-7 for |x| <= 1 with 6.
constexpr float kTanh4[4] = {0.999999463558197f, -0.33326318860054016f, 0.13190296292304993f, -0.04440222308039665f};
constexpr float kTanh6[6] = {0.9999994039535522f, -0.3332904279232025f, 0.13281433284282684f,
                             -0.051605671644210815f, 0.016743112355470657f, -0.0030670592095702887f};

// Reference for a running max that may still be -inf (nothing seen yet): with
// 0 in its place every weight is 2^(-inf) = 0 and not NaN.
__device__ __forceinline__ float chunk_ref(float m) { return m == -INFINITY ? 0.f : m; }

// Element offset of key t's row of a KV head (a bad entry is flagged where it
// was first read).
__device__ __forceinline__ size_t chunk_row_at(const ChunkArgs &a, int b, int kvh, int t) {
  int phys = __ldg(a.tables + (size_t)b * a.max_blocks + t / a.bs);
  if (phys < 0 || (long long)phys >= a.num_blocks) phys = 0;
  return (((size_t)phys * a.bs + t % a.bs) * a.KVH + kvh) * a.D;
}

// One row over keys [t0, t1), all of them visible, on one warp, KEYS at a time:
// m, l and the lane's D / 32 columns of the weighted sum, unnormalised.  The
// tensor-core kernels multiply a whole tile by weights that are 0 for hidden
// keys; where a hidden value is not finite that gives NaN, and the rows that
// show one are done again here, from what they see alone.
template <typename T, int EPL, int KEYS = 1>
__device__ __forceinline__ void chunk_row_exact(const ChunkArgs &a, int b, int kvh, size_t q_row, float slope_log2, int p,
                                             int t0, int t1, float &m, float &l, float (&o)[EPL]) {
  const int lane = threadIdx.x & 31;
  const T *q = reinterpret_cast<const T *>(a.q) + q_row * a.D;
  float qv[EPL];
#pragma unroll
  for (int e = 0; e < EPL; ++e) {
    const int d = lane + 32 * e;
    qv[e] = d < a.D ? to_f32<T>(q[d]) : 0.f;
    o[e] = 0.f;
  }
  m = -INFINITY;
  l = 0.f;
  for (int t = t0; t < t1; t += KEYS) {
    size_t row[KEYS];
    float x[KEYS], mn = m;
#pragma unroll
    for (int k = 0; k < KEYS; ++k) {
      row[k] = chunk_row_at(a, b, kvh, KEYS > 1 ? min(t + k, t1 - 1) : t);
      x[k] = 0.f;
    }
#pragma unroll
    for (int k = 0; k < KEYS; ++k)
#pragma unroll
      for (int e = 0; e < EPL; ++e) {
        const int d = lane + 32 * e;
        if (d < a.D) x[k] = fmaf(qv[e], to_f32<T>((reinterpret_cast<const T *>(a.k_cache) + row[k])[d]), x[k]);
      }
#pragma unroll
    for (int w = 16; w > 0; w >>= 1)
#pragma unroll
      for (int k = 0; k < KEYS; ++k) x[k] += __shfl_xor_sync(0xffffffffu, x[k], w);
#pragma unroll
    for (int k = 0; k < KEYS; ++k) {
      x[k] = chunk_score(a, x[k], slope_log2, p, t + k);
      if (t + k < t1) mn = fmaxf(mn, x[k]);
    }
    const float ref = chunk_ref(mn), c = fast_exp2(m - ref);
    m = mn;
    l *= c;
#pragma unroll
    for (int e = 0; e < EPL; ++e) o[e] *= c;
#pragma unroll
    for (int k = 0; k < KEYS; ++k) {
      if (t + k >= t1) continue;
      const float w = fast_exp2(x[k] - ref);
      l += w;
#pragma unroll
      for (int e = 0; e < EPL; ++e) {
        const int d = lane + 32 * e;
        if (d < a.D) o[e] = fmaf(w, to_f32<T>((reinterpret_cast<const T *>(a.v_cache) + row[k])[d]), o[e]);
      }
    }
  }
}

// Four (or one) output elements of a row.
template <typename T, int VEC>
__device__ __forceinline__ void chunk_put(T *dst, const float (&v)[VEC]) {
  struct __align__(VEC * sizeof(T)) Pack {
    T e[VEC];
  } p;
#pragma unroll
  for (int i = 0; i < VEC; ++i) p.e[i] = from_f32<T>(v[i]);
  *reinterpret_cast<Pack *>(dst) = p;
}

// Joins the nparts parts of `rows` rows from the workspace, by the whole CTA:
//   M = max m_p,  out = sum o_p 2^(m_p - M) / sum l_p 2^(m_p - M).
// The weights 2^(m_p - M) / L are made once, in s_w (room for `room` floats,
// nparts or more), for as many rows at a time as fit; a round trip to L2 then
// brings kR rows x kP parts of a thread.  VEC: columns a thread takes at once
// (4: head_dim a multiple of 4, `out` aligned to 4 elements).
template <typename T, int VEC, typename RowOut, typename Seen>
__device__ void chunk_merge(const ChunkArgs &a, int rows, int nparts, float *s_w, int room, const RowOut &row_out,
                            const Seen &seen) {
  constexpr int kR = 2, kP = 8;
  const int tid = threadIdx.x, nthr = blockDim.x, warp = tid >> 5, lane = tid & 31;
  const int D = a.D, DV = D / VEC, group = min(rows, room / nparts);
  T *out = reinterpret_cast<T *>(a.out);
  for (int g0 = 0; g0 < rows; g0 += group) {
    const int gn = min(group, rows - g0);
    __syncthreads();                                  // s_w is free
    for (int r = warp; r < gn; r += nthr >> 5) {
      const size_t at = row_out(g0 + r) * a.max_parts;
      float M = -INFINITY, L = 0.f;
      for (int p = lane; p < nparts; p += 32) M = fmaxf(M, __ldcg(a.ws_m + at + p));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
      const float ref = chunk_ref(M);
      for (int p = lane; p < nparts; p += 32) {
        const float w = fast_exp2(__ldcg(a.ws_m + at + p) - ref);
        s_w[r * nparts + p] = w;
        L = fmaf(__ldcg(a.ws_l + at + p), w, L);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
      const float inv = 1.f / L;
      __syncwarp();
      for (int p = lane; p < nparts; p += 32) s_w[r * nparts + p] *= inv;
    }
    __syncthreads();
    const int tpr = min(DV, nthr);                    // threads along a row
    const int step = nthr / tpr;                      // rows side by side
    for (int dv = tid % tpr; dv < DV; dv += tpr) {
      for (int r0 = tid / tpr; r0 < gn && tid < step * tpr; r0 += step * kR) {
        float acc[kR][VEC];
        const float *po[kR];
#pragma unroll
        for (int k = 0; k < kR; ++k) {
#pragma unroll
          for (int i = 0; i < VEC; ++i) acc[k][i] = 0.f;
          po[k] = a.ws_o + row_out(g0 + min(r0 + k * step, gn - 1)) * a.max_parts * D + dv * VEC;
        }
        for (int p0 = 0; p0 < nparts; p0 += kP) {
          float v[kR][kP][VEC];
#pragma unroll
          for (int k = 0; k < kR; ++k)
#pragma unroll
            for (int p = 0; p < kP; ++p) {
              const float *src = po[k] + (size_t)min(p0 + p, nparts - 1) * D;
              if constexpr (VEC == 4) {
                const float4 x = __ldcg(reinterpret_cast<const float4 *>(src));
                v[k][p][0] = x.x; v[k][p][1] = x.y; v[k][p][2] = x.z; v[k][p][3] = x.w;
              } else {
                v[k][p][0] = __ldcg(src);
              }
            }
#pragma unroll
          for (int k = 0; k < kR; ++k)
#pragma unroll
            for (int p = 0; p < kP; ++p) {
              if (p0 + p >= nparts) continue;
              const float w = s_w[min(r0 + k * step, gn - 1) * nparts + p0 + p];
#pragma unroll
              for (int i = 0; i < VEC; ++i) acc[k][i] = fmaf(v[k][p][i], w, acc[k][i]);
            }
        }
#pragma unroll
        for (int k = 0; k < kR; ++k) {
          const int r = r0 + k * step;
          if (r >= gn) continue;
          if (!seen(g0 + r)) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) acc[k][i] = 0.f;
          }
          chunk_put<T, VEC>(out + row_out(g0 + r) * D + dv * VEC, acc[k]);
        }
      }
    }
  }
}

// Counts a finished part of a unit (every thread's partial results are
// written); whether it was the last.  One thread publishes for the CTA with
// an acquire-release atomic.  s_scratch: 1 int.
__device__ __forceinline__ bool chunk_last_part(int *counter, int nparts, int *s_scratch) {
  __syncthreads();
  if (threadIdx.x == 0) {
    int prev;
    asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;"
                 : "=r"(prev)
                 : "l"(reinterpret_cast<uint64_t>(counter))
                 : "memory");
    *s_scratch = prev == nparts - 1;
  }
  __syncthreads();
  return *s_scratch != 0;
}

// The end of part `part` of `nparts` of a unit of `rows` rows, by the whole
// CTA: s_m, s_l, s_o (row r at r * ostride) hold the part's state; row_out(r)
// is row r's output row; seen(r) says whether it sees any key at all.  One
// part writes o / l.  Several leave their state in the workspace, and the one
// that `counter` shows to be last joins them.  s_o is overwritten then
// (`room` floats).
template <typename T, typename RowOut, typename Seen>
__device__ void chunk_finish(const ChunkArgs &a, int rows, int part, int nparts, const float *s_m, const float *s_l,
                             float *s_o, int ostride, int room, int *s_scratch, int *counter, const RowOut &row_out,
                             const Seen &seen) {
  const int tid = threadIdx.x, nthr = blockDim.x, D = a.D, DV = D / 4;
  T *out = reinterpret_cast<T *>(a.out);
  if (nparts == 1) {
    for (int i = tid; i < rows * DV; i += nthr) {
      const int r = i / DV, d4 = i - r * DV;
      const float4 v = *reinterpret_cast<const float4 *>(s_o + r * ostride + 4 * d4);
      const bool sees = seen(r);
      const float inv = sees ? 1.f / s_l[r] : 0.f;
      const float x[4] = {sees ? v.x * inv : 0.f, sees ? v.y * inv : 0.f, sees ? v.z * inv : 0.f, sees ? v.w * inv : 0.f};
      chunk_put<T, 4>(out + row_out(r) * D + 4 * d4, x);
    }
    return;
  }
  for (int r = tid; r < rows; r += nthr) {
    const size_t at = row_out(r) * a.max_parts + part;
    a.ws_m[at] = s_m[r];
    a.ws_l[at] = s_l[r];
  }
  for (int i = tid; i < rows * DV; i += nthr) {
    const int r = i / DV, d4 = i - r * DV;
    reinterpret_cast<float4 *>(a.ws_o + (row_out(r) * a.max_parts + part) * D)[d4] =
        *reinterpret_cast<const float4 *>(s_o + r * ostride + 4 * d4);
  }
  if (!chunk_last_part(counter, nparts, s_scratch)) return;
  chunk_merge<T, 4>(a, rows, nparts, s_o, room, row_out, seen);
  if (tid == 0) *counter = 0;  // ready for the next call
}

// go(cap, bias) with a call's score form as constants (.value: kCap..., bool).
template <typename F>
static pkv_status chunk_forms(const ChunkArgs &a, const F &go) {
  auto biased = [&](auto cap) {
    return a.slopes ? go(cap, std::true_type()) : go(cap, std::false_type());
  };
  if (!(a.cap_log2 > 0.f)) return biased(std::integral_constant<int, kCapNone>());
  return a.cap_log2 > kCapShort ? biased(std::integral_constant<int, kCapLarge>())
                                : biased(std::integral_constant<int, kCapUsual>());
}

}  // namespace pkv
