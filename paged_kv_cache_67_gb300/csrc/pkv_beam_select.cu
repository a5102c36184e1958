// pkv_beam_select.cu -- one step of beam search: the K best of W beams x V
// tokens by c_w + x_wv - log sum exp x_w.
//
// Within a beam the order is that of its logits, so a row can be cut into
// pieces that each give their K largest logits and a share of the sum, in one
// pass over the row.  A CTA holds its piece in registers:
//   1. load; maximum m of the piece, sum of 2^(x L - fl(m L)), L = log2 e: the
//      rounding of m L is in the piece's unit, so the sum carries none of it.
//      Where that rounding is no longer small (|m| >= 2^15: it grows with m, and
//      2^ of it with that) sums of 2^((x - m) L), whose difference carries none;
//   2. a bound: the K-th largest of the 256 threads' maxima has K elements at or
//      above it.  Each warp takes its K largest maxima off, one warp-wide maximum
//      at a time, then all do so with the eight warps' lists;
//   3. the elements at or above the bound (K, and a few more) go to shared memory
//      as 64-bit keys -- the logit's bits in their order, then the lowest token --
//      and each counts the keys above its own: its rank.
//      (With the largest of the warps' own bounds some 50 elements came through:
//      64 x 8 beams x 128256 tokens took 113 us.)
// 64 x 8 beams x 128256 bf16: 67 us (116 MB), bound by instructions and the
// barriers between the passes (two issued a cycle); 4 x 32000 fp32: 15 us, latency.
//
// The CTA that finishes a request's last piece joins: a warp a beam merges the
// pieces' sorted keys (lane = piece, K rounds of a warp-wide maximum) and adds
// up the sums in 64 bits; one warp then merges the beams' lists by score in 64
// bits (lane = beam).  Every logit is read once.
//
// Which token comes first must not hang on where a row starts in memory: beams
// with equal logits have to tie.  So thread t of piece i takes the same
// elements of every row, and rows that are not 16-byte aligned are read by
// aligned granules, two for one, and shifted.
#include <algorithm>
#include <type_traits>

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {

constexpr int kBsThreads = 256;
constexpr int kBsWarps = kBsThreads / 32;
constexpr int kBsMost = 32;              // beams, continuations
constexpr int kBsKeys = 512;             // keys of a piece that are ranked by counting
constexpr int kBsParts = 256;            // pieces of a row
constexpr int kBsList = 128;             // keys of a beam's pieces that a warp merges in shared memory
constexpr int kBsSms = 152;              // of the one GPU this library is built for (speed alone)
constexpr long long kBsMaxV = 1LL << 21;
constexpr int kBsMaxB = 16384;

struct BeamSelectArgs {
  float *scores_out;
  int32_t *parents, *tokens;
  uint8_t *finished_out;
  const char *logits;
  const float *scores;
  const uint8_t *finished;
  int *err;
  int *cnt;                              // [B] finished pieces
  unsigned long long *keys;              // [B * W][parts][K]
  double *sums;                          // [B * W][parts]
  float *maxima;                         // [B * W][parts]; NaN: not a number among them
  long long V, stride;
  int W, K, parts, end;
};

// The bits of x in the order of its values (-0 as 0).
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float from_ordered(uint32_t u) {
  return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u);
}
// Larger: the larger logit, of equal ones the lower token.  0: none.
__device__ __forceinline__ unsigned long long beam_key(float x, uint32_t v) {
  return ((unsigned long long)ordered(x) << 32) | (0xffffffffu - v);
}

// Whether a beam's row is to be read.
__device__ __forceinline__ bool beam_live(const BeamSelectArgs &a, long long row) {
  if (a.finished && __ldg(a.finished + row)) return false;
  const float c = __ldg(a.scores + row);
  return c > -INFINITY && c < INFINITY;  // (NaN and +inf are flagged where the request is joined)
}

template <typename T>
constexpr uint32_t kMinusInf = sizeof(T) == 4 ? 0xff800000u : std::is_same<T, __half>::value ? 0xfc00fc00u : 0xff80ff80u;

// 16 bytes from p on, `off` behind an aligned place (off > 0: two aligned loads).
__device__ __forceinline__ uint4 shifted_granule(const char *from, uint32_t off) {
  const uint4 *p = reinterpret_cast<const uint4 *>(from - off);
  const uint4 x = __ldg(p), y = __ldg(p + 1);
  uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
  const uint32_t words = off >> 2;
  if (words & 2)
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
  if (words & 1)
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
  const uint32_t bits = (off & 3) * 8;
  return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits),
                    __funnelshift_r(w[2], w[3], bits), __funnelshift_r(w[3], w[4], bits));
}

// 16 bytes of a row from byte `at` on (a multiple of 16, counted from the
// row's start), whatever the row's alignment; -inf past its end.
template <typename T>
__device__ __forceinline__ uint4 row_granule(const char *row, long long at, long long bytes) {
  const uint32_t off = (uint32_t)(reinterpret_cast<uintptr_t>(row) & 15);
  if (off == 0 && at + 16 <= bytes) return __ldg(reinterpret_cast<const uint4 *>(row + at));
  if (off != 0 && at >= 16 && at + 32 <= bytes) return shifted_granule(row + at, off);
  // the row's ends, element by element
  constexpr int kPer = 16 / sizeof(T);
  union {
    uint4 v;
    uint16_t h[8];
    uint32_t w[4];
  } u;
  u.v = make_uint4(kMinusInf<T>, kMinusInf<T>, kMinusInf<T>, kMinusInf<T>);
#pragma unroll
  for (int e = 0; e < kPer; ++e) {
    const long long b = at + e * (long long)sizeof(T);
    if (b >= bytes) continue;
    if constexpr (sizeof(T) == 2)
      u.h[e] = __ldg(reinterpret_cast<const unsigned short *>(row + b));
    else
      u.w[e] = __ldg(reinterpret_cast<const unsigned int *>(row + b));
  }
  return u.v;
}

template <typename T>
__device__ __forceinline__ float granule_at(const uint4 &g, int e) {
  const uint32_t w[4] = {g.x, g.y, g.z, g.w};
  if constexpr (sizeof(T) == 4) return __uint_as_float(w[e]);
  const uint32_t h = e & 1 ? w[e >> 1] >> 16 : w[e >> 1] & 0xffffu;
  if constexpr (std::is_same<T, __nv_bfloat16>::value) return __uint_as_float(h << 16);
  return __half2float(__ushort_as_half((unsigned short)h));
}

// The largest element of a granule; NaN if there is one.
template <typename T>
__device__ __forceinline__ float granule_max(const uint4 &g) {
  if constexpr (sizeof(T) == 4) {
    float r;
    asm("{.reg .f32 a, b;\n\tmax.NaN.f32 a, %1, %2;\n\tmax.NaN.f32 b, %3, %4;\n\tmax.NaN.f32 %0, a, b;}"
        : "=f"(r) : "f"(__uint_as_float(g.x)), "f"(__uint_as_float(g.y)), "f"(__uint_as_float(g.z)), "f"(__uint_as_float(g.w)));
    return r;
  } else if constexpr (std::is_same<T, __half>::value) {
    uint32_t r;
    asm("{.reg .b32 a, b;\n\tmax.NaN.f16x2 a, %1, %2;\n\tmax.NaN.f16x2 b, %3, %4;\n\tmax.NaN.f16x2 %0, a, b;}"
        : "=r"(r) : "r"(g.x), "r"(g.y), "r"(g.z), "r"(g.w));
    const __half2 h = *reinterpret_cast<const __half2 *>(&r);
    return __half2float(__hmax_nan(__low2half(h), __high2half(h)));
  } else {
    uint32_t r;
    asm("{.reg .b32 a, b;\n\tmax.NaN.bf16x2 a, %1, %2;\n\tmax.NaN.bf16x2 b, %3, %4;\n\tmax.NaN.bf16x2 %0, a, b;}"
        : "=r"(r) : "r"(g.x), "r"(g.y), "r"(g.z), "r"(g.w));
    const __nv_bfloat162 h = *reinterpret_cast<const __nv_bfloat162 *>(&r);
    return __bfloat162float(__hmax_nan(__low2bfloat16(h), __high2bfloat16(h)));
  }
}

__device__ __forceinline__ unsigned long long warp_max_u64(unsigned long long x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const unsigned long long y = __shfl_xor_sync(0xffffffffu, x, o);
    x = y > x ? y : x;
  }
  return x;
}

// The sums' unit is 2^(m L), L = log2 e as fp32 has it, the product as fp32
// rounds it (by 2^-9 at most: a term is below 1.002); from kBsFar on, exact.
constexpr float kBsFar = 32768.f;
__device__ __forceinline__ double beam_unit(float m) {
  return fabsf(m) < kBsFar ? (double)(m * kLog2e) : (double)m * (double)kLog2e;
}

// The request's K best from its pieces, by the whole CTA.
__device__ __noinline__ void beam_join(const BeamSelectArgs &a, int b, unsigned long long (*s_list)[kBsList]) {
  __shared__ unsigned long long s_key[kBsMost][kBsMost];   // a beam's best, sorted
  __shared__ double s_base[kBsMost];                       // c - log sum exp(x - m); finished beams: c
  __shared__ float s_top[kBsMost];                         // m, the largest logit
  __shared__ int s_mode[kBsMost];                          // 0 no proposals, 1 its tokens, 2 itself
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, K = a.K, parts = a.parts;
  for (int w = warp; w < a.W; w += kBsWarps) {
    const long long row = (long long)b * a.W + w;
    const float c = __ldg(a.scores + row);
    const bool done = a.finished && __ldg(a.finished + row);
    int mode = c > -INFINITY && c < INFINITY ? (done ? 2 : 1) : 0;
    bool bad = !(c < INFINITY);
    double base = c;
    float m = -INFINITY;
    if (mode == 1) {
      bool nan = false;
      for (int i = lane; i < parts; i += 32) {
        const float x = __ldcg(a.maxima + row * parts + i);
        nan = nan || !(x < INFINITY);
        m = fmaxf(m, x);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      nan = __any_sync(0xffffffffu, nan);
      double sum = 0.0;
      if (m > -INFINITY)
        for (int i = lane; i < parts; i += 32) {
          const float x = __ldcg(a.maxima + row * parts + i);
          if (x > -INFINITY) sum += __ldcg(a.sums + row * parts + i) * exp2(beam_unit(x) - beam_unit(m));
        }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      bad = nan;
      if (nan || m == -INFINITY) mode = 0;
      base = (double)c - ((beam_unit(m) - (double)m * (double)kLog2e) / (double)kLog2e + log(sum));
    }
    if (mode == 1) {
      // lane = piece (32 apart): its next key not yet taken.  Short lists come
      // to shared memory first: a round then waits for no load from L2.
      const unsigned long long *keys = a.keys + row * parts * K;
      const bool near = parts * K <= kBsList;
      if (near) {
        __syncwarp();
        for (int i = lane; i < parts * K; i += 32) s_list[warp][i] = __ldcg(keys + i);
        __syncwarp();
        if (parts <= 32) {
          unsigned long long head = lane < parts ? s_list[warp][lane * K] : 0;
          int taken = 0;
          for (int k = 0; k < K; ++k) {
            const unsigned long long best = warp_max_u64(head);
            if (lane == 0) s_key[w][k] = best;
            if (best != 0 && head == best) {             // (keys differ: one lane has it)
              ++taken;
              head = taken < K ? s_list[warp][lane * K + taken] : 0;
            }
          }
        }
      }
      if (!near || parts > 32) {
        unsigned long long head[kBsParts / 32];
        uint32_t taken[kBsParts / 32];
#pragma unroll
        for (int j = 0; j < kBsParts / 32; ++j) {
          const int i = lane + 32 * j;
          taken[j] = 0;
          head[j] = i < parts ? __ldcg(keys + (long long)i * K) : 0;
        }
        for (int k = 0; k < K; ++k) {
          unsigned long long best = 0;
#pragma unroll
          for (int j = 0; j < kBsParts / 32; ++j) best = head[j] > best ? head[j] : best;
          best = warp_max_u64(best);
          if (lane == 0) s_key[w][k] = best;
#pragma unroll
          for (int j = 0; j < kBsParts / 32; ++j)
            if (best != 0 && head[j] == best) {
              ++taken[j];
              head[j] = taken[j] < K ? __ldcg(keys + (long long)(lane + 32 * j) * K + taken[j]) : 0;
            }
        }
      }
    }
    if (lane == 0) {
      s_mode[w] = mode;
      s_base[w] = base;
      s_top[w] = m;
      if (bad) raise_flag(a.err, PKV_FLAG_LOGITS);
    }
  }
  __syncthreads();
  if (warp != 0) return;
  // lane = beam: its best proposal not yet taken, -inf: none left.  (A score goes
  // by the difference from the largest logit: of any size, they cancel exactly.)
  const int w = lane;
  const int mode = w < a.W ? s_mode[w] : 0;
  int at = 0;
  auto head_score = [&]() {
    if (mode == 2) return at == 0 ? s_base[w] : -INFINITY;
    if (mode == 0 || at >= K || s_key[w][at] == 0) return (double)-INFINITY;
    return s_base[w] + ((double)from_ordered((uint32_t)(s_key[w][at] >> 32)) - (double)s_top[w]);
  };
  double head = head_score();
  for (int k = 0; k < K; ++k) {
    double best = head;
    int from = lane;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const double x = __shfl_xor_sync(0xffffffffu, best, o);
      const int i = __shfl_xor_sync(0xffffffffu, from, o);
      if (x > best || (x == best && i < from)) {
        best = x;
        from = i;
      }
    }
    if (lane == from) {
      const bool none = best == -INFINITY;
      const int token = none ? -1 : mode == 2 ? a.end : (int)(0xffffffffu - (uint32_t)s_key[w][at]);
      const long long out = (long long)b * K + k;
      a.scores_out[out] = (float)best;
      a.parents[out] = none ? -1 : w;
      a.tokens[out] = token;
      a.finished_out[out] = !none && (mode == 2 || token == a.end);
      ++at;
      head = head_score();
    }
    __syncwarp();
  }
}

// GRANULES 16-byte granules a thread: a piece is kBsThreads * GRANULES of them;
// HELD: the warps' lists' entries that a lane holds, 4 HELD >= K.
template <typename T, int GRANULES, int HELD>
__global__ void __launch_bounds__(kBsThreads, 4) pkv_beam_select_kernel(const __grid_constant__ BeamSelectArgs a) {
  constexpr int kPer = 16 / sizeof(T), E = GRANULES * kPer;
  constexpr long long kPiece = (long long)kBsThreads * E;
  __shared__ float s_f[kBsWarps];
  __shared__ uint32_t s_top[kBsWarps * kBsMost];
  __shared__ unsigned long long s_d[kBsWarps];
  __shared__ int s_n, s_last;
  __shared__ unsigned long long s_keys[kBsKeys];
  __shared__ unsigned long long s_list[kBsWarps][kBsList];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long long row = blockIdx.x / a.parts;
  const int part = (int)(blockIdx.x - row * a.parts), b = (int)(row / a.W);
  if (beam_live(a, row)) {
    const char *base = a.logits + row * a.stride * (long long)sizeof(T);
    const long long bytes = a.V * (long long)sizeof(T), first = part * kPiece;
    uint4 g[GRANULES];
    // inside the row every granule is a load, or two and a shift
    const uint32_t off = (uint32_t)(reinterpret_cast<uintptr_t>(base) & 15);
    const bool inside = (first + kPiece) * (long long)sizeof(T) + 16 <= bytes;
    if (off == 0 && inside) {
#pragma unroll
      for (int i = 0; i < GRANULES; ++i)
        g[i] = __ldg(reinterpret_cast<const uint4 *>(base + first * (long long)sizeof(T)) + i * kBsThreads + tid);
    } else if (part > 0 && inside) {
#pragma unroll
      for (int i = 0; i < GRANULES; ++i)
        g[i] = shifted_granule(base + (first + (long long)(i * kBsThreads + tid) * kPer) * (long long)sizeof(T), off);
    } else {
#pragma unroll
      for (int i = 0; i < GRANULES; ++i) {
        const long long at = (first + (long long)(i * kBsThreads + tid) * kPer) * (long long)sizeof(T);
        g[i] = row_granule<T>(base, at, bytes);
      }
    }
    auto token = [&](int i, int e) { return (uint32_t)first + (uint32_t)(i * kBsThreads + tid) * kPer + e; };
    if (tid == 0) s_n = 0;
    // 1. maximum (NaN where there is one) and sum
    float m = -INFINITY;
    bool nan = false;
#pragma unroll
    for (int i = 0; i < GRANULES; ++i) {
      const float x = granule_max<T>(g[i]);
      nan = nan || !(x < INFINITY);
      m = fmaxf(m, x);
    }
    const float mine = m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    // 2. the warp's K largest of its lanes' maxima, largest first
    uint32_t u = ordered(mine);
    for (int k = 0; k < a.K; ++k) {
      const uint32_t best = __reduce_max_sync(0xffffffffu, u);
      const int from = __ffs(__ballot_sync(0xffffffffu, u == best)) - 1;
      if (lane == from) {
        s_top[warp * a.K + k] = best;
        u = 0;                                             // (below every number's)
      }
    }
    if (lane == 0) s_f[warp] = m;
    const bool any_nan = __syncthreads_or(nan);
#pragma unroll
    for (int k = 0; k < kBsWarps; ++k) m = fmaxf(m, s_f[k]);
    // ... and the K-th of the 8 K: the bound
    uint32_t held[HELD];
#pragma unroll
    for (int j = 0; j < HELD; ++j) held[j] = lane + 32 * j < kBsWarps * a.K ? s_top[lane + 32 * j] : 0;
    for (int k = 0; k < a.K; ++k) {
      uint32_t top = 0;
#pragma unroll
      for (int j = 0; j < HELD; ++j) top = max(top, held[j]);
      u = __reduce_max_sync(0xffffffffu, top);
      const int from = __ffs(__ballot_sync(0xffffffffu, top == u)) - 1;
      if (lane == from) {
        bool gone = false;
#pragma unroll
        for (int j = 0; j < HELD; ++j)
          if (!gone && held[j] == u) {
            held[j] = 0;
            gone = true;
          }
      }
    }
    u = max(u, ordered(-INFINITY));                        // (threads past the row's end have nothing)
    // (a thread's sum in fp32, threads' sums in whole numbers)
    float sum = 0.f;
    const float unit = m > -INFINITY ? m * kLog2e : 0.f;
    auto add_up = [&](auto term) {
#pragma unroll
      for (int i = 0; i < GRANULES; ++i) {
        float part_sum = 0.f;
#pragma unroll
        for (int e = 0; e < kPer; ++e) part_sum += fast_exp2(term(granule_at<T>(g[i], e)));
        sum += part_sum;
      }
    };
    if (fabsf(m) >= kBsFar && m > -INFINITY)
      add_up([&](float x) { return (x - m) * kLog2e; });
    else
      add_up([&](float x) { return fmaf(x, kLog2e, -unit); });
    // a thread's sum is at most 64 and a little: whole units of 2^-20 and of 2^-40
    // add up exactly, in any order, and stay out of the way of the few FP64 units
    const float whole = floorf(sum * 0x1p20f);
    const uint32_t units = __reduce_add_sync(0xffffffffu, (uint32_t)whole);
    const uint32_t parts = __reduce_add_sync(0xffffffffu, (uint32_t)((sum * 0x1p20f - whole) * 0x1p20f));
    if (lane == 0) s_d[warp] = ((unsigned long long)units << 20) + parts;
    // 3. what is at or above the bound, -inf excepted
    const float bound = from_ordered(u);
    if (!any_nan && mine >= bound && mine > -INFINITY) {
#pragma unroll
      for (int i = 0; i < GRANULES; ++i) {
        if (!(granule_max<T>(g[i]) >= bound)) continue;
        uint32_t hits = 0;
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
          const float x = granule_at<T>(g[i], e);
          hits |= x >= bound && x > -INFINITY ? 1u << e : 0u;
        }
        while (hits) {
          const int e = __ffs(hits) - 1, word = sizeof(T) == 4 ? e : e >> 1;
          hits &= hits - 1;
          const uint32_t bits = word < 2 ? (word == 0 ? g[i].x : g[i].y) : (word == 2 ? g[i].z : g[i].w);
          const float x = granule_at<T>(make_uint4(bits, bits, 0, 0), sizeof(T) == 4 ? 0 : e & 1);
          const int n = atomicAdd(&s_n, 1);
          if (n < kBsKeys) s_keys[n] = beam_key(x, token(i, e));
        }
      }
    }
    __syncthreads();
    const int n = s_n;
    const long long out = row * a.parts + part;
    if (tid == kBsThreads - 1) {
      unsigned long long total = 0;
#pragma unroll
      for (int k = 0; k < kBsWarps; ++k) total += s_d[k];
      a.maxima[out] = any_nan ? __int_as_float(0x7fc00000) : m;
      a.sums[out] = (double)total * 0x1p-40;
    }
    unsigned long long *keys = a.keys + out * a.K;
    if (n <= kBsKeys) {
      for (int i = tid; i < n; i += kBsThreads) {
        const unsigned long long key = s_keys[i];
        int rank = 0;
        for (int j = 0; j < n; ++j) rank += s_keys[j] > key;
        if (rank < a.K) keys[rank] = key;
      }
      for (int i = n + tid; i < a.K; i += kBsThreads) keys[i] = 0;
    } else {
      // that many ties at the bound: one at a time, the largest key below the last
      unsigned long long last = ~0ull;
      // (read again: rare, and no reason to hold every element apart)
      for (int k = 0; k < a.K; ++k) {
        unsigned long long best = 0;
#pragma unroll 1
        for (int i = 0; i < E; ++i) {
          const long long v = first + (long long)i * kBsThreads + tid;
          if (v >= a.V) break;
          const float x = to_f32<T>(reinterpret_cast<const T *>(base)[v]);
          const unsigned long long key = x > -INFINITY ? beam_key(x, (uint32_t)v) : 0;
          if (key < last && key > best) best = key;
        }
        best = warp_max_u64(best);
        __syncthreads();
        if (lane == 0) s_keys[warp] = best;
        __syncthreads();
        for (int j = 0; j < kBsWarps; ++j) best = s_keys[j] > best ? s_keys[j] : best;
        if (tid == 0) keys[k] = best;
        last = best;
      }
    }
  }
  // the request's last piece joins them
  __syncthreads();
  if (tid == 0) {
    int prev;
    asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;"
                 : "=r"(prev)
                 : "l"(reinterpret_cast<uint64_t>(a.cnt + b))
                 : "memory");
    s_last = prev == a.W * a.parts - 1;
    if (s_last) a.cnt[b] = 0;                              // ready for the next call
  }
  __syncthreads();
  if (s_last) beam_join(a, b, s_list);
}

struct BeamPlan {
  int granules, parts;
};
// Pieces of a row, `granules` a thread.
static long long beam_parts(int granules, long long V, int el) {
  const long long piece = (long long)kBsThreads * granules * (16 / el);
  return (V + piece - 1) / piece;
}
// Pieces of 2 granules a thread where 8 would not give every SM two CTAs.
static BeamPlan beam_plan(long long rows, long long V, int el) {
  const bool large = rows * beam_parts(8, V, el) >= 2 * kBsSms || beam_parts(2, V, el) > kBsParts;
  const int granules = large ? 8 : 2;
  return {granules, (int)beam_parts(granules, V, el)};
}
// The most pieces that a call of these or any smaller sizes has: fewer rows are
// cut into small pieces again, four of them for a large one at most, of which
// there are fewer than two an SM then.
static long long beam_most_pieces(long long rows, long long V) {
  const long long small = rows * std::min<long long>(beam_parts(2, V, 4), kBsParts);
  return std::max(rows * beam_parts(8, V, 4), std::min<long long>(small, 4 * (2 * kBsSms - 1)));
}

constexpr size_t kBsCntBytes = kBsMaxB * sizeof(int);
static size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
static size_t beam_ws_bytes(long long pieces, int K) {
  return kBsCntBytes + align256((size_t)pieces * K * sizeof(unsigned long long)) +
         align256((size_t)pieces * sizeof(double)) + align256((size_t)pieces * sizeof(float));
}
static bool beam_sizes_ok(int B, int W, int K, int64_t V) { return B >= 0 && W > 0 && K > 0 && V > 0; }

}  // namespace pkv

using namespace pkv;

extern "C" {

PKV_API size_t pkv_beam_select_workspace_size(int B, int W, int K, int64_t V) {
  if (!beam_sizes_ok(B, W, K, V) || W > kBsMost || K > kBsMost || V > kBsMaxV || B > kBsMaxB) return 0;
  return beam_ws_bytes(beam_most_pieces((long long)B * W, V), K);
}

PKV_API pkv_status pkv_beam_select(float *scores_out, int32_t *parents, int32_t *tokens, uint8_t *finished_out,
                                   const void *logits, const float *scores, const uint8_t *finished, int B, int W,
                                   int K, int64_t V, int64_t row_stride, int end_token, pkv_dtype dt, void *workspace,
                                   size_t workspace_bytes, int *err_flags, pkv_stream_t stream) {
  if (!beam_sizes_ok(B, W, K, V) || row_stride < V || end_token < -1 || end_token >= V ||
      (dt != PKV_F32 && dt != PKV_BF16 && dt != PKV_F16))
    return PKV_ERR_INVALID_ARG;
  if (W > kBsMost || K > kBsMost || V > kBsMaxV || B > kBsMaxB) return PKV_ERR_UNSUPPORTED;
  if (B == 0) return PKV_OK;
  if (!scores_out || !parents || !tokens || !finished_out || !logits || !scores) return PKV_ERR_INVALID_ARG;
  auto at = [](const void *p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; };
  const int el = dt == PKV_F32 ? 4 : 2;
  if (!at(scores_out, 4) || !at(parents, 4) || !at(tokens, 4) || !at(scores, 4) || !at(err_flags, 4) || !at(logits, el))
    return PKV_ERR_INVALID_ARG;
  const long long rows = (long long)B * W;
  const BeamPlan plan = beam_plan(rows, V, el);
  const size_t need = beam_ws_bytes(rows * plan.parts, K);
  if (!workspace || workspace_bytes < need || !at(workspace, 256)) return PKV_ERR_WORKSPACE;
  const size_t outs = (size_t)B * K, ins = (size_t)rows;
  const ArgRange written[] = {{scores_out, outs * 4}, {parents, outs * 4}, {tokens, outs * 4}, {finished_out, outs}, {workspace, need}};
  const ArgRange read[] = {{scores, ins * 4}, {finished, ins}, {logits, (size_t)((rows - 1) * row_stride + V) * el}, {err_flags, 4}};
  for (int i = 0; i < 5; ++i) {
    for (int j = 0; j < 4; ++j) {
      const bool same = K == W && ((i == 0 && j == 0 && scores_out == scores) || (i == 3 && j == 1 && finished_out == finished));
      if (!same && overlap(written[i], read[j])) return PKV_ERR_INVALID_ARG;
    }
    for (int j = i + 1; j < 5; ++j)
      if (overlap(written[i], written[j])) return PKV_ERR_INVALID_ARG;
  }
  if (rows * plan.parts > 0x7fffffffLL) return PKV_ERR_UNSUPPORTED;
  BeamSelectArgs a = {};
  a.scores_out = scores_out;
  a.parents = parents;
  a.tokens = tokens;
  a.finished_out = finished_out;
  a.logits = static_cast<const char *>(logits);
  a.scores = scores;
  a.finished = finished;
  a.err = err_flags;
  char *ws = static_cast<char *>(workspace);
  a.cnt = reinterpret_cast<int *>(ws);
  ws += kBsCntBytes;
  a.keys = reinterpret_cast<unsigned long long *>(ws);
  ws += align256((size_t)rows * plan.parts * K * sizeof(unsigned long long));
  a.sums = reinterpret_cast<double *>(ws);
  ws += align256((size_t)rows * plan.parts * sizeof(double));
  a.maxima = reinterpret_cast<float *>(ws);
  a.V = V;
  a.stride = row_stride;
  a.W = W;
  a.K = K;
  a.parts = plan.parts;
  a.end = end_token;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const unsigned grid = (unsigned)(rows * plan.parts);
  auto go = [&](auto type) {
    using T = decltype(type);
    auto held = [&](auto n) {
      if (plan.granules == 8)
        pkv_beam_select_kernel<T, 8, decltype(n)::value><<<grid, kBsThreads, 0, s>>>(a);
      else
        pkv_beam_select_kernel<T, 2, decltype(n)::value><<<grid, kBsThreads, 0, s>>>(a);
    };
    if (K <= 4)
      held(std::integral_constant<int, 1>());
    else if (K <= 8)
      held(std::integral_constant<int, 2>());
    else
      held(std::integral_constant<int, kBsMost / 4>());
  };
  if (dt == PKV_F32)
    go(float());
  else if (dt == PKV_BF16)
    go(__nv_bfloat16());
  else
    go(__half());
  return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // extern "C"
