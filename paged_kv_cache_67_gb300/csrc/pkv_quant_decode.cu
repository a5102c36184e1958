// pkv_quant_decode.cu -- host side of the decode over a quantised cache, and
// its CUDA-core kernel, which takes every shape (see pkv_quant_decode.cuh).
#include <float.h>
#include <math.h>
#include <string.h>

#include <algorithm>

#include "pkv_quant_decode.cuh"

namespace pkv {

constexpr int kQdSms = 152;          // the plan's: of the one GPU this library is built for
constexpr int kQdHeads = 4;          // query heads of a CUDA-core CTA
constexpr int kQdWarps = 8;
constexpr int kQdMaxParts = 256;
constexpr int kQdAutoParts = 64;
constexpr long long kQdMaxKeys = 1LL << 30;

// CUDA cores: warp w takes keys w, w + 8, ... of the part; its lanes hold the
// columns lane, lane + 32, ... of every head's query and sum.
template <typename T, int FMT, int EPL>
__global__ void __launch_bounds__(32 * kQdWarps) pkv_quant_decode_simt_kernel(const __grid_constant__ QuantDecodeArgs a) {
  extern __shared__ __align__(16) float s_o[];     // [warps][heads][D], then the join's weights
  __shared__ float s_wm[kQdWarps][kQdHeads], s_wl[kQdWarps][kQdHeads], s_m[kQdHeads], s_l[kQdHeads];
  __shared__ int s_scratch[1];
  const ChunkArgs &c = a.c;
  const QuantPart p = quant_part(a);
  if (p.nparts == 0) return;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, D = c.D;
  float q[kQdHeads][EPL], o[kQdHeads][EPL], m[kQdHeads], l[kQdHeads];
#pragma unroll
  for (int h = 0; h < kQdHeads; ++h) {
    m[h] = -INFINITY;
    l[h] = 0.f;
#pragma unroll
    for (int e = 0; e < EPL; ++e) {
      const int d = lane + 32 * e;
      o[h][e] = 0.f;
      q[h][e] = h < p.rows && d < D
                    ? to_f32<T>(reinterpret_cast<const T *>(c.q)[((size_t)p.b * c.H + p.head0 + h) * D + d]) : 0.f;
    }
  }
  auto code = [&](const uint8_t *row, int d, float zero) {
    if constexpr (FMT == kInt8) return (float)(int8_t)__ldg(row + d);
    if constexpr (FMT == kE4m3) return half2_to_float2(e4m3x2_to_half2(__ldg(row + d))).x;
    return (float)((__ldg(row + d / 2) >> (d & 1 ? 4 : 0)) & 15) - zero;
  };
  for (int t = max(p.t0, p.lo) + w; t < p.t1; t += kQdWarps) {
    const long long slot = quant_slot(c, p.b, t);
    if (slot < 0) continue;
    const long long blk = slot / c.bs, row = slot * c.KVH + p.kvh;
    const long long at = ((blk * c.KVH + p.kvh) * c.bs + (slot - blk * c.bs)) * quant_params<FMT>();
    const float ks = __ldg(a.kp + at), vs = __ldg(a.vp + at);
    const float kz = FMT == kInt4 ? __ldg(a.kp + at + 1) : 0.f, vz = FMT == kInt4 ? __ldg(a.vp + at + 1) : 0.f;
    const uint8_t *kr = a.k + row * quant_row_bytes<FMT>(D), *vr = a.v + row * quant_row_bytes<FMT>(D);
    float x[kQdHeads] = {}, v[EPL];
#pragma unroll
    for (int e = 0; e < EPL; ++e) {
      const int d = lane + 32 * e;
      const float k = d < D ? code(kr, d, kz) : 0.f;
      v[e] = d < D ? code(vr, d, vz) * vs : 0.f;
#pragma unroll
      for (int h = 0; h < kQdHeads; ++h) x[h] = fmaf(q[h][e], k, x[h]);
    }
#pragma unroll
    for (int s = 16; s > 0; s >>= 1)
#pragma unroll
      for (int h = 0; h < kQdHeads; ++h) x[h] += __shfl_xor_sync(0xffffffffu, x[h], s);
#pragma unroll
    for (int h = 0; h < kQdHeads; ++h) {
      const float y = quant_score(c, x[h] * ks), mn = fmaxf(m[h], y), ref = chunk_ref(mn);
      const float f = exp2f(m[h] - ref), g = exp2f(y - ref);
      m[h] = mn;
      l[h] = fmaf(l[h], f, g);
#pragma unroll
      for (int e = 0; e < EPL; ++e) o[h][e] = fmaf(o[h][e], f, g * v[e]);
    }
  }
  if (lane == 0)
#pragma unroll
    for (int h = 0; h < kQdHeads; ++h) {
      s_wm[w][h] = m[h];
      s_wl[w][h] = l[h];
    }
  __syncthreads();
#pragma unroll
  for (int h = 0; h < kQdHeads; ++h) {
    float M = -INFINITY, L = 0.f;
    for (int i = 0; i < kQdWarps; ++i) M = fmaxf(M, s_wm[i][h]);
    const float ref = chunk_ref(M);
    for (int i = 0; i < kQdWarps; ++i) L += s_wl[i][h] * exp2f(s_wm[i][h] - ref);
    if (threadIdx.x == 0) {
      s_m[h] = M;
      s_l[h] = L;
    }
    const float f = exp2f(m[h] - ref);
#pragma unroll
    for (int e = 0; e < EPL; ++e)
      if (lane + 32 * e < D) s_o[(w * kQdHeads + h) * D + lane + 32 * e] = o[h][e] * f;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < kQdHeads * D; i += 32 * kQdWarps) {
    float sum = 0.f;
    for (int k = 0; k < kQdWarps; ++k) sum += s_o[k * kQdHeads * D + i];
    s_o[i] = sum;
  }
  __syncthreads();
  quant_finish<T>(c, p, s_m, s_l, s_o, D, max(kQdWarps * kQdHeads * D, kQdMaxParts), s_scratch);
}

template <typename T, int FMT, int EPL>
static pkv_status launch_simt_e(const QuantDecodeArgs &a, cudaStream_t stream) {
  static int configured[64];
  auto kern = pkv_quant_decode_simt_kernel<T, FMT, EPL>;
  // (the join needs room for the weights of one row's parts)
  const size_t smem = std::max<size_t>((size_t)kQdWarps * kQdHeads * a.c.D, kQdMaxParts) * sizeof(float);
  if (!allow_smem(kern, smem, configured)) return PKV_ERR_CUDA;
  kern<<<dim3((unsigned)(a.c.chunks * a.c.KVH * a.c.max_parts), (unsigned)a.c.B), 32 * kQdWarps, smem, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

template <typename T, int FMT>
static pkv_status launch_simt_f(const QuantDecodeArgs &a, cudaStream_t stream) {
  return a.c.D <= 128 ? launch_simt_e<T, FMT, 4>(a, stream) : a.c.D <= 256 ? launch_simt_e<T, FMT, 8>(a, stream)
                                                                            : launch_simt_e<T, FMT, 16>(a, stream);
}

template <typename T>
static pkv_status launch_simt_t(const QuantDecodeArgs &a, pkv_quant_format fmt, cudaStream_t stream) {
  switch (fmt) {
    case PKV_QUANT_INT8: return launch_simt_f<T, kInt8>(a, stream);
    case PKV_QUANT_E4M3: return launch_simt_f<T, kE4m3>(a, stream);
    case PKV_QUANT_INT4: return launch_simt_f<T, kInt4>(a, stream);
  }
  return PKV_ERR_INVALID_ARG;
}

struct QuantPlan {
  bool mma;                        // tensor cores
  int heads, chunks;               // query heads of a unit (a CTA), head groups of a KV head
  int P, max_parts;                // CUDA cores: keys of a part, parts
  int grid, least, team;           // tensor cores: CTAs, tiles that a warp takes at least, warps on the same tokens
  size_t bytes;                    // workspace
};

static bool quant_sizes_ok(int B, int H, int KVH, int D, int bs, int max_blocks, int max_n, int partition_size) {
  return B >= 0 && B <= 65535 && H > 0 && H <= 65535 && KVH > 0 && H % KVH == 0 && D > 0 && D <= 512 && bs > 0 &&
         max_blocks >= 0 && max_n >= 0 && partition_size >= 0 && partition_size % 128 == 0;
}

static long long quant_cap(int bs, int max_blocks, int max_n) {
  long long cap = std::min<long long>((long long)max_blocks * bs, kQdMaxKeys);
  if (max_n > 0 && max_n < cap) cap = max_n;
  return std::max<long long>(cap, 1);
}

static long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }

static long long quant_parts_wanted(long long units, long long slots, long long span) {
  units = std::max<long long>(units, 1);
  if (units >= slots) return std::max<long long>(1, std::min(ceil_div(4 * slots, units), span / 1024));
  return std::max<long long>(1, std::min<long long>({2 * slots / units, kQdAutoParts, ceil_div(span, 128)}));
}

static size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// CUDA cores: `cap` keys at most, `span` of them visible.
static void simt_plan(int B, int H, int KVH, int D, long long span, int partition_size, QuantPlan *p) {
  p->heads = std::min(kQdHeads, H / KVH);
  p->chunks = (int)ceil_div(H / KVH, p->heads);
  const long long units = (long long)B * KVH * p->chunks;
  long long P = partition_size;
  if (P == 0) P = std::max<long long>(128, ceil_div(ceil_div(span, quant_parts_wanted(units, 2 * kQdSms, span)), 128) * 128);
  P = std::max(P, ceil_div(ceil_div(span, kQdMaxParts), 128) * 128);
  // more units than the workspace counts: whole
  if (units > kChunkCnt - kChunkCntFirst) P = ceil_div(span, 128) * 128;
  p->P = (int)std::min(P, ceil_div(span, 128) * 128);
  p->max_parts = (int)ceil_div(span, p->P);
}
// `rows`: (query row, part) pairs of a call in parts.
static size_t simt_bytes(size_t rows, int D) {
  return kChunkCnt * sizeof(int) +
         (rows ? 2 * align256(rows * sizeof(float)) + align256(rows * (size_t)D * sizeof(float)) : 0);
}
// The most (unit, part) pairs, in more parts than one, of a call of as many units
// and keys or fewer: a smaller batch is split further (see quant_parts_wanted).
static long long simt_most_pairs(long long units, long long span, int partition_size) {
  if (partition_size) {
    const long long parts = std::min<long long>(kQdMaxParts, ceil_div(span, partition_size));
    return parts > 1 ? units * parts : 0;
  }
  const long long slots = 2 * kQdSms;
  long long most = 0;
  const long long few = std::min(units, slots - 1);
  if (span > 128) most = std::min(2 * slots, few * std::min<long long>(kQdAutoParts, ceil_div(span, 128)));
  if (units >= slots && span >= 2 * 1024) {
    const long long many = std::min(units, 4 * slots - 1);
    most = std::max(most, std::min(4 * slots + many, many * (span / 1024)));
  }
  return most;
}

// Tensor cores: query heads of a unit are four where a head has two columns of
// the product (fp32, or no more heads than that), else eight.
static bool mma_split(pkv_dtype dt, int G) { return dt == PKV_F32 || G <= 4; }
static bool mma_shape(pkv_quant_format fmt, int D) {
  return D == 64 || D == 96 || D == 128 || D == 192 || D == 256 || (D == 80 && fmt != PKV_QUANT_INT4);
}
static long long mma_tiles(int B, long long span) { return B * (ceil_div(span, kQmTok) + 1); }
static void mma_plan(int B, int H, int KVH, int D, long long span, int partition_size, pkv_quant_format fmt, bool split,
                     QuantPlan *p) {
  p->heads = split ? 4 : 8;
  p->chunks = (int)ceil_div(H / KVH, p->heads);
  p->least = std::max(1, partition_size / kQmTok);
  const int params = fmt == PKV_QUANT_INT4 ? 8 : 4, row = fmt == PKV_QUANT_INT4 ? D / 2 : D;
  // one CTA resident everywhere, but no more warps than tiles
  const int units = KVH * p->chunks;
  p->team = units % 8 == 0 ? 8 : units % 4 == 0 ? 4 : units % 2 == 0 ? 2 : 1;
  const long long tiles = ceil_div(mma_tiles(B, span), p->least) * units;
  p->grid = (int)std::min<long long>((long long)kQdSms * qm_ctas(row, params), 2 * ceil_div(tiles, 2 * kQmWarps));
  p->bytes = kChunkCnt * sizeof(int) + (size_t)2 * p->grid * kQmWarps * p->heads * (D + 2) * sizeof(float);
}
constexpr long long kQdMostWarps = (long long)kQmMostCtas * kQdSms * kQmWarps;
constexpr long long power(long long base, int n) { return n == 0 ? 1 : base * power(base, n - 1); }
static_assert(kChunkCntFirst + kQmLevels * kQdMostWarps <= kChunkCnt && kQdMostWarps <= power(kQmFan, kQmLevels),
              "the counters fit the workspace's");

pkv_status launch_quant_mma_int8(const QuantDecodeArgs &a, bool split, pkv_dtype dt, cudaStream_t stream);
pkv_status launch_quant_mma_e4m3(const QuantDecodeArgs &a, bool split, pkv_dtype dt, cudaStream_t stream);
pkv_status launch_quant_mma_int4(const QuantDecodeArgs &a, bool split, pkv_dtype dt, cudaStream_t stream);

}  // namespace pkv

using namespace pkv;

extern "C" {

PKV_API size_t pkv_quant_decode_workspace_size(int B, int H, int num_kv_heads, int head_dim, int block_size,
                                               int max_blocks, int max_context_len, int partition_size) {
  if (!quant_sizes_ok(B, H, num_kv_heads, head_dim, block_size, max_blocks, max_context_len, partition_size)) return 0;
  const long long cap = quant_cap(block_size, max_blocks, max_context_len);
  const int G = H / num_kv_heads;
  const int chunks = (int)ceil_div(G, std::min(kQdHeads, G));
  const long long pairs = simt_most_pairs((long long)B * num_kv_heads * chunks, cap, partition_size);
  // (G rows a KV head over its units)
  size_t most = simt_bytes((size_t)ceil_div(pairs * G, chunks), head_dim);
  for (int f = PKV_QUANT_INT8; f <= PKV_QUANT_INT4; ++f)
    for (int split = 0; split < 2; ++split) {
      if (!mma_shape((pkv_quant_format)f, head_dim)) continue;
      QuantPlan p;
      mma_plan(B, H, num_kv_heads, head_dim, cap, partition_size, (pkv_quant_format)f, split, &p);
      most = std::max(most, p.bytes);
    }
  return most;
}

PKV_API pkv_status pkv_quant_decode_attention(
    void *out, const void *q, const void *k_codes, const void *v_codes, const float *k_params, const float *v_params,
    const int32_t *block_tables, const int32_t *context_lens, int B, int H, int num_kv_heads, int head_dim,
    int block_size, int max_blocks, int64_t num_blocks, float scale, float softcap, int window, pkv_quant_format fmt,
    pkv_dtype dt, int max_context_len, int partition_size, void *workspace, size_t workspace_bytes, int *err_flags,
    pkv_stream_t stream) {
  if (head_dim > 512) return PKV_ERR_UNSUPPORTED;
  if (!quant_sizes_ok(B, H, num_kv_heads, head_dim, block_size, max_blocks, max_context_len, partition_size) ||
      num_blocks < 0 || num_blocks > 0x7fffffffLL || window < 0 || !(softcap >= 0.f) || isinf(softcap) ||
      !isfinite(scale) || (softcap > 0.f && !isfinite(2.f * kLog2e * scale / softcap)) ||
      (fmt != PKV_QUANT_INT8 && fmt != PKV_QUANT_E4M3 && fmt != PKV_QUANT_INT4) ||
      (fmt == PKV_QUANT_INT4 && head_dim % 2) || (dt != PKV_F32 && dt != PKV_BF16 && dt != PKV_F16))
    return PKV_ERR_INVALID_ARG;
  if (B == 0) return PKV_OK;
  if (!out || !q || !k_codes || !v_codes || !k_params || !v_params || !block_tables || !context_lens)
    return PKV_ERR_INVALID_ARG;
  auto at = [](const void *p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; };
  const uintptr_t el = dt == PKV_F32 ? 4 : 2;
  if (!at(out, el) || !at(q, el) || !at(k_params, 4) || !at(v_params, 4) || !at(block_tables, 4) ||
      !at(context_lens, 4) || !at(err_flags, 4))
    return PKV_ERR_INVALID_ARG;
  const int64_t cache_rows = num_blocks * block_size * num_kv_heads;
  const int pbytes = fmt == PKV_QUANT_INT4 ? 8 : 4, G = H / num_kv_heads;
  const long long cap = quant_cap(block_size, max_blocks, max_context_len);
  // (keys are walked from a multiple of 32 on)
  const long long span = window > 0 ? std::min(cap, (long long)window + 31) : cap;
  QuantPlan plan = {};
  // tensor cores where 16-byte copies can read the rows, rows have 32-bit
  // numbers and a KV head's tiles are counted in 32 bits
  plan.mma = mma_shape(fmt, head_dim) && at(k_codes, 16) && at(v_codes, 16) && at(k_params, pbytes) &&
             at(v_params, pbytes) && cache_rows < 0xffffffffLL && mma_tiles(B, span) <= 0x7fffffffLL;
  if (plan.mma) {
    mma_plan(B, H, num_kv_heads, head_dim, span, partition_size, fmt, mma_split(dt, G), &plan);
  } else {
    simt_plan(B, H, num_kv_heads, head_dim, span, partition_size, &plan);
    plan.bytes = simt_bytes(plan.max_parts > 1 ? (size_t)B * H * plan.max_parts : 0, head_dim);
    if ((long long)plan.chunks * num_kv_heads * plan.max_parts > 0x7fffffffLL) return PKV_ERR_UNSUPPORTED;
  }
  const size_t need = plan.bytes;
  if (!workspace || workspace_bytes < need || !at(workspace, 256)) return PKV_ERR_WORKSPACE;
  const size_t rows_bytes = (size_t)B * H * head_dim * el;
  const size_t codes = quant_codes_bytes(fmt, cache_rows, head_dim), params = quant_params_bytes(fmt, cache_rows);
  const ArgRange written[] = {{out, rows_bytes}, {workspace, need}};
  const ArgRange read[] = {{q, rows_bytes}, {k_codes, codes}, {v_codes, codes}, {k_params, params}, {v_params, params},
                           {block_tables, (size_t)B * max_blocks * sizeof(int32_t)},
                           {context_lens, (size_t)B * sizeof(int32_t)}, {err_flags, sizeof(int)}};
  for (const ArgRange &x : written)
    for (const ArgRange &y : read)
      if (overlap(x, y)) return PKV_ERR_INVALID_ARG;
  if (overlap(written[0], written[1])) return PKV_ERR_INVALID_ARG;
  QuantDecodeArgs a;
  memset(&a, 0, sizeof a);
  ChunkArgs &c = a.c;
  c.out = out;
  c.q = q;
  c.tables = block_tables;
  c.lens = context_lens;
  c.err = err_flags;
  c.num_blocks = num_blocks;
  c.total_q = B;
  c.B = B;
  c.H = H;
  c.KVH = num_kv_heads;
  c.D = head_dim;
  c.G = H / num_kv_heads;
  c.bs = block_size;
  c.max_blocks = max_blocks;
  c.max_q = 1;
  c.max_n = (int)std::min<long long>(cap, (long long)max_blocks * block_size);   // (0 for a table without columns)
  c.window = window;
  c.P = plan.P;
  c.max_parts = plan.max_parts;
  c.chunks = plan.chunks;
  c.scale_log2 = scale * kLog2e;
  c.cap_ratio = softcap > 0.f ? scale / softcap : 0.f;
  c.cap_log2 = std::min(softcap * kLog2e, FLT_MAX);
  c.scale_y = softcap > 0.f ? 2.f * kLog2e * scale / softcap : 0.f;
  a.k = static_cast<const uint8_t *>(k_codes);
  a.v = static_cast<const uint8_t *>(v_codes);
  a.kp = k_params;
  a.vp = v_params;
  a.heads = plan.heads;
  // whole chunks of 16 tokens, whose parameters are 16-byte rows of their own too
  a.tma = block_size % 16 == 0 && at(k_params, 16) && at(v_params, 16) && num_blocks > 0;
  a.grid = plan.grid;
  a.least = plan.least;
  a.team = plan.team;
  while ((1LL << a.bs_shift) < block_size) ++a.bs_shift;
  a.bs_mul = (uint32_t)((((1ULL << a.bs_shift) - (uint64_t)block_size) << 32) / (uint64_t)block_size + 1);
  char *ws = static_cast<char *>(workspace);
  c.ws_cnt = reinterpret_cast<int *>(ws);
  ws += kChunkCnt * sizeof(int);
  if (plan.mma) {
    a.states = reinterpret_cast<float *>(ws);
  } else if (plan.max_parts > 1) {
    const size_t rows = (size_t)B * H;
    c.ws_m = reinterpret_cast<float *>(ws);
    ws += align256(rows * plan.max_parts * sizeof(float));
    c.ws_l = reinterpret_cast<float *>(ws);
    ws += align256(rows * plan.max_parts * sizeof(float));
    c.ws_o = reinterpret_cast<float *>(ws);
  }
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (plan.mma) {
    const bool split = mma_split(dt, G);
    switch (fmt) {
      case PKV_QUANT_INT8: return launch_quant_mma_int8(a, split, dt, s);
      case PKV_QUANT_E4M3: return launch_quant_mma_e4m3(a, split, dt, s);
      case PKV_QUANT_INT4: return launch_quant_mma_int4(a, split, dt, s);
    }
  }
  switch (dt) {
    case PKV_F32: return launch_simt_t<float>(a, fmt, s);
    case PKV_BF16: return launch_simt_t<__nv_bfloat16>(a, fmt, s);
    case PKV_F16: return launch_simt_t<__half>(a, fmt, s);
  }
  return PKV_ERR_INVALID_ARG;
}

}  // extern "C"
