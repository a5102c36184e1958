// pkv_chunk.cu -- host side of chunk attention: argument checks, the choice
// of kernel and split, the workspace's layout, the launch.
#include <float.h>
#include <math.h>
#include <string.h>

#include <algorithm>

#include "pkv_chunk.cuh"

namespace pkv {

pkv_status launch_chunk_simt(const ChunkArgs &a, int rows, pkv_dtype dt, cudaStream_t stream);
pkv_status launch_chunk_mma(const ChunkArgs &a, pkv_dtype dt, cudaStream_t stream);
pkv_status launch_chunk_tc(const ChunkArgs &a, pkv_dtype dt, char *scratch, int sms, cudaStream_t stream);
long long chunk_tc_items(int B, long long total_q, int H, int G, int D, int max_q);
size_t chunk_tc_scratch(int B, long long total_q, int H, int G, int D, int max_q, long long parts);

// The plan uses the SM count of the one GPU this library is built for, so
// that the workspace's size needs no device.
constexpr int kPlanSms = 152;
constexpr int kChunkRows = 16;     // packed rows per CTA of the CUDA-core and mma.sync kernels
constexpr int kChunkManyRows = 64; // of the CUDA-core kernel for long chunks
constexpr int kChunkFewRows = 4;   // and for single tokens of small groups
constexpr int kMmaRows = 32;       // packed rows up to which the mma.sync kernel is taken where tcgen05 could be
constexpr int kChunkMaxParts = 64;    // of the automatic split
constexpr int kChunkManyParts = 256;  // of any (a row's weights have to fit the join's shared memory)
constexpr long long kChunkMaxKeys = 1LL << 30;  // keys of a context: positions plus a part stay in 32 bits

struct ChunkPlan {
  int kernel;         // 2 tcgen05, 1 mma.sync, 0 CUDA cores
  int P, max_parts;   // keys per part, parts per row
  int most_parts;     // parts per row of any call of these sizes (the workspace's)
  int rows;           // packed rows per CTA (kernels 0 and 1)
  long long chunks;   // row chunks per (sequence, KV head)
};

static long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }
static size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

static bool device_sms(int *sms) {
  static int cached[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return false;
  *sms = dev < 64 ? cached[dev] : 0;
  if (*sms == 0 && cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return false;
  if (dev < 64) cached[dev] = *sms;
  return *sms > 0;
}

static bool chunk_sizes_ok(int B, int64_t total_q, int H, int KVH, int D, int bs, int max_blocks, int max_q,
                           int max_n, int partition_size) {
  return B >= 0 && B <= 65535 && total_q >= 0 && total_q <= 0x7fffffffLL && H > 0 && H <= 65535 && KVH > 0 &&
         H % KVH == 0 && D > 0 && D <= 512 && bs > 0 && max_blocks >= 0 && max_q >= 0 && max_n >= 0 &&
         partition_size >= 0 && partition_size % 128 == 0;
}

static long long chunk_cap(int bs, int max_blocks, int max_n) {
  long long cap = std::min<long long>((long long)max_blocks * bs, kChunkMaxKeys);
  if (max_n > 0 && max_n < cap) cap = max_n;
  return std::max<long long>(cap, 1);
}

static int chunk_max_q(int64_t total_q, int max_q) {
  return (int)std::max<int64_t>(1, max_q > 0 ? std::min<int64_t>(max_q, total_q) : total_q);
}

// Parts of a unit of the CUDA-core and mma.sync kernels, `slots` CTAs resident.
//  - Units that fill the GPU: a CTA's start and end cost its slot some 7 us,
//    so only contexts of 4096 keys and more are split, 2048 keys or more a
//    part, to even out ragged lengths (512 units: 64 sequences of 2304 keys
//    92 us whole, 105 in two; 512 to 4096 keys 104.4 us at 2048, 108.8 whole).
//  - Fewer units, long contexts: two CTAs a slot of 1024 keys or more (drafts
//    over 16-32k keys: 132 us at 8192 keys, 150 at 2048).
//  - Fewer units, short contexts: one round of CTAs, 128 keys or more, at most
//    32 parts (one sequence of 8192 keys, 8 KV heads: 17 us at 256 keys, 19 at
//    1024, 25 at 128; 128 one-head units of 1087 keys, 152 slots: 28.9 us
//    whole, 46.3 in two); `whole` keys or fewer are not worth the join.
static long long parts_wanted(long long units, long long slots, long long span, long long whole) {
  units = std::max<long long>(units, 1);
  if (units >= slots) return std::max<long long>(1, std::min(ceil_div(4 * slots, units), span / 2048));
  const long long two = std::min<long long>(2 * slots / units, kChunkMaxParts);
  if (span / two >= 1024) return two;
  if (span <= whole) return 1;
  return std::max<long long>(1, std::min<long long>({slots / units, 32, ceil_div(span, 128)}));
}

// Parts of the persistent tcgen05 kernel's items (256 rows x a part): the
// number that gives the shortest estimate, in key tiles of 128, of
//   rounds of items over the SMs x (tiles of a part + 2 to start and end one)
//   + joining the parts (0.015 a part of an item: its 270 KB to and from
//   memory against 2.7 us a tile on one SM of 152; 2 for the launch).
// No part is longer than kTcMaxPart keys (some 25 ms), far inside the kernel's
// bounded waits of 500 ms, which span an item; past 2^28 keys a context's 256
// parts are longer, up to 2^22 keys (some 100 ms).
constexpr int kTcMaxPart = 1 << 20;
static long long tc_parts_wanted(long long items, long long span) {
  const long long fewest = ceil_div(span, kTcMaxPart);
  long long best = fewest;
  double least = 0;
  for (long long p = fewest; p <= kChunkMaxParts && p <= ceil_div(span, 512); ++p) {
    const double cost = (double)ceil_div(items * p, kPlanSms) * (ceil_div(ceil_div(span, p), 128) + 2) +
                        (p > 1 ? 0.015 * items * p + 2 : 0.0);
    if (p == fewest || cost < least) {
      least = cost;
      best = p;
    }
  }
  return best;
}

// `span`: the most keys a unit sees, from its first one's 16-key chunk on
// (where its first part begins); each part has `min_p` keys or more.
static void chunk_split(long long wanted, long long span, int min_p, int partition_size, ChunkPlan *p) {
  long long P = partition_size;
  if (P == 0) P = std::max<long long>(min_p, ceil_div(ceil_div(span, wanted), 128) * 128);
  P = std::min(std::max(P, ceil_div(ceil_div(span, kChunkManyParts), 128) * 128), ceil_div(span, 128) * 128);
  p->P = (int)P;
  p->max_parts = (int)ceil_div(span, P);
  // (of a window's shorter span too: its parts may be a few more where this P
  // was raised)
  p->most_parts = partition_size > 0 ? (int)std::min<long long>(kChunkManyParts, ceil_div(span, partition_size))
                                     : (int)std::min(wanted, ceil_div(span, min_p));
}

static bool chunk_plan(int B, int64_t total_q, int H, int KVH, int D, int bs, int max_blocks, int max_q, int max_n,
                       int window, bool has_prefix, int partition_size, pkv_dtype dt, bool aligned16, ChunkPlan *p) {
  if (!chunk_sizes_ok(B, total_q, H, KVH, D, bs, max_blocks, max_q, max_n, partition_size) || window < 0) return false;
  if (dt != PKV_F32 && dt != PKV_BF16 && dt != PKV_F16) return false;
  const long long mq = chunk_max_q(total_q, max_q), cap = chunk_cap(bs, max_blocks, max_n);
  // 16-bit tensors that TMA can read, in tokens chunks that never span two blocks
  p->kernel = tc_eligible(dt, D, bs) && aligned16 ? 1 : 0;
  const long long unit_rows = mq * (H / KVH);
  // More rows than that go to tcgen05, unless everything is small: 16-row
  // units that are all resident at once, over 1024 keys or fewer, are done
  // before the plan and the larger tiles pay (64 tokens on 64 keys, 8 KV
  // heads: 8.4 us against 16.8; on 1024 keys 22.8 / 27.1; 200 tokens on 1024
  // keys, 400 units, 35 / 31).  By the table's keys, not a window's, so that
  // the workspace knows.
  const bool small = (long long)B * KVH * ceil_div(unit_rows, kChunkRows) <= kPlanSms * (D <= 192 ? 2 : 1) && cap <= 1024;
  if (p->kernel == 1 && unit_rows > kMmaRows && !small) p->kernel = 2;
  p->rows = kChunkRows;
  if (p->kernel == 0) p->rows = unit_rows <= kChunkFewRows ? kChunkFewRows : D <= 256 && unit_rows > 2 * kChunkRows ? kChunkManyRows : kChunkRows;
  p->chunks = ceil_div(mq * (H / KVH), p->rows);
  // a window bounds the keys a unit sees, unless a prefix reaches past it
  const long long span = window > 0 && !has_prefix ? std::min(cap, (long long)window + mq + 63) : cap;
  if (p->kernel == 2) {
    const long long items = chunk_tc_items(B, total_q, H, H / KVH, D, (int)mq);
    // (never more than without a window: the workspace is sized for that)
    chunk_split(std::min(tc_parts_wanted(items, span), tc_parts_wanted(items, cap)), span, 512,
                std::min(partition_size, kTcMaxPart), p);
    return true;
  }
  const int per_sm = p->kernel == 0 ? (p->rows == kChunkManyRows ? 2 : 4) : D <= 192 ? 2 : 1;   // resident CTAs
  const long long units = (long long)B * KVH * p->chunks, slots = (long long)kPlanSms * per_sm;
  const long long whole = p->kernel == 1 ? 640 : 0;   // a tensor-core CTA takes 640 keys in the time of a join
  if (units > kChunkCnt - kChunkCntFirst)   // more than can be counted: whole, whatever the caller asked for
    chunk_split(1, span, 128, 0, p);
  else
    chunk_split(std::min(parts_wanted(units, slots, span, whole), parts_wanted(units, slots, cap, whole)), span, 128,
                partition_size, p);
  return true;
}

// Workspace bytes of a plan.
static size_t chunk_ws_bytes(int kernel, int B, int64_t total_q, int H, int KVH, int D, int max_q, long long parts) {
  size_t bytes = kChunkCnt * sizeof(int);
  if (kernel == 2) bytes += chunk_tc_scratch(B, total_q, H, H / KVH, D, chunk_max_q(total_q, max_q), parts);
  if (parts > 1) {
    const size_t rows = (size_t)total_q * H;
    bytes += 2 * align256(rows * parts * sizeof(float)) + align256(rows * parts * (size_t)D * sizeof(float));
  }
  return bytes;
}

}  // namespace pkv

using namespace pkv;

extern "C" {

PKV_API size_t pkv_chunk_workspace_size(int B, int64_t total_q, int H, int num_kv_heads, int head_dim, int block_size,
                                        int max_blocks, int max_q_len, int max_context_len, int partition_size) {
  size_t most = 0;
  for (int dt = 0; dt < 3; ++dt) {   // fp32, 16-bit, and 16-bit tensors that TMA cannot read
    ChunkPlan p;
    if (!chunk_plan(B, total_q, H, num_kv_heads, head_dim, block_size, max_blocks, max_q_len, max_context_len, 0, false,
                    partition_size, (pkv_dtype)dt, dt == 1, &p))
      return 0;
    most = std::max(most, chunk_ws_bytes(p.kernel, B, total_q, H, num_kv_heads, head_dim, max_q_len, p.most_parts));
  }
  return most;
}

PKV_API int pkv_chunk_plan(int B, int64_t total_q, int H, int num_kv_heads, int head_dim, int block_size, int max_blocks,
                           int max_q_len, int max_context_len, int window, int has_prefix, int partition_size,
                           pkv_dtype dt, int *max_parts, int *kernel) {
  ChunkPlan p;
  if (!chunk_plan(B, total_q, H, num_kv_heads, head_dim, block_size, max_blocks, max_q_len, max_context_len, window,
                  has_prefix != 0, partition_size, dt, true, &p))
    return 0;
  if (max_parts) *max_parts = p.max_parts;
  if (kernel) *kernel = p.kernel;
  return p.P;
}

PKV_API pkv_status pkv_chunk_attention(
    void *out, const void *q, const void *k_cache, const void *v_cache, const int32_t *block_tables,
    const int32_t *cu_seqlens_q, const int32_t *context_lens, const float *slopes, const int32_t *prefix_lens,
    const int32_t *kv_starts, int B, int64_t total_q, int H, int num_kv_heads, int head_dim, int block_size,
    int max_blocks, int64_t num_blocks, float scale, float softcap, int window, pkv_dtype dt, int max_q_len,
    int max_context_len, int partition_size, void *workspace, size_t workspace_bytes, int *err_flags,
    pkv_stream_t stream) {
  if (head_dim > 512) return PKV_ERR_UNSUPPORTED;
  if (!chunk_sizes_ok(B, total_q, H, num_kv_heads, head_dim, block_size, max_blocks, max_q_len, max_context_len,
                      partition_size) ||
      num_blocks < 0 || num_blocks > 0x7fffffffLL || window < 0 || !(softcap >= 0.f) || isinf(softcap) || !isfinite(scale) ||
      (softcap > 0.f && !isfinite(2.f * kLog2e * scale / softcap)))
    return PKV_ERR_INVALID_ARG;
  if (dt != PKV_F32 && dt != PKV_BF16 && dt != PKV_F16) return PKV_ERR_INVALID_ARG;
  // packed rows of a (sequence, KV head), rounded up to a chunk, are counted in 32 bits
  if ((long long)chunk_max_q(total_q, max_q_len) * (H / num_kv_heads) > 0x7fffffffLL - kChunkManyRows) return PKV_ERR_UNSUPPORTED;
  if (B == 0 || total_q == 0) return PKV_OK;
  if (!out || !q || !k_cache || !v_cache || !block_tables || !cu_seqlens_q || !context_lens)
    return PKV_ERR_INVALID_ARG;
  const uintptr_t el = dt == PKV_F32 ? 4 : 2;
  const void *ptrs[4] = {out, q, k_cache, v_cache};
  bool aligned16 = true;
  for (const void *p : ptrs) {
    if (reinterpret_cast<uintptr_t>(p) % el) return PKV_ERR_INVALID_ARG;
    aligned16 = aligned16 && reinterpret_cast<uintptr_t>(p) % 16 == 0;
  }
  const void *p4[] = {block_tables, cu_seqlens_q, context_lens, slopes, prefix_lens, kv_starts, err_flags};
  for (const void *p : p4)
    if (reinterpret_cast<uintptr_t>(p) % 4) return PKV_ERR_INVALID_ARG;
  ChunkPlan plan;
  if (!chunk_plan(B, total_q, H, num_kv_heads, head_dim, block_size, max_blocks, max_q_len, max_context_len, window,
                  prefix_lens != nullptr, partition_size, dt, aligned16, &plan))
    return PKV_ERR_INVALID_ARG;
  const size_t need = chunk_ws_bytes(plan.kernel, B, total_q, H, num_kv_heads, head_dim, max_q_len, plan.max_parts);
  if (!workspace || workspace_bytes < need || reinterpret_cast<uintptr_t>(workspace) % 256) return PKV_ERR_WORKSPACE;
  const size_t rows_bytes = (size_t)total_q * H * head_dim * el;
  const size_t cache_bytes = (size_t)num_blocks * block_size * num_kv_heads * head_dim * el;
  const ArgRange written[] = {{out, rows_bytes}, {workspace, need}};
  const ArgRange read[] = {{q, rows_bytes}, {k_cache, cache_bytes}, {v_cache, cache_bytes},
                           {block_tables, (size_t)B * max_blocks * sizeof(int32_t)},
                           {cu_seqlens_q, (size_t)(B + 1) * sizeof(int32_t)}, {context_lens, (size_t)B * sizeof(int32_t)},
                           {slopes, (size_t)H * sizeof(float)}, {prefix_lens, (size_t)B * sizeof(int32_t)},
                           {kv_starts, (size_t)total_q * sizeof(int32_t)}, {err_flags, sizeof(int)}};
  for (const ArgRange &w : written)
    for (const ArgRange &r : read)
      if (overlap(w, r)) return PKV_ERR_INVALID_ARG;
  if (overlap(written[0], written[1])) return PKV_ERR_INVALID_ARG;
  if (plan.chunks * num_kv_heads * plan.max_parts > 0x7fffffffLL) return PKV_ERR_UNSUPPORTED;
  int sms = 0;
  if (!device_sms(&sms)) return PKV_ERR_CUDA;
  ChunkArgs a;
  memset(&a, 0, sizeof a);
  a.out = out;
  a.q = q;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.tables = block_tables;
  a.cu_q = cu_seqlens_q;
  a.lens = context_lens;
  a.slopes = slopes;
  a.prefix = prefix_lens;
  a.starts = kv_starts;
  a.err = err_flags;
  a.num_blocks = num_blocks;
  a.total_q = total_q;
  a.B = B;
  a.H = H;
  a.KVH = num_kv_heads;
  a.D = head_dim;
  a.G = H / num_kv_heads;
  a.bs = block_size;
  a.max_blocks = max_blocks;
  a.max_q = chunk_max_q(total_q, max_q_len);
  a.max_n = (int)chunk_cap(block_size, max_blocks, max_context_len);
  a.window = window;
  a.P = plan.P;
  a.max_parts = plan.max_parts;
  a.chunks = (int)plan.chunks;
  a.scale_log2 = scale * kLog2e;
  a.cap_ratio = softcap > 0.f ? scale / softcap : 0.f;
  a.cap_log2 = std::min(softcap * kLog2e, FLT_MAX);   // (caps past 2.3e38 stay finite)
  a.scale_y = softcap > 0.f ? 2.f * kLog2e * scale / softcap : scale * kLog2e;
  // the series' powers of scale / cap have to stay in range, and a running
  // max commutes with the cap for a positive scale only
  const double ratio = softcap > 0.f ? (double)scale / softcap : 0.0;
  a.cap_small = a.cap_mid = -1.f;
  if (ratio > 1e-4 && ratio < 1e2) {
    double power = ratio;
    for (int i = 0; i < 4; ++i, power *= ratio * ratio) a.cap_k[i] = (float)(softcap * 1.4426950408889634 * kTanh4[i] * power);
    for (int i = 0; i < 6; ++i) a.cap_c[i] = (float)(softcap * 1.4426950408889634 * kTanh6[i]);
    a.cap_small = (float)(0.5 / ratio);
    a.cap_mid = (float)(1.0 / ratio);
  }
  char *ws = static_cast<char *>(workspace);
  a.ws_cnt = reinterpret_cast<int *>(ws);
  ws += kChunkCnt * sizeof(int);
  char *scratch = ws;
  if (plan.kernel == 2) ws += chunk_tc_scratch(B, total_q, H, a.G, head_dim, a.max_q, plan.max_parts);
  if (plan.max_parts > 1) {
    const size_t rows = (size_t)total_q * H;
    a.ws_m = reinterpret_cast<float *>(ws);
    ws += align256(rows * plan.max_parts * sizeof(float));
    a.ws_l = reinterpret_cast<float *>(ws);
    ws += align256(rows * plan.max_parts * sizeof(float));
    a.ws_o = reinterpret_cast<float *>(ws);
  }
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (plan.kernel == 2) return launch_chunk_tc(a, dt, scratch, sms, s);
  if (plan.kernel == 1) return launch_chunk_mma(a, dt, s);
  return launch_chunk_simt(a, plan.rows, dt, s);
}

}  // extern "C"
