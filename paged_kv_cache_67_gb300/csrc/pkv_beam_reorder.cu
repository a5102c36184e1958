// pkv_beam_reorder.cu -- block tables that follow the chosen beams, with the
// copies of last blocks that two beams would otherwise share.
//
// What a request's children get hangs on that request alone and takes a warp a
// few hundred cycles (lane = child), so every CTA works it out for itself and
// then does its share of the tables and copies: one launch, no CTA waits for
// another.  The copies' sources stay in use under the new tables and their
// targets are blocks that no child uses, so the order of copies is free.
// 32 requests x 8 beams, 16 layers of int8 caches: 21 us, of which a request's
// dependent reads and the copies of a CTA, one after the other, take most.
//   keeps     a child whose last block is not full keeps it if no child before
//             it has the same one there and none holds it whole;
//   takes     the others, in order, the first of the request's own blocks of
//             their column that is in use by no child (their own lane's first).
#include <algorithm>

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {

constexpr int kBrThreads = 256;
constexpr int kBrMost = 32;
constexpr int kBrPools = 256;
constexpr int kBrMaxB = 16384;
constexpr int kBrSms = 152;              // of the one GPU this library is built for (speed alone)

struct BeamPool {
  char *base;
  long long block_bytes, row_bytes;      // row_bytes 0: blocks are copied whole
};
struct BeamReorderArgs {
  int32_t *tables_out, *lens_out;
  int64_t *slots;
  const int32_t *tables, *lens, *parents, *owned;
  const uint8_t *finished;
  int *err;
  long long num_blocks;
  int W, K, max_blocks, bs, num_pools;
  BeamPool pools[kBrPools];
};

// `bytes` bytes by the CTA, 16 at a time where both ends allow.
__device__ __forceinline__ void copy_bytes(char *dst, const char *src, long long bytes) {
  const uintptr_t both = reinterpret_cast<uintptr_t>(dst) | reinterpret_cast<uintptr_t>(src);
  long long done = 0;
  if (both % 16 == 0) {
    const long long n = bytes / 16;
    constexpr int kAhead = 4;            // loads in flight a thread
    for (long long i = threadIdx.x; i < n; i += kBrThreads * kAhead) {
      uint4 v[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j)
        if (i + j * kBrThreads < n) v[j] = reinterpret_cast<const uint4 *>(src)[i + j * kBrThreads];
#pragma unroll
      for (int j = 0; j < kAhead; ++j)
        if (i + j * kBrThreads < n) reinterpret_cast<uint4 *>(dst)[i + j * kBrThreads] = v[j];
    }
    done = n * 16;
  } else if (both % 4 == 0) {
    const long long n = bytes / 4;
    for (long long i = threadIdx.x; i < n; i += kBrThreads) reinterpret_cast<uint32_t *>(dst)[i] = reinterpret_cast<const uint32_t *>(src)[i];
    done = n * 4;
  }
  for (long long i = done + threadIdx.x; i < bytes; i += kBrThreads) dst[i] = src[i];
}

__global__ void __launch_bounds__(kBrThreads) pkv_beam_reorder_kernel(const __grid_constant__ BeamReorderArgs a) {
  constexpr uint32_t kAll = 0xffffffffu;
  __shared__ int s_parent[kBrMost], s_col[kBrMost], s_block[kBrMost];   // column of the next token, its block
  __shared__ int s_src[kBrMost], s_dst[kBrMost], s_rows[kBrMost], s_copies;
  const int b = blockIdx.y, tid = threadIdx.x, lane = tid & 31, K = a.K, MB = a.max_blocks;
  const bool report = blockIdx.x == 0;
  const int32_t *tables = a.tables + (long long)b * a.W * MB, *owned = a.owned + (long long)b * K * MB;
  if (tid < 32) {
    const long long me = (long long)b * K + lane;
    const bool is = lane < K;
    int p = is ? __ldg(a.parents + me) : -1, n = 0;
    bool bad = p < -1 || p >= a.W;
    if (!bad && p >= 0) {
      n = __ldg(a.lens + (long long)b * a.W + p);
      bad = n < 0 || n > (long long)MB * a.bs;
    }
    if (bad) p = -1;
    if (bad && report) raise_flag(a.err, PKV_FLAG_BEAM);
    const bool used = p >= 0;
    const int col = used ? n / a.bs : -1, rest = used ? n - col * a.bs : 0;
    const bool room = used && col < MB;
    const int block = room && rest > 0 ? __ldg(tables + (long long)p * MB + col) : -1;
    // who keeps its last block
    bool keeps = room && rest > 0;
    for (int i = 0; i < K; ++i) {
      const int pi = __shfl_sync(kAll, p, i), ci = __shfl_sync(kAll, col, i), bi = __shfl_sync(kAll, block, i),
                ri = __shfl_sync(kAll, rest, i);
      if (!room || rest == 0 || i == lane || pi < 0) continue;
      if (ci == col && ri > 0 && i < lane && bi == block) keeps = false;
      if (ci > col && __ldg(tables + (long long)pi * MB + col) == block) keeps = false;
    }
    int target = keeps ? block : -1;
    bool none = false;
    // the others, in order
    uint32_t todo = __ballot_sync(kAll, room && !keeps);
    int cur = -1, mine = -1;
    bool free_lane = false;
    while (todo) {
      const int i = __ffs(todo) - 1;
      todo &= todo - 1;
      const int c = __shfl_sync(kAll, col, i);
      if (c != cur) {                    // the request's own blocks of this column, less those in use
        cur = c;
        mine = is ? __ldg(owned + (long long)lane * MB + c) : -1;
        free_lane = is;
        const int use = !used ? -1 : col > c ? __ldg(tables + (long long)p * MB + c) : col == c ? target : -1;
        const bool uses = used && (col > c || (col == c && (keeps || target >= 0)));
        for (int j = 0; j < K; ++j) {
          const int x = __shfl_sync(kAll, use, j);
          const bool y = __shfl_sync(kAll, (int)uses, j);
          if (y && x == mine) free_lane = false;
        }
      }
      const uint32_t frees = __ballot_sync(kAll, free_lane);
      const int from = frees >> i & 1 ? i : frees ? __ffs(frees) - 1 : -1;
      const int got = __shfl_sync(kAll, mine, from < 0 ? 0 : from);
      if (lane == i) {
        target = from < 0 ? -1 : got;
        none = from < 0;
      }
      if (from >= 0 && mine == got) free_lane = false;
    }
    const bool outside = room && !none && (target < 0 || (long long)target >= a.num_blocks);
    const bool src_bad = room && rest > 0 && (block < 0 || (long long)block >= a.num_blocks);
    const bool ended = is && a.finished && __ldg(a.finished + me);
    const bool fine = room && !none && !outside && !src_bad;
    const bool copy = fine && rest > 0 && !keeps;
    const uint32_t copies = __ballot_sync(kAll, copy);
    if (copy) {
      const int at = __popc(copies & ((1u << lane) - 1));
      s_src[at] = block;
      s_dst[at] = target;
      s_rows[at] = rest;
    }
    if (lane == 0) s_copies = __popc(copies);
    if (is) {
      s_parent[lane] = p;
      s_col[lane] = col;
      s_block[lane] = none ? (rest > 0 ? block : __ldg(owned + (long long)lane * MB + col)) : target;
      if (report) {
        const bool next = fine && !ended;
        a.lens_out[me] = used ? n + next : 0;
        a.slots[me] = next ? (long long)target * a.bs + rest : -1;
        if (used && !room && !ended) raise_flag(a.err, PKV_FLAG_CONTEXT_TOO_LONG);
        if (none) raise_flag(a.err, PKV_FLAG_OUT_OF_BLOCKS);
        if (outside || src_bad) raise_flag(a.err, PKV_FLAG_BLOCK_OUT_OF_RANGE);
      }
    }
  }
  __syncthreads();
  int32_t *out = a.tables_out + (long long)b * K * MB;
  for (long long i = (long long)blockIdx.x * kBrThreads + tid; i < (long long)K * MB; i += (long long)gridDim.x * kBrThreads) {
    const int k = (int)(i / MB), c = (int)(i - (long long)k * MB);
    const int p = s_parent[k], col = s_col[k];
    out[i] = c < col ? __ldg(tables + (long long)p * MB + c) : c == col ? s_block[k] : __ldg(owned + i);
  }
  const int items = s_copies * a.num_pools;
  for (int i = blockIdx.x; i < items; i += gridDim.x) {
    const int pool = i / s_copies, k = i - pool * s_copies;
    const BeamPool &x = a.pools[pool];
    copy_bytes(x.base + s_dst[k] * x.block_bytes, x.base + s_src[k] * x.block_bytes,
               x.row_bytes ? x.row_bytes * s_rows[k] : x.block_bytes);
  }
}

}  // namespace pkv

using namespace pkv;

extern "C" PKV_API pkv_status pkv_beam_reorder(int32_t *tables_out, int32_t *lens_out, int64_t *slots,
                                               const int32_t *tables, const int32_t *lens, const int32_t *parents,
                                               const int32_t *owned, const uint8_t *finished, int B, int W, int K,
                                               int max_blocks, int64_t num_blocks, int block_size, int num_pools,
                                               void *const *pools, const int64_t *block_bytes,
                                               const int64_t *row_bytes, int *err_flags, pkv_stream_t stream) {
  if (B < 0 || W <= 0 || K <= 0 || max_blocks <= 0 || num_blocks < 0 || num_blocks > 0x7fffffffLL || block_size <= 0 ||
      num_pools < 0 || (num_pools > 0 && (!pools || !block_bytes || !row_bytes)))
    return PKV_ERR_INVALID_ARG;
  if (W > kBrMost || K > kBrMost || B > kBrMaxB || num_pools > kBrPools) return PKV_ERR_UNSUPPORTED;
  if (B == 0) return PKV_OK;
  if (!tables_out || !lens_out || !slots || !tables || !lens || !parents || !owned) return PKV_ERR_INVALID_ARG;
  auto at = [](const void *p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; };
  if (!at(tables_out, 4) || !at(lens_out, 4) || !at(slots, 8) || !at(tables, 4) || !at(lens, 4) || !at(parents, 4) ||
      !at(owned, 4) || !at(err_flags, 4))
    return PKV_ERR_INVALID_ARG;
  BeamReorderArgs a = {};
  const size_t bk = (size_t)B * K, bw = (size_t)B * W;
  const ArgRange r[] = {{tables_out, bk * max_blocks * 4}, {lens_out, bk * 4}, {slots, bk * 8},       // written
                        {tables, bw * max_blocks * 4}, {lens, bw * 4}, {parents, bk * 4},
                        {owned, bk * max_blocks * 4}, {finished, bk}, {err_flags, 4}};
  for (int i = 0; i < 3; ++i)
    for (int j = i + 1; j < 9; ++j)
      if (overlap(r[i], r[j])) return PKV_ERR_INVALID_ARG;
  for (int i = 0; i < num_pools; ++i) {
    if (block_bytes[i] < 0 || row_bytes[i] < 0 || row_bytes[i] > block_bytes[i] / block_size ||
        block_bytes[i] > (1LL << 40) || (!pools[i] && block_bytes[i] > 0 && num_blocks > 0))
      return PKV_ERR_INVALID_ARG;
    a.pools[i] = {static_cast<char *>(pools[i]), block_bytes[i], row_bytes[i]};
    const ArgRange x = {pools[i], (size_t)(num_blocks * block_bytes[i])};
    for (const ArgRange &y : r)
      if (overlap(x, y)) return PKV_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (overlap(x, ArgRange{pools[j], (size_t)(num_blocks * block_bytes[j])})) return PKV_ERR_INVALID_ARG;
  }
  a.tables_out = tables_out;
  a.lens_out = lens_out;
  a.slots = slots;
  a.tables = tables;
  a.lens = lens;
  a.parents = parents;
  a.owned = owned;
  a.finished = finished;
  a.err = err_flags;
  a.num_blocks = num_blocks;
  a.W = W;
  a.K = K;
  a.max_blocks = max_blocks;
  a.bs = block_size;
  a.num_pools = num_pools;
  // a CTA an item (a pool's copy for one child), up to eight an SM in all
  const long long items = std::max<long long>(1, (long long)num_pools * (K - 1));
  const long long share = std::max<long long>(1, 8LL * kBrSms / B);
  pkv_beam_reorder_kernel<<<dim3((unsigned)std::min(items, share), (unsigned)B), kBrThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(a);
  return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}
