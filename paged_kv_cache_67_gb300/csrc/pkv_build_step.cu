// pkv_build_step.cu -- a serving step's block tables, slots, positions and
// query offsets built on the GPU from the requests' lengths.
//
// With c_b cached and n_b new tokens of request b, h_b blocks held and
// w_b = ceil((c_b + n_b) / bs) wanted:
//   released    R = concat over b of table[b, w_b .. h_b)
//   free stack  F' = F[0 .. count) ++ R
//   needed      block k (over b, then i = h_b .. w_b - 1) = F'[|F'| - 1 - k]
//   token t of request b (t - cu_b is its index): pos = c_b + t - cu_b,
//   slot = table[b, pos / bs] * bs + pos % bs.
// Everything hangs on three exclusive sums over the requests (new tokens,
// needed and released blocks).
//
// One cluster does the step: every CTA makes the three sums for itself in
// shared memory (B <= 16384 requests, a few tiles of 1024), then takes its
// share of the tokens, the needed and the released blocks, finding a token's
// request by a binary search of the sums.  No CTA waits for another until the
// end: table and stack entries that are written are never ones that are read
// (reads: table [0, h), stack below count; writes: table [h, w), stack from
// count on; a needed block that this very step releases is read from the
// releasing row, not from the stack).  The cluster barrier at the end orders
// the outputs that may alias inputs (lengths, counts) behind every read.
#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {

constexpr int kStepThreads = 1024;
constexpr int kStepMaxB = 16384;    // three sums of 4 bytes each in shared memory
constexpr int kStepCluster = 8;     // CTAs of a large step
constexpr int kStepSat = 0x40000000;  // sums saturate here: above every valid total

struct StepArgs {
  int32_t *tables;
  const int32_t *held;
  int32_t *held_out;
  int32_t *free_blocks;
  const int32_t *free_count;
  int32_t *free_count_out;
  const int32_t *cached;
  const int32_t *fresh;
  int32_t *lens;
  int32_t *cu;
  int64_t *slots;
  int32_t *positions;
  int *err;
  long long num_blocks, free_capacity;
  int B, max_blocks, bs, max_tokens;
};

__device__ __forceinline__ int sat_add(int a, int b) {  // both in [0, kStepSat]
  return min(a + b, kStepSat);
}

__device__ __forceinline__ int blocks_for(int tokens, int bs) {  // ceil, no overflow
  return tokens / bs + (tokens % bs != 0);
}

// Last b in [0, B) with start[b] <= x (start[0] = 0 <= x).
__device__ __forceinline__ int owner_of(const int *start, int B, int x) {
  int lo = 0, len = B;
  while (len > 1) {
    const int half = len >> 1;
    if (start[lo + half] <= x) lo += half;
    len -= half;
  }
  return lo;
}

__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

__global__ void __launch_bounds__(kStepThreads) pkv_build_step_kernel(const StepArgs a) {
  extern __shared__ int s_dyn[];
  int *s_new = s_dyn;              // [B] exclusive sums of new tokens
  int *s_need = s_new + a.B;       // [B] of needed blocks
  int *s_back = s_need + a.B;      // [B] of released blocks
  __shared__ int s_warp[3][32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = blockIdx.x, ncta = gridDim.x;

  const int count = *a.free_count;
  int bad = count < 0 || count > a.free_capacity;
  int sum_new = 0, sum_need = 0, sum_back = 0;   // totals of the tiles before
  for (int base = 0; base < a.B; base += kStepThreads) {
    const int b = base + tid;
    int x[3] = {0, 0, 0};
    if (b < a.B) {
      const int c = a.cached[b], n = a.fresh[b], h = a.held[b];
      const bool ok = c >= 0 && n >= 0 && h >= 0 && h <= a.max_blocks &&
                      (long long)c + n <= (long long)a.max_blocks * a.bs &&
                      (long long)c + n <= 0x7fffffffLL && blocks_for(c, a.bs) <= h;
      if (ok) {
        const int w = blocks_for(c + n, a.bs);
        x[0] = min(n, kStepSat);
        x[1] = min(max(w - h, 0), kStepSat);
        x[2] = min(max(h - w, 0), kStepSat);
      }
      bad |= !ok;
    }
    int inc[3] = {x[0], x[1], x[2]};
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        const int y = __shfl_up_sync(0xffffffffu, inc[i], o);
        if (lane >= o) inc[i] = sat_add(inc[i], y);
      }
    }
    if (lane == 31) {
#pragma unroll
      for (int i = 0; i < 3; ++i) s_warp[i][warp] = inc[i];
    }
    __syncthreads();
    int tot[3], pre[3];
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      int v = s_warp[i][lane];                    // the 32 warps' totals, scanned by every warp
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v = sat_add(v, y);
      }
      tot[i] = __shfl_sync(0xffffffffu, v, 31);
      const int before = __shfl_sync(0xffffffffu, v, max(warp - 1, 0));
      pre[i] = warp ? before : 0;
    }
    if (b < a.B) {
      // a sum past the saturation point belongs to a step that is refused below
      s_new[b] = sat_add(sum_new, sat_add(pre[0], inc[0] - x[0]));
      s_need[b] = sat_add(sum_need, sat_add(pre[1], inc[1] - x[1]));
      s_back[b] = sat_add(sum_back, sat_add(pre[2], inc[2] - x[2]));
    }
    sum_new = sat_add(sum_new, tot[0]);
    sum_need = sat_add(sum_need, tot[1]);
    sum_back = sat_add(sum_back, tot[2]);
    __syncthreads();                              // s_warp is written again
  }
  bad |= sum_new >= kStepSat || sum_back >= kStepSat || (long long)count + sum_back > a.free_capacity;
  bad = __syncthreads_or(bad);
  const int top = bad ? 0 : count + sum_back;     // |F'| (at most free_capacity)
  const bool short_of = !bad && sum_need > top;
  const bool ok = !bad && !short_of;
  if (rank == 0 && tid == 0) {
    if (bad) raise_flag(a.err, PKV_FLAG_STEP_INVALID);
    if (short_of) raise_flag(a.err, PKV_FLAG_OUT_OF_BLOCKS);
    if (ok && sum_new > a.max_tokens) raise_flag(a.err, PKV_FLAG_TOKENS_OVER);
  }
  if (!ok) sum_new = sum_need = sum_back = 0;

  // entry i of the table row that request b returns (i counts from w_b)
  auto returned = [&](int r) {
    const int b = owner_of(s_back, a.B, r);
    const int w = blocks_for(a.cached[b] + a.fresh[b], a.bs);
    return a.tables[(size_t)b * a.max_blocks + w + (r - s_back[b])];
  };
  auto needed = [&](int k) {                      // F'[top - 1 - k]
    const int i = top - 1 - k;
    return i < count ? a.free_blocks[i] : returned(i - count);
  };
  auto in_pool = [&](int blk) { return blk >= 0 && (long long)blk < a.num_blocks; };

  const int gid = rank * kStepThreads + tid, gstep = ncta * kStepThreads;
  // tokens (those that the lists have room for): kU of a thread's in flight at once (each is a chain of a search
  // and two dependent loads)
  constexpr int kU = 4;
  for (long long t0 = gid; t0 < a.max_tokens; t0 += (long long)gstep * kU) {
    int pos[kU];
    long long slot[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const long long t = t0 + (long long)u * gstep;
      pos[u] = 0;
      slot[u] = -1;
      if (t < sum_new) {
        const int b = owner_of(s_new, a.B, (int)t);
        pos[u] = a.cached[b] + ((int)t - s_new[b]);
        const int lb = pos[u] / a.bs, h = a.held[b];
        const int blk = lb < h ? a.tables[(size_t)b * a.max_blocks + lb] : needed(s_need[b] + (lb - h));
        if (in_pool(blk)) slot[u] = (long long)blk * a.bs + (pos[u] - lb * a.bs);
        else raise_flag(a.err, PKV_FLAG_BLOCK_OUT_OF_RANGE);
      }
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const long long t = t0 + (long long)u * gstep;
      if (t < a.max_tokens) {
        a.slots[t] = slot[u];
        a.positions[t] = pos[u];
      }
    }
  }
  for (int k = gid; k < sum_need; k += gstep) {
    const int b = owner_of(s_need, a.B, k);
    const int blk = needed(k);
    if (!in_pool(blk)) raise_flag(a.err, PKV_FLAG_BLOCK_OUT_OF_RANGE);
    a.tables[(size_t)b * a.max_blocks + a.held[b] + (k - s_need[b])] = blk;
  }
  for (int r = gid; r < sum_back; r += gstep) a.free_blocks[count + r] = returned(r);
  for (int b = gid; b <= a.B; b += gstep) a.cu[b] = !ok ? 0 : b < a.B ? s_new[b] : sum_new;

  // behind every CTA's last read: the outputs that may be the inputs' memory
  if (ncta > 1) cluster_sync_all();
  else __syncthreads();
  for (int b = gid; b < a.B; b += gstep) {
    const int c = a.cached[b], n = a.fresh[b], h = a.held[b];
    a.lens[b] = ok ? c + n : 0;
    a.held_out[b] = ok ? blocks_for(c + n, a.bs) : h;
  }
  if (gid == 0) *a.free_count_out = ok ? top - sum_need : count;
}

pkv_status launch_build_step(const StepArgs &a, cudaStream_t stream) {
  const size_t smem = (size_t)3 * a.B * sizeof(int);
  static int configured[64] = {0};
  if (!allow_smem(pkv_build_step_kernel, smem, configured)) return PKV_ERR_CUDA;
  const int ctas = a.max_tokens > 4 * kStepThreads ? kStepCluster : 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kStepThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ctas > 1 ? 1 : 0;
  if (cudaLaunchKernelEx(&cfg, pkv_build_step_kernel, a) != cudaSuccess) return PKV_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // namespace pkv

using namespace pkv;

extern "C" PKV_API pkv_status pkv_build_step(
    int32_t *block_tables, const int32_t *held, int32_t *held_out, int32_t *free_blocks,
    const int32_t *free_count, int32_t *free_count_out, const int32_t *cached_lens,
    const int32_t *new_lens, int32_t *context_lens, int32_t *cu_seqlens_q, int64_t *slot_mapping,
    int32_t *positions, int B, int max_blocks, int64_t num_blocks, int block_size,
    int64_t free_capacity, int64_t max_tokens, int *err_flags, pkv_stream_t stream) {
  if (B < 0 || max_blocks < 0 || num_blocks < 0 || num_blocks > 0x7fffffffLL || block_size <= 0 ||
      free_capacity < 0 || free_capacity > 0x7fffffffLL || max_tokens < 0)
    return PKV_ERR_INVALID_ARG;
  if (B > kStepMaxB || max_tokens >= kStepSat || free_capacity >= kStepSat) return PKV_ERR_UNSUPPORTED;
  if (B == 0 && max_tokens == 0) return PKV_OK;
  if (!free_count || !free_count_out || !cu_seqlens_q || (max_tokens > 0 && (!slot_mapping || !positions)) ||
      (free_capacity > 0 && !free_blocks) ||
      (B > 0 && (!held || !held_out || !cached_lens || !new_lens || !context_lens ||
                 (max_blocks > 0 && !block_tables))))
    return PKV_ERR_INVALID_ARG;
  const void *p4[] = {block_tables, held, held_out, free_blocks, free_count, free_count_out,
                      cached_lens, new_lens, context_lens, cu_seqlens_q, positions, err_flags};
  for (const void *p : p4)
    if (reinterpret_cast<uintptr_t>(p) % 4) return PKV_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(slot_mapping) % 8) return PKV_ERR_INVALID_ARG;
  // nothing that is written may overlap another argument, but for the three
  // whole arrays that may be updated in place
  const struct { const void *p; size_t bytes; bool written; int twin; } r[] = {
      {block_tables, (size_t)B * max_blocks * 4, true, -1}, {held, (size_t)B * 4, false, 2},
      {held_out, (size_t)B * 4, true, 1},                   {free_blocks, (size_t)free_capacity * 4, true, -1},
      {free_count, 4, false, 5},                            {free_count_out, 4, true, 4},
      {cached_lens, (size_t)B * 4, false, 8},               {new_lens, (size_t)B * 4, false, -1},
      {context_lens, (size_t)B * 4, true, 6},               {cu_seqlens_q, (size_t)(B + 1) * 4, true, -1},
      {slot_mapping, (size_t)max_tokens * 8, true, -1},     {positions, (size_t)max_tokens * 4, true, -1}};
  constexpr int kArgs = sizeof r / sizeof r[0];
  for (int i = 0; i < kArgs; ++i)
    for (int j = i + 1; j < kArgs; ++j) {
      if (!(r[i].written || r[j].written) || r[i].bytes == 0 || r[j].bytes == 0) continue;
      const uintptr_t x = reinterpret_cast<uintptr_t>(r[i].p), y = reinterpret_cast<uintptr_t>(r[j].p);
      if (x < y + r[j].bytes && y < x + r[i].bytes && !(r[i].twin == j && x == y)) return PKV_ERR_INVALID_ARG;
    }
  StepArgs a = {block_tables, held, held_out, free_blocks, free_count, free_count_out, cached_lens,
                new_lens, context_lens, cu_seqlens_q, slot_mapping, positions, err_flags,
                num_blocks, free_capacity, B, max_blocks, block_size, (int)max_tokens};
  return launch_build_step(a, reinterpret_cast<cudaStream_t>(stream));
}
