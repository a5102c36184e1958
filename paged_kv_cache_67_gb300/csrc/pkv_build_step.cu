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
// shared memory (B <= 16384 requests, up to 16 of a thread), then takes its
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

constexpr int kStepMaxThreads = 1024;
constexpr int kStepMaxB = 16384;    // three sums of 4 bytes each in shared memory
constexpr int kStepSmemB = 8192;    // up to here the cached and held lengths stay there too
constexpr size_t kStepMaxSmem = (size_t)3 * (kStepMaxB + 4) * sizeof(int);  // the most a step asks for
static_assert(kStepMaxSmem >= (size_t)5 * (kStepSmemB + 4) * sizeof(int), "both layouts fit");
constexpr int kStepSmall = 256;     // threads of a small step
constexpr int kStepCluster = 8;     // CTAs of a large step
constexpr int kStepWide = 16;       // of a very large one, where the device has room for it
constexpr int kStepWideFrom = 16384;
constexpr int kStepOneCta = 1024;   // requests or tokens up to which one CTA does the step
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
  uint32_t bs_mul, bs_shift;        // x / bs = (umulhi(x, bs_mul) + x) >> bs_shift for 0 <= x < 2^31
};

__device__ __forceinline__ int sat_add(int a, int b) {  // both in [0, kStepSat]: their sum can be 2^31
  return (int)min((unsigned)a + (unsigned)b, (unsigned)kStepSat);
}

__device__ __forceinline__ int div_bs(const StepArgs &a, int x) {
  return (int)((__umulhi((uint32_t)x, a.bs_mul) + (uint32_t)x) >> a.bs_shift);
}

__device__ __forceinline__ int blocks_for(const StepArgs &a, int tokens) {  // ceil, no overflow
  const int q = div_bs(a, tokens);
  return q + (q * a.bs != tokens);
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

// The same from b on (start[b] <= x), for an owner that is likely near: steps
// that double, then halve.
__device__ __forceinline__ int owner_from(const int *start, int B, int b, int x) {
  int step = 1;
  while (b + step < B && start[b + step] <= x) {
    b += step;
    step <<= 1;
  }
  for (step >>= 1; step > 0; step >>= 1)
    if (b + step < B && start[b + step] <= x) b += step;
  return b;
}

__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// IPT requests of a thread, neighbours, so that one scan over the block makes
// the sums.
template <int IPT>
__global__ void __launch_bounds__(kStepMaxThreads) pkv_build_step_kernel(const StepArgs a) {
  extern __shared__ __align__(16) int s_dyn[];
  const int pad = (a.B + 4) & ~3;  // entries of an array, one more than the requests
  int *s_new = s_dyn;              // [B + 1] exclusive sums of new tokens
  int *s_need = s_new + pad;       // [B + 1] of needed blocks
  int *s_back = s_need + pad;      // [B + 1] of released blocks
  int *s_cached = s_back + pad;    // [B] with B <= kStepSmemB
  int *s_held = s_cached + pad;
  const bool local = a.B <= kStepSmemB;
  __shared__ int s_warp[3][32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nthr = blockDim.x;
  const int rank = blockIdx.x, ncta = gridDim.x;

  const int count = *a.free_count;
  int bad = count < 0 || count > a.free_capacity;
  int c[IPT], n[IPT], h[IPT];
  const int b0 = tid * IPT;
#pragma unroll
  for (int i = 0; i < IPT; ++i) {
    const bool in = b0 + i < a.B;
    c[i] = in ? a.cached[b0 + i] : 0;
    n[i] = in ? a.fresh[b0 + i] : 0;
    h[i] = in ? a.held[b0 + i] : 0;
  }
  int sum[3] = {0, 0, 0}, x[3][IPT];   // this thread's totals, and its requests' own numbers
#pragma unroll
  for (int i = 0; i < IPT; ++i) {
    const bool ok = c[i] >= 0 && n[i] >= 0 && h[i] >= 0 && h[i] <= a.max_blocks &&
                    (long long)c[i] + n[i] <= (long long)a.max_blocks * a.bs &&
                    (long long)c[i] + n[i] <= 0x7fffffffLL && blocks_for(a, c[i]) <= h[i];
    const int w = ok ? blocks_for(a, c[i] + n[i]) : 0;
    x[0][i] = ok ? min(n[i], kStepSat) : 0;
    x[1][i] = ok ? min(max(w - h[i], 0), kStepSat) : 0;
    x[2][i] = ok ? min(max(h[i] - w, 0), kStepSat) : 0;
    bad |= !ok;
    if (local && b0 + i < a.B) {
      s_cached[b0 + i] = c[i];
      s_held[b0 + i] = h[i];
    }
#pragma unroll
    for (int k = 0; k < 3; ++k) sum[k] = sat_add(sum[k], x[k][i]);
  }
  int inc[3] = {sum[0], sum[1], sum[2]};
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const int y = __shfl_up_sync(0xffffffffu, inc[k], o);
      if (lane >= o) inc[k] = sat_add(inc[k], y);
    }
  }
  if (lane == 31) {
#pragma unroll
    for (int k = 0; k < 3; ++k) s_warp[k][warp] = inc[k];
  }
  bad = __syncthreads_or(bad);
  int total[3];
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    int v = lane < nthr / 32 ? s_warp[k][lane] : 0;  // the warps' totals, scanned by every warp
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v = sat_add(v, y);
    }
    total[k] = __shfl_sync(0xffffffffu, v, 31);
    const int before = __shfl_sync(0xffffffffu, v, max(warp - 1, 0));
    // (a sum past the saturation point belongs to a step that is refused below)
    int at = sat_add(warp ? before : 0, inc[k] - sum[k]);
    int *dst = k == 0 ? s_new : k == 1 ? s_need : s_back;
#pragma unroll
    for (int i = 0; i < IPT; ++i) {
      if (b0 + i < a.B) dst[b0 + i] = at;
      at = sat_add(at, x[k][i]);
    }
    if (tid == 0) dst[a.B] = total[k];
  }
  __syncthreads();
  int sum_new = total[0], sum_need = total[1], sum_back = total[2];
  bad |= sum_new >= kStepSat || sum_back >= kStepSat || (long long)count + sum_back > a.free_capacity;
  const int top = bad ? 0 : count + sum_back;     // |F'| (at most free_capacity)
  const bool short_of = !bad && sum_need > top;
  const bool ok = !bad && !short_of;
  if (rank == 0 && tid == 0) {
    if (bad) raise_flag(a.err, PKV_FLAG_STEP_INVALID);
    if (short_of) raise_flag(a.err, PKV_FLAG_OUT_OF_BLOCKS);
    if (ok && sum_new > a.max_tokens) raise_flag(a.err, PKV_FLAG_TOKENS_OVER);
  }
  if (!ok) sum_new = sum_need = sum_back = 0;

  auto cached_of = [&](int b) { return local ? s_cached[b] : a.cached[b]; };
  auto held_of = [&](int b) { return local ? s_held[b] : a.held[b]; };
  auto want_of = [&](int b) { return blocks_for(a, cached_of(b) + (s_new[b + 1] - s_new[b])); };
  auto returned = [&](int r) {                    // released block r, from its table row
    const int b = owner_of(s_back, a.B, r);
    return a.tables[(size_t)b * a.max_blocks + want_of(b) + (r - s_back[b])];
  };
  auto needed = [&](int k) {                      // F'[top - 1 - k]
    const int i = top - 1 - k;
    return i < count ? a.free_blocks[i] : returned(i - count);
  };
  auto in_pool = [&](int blk) { return blk >= 0 && (long long)blk < a.num_blocks; };

  // Tokens (those that the lists have room for) from the first warps on,
  // needed blocks from the last on, released ones from the middle, so that
  // the three run side by side in a small step.
  const int gid = rank * nthr + tid, gstep = ncta * nthr;
  constexpr int kU = 2;                           // chains of a lane in flight in a large one
  const int nu = a.max_tokens > gstep ? kU : 1;
  for (int w0 = gid >> 5; (long long)w0 * 32 * nu < a.max_tokens; w0 += gstep >> 5) {
    const int first = w0 * 32 * nu + lane;
    int pos[kU], blk[kU], off[kU], b = 0;
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int t = first + 32 * u;
      pos[u] = off[u] = 0;
      blk[u] = -1;
      if (u < nu && t < sum_new && t < a.max_tokens) {
        b = u == 0 ? owner_of(s_new, a.B, t) : owner_from(s_new, a.B, b, t);
        pos[u] = cached_of(b) + (t - s_new[b]);
        const int lb = div_bs(a, pos[u]), held = held_of(b);
        off[u] = pos[u] - lb * a.bs;
        blk[u] = lb < held ? a.tables[(size_t)b * a.max_blocks + lb] : needed(s_need[b] + (lb - held));
      }
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int t = first + 32 * u;
      if (u < nu && t < a.max_tokens) {
        const bool fits = in_pool(blk[u]);
        if (!fits && t < sum_new) raise_flag(a.err, PKV_FLAG_BLOCK_OUT_OF_RANGE);
        a.slots[t] = fits ? (long long)blk[u] * a.bs + off[u] : -1;
        a.positions[t] = pos[u];
      }
    }
  }
  for (int k = gstep - 1 - gid; k < sum_need; k += gstep) {
    const int b = owner_of(s_need, a.B, k);
    const int blk = needed(k);
    if (!in_pool(blk)) raise_flag(a.err, PKV_FLAG_BLOCK_OUT_OF_RANGE);
    a.tables[(size_t)b * a.max_blocks + held_of(b) + (k - s_need[b])] = blk;
  }
  const int mid = gid >= gstep / 2 ? gid - gstep / 2 : gid + gstep - gstep / 2;
  for (int r = mid; r < sum_back; r += gstep) a.free_blocks[count + r] = returned(r);
  for (int b = gid; b <= a.B; b += gstep) a.cu[b] = ok ? s_new[b] : 0;

  // behind every CTA's last read: the outputs that may be the inputs' memory
  if (ncta > 1) cluster_sync_all();
  else __syncthreads();
  for (int b = gid; b < a.B; b += gstep) {
    // both read before either is written: above kStepSmemB they are the memory
    // that lens and held_out may be
    const int total_b = cached_of(b) + (s_new[b + 1] - s_new[b]), hb = held_of(b);
    a.lens[b] = ok ? total_b : 0;
    a.held_out[b] = ok ? blocks_for(a, total_b) : hb;
  }
  if (gid == 0) *a.free_count_out = ok ? top - sum_need : count;
}

// Whether clusters of kStepWide CTAs (past the portable 8) fit this device.
template <int IPT>
static bool wide_fits() {
  static int known[64] = {0};      // 0 unknown, 1 yes, 2 no
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return false;
  if (known[dev] == 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kStepWide);
    cfg.blockDim = dim3(kStepMaxThreads);
    cfg.dynamicSmemBytes = kStepMaxSmem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kStepWide;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    const bool ok = cudaFuncSetAttribute(pkv_build_step_kernel<IPT>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
                    cudaOccupancyMaxActiveClusters(&n, pkv_build_step_kernel<IPT>, &cfg) == cudaSuccess && n > 0;
    if (!ok) cudaGetLastError();
    known[dev] = ok ? 1 : 2;
  }
  return known[dev] == 1;
}

template <int IPT>
static pkv_status launch_step(const StepArgs &a, int ctas, int threads, cudaStream_t stream) {
  const size_t smem = (size_t)(a.B <= kStepSmemB ? 5 : 3) * ((a.B + 4) & ~3) * sizeof(int);
  static int configured[64] = {0};
  if (!allow_smem(pkv_build_step_kernel<IPT>, kStepMaxSmem, configured)) return PKV_ERR_CUDA;
  if (ctas == kStepWide && !wide_fits<IPT>()) ctas = kStepCluster;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ctas > 1 ? 1 : 0;
  if (cudaLaunchKernelEx(&cfg, pkv_build_step_kernel<IPT>, a) != cudaSuccess) return PKV_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

pkv_status launch_build_step(const StepArgs &a, cudaStream_t stream) {
  const int most = a.B > a.max_tokens ? a.B : a.max_tokens;
  const int ctas = most > kStepWideFrom ? kStepWide : most > kStepOneCta ? kStepCluster : 1;
  const int threads = most <= kStepSmall ? kStepSmall : kStepMaxThreads;   // fewer warps start and meet faster
  if (a.B <= threads) return launch_step<1>(a, ctas, threads, stream);
  if (a.B <= 4 * threads) return launch_step<4>(a, ctas, threads, stream);
  return launch_step<kStepMaxB / kStepMaxThreads>(a, ctas, threads, stream);
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
                num_blocks, free_capacity, B, max_blocks, block_size, (int)max_tokens, 0, 0};
  // x / bs for 31-bit x by one product (Granlund and Montgomery 1994): with
  // s = ceil(log2 bs), m = floor(2^32 (2^s - bs) / bs) + 1
  while ((1LL << a.bs_shift) < block_size) ++a.bs_shift;
  a.bs_mul = (uint32_t)(((1ULL << 32) * ((1ULL << a.bs_shift) - block_size)) / block_size + 1);
  return launch_build_step(a, reinterpret_cast<cudaStream_t>(stream));
}
