// pkv_quant_decode.cuh -- what the decode kernels over a quantised cache share.
//
// One new token per sequence.  Rows are the query heads of a KV head, a few of
// them a unit (a.chunks head groups a KV head).  The visible keys are
// [lo, n), lo = max(0, n - window), walked from lo & ~31 on.
#pragma once

#include "pkv_chunk.cuh"
#include "pkv_quant.cuh"

namespace pkv {

// Shape of the tensor-core kernel: tokens of a tile, pairs of warps of a CTA, and
// its rings: as many tiles as let two CTAs share an SM's 228 KB (1 KB of it a
// CTA's own), at least two and at most six; rows too wide for that have one CTA.
constexpr int kQmTok = 32;
constexpr int kQmHalves = kQmTok / 16;
constexpr int kQmWarps = 4;
constexpr int kQmThreads = 2 * 32 * kQmWarps;
constexpr int kQmRegsCompute = 200, kQmRegsFill = 48;   // of two CTAs an SM: 128 a thread in all
constexpr int kQmGroups = 32 * kQmWarps;   // groups of sequences whose first tiles a CTA keeps
constexpr int kQmMostCtas = 2;
constexpr int kQmFan = 16;                 // states joined at once
constexpr int kQmLevels = 3;               // joins one after the other: kQmFan^kQmLevels warps
constexpr int kQmMostStages = 6;
// (the rings begin at a multiple of 1 KB; barriers, first tiles, a scan's sums)
constexpr int kQmPre = 1024 + 16 * kQmWarps * kQmMostStages + 4 * (kQmGroups + 2 + kQmWarps);
constexpr int qm_tile(int row, int params) { return kQmWarps * kQmTok * 2 * (row + params); }
constexpr int qm_ctas(int row, int params) { return 2 * qm_tile(row, params) + kQmPre <= 113 * 1024 ? 2 : 1; }
constexpr int qm_stages(int row, int params) {
  const int n = ((qm_ctas(row, params) == 2 ? 113 : 227) * 1024 - kQmPre) / qm_tile(row, params);
  return n > kQmMostStages ? kQmMostStages : n;
}
constexpr int qm_smem(int row, int params) { return qm_stages(row, params) * qm_tile(row, params) + kQmPre; }
// Bytes of a row that lie together in the ring: a power of two is swizzled by
// TMA over itself, others are conflict-free or nearly so as they are.
constexpr int qm_box(int row) { return row % 128 == 0 ? 128 : row == 192 ? 64 : row; }

struct QuantDecodeArgs {
  ChunkArgs c;                     // q, out, tables, lens, sizes, score form, split, workspace
  const uint8_t *k, *v;            // codes
  const float *kp, *vp;            // parameters
  int heads;                       // query heads of a unit
  float *states;                   // tensor cores: two places a warp for states to be joined
  int tma;                         // blocks of whole 16-token chunks, read by TMA
  int grid, least, team;           // its CTAs; tiles that a warp takes at least; warps that walk the same tokens
  uint32_t bs_mul;                 // t / block_size = (umulhi(t, bs_mul) + t) >> bs_shift for t < 2^31
  int bs_shift;
};

// A CTA's place in the grid and its keys [t0, t1); nparts 0: nothing to do.
struct QuantPart {
  int b, kvh, chunk, part, nparts, n, lo, t0, t1, head0, rows, unit;
};
__device__ __forceinline__ QuantPart quant_part(const QuantDecodeArgs &a) {
  QuantPart p;
  const ChunkArgs &c = a.c;
  // head groups and KV heads of the same tokens side by side: their parameters
  // share sectors, their keys a read
  p.b = blockIdx.y;
  const int x = blockIdx.x;
  p.chunk = x % c.chunks;
  p.kvh = x / c.chunks % c.KVH;
  p.part = x / (c.chunks * c.KVH);
  p.unit = (p.b * c.KVH + p.kvh) * c.chunks + p.chunk;
  p.head0 = p.kvh * c.G + p.chunk * a.heads;
  p.rows = min(a.heads, c.G - p.chunk * a.heads);
  int n = __ldg(c.lens + p.b);
  const bool report = x == 0 && threadIdx.x == 0;
  if (n < 0) {
    if (report) raise_flag(c.err, PKV_FLAG_CONTEXT_NEGATIVE);
    n = 0;
  }
  const long long cap = (long long)c.max_blocks * c.bs;
  if (n > cap) {
    if (report) raise_flag(c.err, PKV_FLAG_CONTEXT_TOO_LONG);
    n = (int)cap;
  }
  if (n > c.max_n) {               // the host's bound sized the split: what lies past it is not read
    if (report) raise_flag(c.err, PKV_FLAG_CONTEXT_OVER_HINT);
    n = c.max_n;
  }
  p.n = n;
  p.lo = c.window > 0 ? max(0, n - c.window) : 0;
  const int base = p.lo & ~31;
  p.nparts = max(1, (n - base + c.P - 1) / c.P);
  if (p.part >= p.nparts) p.nparts = 0;
  p.t0 = base + p.part * c.P;
  p.t1 = min(n, p.t0 + c.P);
  return p;
}

// Slot of key t, or -1 where its table entry names no block (flagged).
__device__ __forceinline__ long long quant_slot(const ChunkArgs &c, int b, int t) {
  const int lb = t / c.bs, phys = __ldg(c.tables + (size_t)b * c.max_blocks + lb);
  if (phys < 0 || (long long)phys >= c.num_blocks) {
    raise_flag(c.err, PKV_FLAG_BLOCK_OUT_OF_RANGE);
    return -1;
  }
  return (long long)phys * c.bs + (t - lb * c.bs);
}

// As chunk_finish, for any head_dim (vectors of 4 where they fit).
template <typename T>
__device__ __noinline__ void quant_finish(const ChunkArgs &a, const QuantPart &p, const float *s_m, const float *s_l, float *s_o,
                             int ostride, int room, int *s_scratch) {
  auto row_out = [&](int r) { return (size_t)p.b * a.H + p.head0 + r; };
  const bool sees = p.n > p.lo;
  auto seen = [&](int) { return sees; };
  int *counter = a.ws_cnt + kChunkCntFirst + p.unit;
  if (a.D % 4 == 0 && reinterpret_cast<uintptr_t>(a.out) % 16 == 0) {
    chunk_finish<T>(a, p.rows, p.part, p.nparts, s_m, s_l, s_o, ostride, room, s_scratch, counter, row_out, seen);
    return;
  }
  const int tid = threadIdx.x, nthr = blockDim.x, D = a.D;
  if (p.nparts == 1) {
    for (int i = tid; i < p.rows * D; i += nthr) {
      const int r = i / D, d = i - r * D;
      reinterpret_cast<T *>(a.out)[row_out(r) * D + d] = from_f32<T>(sees ? s_o[r * ostride + d] / s_l[r] : 0.f);
    }
    return;
  }
  for (int r = tid; r < p.rows; r += nthr) {
    a.ws_m[row_out(r) * a.max_parts + p.part] = s_m[r];
    a.ws_l[row_out(r) * a.max_parts + p.part] = s_l[r];
  }
  for (int i = tid; i < p.rows * D; i += nthr) {
    const int r = i / D, d = i - r * D;
    a.ws_o[(row_out(r) * a.max_parts + p.part) * D + d] = s_o[r * ostride + d];
  }
  if (!chunk_last_part(counter, p.nparts, s_scratch)) return;
  chunk_merge<T, 1>(a, p.rows, p.nparts, s_o, room, row_out, seen);
  if (tid == 0) *counter = 0;
}

// The capped or plain score in log2 units from the raw product.
__device__ __forceinline__ float quant_score(const ChunkArgs &a, float dot) {
  return a.cap_log2 > 0.f ? chunk_cap(a, dot) : dot * a.scale_log2;
}

}  // namespace pkv
