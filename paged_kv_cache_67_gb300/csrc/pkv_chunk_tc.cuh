// pkv_chunk_tc.cuh -- chunk attention for bf16 / fp16 and many rows per key
// (long chunks, drafts of grouped heads), head_dim 64 to 256, on the
// 5th-generation tensor cores (see pkv_chunk.cuh for rows, masks and scores).
//
// Three launches.
//   plan   (one CTA) lists the units of work: 256 packed rows (two 128-row
//          tiles; one at head_dim 192 and 256) of a sequence x one part of the keys they see, most key
//          tiles first, so that the long ones start first.
//   main   persistent, a CTA per SM, claims (unit, head subgroup) items from
//          a counter; roles as in causal prefill: two softmax warpgroups, one
//          per tile and one row per thread, a producer that streams the K and
//          V tiles (128 keys), a thread that issues S = Q K^T and O += P V
//          into tensor memory, and a scheduler that claims, works out and
//          publishes items and loads their queries.
//   merge  (only when the keys are split) joins the parts' (m, l, O).
// Packing.  With G' the largest power of two that divides the G query heads
// of a KV head, a tile is 128 / G' queries x G' heads: one TMA box brings it
// into the tile's row order, a K/V tile serves G' heads at once, and a tile
// spans fewer positions, so fewer keys are multiplied only to be masked.
// A unit of one row tile (128 rows or fewer) gives both warpgroups the same
// rows and every other key tile each: one group's softmax hides behind the
// other's products, and group 0 joins the two states at the end, reading
// group 1's O from tensor memory.
// Units whose keys a window or document mask cuts start at the first key any
// of their rows sees (its 16-key chunk): tiles before it are never loaded.
// Values that no row sees are zeroed in the tile; a row that still ends not
// finite because a hidden value is not (0 * inf) is noted, and its warp does it
// again key by key once the CTA has no more items: no wait spans that.
// Every wait is bounded, as in prefill.
#pragma once

#include <string.h>

#include <type_traits>

#include "pkv_attn_tc.cuh"
#include "pkv_chunk.cuh"
#include "pkv_tcgen05.cuh"

namespace pkv {

constexpr int kCtRows = 128;     // packed rows per softmax warpgroup (MMA M)
constexpr int kCtMaxGroups = 2;  // row tiles per item: 2, or 1 where O's columns leave no room for a second (D > 128)
constexpr int kCtTile = 128;     // keys per tile
constexpr int kCtMaxStages = 4;  // of the K ring, and of the V ring
// Warps: four softmax warps per group, then K producer, MMA, scheduler and V
// producer.  Registers with two groups: the launch has 384 x 168 = 64512; the
// softmax warps take 200 each and the others 104 (256 x 200 + 128 x 104 =
// 64512).  At 216 / 72 the MMA issuer spills (plain scores 1065 TFLOP/s
// against 1121), at 184 / 136 the softmax does.  One group needs no split.
constexpr int kCtRegsLaunch = 168, kCtRegsSoftmax = 200, kCtRegsOther = 104;
static_assert(32 * 4 * kCtMaxGroups * kCtRegsSoftmax + 128 * kCtRegsOther <= 32 * (4 * kCtMaxGroups + 4) * kCtRegsLaunch,
              "the split cannot exceed what the launch holds");
__host__ __device__ constexpr int ct_groups(int D) { return D <= 128 ? 2 : 1; }
constexpr int kCtQRegion = kCtRows * 128;      // 128 rows x 64 elements of 16 bits
constexpr int kCtKVRegion = kCtTile * 128;
constexpr int kCtPlanThreads = 1024;
constexpr int kCtSat = 1 << 29;                // sums of tiles stop here (query offsets that overlap can add up to anything)
constexpr int kCtClasses = 256;                // plan: key tiles of a unit, the most first

struct __align__(16) CtUnit {    // 32 bytes, written by the plan
  int b, i0, part, nparts;       // sequence, first query; part of the keys
  int t0, t1, lo, pad;           // the part's keys [t0, t1) (t1 = 0: no row sees any); first key seen by the unit
};

struct CtArgs {
  ChunkArgs c;
  int *n_units;                  // written by the plan
  int4 *tiles;                   // [tiles_cap] (sequence, tile, first key seen, one past the last)
  CtUnit *units;                 // [units_cap]
  int2 *redo;                    // [units_cap * subs][softmax warps] (rows to do again, the warp's next noted item)
  int tiles_cap, units_cap;
  int gshift;                    // log2 of the packed heads G'
  int subs;                      // head subgroups: H / G'
  int bshift;                    // log2 of the keys in one TMA box: 16 .. 64, a divisor of block_size
};

// ---------------------------------------------------------------------- main

template <int D>
struct CtShape {
  static constexpr int kGroups = ct_groups(D);
  static constexpr int kSoftmaxWarps = 4 * kGroups;
  static constexpr int kThreads = 32 * (kSoftmaxWarps + 4);
  static constexpr int kReaders = 3 + kSoftmaxWarps;            // of a published item
  static constexpr int kRegions = D / 64;
  static constexpr int kQBytes = kRegions * kCtQRegion;         // one group's query tile
  static constexpr int kKVBytes = kRegions * kCtKVRegion;       // one K (or V) tile
  static constexpr int kQOff = 0;                               // [group]
  static constexpr int kKStages = D == 64 ? 4 : D <= 192 ? 2 : 1, kVStages = D == 64 ? 4 : D == 128 ? 3 : 1;
  static constexpr int kKOff = kQOff + kGroups * kQBytes;       // [stage]
  static constexpr int kVOff = kKOff + kKStages * kKVBytes;     // [stage]
  static constexpr int kBarOff = kVOff + kVStages * kKVBytes;
  static constexpr int kPairOff = kBarOff + 1024;               // group 1's m, l of 128 rows
  static constexpr int kSmem = kPairOff + 1024 + 1024;          // + alignment slack
  // Tensor memory, 512 columns.  Two groups: S (128 columns, P over its first
  // half) and O (D columns) in 256 each.  One: S buffer 0, O in columns 128 to
  // 383, S buffer 1.
  static constexpr uint32_t kTmemCols = 512;
  __device__ __forceinline__ static uint32_t s_col(int g) { return (kGroups == 2 ? 256 : 384) * g; }
};

// One work item as every role sees it.  kind: 1 work, 2 no row sees a key
// (zero rows to write), -1 no more items.
struct __align__(16) CtItem {
  int kind, sub, b, i0;          // head subgroup, sequence, first query in the sequence
  int q0, qlen, n, w;            // the sequence's first row; the item's number
  int t0, t1, lo, part;          // the part's keys, the unit's first seen key
  int nt[kCtMaxGroups];             // key tiles each group works on
  int ntiles;                    // key tiles the item loads
  int nparts;                    // negative: both groups share one row tile (then -nparts parts)
  __device__ __forceinline__ bool pair() const { return nparts < 0; }
  __device__ __forceinline__ int parts() const { return nparts < 0 ? -nparts : nparts; }
};
static_assert(sizeof(CtItem) == 64, "four 16-byte words");

// Rows `rows` (bits: lanes) of the warp's 32 of item w, which ended not finite
// with a key of the part hidden: where a value that was multiplied by a hidden
// key's 0 is not finite, again from what the row sees alone.  g, r: the lane's
// row tile and row, as in the softmax.  (Inlined, it cost the softmax registers:
// four capped prompt chunks 170 us, 167 so.)
template <int D, typename T, bool BIAS>
__device__ __noinline__ void ct_redo(const CtArgs &ta, unsigned w, unsigned rows, int g, int r) {
  constexpr int kGroups = ct_groups(D), EPL = D / 32;
  constexpr int kKeys = 32 / EPL;                // keys whose loads are in flight together
  const ChunkArgs &a = ta.c;
  const int lane = threadIdx.x & 31;
  const int per = kCtRows >> ta.gshift;
  CtUnit u;
  reinterpret_cast<int4 *>(&u)[0] = __ldcg(reinterpret_cast<const int4 *>(ta.units + w / (unsigned)ta.subs));
  reinterpret_cast<int4 *>(&u)[1] = __ldcg(reinterpret_cast<const int4 *>(ta.units + w / (unsigned)ta.subs) + 1);
  const int sub = (int)(w % (unsigned)ta.subs), kvh = (sub << ta.gshift) / a.G;
  const ChunkSeq s = chunk_seq(a, u.b, false);
  const int queries = min(kGroups * per, s.qlen - u.i0);
  const int qi = (kGroups == 2 && queries <= per ? 0 : g * per) + (r >> ta.gshift);
  const int i = u.i0 + min(qi, queries - 1), p = s.n - s.qlen + i;
  const int h = (sub << ta.gshift) + (r & ((1 << ta.gshift) - 1));
  const size_t q_row = (size_t)(s.q0 + i) * a.H + h;
  const float slope = BIAS ? __ldg(a.slopes + h) * kLog2e : 0.f;
  int lo, hi;
  chunk_visible(a, s, i, lo, hi);
  const bool seen = hi > lo;
  const int rlo = max(lo, u.t0), rhi = min(hi, u.t1);
  const bool mine = (rows >> lane) & 1, some = mine && rhi > rlo;
  // The keys [from, u.t1) were multiplied; the row's are one interval of them,
  // so what counts is the first key with a value that is not finite before the
  // rows' own, and the last behind them.
  const int from = max(u.t0, u.lo);
  const int before = __reduce_max_sync(0xffffffffu, some ? rlo : from);
  const int behind = __reduce_min_sync(0xffffffffu, some ? rhi : u.t1);
  auto odd_value = [&](int t) {                  // key t's row of V, by the warp
    float z = 0.f;
    const T *v = reinterpret_cast<const T *>(a.v_cache) + chunk_row_at(a, u.b, kvh, t) + lane;
#pragma unroll
    for (int e = 0; e < EPL; ++e) z = fmaf(to_f32<T>(v[32 * e]), 0.f, z);
    return z != 0.f;
  };
  int first = 0x7fffffff, last = -1;
  for (int t = from; t < before && first > t; t += kKeys) {
#pragma unroll
    for (int k = 0; k < kKeys; ++k)
      if (t + k < before && odd_value(t + k)) first = min(first, t + k);
    first = __reduce_min_sync(0xffffffffu, first);
  }
  for (int t = u.t1 - 1; t >= behind && last < 0; t -= kKeys) {
#pragma unroll
    for (int k = 0; k < kKeys; ++k)
      if (t - k >= behind && odd_value(t - k)) last = max(last, t - k);
    last = __reduce_max_sync(0xffffffffu, last);
  }
  unsigned again = __ballot_sync(0xffffffffu, mine && (!some || first < rlo || last >= rhi));
  while (again) {
    const int src = __ffs(again) - 1;
    again &= again - 1;
    const size_t row = __shfl_sync(0xffffffffu, (unsigned long long)q_row, src);
    const bool any_key = __shfl_sync(0xffffffffu, (int)seen, src);
    float em, el, eo[EPL];
    chunk_row_exact<T, EPL, kKeys>(a, u.b, kvh, row, __shfl_sync(0xffffffffu, slope, src), __shfl_sync(0xffffffffu, p, src),
                                   __shfl_sync(0xffffffffu, rlo, src), __shfl_sync(0xffffffffu, rhi, src), em, el, eo);
    const size_t at = row * a.max_parts + u.part;
#pragma unroll
    for (int e = 0; e < EPL; ++e) {
      const int d = lane + 32 * e;
      if (u.nparts == 1)
        reinterpret_cast<T *>(a.out)[row * D + d] = from_f32<T>(any_key ? eo[e] / el : 0.f);
      else
        a.ws_o[at * D + d] = eo[e];
    }
    if (u.nparts > 1 && lane == 0) {
      a.ws_m[at] = em;
      a.ws_l[at] = el;
    }
  }
}

template <int D, typename T, int CAP, bool BIAS>
__global__ void __launch_bounds__(CtShape<D>::kThreads, 1)
    pkv_chunk_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                        const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CtArgs ta) {
  using Sh = CtShape<D>;
  constexpr int kGroups = Sh::kGroups, kSoftmaxWarps = Sh::kSoftmaxWarps;
  const ChunkArgs &a = ta.c;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t *bars = reinterpret_cast<uint64_t *>(sm + Sh::kBarOff);
  uint64_t *k_full = bars;                       // [kCtMaxStages]: K and V arrive and are
  uint64_t *v_full = k_full + kCtMaxStages;      // released separately, each through its
  uint64_t *k_empty = v_full + kCtMaxStages;     // own ring and producer
  uint64_t *v_empty = k_empty + kCtMaxStages;
  uint64_t *q_full = v_empty + kCtMaxStages;     // [groups]: the group's query tile landed
  uint64_t *q_empty = q_full + kCtMaxGroups;     // its last S of an item done
  uint64_t *s_full = q_empty + kCtMaxGroups;     // S of its current tile (one group: of S buffer tile & 1)
  uint64_t *p_full = s_full + kCtMaxGroups;      // P of its current tile (the same)
  uint64_t *o_done = p_full + kCtMaxGroups;      // its last P . V of an item done (one group: every P . V, [0])
  uint64_t *item_full = o_done + kCtMaxGroups;      // [2]
  uint64_t *item_empty = item_full + 2;          // [2]
  uint64_t *pair_full = item_empty + 2;          // group 1's state of a shared row tile is there
  uint64_t *pair_empty = pair_full + 1;          // group 0 has read it
  uint64_t *mma_done = pair_empty + 1;
  uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(mma_done + 1);
  int *abort_flag = reinterpret_cast<int *>(mma_done + 2);
  CtItem *items = reinterpret_cast<CtItem *>(bars + 36);  // [2], 16-byte aligned
  static_assert(4 * kCtMaxStages + 5 * kCtMaxGroups + 4 + 3 + 2 <= 36, "the barriers end before the items");
  float *s_pair = reinterpret_cast<float *>(sm + Sh::kPairOff);  // [2][128]

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    for (int s = 0; s < kCtMaxStages; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&v_full[s], 1);
      mbar_init(&k_empty[s], 1);
      mbar_init(&v_empty[s], 1);
    }
    for (int g = 0; g < kCtMaxGroups; ++g) {
      mbar_init(&q_full[g], 1);
      mbar_init(&q_empty[g], 1);
      mbar_init(&s_full[g], 1);
      mbar_init(&p_full[g], 128);
      mbar_init(&o_done[g], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&item_full[s], 1);
      mbar_init(&item_empty[s], Sh::kReaders);
    }
    mbar_init(pair_full, 128);
    mbar_init(pair_empty, 128);
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tensormap(&tmQ);
    prefetch_tensormap(&tmK);
    prefetch_tensormap(&tmV);
  }
  if (warp == kSoftmaxWarps) tmem_alloc(tmem_holder, Sh::kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  constexpr bool bf16 = std::is_same<T, __nv_bfloat16>::value;
  const int gheads = 1 << ta.gshift;               // heads packed in a tile
  const int per = kCtRows >> ta.gshift;            // queries per row tile

  auto abort_cta = [&]() {
    raise_flag(a.err, PKV_FLAG_TIMEOUT);
    *(volatile int *)abort_flag = 1;
  };
  // (a warp that goes on or gives up as one takes this into its vote)
  auto aborted = [&]() { return *(volatile int *)abort_flag != 0; };

  if (warp >= kSoftmaxWarps) {
    if constexpr (kGroups == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kCtRegsOther));
    if (warp == kSoftmaxWarps + 2) {
      // ------------------------------------------------------------ scheduler
      griddep_wait();                                // the plan's units (every other role waits for an item)
      const unsigned total = (unsigned)*(volatile int *)ta.n_units * (unsigned)ta.subs;
      unsigned w = blockIdx.x;
      int it = 0, ig[kCtMaxGroups] = {0, 0};
      bool ok = true;
      while (true) {
        CtItem item;
        memset(&item, 0, sizeof item);
        item.kind = -1;
        if (w < total) {
          const int4 *up = reinterpret_cast<const int4 *>(ta.units + w / (unsigned)ta.subs);
          const int4 u0 = __ldcg(up), u1 = __ldcg(up + 1);
          const ChunkSeq s = chunk_seq(a, u0.x, false);
          item.sub = (int)(w % (unsigned)ta.subs);
          item.b = u0.x;
          item.i0 = u0.y;
          item.part = u0.z;
          item.nparts = u0.w;
          item.t0 = u1.x;
          item.t1 = u1.y;
          item.lo = u1.z;
          item.q0 = s.q0;
          item.qlen = s.qlen;
          item.n = s.n;
          item.w = (int)w;
          const int queries = min(kGroups * per, s.qlen - item.i0);
          item.kind = item.t1 > 0 ? 1 : 2;
          if (item.kind == 1) {
            // one past the last key the group's rows see before the part's end
            // (at least one tile, so that a present group always has work)
            auto tiles_to = [&](int i) {
              const int hi = min(item.t1, max(s.n - s.qlen + i + 1, s.prefix));
              return max(1, (hi - item.t0 + kCtTile - 1) / kCtTile);
            };
            item.nt[0] = tiles_to(item.i0 + min(per, queries) - 1);
            item.nt[1] = queries > per ? tiles_to(item.i0 + queries - 1) : 0;
            item.ntiles = max(item.nt[0], item.nt[1]);
            if (kGroups == 2 && queries <= per) {
              item.nparts = -item.nparts;
              item.nt[1] = item.ntiles / 2;
              item.nt[0] = item.ntiles - item.nt[1];
            }
          }
        }
        const int slot = it & 1;
        if (it >= 2) {
          ok = __all_sync(0xffffffffu, mbar_wait_bounded(&item_empty[slot], ((it >> 1) - 1) & 1));
          if (!ok) break;
        }
        if (lane == 0) {
          items[slot] = item;
          mbar_arrive(&item_full[slot]);
        }
        __syncwarp();
        ++it;
        if (item.kind < 0) break;
        if (item.kind == 1) {
#pragma unroll
          for (int g = 0; g < kGroups; ++g) {
            if (!ok || item.nt[g] == 0) continue;
            if (ig[g] > 0) {
              ok = __all_sync(0xffffffffu, mbar_wait_bounded(&q_empty[g], (ig[g] - 1) & 1) && !aborted());
              if (!ok) break;
            }
            if (lane == 0) mbar_arrive_expect_tx(&q_full[g], (uint32_t)Sh::kQBytes);
            __syncwarp();
            if (lane < Sh::kRegions)
              tma_load_3d_keep(sm + Sh::kQOff + g * Sh::kQBytes + lane * kCtQRegion, &tmQ, &q_full[g], 64 * lane,
                               item.sub << ta.gshift, item.q0 + item.i0 + (item.pair() ? 0 : g * per));
            ++ig[g];
          }
          if (!ok) break;
        }
        unsigned nw = 0;
        if (lane == 0) nw = (unsigned)atomicAdd(a.ws_cnt, 1) + gridDim.x;
        w = __shfl_sync(0xffffffffu, nw, 0);
      }
      if (!ok && lane == 0) abort_cta();
      if (a.max_parts > 1) griddep_launch_dependents();  // the merge: it reads nothing before it has waited
      // the last query tiles land before the CTA can end (bounded)
#pragma unroll
      for (int g = 0; g < kGroups; ++g)
        if (ig[g] > 0) mbar_wait_bounded(&q_full[g], (ig[g] - 1) & 1);
    } else if (warp == kSoftmaxWarps || warp == kSoftmaxWarps + 3) {
      // ----------------------------------------------------------- producers
      // one warp streams the keys, one the values: per item and tile the boxes
      // (one per lane: some keys of one 64-column region) once the tile that
      // used the stage before has been read.  In one warp a tile's keys would
      // wait behind the values before them.
      const bool is_v = warp != kSoftmaxWarps;
      const int stages = is_v ? Sh::kVStages : Sh::kKStages;
      uint64_t *full = is_v ? v_full : k_full, *empty = is_v ? v_empty : k_empty;
      const CUtensorMap *map = is_v ? &tmV : &tmK;
      uint8_t *ring_base = sm + (is_v ? Sh::kVOff : Sh::kKOff);
      const int nboxes = kCtTile >> ta.bshift, per_tensor = nboxes * Sh::kRegions;
      const int region = (lane % per_tensor) / nboxes, chunk = lane % nboxes;
      int it = 0, issued = 0, stage = 0;
      uint32_t parity = 1;            // of the stage's release: passes at once in the first round
      bool ok = true;
      while (ok) {
        const int slot = it & 1;
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(&item_full[slot], (it >> 1) & 1));
        if (!ok) break;
        const CtItem item = items[slot];
        __syncwarp();
        if (lane == 0) mbar_arrive(&item_empty[slot]);
        ++it;
        if (item.kind < 0) break;
        const int kvh = (item.sub << ta.gshift) / a.G;
        for (int j = 0; j < item.ntiles; ++j) {
          const int tok0 = item.t0 + j * kCtTile;
          const int valid_chunks = min(nboxes, (item.t1 - tok0 + (1 << ta.bshift) - 1) >> ta.bshift);
          const uint32_t bytes = (uint32_t)(valid_chunks * Sh::kRegions * (128 << ta.bshift));
          int phys = 0;
          if (lane < valid_chunks) phys = __ldg(a.tables + (size_t)item.b * a.max_blocks + (tok0 + (lane << ta.bshift)) / a.bs);
          ok = __all_sync(0xffffffffu, mbar_wait_bounded(&empty[stage], parity) && !aborted());
          if (!ok) break;
          if (lane < valid_chunks && (phys < 0 || (long long)phys >= a.num_blocks)) {
            raise_flag(a.err, PKV_FLAG_BLOCK_OUT_OF_RANGE);
            phys = 0;
          }
          phys = __shfl_sync(0xffffffffu, phys, chunk);
          if (lane == 0) mbar_arrive_expect_tx(&full[stage], bytes);
          __syncwarp();
          if (lane < per_tensor && chunk < valid_chunks) {
            const int t = tok0 + (chunk << ta.bshift);
            tma_load_4d_keep(ring_base + stage * Sh::kKVBytes + region * kCtKVRegion + chunk * (128 << ta.bshift), map,
                             &full[stage], region * 64, kvh, t % a.bs, phys);
          }
          ++issued;
          if (++stage == stages) {
            stage = 0;
            parity ^= 1;
          }
        }
      }
      if (!ok && lane == 0) abort_cta();
      // the last fills land before the CTA can end (bounded)
      for (int r = max(0, issued - stages); r < issued; ++r) mbar_wait_bounded(&full[r % stages], (r / stages) & 1);
    } else if (warp == kSoftmaxWarps + 1) {
      // ------------------------------------------------------------ MMA issuer
      if (lane == 0) {
        const uint32_t idesc_s = umma_idesc_f16(128, kCtTile, bf16, false);
        const uint32_t idesc_o = umma_idesc_f16(128, D, bf16, true);
        auto kv_base = [&](int ring, bool v) {
          return smem_u32(v ? sm + Sh::kVOff + (ring % Sh::kVStages) * Sh::kKVBytes
                            : sm + Sh::kKOff + (ring % Sh::kKStages) * Sh::kKVBytes);
        };
        // g: the group, or with one group the S buffer
        auto issue_s = [&](int g, int ring) {  // S_g = Q_g . K^T over D in 16-wide steps
          const uint32_t qb = smem_u32(sm + Sh::kQOff + (kGroups == 2 ? g : 0) * Sh::kQBytes), kb = kv_base(ring, false);
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            umma_f16(tmem + Sh::s_col(g), umma_desc_sw128(qb + (k >> 2) * kCtQRegion + (k & 3) * 32, 16, 1024),
                     umma_desc_sw128(kb + (k >> 2) * kCtKVRegion + (k & 3) * 32, 16, 1024), idesc_s,
                     k > 0);
          umma_commit(&s_full[g]);
        };
        auto issue_pv = [&](int g, int ring, bool acc) {  // O_g (+)= P_g . V, P from tensor memory
          const uint32_t vb = kv_base(ring, true);
#pragma unroll
          for (int k = 0; k < kCtTile / 16; ++k)
            umma_f16_tmem_a(tmem + (kGroups == 2 ? 256 * g + 128 : 128), tmem + Sh::s_col(g) + 8 * k,
                            umma_desc_sw128(vb + k * 2048, kCtKVRegion, 1024), idesc_o, acc || k > 0);
        };
        // Per item: S of the first tile of both groups; then per tile and
        // group, as soon as P_g(j) arrives: P_g(j) . V_j, then S_g(j+1).  The
        // products of one thread run in issue order, so S_g(j+1) -- written
        // over P_g(j) -- starts after P_g(j) . V_j has read it, and the commit
        // that signals S_g(j+1) also covers P_g(j) . V_j (O is final for tile
        // j when the softmax sees S_g(j+1)).  The next item's first product
        // into O (no accumulate) comes after the softmax's first P of that
        // item, which the softmax writes only once it has read the previous O.
        // Group 0 (the earlier query rows) needs no more KV tiles than group
        // 1: once its last product of an item is issued, group 0's first S of
        // the next item is issued as soon as that item, its query tile and its
        // first keys are there, so group 0's softmax starts on the next item
        // while group 1 finishes this one.
        int it = 0, ring0 = 0, ig[kCtMaxGroups] = {0, 0}, tcnt[kCtMaxGroups] = {0, 0};
        CtItem nx;
        bool have_nx = false;   // the next item is read already
        bool early = false;     // ... and group 0's first S of it issued
        bool ok = true;
        while (ok) {
          CtItem item;
          if (have_nx) {
            item = nx;
            have_nx = false;
          } else {
            const int slot = it & 1;
            ok = mbar_wait_bounded(&item_full[slot], (it >> 1) & 1);
            if (!ok) break;
            item = items[slot];
            mbar_arrive(&item_empty[slot]);
            ++it;
          }
          if (item.kind < 0) break;
          if (item.ntiles == 0) continue;
          const bool pre = early;
          early = false;
          if constexpr (kGroups == 1) {
            // One row tile: S of tile t goes to buffer t & 1 (t counts over all
            // items), so the next S is made while the softmax works on this one,
            // as soon as its keys are there, and before or after P . V as they
            // and P arrive.  A buffer's P is read by a product issued before
            // the S that overwrites it.
            auto start_s = [&](int ring, bool last) {
              ok = ok && mbar_wait_bounded(&k_full[ring % Sh::kKStages], (ring / Sh::kKStages) & 1);
              if (!ok) return;
              tc_fence_after();
              issue_s(ring & 1, ring);
              if (last) umma_commit(&q_empty[0]);
              umma_commit(&k_empty[ring % Sh::kKStages]);
            };
            ok = mbar_wait_bounded(&q_full[0], ig[0] & 1);
            start_s(ring0, item.ntiles == 1);
            for (int j = 0; ok && j < item.ntiles; ++j) {
              const int ring = ring0 + j, nr = ring + 1;
              bool started = j + 1 >= item.ntiles;
              const unsigned long long t0 = global_timer_ns();
              while (!mbar_test_wait(&p_full[ring & 1], (ring >> 1) & 1)) {
                if (!started && mbar_test_wait(&k_full[nr % Sh::kKStages], (nr / Sh::kKStages) & 1)) {
                  start_s(nr, j + 2 == item.ntiles);
                  started = true;
                }
                if (global_timer_ns() - t0 > kWaitLimitNs) {
                  ok = false;
                  break;
                }
              }
              if (ok) ok = mbar_wait_bounded(&v_full[ring % Sh::kVStages], (ring / Sh::kVStages) & 1);
              if (!ok) break;
              tc_fence_after();
              issue_pv(ring & 1, ring, j > 0);
              umma_commit(&v_empty[ring % Sh::kVStages]);
              umma_commit(&o_done[0]);
              if (!started) start_s(nr, j + 2 == item.ntiles);
            }
            ring0 += item.ntiles;
            if (ok && aborted()) ok = false;
            ++ig[0];
            continue;
          }
          if (kGroups == 2 && item.pair()) {
            // tile j belongs to group j & 1
            auto start_s = [&](int j) {  // S of tile j, and what its products free
              const int g = j & 1, ring = ring0 + j;
              if (!(j == 0 && pre)) {
                ok = ok && mbar_wait_bounded(&k_full[ring % Sh::kKStages], (ring / Sh::kKStages) & 1);
                if (ok && j < 2) ok = mbar_wait_bounded(&q_full[g], ig[g] & 1);
                if (!ok) return;
                tc_fence_after();
                issue_s(g, ring);
                if (j + 2 >= item.ntiles) umma_commit(&q_empty[g]);
              }
              umma_commit(&k_empty[ring % Sh::kKStages]);
            };
            for (int j = 0; ok && j < min(2, item.ntiles); ++j) start_s(j);
            for (int j = 0; ok && j < item.ntiles; ++j) {
              const int g = j & 1, ring = ring0 + j;
              ok = mbar_wait_bounded(&p_full[g], tcnt[g] & 1);
              ++tcnt[g];
              if (ok) ok = mbar_wait_bounded(&v_full[ring % Sh::kVStages], (ring / Sh::kVStages) & 1);
              if (!ok) break;
              tc_fence_after();
              issue_pv(g, ring, j >= 2);
              umma_commit(&v_empty[ring % Sh::kVStages]);
              if (j + 2 < item.ntiles) start_s(j + 2);
              else umma_commit(&o_done[g]);
            }
            ring0 += item.ntiles;
            if (ok && aborted()) ok = false;
#pragma unroll
            for (int g = 0; g < kGroups; ++g) ig[g] += item.nt[g] > 0;
            continue;
          }
          ok = mbar_wait_bounded(&k_full[ring0 % Sh::kKStages], (ring0 / Sh::kKStages) & 1);
#pragma unroll
          for (int g = 0; g < kGroups; ++g)
            if (ok && item.nt[g] > 0 && !(g == 0 && pre)) ok = mbar_wait_bounded(&q_full[g], ig[g] & 1);
          if (!ok || aborted()) {
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll
          for (int g = 0; g < kGroups; ++g) {
            if (item.nt[g] == 0 || (g == 0 && pre)) continue;
            issue_s(g, ring0);
            if (item.nt[g] == 1) umma_commit(&q_empty[g]);  // the group's last S of the item
          }
          umma_commit(&k_empty[ring0 % Sh::kKStages]);
          const int ring_next = ring0 + item.ntiles;
          // group 0's first S of the next item, if everything it reads is
          // there (never waits)
          auto try_early = [&]() {
            if (early) return;
            if (!have_nx) {
              const int slot = it & 1;
              if (!mbar_test_wait(&item_full[slot], (it >> 1) & 1)) return;
              nx = items[slot];
              mbar_arrive(&item_empty[slot]);
              ++it;
              have_nx = true;
            }
            if (nx.kind != 1) return;
            if (!mbar_test_wait(&k_full[ring_next % Sh::kKStages], (ring_next / Sh::kKStages) & 1) ||
                !mbar_test_wait(&q_full[0], (ig[0] + 1) & 1))
              return;
            tc_fence_after();
            issue_s(0, ring_next);
            if (nx.nt[0] == 1) umma_commit(&q_empty[0]);
            early = true;
          };
          for (int j = 0; ok && j < item.ntiles; ++j) {
            const int ring = ring0 + j;
            bool v_ready = false, k_ready = false;
#pragma unroll
            for (int g = 0; g < kGroups; ++g) {
              if (!ok || j >= item.nt[g]) continue;
              if (g == 1 && j + 1 >= item.nt[0]) {
                // group 0 is done with this item: look for its next one while
                // group 1's P is not there yet
                const unsigned long long t0 = global_timer_ns();
                while (!mbar_test_wait(&p_full[1], tcnt[1] & 1)) {
                  try_early();
                  if (global_timer_ns() - t0 > kWaitLimitNs) break;
                }
              }
              ok = mbar_wait_bounded(&p_full[g], tcnt[g] & 1);
              ++tcnt[g];
              if (!ok) break;
              if (!v_ready) {
                ok = mbar_wait_bounded(&v_full[ring % Sh::kVStages], (ring / Sh::kVStages) & 1);
                if (!ok) break;
                v_ready = true;
              }
              tc_fence_after();
              issue_pv(g, ring, j > 0);
              // the tile's last P . V: its V slot is free once that has run
              if (g == kGroups - 1 || j >= item.nt[1]) umma_commit(&v_empty[ring % Sh::kVStages]);
              if (j + 1 < item.nt[g]) {
                if (!k_ready) {
                  ok = mbar_wait_bounded(&k_full[(ring + 1) % Sh::kKStages], ((ring + 1) / Sh::kKStages) & 1);
                  if (!ok) break;
                  k_ready = true;
                }
                issue_s(g, ring + 1);
                if (j + 2 == item.nt[g]) umma_commit(&q_empty[g]);
              } else {
                umma_commit(&o_done[g]);  // the group's last product of the item
              }
            }
            if (!ok) break;
            if (j + 1 < item.ntiles) umma_commit(&k_empty[(ring + 1) % Sh::kKStages]);
          }
          ring0 = ring_next;
          if (ok && aborted()) ok = false;
#pragma unroll
          for (int g = 0; g < kGroups; ++g) ig[g] += item.nt[g] > 0;
        }
        if (!ok) abort_cta();
        umma_commit(mma_done);  // every product issued above has completed when this arrives
        mbar_wait_bounded(mma_done, 0);
      }
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------ softmax
    if constexpr (kGroups == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kCtRegsSoftmax));
    const int g = warp >> 2;                            // warpgroup = row tile
    const int quarter = warp & 3;
    const int r = 32 * quarter + lane;                  // row in the tile = tensor-memory lane
    const uint32_t lane_off = (uint32_t)(32 * quarter) << 16;
    const uint32_t tmem_o = tmem + 256 * g + 128 + lane_off;
    const float sl2 = a.scale_y;
    // scores may stay raw until the exponent when nothing but a positive
    // scale stands between (the max commutes with it)
    const bool raw = !CAP && !BIAS && sl2 > 0.f;
    const float mul = raw ? sl2 : 1.f;
    int it = 0, ring0 = 0, ig = 0, tcnt = 0, npair = 0;
    int redo = -1;                                      // the item noted last
    bool ok = true;
    while (true) {
      const int slot = it & 1;
      ok = mbar_wait_bounded(&item_full[slot], (it >> 1) & 1);
      if (!__all_sync(0xffffffffu, ok)) {
        ok = false;
        break;
      }
      const CtItem item = items[slot];
      __syncwarp();
      if (lane == 0) mbar_arrive(&item_empty[slot]);
      ++it;
      if (item.kind < 0) break;
      // this thread's row: query i of the sequence, head h (rows past the
      // item's last query mirror it and are not written)
      const bool pair = kGroups == 2 && item.pair();
      const int qi = (pair ? 0 : g * per) + (r >> ta.gshift);
      const int queries = min(kGroups * per, item.qlen - item.i0);
      const bool real_row = qi < queries;
      const bool live = __any_sync(0xffffffffu, real_row);  // a warp without rows only keeps the barriers going
      const int i = item.i0 + min(qi, queries - 1);
      const int h = (item.sub << ta.gshift) + (r & (gheads - 1));
      const size_t q_row = (size_t)(item.q0 + i) * a.H + h;
      T *orow = reinterpret_cast<T *>(a.out) + q_row * D;
      const int my_tiles = item.kind == 1 ? (g == 0 ? item.nt[0] : item.nt[1]) : 0;
      if (item.kind == 2 && real_row) {
        for (int c = 0; c < D / 8; ++c) reinterpret_cast<uint4 *>(orow)[c] = make_uint4(0, 0, 0, 0);
      }
      if (my_tiles == 0) {
        ring0 += item.ntiles;
        continue;
      }
      ChunkSeq sq;
      sq.q0 = item.q0;
      sq.qlen = item.qlen;
      sq.n = item.n;
      sq.prefix = a.prefix ? min(max(__ldg(a.prefix + item.b), 0), item.n) : 0;
      int lo, hi;
      chunk_visible(a, sq, i, lo, hi);
      const int p = item.n - item.qlen + i;
      const float slope = BIAS ? __ldg(a.slopes + h) * kLog2e : 0.f;
      float2 d_bias[4];                                 // slope x columns 0 .. 7
#pragma unroll
      for (int c = 0; c < 4; ++c) d_bias[c] = make_float2(slope * (float)(2 * c), slope * (float)(2 * c + 1));
      float m_used = -INFINITY, l = 0.f;
      for (int j = 0; j < my_tiles; ++j) {
        const int jt = pair ? 2 * j + g : j;           // the item's tile
        const int t0 = item.t0 + jt * kCtTile;
        const int ring = ring0 + jt;
        const int sb = kGroups == 2 ? g : ring & 1;    // its S (and P) and their barriers
        const uint32_t tmem_sp = tmem + Sh::s_col(sb) + lane_off;
        ok = mbar_wait_bounded(&s_full[sb], (kGroups == 2 ? tcnt : ring >> 1) & 1);
        ++tcnt;
        if (!__all_sync(0xffffffffu, ok && !aborted())) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (live) {
        uint32_t sa[64], sb[64];
        tmem_ld64_nowait(tmem_sp, sa);
        tmem_ld64_nowait(tmem_sp + 64, sb);
        tmem_wait_ld_bind64(sa);
        reg_bind64(sb);
        float sc[128];
#pragma unroll
        for (int c = 0; c < 64; ++c) {
          sc[c] = __uint_as_float(sa[c]);
          sc[64 + c] = __uint_as_float(sb[c]);
        }
        const bool cut = t0 < lo || t0 + kCtTile > hi;   // some of the tile is hidden from the row
        auto hide = [&](float v) {  // v in the hidden columns: a bit per column, not two comparisons
#pragma unroll
          for (int k = 0; k < 128; k += 32) {
            const int from = min(max(lo - t0 - k, 0), 32), to = min(max(hi - t0 - k, 0), 32);
            const uint32_t seen_bits = (uint32_t)((1ull << to) - 1ull) & ~(uint32_t)((1ull << from) - 1ull);
#pragma unroll
            for (int c = 0; c < 32; ++c) sc[k + c] = (seen_bits >> c) & 1u ? sc[k + c] : v;
          }
        };
        // Where a row sees no key past its position, its bias slope (j - p) is
        // linear in the column: slope (c mod 8) goes in with the score, and
        // the rest, one number per 8 columns, only into the max and the
        // exponent.
        const bool linear = BIAS && (!a.prefix || __all_sync(0xffffffffu, t0 + kCtTile - 1 <= p));
        const float base = BIAS ? slope * (float)(t0 - p) : 0.f;
        auto block_bias = [&](int c) { return linear ? fmaf(slope, (float)(c & ~7), base) : 0.f; };
        // Capped scores: |q . k| over the tile picks the way to its tanh.  The
        // usual tile is near 0, where 4 terms do; without a bias they are
        // then evaluated inside the exponent, straight from the raw scores.
        bool fused = false;
        float mx_raw = -INFINITY;
        if (CAP == kCapLarge) {
          // the scores of a large cap are near 0 as a rule: then no branch per score
          if (cut) hide(0.f);
          float far = 0.f;
#pragma unroll
          for (int c = 0; c < 128; ++c) far = fmaxf(far, fabsf(sc[c]));
          if (__all_sync(0xffffffffu, !real_row || far * fabsf(a.cap_ratio) < kCapNear)) {
#pragma unroll
            for (int c = 0; c < 128; ++c) sc[c] = chunk_cap_near(a, sc[c]);
          } else {
#pragma unroll
            for (int c = 0; c < 128; ++c) sc[c] = chunk_cap(a, sc[c]);
          }
        } else if (CAP && !BIAS) {
          if (cut) {  // hidden columns hold whatever was there: they have no say
            hide(0.f);
          }
          float mn_raw = INFINITY;
#pragma unroll
          for (int c = 0; c < 128; c += 2) {
            mx_raw = max3f(mx_raw, sc[c], sc[c + 1]);
            mn_raw = min3f(mn_raw, sc[c], sc[c + 1]);
          }
          const float far = real_row ? fmaxf(mx_raw, -mn_raw) : 0.f;
          fused = __all_sync(0xffffffffu, !cut && far <= a.cap_small);
          if (!fused && __all_sync(0xffffffffu, far <= a.cap_mid)) {
            const float2 rt = kept_pair(a.cap_ratio);
            float2 kc[6];
#pragma unroll
            for (int e = 0; e < 6; ++e) kc[e] = kept_pair(a.cap_c[e]);
#pragma unroll
            for (int c = 0; c < 128; c += 2) {
              const float2 x = fmul2(make_float2(sc[c], sc[c + 1]), rt), z = fmul2(x, x);
              float2 q = ffma2(z, kc[5], kc[4]);
#pragma unroll
              for (int e = 3; e >= 0; --e) q = ffma2(z, q, kc[e]);
              q = fmul2(x, q);
              sc[c] = q.x;
              sc[c + 1] = q.y;
            }
          } else if (!fused) {
#pragma unroll
            for (int c = 0; c < 128; ++c) sc[c] = chunk_capped(sc[c] * sl2, a.cap_log2);
          }
        } else if (CAP) {
#pragma unroll
          for (int c = 0; c < 128; ++c) sc[c] = chunk_capped(sc[c] * sl2, a.cap_log2);
        } else if (!raw && !BIAS) {
#pragma unroll
          for (int c = 0; c < 128; ++c) sc[c] *= sl2;
        }
        if (BIAS) {
          const float f = CAP ? 1.f : sl2;
          if (linear) {
            const float2 f2 = kept_pair(f);
#pragma unroll
            for (int c = 0; c < 128; c += 2) {
              const float2 x = ffma2(make_float2(sc[c], sc[c + 1]), f2, d_bias[(c >> 1) & 3]);
              sc[c] = x.x;
              sc[c + 1] = x.y;
            }
          } else {
            const float away = (float)(t0 - p);
#pragma unroll
            for (int c = 0; c < 128; ++c) sc[c] = fmaf(sc[c], f, -slope * fabsf(away + (float)c));
          }
        }
        if (cut) {
          hide(-INFINITY);
        }
        float mx = -INFINITY;
        if (fused) {
          const float z = mx_raw * mx_raw;
          mx = mx_raw * fmaf(z, fmaf(z, fmaf(z, a.cap_k[3], a.cap_k[2]), a.cap_k[1]), a.cap_k[0]);
        } else if (BIAS) {
#pragma unroll
          for (int c = 0; c < 128; c += 8) {
            float m8 = max3f(sc[c], sc[c + 1], sc[c + 2]);
            m8 = max3f(m8, sc[c + 3], sc[c + 4]);
            m8 = max3f(m8, sc[c + 5], sc[c + 6]);
            mx = fmaxf(mx, fmaxf(m8, sc[c + 7]) + block_bias(c));
          }
        } else {
#pragma unroll
          for (int c = 0; c < 128; c += 2) mx = max3f(mx, sc[c], sc[c + 1]);
          if (raw) mx *= sl2;
        }
        // the reference max moves only when the row max exceeds it by 2^8
        const float m_new = (mx > m_used + 8.f) ? mx : m_used;
        const float ref = chunk_ref(m_new);            // nothing seen yet: weights 0, not NaN
        const float alpha = fast_exp2(m_used - ref);   // 0 before the first key seen
        const bool rescale = __any_sync(0xffffffffu, m_new != m_used) && j > 0;
        l *= alpha;
        m_used = m_new;
        // The sum takes the weights as they are, the product with V rounds them
        // to T.  Summing the rounded ones makes up for part of that (against 64
        // bits, capped prompts 0.00210 for 0.00228, packed documents 0.00180 for
        // 0.00191; rounding the output alone gives 0.00166) and costs the
        // unpacking: 184 us for 168, 302 for 279.
        float2 lsum = make_float2(0.f, 0.f);
        auto weights = [&](const auto &exponent) {       // P = 2^exponent(pair), and its sum
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            uint32_t pk[32];
#pragma unroll
            for (int c2 = 0; c2 < 32; ++c2) {
              const int c = 64 * hf + 2 * c2;
              float2 x = exponent(make_float2(sc[c], sc[c + 1]), c);
              x.x = fast_exp2(x.x);
              x.y = fast_exp2(x.y);
              lsum = fadd2(lsum, x);
              pk[c2] = PackPair<T>::pack(x.x, x.y);
            }
            tmem_st32u_nowait(tmem_sp + 32 * hf, pk);
          }
        };
        const float2 nref = kept_pair(-ref);
        if (CAP == kCapUsual && !BIAS && fused) {
          const float2 k0 = kept_pair(a.cap_k[0]), k1 = kept_pair(a.cap_k[1]);
          const float2 k2 = kept_pair(a.cap_k[2]), k3 = kept_pair(a.cap_k[3]);
          weights([&](float2 x, int) {
            const float2 z = fmul2(x, x);
            return ffma2(x, ffma2(z, ffma2(z, ffma2(z, k3, k2), k1), k0), nref);
          });
        } else if (BIAS) {
          weights([&](float2 x, int c) {
            const float e = block_bias(c) - ref;
            return fadd2(x, make_float2(e, e));
          });
        } else if (CAP) {
          weights([&](float2 x, int) { return fadd2(x, nref); });
        } else {
          const float2 mul2 = kept_pair(mul);
          weights([&](float2 x, int) { return ffma2(x, mul2, nref); });
        }
        tmem_wait_st();
        l += lsum.x + lsum.y;
        // O is final for tile j - 1 here with two groups (the commit that
        // signalled S_g(j) covers P_g(j - 1) . V); with one it may still run
        if (rescale) {
          if (kGroups == 1) {
            ok = mbar_wait_bounded(&o_done[0], (ring - 1) & 1);
            tc_fence_after();
          }
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            float v[32];
            tmem_ld32(tmem_o + 32 * c, v);
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] *= alpha;
            tmem_st32(tmem_o + 32 * c, v);
          }
        }
        }
        if (kGroups == 1) {
          // the product before the item's last is waited for here, so that the
          // wait for the last one below looks at its phase and no other
          if (j > 0 && j + 1 == my_tiles) ok = ok && mbar_wait_bounded(&o_done[0], (ring - 1) & 1);
          if (!__all_sync(0xffffffffu, ok)) {
            ok = false;
            break;
          }
        }
        // the tile's values that no row of the unit sees become 0 (they may
        // hold anything, and 0 * NaN would poison the product)
        const bool ragged = t0 < item.lo || t0 + kCtTile > item.t1;
        if (ragged) {
          ok = mbar_wait_bounded(&v_full[ring % Sh::kVStages], (ring / Sh::kVStages) & 1);
          if (!__all_sync(0xffffffffu, ok)) {
            ok = false;
            break;
          }
          if (t0 + r < item.lo || t0 + r >= item.t1) {
            uint8_t *vrow = sm + Sh::kVOff + (ring % Sh::kVStages) * Sh::kKVBytes + r * 128;
#pragma unroll
            for (int rg = 0; rg < Sh::kRegions; ++rg)
#pragma unroll
              for (int c = 0; c < 8; ++c)
                *reinterpret_cast<uint4 *>(vrow + rg * kCtKVRegion + c * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_shared();  // the zeros before the product reads them
        }
        tc_fence_before();
        mbar_arrive(&p_full[sb]);
      }
      if (!ok) break;
      if (kGroups == 2) {
        ok = mbar_wait_bounded(&o_done[g], ig & 1);
      } else {
        ok = mbar_wait_bounded(&o_done[0], (ring0 + my_tiles - 1) & 1);
      }
      ++ig;
      if (!__all_sync(0xffffffffu, ok && !aborted())) {
        ok = false;
        break;
      }
      tc_fence_after();
      float scale0 = 1.f, scale1 = 0.f;                 // of this group's O, and of group 1's in a shared tile
      if (pair && item.nt[1] > 0) {
        if (g == 1) {                                   // hand the state over, and go on once it has been read
          s_pair[r] = m_used;
          s_pair[kCtRows + r] = l;
          tc_fence_before();
          mbar_arrive(pair_full);
          ok = __all_sync(0xffffffffu, mbar_wait_bounded(pair_empty, npair & 1));
          ++npair;
          if (!ok) break;
          ring0 += item.ntiles;
          continue;
        }
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(pair_full, npair & 1));
        ++npair;
        if (!ok) break;
        tc_fence_after();
        const float m1 = s_pair[r], l1 = s_pair[kCtRows + r];
        const float M = fmaxf(m_used, m1), ref = chunk_ref(M);
        scale0 = fast_exp2(m_used - ref);
        scale1 = fast_exp2(m1 - ref);
        m_used = M;
        l = l * scale0 + l1 * scale1;
      }
      // the row: O / l, or with several parts (m, l, O) to the workspace
      const bool seen = hi > lo;
      const float inv_l = seen ? 1.f / l : 0.f;
      const size_t at = q_row * a.max_parts + item.part;
      float odd = 0.f;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        if (!live) break;
        float v[32];
        tmem_ld32(tmem_o + 32 * c, v);
        if (pair && item.nt[1] > 0) {
          float v1[32];
          tmem_ld32(tmem_o + 256 + 32 * c, v1);
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = fmaf(v[e], scale0, v1[e] * scale1);
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) odd = fmaf(v[e], 0.f, odd);
        if (!real_row) continue;
        if (item.parts() == 1) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 16; ++e)
            pk[e] = seen ? PackPair<T>::pack(v[2 * e] * inv_l, v[2 * e + 1] * inv_l) : 0u;
          uint4 *dst = reinterpret_cast<uint4 *>(orow + 32 * c);
#pragma unroll
          for (int c4 = 0; c4 < 4; ++c4) dst[c4] = make_uint4(pk[4 * c4], pk[4 * c4 + 1], pk[4 * c4 + 2], pk[4 * c4 + 3]);
        } else {
          float4 *dst = reinterpret_cast<float4 *>(a.ws_o + at * D + 32 * c);
#pragma unroll
          for (int c4 = 0; c4 < 8; ++c4) dst[c4] = make_float4(v[4 * c4], v[4 * c4 + 1], v[4 * c4 + 2], v[4 * c4 + 3]);
        }
      }
      if (pair && item.nt[1] > 0) {
        tc_fence_before();
        mbar_arrive(pair_empty);
      }
      if (real_row && item.parts() > 1) {
        a.ws_m[at] = m_used;
        a.ws_l[at] = l;
      }
      // rows that are not finite although a key of the part is hidden from
      // them: noted for the end
      const unsigned again = __ballot_sync(0xffffffffu, real_row && odd != 0.f && (lo > item.t0 || hi < item.t1));
      if (again) {
        if (lane == 0) ta.redo[(size_t)item.w * kSoftmaxWarps + warp] = make_int2((int)again, redo);
        redo = item.w;
      }
      ring0 += item.ntiles;
    }
    if (!ok && lane == 0) abort_cta();
    __syncwarp();
    while (ok && redo >= 0) {
      const volatile int2 *note = ta.redo + (size_t)redo * kSoftmaxWarps + warp;
      const unsigned rows = (unsigned)note->x;
      const int next = note->y;
      ct_redo<D, T, BIAS>(ta, (unsigned)redo, rows, g, r);
      redo = next;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kSoftmaxWarps) tmem_dealloc(tmem, Sh::kTmemCols);
  if (tid == 0) {
    // the last CTA puts the counters back (every claim's value was used
    // before the barrier, so it is performed already)
    if (atomicAdd(a.ws_cnt + 1, 1) == (int)gridDim.x - 1) {
      atomicExch(a.ws_cnt, 0);
      atomicExch(a.ws_cnt + 1, 0);
    }
  }
}

// --------------------------------------------------------------------- merge

// One warp per output row: out = sum_p o_p 2^(m_p - M) / sum_p l_p 2^(m_p - M)
// over the row's parts; rows of units with one part are written already.
// blockIdx.y: the part-0 entries of the unit list lead to the rows.
template <int D, typename T>
__global__ void __launch_bounds__(256) pkv_chunk_merge_kernel(const __grid_constant__ CtArgs ta) {
  griddep_wait();
  const ChunkArgs &a = ta.c;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int kRows = ct_groups(D) * kCtRows;
  const int per = kRows >> ta.gshift;
  const int units = *ta.n_units;
  // 8 rows (one per warp) of a unit's rows x subs per block of work
  const long long blocks_per_unit = (long long)ta.subs * (kRows / 8);
  for (long long w = blockIdx.x; w < units * blocks_per_unit; w += gridDim.x) {
    const int un = (int)(w / blocks_per_unit), rest = (int)(w - un * blocks_per_unit);
    const CtUnit u = ta.units[un];
    if (u.part != 0 || u.nparts == 1) continue;
    const int sub = rest / (kRows / 8), r = (rest % (kRows / 8)) * 8 + warp;
    const ChunkSeq s = chunk_seq(a, u.b, false);
    const int i = u.i0 + (r >> ta.gshift);
    if (i >= min(s.qlen, u.i0 + per)) continue;
    const size_t row = (size_t)(s.q0 + i) * a.H + (sub << ta.gshift) + (r & ((1 << ta.gshift) - 1));
    int lo, hi;
    chunk_visible(a, s, i, lo, hi);
    const float *pm = a.ws_m + row * a.max_parts, *pl = a.ws_l + row * a.max_parts;
    constexpr int EPL = D / 32;
    float M = -INFINITY;
    for (int p = lane; p < u.nparts; p += 32) M = fmaxf(M, pm[p]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    const float ref = chunk_ref(M);
    float L = 0.f, acc[EPL];
#pragma unroll
    for (int e = 0; e < EPL; ++e) acc[e] = 0.f;
#pragma unroll 4
    for (int p = 0; p < u.nparts; ++p) {
      const float wt = fast_exp2(pm[p] - ref);
      L = fmaf(pl[p], wt, L);
      const float *po = a.ws_o + (row * a.max_parts + p) * D + lane * EPL;
#pragma unroll
      for (int e = 0; e < EPL; ++e) acc[e] = fmaf(po[e], wt, acc[e]);
    }
    const float inv = hi > lo ? 1.f / L : 0.f;
    T *orow = reinterpret_cast<T *>(a.out) + row * D + lane * EPL;
#pragma unroll
    for (int e = 0; e < EPL; ++e) orow[e] = from_f32<T>(hi > lo ? acc[e] * inv : 0.f);
  }
}

// ---------------------------------------------------------------- host side

// The plan's launch (pkv_chunk_tc.cu).
bool launch_ct_plan(const CtArgs &a, cudaStream_t stream);

template <typename... KArgs, typename... Args>
static bool launch_after(void (*kern)(KArgs...), int ctas, int threads, size_t smem, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...) == cudaSuccess;
}

template <int D, typename T, int CAP, bool BIAS>
static pkv_status launch_ct(const CtArgs &a, const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv, int sms,
                            cudaStream_t stream) {
  auto kern = pkv_chunk_tc_kernel<D, T, CAP, BIAS>;
  static int configured[64] = {0};
  if (!allow_smem(kern, CtShape<D>::kSmem, configured)) return PKV_ERR_CUDA;
  if (!launch_ct_plan(a, stream)) return PKV_ERR_CUDA;
  const long long most = (long long)a.units_cap * a.subs;
  const int ctas = (int)(most < sms ? most : sms);
  if (!launch_after(kern, ctas, CtShape<D>::kThreads, CtShape<D>::kSmem, stream, mq, mk, mv, a)) return PKV_ERR_CUDA;
  if (a.c.max_parts > 1 && !launch_after(pkv_chunk_merge_kernel<D, T>, sms * 8, 256, 0, stream, a)) return PKV_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

template <int D, typename T>
static pkv_status launch_ct_form(const CtArgs &a, const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv,
                                 int sms, cudaStream_t s) {
  return chunk_forms(a.c, [&](auto cap, auto bias) { return launch_ct<D, T, cap.value, bias.value>(a, mq, mk, mv, sms, s); });
}

template <int D>
static pkv_status launch_ct_dt(const CtArgs &a, pkv_dtype dt, const CUtensorMap &mq, const CUtensorMap &mk,
                               const CUtensorMap &mv, int sms, cudaStream_t s) {
  return dt == PKV_BF16 ? launch_ct_form<D, __nv_bfloat16>(a, mq, mk, mv, sms, s)
                        : launch_ct_form<D, __half>(a, mq, mk, mv, sms, s);
}

}  // namespace pkv
