// pkv_chunk_tc.cu -- the tcgen05 chunk attention's plan kernel and host side,
// and its instances for head_dim 64 and 128 (pkv_chunk_tc.cuh has the kernel).
#include "pkv_chunk_tc.cuh"

namespace pkv {

// ---------------------------------------------------------------------- plan

// Keys that the rows of queries [i0, i1) see: the first, and one past the
// last.  kCtLanes lanes of a warp work on a tile together.  Without kv_starts
// both bounds rise with the query; with them the first key is the least over
// the queries that see any, 16 loads of a lane in flight.
constexpr int kCtLanes = 4;
__device__ __forceinline__ void ct_span(const ChunkArgs &a, const ChunkSeq &s, int i0, int i1, int sub, int &lo, int &hi) {
  lo = 0x7fffffff;
  hi = 0;
  auto take = [&](int i, int start) {
    const int p = s.n - s.qlen + i, h = max(p + 1, s.prefix);
    const int l = max(a.window > 0 ? max(0, p - a.window + 1) : 0, start);
    if (l < h) {
      lo = min(lo, l);
      hi = max(hi, h);
    }
  };
  if (a.starts) {
    constexpr int kU = 16;
    for (int i = i0 + sub; i < i1; i += kCtLanes * kU) {
      int st[kU];
#pragma unroll
      for (int k = 0; k < kU; ++k) st[k] = i + kCtLanes * k < i1 ? __ldg(a.starts + s.q0 + i + kCtLanes * k) : 0x7fffffff;
#pragma unroll
      for (int k = 0; k < kU; ++k)
        if (i + kCtLanes * k < i1) take(i + kCtLanes * k, st[k]);
    }
  } else if (i1 > i0) {
    take(i0, 0);
    take(i1 - 1, 0);
  }
#pragma unroll
  for (int o = kCtLanes / 2; o > 0; o >>= 1) {
    lo = min(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = max(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
}

__global__ void __launch_bounds__(kCtPlanThreads) pkv_chunk_plan_kernel(const CtArgs a) {
  __shared__ int s_cls[kCtClasses];
  __shared__ int s_warp[32];
  __shared__ int s_first[kCtPlanThreads];    // B <= kCtPlanThreads: a sequence's first tile
  __shared__ ChunkSeq s_seq[kCtPlanThreads];
  griddep_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (ct_groups(a.c.D) * kCtRows) >> a.gshift;   // queries per unit
  const bool one_scan = a.c.B <= kCtPlanThreads;   // tiles are then found by a search, else listed first
  for (int i = tid; i < kCtClasses; i += kCtPlanThreads) s_cls[i] = 0;
  int total = 0;
  for (int base = 0; base < a.c.B; base += kCtPlanThreads) {
    const int b = base + tid;
    int cnt = 0;
    if (b < a.c.B) {
      const ChunkSeq s = chunk_seq(a.c, b, true);
      cnt = min((s.qlen + per - 1) / per, kCtSat);
      if (one_scan) s_seq[b] = s;
    }
    int inc = cnt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc = min(inc + y, kCtSat);
    }
    if (lane == 31) s_warp[warp] = inc;
    __syncthreads();
    int v = s_warp[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v = min(v + y, kCtSat);
    }
    const int before = __shfl_sync(0xffffffffu, v, max(warp - 1, 0));
    const int at = min(total + min((warp ? before : 0) + (inc - cnt), kCtSat), kCtSat);
    total = min(total + __shfl_sync(0xffffffffu, v, 31), kCtSat);
    if (one_scan) {
      s_first[tid] = at;
    } else {
      for (int t = 0; t < cnt && at + t < a.tiles_cap; ++t) a.tiles[at + t] = make_int4(b, t, 0, 0);
    }
    __syncthreads();
  }
  // (query offsets that overlap could make more tiles than there is room for)
  if (total > a.tiles_cap && tid == 0) raise_flag(a.c.err, PKV_FLAG_QUERY_LEN);
  total = min(total, a.tiles_cap);
  __syncthreads();
  // each tile's parts: counted by their key tiles, then placed by them
  for (int pass = 0; pass < 2; ++pass) {
    for (int n0 = 0; n0 < total; n0 += kCtPlanThreads / kCtLanes) {
      const int n = n0 + tid / kCtLanes, sub = tid & (kCtLanes - 1);
      int4 bt = make_int4(0, 0, 0, 0);
      if (n < total && (pass == 1 || !one_scan)) bt = a.tiles[n];
      int lo = bt.z, hi = bt.w;
      if (pass == 0) {
        ChunkSeq s = {0, 0, 0, 0};
        if (n < total && one_scan) {           // the last sequence that starts at or before tile n
          int b = 0, len = a.c.B;
          while (len > 1) {
            const int half = len >> 1;
            if (s_first[b + half] <= n) b += half;
            len -= half;
          }
          bt.x = b;
          bt.y = n - s_first[b];
          s = s_seq[b];
        } else if (n < total) {
          s = chunk_seq(a.c, bt.x, false);
        }
        ct_span(a.c, s, bt.y * per, min(s.qlen, bt.y * per + per), sub, lo, hi);
        if (n < total && sub == 0) a.tiles[n] = make_int4(bt.x, bt.y, lo, hi);
      }
      const int i0 = bt.y * per;
      if (n >= total) continue;
      const int base = hi > 0 ? lo & -(1 << a.bshift) : 0;
      const int nparts = max(1, (hi - base + a.c.P - 1) / a.c.P);
      for (int p = sub; p < nparts; p += kCtLanes) {
        const int t0 = base + p * a.c.P, t1 = min(hi, t0 + a.c.P);
        const int cls = kCtClasses - 1 - min(kCtClasses - 1, (t1 - t0 + kCtTile - 1) / kCtTile);
        const int at = atomicAdd(&s_cls[cls], 1);
        if (pass && at < a.units_cap) {
          CtUnit u = {bt.x, i0, p, nparts, t0, t1, lo, 0};
          reinterpret_cast<int4 *>(a.units + at)[0] = make_int4(u.b, u.i0, u.part, u.nparts);
          reinterpret_cast<int4 *>(a.units + at)[1] = make_int4(u.t0, u.t1, u.lo, u.pad);
        }
      }
    }
    __syncthreads();
    if (pass == 0) {             // counts -> first places
      int v = tid < kCtClasses ? s_cls[tid] : 0, inc = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
      }
      if (lane == 31) s_warp[warp] = inc;
      __syncthreads();
      int before = 0, all = 0;
      for (int i = 0; i < kCtClasses / 32; ++i) {
        if (i < warp) before += s_warp[i];
        all += s_warp[i];
      }
      if (tid < kCtClasses) s_cls[tid] = before + inc - v;
      if (tid == 0) *a.n_units = min(all, a.units_cap);
      __syncthreads();
    }
  }
}

// ---------------------------------------------------------------- host side

static long long ct_tiles_cap(int B, long long total_q, int max_q, int per) {
  const long long by_rows = total_q / per + B, by_seq = (long long)B * ((max_q + per - 1) / per);
  return by_rows < by_seq ? by_rows : by_seq;
}

int chunk_tc_gshift(int G) {     // log2 of the heads packed in a tile
  int s = 0;
  while (s < 7 && G % (2 << s) == 0) ++s;
  return s;
}

long long chunk_tc_items(int B, long long total_q, int H, int G, int D, int max_q) {
  const int sh = chunk_tc_gshift(G);
  return ct_tiles_cap(B, total_q, max_q, (ct_groups(D) * kCtRows) >> sh) * (H >> sh);
}

static size_t ct_align(size_t x) { return (x + 255) & ~size_t(255); }

// Notes of rows to do again, of an item: one per softmax warp.
static size_t ct_notes(int D) { return 4 * ct_groups(D) * sizeof(int2); }

size_t chunk_tc_scratch(int B, long long total_q, int H, int G, int D, int max_q, long long parts) {
  const int sh = chunk_tc_gshift(G);
  const long long tiles = ct_tiles_cap(B, total_q, max_q, (ct_groups(D) * kCtRows) >> sh);
  return 256 + ct_align(tiles * sizeof(int4)) + ct_align(tiles * parts * sizeof(CtUnit)) +
         ct_align(tiles * parts * (H >> sh) * ct_notes(D));
}

bool launch_ct_plan(const CtArgs &a, cudaStream_t stream) {
  pkv_chunk_plan_kernel<<<1, kCtPlanThreads, 0, stream>>>(a);
  return cudaGetLastError() == cudaSuccess;
}

// head_dim 192 and 256 (pkv_chunk_tc_wide.cu: the instances compile side by side)
pkv_status launch_chunk_tc_wide(const CtArgs &a, pkv_dtype dt, const CUtensorMap &mq, const CUtensorMap &mk,
                                const CUtensorMap &mv, int sms, cudaStream_t stream);

// `scratch`: chunk_tc_scratch(...) bytes of the workspace, 256-byte aligned.
pkv_status launch_chunk_tc(const ChunkArgs &c, pkv_dtype dt, char *scratch, int sms, cudaStream_t stream) {
  CtArgs a;
  memset(&a, 0, sizeof a);
  a.c = c;
  a.gshift = chunk_tc_gshift(c.G);
  a.subs = c.H >> a.gshift;
  a.bshift = c.bs % 64 == 0 ? 6 : c.bs % 32 == 0 ? 5 : 4;
  const long long tiles = ct_tiles_cap(c.B, c.total_q, c.max_q, (ct_groups(c.D) * kCtRows) >> a.gshift);
  if (tiles >= kCtSat || tiles * c.max_parts * a.subs > 0x7fffffffLL) return PKV_ERR_UNSUPPORTED;
  a.tiles_cap = (int)tiles;
  a.units_cap = (int)(tiles * c.max_parts);
  a.n_units = reinterpret_cast<int *>(scratch);
  scratch += 256;
  a.tiles = reinterpret_cast<int4 *>(scratch);
  scratch += ct_align(tiles * sizeof(int4));
  a.units = reinterpret_cast<CtUnit *>(scratch);
  scratch += ct_align(tiles * c.max_parts * sizeof(CtUnit));
  a.redo = reinterpret_cast<int2 *>(scratch);
  CUtensorMap mq, mk, mv;
  if (!encode_packed_map(&mq, c.q, dt, c.total_q, c.H, c.D, 1 << a.gshift, kCtRows >> a.gshift) ||
      !encode_cache_map(&mk, c.k_cache, dt, c.num_blocks, c.bs, c.KVH, c.D, 1 << a.bshift) ||
      !encode_cache_map(&mv, c.v_cache, dt, c.num_blocks, c.bs, c.KVH, c.D, 1 << a.bshift))
    return PKV_ERR_CUDA;
  switch (c.D) {
    case 64: return launch_ct_dt<64>(a, dt, mq, mk, mv, sms, stream);
    case 128: return launch_ct_dt<128>(a, dt, mq, mk, mv, sms, stream);
  }
  return launch_chunk_tc_wide(a, dt, mq, mk, mv, sms, stream);
}

}  // namespace pkv
