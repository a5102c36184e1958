// pkv_chunk_mma.cu -- chunk attention for bf16 / fp16 and few rows per key:
// single tokens and short drafts, where reading K and V once bounds the call
// (see pkv_chunk.cuh for the rows, masks and scores).
//
// CTA = (part of the context, 16 packed rows of a KV head, sequence), W warps.
// A part is walked in chunks of 16 tokens (block_size is a multiple of 16, so
// a chunk lies in one block); warp w takes chunks w, w + W, ...; chunk c passes
// through stage c mod R of a ring in shared memory, filled by two 5-D TMA boxes
// (the chunk's K and V rows of this head), and the warp that is done with chunk
// c fetches chunk c + R into its stage.  The 16 rows are one m16n8k16 tile:
//   S[16 x 16] = Q K^T, scores and masks, online softmax in registers,
//   O[16 x D] += P V,
// and the warps' states are merged in shared memory at the end.  No barrier
// separates the warps in between; a chunk that every row sees whole (the usual
// one) skips the masks.
#include <string.h>

#include "pkv_chunk.cuh"

namespace pkv {

constexpr int kCmTok = 16;
constexpr int kCmRows = 16;
constexpr int kCmBox = 16 * 128;      // one box: 16 rows of 64 elements

template <int D>
struct CmShape {
  static constexpr int kSteps = D / 16;
  static constexpr int kBoxes = D / 64;
  static constexpr int kStage = 2 * kBoxes * kCmBox;             // K and V of one chunk
  // Two CTAs of 4 warps an SM; at 256, where 12 stages fill the
  // shared memory, one of 8.  (4 warps there left each scheduler one, which
  // waited for its own products: 16 heads on 8192 keys 28.9 us, 22.2 with 8; on
  // 640 whole 18.6 / 16.3; 64 sequences of 4096 62.9 / 58.9.  128 of 1087 lose,
  // 27.0 / 28.8: fewer stages are ahead of the warps.  Two CTAs of 4 warps and 6
  // stages: 8192 keys 29.1, 128 of 1087 in two parts 38.5.)
  static constexpr int kWarps = D <= 192 ? 4 : 8;
  static constexpr int kStages = D <= 64 ? 24 : D <= 128 ? 12 : D <= 192 ? 8 : 12;
  // a stage is always the same warp's: its next chunk cannot be looked for
  // before it is asked for
  static constexpr bool kOwn = kStages % kWarps == 0;
  static constexpr int kRing = kStages * kStage;
  static constexpr int kQStride = D + 8;
  static constexpr int kOStride = D + 8;
  static constexpr bool kQInRegs = D <= 128;
  static constexpr int kSmem = 1024 + kRing + kCmRows * kQStride * 2 + kStages * 8 +
                               4 * (2 * kWarps * kCmRows + 3 * kCmRows) + 4 * (2 * kCmRows + 4 + kStages);
  static_assert(kWarps * kCmRows * kOStride * 4 <= kRing, "the warps' states fit the ring");
  static_assert(kStages >= kWarps, "every warp's first chunk is in the first fill");
};

__device__ __forceinline__ void st_release_cta(int *p, int v) {
  asm volatile("st.release.cta.shared::cta.s32 [%0], %1;" ::"r"(smem_u32(p)), "r"(v) : "memory");
}

// Wait until *p is v; false after kWaitLimitNs.
__device__ __forceinline__ bool flag_wait_bounded(const int *p, int v) {
  auto is = [&]() {
    int x;
    asm volatile("ld.acquire.cta.shared::cta.s32 %0, [%1];" : "=r"(x) : "r"(smem_u32(p)) : "memory");
    return x == v;
  };
  if (is()) return true;
  const unsigned long long t0 = global_timer_ns();
  while (!is()) {
    if (global_timer_ns() - t0 > kWaitLimitNs) return false;
  }
  return true;
}

template <int D, typename T, int CAP, bool BIAS>
__global__ void __launch_bounds__(32 * CmShape<D>::kWarps, 1)
    pkv_chunk_mma_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                         const ChunkArgs a) {
  using Sh = CmShape<D>;
  using Mma = MmaOp<T>;
  constexpr int R = Sh::kStages, W = Sh::kWarps;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  T *sQ = reinterpret_cast<T *>(ring + Sh::kRing);
  uint64_t *bars = reinterpret_cast<uint64_t *>(sQ + kCmRows * Sh::kQStride);
  float *s_wm = reinterpret_cast<float *>(bars + R);           // [W][16]
  float *s_wl = s_wm + W * kCmRows;                              // [W][16]
  float *s_m = s_wl + W * kCmRows;                               // [16]
  float *s_l = s_m + kCmRows;                                    // [16]
  float *s_slope = s_l + kCmRows;                                // [16]
  int *s_lo = reinterpret_cast<int *>(s_slope + kCmRows);        // [16]
  int *s_hi = s_lo + kCmRows;                                    // [16]
  int *s_scratch = s_hi + kCmRows;
  int *s_asked = s_scratch + 4;                                  // [R] chunk that a stage was last filled with

  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  // row chunks of the same keys are neighbours in the grid, so that the second
  // finds in L2 what the first has read
  const int b = blockIdx.y, chunk = blockIdx.x % a.chunks, unit = blockIdx.x / a.chunks;
  const int kvh = unit / a.max_parts, part = unit - kvh * a.max_parts;
  const ChunkSeq sq = chunk_seq(a, b, blockIdx.x == 0 && tid == 0);
  const int rows = min(kCmRows, sq.qlen * a.G - chunk * kCmRows);
  if (rows <= 0) return;
  const int r_first = chunk * kCmRows;
  auto row_query = [&](int r) { return (r_first + r) / a.G; };
  auto row_head = [&](int r) { return kvh * a.G + (r_first + r) % a.G; };
  auto row_out = [&](int r) { return (size_t)(sq.q0 + row_query(r)) * a.H + row_head(r); };

  // every warp works the rows' ranges out for itself: lane = row (rows past
  // the last mirror it, so that they leave the bounds as they are)
  int lo = 0, hi = 0;
  {
    const int r = min(lane & 15, rows - 1);
    chunk_visible(a, sq, row_query(r), lo, hi);
    if (w == 0 && lane < kCmRows) {
      s_lo[lane] = lo;
      s_hi[lane] = hi;
      if (BIAS) s_slope[lane] = __ldg(a.slopes + row_head(r)) * kLog2e;
    }
  }
  const int lo_min = __reduce_min_sync(0xffffffffu, hi > lo ? lo : 0x7fffffff);
  const int hi_max = __reduce_max_sync(0xffffffffu, hi);
  const int lo_max = __reduce_max_sync(0xffffffffu, hi > lo ? lo : 0x7fffffff);  // all rows see [lo_max, hi_min)
  const int hi_min = __reduce_min_sync(0xffffffffu, hi);
  const int base = hi_max > 0 ? lo_min & ~15 : 0;
  const int nparts = max(1, (hi_max - base + a.P - 1) / a.P);
  if (part >= nparts) return;
  const int t0 = base + part * a.P, t1 = min(hi_max, t0 + a.P);
  const int nchunks = t1 > t0 ? (t1 - t0 + kCmTok - 1) / kCmTok : 0;
  const int nch_w = nchunks > w ? (nchunks - w + W - 1) / W : 0;

  if (lane == 0) {
    for (int s = w; s < R; s += W) mbar_init(&bars[s], 1);
    fence_mbar_init();
  }
  __syncwarp();
  const uint64_t policy = l2_evict_first_policy();
  // The chunks this warp asks for: w, w + W, ... of the first fill, then the
  // ones R behind those it is done with.
  const int first = (R - w + W - 1) / W;
  auto asks = [&](int i) { return i < first ? w + W * i : w + R + W * (i - first); };
  int tbl_batch = -1, my_phys = 0;
  auto issue = [&](int i) {             // the i-th of them
    const int c = asks(i);
    if (c >= nchunks) return;
    if ((i >> 5) != tbl_batch) {        // table entries: one load per lane for 32 chunks
      tbl_batch = i >> 5;
      const int cl = asks(tbl_batch * 32 + lane);
      my_phys = 0;
      if (cl < nchunks) {
        my_phys = __ldg(a.tables + (size_t)b * a.max_blocks + (t0 + kCmTok * cl) / a.bs);
        if (my_phys < 0 || (long long)my_phys >= a.num_blocks) {
          raise_flag(a.err, PKV_FLAG_BLOCK_OUT_OF_RANGE);
          my_phys = 0;
        }
      }
    }
    const int phys = __shfl_sync(0xffffffffu, my_phys, i & 31);
    const int row0 = (t0 + kCmTok * c) % a.bs, slot = c % R;
    uint8_t *st = ring + (size_t)slot * Sh::kStage;
    if (lane == 0) {
      mbar_arrive_expect_tx(&bars[slot], Sh::kStage);
      st_release_cta(&s_asked[slot], c);
    }
    __syncwarp();
    if (lane < 2)
      tma_load_5d(st + lane * Sh::kBoxes * kCmBox, lane ? &tmV : &tmK, &bars[slot], 0, row0, 0, kvh, phys, policy);
  };
  for (int i = 0; i < first; ++i) issue(i);

  // query rows (zeros past the last) while the first chunks are in flight
  for (int i = tid; i < kCmRows * (D / 8); i += blockDim.x) {
    const int r = i / (D / 8), c = i - r * (D / 8);
    uint4 v = make_uint4(0, 0, 0, 0);
    if (r < rows) v = __ldg(reinterpret_cast<const uint4 *>(reinterpret_cast<const T *>(a.q) + row_out(r) * D) + c);
    *reinterpret_cast<uint4 *>(sQ + r * Sh::kQStride + c * 8) = v;
  }
  __syncthreads();
  const uint32_t q_addr = smem_u32(sQ) + (((lane & 7) + ((lane >> 3) & 1) * 8) * Sh::kQStride + (lane >> 4) * 8) * 2;
  uint32_t qf[Sh::kQInRegs ? Sh::kSteps : 1][4];
  if constexpr (Sh::kQInRegs) {
#pragma unroll
    for (int kk = 0; kk < Sh::kSteps; ++kk) ldsm_x4(q_addr + kk * 32, qf[kk][0], qf[kk][1], qf[kk][2], qf[kk][3]);
  }

  // this lane's two rows: fragment rows lane / 4 and lane / 4 + 8
  const int r0 = lane >> 2, r1 = r0 + 8;
  const int lo0 = s_lo[r0], hi0 = s_hi[r0], lo1 = s_lo[r1], hi1 = s_hi[r1];
  float slope0 = 0.f, slope1 = 0.f;
  int p0 = 0, p1 = 0;
  if (BIAS) {
    slope0 = s_slope[r0];
    slope1 = s_slope[r1];
    p0 = sq.n - sq.qlen + row_query(min(r0, rows - 1));
    p1 = sq.n - sq.qlen + row_query(min(r1, rows - 1));
  }
  float o[D / 8][4];
#pragma unroll
  for (int nt = 0; nt < D / 8; ++nt) o[nt][0] = o[nt][1] = o[nt][2] = o[nt][3] = 0.f;
  float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
  const int k_row = (lane & 7) + ((lane >> 4) << 3), k_col = (lane >> 3) & 1;
  const int v_row = (lane & 7) + (((lane >> 3) & 1) << 3), v_col = lane >> 4;
  const int sw = lane & 7;

  int i = 0;
  for (; i < nch_w; ++i) {
    const int c = w + W * i, slot = c % R;
    // a stage that passes from warp to warp: its barrier's parity says nothing
    // until the chunk was asked for
    const bool ok = (Sh::kOwn || flag_wait_bounded(&s_asked[slot], c)) && mbar_wait_bounded(&bars[slot], (c / R) & 1);
    if (!__all_sync(0xffffffffu, ok)) {
      if (lane == 0) raise_flag(a.err, PKV_FLAG_TIMEOUT);
      break;
    }
    const int c0 = t0 + kCmTok * c;
    const uint32_t kb = smem_u32(ring + (size_t)slot * Sh::kStage), vb = kb + Sh::kBoxes * kCmBox;
    // S = Q K^T; even and odd steps apart (two shorter chains)
    float sacc[2][2][4] = {};
#pragma unroll
    for (int kk = 0; kk < Sh::kSteps; ++kk) {
      uint32_t b0, b1, b2, b3, af[4];
      ldsm_x4(kb + (kk >> 2) * kCmBox + k_row * 128 + (((((kk & 3) << 1) + k_col) ^ sw) << 4), b0, b1, b2, b3);
      if constexpr (Sh::kQInRegs) {
        af[0] = qf[kk][0]; af[1] = qf[kk][1]; af[2] = qf[kk][2]; af[3] = qf[kk][3];
      } else {
        ldsm_x4(q_addr + kk * 32, af[0], af[1], af[2], af[3]);
      }
      Mma::run(sacc[kk & 1][0], af, b0, b1);
      Mma::run(sacc[kk & 1][1], af, b2, b3);
    }
    float x[2][4];
#pragma unroll
    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float t = sacc[0][nt][e] + sacc[1][nt][e];
        if (CAP == kCapLarge) {
          t = chunk_cap(a, t);
        } else {
          t *= a.scale_y;
          if (CAP) t = chunk_capped(t, a.cap_log2);
        }
        if (BIAS) {
          const int j = c0 + nt * 8 + (lane & 3) * 2 + (e & 1);
          t = fmaf(e < 2 ? -slope0 : -slope1, fabsf((float)((e < 2 ? p0 : p1) - j)), t);
        }
        x[nt][e] = t;
      }
    const bool whole = c0 >= lo_max && c0 + kCmTok <= min(hi_min, t1);
    uint32_t vm0 = 0xffffffffu, vm1 = 0xffffffffu;
    if (!whole) {
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = c0 + nt * 8 + (lane & 3) * 2 + (e & 1);
          const bool vis = j < t1 && (e < 2 ? j >= lo0 && j < hi0 : j >= lo1 && j < hi1);
          x[nt][e] = vis ? x[nt][e] : -INFINITY;
        }
      // values that no row sees become 0 (they may hold anything)
      const int tk = c0 + (lane & 3) * 2;
      auto live = [&](int j) { return j >= lo_min && j < t1; };
      vm0 = (live(tk) ? 0x0000ffffu : 0u) | (live(tk + 1) ? 0xffff0000u : 0u);
      vm1 = (live(tk + 8) ? 0x0000ffffu : 0u) | (live(tk + 9) ? 0xffff0000u : 0u);
    }
    float mx0 = fmaxf(fmaxf(x[0][0], x[0][1]), fmaxf(x[1][0], x[1][1]));
    float mx1 = fmaxf(fmaxf(x[0][2], x[0][3]), fmaxf(x[1][2], x[1][3]));
    mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 1));
    mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 1));
    mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 2));
    mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 2));
    const float mn0 = fmaxf(m0, mx0), mn1 = fmaxf(m1, mx1);
    if (__any_sync(0xffffffffu, mn0 > m0 || mn1 > m1)) {
      const float f0 = fast_exp2(m0 - chunk_ref(mn0)), f1 = fast_exp2(m1 - chunk_ref(mn1));
      l0 *= f0;
      l1 *= f1;
#pragma unroll
      for (int nt = 0; nt < D / 8; ++nt) {
        o[nt][0] *= f0; o[nt][1] *= f0;
        o[nt][2] *= f1; o[nt][3] *= f1;
      }
      m0 = mn0;
      m1 = mn1;
    }
    const float e0 = chunk_ref(m0), e1 = chunk_ref(m1);
    // weights in 16 bits, and the sum of the rounded ones: it hides behind the loads here
    uint32_t pa[4];
    pa[0] = Mma::pack(fast_exp2(x[0][0] - e0), fast_exp2(x[0][1] - e0), l0);
    pa[1] = Mma::pack(fast_exp2(x[0][2] - e1), fast_exp2(x[0][3] - e1), l1);
    pa[2] = Mma::pack(fast_exp2(x[1][0] - e0), fast_exp2(x[1][1] - e0), l0);
    pa[3] = Mma::pack(fast_exp2(x[1][2] - e1), fast_exp2(x[1][3] - e1), l1);
#pragma unroll
    for (int dp = 0; dp < Sh::kSteps; ++dp) {
      uint32_t b0, b1, b2, b3;
      ldsm_x4_trans(vb + (dp >> 2) * kCmBox + v_row * 128 + (((((dp & 3) << 1) + v_col) ^ sw) << 4), b0, b1, b2, b3);
      b0 &= vm0; b1 &= vm1; b2 &= vm0; b3 &= vm1;
      Mma::run(o[2 * dp], pa, b0, b1);
      Mma::run(o[2 * dp + 1], pa, b2, b3);
    }
    __syncwarp();
    issue(first + i);
  }
  l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
  l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
  l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
  l1 += __shfl_xor_sync(0xffffffffu, l1, 2);

  // merge the warps' states (the ring is free then)
  if ((lane & 3) == 0) {
    s_wm[w * kCmRows + r0] = m0;
    s_wm[w * kCmRows + r1] = m1;
    s_wl[w * kCmRows + r0] = l0;
    s_wl[w * kCmRows + r1] = l1;
  }
  if (__syncthreads_or(i < nch_w)) {  // a warp gave up: let the copies already asked for land (bounded)
    for (int s = w; s < min(R, nchunks); s += W) mbar_wait_bounded(&bars[s], (s_asked[s] / R) & 1);
    __syncthreads();
  }
  float M0 = -INFINITY, M1 = -INFINITY;
#pragma unroll
  for (int ww = 0; ww < W; ++ww) {
    M0 = fmaxf(M0, s_wm[ww * kCmRows + r0]);
    M1 = fmaxf(M1, s_wm[ww * kCmRows + r1]);
  }
  const float f0 = fast_exp2(m0 - chunk_ref(M0)), f1 = fast_exp2(m1 - chunk_ref(M1));
  float *sO = reinterpret_cast<float *>(ring);  // [W][16][kOStride]
  if (r0 < rows) {
#pragma unroll
    for (int nt = 0; nt < D / 8; ++nt)
      *reinterpret_cast<float2 *>(sO + (w * kCmRows + r0) * Sh::kOStride + nt * 8 + (lane & 3) * 2) =
          make_float2(o[nt][0] * f0, o[nt][1] * f0);
  }
  if (r1 < rows) {
#pragma unroll
    for (int nt = 0; nt < D / 8; ++nt)
      *reinterpret_cast<float2 *>(sO + (w * kCmRows + r1) * Sh::kOStride + nt * 8 + (lane & 3) * 2) =
          make_float2(o[nt][2] * f1, o[nt][3] * f1);
  }
  if (tid < kCmRows) {
    float M = -INFINITY, L = 0.f;
    for (int ww = 0; ww < W; ++ww) M = fmaxf(M, s_wm[ww * kCmRows + tid]);
    for (int ww = 0; ww < W; ++ww)
      L += s_wl[ww * kCmRows + tid] * fast_exp2(s_wm[ww * kCmRows + tid] - chunk_ref(M));
    s_m[tid] = M;
    s_l[tid] = L;
  }
  if (tid == 0) *s_scratch = 0;
  __syncthreads();
  for (int e = tid; e < rows * (D / 4); e += blockDim.x) {
    const int r = e / (D / 4), d = (e - r * (D / 4)) * 4;
    float4 acc = *reinterpret_cast<const float4 *>(sO + r * Sh::kOStride + d);
#pragma unroll
    for (int ww = 1; ww < W; ++ww) {
      const float4 v = *reinterpret_cast<const float4 *>(sO + (ww * kCmRows + r) * Sh::kOStride + d);
      acc.x += v.x; acc.y += v.y; acc.z += v.z; acc.w += v.w;
    }
    *reinterpret_cast<float4 *>(sO + r * Sh::kOStride + d) = acc;
    // not finite, and some key of the part is hidden from the row: its rows
    // are looked at again below
    const float z = (acc.x + acc.y + acc.z + acc.w) * 0.f;
    if (z != 0.f && (s_lo[r] > t0 || s_hi[r] < t1)) atomicOr(s_scratch, 1 << r);
  }
  __syncthreads();
  const int again = *s_scratch;
  if (again) {
    for (int r = w; r < rows; r += W) {
      if (!((again >> r) & 1)) continue;
      float m, l, acc[D / 32];
      chunk_row_exact<T, D / 32>(a, b, kvh, row_out(r), BIAS ? s_slope[r] : 0.f, sq.n - sq.qlen + row_query(r),
                                 max(t0, s_lo[r]), min(t1, s_hi[r]), m, l, acc);
#pragma unroll
      for (int e = 0; e < D / 32; ++e) sO[r * Sh::kOStride + lane + 32 * e] = acc[e];
      if (lane == 0) {
        s_m[r] = m;
        s_l[r] = l;
      }
    }
    __syncthreads();
  }
  chunk_finish<T>(a, rows, part, nparts, s_m, s_l, sO, Sh::kOStride, Sh::kRing / 4, s_scratch,
                  a.ws_cnt + kChunkCntFirst + ((size_t)b * a.KVH + kvh) * a.chunks + chunk, row_out,
                  [&](int r) { return s_hi[r] > s_lo[r]; });
}

template <int D, typename T, int CAP, bool BIAS>
static pkv_status launch_cm(const ChunkArgs &a, const CUtensorMap &mk, const CUtensorMap &mv, cudaStream_t stream) {
  auto kern = pkv_chunk_mma_kernel<D, T, CAP, BIAS>;
  static int configured[64] = {0};
  if (!allow_smem(kern, CmShape<D>::kSmem, configured)) return PKV_ERR_CUDA;
  const dim3 grid((unsigned)((long long)a.max_parts * a.KVH * a.chunks), a.B);
  kern<<<grid, 32 * CmShape<D>::kWarps, CmShape<D>::kSmem, stream>>>(mk, mv, a);
  return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

template <int D, typename T>
static pkv_status launch_cm_form(const ChunkArgs &a, const CUtensorMap &mk, const CUtensorMap &mv, cudaStream_t stream) {
  return chunk_forms(a, [&](auto cap, auto bias) { return launch_cm<D, T, cap.value, bias.value>(a, mk, mv, stream); });
}

template <typename T>
static pkv_status launch_cm_dt(const ChunkArgs &a, const CUtensorMap &mk, const CUtensorMap &mv, cudaStream_t stream) {
  switch (a.D) {
    case 64: return launch_cm_form<64, T>(a, mk, mv, stream);
    case 128: return launch_cm_form<128, T>(a, mk, mv, stream);
    case 192: return launch_cm_form<192, T>(a, mk, mv, stream);
    case 256: return launch_cm_form<256, T>(a, mk, mv, stream);
  }
  return PKV_ERR_UNSUPPORTED;
}

pkv_status launch_chunk_mma(const ChunkArgs &a, pkv_dtype dt, cudaStream_t stream) {
  CUtensorMap mk, mv;
  if (!encode_chunk_map(&mk, a.k_cache, dt, a.num_blocks, a.bs, a.KVH, a.D) ||
      !encode_chunk_map(&mv, a.v_cache, dt, a.num_blocks, a.bs, a.KVH, a.D))
    return PKV_ERR_CUDA;
  return dt == PKV_BF16 ? launch_cm_dt<__nv_bfloat16>(a, mk, mv, stream) : launch_cm_dt<__half>(a, mk, mv, stream);
}

}  // namespace pkv
