// pkv_chunk_simt.cuh -- chunk attention on the CUDA cores: any dtype, any
// head_dim up to 512, any block size and alignment (see pkv_chunk.cuh for the
// rows, masks and scores).  It serves fp32, whose accuracy rules out 16-bit
// products, and the shapes that the tensor-core kernels do not take.
//
// CTA = (part of the context, RT packed rows of a KV head, sequence), 128
// threads; 32 keys at a time pass through shared memory.
//   RT = 4 and 16, few rows per key, bound by instructions and loads:
//     S    RT = 16: thread = key x 4 rows, a key vector against four query
//          vectors; RT = 4: thread = key x 4 rows x a quarter of D (its warp's),
//          the quarters added up by the softmax
//     O    thread = columns tid, tid + 128, ... x RT rows
//   RT = 64, long chunks, bound by the multiply-adds: 8 row groups x 16 columns
//     S    thread = 8 rows x 2 keys: 10 shared loads feed 64 multiply-adds per
//          4 columns of D, the query loads broadcast over 16 lanes
//     O    thread = 8 rows x columns 4 tx + 64 j
// The next tile's keys load while this one's softmax and O run, its values
// while the next S runs (cp.async, one buffer each: with two, fewer CTAs fit an
// SM and decode at head_dim 128 took 880 us for 489); block-table entries are
// read a tile ahead of that.
#pragma once

#include "pkv_chunk.cuh"

namespace pkv {

constexpr int kCsTok = 32;
constexpr int kCsThreads = 128;

// Elements of a padded row: 16-byte steps, and 16 bytes that turn the banks.
template <typename T>
__host__ __device__ constexpr int cs_stride(int D) {
  return (D * (int)sizeof(T) + 15) / 16 * 16 / (int)sizeof(T) + 16 / (int)sizeof(T);
}

template <typename T, int RT>
static size_t cs_smem(int D) {
  return (size_t)RT * cs_stride<float>(D) * 4 + 2 * (size_t)kCsTok * cs_stride<T>(D) * sizeof(T) +
         4 * (size_t)((RT == 4 ? 16 : RT) * (kCsTok + 4) + kCsTok * (RT + 4) + 4 * RT) + 4 * (2 * RT + 4) + 2 * kCsTok * sizeof(long long);
}

__device__ __forceinline__ void cs_copy16(uint32_t dst, const void *src, bool live) {  // zeros when not live
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cs_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cs_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Four consecutive elements (16-byte, or 8-byte aligned for 16-bit types) as fp32.
__device__ __forceinline__ float4 cs_ld4(const float *p) { return *reinterpret_cast<const float4 *>(p); }
template <typename T>
__device__ __forceinline__ float4 cs_ld4(const T *p) {
  const uint2 v = *reinterpret_cast<const uint2 *>(p);
  const T *e = reinterpret_cast<const T *>(&v);
  return make_float4(to_f32<T>(e[0]), to_f32<T>(e[1]), to_f32<T>(e[2]), to_f32<T>(e[3]));
}

// EP: column steps of a thread in O (RT = 64: of 64, else of 128).  AL:
// cache rows are whole, aligned 16-byte vectors, and out is aligned.
template <typename T, int RT, int EP, bool AL>
__global__ void __launch_bounds__(kCsThreads) pkv_chunk_simt_kernel(const ChunkArgs a) {
  extern __shared__ __align__(16) uint8_t s_raw[];
  const int D = a.D, QS = cs_stride<float>(D), KS = cs_stride<T>(D);
  constexpr int kSS = kCsTok + 4, kPS = RT + 4;
  float *sQ = reinterpret_cast<float *>(s_raw);       // [RT][QS]
  T *sK = reinterpret_cast<T *>(sQ + RT * QS);        // [32][KS]
  T *sV = sK + kCsTok * KS;                           // [32][KS]
  float *sS = reinterpret_cast<float *>(sV + kCsTok * KS);  // [RT][kSS] scores
  float *sP = sS + (RT == 4 ? 16 : RT) * kSS;         // [32][kPS] weights, transposed  (RT = 4: sS is [4 quarters][4])
  float *s_alpha = sP + kCsTok * kPS;                 // [RT]
  float *s_m = s_alpha + RT, *s_l = s_m + RT, *s_slope = s_l + RT;  // [RT]
  int *s_lo = reinterpret_cast<int *>(s_slope + RT);  // [RT]
  int *s_hi = s_lo + RT;                              // [RT]
  int *s_flag = s_hi + RT;                            // [0] last part / rows to do again, [1] first key, [2] one past the last
  long long *s_row = reinterpret_cast<long long *>(s_flag + 4);  // [2][32] element offset of a key's row, or -1

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, tx = tid & 15, ty = tid >> 4;
  const int b = blockIdx.y, slotp = blockIdx.x % a.max_parts, unit = blockIdx.x / a.max_parts;
  const int kvh = unit / a.chunks, chunk = a.chunks - 1 - (unit - kvh * a.chunks);  // the longest chunks first
  const ChunkSeq sq = chunk_seq(a, b, blockIdx.x == 0 && tid == 0);
  const int rows = min(RT, sq.qlen * a.G - chunk * RT);
  if (rows <= 0) return;
  auto row_query = [&](int r) { return (chunk * RT + r) / a.G; };
  auto row_head = [&](int r) { return kvh * a.G + (chunk * RT + r) % a.G; };
  auto out_row = [&](int r) { return (size_t)(sq.q0 + row_query(r)) * a.H + row_head(r); };
  if (tid == 0) {
    s_flag[1] = 0x7fffffff;
    s_flag[2] = 0;
  }
  __syncthreads();
  if (tid < RT) {
    int lo = 0, hi = 0;
    float slope = 0.f;
    if (tid < rows) {
      chunk_visible(a, sq, row_query(tid), lo, hi);
      if (a.slopes) slope = __ldg(a.slopes + row_head(tid)) * kLog2e;
    }
    s_lo[tid] = lo;
    s_hi[tid] = hi;
    s_slope[tid] = slope;
    if (hi > lo) {
      atomicMin(s_flag + 1, lo);
      atomicMax(s_flag + 2, hi);
    }
  }
  __syncthreads();
  const int lo_min = s_flag[1], hi_max = s_flag[2];
  // the unit's parts begin at its first visible key, on a multiple of 16
  const int base = hi_max > 0 ? lo_min & ~15 : 0;
  const int nparts = max(1, (hi_max - base + a.P - 1) / a.P);
  if (slotp >= nparts) return;
  // (no row sees a key: the empty part [0, 0), from which t0 + tid is no overflow)
  const int t0 = hi_max > 0 ? max(lo_min, base + slotp * a.P) : 0, t1 = min(hi_max, base + (slotp + 1) * a.P);

  // element offset of key t's row, -1 past the part's end
  auto table_entry = [&](int t) { return t < t1 ? __ldg(a.tables + (size_t)b * a.max_blocks + t / a.bs) : 0; };
  auto key_row = [&](int t, int phys) -> long long {
    if (t >= t1) return -1;
    const int lb = t / a.bs;
    if (phys < 0 || (long long)phys >= a.num_blocks) {
      raise_flag(a.err, PKV_FLAG_BLOCK_OUT_OF_RANGE);
      phys = 0;
    }
    return (((long long)phys * a.bs + (t - lb * a.bs)) * a.KVH + kvh) * D;
  };
  const int row_pieces = max(1, D * (int)sizeof(T) / 16), first_row = tid / row_pieces, first_piece = tid % row_pieces;
  auto fetch = [&](T *dst, const void *cache, int tile) {  // 32 rows into shared memory
    const T *src = reinterpret_cast<const T *>(cache);
    const long long *rowp = s_row + (tile & 1) * kCsTok;
    if constexpr (AL) {
      const int pieces = row_pieces;
      auto copy = [&](int t, int c) {
        const long long row = rowp[t];
        cs_copy16(smem_u32(dst + t * KS) + 16 * c, reinterpret_cast<const uint4 *>(src + (row < 0 ? 0 : row)) + c, row >= 0);
      };
      if (kCsThreads % pieces == 0) {           // a thread keeps to one piece of the row
#pragma unroll 4
        for (int t = first_row; t < kCsTok; t += kCsThreads / pieces) copy(t, first_piece);
      } else {
        for (int i = tid; i < kCsTok * pieces; i += kCsThreads) copy(i / pieces, i % pieces);
      }
    } else {
      for (int t = warp; t < kCsTok; t += kCsThreads / 32) {
        const long long row = rowp[t];
        for (int d = lane; d < KS; d += 32) dst[t * KS + d] = (row >= 0 && d < D) ? src[row + d] : from_f32<T>(0.f);
      }
    }
    cs_commit();
  };
  const int ntiles = t1 > t0 ? (t1 - t0 + kCsTok - 1) / kCsTok : 0;
  if (tid < 2 * kCsTok) s_row[tid] = key_row(t0 + tid, table_entry(t0 + tid));   // the first two tiles
  __syncthreads();
  if (ntiles > 0) {
    fetch(sK, a.k_cache, 0);
    fetch(sV, a.v_cache, 0);
  }
  for (int r = warp; r < RT; r += kCsThreads / 32)
    for (int d = lane; d < QS; d += 32)
      sQ[r * QS + d] = (r < rows && d < D) ? to_f32<T>(reinterpret_cast<const T *>(a.q)[out_row(r) * D + d]) : 0.f;

  constexpr int kOR = RT == 64 ? 8 : RT, kOC = RT == 64 ? 4 * EP : EP;  // rows and columns of O a thread holds
  float o[kOR][kOC];
#pragma unroll
  for (int r = 0; r < kOR; ++r)
#pragma unroll
    for (int e = 0; e < kOC; ++e) o[r][e] = 0.f;
  constexpr int kTpr = kCsThreads / RT, kXs = kCsTok / kTpr;            // softmax: threads a row, keys a thread
  const int srow = tid / kTpr, sub = tid % kTpr;
  float m = -INFINITY, l = 0.f;

  for (int tile = 0; tile < ntiles; ++tile) {
    const int key0 = t0 + tile * kCsTok;
    cs_wait<1>();
    __syncthreads();                            // this tile's keys are there
    if constexpr (RT == 4) {                    // key `lane`, four rows, the warp's quarter of the columns
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
      const T *kr = sK + lane * KS;
      const float4 *qr = reinterpret_cast<const float4 *>(sQ);
      const int quads = (D + 3) / 4, from = quads * warp / 4, to = quads * (warp + 1) / 4;
#pragma unroll 4
      for (int d = from; d < to; ++d) {
        const float4 kx = cs_ld4(kr + 4 * d);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float4 qx = qr[r * (QS / 4) + d];
          acc[r] = fmaf(qx.x, kx.x, fmaf(qx.y, kx.y, fmaf(qx.z, kx.z, fmaf(qx.w, kx.w, acc[r]))));
        }
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) sS[(4 * warp + r) * kSS + lane] = acc[r];
    } else if constexpr (RT == 16) {            // key `lane`, rows 4 * warp ..
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
      const T *kr = sK + lane * KS;
      const float4 *qr = reinterpret_cast<const float4 *>(sQ + 4 * warp * QS);
#pragma unroll 4
      for (int d = 0; d < (D + 3) / 4; ++d) {
        const float4 kx = cs_ld4(kr + 4 * d);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float4 qx = qr[r * (QS / 4) + d];
          acc[r] = fmaf(qx.x, kx.x, fmaf(qx.y, kx.y, fmaf(qx.z, kx.z, fmaf(qx.w, kx.w, acc[r]))));
        }
      }
      const int j = key0 + lane;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int rr = 4 * warp + r;
        const bool vis = j < t1 && j >= s_lo[rr] && j < s_hi[rr];
        sS[rr * kSS + lane] = vis ? chunk_score(a, acc[r], s_slope[rr], sq.n - sq.qlen + row_query(rr), j) : -INFINITY;
      }
    } else {
      float acc[8][2];
#pragma unroll
      for (int r = 0; r < 8; ++r) acc[r][0] = acc[r][1] = 0.f;
      const T *k0 = sK + tx * KS, *k1 = sK + (tx + 16) * KS;
      const float4 *qr = reinterpret_cast<const float4 *>(sQ + 8 * ty * QS);
#pragma unroll 2
      for (int d = 0; d < (D + 3) / 4; ++d) {
        const float4 ka = cs_ld4(k0 + 4 * d), kb = cs_ld4(k1 + 4 * d);
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          const float4 qx = qr[r * (QS / 4) + d];
          acc[r][0] = fmaf(qx.x, ka.x, fmaf(qx.y, ka.y, fmaf(qx.z, ka.z, fmaf(qx.w, ka.w, acc[r][0]))));
          acc[r][1] = fmaf(qx.x, kb.x, fmaf(qx.y, kb.y, fmaf(qx.z, kb.z, fmaf(qx.w, kb.w, acc[r][1]))));
        }
      }
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        const int rr = 8 * ty + r;
        const int lo = s_lo[rr], hi = min(s_hi[rr], t1), p = sq.n - sq.qlen + row_query(rr);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int j = key0 + tx + 16 * k;
          sS[rr * kSS + tx + 16 * k] = j >= lo && j < hi ? chunk_score(a, acc[r][k], s_slope[rr], p, j) : -INFINITY;
        }
      }
    }
    // table entries of the tile after the next, looked at only at the end
    const int next_key = key0 + 2 * kCsTok + tid, next_phys = tid < kCsTok ? table_entry(next_key) : 0;
    __syncthreads();                            // scores there, keys free
    if (tile + 1 < ntiles) fetch(sK, a.k_cache, tile + 1);
    else cs_commit();
    {
      float x[kXs], mx = -INFINITY;
#pragma unroll
      for (int i = 0; i < kXs; ++i) {
        if constexpr (RT == 4) {                // the quarters' sum, and the score
          const float dot = (sS[srow * kSS + sub] + sS[(4 + srow) * kSS + sub]) + (sS[(8 + srow) * kSS + sub] + sS[(12 + srow) * kSS + sub]);
          const int j = key0 + sub;
          const bool vis = j < t1 && j >= s_lo[srow] && j < s_hi[srow];
          x[i] = vis ? chunk_score(a, dot, s_slope[srow], sq.n - sq.qlen + row_query(srow), j) : -INFINITY;
        } else {
          x[i] = sS[srow * kSS + sub + kTpr * i];
        }
        mx = fmaxf(mx, x[i]);
      }
#pragma unroll
      for (int w = 1; w < kTpr; w <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
      const float mn = fmaxf(m, mx), ref = chunk_ref(mn);
      const float alpha = fast_exp2(m - ref);
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < kXs; ++i) {
        const float p = fast_exp2(x[i] - ref);
        sum += p;
        sP[(sub + kTpr * i) * kPS + srow] = p;
      }
#pragma unroll
      for (int w = 1; w < kTpr; w <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
      l = fmaf(l, alpha, sum);
      m = mn;
      if (sub == 0) s_alpha[srow] = alpha;
    }
    cs_wait<1>();
    __syncthreads();                            // weights and this tile's values are there
    const int r0 = RT == 64 ? 8 * ty : 0;
#pragma unroll
    for (int r = 0; r < kOR; ++r) {
      const float al = s_alpha[r0 + r];
#pragma unroll
      for (int e = 0; e < kOC; ++e) o[r][e] *= al;
    }
#pragma unroll 2
    for (int t = 0; t < kCsTok; ++t) {
      float p[kOR];
#pragma unroll
      for (int r4 = 0; r4 < kOR / 4; ++r4) {
        const float4 v = *reinterpret_cast<const float4 *>(sP + t * kPS + r0 + 4 * r4);
        p[4 * r4] = v.x; p[4 * r4 + 1] = v.y; p[4 * r4 + 2] = v.z; p[4 * r4 + 3] = v.w;
      }
      if constexpr (RT != 64) {
#pragma unroll
        for (int e = 0; e < EP; ++e) {
          const int d = tid + kCsThreads * e;
          const float v = d < D ? to_f32<T>(sV[t * KS + d]) : 0.f;
#pragma unroll
          for (int r = 0; r < RT; ++r) o[r][e] = fmaf(p[r], v, o[r][e]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < EP; ++j) {
          const int d = 4 * tx + 64 * j;
          const float4 v = d < D ? cs_ld4(sV + t * KS + d) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int r = 0; r < 8; ++r) {
            o[r][4 * j] = fmaf(p[r], v.x, o[r][4 * j]);
            o[r][4 * j + 1] = fmaf(p[r], v.y, o[r][4 * j + 1]);
            o[r][4 * j + 2] = fmaf(p[r], v.z, o[r][4 * j + 2]);
            o[r][4 * j + 3] = fmaf(p[r], v.w, o[r][4 * j + 3]);
          }
        }
      }
    }
    __syncthreads();                            // values and weights free
    if (tile + 1 < ntiles) fetch(sV, a.v_cache, tile + 1);
    else cs_commit();
    // (read again only after the next barriers: K of tile + 2 is fetched behind two of them)
    if (tid < kCsTok) s_row[(tile & 1) * kCsTok + tid] = key_row(next_key, next_phys);
  }
  cs_wait<0>();
  if (sub == 0) {
    s_m[srow] = m;
    s_l[srow] = l;
  }
  unsigned long long *s_again = reinterpret_cast<unsigned long long *>(s_row);
  __syncthreads();
  if (tid == 0) *s_again = 0;
  __syncthreads();

  // the rows; those that are not finite although a key of the part is hidden
  // from them (0 * inf) are done again below, from what they see alone
  T *out = reinterpret_cast<T *>(a.out);
#pragma unroll
  for (int r = 0; r < kOR; ++r) {
    const int rr = RT == 64 ? 8 * ty + r : r;
    if (rr >= rows) continue;
    const size_t row = out_row(rr), at = row * a.max_parts + slotp;
    const bool seen = s_hi[rr] > s_lo[rr];
    float odd = 0.f;
#pragma unroll
    for (int e = 0; e < kOC; ++e) {
      const int d = RT == 64 ? 4 * tx + 64 * (e / 4) + e % 4 : tid + kCsThreads * e;
      if (d >= D) continue;
      odd = fmaf(o[r][e], 0.f, odd);
      if (nparts == 1) out[row * D + d] = from_f32<T>(seen ? o[r][e] / s_l[rr] : 0.f);
      else a.ws_o[at * D + d] = o[r][e];
    }
    if (odd != 0.f && (s_lo[rr] > t0 || s_hi[rr] < t1)) atomicOr(s_again, 1ull << rr);
  }
  if (nparts > 1 && tid < rows) {
    const size_t at = out_row(tid) * a.max_parts + slotp;
    a.ws_m[at] = s_m[tid];
    a.ws_l[at] = s_l[tid];
  }
  __syncthreads();
  const unsigned long long again = *s_again;
  for (int r = warp; again && r < rows; r += kCsThreads / 32) {
    if (!((again >> r) & 1)) continue;
    constexpr int kE = RT == 64 ? 2 * EP : 4 * EP;  // 32-column steps of a row
    float em, el, eo[kE];
    chunk_row_exact<T, kE>(a, b, kvh, out_row(r), s_slope[r], sq.n - sq.qlen + row_query(r), max(t0, s_lo[r]),
                           min(t1, s_hi[r]), em, el, eo);
    const size_t row = out_row(r), at = row * a.max_parts + slotp;
#pragma unroll
    for (int e = 0; e < kE; ++e) {
      const int d = lane + 32 * e;
      if (d >= D) continue;
      if (nparts == 1) out[row * D + d] = from_f32<T>(s_hi[r] > s_lo[r] ? eo[e] / el : 0.f);
      else a.ws_o[at * D + d] = eo[e];
    }
    if (nparts > 1 && lane == 0) {
      a.ws_m[at] = em;
      a.ws_l[at] = el;
    }
  }
  if (nparts == 1) return;
  int *counter = a.ws_cnt + kChunkCntFirst + ((size_t)b * a.KVH + kvh) * a.chunks + chunk;
  if (!chunk_last_part(counter, nparts, s_flag)) return;
  // (everything before the rows' bounds is free now)
  const int room = (int)(reinterpret_cast<float *>(s_alpha) - reinterpret_cast<float *>(s_raw));
  auto seen = [&](int r) { return s_hi[r] > s_lo[r]; };
  chunk_merge<T, AL ? 4 : 1>(a, rows, nparts, reinterpret_cast<float *>(s_raw), room, out_row, seen);
  if (tid == 0) *counter = 0;
}

template <typename T, int RT, int EP>
static pkv_status launch_cs(const ChunkArgs &a, cudaStream_t stream) {
  const dim3 grid((unsigned)((long long)a.max_parts * a.KVH * a.chunks), a.B);
  const size_t smem = cs_smem<T, RT>(a.D);
  const bool aligned = a.D * sizeof(T) % 16 == 0 && reinterpret_cast<uintptr_t>(a.k_cache) % 16 == 0 &&
                       reinterpret_cast<uintptr_t>(a.v_cache) % 16 == 0 &&
                       reinterpret_cast<uintptr_t>(a.out) % 16 == 0;
  auto go = [&](auto kern, int *configured) {
    if (!allow_smem(kern, smem, configured)) return PKV_ERR_CUDA;
    kern<<<grid, kCsThreads, smem, stream>>>(a);
    return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
  };
  static int configured[2][64] = {{0}};
  return aligned ? go(pkv_chunk_simt_kernel<T, RT, EP, true>, configured[0])
                 : go(pkv_chunk_simt_kernel<T, RT, EP, false>, configured[1]);
}

template <typename T>
static pkv_status launch_cs_dt(const ChunkArgs &a, int rows, cudaStream_t stream) {
  if (rows == 64) {
    if (a.D <= 64) return launch_cs<T, 64, 1>(a, stream);
    return a.D <= 128 ? launch_cs<T, 64, 2>(a, stream) : launch_cs<T, 64, 4>(a, stream);
  }
  if (rows == 4) {
    if (a.D <= 128) return launch_cs<T, 4, 1>(a, stream);
    return a.D <= 256 ? launch_cs<T, 4, 2>(a, stream) : launch_cs<T, 4, 4>(a, stream);
  }
  if (a.D <= 128) return launch_cs<T, 16, 1>(a, stream);
  return a.D <= 256 ? launch_cs<T, 16, 2>(a, stream) : launch_cs<T, 16, 4>(a, stream);
}

}  // namespace pkv
