// pkv_chunk_simt.cu -- chunk attention on the CUDA cores: any dtype, any
// head_dim up to 512, any block size and alignment (see pkv_chunk.cuh for the
// rows, masks and scores).  It serves fp32, whose accuracy rules out 16-bit
// products, and the shapes that the tensor-core kernels do not take.
//
// CTA = (part of the context, 16 packed rows of a KV head, sequence), 128
// threads.  Keys and values pass through shared memory as fp32, 32 tokens at
// a time:
//   S[16 x 32]   thread = token x 4 rows: one key vector against four query
//                vectors, so a 16-byte shared load feeds 16 multiply-adds
//   softmax      8 threads a row: running max m and sum l in registers
//   O[16 x D]    thread = columns tid, tid + 128, ...; 16 rows each
// The multiply-adds bound long chunks, the loads single tokens.
#include "pkv_chunk.cuh"

namespace pkv {

constexpr int kCsRows = 16;
constexpr int kCsTok = 32;
constexpr int kCsThreads = 128;

__host__ __device__ inline int cs_row_floats(int D) { return (D + 3) / 4 * 4 + 4; }  // padded rows: no bank conflicts

size_t chunk_simt_smem(int D) {
  return sizeof(float) * ((size_t)(kCsRows + 2 * kCsTok) * cs_row_floats(D) + 2 * kCsRows * (kCsTok + 4) +
                          4 * kCsRows) + sizeof(int) * (2 * kCsRows + 4);
}

template <typename T, int EPT>
__global__ void __launch_bounds__(kCsThreads) pkv_chunk_simt_kernel(const ChunkArgs a) {
  extern __shared__ __align__(16) float s_f[];
  const int D = a.D, RS = cs_row_floats(D);
  float *sQ = s_f;                              // [16][RS]
  float *sK = sQ + kCsRows * RS;                // [32][RS]
  float *sV = sK + kCsTok * RS;                 // [32][RS]
  float *sS = sV + kCsTok * RS;                 // [16][36] scores
  float *sP = sS + kCsRows * (kCsTok + 4);      // [32][16] weights, transposed (fits [16][36])
  float *s_alpha = sP + kCsRows * (kCsTok + 4); // [16]
  float *s_m = s_alpha + kCsRows;               // [16]
  float *s_l = s_m + kCsRows;                   // [16]
  float *s_slope = s_l + kCsRows;               // [16]
  int *s_lo = reinterpret_cast<int *>(s_slope + kCsRows);  // [16]
  int *s_hi = s_lo + kCsRows;                   // [16]
  int *s_flag = s_hi + kCsRows;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.y, slotp = blockIdx.x % a.max_parts, unit = blockIdx.x / a.max_parts;
  const int kvh = unit / a.chunks, chunk = unit - kvh * a.chunks;
  const ChunkSeq sq = chunk_seq(a, b, blockIdx.x == 0 && tid == 0);
  const int rows = min(kCsRows, sq.qlen * a.G - chunk * kCsRows);
  if (rows <= 0) return;
  // row r of the chunk: packed row chunk * 16 + r = query * G + head of the group
  auto row_query = [&](int r) { return (chunk * kCsRows + r) / a.G; };
  auto row_head = [&](int r) { return kvh * a.G + (chunk * kCsRows + r) % a.G; };
  if (tid < kCsRows) {
    int lo = 0, hi = 0;
    float slope = 0.f;
    if (tid < rows) {
      chunk_visible(a, sq, row_query(tid), lo, hi);
      if (a.slopes) slope = __ldg(a.slopes + row_head(tid)) * kLog2e;
    }
    s_lo[tid] = lo;
    s_hi[tid] = hi;
    s_slope[tid] = slope;
  }
  __syncthreads();
  int lo_min = 0x7fffffff, hi_max = 0;
  for (int r = 0; r < rows; ++r)
    if (s_hi[r] > s_lo[r]) {
      lo_min = min(lo_min, s_lo[r]);
      hi_max = max(hi_max, s_hi[r]);
    }
  // the unit's parts begin at its first visible key's 16-key chunk
  const int base = hi_max > 0 ? lo_min & ~15 : 0;
  const int nparts = max(1, (hi_max - base + a.P - 1) / a.P);
  if (slotp >= nparts) return;
  const int t0 = max(lo_min, base + slotp * a.P), t1 = min(hi_max, base + (slotp + 1) * a.P);

  for (int i = tid; i < kCsRows * RS; i += kCsThreads) {
    const int r = i / RS, d = i - r * RS;
    sQ[i] = (r < rows && d < D)
                ? to_f32<T>(reinterpret_cast<const T *>(a.q)[((size_t)(sq.q0 + row_query(r)) * a.H + row_head(r)) * D + d])
                : 0.f;
  }

  float o[kCsRows][EPT];
#pragma unroll
  for (int r = 0; r < kCsRows; ++r)
#pragma unroll
    for (int e = 0; e < EPT; ++e) o[r][e] = 0.f;
  const int srow = tid >> 3, sub = tid & 7;     // softmax: row and its eighth
  float m = -INFINITY, l = 0.f;

  const T *kc = reinterpret_cast<const T *>(a.k_cache);
  const T *vc = reinterpret_cast<const T *>(a.v_cache);
  for (int tile = t0; tile < t1; tile += kCsTok) {
    const int cnt = min(kCsTok, t1 - tile);
    __syncthreads();                            // the previous tile is no longer read
    bool odd = false;                           // a value that is not finite
    for (int t = warp; t < kCsTok; t += kCsThreads / 32) {
      const T *kp = kc, *vp = vc;
      if (t < cnt) {
        const int lb = (tile + t) / a.bs;
        int phys = __ldg(a.tables + (size_t)b * a.max_blocks + lb);
        if (phys < 0 || (long long)phys >= a.num_blocks) {
          if (lane == 0) raise_flag(a.err, PKV_FLAG_BLOCK_OUT_OF_RANGE);
          phys = 0;
        }
        const size_t row = (((size_t)phys * a.bs + (tile + t - lb * a.bs)) * a.KVH + kvh) * D;
        kp += row;
        vp += row;
      }
      for (int d = lane; d < RS; d += 32) {
        const bool live = t < cnt && d < D;
        const float kx = live ? to_f32<T>(kp[d]) : 0.f, vx = live ? to_f32<T>(vp[d]) : 0.f;
        sK[t * RS + d] = kx;
        sV[t * RS + d] = vx;
        odd |= !(fabsf(vx) < INFINITY);
      }
    }
    const bool any_odd = __syncthreads_or(odd);
    {                                           // scores: token `lane`, rows 4 * warp ..
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
      const float4 *kr = reinterpret_cast<const float4 *>(sK + lane * RS);
      const float4 *qr = reinterpret_cast<const float4 *>(sQ + 4 * warp * RS);
      for (int d = 0; d < (D + 3) / 4; ++d) {
        const float4 kx = kr[d];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float4 qx = qr[r * (RS / 4) + d];
          acc[r] = fmaf(qx.x, kx.x, fmaf(qx.y, kx.y, fmaf(qx.z, kx.z, fmaf(qx.w, kx.w, acc[r]))));
        }
      }
      const int j = tile + lane;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int rr = 4 * warp + r;
        const bool vis = j < t1 && j >= s_lo[rr] && j < s_hi[rr];
        sS[rr * (kCsTok + 4) + lane] =
            vis ? chunk_score(a, acc[r], s_slope[rr], sq.n - sq.qlen + row_query(rr), j) : -INFINITY;
      }
    }
    __syncthreads();
    {                                           // softmax: 8 threads a row, 4 tokens each
      float x[4], mx = -INFINITY;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[i] = sS[srow * (kCsTok + 4) + sub + 8 * i];
        mx = fmaxf(mx, x[i]);
      }
#pragma unroll
      for (int w = 1; w < 8; w <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
      const float mn = fmaxf(m, mx);
      const float base = mn == -INFINITY ? 0.f : mn;   // nothing seen yet: every weight 0, not NaN
      const float alpha = fast_exp2(m - base);
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float p = fast_exp2(x[i] - base);
        sum += p;
        sP[(sub + 8 * i) * kCsRows + srow] = p;
      }
#pragma unroll
      for (int w = 1; w < 8; w <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
      l = fmaf(l, alpha, sum);
      m = mn;
      if (sub == 0) s_alpha[srow] = alpha;
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kCsRows; ++r) {
      const float al = s_alpha[r];
#pragma unroll
      for (int e = 0; e < EPT; ++e) o[r][e] *= al;
    }
    if (!any_odd) {
#pragma unroll 4
      for (int t = 0; t < kCsTok; ++t) {
        float v[EPT];
#pragma unroll
        for (int e = 0; e < EPT; ++e) {
          const int d = tid + kCsThreads * e;
          v[e] = d < D ? sV[t * RS + d] : 0.f;
        }
        const float4 *pr = reinterpret_cast<const float4 *>(sP + t * kCsRows);
#pragma unroll
        for (int r4 = 0; r4 < kCsRows / 4; ++r4) {
          const float4 p = pr[r4];
#pragma unroll
          for (int e = 0; e < EPT; ++e) {
            o[4 * r4][e] = fmaf(p.x, v[e], o[4 * r4][e]);
            o[4 * r4 + 1][e] = fmaf(p.y, v[e], o[4 * r4 + 1][e]);
            o[4 * r4 + 2][e] = fmaf(p.z, v[e], o[4 * r4 + 2][e]);
            o[4 * r4 + 3][e] = fmaf(p.w, v[e], o[4 * r4 + 3][e]);
          }
        }
      }
    } else {                                    // only what a row sees may reach it
      for (int t = 0; t < cnt; ++t) {
        float v[EPT];
#pragma unroll
        for (int e = 0; e < EPT; ++e) {
          const int d = tid + kCsThreads * e;
          v[e] = d < D ? sV[t * RS + d] : 0.f;
        }
#pragma unroll
        for (int r = 0; r < kCsRows; ++r)
          if (tile + t >= s_lo[r] && tile + t < s_hi[r])
#pragma unroll
            for (int e = 0; e < EPT; ++e) o[r][e] = fmaf(sP[t * kCsRows + r], v[e], o[r][e]);
      }
    }
  }
  if (sub == 0) {
    s_m[srow] = m;
    s_l[srow] = l;
  }
  __syncthreads();

  T *out = reinterpret_cast<T *>(a.out);
  auto out_row = [&](int r) { return (size_t)(sq.q0 + row_query(r)) * a.H + row_head(r); };
  if (nparts == 1) {
#pragma unroll
    for (int r = 0; r < kCsRows; ++r)
      if (r < rows)
#pragma unroll
        for (int e = 0; e < EPT; ++e) {
          const int d = tid + kCsThreads * e;
          if (d < D) out[out_row(r) * D + d] = from_f32<T>(s_hi[r] > s_lo[r] ? o[r][e] / s_l[r] : 0.f);
        }
    return;
  }
#pragma unroll
  for (int r = 0; r < kCsRows; ++r)
    if (r < rows) {
      const size_t at = out_row(r) * a.max_parts + slotp;
      if (tid == 0) {
        a.ws_m[at] = s_m[r];
        a.ws_l[at] = s_l[r];
      }
#pragma unroll
      for (int e = 0; e < EPT; ++e) {
        const int d = tid + kCsThreads * e;
        if (d < D) a.ws_o[at * D + d] = o[r][e];
      }
    }
  __syncthreads();
  int *counter = a.ws_cnt + kChunkCntFirst + ((size_t)b * a.KVH + kvh) * a.chunks + chunk;
  if (tid == 0) {
    int prev;
    asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;"
                 : "=r"(prev)
                 : "l"(reinterpret_cast<uint64_t>(counter))
                 : "memory");
    *s_flag = prev == nparts - 1;
  }
  __syncthreads();
  if (!*s_flag) return;
  // the last part merges: out = sum_p o_p 2^(m_p - M) / sum_p l_p 2^(m_p - M)
  for (int i = tid; i < rows * D; i += kCsThreads) {
    const int r = i / D, d = i - r * D;
    const size_t at = out_row(r) * a.max_parts;
    float M = -INFINITY, L = 0.f, acc = 0.f;
    for (int p = 0; p < nparts; ++p) M = fmaxf(M, __ldcg(a.ws_m + at + p));
    const float base = M == -INFINITY ? 0.f : M;
    for (int p = 0; p < nparts; ++p) {
      const float w = fast_exp2(__ldcg(a.ws_m + at + p) - base);
      L = fmaf(__ldcg(a.ws_l + at + p), w, L);
      acc = fmaf(__ldcg(a.ws_o + (at + p) * D + d), w, acc);
    }
    out[out_row(r) * D + d] = from_f32<T>(s_hi[r] > s_lo[r] ? acc / L : 0.f);
  }
  if (tid == 0) *counter = 0;
}

template <typename T>
static pkv_status launch_chunk_simt_t(const ChunkArgs &a, cudaStream_t stream) {
  const dim3 grid((unsigned)((long long)a.max_parts * a.KVH * a.chunks), a.B);
  const size_t smem = chunk_simt_smem(a.D);
  if (a.D <= 128) {
    static int configured[64] = {0};
    if (!allow_smem(pkv_chunk_simt_kernel<T, 1>, smem, configured)) return PKV_ERR_CUDA;
    pkv_chunk_simt_kernel<T, 1><<<grid, kCsThreads, smem, stream>>>(a);
  } else if (a.D <= 256) {
    static int configured[64] = {0};
    if (!allow_smem(pkv_chunk_simt_kernel<T, 2>, smem, configured)) return PKV_ERR_CUDA;
    pkv_chunk_simt_kernel<T, 2><<<grid, kCsThreads, smem, stream>>>(a);
  } else {
    static int configured[64] = {0};
    if (!allow_smem(pkv_chunk_simt_kernel<T, 4>, smem, configured)) return PKV_ERR_CUDA;
    pkv_chunk_simt_kernel<T, 4><<<grid, kCsThreads, smem, stream>>>(a);
  }
  return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

pkv_status launch_chunk_simt(const ChunkArgs &a, pkv_dtype dt, cudaStream_t stream) {
  switch (dt) {
    case PKV_F32: return launch_chunk_simt_t<float>(a, stream);
    case PKV_BF16: return launch_chunk_simt_t<__nv_bfloat16>(a, stream);
    case PKV_F16: return launch_chunk_simt_t<__half>(a, stream);
  }
  return PKV_ERR_INVALID_ARG;
}

}  // namespace pkv
