// pkv_quant_decode_mma.cuh -- decode over a quantised cache on the tensor
// cores (see pkv_quant_decode.cuh for parts and rows).
//
// Codes are whole numbers up to 255 or e4m3 values: exact in fp16.  So both
// products run as fp16 x fp16 -> fp32 on the codes themselves and the scales
// stay outside:
//   x_j = sk_j (q . ck_j),   O = sum_j (p_j sv_j) cv_j,   out = O / sum_j p_j.
// Tokens are the products' M (16 a tile), query heads their N = 8, so a code is
// unpacked once for 8 heads:
//   S^T[16 tokens x 8] = CK[16 x D] Q^T[D x 8],   O^T[D x 8] += CV^T[D x 16] W[16 x 8].
// q is scaled by a power of two a row (its largest element to [2^14, 2^15)),
// so that fp16 holds bf16's range; the weights w_j = p_j sv_j by another, of the
// largest value scale that the warp has met, so that w <= 2^15 whatever the
// scales are.  What falls below fp16 there is under 2^-30 of the largest value.
//
// SPLIT: columns 0-3 hold four heads, columns 4-7 what fp16 leaves of them: a
// query or a weight is hi + lo, good to 2^-23.  fp32 always, other types where
// the KV head has four query heads or fewer (the columns are free then).  bf16
// goes without: its queries are exact and the weights' half step, 2^-11, is an
// eighth of what it rounds off the output.  fp16 with more heads, where it would
// be as much as the output's own, has the rest of the weights in another turn of
// the second product.
//
// The running maximum is raised only when some score passes it by 2^8: one vote
// a tile of 32 tokens instead of three exchanges a head.
//
// CTA = 4 warps; warp w takes tiles w, w + 4, ... of 32 tokens through a ring of
// its own in shared memory, filled by 16-byte cp.async row by row (a row's place
// comes from the block table, so any block size will do), with no barrier
// between the warps.  Rows are padded to an odd number of 16-byte chunks: the
// 4-byte fragment loads of K and the transposing ldmatrix of V both touch every
// bank once.
#pragma once

#include "pkv_quant_decode.cuh"

namespace pkv {

constexpr int kQmTok = 32;
constexpr int kQmWarps = 4;

template <int D, int FMT, int NT>
struct QmShape {
  static constexpr int kRow = quant_row_bytes<FMT>(D);
  static constexpr int kChunks = kRow / 16;
  static constexpr int kStride = 16 * (kChunks | 1);                  // an odd number of chunks
  static constexpr int kParams = 4 * quant_params<FMT>();             // bytes a row
  static constexpr int kStage = kQmTok * 2 * (kStride + kParams);
  static constexpr int kCols = 8 * NT;
  static constexpr int kOStride = D + 4;
  // two CTAs an SM and more, whichever the registers allow
  static constexpr int kStages = kStage * kQmWarps * 3 <= 110 * 1024 ? 3 : 2;
  static constexpr int kRing = kStages * kStage * kQmWarps;
  static constexpr int kOut = kQmWarps * kCols * kOStride * 4;
  static constexpr int kMain = kRing > kOut ? kRing : kOut;
  static constexpr int kSmem = kMain + 4 * (2 * kQmWarps * kCols + 2 * kCols + 4);
  static_assert(kMain >= 1024, "the join's weights fit");
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_small(uint32_t dst, const void *src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ float lds_f32(uint32_t addr) { return __uint_as_float(lds32(addr)); }
__device__ __forceinline__ void ldsm_x2_trans(uint32_t addr, uint32_t &r0, uint32_t &r1) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0, %1}, [%2];" : "=r"(r0), "=r"(r1) : "r"(addr));
}
// An 8x8 tile of 16-bit elements, transposed across the warp.
__device__ __forceinline__ uint32_t movm_trans(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t hsub2_u(uint32_t a, uint32_t b) {
  __half2 r = __hsub2(*reinterpret_cast<__half2 *>(&a), *reinterpret_cast<__half2 *>(&b));
  return *reinterpret_cast<uint32_t *>(&r);
}
__device__ __forceinline__ uint32_t hfma2_u(uint32_t a, uint32_t b, uint32_t c) {
  __half2 r = __hfma2(*reinterpret_cast<__half2 *>(&a), *reinterpret_cast<__half2 *>(&b), *reinterpret_cast<__half2 *>(&c));
  return *reinterpret_cast<uint32_t *>(&r);
}
__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
  __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t *>(&v);
}

// Four codes of a word (one K row; of V's ldmatrix word, two columns of token
// 2t and the same of token 2t + 1) as two pairs of halves.
// int8: bytes (0, 2) and (1, 3): a byte with its top bit turned, code + 128, in
// the low bits of the half 1024 is 1152 + code exactly: one and-xor, one subtract.
// e4m3: K's bytes (0, 1) and (2, 3), V's as int8's.
template <int FMT, bool V>
__device__ __forceinline__ void code_pairs(uint32_t w, uint32_t &p0, uint32_t &p1) {
  if constexpr (FMT == kInt8) {
    p0 = hsub2_u((w & 0x00ff00ffu) ^ 0x64806480u, 0x64806480u);
    p1 = hsub2_u(((w >> 8) & 0x00ff00ffu) ^ 0x64806480u, 0x64806480u);
  } else {
    if (V) w = __byte_perm(w, 0, 0x3120);
    p0 = e4m3x2_to_half2((uint16_t)w);
    p1 = e4m3x2_to_half2((uint16_t)(w >> 16));
  }
}
// Eight 4-bit codes of a word, less the zero points: pairs (nibbles i, i + 4).
// z1 = 1024 + zero of the two halves' tokens, z16 = -(64 + zero): a nibble in
// bits 4-7 of the half 1024 + 16 c is brought down by a multiply-add, exactly.
__device__ __forceinline__ void nibble_pairs(uint32_t w, uint32_t z1, uint32_t z16, uint32_t (&p)[4]) {
  const uint32_t u = w >> 8;
  constexpr uint32_t kSixteenth = 0x2c002c00u;
  p[0] = hsub2_u((w & 0x000f000fu) | 0x64006400u, z1);
  p[1] = hfma2_u((w & 0x00f000f0u) | 0x64006400u, kSixteenth, z16);
  p[2] = hsub2_u((u & 0x000f000fu) | 0x64006400u, z1);
  p[3] = hfma2_u((u & 0x00f000f0u) | 0x64006400u, kSixteenth, z16);
}

// t / bs for t < 2^31 by a multiplication (mul, shift from the host).
__device__ __forceinline__ int div_by(int t, uint32_t mul, int shift) {
  return (int)((__umulhi((uint32_t)t, mul) + (uint32_t)t) >> shift);
}

template <int D, int FMT, int NT, bool SPLIT>
__global__ void __launch_bounds__(32 * kQmWarps) pkv_quant_decode_mma_kernel(const __grid_constant__ QuantDecodeArgs a,
                                                                             const int dt) {
  static_assert(NT == 1 || !SPLIT, "a split head's columns are in one tile");
  using Sh = QmShape<D, FMT, NT>;
  constexpr int W = kQmWarps, S = Sh::kStages, kSteps = D / 16, kHeads = SPLIT ? 4 : 8 * NT;
  extern __shared__ __align__(16) uint8_t ring[];
  float *s_wm = reinterpret_cast<float *>(ring + Sh::kMain);     // [W][cols] maxima, sums
  float *s_wl = s_wm + W * Sh::kCols;
  float *s_m = s_wl + W * Sh::kCols;                             // [cols]
  float *s_l = s_m + Sh::kCols;
  int *s_scratch = reinterpret_cast<int *>(s_l + Sh::kCols);
  const ChunkArgs &c = a.c;
  const QuantPart p = quant_part(a);
  if (p.nparts == 0) return;
  const bool rest = SPLIT ? dt != PKV_BF16 : dt == PKV_F16;   // weights of two parts
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, g = lane >> 2, t4 = lane & 3;
  const int ntiles = p.t1 > p.t0 ? (p.t1 - p.t0 + kQmTok - 1) / kQmTok : 0;
  const int mine = ntiles > w ? (ntiles - w + W - 1) / W : 0;
  const int first = max(p.t0, p.lo);
  uint8_t *my_ring = ring + (size_t)w * S * Sh::kStage;
  const uint32_t ring_at = smem_u32(my_ring);

  // Tile i of this warp into stage i mod S.  Lane r looks up token r's block one
  // tile ahead, so that the table entry is there when it is needed; what is
  // not visible is filled with zeros and not read.  (Rows of the cache are fewer
  // than 2^32 - 1 here.)
  constexpr bool kEven = 32 % Sh::kChunks == 0;          // a lane keeps to one chunk of the rows
  const int32_t *table = c.tables + (size_t)p.b * c.max_blocks;
  const uint8_t *k_at = a.k + lane % Sh::kChunks * 16, *v_at = a.v + lane % Sh::kChunks * 16;
  const uint32_t st_even = ring_at + lane / Sh::kChunks * Sh::kStride + lane % Sh::kChunks * 16;
  int next_phys = 0, next_off = -1;
  auto look_up = [&](int i) {
    const int t = p.t0 + kQmTok * (w + W * i) + lane;
    next_off = -1;
    if (i < mine && t >= first && t < p.t1) {
      const int lb = div_by(t, a.bs_mul, a.bs_shift);
      next_off = t - lb * c.bs;
      next_phys = __ldg(table + lb);
    }
  };
  auto issue = [&](int i) {
    if (i < mine) {
      bool in = next_off >= 0;
      if (in && (next_phys < 0 || (long long)next_phys >= c.num_blocks)) {
        raise_flag(c.err, PKV_FLAG_BLOCK_OUT_OF_RANGE);
        in = false;
      }
      const uint32_t phys = (uint32_t)next_phys, off = (uint32_t)next_off;
      const uint32_t row = in ? (phys * (uint32_t)c.bs + off) * (uint32_t)c.KVH + (uint32_t)p.kvh : 0xffffffffu;
      const uint32_t num = in ? (phys * (uint32_t)c.KVH + (uint32_t)p.kvh) * (uint32_t)c.bs + off : 0u;
      const uint32_t stage = (i % S) * Sh::kStage, st = ring_at + stage;
      const uint32_t pa = st + 2 * kQmTok * Sh::kStride + lane * Sh::kParams;
      cp_async_small<Sh::kParams>(pa, a.kp + (size_t)num * quant_params<FMT>(), in ? Sh::kParams : 0);
      cp_async_small<Sh::kParams>(pa + kQmTok * Sh::kParams, a.vp + (size_t)num * quant_params<FMT>(), in ? Sh::kParams : 0);
      if (kEven && __all_sync(0xffffffffu, in)) {
#pragma unroll
        for (int j = 0; j < Sh::kChunks; ++j) {
          const uint32_t from = __shfl_sync(0xffffffffu, row, lane / Sh::kChunks + j * (32 / Sh::kChunks));
          const uint32_t to = st_even + stage + j * (32 / Sh::kChunks) * Sh::kStride;
          cp_async16(to, k_at + (size_t)from * Sh::kRow, 16);
          cp_async16(to + kQmTok * Sh::kStride, v_at + (size_t)from * Sh::kRow, 16);
        }
      } else {
#pragma unroll
        for (int j = 0; j < Sh::kChunks; ++j) {
          const int idx = lane + 32 * j, r = idx / Sh::kChunks, ch = idx - r * Sh::kChunks;
          const uint32_t from = __shfl_sync(0xffffffffu, row, r);
          const bool has = from != 0xffffffffu;
          const size_t at = has ? (size_t)from * Sh::kRow + ch * 16 : 0;
          const uint32_t to = st + r * Sh::kStride + ch * 16;
          cp_async16(to, a.k + at, has ? 16 : 0);
          cp_async16(to + kQmTok * Sh::kStride, a.v + at, has ? 16 : 0);
        }
      }
      look_up(i + 1);
    }
    cp_async_commit();
  };
  look_up(0);
#pragma unroll
  for (int i = 0; i < S - 1; ++i) issue(i);

  // The queries, scaled, as the product's B: column g of a tile is a head (or
  // what fp16 left of head g - 4); warp-wide maximum of a row's elements.
  auto q_at = [&](int h, int d) {
    const size_t i = ((size_t)p.b * c.H + p.head0 + h) * D + d;
    return dt == PKV_F32 ? reinterpret_cast<const float *>(c.q)[i]
         : dt == PKV_BF16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(c.q)[i])
                          : __half2float(reinterpret_cast<const __half *>(c.q)[i]);
  };
  // scores in log2 units, or what their cap wants (see chunk_capped: its error
  // does for 16-bit types; chunk_cap)
  const int cap = !(c.cap_log2 > 0.f) ? kCapNone : dt != PKV_F32 && c.cap_log2 <= kCapShort ? kCapUsual : kCapLarge;
  const float score_unit = cap == kCapNone ? c.scale_log2 : cap == kCapUsual ? c.scale_y : 1.f;
  uint32_t qf[NT][kSteps][2];
  float qs[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int col_head = SPLIT ? g & 3 : 8 * nt + g;
    const bool has = col_head < p.rows, low = SPLIT && g >= 4;
    float v[kSteps][4], big = 0.f;
#pragma unroll
    for (int ks = 0; ks < kSteps; ++ks)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        // the column of A's element (see code_pairs, nibble_pairs)
        const int d = FMT == kInt4   ? (ks >> 1) * 32 + 8 * t4 + 2 * (ks & 1) + (e >> 1) + 4 * (e & 1)
                      : FMT == kInt8 ? ks * 16 + 4 * t4 + (e >> 1) + 2 * (e & 1)
                                     : ks * 16 + 4 * t4 + e;
        v[ks][e] = has ? q_at(col_head, d) : 0.f;
        big = fmaxf(big, fabsf(v[ks][e]));
      }
    big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
    big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
    // 2^(14 - floor(log2 big)), both ends within fp32's exponents
    const int ex = min(max((__float_as_int(big) >> 23) - 127, -100), 100);
    const float up = __int_as_float((14 - ex + 127) << 23), down = __int_as_float((ex - 14 + 127) << 23);
#pragma unroll
    for (int ks = 0; ks < kSteps; ++ks)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x = v[ks][2 * e] * up, y = v[ks][2 * e + 1] * up;
        if (low) {
          x = dt == PKV_F32 ? x - __half2float(__float2half_rn(x)) : x;
          y = dt == PKV_F32 ? y - __half2float(__float2half_rn(y)) : y;
        }
        qf[nt][ks][e] = half2_bits(x, y);
      }
    // this lane's score columns are 2 t4, 2 t4 + 1
    qs[nt][0] = __shfl_sync(0xffffffffu, down, 8 * t4) * score_unit;
    qs[nt][1] = __shfl_sync(0xffffffffu, down, 8 * t4 + 4) * score_unit;
  }

  float o[NT][kSteps][4] = {};
  float m[NT][2], l[NT][2];
  // O's unit is 2^(ve - kUnit): ve the largest exponent of a value's scale so far
  // (fp32's biased one; from 2^-97 on, NaN and infinity aside)
  constexpr int kUnit = 127 + 6;
  int ve = 30;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      m[nt][e] = -INFINITY;
      l[nt][e] = 0.f;
    }

  for (int i = 0; i < mine; ++i) {
    cp_async_wait<S - 2>();
    __syncwarp();                                        // (and every lane is done with tile i - 1, whose stage is next)
    issue(i + S - 1);
    const uint32_t kb = ring_at + (i % S) * Sh::kStage, vb = kb + kQmTok * Sh::kStride;
    const uint32_t kpb = vb + kQmTok * Sh::kStride, vpb = kpb + kQmTok * Sh::kParams;
    const int tile0 = p.t0 + kQmTok * (w + W * i);
    const bool whole = tile0 >= first && tile0 + kQmTok <= p.t1;
    float x[2][NT][4], sv[2][2];
    int ve_new = ve;
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
      const int r0 = mt * 16 + g, r1 = r0 + 8;
      float s[NT][4] = {};
      const uint32_t k0 = kb + r0 * Sh::kStride + 4 * t4, k1 = k0 + 8 * Sh::kStride;
      if constexpr (FMT == kInt4) {
        const uint32_t z0 = half2_bits(lds_f32(kpb + r0 * 8 + 4), 0.f) & 0xffffu, z1 = half2_bits(lds_f32(kpb + r1 * 8 + 4), 0.f) & 0xffffu;
        const uint32_t zz0 = z0 | (z0 << 16), zz1 = z1 | (z1 << 16);
        const uint32_t a1 = hfma2_u(zz0, 0x3c003c00u, 0x64006400u), b1 = hfma2_u(zz1, 0x3c003c00u, 0x64006400u);   // 1024 + z
        const uint32_t a16 = hfma2_u(zz0, 0xbc00bc00u, 0xd400d400u), b16 = hfma2_u(zz1, 0xbc00bc00u, 0xd400d400u); // -64 - z
#pragma unroll
        for (int k2 = 0; k2 < D / 32; ++k2) {
          uint32_t f0[4], f1[4];
          nibble_pairs(lds32(k0 + k2 * 16), a1, a16, f0);
          nibble_pairs(lds32(k1 + k2 * 16), b1, b16, f1);
          const uint32_t A[4] = {f0[0], f1[0], f0[1], f1[1]}, B[4] = {f0[2], f1[2], f0[3], f1[3]};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            MmaOp<__half>::run(s[nt], A, qf[nt][2 * k2][0], qf[nt][2 * k2][1]);
            MmaOp<__half>::run(s[nt], B, qf[nt][2 * k2 + 1][0], qf[nt][2 * k2 + 1][1]);
          }
        }
      } else {
#pragma unroll
        for (int ks = 0; ks < kSteps; ++ks) {
          uint32_t A[4];
          code_pairs<FMT, false>(lds32(k0 + ks * 16), A[0], A[2]);
          code_pairs<FMT, false>(lds32(k1 + ks * 16), A[1], A[3]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) MmaOp<__half>::run(s[nt], A, qf[nt][ks][0], qf[nt][ks][1]);
        }
      }
      const float sk0 = lds_f32(kpb + r0 * Sh::kParams), sk1 = lds_f32(kpb + r1 * Sh::kParams);
      sv[mt][0] = lds_f32(vpb + r0 * Sh::kParams);
      sv[mt][1] = lds_f32(vpb + r1 * Sh::kParams);
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const int ex = (__float_as_int(sv[mt][hf]) >> 23) & 255;
        if (ex != 255) ve_new = max(ve_new, ex);
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if (SPLIT && dt == PKV_F32) {
#pragma unroll
          for (int e = 0; e < 4; ++e) s[nt][e] += __shfl_xor_sync(0xffffffffu, s[nt][e], 2);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) x[mt][nt][e] = s[nt][e] * qs[nt][e & 1] * (e < 2 ? sk0 : sk1);
      }
    }
    if (cap != kCapNone) {
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            x[mt][nt][e] = cap == kCapUsual ? chunk_capped(x[mt][nt][e], c.cap_log2) : chunk_cap(c, x[mt][nt][e]);
    }
    if (!whole) {
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const int t = tile0 + mt * 16 + hf * 8 + g;
          if (t >= first && t < p.t1) continue;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) x[mt][nt][2 * hf] = x[mt][nt][2 * hf + 1] = -INFINITY;
        }
    }
    // raise the maxima where a score passes them by 2^8, and O's unit where a
    // value's scale passes it
    bool over = ve_new > ve;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const float m0 = m[nt][0] + 8.f, m1 = m[nt][1] + 8.f;
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
        over = over || x[mt][nt][0] > m0 || x[mt][nt][1] > m1 || x[mt][nt][2] > m0 || x[mt][nt][3] > m1;
    }
    if (__any_sync(0xffffffffu, over)) {
      ve_new = __reduce_max_sync(0xffffffffu, ve_new);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float top = fmaxf(fmaxf(x[0][nt][e], x[0][nt][e + 2]), fmaxf(x[1][nt][e], x[1][nt][e + 2]));
#pragma unroll
          for (int sh = 4; sh < 32; sh <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, sh));
          top = fmaxf(top, m[nt][e]);
          const float d = m[nt][e] - chunk_ref(top), f = fast_exp2(d + (float)(ve - ve_new));
          l[nt][e] *= fast_exp2(d);
          m[nt][e] = top;
#pragma unroll
          for (int ks = 0; ks < kSteps; ++ks) {
            o[nt][ks][e] *= f;
            o[nt][ks][e + 2] *= f;
          }
        }
      ve = ve_new;
    }
    const float unit = __int_as_float((127 + kUnit - ve) << 23);    // 2^(kUnit - ve)
    // weights, as the product's B
    uint32_t wb[2][NT][2], wl[2][NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const float r0 = chunk_ref(m[nt][0]), r1 = chunk_ref(m[nt][1]);
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const float p0 = fast_exp2(x[mt][nt][2 * hf] - r0), p1 = fast_exp2(x[mt][nt][2 * hf + 1] - r1);
          const float s1 = sv[mt][hf] * unit, w0 = p0 * s1, w1 = p1 * s1;
          l[nt][0] += p0;
          l[nt][1] += p1;
          __half2 h = __floats2half2_rn(w0, w1);
          if (rest) {
            const float2 f = __half22float2(h);
            const __half2 lo = __floats2half2_rn(w0 - f.x, w1 - f.y);
            if (SPLIT) {
              if (t4 >= 2) h = lo;
            } else {
              wl[mt][nt][hf] = movm_trans(*reinterpret_cast<const uint32_t *>(&lo));
            }
          }
          wb[mt][nt][hf] = movm_trans(*reinterpret_cast<uint32_t *>(&h));
        }
    }
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
      const uint32_t va = vb + (mt * 16 + (lane & 15)) * Sh::kStride + (lane >> 4) * 16;
      if constexpr (FMT == kInt4) {
        // tokens 2 t4, 2 t4 + 1 (and 8 behind them) of this half tile
        uint32_t z1[2], z16[2];
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const uint32_t z = half2_bits(lds_f32(vpb + (mt * 16 + 8 * hf + 2 * t4) * 8 + 4),
                                        lds_f32(vpb + (mt * 16 + 8 * hf + 2 * t4 + 1) * 8 + 4));
          z1[hf] = hfma2_u(z, 0x3c003c00u, 0x64006400u);
          z16[hf] = hfma2_u(z, 0xbc00bc00u, 0xd400d400u);
        }
        auto block = [&](int ch, uint32_t r0, uint32_t r1) {      // 32 columns of 16 tokens
          uint32_t f0[4], f1[4];
          nibble_pairs(r0, z1[0], z16[0], f0);
          nibble_pairs(r1, z1[1], z16[1], f1);
#pragma unroll
          for (int q2 = 0; q2 < 2; ++q2) {
            const uint32_t A[4] = {f0[2 * q2], f0[2 * q2 + 1], f1[2 * q2], f1[2 * q2 + 1]};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              MmaOp<__half>::run(o[nt][2 * ch + q2], A, wb[mt][nt][0], wb[mt][nt][1]);
              if (!SPLIT && rest) MmaOp<__half>::run(o[nt][2 * ch + q2], A, wl[mt][nt][0], wl[mt][nt][1]);
            }
          }
        };
#pragma unroll
        for (int ch = 0; ch + 1 < Sh::kChunks; ch += 2) {
          uint32_t r0, r1, r2, r3;
          ldsm_x4_trans(va + ch * 16, r0, r1, r2, r3);
          block(ch, r0, r1);
          block(ch + 1, r2, r3);
        }
        if constexpr (Sh::kChunks & 1) {
          uint32_t r0, r1;
          ldsm_x2_trans(vb + (mt * 16 + (lane & 15)) * Sh::kStride + (Sh::kChunks - 1) * 16, r0, r1);
          block(Sh::kChunks - 1, r0, r1);
        }
      } else {
        auto block = [&](int ch, uint32_t r0, uint32_t r1) {      // 16 columns of 16 tokens
          uint32_t A[4];
          code_pairs<FMT, true>(r0, A[0], A[1]);
          code_pairs<FMT, true>(r1, A[2], A[3]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            MmaOp<__half>::run(o[nt][ch], A, wb[mt][nt][0], wb[mt][nt][1]);
            if (!SPLIT && rest) MmaOp<__half>::run(o[nt][ch], A, wl[mt][nt][0], wl[mt][nt][1]);
          }
        };
#pragma unroll
        for (int ch = 0; ch + 1 < Sh::kChunks; ch += 2) {
          uint32_t r0, r1, r2, r3;
          ldsm_x4_trans(va + ch * 16, r0, r1, r2, r3);
          block(ch, r0, r1);
          block(ch + 1, r2, r3);
        }
        if constexpr (Sh::kChunks & 1) {
          uint32_t r0, r1;
          ldsm_x2_trans(vb + (mt * 16 + (lane & 15)) * Sh::kStride + (Sh::kChunks - 1) * 16, r0, r1);
          block(Sh::kChunks - 1, r0, r1);
        }
      }
    }
  }
  cp_async_wait<0>();

  // Merge the warps.  Column sums over the lanes of a column first.
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int sh = 4; sh < 32; sh <<= 1) l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], sh);
      if (g == 0) {
        const int at = w * Sh::kCols + 8 * nt + 2 * t4 + e;
        s_wm[at] = m[nt][e];
        s_wl[at] = l[nt][e];
      }
    }
  __syncthreads();                                       // (every ring is free too)
  float *s_o = reinterpret_cast<float *>(ring);          // [W][cols][kOStride]
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int col = 8 * nt + 2 * t4 + e;
      float M = -INFINITY;
#pragma unroll
      for (int k = 0; k < W; ++k) M = fmaxf(M, s_wm[k * Sh::kCols + col]);
      const float f = exp2f(m[nt][e] - chunk_ref(M) + (float)(ve - kUnit));
      float *dst = s_o + (w * Sh::kCols + col) * Sh::kOStride;
#pragma unroll
      for (int ks = 0; ks < kSteps; ++ks) {
        // rows g and g + 8 of tile ks are columns of V (see code_pairs, nibble_pairs)
        const int d = FMT == kInt4 ? (ks >> 1) * 32 + 4 * g + 2 * (ks & 1) : ks * 16 + 2 * g;
        *reinterpret_cast<float2 *>(dst + d) = make_float2(o[nt][ks][e] * f, o[nt][ks][e + 2] * f);
      }
    }
  if (threadIdx.x < Sh::kCols) {
    const int col = threadIdx.x;
    float M = -INFINITY, L = 0.f;
    for (int k = 0; k < W; ++k) M = fmaxf(M, s_wm[k * Sh::kCols + col]);
    for (int k = 0; k < W; ++k) L += s_wl[k * Sh::kCols + col] * exp2f(s_wm[k * Sh::kCols + col] - chunk_ref(M));
    if (col < kHeads) {
      s_m[col] = M;
      s_l[col] = L;
    }
  }
  __syncthreads();
  // sum the warps (and a head's two columns) into the head's first row, which
  // only the thread that writes it reads
  for (int i = threadIdx.x; i < kHeads * D; i += 32 * W) {
    const int r = i / D, d = i - r * D, col = r;
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < W; ++k) {
      sum += s_o[(k * Sh::kCols + col) * Sh::kOStride + d];
      if (SPLIT && rest) sum += s_o[(k * Sh::kCols + col + 4) * Sh::kOStride + d];
    }
    s_o[r * Sh::kOStride + d] = sum;
  }
  __syncthreads();
  constexpr int kRoom = Sh::kMain / 4;
  if (dt == PKV_F32)
    quant_finish<float>(c, p, s_m, s_l, s_o, Sh::kOStride, kRoom, s_scratch);
  else if (dt == PKV_BF16)
    quant_finish<__nv_bfloat16>(c, p, s_m, s_l, s_o, Sh::kOStride, kRoom, s_scratch);
  else
    quant_finish<__half>(c, p, s_m, s_l, s_o, Sh::kOStride, kRoom, s_scratch);
}

template <int D, int FMT, int NT, bool SPLIT>
static pkv_status launch_qm(const QuantDecodeArgs &a, pkv_dtype dt, cudaStream_t stream) {
  static int configured[64];
  auto kern = pkv_quant_decode_mma_kernel<D, FMT, NT, SPLIT>;
  constexpr int kSmem = QmShape<D, FMT, NT>::kSmem;
  if (!allow_smem(kern, kSmem, configured)) return PKV_ERR_CUDA;
  kern<<<dim3((unsigned)(a.c.chunks * a.c.KVH * a.c.max_parts), (unsigned)a.c.B), 32 * kQmWarps, kSmem, stream>>>(a, (int)dt);
  return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

template <int D, int FMT>
static pkv_status launch_qm_d(const QuantDecodeArgs &a, int tiles, bool split, pkv_dtype dt, cudaStream_t stream) {
  if (split) return launch_qm<D, FMT, 1, true>(a, dt, stream);
  return launch_qm<D, FMT, 1, false>(a, dt, stream);
}

// Every head_dim of a format.
template <int FMT>
static pkv_status launch_qm_f(const QuantDecodeArgs &a, int tiles, bool split, pkv_dtype dt, cudaStream_t stream) {
  switch (a.c.D) {
    case 64: return launch_qm_d<64, FMT>(a, tiles, split, dt, stream);
    case 80:
      if constexpr (FMT != kInt4) return launch_qm_d<80, FMT>(a, tiles, split, dt, stream);
      break;
    case 96: return launch_qm_d<96, FMT>(a, tiles, split, dt, stream);
    case 128: return launch_qm_d<128, FMT>(a, tiles, split, dt, stream);
    case 192: return launch_qm_d<192, FMT>(a, tiles, split, dt, stream);
    case 256: return launch_qm_d<256, FMT>(a, tiles, split, dt, stream);
  }
  return PKV_ERR_UNSUPPORTED;
}

}  // namespace pkv
