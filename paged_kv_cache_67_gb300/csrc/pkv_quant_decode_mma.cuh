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
// query or a weight is hi + lo, good to 2^-22.  fp32 always, other types where
// the KV head has four query heads or fewer (the columns are free then).  16-bit
// types with more heads, whose queries are exact in one column, have the rest of
// the weights in another turn of the second product.  (Weights of one fp16
// number, 2^-11 each, would move bf16 outputs by a step in places: the second
// turn takes 64 x 512-4096 keys of 8 heads of 128, int8, 64 query heads, from
// 76.2 to 77.2 us.)
//
// The running maximum is raised only when some score passes it by 2^8: one vote
// a tile instead of three exchanges a head.
//
// Work.  All tiles of all units -- a unit is a sequence's visible keys for one
// head group of a KV head -- stand in one line, and every warp of a grid that
// fills the GPU once takes an equal stretch of it: lengths may be as ragged as
// they like.  Warps run by themselves, with no barrier over the CTA: each has a
// ring in shared memory and a second warp that fills it (across the ends of units
// too): asking for a tile takes as long as computing on it, some 1300 cycles.  Where blocks are whole
// chunks of 16 tokens, TMA brings them, a box of K and one of V a chunk; any other
// block size goes row by row, 16 bytes a cp.async, to the same places.  (All by
// cp.async, a batch of 64 x 2304 keys took 79 us, and 88 with the arithmetic
// left out.)
// A warp that has a whole unit writes its output.  The others leave the states
// (max, sum, weighted sum) of the unit they began in and the one they end in, two
// places a warp, and the last one done of up to 16 neighbours joins them, then of
// up to 16 such groups, until the unit is one.
//
// Measured: 64 x 512-4096 keys of 8 heads of 128, int8, 32 query heads: 60-61.7 us,
// 5.1 TB/s (4 bits 56 us, 3.0 TB/s); 8 x 16-32k keys, e4m3, capped: 75-77 us,
// 5.3 TB/s.  What bounds it: a tile is a chain of some 1600 cycles in each of an
// SM's eight computing warps.  One KV head of 16 heads of 256, 4 bits, 128 x 1-8192
// keys: 56 us, where the 16-bit cache's kernel takes 35 (two units unpack every
// key, and start and end for every short sequence).
//
// Rows in the ring are swizzled as TMA does it: the 4-byte fragment loads of K
// and the transposing ldmatrix of V both touch every bank once.
#pragma once

#include <string.h>

#include "pkv_quant_decode.cuh"

namespace pkv {

template <int D, int FMT>
struct QmShape {
  static constexpr int kRow = quant_row_bytes<FMT>(D);
  static constexpr int kChunks = kRow / 16;
  static constexpr int kBox = qm_box(kRow);                           // bytes of a row that lie together
  static constexpr int kSwizzle = kBox == 128 ? 0x70 : kBox == 64 ? 0x30 : kBox == 32 ? 0x10 : 0;
  static constexpr int kParams = 4 * quant_params<FMT>();             // bytes a row
  static constexpr int kHalf = 16 * kRow;                             // 16 tokens' rows of K or V
  static constexpr int kCodes = 2 * kQmHalves * kHalf;                // of a tile: K's halves, V's
  static constexpr int kStages = qm_stages(kRow, kParams);
  static constexpr int kSmem = qm_smem(kRow, kParams);
  static constexpr int kCtas = qm_ctas(kRow, kParams);
  static_assert(kHalf % 128 == 0 && (kSwizzle == 0 || kHalf % (8 * kBox) == 0), "the swizzle's period");
};
// Where chunk ch of row r of a half lies in it.
template <int ROW, int BOX, int MASK>
__device__ __forceinline__ int qm_at(int r, int ch) {
  constexpr int kPer = BOX / 16;
  const int in = r * BOX + ch % kPer * 16;
  return ch / kPer * (16 * BOX) + (in ^ ((in >> 3) & MASK));
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_small(uint32_t dst, const void *src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N), "r"(bytes) : "memory");
}
// As mbar_wait_bounded; the warp sleeps up to a millisecond at a time: looking
// again and again took a third of this kernel's instructions from the warps that
// compute.
__device__ __forceinline__ bool mbar_sleep_bounded(uint64_t *bar, uint32_t parity) {
  auto done = [&]() {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(1000000u)
        : "memory");
    return ok != 0;
  };
  if (done()) return true;
  const unsigned long long t0 = global_timer_ns();
  while (!done()) {
    if (global_timer_ns() - t0 > kWaitLimitNs) return false;
  }
  return true;
}
// Arrives on `bar` once this thread's cp.async so far are done.
__device__ __forceinline__ void cp_async_arrive(uint64_t *bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
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

// (w & m) ^ c and (w & m) | c in one instruction each (written out, or two
// constants become two instructions).
__device__ __forceinline__ uint32_t and_xor(uint32_t w, uint32_t m, uint32_t c) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0x6a;" : "=r"(r) : "r"(w), "r"(m), "r"(c));
  return r;
}
__device__ __forceinline__ uint32_t and_or(uint32_t w, uint32_t m, uint32_t c) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(r) : "r"(w), "r"(m), "r"(c));
  return r;
}

// Four codes of a word (one K row; of V's ldmatrix word, two columns of token
// 2t and the same of token 2t + 1) as two pairs of halves.
// (Whole numbers become halves by their bits, as is usual: or-ed into the low
// bits of 1024, whose unit in fp16 is 1.)
// int8: bytes (0, 2) and (1, 3): a byte with its top bit turned, code + 128, in
// the low bits of the half 1024 is 1152 + code exactly: one and-xor, one subtract.
// e4m3: K's bytes (0, 1) and (2, 3), V's as int8's.
template <int FMT, bool V>
__device__ __forceinline__ void code_pairs(uint32_t w, uint32_t &p0, uint32_t &p1) {
  if constexpr (FMT == kInt8) {
    p0 = hsub2_u(and_xor(w, 0x00ff00ffu, 0x64806480u), 0x64806480u);
    p1 = hsub2_u(and_xor(w >> 8, 0x00ff00ffu, 0x64806480u), 0x64806480u);
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
  p[0] = hsub2_u(and_or(w, 0x000f000fu, 0x64006400u), z1);
  p[1] = hfma2_u(and_or(w, 0x00f000f0u, 0x64006400u), kSixteenth, z16);
  p[2] = hsub2_u(and_or(u, 0x000f000fu, 0x64006400u), z1);
  p[3] = hfma2_u(and_or(u, 0x00f000f0u, 0x64006400u), kSixteenth, z16);
}

// t / bs for t < 2^31 by a multiplication (mul, shift from the host).
__device__ __forceinline__ int div_by(int t, uint32_t mul, int shift) {
  return (int)((__umulhi((uint32_t)t, mul) + (uint32_t)t) >> shift);
}

// N times four consecutive elements of a query row, place(i) the first of the
// i-th: every load is on its way before the first is looked at.
template <int N, typename Place>
__device__ __forceinline__ void q_fours(const void *q, int dt, bool aligned, const Place &place, float4 (&v)[N]) {
  if (dt == PKV_F32) {
    const float *p = reinterpret_cast<const float *>(q);
    if (aligned) {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = __ldg(reinterpret_cast<const float4 *>(p + place(i)));
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = make_float4(__ldg(p + place(i)), __ldg(p + place(i) + 1), __ldg(p + place(i) + 2), __ldg(p + place(i) + 3));
    }
    return;
  }
  const unsigned short *p = reinterpret_cast<const unsigned short *>(q);
  uint2 w[N];
  if (aligned) {
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = __ldg(reinterpret_cast<const uint2 *>(p + place(i)));
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      w[i] = make_uint2(__ldg(p + place(i)) | ((uint32_t)__ldg(p + place(i) + 1) << 16),
                        __ldg(p + place(i) + 2) | ((uint32_t)__ldg(p + place(i) + 3) << 16));
  }
  if (dt == PKV_BF16) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      v[i] = make_float4(__uint_as_float(w[i].x << 16), __uint_as_float(w[i].x & 0xffff0000u), __uint_as_float(w[i].y << 16),
                         __uint_as_float(w[i].y & 0xffff0000u));
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float2 a = half2_to_float2(w[i].x), b = half2_to_float2(w[i].y);
      v[i] = make_float4(a.x, a.y, b.x, b.y);
    }
  }
}

// Two (four) neighbouring elements of an output row.
__device__ __forceinline__ void put_two(void *out, size_t at, int dt, bool aligned, float x, float y) {
  if (dt == PKV_F32) {
    float *p = reinterpret_cast<float *>(out) + at;
    if (aligned) { *reinterpret_cast<float2 *>(p) = make_float2(x, y); return; }
    p[0] = x; p[1] = y;
    return;
  }
  uint32_t w;
  if (dt == PKV_BF16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
    w = *reinterpret_cast<const uint32_t *>(&v);
  } else {
    w = half2_bits(x, y);
  }
  unsigned short *p = reinterpret_cast<unsigned short *>(out) + at;
  if (aligned) { *reinterpret_cast<uint32_t *>(p) = w; return; }
  p[0] = (unsigned short)w; p[1] = (unsigned short)(w >> 16);
}

// N pairs of neighbouring elements of an output row that begins at element `at`:
// the i-th at column(i).  (The type is looked at once, not for every pair.)
template <int N, typename Column, typename Pair>
__device__ __forceinline__ void put_pairs(void *out, size_t at, int dt, bool aligned, const Column &column, const Pair &pair) {
  if (aligned && dt == PKV_BF16) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float2 v = pair(i);
      *reinterpret_cast<__nv_bfloat162 *>(reinterpret_cast<__nv_bfloat16 *>(out) + at + column(i)) = __floats2bfloat162_rn(v.x, v.y);
    }
  } else if (aligned && dt == PKV_F16) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float2 v = pair(i);
      *reinterpret_cast<__half2 *>(reinterpret_cast<__half *>(out) + at + column(i)) = __floats2half2_rn(v.x, v.y);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float2 v = pair(i);
      put_two(out, at + column(i), dt, aligned, v.x, v.y);
    }
  }
}

// A place in the line of tiles: tile `tile` of `tiles` of a team's unit `unit` of
// sequence b, this warp's KV head.
struct QmAt {
  int b, unit, kvh, tile, tiles, first, n, base;
};

// Sequence b's visible keys and tiles of them.
__device__ __forceinline__ void qm_keys(const ChunkArgs &c, int b, QmAt &s) {
  int n = __ldg(c.lens + b);
  n = min(max(n, 0), c.max_n);             // (max_n is at most the table's keys)
  s.n = n;
  s.first = c.window > 0 ? max(0, n - c.window) : 0;
  s.base = s.first & ~(kQmTok - 1);
  s.tiles = (n - s.base + kQmTok - 1) / kQmTok;
}

template <int D, int FMT, bool SPLIT>
__global__ void __launch_bounds__(kQmThreads, QmShape<D, FMT>::kCtas)
    pkv_quant_decode_mma_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                                const __grid_constant__ QuantDecodeArgs a, const int dt) {
  using Sh = QmShape<D, FMT>;
  constexpr int S = Sh::kStages, kSteps = D / 16, kHeads = SPLIT ? 4 : 8;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t *codes_all = smem, *params_all = smem + kQmWarps * S * Sh::kCodes;
  uint64_t *bars_all = reinterpret_cast<uint64_t *>(params_all + kQmWarps * S * 2 * kQmTok * Sh::kParams);
  int *s_first = reinterpret_cast<int *>(bars_all + 2 * kQmWarps * S);       // [groups + 1] tiles of one (KV head, head group)
  int *s_warp = s_first + kQmGroups + 2;
  const ChunkArgs &c = a.c;
  const bool producer = threadIdx.x >= 32 * kQmWarps;         // warp w + 4 fills warp w's ring
  const int lane = threadIdx.x & 31, w = (threadIdx.x >> 5) % kQmWarps, g = lane >> 2, t4 = lane & 3;
  const bool q16 = reinterpret_cast<uintptr_t>(c.q) % 16 == 0, out8 = reinterpret_cast<uintptr_t>(c.out) % 8 == 0;

  // ---- the line: first tiles of kQmGroups groups of sequences
  const int per = (c.B + kQmGroups - 1) / kQmGroups;
  {
    int sum = 0;
    for (int b = threadIdx.x * per; !producer && b < min(c.B, (int)(threadIdx.x + 1) * per); ++b) {
      QmAt s;
      qm_keys(c, b, s);
      sum += s.tiles;                       // (fewer than 2^31 in all: the host's check)
      if (blockIdx.x == 0) {
        const int n = __ldg(c.lens + b);
        if (n < 0) raise_flag(c.err, PKV_FLAG_CONTEXT_NEGATIVE);
        if ((long long)n > (long long)c.max_blocks * c.bs) raise_flag(c.err, PKV_FLAG_CONTEXT_TOO_LONG);
        else if (n > c.max_n) raise_flag(c.err, PKV_FLAG_CONTEXT_OVER_HINT);
      }
    }
    int scan = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, scan, o);
      if (lane >= o) scan += x;
    }
    if (!producer && lane == 31) s_warp[w] = scan;
    if (threadIdx.x == 0) s_first[0] = 0;
    if (threadIdx.x < 2 * kQmWarps * S) {
      // full: the copies' lanes (and the one that asks for boxes); then free again
      mbar_init(&bars_all[threadIdx.x], threadIdx.x >= kQmWarps * S ? 1 : a.tma ? 33 : 32);
      fence_mbar_init();
    }
    __syncthreads();
    if (!producer) {
      for (int k = 0; k < w; ++k) scan += s_warp[k];
      s_first[threadIdx.x + 1] = scan;
    }
    __syncthreads();
  }
  // A team of `team` neighbouring warps (of one CTA, or two) walks the same
  // tokens for neighbouring units, so that a token's rows, which lie together,
  // are read together; the line is one of teams' units.
  const int team = a.team, per_b = c.KVH * c.chunks / team;
  const long long total = (long long)s_first[kQmGroups] * per_b;
  const long long warps = (long long)gridDim.x * kQmWarps;
  const long long teams = warps / team;
  const long long share = max((total + teams - 1) / teams, (long long)a.least);
  const int mate = team > kQmWarps ? (blockIdx.x % (team / kQmWarps)) * kQmWarps + w : w % team;
  // neighbours in the line are on different SMs: short lines use them all
  const int me = team > kQmWarps ? blockIdx.x / (team / kQmWarps) : w / team * gridDim.x + blockIdx.x;
  const long long begin = me * share;
  const int mine = begin < total && me < teams ? (int)min(share, total - begin) : 0;

  QmAt cur = {};
  long long unit0 = 0;                      // the current unit's first tile in the line
  if (mine > 0) {
    // the group by bisection, its sequence 32 at a time, then the unit
    int lo = 0, hi = kQmGroups - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if ((long long)s_first[mid] * per_b <= begin) lo = mid; else hi = mid - 1;
    }
    long long at = (long long)s_first[lo] * per_b;
    int b = lo * per;
    for (;;) {
      QmAt s;
      s.tiles = 0;
      if (b + lane < c.B) qm_keys(c, b + lane, s);
      int scan = s.tiles;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, scan, o);
        if (lane >= o) scan += x;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, at + (long long)scan * per_b > begin);
      if (past) {
        const int k = __ffs(past) - 1;
        at += (long long)(__shfl_sync(0xffffffffu, scan, k) - __shfl_sync(0xffffffffu, s.tiles, k)) * per_b;
        b += k;
        break;
      }
      at += (long long)__shfl_sync(0xffffffffu, scan, 31) * per_b;
      b += 32;                              // (begin < total: some sequence has the tile)
    }
    qm_keys(c, b, cur);
    cur.b = b;
    const int off = (int)(begin - at), unit = off / cur.tiles;
    cur.tile = off - unit * cur.tiles;
    cur.unit = unit;
    cur.kvh = (unit * team + mate) / c.chunks;
    unit0 = begin - cur.tile;
  }
  // the next tile's place; whether it is another unit's
  auto advance = [&](QmAt &s) {
    if (++s.tile < s.tiles) return false;
    s.tile = 0;
    if (++s.unit == per_b) {
      s.unit = 0;
      do qm_keys(c, ++s.b, s); while (s.tiles == 0);   // (only called where a tile follows)
    }
    s.kvh = (s.unit * team + mate) / c.chunks;
    return true;
  };

  // ---- the ring.  Tile i of this warp into stage i mod S: K's and V's halves of
  // 16 tokens, then their parameters.  Block table entries are looked up one tile
  // ahead, so that they are there when they are needed.  What holds no visible
  // key is not read.
  uint64_t *bars = bars_all + w * S, *free_bars = bars_all + (kQmWarps + w) * S;
  uint8_t *codes = codes_all + w * S * Sh::kCodes, *params = params_all + w * S * 2 * kQmTok * Sh::kParams;
  const uint32_t codes_at = smem_u32(codes), params_at = smem_u32(params);
  const uint64_t policy = l2_evict_first_policy();
  QmAt ahead = cur;
  // TMA: every lane has the halves' entries, one lane asks for their copies; else
  // lane r's rows are token r's.
  int next_phys[kQmHalves], next_off[kQmHalves];
  auto look_up = [&](const QmAt &s) {
#pragma unroll
    for (int h = 0; h < kQmHalves; ++h) {
      const int t = s.base + kQmTok * s.tile + (a.tma ? 16 * h : lane);
      next_off[h] = -1;
      if (a.tma ? t + 16 > s.first && t < s.n : h == 0 && lane < kQmTok && t >= s.first && t < s.n) {
        const int lb = div_by(t, a.bs_mul, a.bs_shift);
        next_off[h] = t - lb * c.bs;
        next_phys[h] = __ldg(c.tables + (size_t)s.b * c.max_blocks + lb);
      }
    }
  };
  auto issue = [&](int i) {
    if (i >= mine) return;
    const int st = i % S;
    bool in[kQmHalves];
#pragma unroll
    for (int h = 0; h < kQmHalves; ++h) {
      in[h] = next_off[h] >= 0;
      if (in[h] && (uint32_t)next_phys[h] >= (uint32_t)c.num_blocks) {   // (num_blocks is below 2^31)
        raise_flag(c.err, PKV_FLAG_BLOCK_OUT_OF_RANGE);
        in[h] = false;
      }
    }
    const uint32_t kvh = (uint32_t)ahead.kvh;
    // (rows of the cache are fewer than 2^32 - 1 here)
    auto number = [&](int h) { return ((uint32_t)next_phys[h] * (uint32_t)c.KVH + kvh) * (uint32_t)c.bs + (uint32_t)next_off[h]; };
    const uint32_t params_to = params_at + (st * 2 * kQmTok + lane) * Sh::kParams;
    if (a.tma) {
      if (lane == 0) {
        int halves = 0;
#pragma unroll
        for (int h = 0; h < kQmHalves; ++h) halves += in[h];
        mbar_arrive_expect_tx(&bars[st], halves * 2 * Sh::kHalf);
#pragma unroll
        for (int h = 0; h < kQmHalves; ++h) {
          if (!in[h]) continue;
          uint8_t *to = codes + st * Sh::kCodes + h * Sh::kHalf;
          tma_load_5d(to, &tmK, &bars[st], 0, next_off[h], 0, (int)kvh, next_phys[h], policy);
          tma_load_5d(to + kQmHalves * Sh::kHalf, &tmV, &bars[st], 0, next_off[h], 0, (int)kvh, next_phys[h], policy);
        }
      }
      __syncwarp();
      // lane r token r's parameters
      const int h = lane / 16;
      if (h == 0 ? in[0] : in[kQmHalves - 1]) {
        const size_t num = (size_t)(h == 0 ? number(0) : number(kQmHalves - 1)) + (lane & 15);
        cp_async_small<Sh::kParams>(params_to, a.kp + num * quant_params<FMT>(), Sh::kParams);
        cp_async_small<Sh::kParams>(params_to + kQmTok * Sh::kParams, a.vp + num * quant_params<FMT>(), Sh::kParams);
      }
    } else {
      const uint32_t row = in[0] ? ((uint32_t)next_phys[0] * (uint32_t)c.bs + (uint32_t)next_off[0]) * (uint32_t)c.KVH + kvh : 0xffffffffu;
      if (in[0]) {
        const size_t num = (size_t)number(0) * quant_params<FMT>();
        cp_async_small<Sh::kParams>(params_to, a.kp + num, Sh::kParams);
        cp_async_small<Sh::kParams>(params_to + kQmTok * Sh::kParams, a.vp + num, Sh::kParams);
      }
#pragma unroll
      for (int j = 0; j < (kQmTok * Sh::kChunks + 31) / 32; ++j) {
        const int idx = lane + 32 * j, r = idx / Sh::kChunks, ch = idx - r * Sh::kChunks;
        const uint32_t from = __shfl_sync(0xffffffffu, row, r & 31);
        if (r < kQmTok && from != 0xffffffffu) {
          const uint32_t to = codes_at + st * Sh::kCodes + (r >> 4) * Sh::kHalf + qm_at<Sh::kRow, Sh::kBox, Sh::kSwizzle>(r & 15, ch);
          cp_async16(to, a.k + (size_t)from * Sh::kRow + ch * 16, 16);
          cp_async16(to + kQmHalves * Sh::kHalf, a.v + (size_t)from * Sh::kRow + ch * 16, 16);
        }
      }
    }
    cp_async_arrive(&bars[st]);
    if (i + 1 < mine) {
      advance(ahead);
      look_up(ahead);
    }
  };
  // Two CTAs an SM are launched with 128 registers a thread: the warps that fill
  // the rings leave some of theirs to those that compute.  (Every warp comes here.)
  if (producer) {
    if constexpr (Sh::kCtas == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kQmRegsFill));
    if (mine > 0) look_up(ahead);
    for (int i = 0; i < mine; ++i) {
      if (i >= S && !__all_sync(0xffffffffu, mbar_sleep_bounded(&free_bars[i % S], (i / S - 1) & 1))) {
        // give up, once the copies that were asked for have landed (bounded)
        if (lane == 0) raise_flag(c.err, PKV_FLAG_TIMEOUT);
        for (int k = max(0, i - S); k < i; ++k) mbar_sleep_bounded(&bars[k % S], (k / S) & 1);
        return;
      }
      issue(i);
    }
    // sequences without a visible key
    for (int b = blockIdx.x; b < c.B; b += gridDim.x) {
      QmAt s;
      qm_keys(c, b, s);
      if (s.tiles == 0)
        for (int i = threadIdx.x - 32 * kQmWarps; i < c.H * D / 2; i += 32 * kQmWarps)
          put_two(c.out, (size_t)b * c.H * D + 2 * i, dt, out8, 0.f, 0.f);
    }
    return;
  }
  if constexpr (Sh::kCtas == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kQmRegsCompute));
  if (mine == 0) return;
  // this lane's places in a half: K's row g (and g + 8, half a box further) at
  // chunk j of a box, V's row lane mod 16 at chunk j and, from lane 16 on, j + 1
  constexpr int kPer = Sh::kBox / 16;
  int k_place[kPer], v_place[(kPer + 1) / 2];
#pragma unroll
  for (int j = 0; j < kPer; ++j) k_place[j] = qm_at<Sh::kRow, Sh::kBox, Sh::kSwizzle>(g, j) + 4 * t4;
#pragma unroll
  for (int j = 0; j < (kPer + 1) / 2; ++j)
    v_place[j] = qm_at<Sh::kRow, Sh::kBox, Sh::kSwizzle>(lane & 15, min(2 * j + (lane >> 4), kPer - 1));

  // ---- a unit's state
  // scores in log2 units, or what their cap wants (see chunk_capped: its error
  // does for 16-bit types; chunk_cap)
  const int cap = !(c.cap_log2 > 0.f) ? kCapNone : dt != PKV_F32 && c.cap_log2 <= kCapShort ? kCapUsual : kCapLarge;
  const float score_unit = cap == kCapNone ? c.scale_log2 : cap == kCapUsual ? c.scale_y : 1.f;
  uint32_t qf[kSteps][2];
  float qs[2], o[kSteps][4], m[2], l[2];
  // O's unit is 2^(ve - kUnit): ve the largest exponent of a value's scale so far
  // (fp32's biased one; from 2^-97 on, NaN and infinity aside)
  constexpr int kUnit = 127 + 6;
  int ve;
  // The queries, scaled, as the product's B: column g is a head (or what fp16
  // left of head g - 4).
  auto start = [&]() {
    const int head = ((cur.unit * team + mate) - cur.kvh * c.chunks) * kHeads + (SPLIT ? g & 3 : g);
    const bool has = head < c.G, low = SPLIT && g >= 4;
    // (columns past the last head have a head's row, times 0)
    const size_t row = ((size_t)cur.b * c.H + cur.kvh * c.G + (has ? head : 0)) * D;
    float4 v[kSteps];
    // int4: a lane's eight columns of 32 are those of two steps
    q_fours<kSteps>(c.q, dt, q16, [&](int ks) {
      return row + (FMT == kInt4 ? (ks >> 1) * 32 + 8 * t4 + 4 * (ks & 1) : ks * 16 + 4 * t4);
    }, v);
    float big = 0.f;
#pragma unroll
    for (int ks = 0; ks < kSteps; ++ks) {
      if (!has) v[ks] = make_float4(0.f, 0.f, 0.f, 0.f);
      big = fmaxf(fmaxf(big, fmaxf(fabsf(v[ks].x), fabsf(v[ks].y))), fmaxf(fabsf(v[ks].z), fabsf(v[ks].w)));
    }
    big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
    big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
    // 2^(14 - floor(log2 big)), both ways a normal number; no more than the type's
    // largest (an infinity stays one), no less than 2^-100
    const int ex = min(max((__float_as_int(big) >> 23) - 127, -100), 127);
    const float up = __int_as_float((14 - ex + 127) << 23), down = __int_as_float((ex - 14 + 127) << 23);
    auto part = [&](float x, float y) {
      x *= up;
      y *= up;
      if (low && dt == PKV_F32) {
        x -= __half2float(__float2half_rn(x));
        y -= __half2float(__float2half_rn(y));
      }
      return half2_bits(x, y);
    };
#pragma unroll
    for (int ks = 0; ks < kSteps; ++ks) {
      if constexpr (FMT == kInt4) {          // nibble pairs (i, i + 4): step 0 i = 0, 1, step 1 i = 2, 3
        if (ks & 1) continue;
        const float4 &x = v[ks], &y = v[ks + 1];
        qf[ks][0] = part(x.x, y.x);
        qf[ks][1] = part(x.y, y.y);
        qf[ks + 1][0] = part(x.z, y.z);
        qf[ks + 1][1] = part(x.w, y.w);
      } else if constexpr (FMT == kInt8) {
        qf[ks][0] = part(v[ks].x, v[ks].z);
        qf[ks][1] = part(v[ks].y, v[ks].w);
      } else {
        qf[ks][0] = part(v[ks].x, v[ks].y);
        qf[ks][1] = part(v[ks].z, v[ks].w);
      }
    }
    // this lane's score columns are 2 t4, 2 t4 + 1
    qs[0] = __shfl_sync(0xffffffffu, down, 8 * t4) * score_unit;
    qs[1] = __shfl_sync(0xffffffffu, down, 8 * t4 + 4) * score_unit;
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.f;
    ve = 30;
#pragma unroll
    for (int ks = 0; ks < kSteps; ++ks) o[ks][0] = o[ks][1] = o[ks][2] = o[ks][3] = 0.f;
  };

  // ---- the end of this warp's part of the unit
  float *ws_m = a.states, *ws_l = ws_m + 2 * warps * kHeads, *ws_o = ws_l + 2 * warps * kHeads;
  auto finish = [&]() {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int sh = 4; sh < 32; sh <<= 1) l[e] += __shfl_xor_sync(0xffffffffu, l[e], sh);
    }
    if (SPLIT) {                             // a head's two columns
#pragma unroll
      for (int ks = 0; ks < kSteps; ++ks)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[ks][e] += __shfl_xor_sync(0xffffffffu, o[ks][e], 2);
    }
    const int chunk = (cur.unit * team + mate) - cur.kvh * c.chunks, rows = min(kHeads, c.G - chunk * kHeads);
    const size_t out_row = (size_t)cur.b * c.H + cur.kvh * c.G + chunk * kHeads;
    const long long first = unit0 / share, last = (unit0 + cur.tiles - 1) / share;
    const float unit = exp2f((float)(ve - kUnit));
    // columns of V that tile ks's rows g and g + 8 are (see code_pairs, nibble_pairs)
    auto column = [&](int ks) { return FMT == kInt4 ? (ks >> 1) * 32 + 4 * g + 2 * (ks & 1) : ks * 16 + 2 * g; };
    if (first == last) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int col = 2 * t4 + e;
        if (col >= rows) continue;
        const float inv = unit / l[e];
        put_pairs<kSteps>(c.out, (out_row + col) * D, dt, out8, column, [&](int ks) { return make_float2(o[ks][e] * inv, o[ks][e + 2] * inv); });
      }
      return;
    }
    // place of fragment f (team first + f): its own end, the others' beginning
    auto place = [&](long long f) { return ((2 * (first + f) + (f == 0)) * team + mate) * kHeads; };
    long long f = me - first;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int col = 2 * t4 + e;
      if (col >= rows) continue;
      const size_t at = place(f) + col;
      if (g == 0) {
        __stcg(ws_m + at, m[e]);
        __stcg(ws_l + at, l[e]);
      }
#pragma unroll
      for (int ks = 0; ks < kSteps; ++ks)
        __stcg(reinterpret_cast<float2 *>(ws_o + at * D + column(ks)), make_float2(o[ks][e] * unit, o[ks][e + 2] * unit));
    }
    long long count = last - first + 1, stride = 1;
    for (int level = 0; count > 1; ++level) {
      const long long group = f / kQmFan;
      const int size = (int)min((long long)kQmFan, count - group * kQmFan);
      const long long head = group * kQmFan * stride;       // the group's first fragment
      count = (count + kQmFan - 1) / kQmFan;
      if (size > 1) {
        // (the counter of the group's first warp: no other group of two or more
        // at this level begins there)
        int *counter = c.ws_cnt + kChunkCntFirst + level * warps + (first + head) * team + mate;
        int prev = 0;
        __syncwarp();
        if (lane == 0)
          asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;"
                       : "=r"(prev)
                       : "l"(reinterpret_cast<uint64_t>(counter))
                       : "memory");
        prev = __shfl_sync(0xffffffffu, prev, 0);
        if (prev != size - 1) return;
        if (lane == 0) *counter = 0;         // ready for the next call
        __syncwarp();
        // as many heads at once as registers take: a round trip to L2 for their
        // maxima and sums, then one for every other source
        constexpr int kVec = (D + 127) / 128, kGroup = kHeads * kVec <= 8 ? kHeads : 4, kAhead = 2;
        const size_t to = place(head);
#pragma unroll 1
        for (int h0 = 0; h0 < rows; h0 += kGroup) {
          const size_t from = place(head + min(lane, size - 1) * stride) + h0;
          float wt[kGroup], M[kGroup], L[kGroup];
#pragma unroll
          for (int h = 0; h < kGroup; ++h) {
            wt[h] = lane < size && h0 + h < rows ? __ldcg(ws_m + from + h) : -INFINITY;
            L[h] = lane < size && h0 + h < rows ? __ldcg(ws_l + from + h) : 0.f;
          }
#pragma unroll
          for (int h = 0; h < kGroup; ++h) {
            M[h] = wt[h];
#pragma unroll
            for (int sh = 16; sh > 0; sh >>= 1) M[h] = fmaxf(M[h], __shfl_xor_sync(0xffffffffu, M[h], sh));
            wt[h] = fast_exp2(wt[h] - chunk_ref(M[h]));
            L[h] *= wt[h];
#pragma unroll
            for (int sh = 16; sh > 0; sh >>= 1) L[h] += __shfl_xor_sync(0xffffffffu, L[h], sh);
          }
          float4 acc[kGroup][kVec];
#pragma unroll
          for (int h = 0; h < kGroup; ++h)
#pragma unroll
            for (int k = 0; k < kVec; ++k) acc[h][k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
          for (int j0 = 0; j0 < size; j0 += kAhead) {
            float4 y[kAhead][kGroup][kVec];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
              const float4 *src = reinterpret_cast<const float4 *>(ws_o + (place(head + min(j0 + j, size - 1) * stride) + h0) * D);
#pragma unroll
              for (int h = 0; h < kGroup; ++h)
#pragma unroll
                for (int k = 0; k < kVec; ++k)
                  y[j][h][k] = h0 + h < rows && lane + 32 * k < D / 4 ? __ldcg(src + h * (D / 4) + lane + 32 * k) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
              const bool has = j0 + j < size;
#pragma unroll
              for (int h = 0; h < kGroup; ++h) {
                float x = __shfl_sync(0xffffffffu, wt[h], j0 + j);
                if (!has) continue;
#pragma unroll
                for (int k = 0; k < kVec; ++k) {
                  acc[h][k].x = fmaf(x, y[j][h][k].x, acc[h][k].x);
                  acc[h][k].y = fmaf(x, y[j][h][k].y, acc[h][k].y);
                  acc[h][k].z = fmaf(x, y[j][h][k].z, acc[h][k].z);
                  acc[h][k].w = fmaf(x, y[j][h][k].w, acc[h][k].w);
                }
              }
            }
          }
          __syncwarp();                      // (every lane has read the group's first state)
#pragma unroll
          for (int h = 0; h < kGroup; ++h) {
            if (h0 + h >= rows) break;
            const float inv = 1.f / L[h];
#pragma unroll
            for (int k = 0; k < kVec; ++k) {
              const int d = 4 * (lane + 32 * k);
              if (d >= D) continue;
              const float4 &y = acc[h][k];
              if (count > 1)
                __stcg(reinterpret_cast<float4 *>(ws_o + (to + h0 + h) * D + d), y);
              else
                put_pairs<2>(c.out, (out_row + h0 + h) * D + d, dt, out8, [](int i) { return 2 * i; },
                             [&](int i) { return i == 0 ? make_float2(y.x * inv, y.y * inv) : make_float2(y.z * inv, y.w * inv); });
            }
            if (count > 1 && lane == 0) {
              __stcg(ws_m + to + h0 + h, M[h]);
              __stcg(ws_l + to + h0 + h, L[h]);
            }
          }
        }
      }
      f = group;
      stride *= kQmFan;
    }
  };

  start();
  for (int i = 0; i < mine; ++i) {
    const int st = i % S;
    if (!__all_sync(0xffffffffu, mbar_sleep_bounded(&bars[st], (i / S) & 1))) {
      if (lane == 0) raise_flag(c.err, PKV_FLAG_TIMEOUT);   // (the warp that fills the ring gives up too)
      return;
    }
    const uint32_t kb = codes_at + st * Sh::kCodes, vb = kb + kQmHalves * Sh::kHalf;
    const uint32_t kpb = params_at + st * 2 * kQmTok * Sh::kParams, vpb = kpb + kQmTok * Sh::kParams;
    const int tile0 = cur.base + kQmTok * cur.tile;
    const bool whole = tile0 >= cur.first && tile0 + kQmTok <= cur.n;
    if (!whole) {
      // values that no query sees, and their parameters, become 0: they may be anything
      const int t = tile0 + lane;
      if (lane < kQmTok && !(t >= cur.first && t < cur.n)) {
#pragma unroll
        for (int ch = 0; ch < Sh::kChunks; ++ch)
          st_shared_v4(vb + (lane >> 4) * Sh::kHalf + qm_at<Sh::kRow, Sh::kBox, Sh::kSwizzle>(lane & 15, ch), make_uint4(0, 0, 0, 0));
        float *to = reinterpret_cast<float *>(params + (st * 2 * kQmTok + kQmTok + lane) * Sh::kParams);
#pragma unroll
        for (int k = 0; k < quant_params<FMT>(); ++k) to[k] = 0.f;
      }
      fence_proxy_async_shared();
      __syncwarp();
    }
    float x[kQmHalves][4], sv[kQmHalves][2];
    int ve_new = ve;
#pragma unroll
    for (int mt = 0; mt < kQmHalves; ++mt) {
      const int r0 = mt * 16 + g, r1 = r0 + 8;
      float s[2][4] = {};                                // (two chains)
      const uint32_t kh = kb + mt * Sh::kHalf;
      auto k_word = [&](int ch, int up) {                // chunk ch of row g (+ 8)
        return lds32(kh + ch / kPer * (16 * Sh::kBox) + up * 8 * Sh::kBox + k_place[ch % kPer]);
      };
      if constexpr (FMT == kInt4) {
        const uint32_t z0 = half2_bits(lds_f32(kpb + r0 * 8 + 4), 0.f) & 0xffffu, z1 = half2_bits(lds_f32(kpb + r1 * 8 + 4), 0.f) & 0xffffu;
        const uint32_t zz0 = z0 | (z0 << 16), zz1 = z1 | (z1 << 16);
        const uint32_t a1 = hfma2_u(zz0, 0x3c003c00u, 0x64006400u), b1 = hfma2_u(zz1, 0x3c003c00u, 0x64006400u);   // 1024 + z
        const uint32_t a16 = hfma2_u(zz0, 0xbc00bc00u, 0xd400d400u), b16 = hfma2_u(zz1, 0xbc00bc00u, 0xd400d400u); // -64 - z
#pragma unroll
        for (int k2 = 0; k2 < D / 32; ++k2) {
          uint32_t f0[4], f1[4];
          nibble_pairs(k_word(k2, 0), a1, a16, f0);
          nibble_pairs(k_word(k2, 1), b1, b16, f1);
          const uint32_t A[4] = {f0[0], f1[0], f0[1], f1[1]}, B[4] = {f0[2], f1[2], f0[3], f1[3]};
          MmaOp<__half>::run(s[0], A, qf[2 * k2][0], qf[2 * k2][1]);
          MmaOp<__half>::run(s[1], B, qf[2 * k2 + 1][0], qf[2 * k2 + 1][1]);
        }
      } else {
#pragma unroll
        for (int ks = 0; ks < kSteps; ++ks) {
          uint32_t A[4];
          code_pairs<FMT, false>(k_word(ks, 0), A[0], A[2]);
          code_pairs<FMT, false>(k_word(ks, 1), A[1], A[3]);
          MmaOp<__half>::run(s[ks & 1], A, qf[ks][0], qf[ks][1]);
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
      for (int e = 0; e < 4; ++e) {
        float y = s[0][e] + s[1][e];
        if (SPLIT && dt == PKV_F32) y += __shfl_xor_sync(0xffffffffu, y, 2);
        // (scales first: the codes' product with a large query may pass fp32 where
        // the score does not)
        x[mt][e] = y * (qs[e & 1] * (e < 2 ? sk0 : sk1));
      }
    }
    if (cap != kCapNone) {
#pragma unroll
      for (int mt = 0; mt < kQmHalves; ++mt)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          x[mt][e] = cap == kCapUsual ? chunk_capped(x[mt][e], c.cap_log2) : chunk_cap(c, x[mt][e]);
    }
    if (!whole) {
#pragma unroll
      for (int mt = 0; mt < kQmHalves; ++mt)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const int t = tile0 + mt * 16 + hf * 8 + g;
          if (t >= cur.first && t < cur.n) continue;
          x[mt][2 * hf] = x[mt][2 * hf + 1] = -INFINITY;
        }
    }
    // raise the maxima where a score passes them by 2^8, and O's unit where a
    // value's scale passes it
    const float m0 = m[0] + 8.f, m1 = m[1] + 8.f;
    bool over = ve_new > ve;
#pragma unroll
    for (int mt = 0; mt < kQmHalves; ++mt) over = over || x[mt][0] > m0 || x[mt][1] > m1 || x[mt][2] > m0 || x[mt][3] > m1;
    if (__any_sync(0xffffffffu, over)) {
      ve_new = __reduce_max_sync(0xffffffffu, ve_new);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float top = -INFINITY;
#pragma unroll
        for (int mt = 0; mt < kQmHalves; ++mt) top = fmaxf(top, fmaxf(x[mt][e], x[mt][e + 2]));
#pragma unroll
        for (int sh = 4; sh < 32; sh <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, sh));
        top = fmaxf(top, m[e]);
        const float d = m[e] - chunk_ref(top), f = fast_exp2(d + (float)(ve - ve_new));
        l[e] *= fast_exp2(d);
        m[e] = top;
#pragma unroll
        for (int ks = 0; ks < kSteps; ++ks) {
          o[ks][e] *= f;
          o[ks][e + 2] *= f;
        }
      }
      ve = ve_new;
    }
    const float unit = __int_as_float((127 + kUnit - ve) << 23);    // 2^(kUnit - ve)
    // weights, as the product's B
    uint32_t wb[kQmHalves][2], wl[kQmHalves][2];
    const float r0 = chunk_ref(m[0]), r1 = chunk_ref(m[1]);
#pragma unroll
    for (int mt = 0; mt < kQmHalves; ++mt)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const float p0 = fast_exp2(x[mt][2 * hf] - r0), p1 = fast_exp2(x[mt][2 * hf + 1] - r1);
        const float s1 = sv[mt][hf] * unit, w0 = p0 * s1, w1 = p1 * s1;
        l[0] += p0;
        l[1] += p1;
        __half2 h = __floats2half2_rn(w0, w1);
        const float2 f = __half22float2(h);
        const __half2 lo = __floats2half2_rn(w0 - f.x, w1 - f.y);
        if (SPLIT) {
          if (t4 >= 2) h = lo;
        } else {
          wl[mt][hf] = movm_trans(*reinterpret_cast<const uint32_t *>(&lo));
        }
        wb[mt][hf] = movm_trans(*reinterpret_cast<uint32_t *>(&h));
      }
#pragma unroll
    for (int mt = 0; mt < kQmHalves; ++mt) {
      const uint32_t vh = vb + mt * Sh::kHalf;
      auto product = [&](int ks, const uint32_t (&A)[4]) {
        MmaOp<__half>::run(o[ks], A, wb[mt][0], wb[mt][1]);
        if (!SPLIT) MmaOp<__half>::run(o[ks], A, wl[mt][0], wl[mt][1]);
      };
      uint32_t z1[2], z16[2];                // int4: tokens 2 t4, 2 t4 + 1 (and 8 behind them) of this half tile
      if constexpr (FMT == kInt4) {
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const uint32_t z = half2_bits(lds_f32(vpb + (mt * 16 + 8 * hf + 2 * t4) * 8 + 4),
                                        lds_f32(vpb + (mt * 16 + 8 * hf + 2 * t4 + 1) * 8 + 4));
          z1[hf] = hfma2_u(z, 0x3c003c00u, 0x64006400u);
          z16[hf] = hfma2_u(z, 0xbc00bc00u, 0xd400d400u);
        }
      }
      auto block = [&](int ch, uint32_t w0, uint32_t w1) {        // a chunk's columns of 16 tokens
        if constexpr (FMT == kInt4) {
          uint32_t f0[4], f1[4];
          nibble_pairs(w0, z1[0], z16[0], f0);
          nibble_pairs(w1, z1[1], z16[1], f1);
#pragma unroll
          for (int q2 = 0; q2 < 2; ++q2) {
            const uint32_t A[4] = {f0[2 * q2], f0[2 * q2 + 1], f1[2 * q2], f1[2 * q2 + 1]};
            product(2 * ch + q2, A);
          }
        } else {
          uint32_t A[4];
          code_pairs<FMT, true>(w0, A[0], A[1]);
          code_pairs<FMT, true>(w1, A[2], A[3]);
          product(ch, A);
        }
      };
#pragma unroll
      for (int ch = 0; ch + 1 < Sh::kChunks; ch += 2) {
        uint32_t w0, w1, w2, w3;
        ldsm_x4_trans(vh + ch / kPer * (16 * Sh::kBox) + v_place[ch % kPer / 2], w0, w1, w2, w3);
        block(ch, w0, w1);
        block(ch + 1, w2, w3);
      }
      if constexpr (Sh::kChunks & 1) {               // (one box then; lanes below 16 give the rows)
        uint32_t w0, w1;
        ldsm_x2_trans(vh + v_place[kPer / 2], w0, w1);
        block(Sh::kChunks - 1, w0, w1);
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&free_bars[st]);
    const bool ends = cur.tile + 1 == cur.tiles;
    if (ends || i + 1 == mine) finish();
    if (i + 1 < mine && advance(cur)) {
      unit0 = begin + i + 1;
      start();
    }
  }
}

template <int D, int FMT, bool SPLIT>
static pkv_status launch_qm(const QuantDecodeArgs &a, pkv_dtype dt, cudaStream_t stream) {
  static int configured[64];
  using Sh = QmShape<D, FMT>;
  auto kern = pkv_quant_decode_mma_kernel<D, FMT, SPLIT>;
  if (!allow_smem(kern, Sh::kSmem, configured)) return PKV_ERR_CUDA;
  if constexpr (Sh::kCtas == 2) {
    // the two shares of registers come out of what a CTA is launched with; a build
    // that gave it fewer would wait for them
    static int regs;
    int n = __atomic_load_n(&regs, __ATOMIC_RELAXED);
    if (n == 0) {
      cudaFuncAttributes attr;
      if (cudaFuncGetAttributes(&attr, kern) != cudaSuccess) return PKV_ERR_CUDA;
      n = attr.numRegs;
      __atomic_store_n(&regs, n, __ATOMIC_RELAXED);
    }
    if (n * kQmThreads < (kQmRegsCompute + kQmRegsFill) * (kQmThreads / 2)) return PKV_ERR_UNSUPPORTED;
  }
  CUtensorMap maps[2];
  memset(maps, 0, sizeof maps);
  if (a.tma && (!encode_codes_map(&maps[0], a.k, a.c.num_blocks, a.c.bs, a.c.KVH, Sh::kRow, Sh::kBox) ||
                !encode_codes_map(&maps[1], a.v, a.c.num_blocks, a.c.bs, a.c.KVH, Sh::kRow, Sh::kBox)))
    return PKV_ERR_CUDA;
  kern<<<(unsigned)a.grid, kQmThreads, Sh::kSmem, stream>>>(maps[0], maps[1], a, (int)dt);
  return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

template <int D, int FMT>
static pkv_status launch_qm_d(const QuantDecodeArgs &a, bool split, pkv_dtype dt, cudaStream_t stream) {
  return split ? launch_qm<D, FMT, true>(a, dt, stream) : launch_qm<D, FMT, false>(a, dt, stream);
}

// Every head_dim of a format.
template <int FMT>
static pkv_status launch_qm_f(const QuantDecodeArgs &a, bool split, pkv_dtype dt, cudaStream_t stream) {
  switch (a.c.D) {
    case 64: return launch_qm_d<64, FMT>(a, split, dt, stream);
    case 80:
      if constexpr (FMT != kInt4) return launch_qm_d<80, FMT>(a, split, dt, stream);
      break;
    case 96: return launch_qm_d<96, FMT>(a, split, dt, stream);
    case 128: return launch_qm_d<128, FMT>(a, split, dt, stream);
    case 192: return launch_qm_d<192, FMT>(a, split, dt, stream);
    case 256: return launch_qm_d<256, FMT>(a, split, dt, stream);
  }
  return PKV_ERR_UNSUPPORTED;
}

}  // namespace pkv
