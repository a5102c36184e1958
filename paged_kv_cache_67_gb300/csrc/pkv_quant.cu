// pkv_quant.cu -- new tokens quantised as they are written to a paged cache,
// and cached rows read back as numbers.
//
// A row is one token's head_dim values of one KV head.  Its scale hangs on its
// largest magnitude, so a row is held in registers between the two looks at
// it: a group of L lanes (a power of two) takes the row of K and the row of V
// of one (token, head), VEC elements a lane at a time, finds both extremes
// with log2 L exchanges and writes the codes.  Every element is read once and
// every code written once.  16384 tokens of 8 heads of 128, bf16 to e4m3: 28.8 us,
// 3.5 TB/s, bound by instructions (three issued a cycle: extremes, conversions,
// packing); 32768 tokens read back from int8: 41 us, 4.9 TB/s, waiting for loads.
#include <string.h>

#include "pkv_quant.cuh"

namespace pkv {

constexpr int kQuantThreads = 256;
constexpr float kQuantTiny = 7.888609052210118e-31f;   // 2^-100

// t / d for t < 2^31 by a multiplication: a division costs as much as a row's
// arithmetic.
struct QuantDiv {
  uint32_t mul;
  int shift;
};
static QuantDiv quant_div(uint32_t d) {
  QuantDiv r = {0, 0};
  while ((1ULL << r.shift) < d) ++r.shift;
  r.mul = (uint32_t)((((1ULL << r.shift) - (uint64_t)d) << 32) / d + 1);
  return r;
}
__device__ __forceinline__ uint32_t div_by(uint32_t t, const QuantDiv &d) { return (__umulhi(t, d.mul) + t) >> d.shift; }

// The larger (smaller) of two; NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

struct QuantRowsArgs {
  char *codes[2];          // k, v
  float *params[2];
  char *x[2];              // dense rows (written by the read kernel)
  const int64_t *slots;
  int *err;
  long long T, stride[2], capacity;   // strides in elements
  int bs, KVH, D, lanes, vecs;        // lanes of a group, vectors of a row
  QuantDiv by_kvh, by_bs;             // (rows of a launch are fewer than 2^31)
  int small;                          // slots are, too
};

// 16 bytes, or (fewer) elements at their own alignment.
template <typename T, int VEC>
struct alignas(sizeof(T) * VEC == 16 ? 16 : sizeof(T)) QuantVec {
  T e[VEC];
};
template <int BYTES>
struct __align__(BYTES) QuantBytes {
  uint8_t b[BYTES];
};

template <int FMT, int VEC>
struct QuantCodes {
  static constexpr int kBytes = FMT == kInt4 ? VEC / 2 : VEC;
  using Pack = QuantBytes<kBytes>;
};

// (token, head) of this lane's group; false past the last, for padding and for
// slots past the pool.
__device__ __forceinline__ bool quant_row(const QuantRowsArgs &a, long long &t, int &h, long long &slot, int &at) {
  const uint32_t lane = threadIdx.x & 31, group = lane / a.lanes;     // (a.lanes: a power of two)
  at = (int)(lane - group * a.lanes);
  const uint32_t row = (blockIdx.x * (kQuantThreads / 32) + (threadIdx.x >> 5)) * (32 / a.lanes) + group;
  const uint32_t token = div_by(row, a.by_kvh);
  t = token;
  h = (int)(row - token * a.KVH);
  if (t >= a.T) return false;
  slot = __ldg(a.slots + t);
  if (slot < 0) return false;
  if (slot >= a.capacity) {
    if (h == 0 && at == 0) raise_flag(a.err, PKV_FLAG_SLOT_OUT_OF_RANGE);
    return false;
  }
  return true;
}

template <typename T, int VEC, int NV, int FMT>
__global__ void __launch_bounds__(kQuantThreads) pkv_quant_write_kernel(const __grid_constant__ QuantRowsArgs a) {
  using V = QuantVec<T, VEC>;
  using C = QuantCodes<FMT, VEC>;
  long long t, slot;
  int h, at;
  const bool has = quant_row(a, t, h, slot, at);
  V x[2][NV];
  float lo[2], hi[2];
  // both rows' loads before anything is looked at
#pragma unroll
  for (int s = 0; s < 2; ++s)
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = at + i * a.lanes;
#pragma unroll
      for (int e = 0; e < VEC; ++e) x[s][i].e[e] = from_f32<T>(0.f);
      if (has && v < a.vecs)
        x[s][i] = *(reinterpret_cast<const V *>(reinterpret_cast<const T *>(a.x[s]) + t * a.stride[s] + (long long)h * a.D) + v);
    }
  // lo, hi: the row's ends, 0 among them (int8, e4m3: hi its largest magnitude);
  // NaN where it holds one
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    lo[s] = hi[s] = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float f = to_f32<T>(x[s][i].e[e]);
        if constexpr (FMT == kInt4) {
          lo[s] = min_nan(lo[s], f);
          hi[s] = max_nan(hi[s], f);
        } else {
          hi[s] = max_nan(hi[s], fabsf(f));
        }
      }
  }
  for (int o = a.lanes >> 1; o > 0; o >>= 1) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      if constexpr (FMT == kInt4) lo[s] = min_nan(lo[s], __shfl_xor_sync(0xffffffffu, lo[s], o));
      hi[s] = max_nan(hi[s], __shfl_xor_sync(0xffffffffu, hi[s], o));
    }
  }
  if (!has) return;
  constexpr float kTop = FMT == kInt8 ? 127.f : FMT == kE4m3 ? 448.f : 15.f;
  const long long blk = a.small ? (long long)div_by((uint32_t)slot, a.by_bs) : slot / a.bs;
  const int off = (int)(slot - blk * a.bs);
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const float span = FMT == kInt4 ? hi[s] - lo[s] : hi[s];
    const bool ok = span <= 3.402823466e38f;               // (neither NaN nor infinite)
    const bool fine = ok && span >= kQuantTiny;
    // (reciprocals, as pkv.h defines them: 2^-23 off where quotients would be 2^-24,
    // next to a code's half step of 2^-9 and more; quotients took 16384 tokens to int8
    // from 26.8 to 28.7 us, to e4m3 from 27.6 to 28.8)
    const float inv = fine ? __fmul_rn(__frcp_rn(span), kTop) : 0.f;
    const float scale = fine ? __fmul_rn(span, 1.f / kTop) : ok ? 0.f : __int_as_float(0x7fc00000);
    const int zero = FMT == kInt4 && fine ? rint_product(-lo[s], inv) : 0;
    if (at == 0) {
      float *p = a.params[s] + ((blk * a.KVH + h) * a.bs + off) * quant_params<FMT>();
      if (FMT == kInt4)
        p[0] = scale, p[1] = (float)zero;
      else
        p[0] = scale;
    }
    typename C::Pack *dst = reinterpret_cast<typename C::Pack *>(a.codes[s] + (slot * a.KVH + h) * quant_row_bytes<FMT>(a.D));
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = at + i * a.lanes;
      if (v >= a.vecs) continue;
      typename C::Pack out;
      if (!fine) {                                       // (an infinity times 0 would be NaN)
#pragma unroll
        for (int e = 0; e < C::kBytes; ++e) out.b[e] = 0;
        dst[v] = out;
        continue;
      }
      float f[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) f[e] = to_f32<T>(x[s][i].e[e]);
      if constexpr (FMT == kInt8 && VEC % 4 == 0) {
        // four at a time: a sum's low byte is its code
        uint32_t w[VEC / 4];
#pragma unroll
        for (int e = 0; e < VEC; e += 4) {
          uint32_t b[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) b[k] = __float_as_uint(fmaf(f[e + k], inv, kRintMagic));
          w[e / 4] = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
        }
        memcpy(&out, w, sizeof out);
      } else if constexpr (FMT == kInt8) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) out.b[e] = (uint8_t)rint_product(f[e], inv);
      } else if constexpr (FMT == kE4m3 && VEC % 4 == 0) {
        uint32_t w[VEC / 4];
#pragma unroll
        for (int e = 0; e < VEC; e += 4)
          w[e / 4] = __byte_perm(e4m3x2_from(f[e] * inv, f[e + 1] * inv), e4m3x2_from(f[e + 2] * inv, f[e + 3] * inv), 0x5410);
        memcpy(&out, w, sizeof out);
      } else if constexpr (FMT == kE4m3) {
        if constexpr (VEC == 1) {
          out.b[0] = (uint8_t)e4m3x2_from(f[0] * inv, 0.f);
        } else {
#pragma unroll
          for (int e = 0; e < VEC; e += 2) {
            const uint32_t two = e4m3x2_from(f[e] * inv, f[e + 1] * inv);
            out.b[e] = (uint8_t)two;
            out.b[e + 1] = (uint8_t)(two >> 8);
          }
        }
      } else {
#pragma unroll
        for (int e = 0; e < VEC; e += 2) {
          const int c0 = min(max(rint_product(f[e], inv) + zero, 0), 15);
          const int c1 = min(max(rint_product(f[e + 1], inv) + zero, 0), 15);
          out.b[e / 2] = (uint8_t)(c0 | (c1 << 4));
        }
      }
      dst[v] = out;
    }
  }
}

template <typename T, int VEC, int NV, int FMT>
__global__ void __launch_bounds__(kQuantThreads) pkv_quant_read_kernel(const __grid_constant__ QuantRowsArgs a) {
  using V = QuantVec<T, VEC>;
  using C = QuantCodes<FMT, VEC>;
  long long t, slot;
  int h, at;
  if (!quant_row(a, t, h, slot, at)) return;
  const long long blk = a.small ? (long long)div_by((uint32_t)slot, a.by_bs) : slot / a.bs;
  const int off = (int)(slot - blk * a.bs);
  typename C::Pack in[2][NV];
  float scale[2], zero[2];
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const float *p = a.params[s] + ((blk * a.KVH + h) * a.bs + off) * quant_params<FMT>();
    scale[s] = __ldg(p);
    zero[s] = FMT == kInt4 ? __ldg(p + 1) : 0.f;
    const typename C::Pack *src =
        reinterpret_cast<const typename C::Pack *>(a.codes[s] + (slot * a.KVH + h) * quant_row_bytes<FMT>(a.D));
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (at + i * a.lanes < a.vecs) in[s][i] = src[at + i * a.lanes];
  }
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    V *dst = reinterpret_cast<V *>(reinterpret_cast<T *>(a.x[s]) + t * a.stride[s] + (long long)h * a.D);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = at + i * a.lanes;
      if (v >= a.vecs) continue;
      V out;
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        float c;
        if constexpr (FMT == kInt8)
          c = (float)(int8_t)in[s][i].b[e];
        else if constexpr (FMT == kE4m3)
          c = half2_to_float2(e4m3x2_to_half2(in[s][i].b[e])).x;
        else
          c = (float)((in[s][i].b[e / 2] >> (e & 1 ? 4 : 0)) & 15) - zero[s];
        out.e[e] = from_f32<T>(c * scale[s]);
      }
      dst[v] = out;
    }
  }
}

template <typename T, int VEC, int NV, int FMT>
static pkv_status launch_rows(const QuantRowsArgs &a, bool read, cudaStream_t stream) {
  // fewer than 2^31 rows a launch
  const long long most = 0x40000000LL / a.KVH;
  for (long long t0 = 0; t0 < a.T; t0 += most) {
    QuantRowsArgs b = a;
    b.T = a.T - t0 < most ? a.T - t0 : most;
    b.slots += t0;
    for (int s = 0; s < 2; ++s) b.x[s] += t0 * a.stride[s] * (long long)sizeof(T);
    const long long per_cta = kQuantThreads / a.lanes, blocks = (b.T * a.KVH + per_cta - 1) / per_cta;
    if (read)
      pkv_quant_read_kernel<T, VEC, NV, FMT><<<(unsigned)blocks, kQuantThreads, 0, stream>>>(b);
    else
      pkv_quant_write_kernel<T, VEC, NV, FMT><<<(unsigned)blocks, kQuantThreads, 0, stream>>>(b);
    if (cudaGetLastError() != cudaSuccess) return PKV_ERR_CUDA;
  }
  return PKV_OK;
}

template <typename T, int VEC, int FMT>
static pkv_status launch_rows_v(QuantRowsArgs &a, bool read, cudaStream_t stream) {
  constexpr int kMost = 512 / (32 * VEC);              // vectors of a lane at head_dim 512
  a.vecs = a.D / VEC;
  for (a.lanes = 1; a.lanes < 32 && a.lanes < a.vecs;) a.lanes *= 2;
  return a.vecs <= 32 ? launch_rows<T, VEC, 1, FMT>(a, read, stream) : launch_rows<T, VEC, kMost, FMT>(a, read, stream);
}

// 16-byte vectors of the dense rows where every row start allows them, else
// one element (4 bits: two, a byte of codes) at a time.
template <typename T, int FMT>
static pkv_status launch_rows_t(QuantRowsArgs &a, bool read, cudaStream_t stream) {
  constexpr int kVec = 16 / sizeof(T), kPack = FMT == kInt4 ? kVec / 2 : kVec;
  bool wide = a.D % kVec == 0;
  for (int s = 0; s < 2; ++s)
    wide = wide && reinterpret_cast<uintptr_t>(a.x[s]) % 16 == 0 && a.stride[s] % kVec == 0 &&
           reinterpret_cast<uintptr_t>(a.codes[s]) % kPack == 0;
  if (wide) return launch_rows_v<T, kVec, FMT>(a, read, stream);
  if constexpr (FMT == kInt4) {
    return launch_rows_v<T, 2, FMT>(a, read, stream);
  } else {
    return launch_rows_v<T, 1, FMT>(a, read, stream);
  }
}

template <typename T>
static pkv_status launch_rows_f(QuantRowsArgs &a, pkv_quant_format fmt, bool read, cudaStream_t stream) {
  switch (fmt) {
    case PKV_QUANT_INT8: return launch_rows_t<T, kInt8>(a, read, stream);
    case PKV_QUANT_E4M3: return launch_rows_t<T, kE4m3>(a, read, stream);
    case PKV_QUANT_INT4: return launch_rows_t<T, kInt4>(a, read, stream);
  }
  return PKV_ERR_INVALID_ARG;
}

// Whether rows of `row` bytes, `stride` apart from each other, at x and at y meet
// nowhere (`count` of each: the two halves of one buffer's rows do not).
static bool rows_apart(const void *x, const void *y, int64_t count, size_t row, size_t stride) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(x), b = reinterpret_cast<uintptr_t>(y);
  const size_t off = a < b ? b - a : a - b;
  if (count > 1 && off < (size_t)(count - 1) * stride + row) return off % stride >= row && off % stride <= stride - row;
  return off >= row;
}

// Both calls: `x` is read (write) or written (read).
static pkv_status quant_rows(void *const (&codes)[2], float *const (&params)[2], void *const (&x)[2],
                             const int64_t *slots, int64_t T, const int64_t (&stride)[2], int64_t num_blocks, int bs,
                             int KVH, int D, pkv_quant_format fmt, pkv_dtype dt, bool read, int *err,
                             cudaStream_t stream) {
  if ((fmt != PKV_QUANT_INT8 && fmt != PKV_QUANT_E4M3 && fmt != PKV_QUANT_INT4) ||
      (dt != PKV_F32 && dt != PKV_BF16 && dt != PKV_F16))
    return PKV_ERR_INVALID_ARG;
  if (T < 0 || T > 0x7fffffffLL || num_blocks < 0 || num_blocks > 0x7fffffffLL || bs <= 0 || KVH <= 0 || KVH > 65535 ||
      D <= 0 || (fmt == PKV_QUANT_INT4 && D % 2) || stride[0] < (int64_t)KVH * D || stride[1] < (int64_t)KVH * D)
    return PKV_ERR_INVALID_ARG;
  if (D > 512) return PKV_ERR_UNSUPPORTED;
  if (T == 0) return PKV_OK;
  const size_t el = dt == PKV_F32 ? 4 : 2;
  if (!slots || reinterpret_cast<uintptr_t>(slots) % 8 || reinterpret_cast<uintptr_t>(err) % 4) return PKV_ERR_INVALID_ARG;
  QuantRowsArgs a = {};
  const int64_t rows = num_blocks * bs * KVH;
  ArgRange r[8];
  for (int s = 0; s < 2; ++s) {
    if (!codes[s] || !params[s] || !x[s] || reinterpret_cast<uintptr_t>(x[s]) % el ||
        reinterpret_cast<uintptr_t>(params[s]) % 4)
      return PKV_ERR_INVALID_ARG;
    r[s] = {codes[s], quant_codes_bytes(fmt, rows, D)};
    r[2 + s] = {params[s], quant_params_bytes(fmt, rows)};
    r[4 + s] = {x[s], (size_t)((T - 1) * stride[s] + (int64_t)KVH * D) * el};
    a.codes[s] = static_cast<char *>(codes[s]);
    a.params[s] = params[s];
    a.x[s] = static_cast<char *>(x[s]);
    a.stride[s] = stride[s];
  }
  r[6] = {slots, (size_t)T * sizeof(int64_t)};
  r[7] = {err, sizeof(int)};
  // what is written overlaps nothing else (two dense inputs, and two caches
  // that are only read, may)
  for (int i = 0; i < 8; ++i)
    for (int j = i + 1; j < 8; ++j) {
      const bool wi = read ? i == 4 || i == 5 : i < 4, wj = read ? j == 4 || j == 5 : j < 4;
      if (i == 4 && j == 5 && stride[0] == stride[1] && rows_apart(x[0], x[1], T, (size_t)KVH * D * el, (size_t)stride[0] * el)) continue;
      if ((wi || wj) && overlap(r[i], r[j])) return PKV_ERR_INVALID_ARG;
    }
  a.slots = slots;
  a.err = err;
  a.T = T;
  a.capacity = num_blocks * bs;
  a.bs = bs;
  a.by_kvh = quant_div((uint32_t)KVH);
  a.by_bs = quant_div((uint32_t)bs);
  a.small = a.capacity <= 0x7fffffffLL;
  a.KVH = KVH;
  a.D = D;
  switch (dt) {
    case PKV_F32: return launch_rows_f<float>(a, fmt, read, stream);
    case PKV_BF16: return launch_rows_f<__nv_bfloat16>(a, fmt, read, stream);
    case PKV_F16: return launch_rows_f<__half>(a, fmt, read, stream);
  }
  return PKV_ERR_INVALID_ARG;
}

}  // namespace pkv

using namespace pkv;

extern "C" {

PKV_API pkv_status pkv_quant_write(void *k_codes, void *v_codes, float *k_params, float *v_params, const void *k,
                                   const void *v, const int64_t *slot_mapping, int64_t num_tokens,
                                   int64_t k_token_stride, int64_t v_token_stride, int64_t num_blocks, int block_size,
                                   int num_kv_heads, int head_dim, pkv_quant_format fmt, pkv_dtype dt, int *err_flags,
                                   pkv_stream_t stream) {
  return quant_rows({k_codes, v_codes}, {k_params, v_params}, {const_cast<void *>(k), const_cast<void *>(v)},
                    slot_mapping, num_tokens, {k_token_stride, v_token_stride}, num_blocks, block_size, num_kv_heads,
                    head_dim, fmt, dt, false, err_flags, reinterpret_cast<cudaStream_t>(stream));
}

PKV_API pkv_status pkv_quant_read(void *k_out, void *v_out, const void *k_codes, const void *v_codes,
                                  const float *k_params, const float *v_params, const int64_t *slot_mapping,
                                  int64_t num_tokens, int64_t k_out_stride, int64_t v_out_stride, int64_t num_blocks,
                                  int block_size, int num_kv_heads, int head_dim, pkv_quant_format fmt, pkv_dtype dt,
                                  int *err_flags, pkv_stream_t stream) {
  return quant_rows({const_cast<void *>(k_codes), const_cast<void *>(v_codes)},
                    {const_cast<float *>(k_params), const_cast<float *>(v_params)}, {k_out, v_out}, slot_mapping,
                    num_tokens, {k_out_stride, v_out_stride}, num_blocks, block_size, num_kv_heads, head_dim, fmt, dt,
                    true, err_flags, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
