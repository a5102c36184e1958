// pkv_rope_write.cu -- rotary positions over several axes, fused with the
// paged write: q rotated into q_out, k rotated into the cache, v copied there.
//
// Pair j of a head, (x, y), turns by the angle of position pos[axis(j)]:
//   (x, y) -> (x c - y s, y c + x s),   c, s = cos_sin[pos][j], [pairs + j]
// in fp32, rounded once.  Every element is read once and written once, so
// memory bounds it; what it must not do is read the angle table (8 bytes a
// pair, more than the 4 bytes of a 16-bit pair itself) once per head.
//
// So a lane keeps to one unit of a head -- VEC pairs, two vectors of VEC
// elements: columns j and j + pairs, or 2 VEC neighbours when interleaved --
// with its cosines and sines in registers, and runs over the token's heads.
// A warp's lanes cover 32 / U heads of U units side by side (coalesced), a
// token is shared by `wpt` warps.  The columns behind rot_dim are units that
// copy, the value heads are copied by every unit.
#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {

constexpr int kRopeWarps = 4;
constexpr int kRopeMaxPairs = 256;

struct RopeArgs {
  char *q_out, *kc, *vc;
  const char *q, *k, *v;
  const float *cos_sin;
  const int32_t *pos;
  const int64_t *slots;
  int *err;
  long long T, q_stride, k_stride, v_stride, pos_stride;  // strides in elements
  long long max_pos, capacity;
  int axes, H, KVH, D, pairs, interleaved;
  int wpt;                              // warps per token
  int stream;                           // the stores outrun L2
  uint32_t used_axes;                   // axes that turn a pair
  int quads;                            // the table's four-pair groups can be read as vectors
  uint32_t axis2[kRopeMaxPairs / 16];   // axis of pair j: two bits
};

template <typename T, int VEC>
struct __align__(sizeof(T) * VEC) RopeVec {
  T e[VEC];
};

// A vector's store; with `stream` marked as read by nobody soon (st.cs).
template <typename T, int VEC>
__device__ __forceinline__ void rope_store(T *dst, const RopeVec<T, VEC> &v, int stream) {
  constexpr int kBytes = sizeof(T) * VEC;
  if (kBytes == 16 && stream) {
    const uint4 u = *reinterpret_cast<const uint4 *>(&v);
    __stcs(reinterpret_cast<uint4 *>(dst), u);
  } else {
    *reinterpret_cast<RopeVec<T, VEC> *>(dst) = v;
  }
}

template <typename T, int VEC>
__global__ void __launch_bounds__(32 * kRopeWarps) pkv_rope_write_kernel(const __grid_constant__ RopeArgs a) {
  using V = RopeVec<T, VEC>;
  const int lane = threadIdx.x & 31;
  const long long gw = (long long)blockIdx.x * kRopeWarps + (threadIdx.x >> 5);
  const long long t = gw / a.wpt;
  const int part = (int)(gw - t * a.wpt);
  if (t >= a.T) return;
  // slot, positions and the first heads' vectors are independent loads: all in
  // flight before the first is looked at
  const long long slot = __ldg(a.slots + t);
  int pos[4] = {0, 0, 0, 0};
#pragma unroll
  for (int ax = 0; ax < 4; ++ax)
    if (ax < a.axes) pos[ax] = __ldg(a.pos + ax * a.pos_stride + t);
  const int pairs = a.pairs, D = a.D;
  const int rot_units = pairs / VEC;
  const int units = rot_units + (D - 2 * pairs + 2 * VEC - 1) / (2 * VEC);
  const int hpw = units >= 32 ? 1 : 32 / units;           // heads side by side in a warp
  const int hl = units >= 32 ? 0 : lane / units;
  const int heads = a.H + 2 * a.KVH;
  const T *qs = reinterpret_cast<const T *>(a.q) + t * a.q_stride;
  const T *ks = reinterpret_cast<const T *>(a.k) + t * a.k_stride;
  const T *vs = reinterpret_cast<const T *>(a.v) + t * a.v_stride;
  const bool in_pool = slot < a.capacity;
  const int hstep = a.wpt * hpw;

  for (int u0 = 0; u0 < units; u0 += 32) {                // one pass unless a head has more than 32 units
    const int unit = units >= 32 ? u0 + lane : lane - hl * units;
    const bool has = hl < hpw && unit < units;
    const bool turns = unit < rot_units;
    int e0, e1;                                           // the unit's two vectors
    if (turns) {
      e0 = a.interleaved ? 2 * unit * VEC : unit * VEC;
      e1 = a.interleaved ? e0 + VEC : pairs + unit * VEC;
    } else {
      e0 = 2 * pairs + (unit - rot_units) * 2 * VEC;
      e1 = e0 + VEC;
    }
    const bool second = e1 < D;
    V x, y;
    auto load = [&](int h) {
      if (has && h < heads) {
        const T *src = h < a.H ? qs + h * D : h < a.H + a.KVH ? ks + (h - a.H) * D : vs + (h - a.H - a.KVH) * D;
        x = *reinterpret_cast<const V *>(src + e0);
        if (second) y = *reinterpret_cast<const V *>(src + e1);
      }
    };
    int h = part * hpw + hl;
    load(h);
    if (u0 == 0) {
      if (slot < 0) return;                               // padding token
      bool ok = true;
#pragma unroll
      for (int ax = 0; ax < 4; ++ax)
        if ((a.used_axes >> ax) & 1) ok = ok && pos[ax] >= 0 && pos[ax] < a.max_pos;
      if (!ok) {
        if (lane == 0 && part == 0) raise_flag(a.err, PKV_FLAG_POSITION);
        return;
      }
      if (!in_pool && lane == 0 && part == 0) raise_flag(a.err, PKV_FLAG_SLOT_OUT_OF_RANGE);
    }
    if (!has) continue;
    T *qd = reinterpret_cast<T *>(a.q_out) + t * (long long)a.H * D;
    T *kd = reinterpret_cast<T *>(a.kc) + (in_pool ? slot : 0) * (long long)a.KVH * D;
    T *vd = reinterpret_cast<T *>(a.vc) + (in_pool ? slot : 0) * (long long)a.KVH * D;
    float c[VEC], s[VEC];
    if (turns) {
      auto row_of = [&](int j) {
        const int ax = (a.axis2[j >> 4] >> (2 * (j & 15))) & 3;
        const int p = ax == 0 ? pos[0] : ax == 1 ? pos[1] : ax == 2 ? pos[2] : pos[3];
        return a.cos_sin + (long long)p * (2 * pairs) + j;
      };
      if (VEC % 4 == 0 && a.quads) {                      // four pairs of one axis: one load
#pragma unroll
        for (int i = 0; i < VEC / 4; ++i) {
          const float *row = row_of(unit * VEC + 4 * i);
          const float4 cv = __ldg(reinterpret_cast<const float4 *>(row));
          const float4 sv = __ldg(reinterpret_cast<const float4 *>(row + pairs));
          c[4 * i] = cv.x; c[4 * i + 1] = cv.y; c[4 * i + 2] = cv.z; c[4 * i + 3] = cv.w;
          s[4 * i] = sv.x; s[4 * i + 1] = sv.y; s[4 * i + 2] = sv.z; s[4 * i + 3] = sv.w;
        }
      } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const float *row = row_of(unit * VEC + i);
          c[i] = __ldg(row);
          s[i] = __ldg(row + pairs);
        }
      }
    }
    // one head at a time: more loads in flight a lane cost registers and with
    // them warps (two heads 93 us, four 103, one 77 at 16384 tokens of 32 + 8
    // + 8 heads of 128)
    for (; h < heads; h += hstep) {
      if (h != part * hpw + hl) load(h);
      if (h >= a.H && !in_pool) continue;
      T *dst = h < a.H ? qd + h * D : h < a.H + a.KVH ? kd + (h - a.H) * D : vd + (h - a.H - a.KVH) * D;
      if (turns && h < a.H + a.KVH) {
        float fx[VEC], fy[VEC];
#pragma unroll
        for (int n = 0; n < VEC; ++n) {
          fx[n] = to_f32<T>(x.e[n]);
          fy[n] = to_f32<T>(y.e[n]);
        }
        if (a.interleaved) {                              // pairs are neighbours: x holds the first VEC / 2 of them
          float z[2 * VEC];
#pragma unroll
          for (int n = 0; n < VEC; ++n) {
            z[n] = fx[n];
            z[VEC + n] = fy[n];
          }
#pragma unroll
          for (int n = 0; n < VEC; ++n) {
            const float p = z[2 * n], q = z[2 * n + 1];
            z[2 * n] = fmaf(p, c[n], -(q * s[n]));
            z[2 * n + 1] = fmaf(q, c[n], p * s[n]);
          }
#pragma unroll
          for (int n = 0; n < VEC; ++n) {
            x.e[n] = from_f32<T>(z[n]);
            y.e[n] = from_f32<T>(z[VEC + n]);
          }
        } else {
#pragma unroll
          for (int n = 0; n < VEC; ++n) {
            x.e[n] = from_f32<T>(fmaf(fx[n], c[n], -(fy[n] * s[n])));
            y.e[n] = from_f32<T>(fmaf(fy[n], c[n], fx[n] * s[n]));
          }
        }
      }
      rope_store(dst + e0, x, a.stream);
      if (second) rope_store(dst + e1, y, a.stream);
    }
  }
}

// Widest vector (elements) that every row start, stride and unit edge allows.
static int rope_vec(const RopeArgs &a, int el) {
  const long long strides[] = {a.q_stride, a.k_stride, a.v_stride};
  const void *ptrs[] = {a.q_out, a.kc, a.vc, a.q, a.k, a.v};
  for (int vec = 16 / el; vec > 1; vec >>= 1) {
    if (a.D % vec || a.pairs % vec) continue;
    bool ok = true;
    for (long long s : strides) ok = ok && s % vec == 0;
    for (const void *p : ptrs) ok = ok && reinterpret_cast<uintptr_t>(p) % (vec * el) == 0;
    if (ok) return vec;
  }
  return 1;
}

template <typename T, int VEC>
static pkv_status launch_rope_v(RopeArgs &a, cudaStream_t stream) {
  const int units = a.pairs / VEC + (a.D - 2 * a.pairs + 2 * VEC - 1) / (2 * VEC);
  const int hpw = units >= 32 ? 1 : 32 / units;
  const int groups = (a.H + 2 * a.KVH + hpw - 1) / hpw;   // warp-wide groups of heads of a token
  // few tokens: spread a token's heads over warps until the GPU holds about
  // 16 warps an SM (152 SMs, those of the one GPU this library is built for;
  // another count costs speed alone); many: one warp walks all heads and reads
  // its angles once
  const long long want = (152LL * 16 + a.T - 1) / a.T;
  // what is written stays in L2 for the attention that reads it next, unless
  // it could not (402 MB of rows: 72 us with streaming stores, 77 without)
  a.stream = a.T * (a.H + 2LL * a.KVH) * a.D * (long long)sizeof(T) > (64LL << 20);
  a.wpt = (int)(want < 1 ? 1 : want > groups ? groups : want);
  const long long blocks = (a.T * a.wpt + kRopeWarps - 1) / kRopeWarps;
  if (blocks > 0x7fffffffLL) return PKV_ERR_UNSUPPORTED;
  pkv_rope_write_kernel<T, VEC><<<(unsigned)blocks, 32 * kRopeWarps, 0, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

template <typename T>
static pkv_status launch_rope_t(RopeArgs &a, cudaStream_t stream) {
  switch (rope_vec(a, (int)sizeof(T))) {
    case 8:
      if constexpr (sizeof(T) == 2) return launch_rope_v<T, 8>(a, stream);
    case 4: return launch_rope_v<T, 4>(a, stream);
    case 2: return launch_rope_v<T, 2>(a, stream);
  }
  return launch_rope_v<T, 1>(a, stream);
}

}  // namespace pkv

using namespace pkv;

extern "C" PKV_API pkv_status pkv_rope_write(
    void *q_out, void *k_cache, void *v_cache, const void *q, const void *k, const void *v,
    const float *cos_sin, const int32_t *positions, const uint8_t *pair_axis,
    const int64_t *slot_mapping, int64_t num_tokens, int64_t q_token_stride,
    int64_t k_token_stride, int64_t v_token_stride, int64_t positions_stride, int num_axes, int H,
    int num_kv_heads, int head_dim, int rot_dim, int interleaved, int64_t max_position,
    int64_t num_blocks, int block_size, pkv_dtype dt, int *err_flags, pkv_stream_t stream) {
  if (dt != PKV_F32 && dt != PKV_BF16 && dt != PKV_F16) return PKV_ERR_INVALID_ARG;
  if (num_tokens < 0 || num_tokens > 0x7fffffffLL || num_blocks < 0 || num_blocks > 0x7fffffffLL ||
      block_size <= 0 || H <= 0 || H > 65535 || num_kv_heads <= 0 || num_kv_heads > 65535 ||
      head_dim <= 0 || rot_dim < 0 || rot_dim > head_dim || rot_dim % 2 || num_axes < 1 ||
      num_axes > 4 || max_position < 0 || positions_stride < 0 ||
      (num_axes > 1 && positions_stride > 0 && positions_stride < num_tokens))
    return PKV_ERR_INVALID_ARG;
  if (head_dim > 512) return PKV_ERR_UNSUPPORTED;
  if (q_token_stride < (int64_t)H * head_dim || k_token_stride < (int64_t)num_kv_heads * head_dim ||
      v_token_stride < (int64_t)num_kv_heads * head_dim ||
      (q_out == q && q_token_stride != (int64_t)H * head_dim))
    return PKV_ERR_INVALID_ARG;
  RopeArgs a = {};
  a.quads = rot_dim % 8 == 0 && reinterpret_cast<uintptr_t>(cos_sin) % 16 == 0;
  for (int j = 0; j < rot_dim / 2; ++j) {
    const int axis = pair_axis ? pair_axis[j] : 0;
    if (axis >= num_axes) return PKV_ERR_INVALID_ARG;
    a.axis2[j >> 4] |= (uint32_t)axis << (2 * (j & 15));
    a.used_axes |= 1u << axis;
    if (pair_axis && axis != pair_axis[j & ~3]) a.quads = 0;   // a group over two axes
  }
  if (num_tokens == 0) return PKV_OK;
  if (!q_out || !k_cache || !v_cache || !q || !k || !v || !positions || !slot_mapping ||
      (rot_dim > 0 && !cos_sin))
    return PKV_ERR_INVALID_ARG;
  const uintptr_t el = dt == PKV_F32 ? 4 : 2;
  // (rows that lie between another tensor's rows would do, but no caller has them)
  auto rows = [&](const void *p, int64_t stride, int64_t row) { return ArgRange{p, (size_t)((num_tokens - 1) * stride + row) * el}; };
  const int64_t q_row = (int64_t)H * head_dim, kv_row = (int64_t)num_kv_heads * head_dim;
  const size_t cache = (size_t)num_blocks * block_size * kv_row * el;
  const ArgRange out = rows(q_out, q_row, q_row), kc = {k_cache, cache}, vc = {v_cache, cache};
  const ArgRange others[] = {rows(k, k_token_stride, kv_row), rows(v, v_token_stride, kv_row), kc, vc,
                             {cos_sin, (size_t)max_position * rot_dim * sizeof(float)},
                             {positions, (size_t)((num_axes - 1) * positions_stride + num_tokens) * sizeof(int32_t)},
                             {slot_mapping, (size_t)num_tokens * sizeof(int64_t)}};
  for (const ArgRange &x : others)
    if (overlap(out, x)) return PKV_ERR_INVALID_ARG;
  if ((q_out != q && overlap(out, rows(q, q_token_stride, q_row))) || overlap(kc, vc)) return PKV_ERR_INVALID_ARG;
  const void *ptrs[] = {q_out, k_cache, v_cache, q, k, v};
  for (const void *p : ptrs)
    if (reinterpret_cast<uintptr_t>(p) % el) return PKV_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(cos_sin) % 4 || reinterpret_cast<uintptr_t>(positions) % 4 ||
      reinterpret_cast<uintptr_t>(err_flags) % 4 || reinterpret_cast<uintptr_t>(slot_mapping) % 8)
    return PKV_ERR_INVALID_ARG;
  a.q_out = static_cast<char *>(q_out);
  a.kc = static_cast<char *>(k_cache);
  a.vc = static_cast<char *>(v_cache);
  a.q = static_cast<const char *>(q);
  a.k = static_cast<const char *>(k);
  a.v = static_cast<const char *>(v);
  a.cos_sin = cos_sin;
  a.pos = positions;
  a.slots = slot_mapping;
  a.err = err_flags;
  a.T = num_tokens;
  a.q_stride = q_token_stride;
  a.k_stride = k_token_stride;
  a.v_stride = v_token_stride;
  a.pos_stride = positions_stride;
  a.max_pos = max_position;
  a.capacity = num_blocks * block_size;
  a.axes = num_axes;
  a.H = H;
  a.KVH = num_kv_heads;
  a.D = head_dim;
  a.pairs = rot_dim / 2;
  a.interleaved = interleaved != 0;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  switch (dt) {
    case PKV_F32: return launch_rope_t<float>(a, s);
    case PKV_BF16: return launch_rope_t<__nv_bfloat16>(a, s);
    case PKV_F16: return launch_rope_t<__half>(a, s);
  }
  return PKV_ERR_INVALID_ARG;
}
