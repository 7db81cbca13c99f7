// The rows that the encode kernels quantise: one role's [B][Hkv][n_rows][128]
// fp16 array (vqkv_encode), or both roles' rows of a ragged batch as they come
// out of a projection, keys rotated on the way (vqkv_append).
#pragma once

#include <cuda_bf16.h>

#include <type_traits>

#include "common.cuh"
#include "encode_common.cuh"
#include "internal.h"

namespace vqkv {
namespace {

// Where row r belongs.
struct RowPlace {
  int b;       // sequence
  int t;       // cache position, -1: nothing to encode
  int angle;   // position of its rotation (append)
};

// Cosines and sines of a lane's four channels; a rotation by nothing where
// they are not rotated.
struct Turn {
  float4 c, s;
};

// x c + q s in pairs of fp32: the products' errors are exact, so the result is
// the correctly rounded fp32 except where the exact value lies within about
// 2^-20 ulp of a rounding boundary (as in the key transform).  A rounding here
// that depended on the order of operations could change a code.
__device__ __forceinline__ float turned(float x, float c, float q, float s) {
  const float p = __fmul_rn(x, c), r = __fmul_rn(q, s);
  const float pe = __fmaf_rn(x, c, -p), re = __fmaf_rn(q, s, -r);
  const df sum = two_sum(p, r);
  return __fadd_rn(sum.h, __fadd_rn(sum.l, __fadd_rn(pe, re)));
}

// The lane's four values of a row of any type the calls take.
__device__ __forceinline__ uint4 load_four(const char* row, int lane, int dtype) {
  if (dtype == VQKV_DTYPE_F32) return __ldg(reinterpret_cast<const uint4*>(row) + lane);
  const uint2 v = __ldg(reinterpret_cast<const uint2*>(row) + lane);
  return make_uint4(v.x, v.y, 0u, 0u);
}
__device__ __forceinline__ void four_floats(uint4 raw, int dtype, float (&v)[4]) {
  if (dtype == VQKV_DTYPE_F32) {
    v[0] = __uint_as_float(raw.x), v[1] = __uint_as_float(raw.y);
    v[2] = __uint_as_float(raw.z), v[3] = __uint_as_float(raw.w);
  } else if (dtype == VQKV_DTYPE_BF16) {   // the upper halves of the fp32 values
    v[0] = __uint_as_float(raw.x << 16), v[1] = __uint_as_float(raw.x & 0xffff0000u);
    v[2] = __uint_as_float(raw.y << 16), v[3] = __uint_as_float(raw.y & 0xffff0000u);
  } else {
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&raw.x));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&raw.y));
    v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
  }
}

template <bool APPEND>
struct Rows;

template <>
struct Rows<false> {
  using Params = EncodeParams;
  using Raw = uint2;
  const EncodeParams& p;
  const int kvh;
  __device__ __forceinline__ explicit Rows(const EncodeParams& a) : p(a), kvh(blockIdx.y) {}
  // This CTA's number among those that share its (KV head, role)'s rows.
  __device__ __forceinline__ int cta() const { return (int)blockIdx.x; }
  __device__ __forceinline__ int ctas() const { return (int)gridDim.x; }
  __device__ __forceinline__ int count() const { return p.B * p.n_rows; }
  __device__ __forceinline__ int angle(int) const { return 0; }
  __device__ __forceinline__ RowPlace place(int r, int, bool report) {
    const int b = r / p.n_rows, n = r - b * p.n_rows;
    const int t = p.pos[b] + n;
    if (t < 0 || t >= p.cap_len) {
      if (report && p.err) atomicOr(p.err, VQKV_DEVERR_POSITION);
      return {b, -1, 0};
    }
    return {b, t, 0};
  }
  __device__ __forceinline__ const __half* row_ptr(int r) const {
    const int b = r / p.n_rows, n = r - b * p.n_rows;
    return p.x + (((size_t)b * p.Hkv + kvh) * p.n_rows + n) * kHeadDim;
  }
  __device__ __forceinline__ Raw load(int r, int lane) const {
    return *reinterpret_cast<const uint2*>(row_ptr(r) + 4 * lane);
  }
  __device__ __forceinline__ Turn turn(int, int) const { return {}; }
  __device__ __forceinline__ void values(Raw raw, const Turn&, int, float (&v)[4]) const {
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&raw.x));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&raw.y));
    v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
  }
  __device__ __forceinline__ void row(const RowPlace&, int r, int lane, float (&x)[4]) const {
    transform_row(row_ptr(r), p.role == VQKV_ROLE_K ? p.s + (size_t)kvh * kHeadDim : nullptr, lane, x);
  }
};

// Rows are the batch's tokens; those behind the last sequence (and before the
// first) are padding.
template <>
struct Rows<true> {
  using Params = AppendParams;
  using Raw = uint4;
  const AppendParams& a;
  EncodeParams p;          // this CTA's role
  const int kvh;
  const char* x;           // its rows
  long long token_stride;  // bytes
  int b = 0, first = 0, last = 0, pos = 0;   // the sequence of the last row placed: its tokens, its first one's position
  __device__ __forceinline__ explicit Rows(const AppendParams& a_)
      : a(a_), p(a_.both), kvh(blockIdx.y) {
    const int role = (int)blockIdx.x >= a.key_ctas ? VQKV_ROLE_V : VQKV_ROLE_K, bytes = a.dtype == VQKV_DTYPE_F32 ? 4 : 2;
    p.role = role;
    p.s = role == VQKV_ROLE_K ? p.s : nullptr;
    p.cb = a.cb[role];
    p.codes = a.codes[role];
    x = static_cast<const char*>(a.x[role]) + (long long)kvh * a.head_stride[role] * bytes;
    token_stride = a.token_stride[role] * bytes;
  }
  __device__ __forceinline__ int cta() const { return (int)blockIdx.x - (p.role == VQKV_ROLE_V ? a.key_ctas : 0); }
  __device__ __forceinline__ int ctas() const { return p.role == VQKV_ROLE_V ? (int)gridDim.x - a.key_ctas : a.key_ctas; }
  __device__ __forceinline__ int count() const { return a.n_tokens; }
  // Called by whole warps: the sequence is the last one that starts at or
  // before token r, found by 32 probes at a time.  Every index read lies in
  // [0, B] whatever the starts hold.
  // angle: that of token r (its load is a memory latency of its own).
  __device__ __forceinline__ int angle(int r) const { return a.rope_pos != nullptr ? __ldg(a.rope_pos + r) : 0; }
  __device__ __forceinline__ RowPlace place(int r, int angle, bool report) {
    if (!(first <= r && r < last)) {
      const int lane = threadIdx.x & 31;
      int lo = 0, hi = p.B;
      while (hi - lo > 1) {
        const int step = (hi - lo + 31) >> 5, at = lo + lane * step;
        const unsigned below = __ballot_sync(0xffffffffu, at < hi && __ldg(a.row_start + at) <= r);
        if (below) lo += (31 - __clz(below)) * step;
        hi = below ? min(hi, lo + step) : lo + 1;
      }
      b = lo;
      first = __ldg(a.row_start + lo), last = __ldg(a.row_start + lo + 1);
      pos = __ldg(a.pos + lo);
      if (!(first <= r && r < last)) {
        last = first;
        return {b, -1, 0};
      }
    }
    const long long t = (long long)pos + ((long long)r - first);
    const bool in_cache = t >= 0 && t < p.cap_len;
    bool turns = true;
    if (a.table != nullptr) {
      if (a.rope_pos == nullptr) angle = in_cache ? (int)t : 0;
      turns = angle >= 0 && angle < a.n_table;
    }
    if (!in_cache || !turns) {
      if (report && p.err) atomicOr(p.err, VQKV_DEVERR_POSITION);
      return {b, -1, 0};
    }
    return {b, (int)t, angle};
  }
  __device__ __forceinline__ Raw load(int r, int lane) const {
    return load_four(x + r * token_stride, lane, a.dtype);
  }
  __device__ __forceinline__ Turn turn(int angle, int lane) const {
    Turn u{make_float4(1.f, 1.f, 1.f, 1.f), make_float4(0.f, 0.f, 0.f, 0.f)};
    if (a.table == nullptr || p.role != VQKV_ROLE_K || 4 * lane >= a.rot) return u;
    const float* row = a.table + (size_t)angle * a.rot;
    const int half = a.rot >> 1;
    if (a.interleaved) {
      const float2 c = __ldg(reinterpret_cast<const float2*>(row + 2 * lane));
      const float2 s = __ldg(reinterpret_cast<const float2*>(row + half + 2 * lane));
      u.c = make_float4(c.x, c.x, c.y, c.y);
      u.s = make_float4(-s.x, s.x, -s.y, s.y);
    } else {
      const bool upper = 4 * lane >= half;
      const int i = 4 * lane - (upper ? half : 0);
      u.c = __ldg(reinterpret_cast<const float4*>(row + i));
      u.s = __ldg(reinterpret_cast<const float4*>(row + half + i));
      if (!upper) u.s = make_float4(-u.s.x, -u.s.y, -u.s.z, -u.s.w);
    }
    return u;
  }
  __device__ __forceinline__ void rotate(float (&v)[4], const Turn& u, int lane) const {
    float q[4];
    if (a.interleaved) {
      q[0] = v[1], q[1] = v[0], q[2] = v[3], q[3] = v[2];
    } else {   // the other half's lane
      const int eighth = a.rot >> 3, other = lane < eighth ? lane + eighth : lane < 2 * eighth ? lane - eighth : lane;
#pragma unroll
      for (int i = 0; i < 4; ++i) q[i] = __shfl_sync(0xffffffffu, v[i], other);
    }
    if (4 * lane < a.rot) {
      v[0] = turned(v[0], u.c.x, q[0], u.s.x), v[1] = turned(v[1], u.c.y, q[1], u.s.y);
      v[2] = turned(v[2], u.c.z, q[2], u.s.z), v[3] = turned(v[3], u.c.w, q[3], u.s.w);
    }
  }
  // A row's values as they are encoded: a key's after its rotation.
  __device__ __forceinline__ void values(Raw raw, const Turn& u, int lane, float (&v)[4]) const {
    four_floats(raw, a.dtype, v);
    if (p.role == VQKV_ROLE_K && a.table != nullptr) rotate(v, u, lane);
  }
  __device__ __forceinline__ void transform(Raw raw, const Turn& u, float4 s, float4 rs, int lane, float (&x)[4]) const {
    values(raw, u, lane, x);
    if (p.role != VQKV_ROLE_K) return;
    const float v[4] = {x[0], x[1], x[2], x[3]};
    transform_key_values(v, s, rs, lane, x);
  }
  __device__ __forceinline__ void row(const RowPlace& w, int r, int lane, float (&x)[4]) const {
    const Raw raw = load(r, lane);
    const Turn u = turn(w.angle, lane);
    float4 s = make_float4(1.f, 1.f, 1.f, 1.f);
    if (p.role == VQKV_ROLE_K) s = __ldg(reinterpret_cast<const float4*>(p.s + (size_t)kvh * kHeadDim + 4 * lane));
    transform(raw, u, s, make_float4(__frcp_rn(s.x), __frcp_rn(s.y), __frcp_rn(s.z), __frcp_rn(s.w)), lane, x);
  }
};

}  // namespace
}  // namespace vqkv
