// Query transform and centroid-gather helpers shared by the attention kernels
// over packed codes (decode.cu, decode_tree.cu).
#pragma once

#include "common.cuh"
#include "internal.h"

namespace vqkv {
namespace {

// The lane's 4 channels of query column col0 + warp (query c / g, head
// c % g) and their smoothing factors, for warps 0..nloc-1.
struct QueryLoad {
  uint2 q;
  float4 s;
};
__device__ __forceinline__ QueryLoad load_query(const DecodeParams& p, int b, int kvh, int warp, int lane, int col0,
                                                int nloc) {
  QueryLoad r{make_uint2(0u, 0u), make_float4(0.f, 0.f, 0.f, 0.f)};
  if (warp < nloc) {
    const int c = col0 + warp;
    const int m = c / p.g, hq = kvh * p.g + c - m * p.g;
    r.q = *reinterpret_cast<const uint2*>(p.q + (((size_t)b * p.M + m) * p.Hq + hq) * kHeadDim + 4 * lane);
    r.s = *reinterpret_cast<const float4*>(p.s + (size_t)kvh * kHeadDim + 4 * lane);
  }
  return r;
}

// q' of the CTA's softmax column col0 + warp into row `warp` of s_qp (fp32,
// scaled, rows `pitch` floats apart), by warps 0..nloc-1.
__device__ __forceinline__ void transform_query(const DecodeParams& p, const QueryLoad& r, int warp, int lane,
                                                float* s_qp, int pitch, int nloc) {
  if (warp < nloc) {
    const __half2 q01 = *reinterpret_cast<const __half2*>(&r.q.x);
    const __half2 q23 = *reinterpret_cast<const __half2*>(&r.q.y);
    float v[4] = {__low2float(q01) * r.s.x, __high2float(q01) * r.s.y, __low2float(q23) * r.s.z,
                  __high2float(q23) * r.s.w};
    fwht128_f32(v, lane);
    float4 o = make_float4(v[0] * p.qscale, v[1] * p.qscale, v[2] * p.qscale, v[3] * p.qscale);
    *reinterpret_cast<float4*>(s_qp + warp * pitch + 4 * lane) = o;
  }
}

// Shared-memory offset of a gathered centroid: one byte permute puts code
// byte K of `codes` into bits 8..15 and the lane's replica offset (byte 0 of
// `lane_byte`) into bits 0..7: (code << 8) | replica offset.
template <int K>
__device__ __forceinline__ uint32_t cb_offset(uint32_t codes, uint32_t lane_byte) {
  return __byte_perm(codes, lane_byte, 0x5504 | (K << 4));
}

template <typename T>
__device__ __forceinline__ T lds_at(const unsigned char* base, uint32_t off) {
  return *reinterpret_cast<const T*>(base + off);
}

// 24-bit code pair at byte b (a multiple of 3) of a lane's run of words.
template <int LW>
__device__ __forceinline__ uint32_t pair_at(const uint32_t (&w)[LW], int b) {
  const int i = b >> 2, sh = (b & 3) * 8;
  return (sh <= 8 ? (w[i] >> sh) : __funnelshift_r(w[i], w[i + 1], sh)) & 0xffffffu;
}

// 10-bit code at bit b of a lane's run words (b is a constant after
// unrolling, so the word indices are too).
template <int N>
__device__ __forceinline__ uint32_t bits10(const uint32_t (&w)[N], int b) {
  const int i = b >> 5, sh = b & 31;
  return (i + 1 < N ? __funnelshift_r(w[i], w[i + 1], sh) : w[i] >> sh) & 0x3ffu;
}

// Byte offset of centroid c in copy `rep` of a 1024-entry codebook whose four
// copies are interleaved in 128-byte rows: copy r holds its even / odd
// entries in 16-byte bank groups 2r / 2r+1.
__device__ __forceinline__ uint32_t cb10_offset(uint32_t c) { return ((c >> 1) << 7) | ((c & 1u) << 4); }

// 24-bit code pair k (bytes 3k..3k+2) of a lane's 12-byte run (3 words).
__device__ __forceinline__ uint32_t pair24(uint32_t w0, uint32_t w1, uint32_t w2, int k) {
  if (k == 0) return w0 & 0xffffffu;
  if (k == 1) return __funnelshift_r(w0, w1, 24) & 0xffffffu;
  if (k == 2) return __funnelshift_r(w1, w2, 16) & 0xffffffu;
  return w2 >> 8;
}

}  // namespace
}  // namespace vqkv
