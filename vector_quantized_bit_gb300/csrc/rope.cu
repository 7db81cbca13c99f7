// Rotary positions for sm_103a: the table of cosines and sines, and the rotation
// of query or key rows (the pages leave rotary positions outside the method;
// models rotate queries and keys before the cache sees them).
#include <cuda_bf16.h>

#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace vqkv {
namespace {

// ------------------------------------------------------------------ table
// Row p holds cos(p f_i) for i < rot / 2, then sin(p f_i), times an amplitude.
// The angle in turns is p * f_i / 2 pi; its whole turns do not matter, so with
// f_i / 2 pi as a 64-bit fraction the 64-bit product's overflow is the range
// reduction: exact for any 32-bit p but for the fraction's own rounding (2^-65
// turns times p).  The nearest quarter turn is split off and the rest, at most
// an eighth of a turn, goes to sincospif as a number of 24 bits or more.
// One thread: four pairs of one position, two 16-byte stores.
__global__ void __launch_bounds__(256) rope_table_kernel(const __grid_constant__ RopeTableParams p) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int quads = p.rot >> 3;   // four-pair pieces of a row
  const long long pieces = (long long)p.n_pos * quads;
  for (long long k = (long long)blockIdx.x * 256 + threadIdx.x; k < pieces; k += (long long)gridDim.x * 256) {
    const int pos = (int)(k / quads), i = 4 * (int)(k - (long long)pos * quads);
    float c[4], s[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const unsigned long long turn = p.step[i + j] * (unsigned long long)pos;
      const unsigned top = (unsigned)((turn + (1ull << 31)) >> 32);          // turns in units of 2^-32
      const unsigned quarter = (top + (1u << 29)) >> 30;
      const float rest = (float)(int)(top - (quarter << 30)) * 4.656612873077393e-10f;   // half turns: 2^-31 each
      float a, b;
      sincospif(rest, &a, &b);
      const float y = quarter & 1 ? b : a, x = quarter & 1 ? a : b;           // quarter turns swap and negate
      s[j] = (quarter & 2 ? -y : y) * p.amplitude;
      c[j] = ((quarter + 1) & 2 ? -x : x) * p.amplitude;
    }
    float* row = p.table + (size_t)pos * p.rot + i;
    *reinterpret_cast<float4*>(row) = make_float4(c[0], c[1], c[2], c[3]);
    *reinterpret_cast<float4*>(row + (p.rot >> 1)) = make_float4(s[0], s[1], s[2], s[3]);
  }
}

// ------------------------------------------------------------------ rotation
// (y_i, z_i) = (a c - b s, b c + a s) over the row's pairs.  A row is 16 pieces of
// two four-channel halves: a piece u below rot / 8 holds pairs 4u .. 4u + 3 (both
// members, so no thread needs another's channels, and the rotation may be in
// place), the others channels that pass through.  A thread keeps one piece's
// cosines and sines and takes it in ROWS heads of its token.
template <typename T>
struct Four;   // four channels of a type
template <>
struct Four<float> {
  using Word = float4;
  static __device__ __forceinline__ void get(Word w, float (&v)[4]) { v[0] = w.x, v[1] = w.y, v[2] = w.z, v[3] = w.w; }
  static __device__ __forceinline__ Word put(const float (&v)[4]) { return make_float4(v[0], v[1], v[2], v[3]); }
};
template <>
struct Four<__half> {
  using Word = uint2;
  static __device__ __forceinline__ void get(Word w, float (&v)[4]) {
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&w.x));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&w.y));
    v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
  }
  static __device__ __forceinline__ Word put(const float (&v)[4]) {
    return make_uint2(pack_half2(v[0], v[1]), pack_half2(v[2], v[3]));
  }
};
template <>
struct Four<__nv_bfloat16> {
  using Word = uint2;
  static __device__ __forceinline__ void get(Word w, float (&v)[4]) {   // the upper halves of the fp32 values
    v[0] = __uint_as_float(w.x << 16), v[1] = __uint_as_float(w.x & 0xffff0000u);
    v[2] = __uint_as_float(w.y << 16), v[3] = __uint_as_float(w.y & 0xffff0000u);
  }
  static __device__ __forceinline__ Word put(const float (&v)[4]) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
    return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  }
};

constexpr int RP_THREADS = 256, RP_PIECES = 16, RP_HEADS = RP_THREADS / RP_PIECES;

template <typename T, int ROWS>
__global__ void __launch_bounds__(RP_THREADS) rope_kernel(const __grid_constant__ RopeParams p) {
  using F = Four<T>;
  using Word = typename F::Word;
  grid_dependency_wait();
  grid_dependents_launch();
  const int t = blockIdx.x, u = threadIdx.x & (RP_PIECES - 1);
  const int h0 = (int)blockIdx.y * (RP_HEADS * ROWS) + (threadIdx.x >> 4);
  const bool turns = 8 * u < p.rot;
  const bool split = turns && !p.interleaved;
  const int lo = split ? 4 * u : 8 * u, hi = split ? lo + (p.rot >> 1) : lo + 4;
  const T* x = static_cast<const T*>(p.x) + (long long)t * p.x_token;
  T* out = static_cast<T*>(p.out) + (long long)t * p.out_token;
  const int pos = __ldg(p.pos + t);
  Word a[ROWS], b[ROWS];
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const int h = h0 + i * RP_HEADS;
    if (h < p.H) {
      const T* row = x + (long long)h * p.x_head;
      a[i] = *reinterpret_cast<const Word*>(row + lo);
      b[i] = *reinterpret_cast<const Word*>(row + hi);
    }
  }
  if (pos < 0 || pos >= p.n_pos) {
    if (threadIdx.x == 0 && blockIdx.y == 0 && p.err) atomicOr(p.err, VQKV_DEVERR_POSITION);
    return;
  }
  float4 c = make_float4(1.f, 1.f, 1.f, 1.f), s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (turns) {
    const float* row = p.table + (size_t)pos * p.rot + 4 * u;
    c = __ldg(reinterpret_cast<const float4*>(row));
    s = __ldg(reinterpret_cast<const float4*>(row + (p.rot >> 1)));
    if (p.transpose) s = make_float4(-s.x, -s.y, -s.z, -s.w);
  }
  const float cv[4] = {c.x, c.y, c.z, c.w}, sv[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const int h = h0 + i * RP_HEADS;
    if (h >= p.H) break;
    if (turns) {
      float v[4], w[4];
      F::get(a[i], v);
      F::get(b[i], w);
      if (p.interleaved) {   // the halves hold two pairs each
        float y[4], z[4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          y[2 * j] = v[2 * j] * cv[j] - v[2 * j + 1] * sv[j], y[2 * j + 1] = v[2 * j + 1] * cv[j] + v[2 * j] * sv[j];
          z[2 * j] = w[2 * j] * cv[2 + j] - w[2 * j + 1] * sv[2 + j];
          z[2 * j + 1] = w[2 * j + 1] * cv[2 + j] + w[2 * j] * sv[2 + j];
        }
        a[i] = F::put(y), b[i] = F::put(z);
      } else {
        float y[4], z[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = v[j] * cv[j] - w[j] * sv[j], z[j] = w[j] * cv[j] + v[j] * sv[j];
        a[i] = F::put(y), b[i] = F::put(z);
      }
    }
    T* row = out + (long long)h * p.out_head;
    *reinterpret_cast<Word*>(row + lo) = a[i];
    *reinterpret_cast<Word*>(row + hi) = b[i];
  }
}

template <typename T>
cudaError_t launch_rope_of(const RopeParams& p, int sms, cudaStream_t stream) {
  // four heads a thread where that still fills the GPU
  const int per4 = RP_HEADS * 4;
  if ((long long)p.T * ((p.H + per4 - 1) / per4) >= 4 * sms)
    return launch_pdl(rope_kernel<T, 4>, dim3(p.T, (p.H + per4 - 1) / per4), dim3(RP_THREADS), 0, stream, p);
  return launch_pdl(rope_kernel<T, 1>, dim3(p.T, (p.H + RP_HEADS - 1) / RP_HEADS), dim3(RP_THREADS), 0, stream, p);
}

}  // namespace

cudaError_t launch_rope_table(const RopeTableParams& p, cudaStream_t stream) {
  const long long blocks = ((long long)p.n_pos * (p.rot >> 3) + 255) / 256;
  return launch_pdl(rope_table_kernel, dim3((unsigned)std::min<long long>(blocks, 1 << 20)), dim3(256), 0, stream, p);
}

cudaError_t launch_rope(const RopeParams& p, int sms, cudaStream_t stream) {
  if (p.dtype == VQKV_DTYPE_F32) return launch_rope_of<float>(p, sms, stream);
  if (p.dtype == VQKV_DTYPE_BF16) return launch_rope_of<__nv_bfloat16>(p, sms, stream);
  return launch_rope_of<__half>(p, sms, stream);
}

}  // namespace vqkv
