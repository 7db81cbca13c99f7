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
// an eighth of a turn, is a number of 24 bits or more for the series.
// One thread: the same four pairs of RT_ROWS positions, two 16-byte stores each.  Its
// steps come out of the parameters once (lanes with different indices read them one
// after another), and from position to position the turn only grows by an exact 64-bit
// sum.  Bound by the stores: 196,608 x 128 take 19 us (5.3 TB/s), issue slots 69 % busy
// (with sincospif and a 64-bit product per element 49 us, bound by issue).
// sin and cos of a number x of half turns, |x| <= 1/4: Taylor's series, whose first
// terms left out are below (pi / 4)^11 / 11! = 2e-9 and (pi / 4)^12 / 12! = 2e-10.
__device__ __forceinline__ void sincos_half_turns(float x, float& s, float& c) {
  const float y = x * x;
  s = x * __fmaf_rn(y, __fmaf_rn(y, __fmaf_rn(y, __fmaf_rn(y, 0.0821458866f, -0.599264529f), 2.55016404f), -5.16771278f), 3.14159265f);
  c = __fmaf_rn(y, __fmaf_rn(y, __fmaf_rn(y, __fmaf_rn(y, __fmaf_rn(y, -0.0258068914f, 0.23533063f), -1.33526277f), 4.05871213f), -4.9348022f), 1.f);
}

constexpr int RT_THREADS = 256, RT_ROWS = 8;
__global__ void __launch_bounds__(RT_THREADS) rope_table_kernel(const __grid_constant__ RopeTableParams p) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int quads = p.rot >> 3, rows = RT_THREADS / quads;   // four-pair pieces of a row; rows of a round
  const int r = threadIdx.x / quads, i = 4 * (threadIdx.x - r * quads);
  if (r >= rows) return;
  long long pos = (long long)blockIdx.x * (rows * RT_ROWS) + r;
  unsigned long long turn[4], step[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    turn[j] = p.step[i + j] * (unsigned long long)pos;
    step[j] = p.step[i + j] * (unsigned long long)rows;
  }
  float* row = p.table + pos * p.rot + i;
#pragma unroll 2
  for (int n = 0; n < RT_ROWS && pos < p.n_pos; ++n, pos += rows, row += (long long)rows * p.rot) {
    float c[4], s[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const unsigned top = (unsigned)((turn[j] + (1ull << 31)) >> 32);       // turns in units of 2^-32
      turn[j] += step[j];
      const unsigned quarter = (top + (1u << 29)) >> 30;
      const float rest = (float)(int)(top - (quarter << 30)) * 4.656612873077393e-10f;   // half turns: 2^-31 each
      float a, b;
      sincos_half_turns(rest, a, b);
      const float y = quarter & 1 ? b : a, x = quarter & 1 ? a : b;           // quarter turns swap and negate
      s[j] = (quarter & 2 ? -y : y) * p.amplitude;
      c[j] = ((quarter + 1) & 2 ? -x : x) * p.amplitude;
    }
    *reinterpret_cast<float4*>(row) = make_float4(c[0], c[1], c[2], c[3]);
    *reinterpret_cast<float4*>(row + (p.rot >> 1)) = make_float4(s[0], s[1], s[2], s[3]);
  }
}

// ------------------------------------------------------------------ rotation
// (y_i, z_i) = (a c - b s, b c + a s) over the row's pairs.  A row is 16 pieces of
// two four-channel halves: a piece u below rot / 8 holds pairs 4u .. 4u + 3 (both
// members, so no thread needs another's channels, and the rotation may be in
// place), the others channels that pass through.  A thread takes one piece of ROWS
// heads of each of TOKENS tokens, all its loads in flight before the first is used.
// Bound by memory: 16,384 bf16 tokens of 32 heads 45 us (6.0 TB/s), 8,191 fp32 ones of
// 40 heads 50 us (6.8 TB/s).
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

template <typename T, int ROWS, int TOKENS>
__global__ void __launch_bounds__(RP_THREADS) rope_kernel(const __grid_constant__ RopeParams p) {
  using F = Four<T>;
  using Word = typename F::Word;
  grid_dependency_wait();
  grid_dependents_launch();
  const int t0 = blockIdx.x * TOKENS, u = threadIdx.x & (RP_PIECES - 1);
  const int h0 = (int)blockIdx.y * (RP_HEADS * ROWS) + (threadIdx.x >> 4);
  const bool turns = 8 * u < p.rot;
  const bool split = turns && !p.interleaved;
  const int lo = split ? 4 * u : 8 * u, hi = split ? lo + (p.rot >> 1) : lo + 4;
  int pos[TOKENS];
  Word a[TOKENS][ROWS], b[TOKENS][ROWS];
#pragma unroll
  for (int k = 0; k < TOKENS; ++k) pos[k] = t0 + k < p.T ? __ldg(p.pos + t0 + k) : 0;
#pragma unroll
  for (int k = 0; k < TOKENS; ++k)
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      const int h = h0 + i * RP_HEADS;
      if (h < p.H && t0 + k < p.T) {
        const T* row = static_cast<const T*>(p.x) + (long long)(t0 + k) * p.x_token + (long long)h * p.x_head;
        a[k][i] = *reinterpret_cast<const Word*>(row + lo);
        b[k][i] = *reinterpret_cast<const Word*>(row + hi);
      }
    }
#pragma unroll
  for (int k = 0; k < TOKENS; ++k) {
    if (t0 + k >= p.T) break;
    if (pos[k] < 0 || pos[k] >= p.n_pos) {
      if (threadIdx.x == 0 && blockIdx.y == 0 && p.err) atomicOr(p.err, VQKV_DEVERR_POSITION);
      continue;
    }
    float4 c = make_float4(1.f, 1.f, 1.f, 1.f), s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (turns) {
      const float* row = p.table + (size_t)pos[k] * p.rot + 4 * u;
      c = __ldg(reinterpret_cast<const float4*>(row));
      s = __ldg(reinterpret_cast<const float4*>(row + (p.rot >> 1)));
      if (p.transpose) s = make_float4(-s.x, -s.y, -s.z, -s.w);
    }
    const float cv[4] = {c.x, c.y, c.z, c.w}, sv[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      const int h = h0 + i * RP_HEADS;
      if (h >= p.H) break;
      Word y4 = a[k][i], z4 = b[k][i];
      if (turns) {
        float v[4], w[4], y[4], z[4];
        F::get(y4, v);
        F::get(z4, w);
        if (p.interleaved) {   // the halves hold two pairs each
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            y[2 * j] = v[2 * j] * cv[j] - v[2 * j + 1] * sv[j], y[2 * j + 1] = v[2 * j + 1] * cv[j] + v[2 * j] * sv[j];
            z[2 * j] = w[2 * j] * cv[2 + j] - w[2 * j + 1] * sv[2 + j];
            z[2 * j + 1] = w[2 * j + 1] * cv[2 + j] + w[2 * j] * sv[2 + j];
          }
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) y[j] = v[j] * cv[j] - w[j] * sv[j], z[j] = w[j] * cv[j] + v[j] * sv[j];
        }
        y4 = F::put(y), z4 = F::put(z);
      }
      T* row = static_cast<T*>(p.out) + (long long)(t0 + k) * p.out_token + (long long)h * p.out_head;
      *reinterpret_cast<Word*>(row + lo) = y4;
      *reinterpret_cast<Word*>(row + hi) = z4;
    }
  }
}

// Three or four rows a thread where that still fills the GPU: of one token, or of two
// or four where a token has only two or one (32 heads of 16,384 bf16 tokens: 50 us with
// two rows of one token).
template <typename T, int ROWS, int TOKENS>
cudaError_t launch_rope_as(const RopeParams& p, cudaStream_t stream) {
  constexpr int per = RP_HEADS * ROWS;
  return launch_pdl(rope_kernel<T, ROWS, TOKENS>, dim3((p.T + TOKENS - 1) / TOKENS, (p.H + per - 1) / per), dim3(RP_THREADS), 0,
                    stream, p);
}
template <typename T>
cudaError_t launch_rope_of(const RopeParams& p, int sms, cudaStream_t stream) {
  if ((long long)p.T * p.H < 64LL * 4 * sms) return launch_rope_as<T, 1, 1>(p, stream);
  if (p.H <= RP_HEADS) return launch_rope_as<T, 1, 4>(p, stream);
  if (p.H <= 2 * RP_HEADS) return launch_rope_as<T, 2, 2>(p, stream);
  if (p.H <= 3 * RP_HEADS) return launch_rope_as<T, 3, 1>(p, stream);
  return launch_rope_as<T, 4, 1>(p, stream);
}

}  // namespace

cudaError_t launch_rope_table(const RopeTableParams& p, cudaStream_t stream) {
  const int rows = RT_THREADS / (p.rot >> 3) * RT_ROWS;
  return launch_pdl(rope_table_kernel, dim3((unsigned)(((long long)p.n_pos + rows - 1) / rows)), dim3(RT_THREADS), 0, stream, p);
}

cudaError_t launch_rope(const RopeParams& p, int sms, cudaStream_t stream) {
  if (p.dtype == VQKV_DTYPE_F32) return launch_rope_of<float>(p, sms, stream);
  if (p.dtype == VQKV_DTYPE_BF16) return launch_rope_of<__nv_bfloat16>(p, sms, stream);
  return launch_rope_of<__half>(p, sms, stream);
}

}  // namespace vqkv
