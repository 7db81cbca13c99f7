// Cross attention over a packed cache (vqkv_cross_attn): ragged queries, each of
// which sees all cached tokens of its sequence.  The kernel is that of the draft
// trees (decode_tree.cu) with other work units: an item is a group of up to 64 or
// 128 of a sequence's columns (query, head of the KV head), its units the tiles of
// 64 tokens.  All items' units in order are cut into equal shares; a CTA of a KV head
// takes one share, or two side by side (items of 64 columns: STREAMS in tile_attn.cuh).
// A share has a piece of an item that began before it and one that ends behind it at
// most, so two partials per share hold whatever the cut leaves for
// cross_combine_kernel.
//
// The scores come from both fp16 parts of q' (above 64 columns: ONE_O in
// tile_attn.cuh).  One part is off by 2^-12 rms, and a weight by that times its score
// in nats, a size that has no bound: fp16 results with errors of 2.7e-4 (2.1e-4 is the
// output's own rounding) had 3.7e-4; bf16 ones, rounded to 1.7e-3 rms, 1.9e-3 at
// scores of 11 nats rms and 2.1e-3 at 22.  With one part and up to 256 columns per
// dequantised tile the ragged bf16 prompts below took 90 us.
//
// Bound: the chain of a tile (scores, softmax, P V) against dequantisation that only
// 64 or 128 columns share, as in the draft trees.  2,048 queries of 32 heads over
// 32,768 tokens at 2 bit: 1.19 ms (0.92 PFLOP/s of the two products, 1.38 with the
// low parts); 12 ragged prompts of 33 to 448 tokens over paged 4-bit states of 600 to
// 1,500: 112 us, about a sixth of them q' and the merge.
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "tile_attn.cuh"

namespace vqkv {
namespace {

// Four consecutive values of an output row, whose address is a multiple of 2 bytes.
__device__ __forceinline__ void store_four(const DecodeParams& p, __half* dst, float4 w) {
  if (!p.bf16) {
    store_out4(dst, w);
    return;
  }
  const __nv_bfloat162 a = __floats2bfloat162_rn(w.x, w.y), b = __floats2bfloat162_rn(w.z, w.w);
  const uint2 h = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  if ((reinterpret_cast<uintptr_t>(dst) & 7) == 0) {
    *reinterpret_cast<uint2*>(dst) = h;
  } else {
    dst[0] = __ushort_as_half((unsigned short)h.x), dst[1] = __ushort_as_half((unsigned short)(h.x >> 16));
    dst[2] = __ushort_as_half((unsigned short)h.y), dst[3] = __ushort_as_half((unsigned short)(h.y >> 16));
  }
}

// q' of every column, as the attention kernel's threads load it (tree_query_kernel's
// image): sequence b's groups of 32 columns (PAIR: 16) start at cross_query_slot.
// Columns past a sequence's last are neither written nor read.  Four threads per
// column.  PAIR: a group's 16 columns' high and low parts side by side; else a group's
// high parts, then its low ones.
template <bool PAIR>
__global__ void __launch_bounds__(128) cross_query_kernel(const __grid_constant__ DecodeParams p, uint4* qx) {
  constexpr int W = PAIR ? 16 : 32;
  __shared__ int s_start[kFlatMaxB + 1];
  __shared__ float4 s_s[4][9];   // s, 32 channels a row, rows in different banks
  grid_dependency_wait();
  grid_dependents_launch();
  const int kvh = blockIdx.y, part = threadIdx.x & 3;
  const long long col = (long long)blockIdx.x * 32 + (threadIdx.x >> 2);
  const bool any = col < (long long)p.n_rows * p.g;
  const int row = any ? (int)(col / p.g) : 0, h = any ? (int)(col - (long long)row * p.g) : 0;
  const uint2* q = reinterpret_cast<const uint2*>(p.q + (long long)row * p.q_row + (kvh * p.g + h) * kHeadDim + 32 * part);
  uint2 x[8];   // in flight while the row's sequence is looked up
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = q[i];
  if (threadIdx.x < kHeadDim / 4)
    s_s[threadIdx.x >> 3][threadIdx.x & 7] = __ldg(reinterpret_cast<const float4*>(p.s + (size_t)kvh * kHeadDim) + threadIdx.x);
  for (int i = threadIdx.x; i <= p.B; i += 128) s_start[i] = __ldg(p.row_start + i);
  __syncthreads();
  const int lo = sequence_of(s_start, p.B, row);   // the last sequence that starts at or before the row
  const RowRange rows = rows_between(p, s_start[lo], s_start[lo + 1]);
  const bool in = any && row >= rows.first && row - rows.first < rows.n;   // both in [0, n_rows]
  float v[32];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float4 f = s_s[part][i];
    float2 a, b;
    if (p.bf16) {   // the upper halves of the fp32 values
      a = make_float2(__uint_as_float(x[i].x << 16), __uint_as_float(x[i].x & 0xffff0000u));
      b = make_float2(__uint_as_float(x[i].y << 16), __uint_as_float(x[i].y & 0xffff0000u));
    } else {
      a = __half22float2(*reinterpret_cast<const __half2*>(&x[i].x));
      b = __half22float2(*reinterpret_cast<const __half2*>(&x[i].y));
    }
    v[4 * i] = a.x * f.x, v[4 * i + 1] = a.y * f.y, v[4 * i + 2] = b.x * f.z, v[4 * i + 3] = b.y * f.w;
  }
  fwht_column(v, part, p.qscale);
  if (!in) return;
  const int c = (row - rows.first) * p.g + h;
  const size_t slot = (size_t)kvh * (cross_query_slot(p.n_rows, p.B, p.g, W) + 1) + cross_query_slot(rows.first, lo, p.g, W) + c / W;
  uint4* dst = qx + ((PAIR ? slot : 2 * slot) * 16 + 4 * part) * 32 + (c & (W - 1));
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t w[4], low[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x = v[8 * j + 2 * i], y = v[8 * j + 2 * i + 1];
      const __half2 f = __floats2half2_rn(x, y);
      w[i] = *reinterpret_cast<const uint32_t*>(&f);
      low[i] = pack_half2(x - __low2float(f), y - __high2float(f));
    }
    dst[32 * j] = make_uint4(w[0], w[1], w[2], w[3]);
    dst[32 * j + (PAIR ? 16 : 16 * 32)] = make_uint4(low[0], low[1], low[2], low[3]);
  }
}

// Merges of the items that several shares overlap.  Of share `split`'s two partials
// the second is an item's first part, the first any other.
__device__ __forceinline__ const float4* cross_partial(const DecodeParams& p, int kvh, int split, int part, int cols) {
  return reinterpret_cast<const float4*>(p.partials) +
         (((size_t)kvh * p.n_splits + split + part) * 2 + (part == 0)) * (cols * kPartialStride / 4);
}

// Few partials per item: the item that share blockIdx.x begins, if it does not end
// it.  Lane = column of 32, warp = 16 channels: every load is 512 neighbouring bytes.
__global__ void __launch_bounds__(256) cross_combine_kernel(const __grid_constant__ DecodeParams p, int cols) {
  const int split = blockIdx.x, kvh = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_dependency_wait();
  grid_dependents_launch();
  const int4 item = __ldcg(reinterpret_cast<const int4*>(p.tickets) + split);
  if (item.z == 0) return;
  const RowRange rows = row_range(p, item.x, false);
  const int cl = blockIdx.z * 32 + lane, c = item.y * cols + cl;
  if (cl >= cols || c >= rows.n * p.g) return;
  float M = kMInit, l = 0.f, O[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) O[i] = 0.f;
  constexpr int U = 2;
  for (int i0 = 0; i0 < item.z; i0 += U) {
    float2 ml[U];
    float4 o[U][4];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      ml[u] = make_float2(kMInit, 0.f);
      if (i0 + u < item.z) {
        const float4* at = cross_partial(p, kvh, split, i0 + u, cols);
        ml[u] = __ldcg(reinterpret_cast<const float2*>(at + 32 * cols) + cl);
#pragma unroll
        for (int k = 0; k < 4; ++k) o[u][k] = __ldcg(at + (4 * warp + k) * cols + cl);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) o[u][k] = make_float4(0.f, 0.f, 0.f, 0.f);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float n = fmaxf(M, ml[u].x), fa = fast_exp2(M - n), fb = fast_exp2(ml[u].x - n);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        O[4 * k] = O[4 * k] * fa + o[u][k].x * fb, O[4 * k + 1] = O[4 * k + 1] * fa + o[u][k].y * fb;
        O[4 * k + 2] = O[4 * k + 2] * fa + o[u][k].z * fb, O[4 * k + 3] = O[4 * k + 3] * fa + o[u][k].w * fb;
      }
      l = l * fa + ml[u].y * fb;
      M = n;
    }
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  __half* dst = p.out + cross_out_row(p, rows.first, kvh, c) + 16 * warp;
#pragma unroll
  for (int k = 0; k < 4; ++k)
    store_four(p, dst + 4 * k, make_float4(O[4 * k] * inv, O[4 * k + 1] * inv, O[4 * k + 2] * inv, O[4 * k + 3] * inv));
}

// Many partials per item (few items): a block per column, a warp per every eighth
// part, lane = 4 channels; item blockIdx.x of groups_max per sequence.
constexpr int CW_WARPS = 8;
__global__ void __launch_bounds__(CW_WARPS * 32) cross_combine_wide_kernel(const __grid_constant__ DecodeParams p, int cols,
                                                                           int groups_max) {
  constexpr int U = 8;
  __shared__ int s_pref[kFlatMaxB + 1];
  __shared__ float4 s_o[CW_WARPS][32];
  __shared__ float2 s_ml[CW_WARPS];
  const int kvh = blockIdx.y, cl = blockIdx.z, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_dependency_wait();
  grid_dependents_launch();
  item_prefix<tr::TOK>(p, cols, s_pref, false);
  const int T = s_pref[p.B], S = min(p.n_splits, T);
  const int b = blockIdx.x / groups_max, group = blockIdx.x - b * groups_max;
  const int all = (clamped_len(p, b) + tr::TOK - 1) / tr::TOK;
  if (s_pref[b] + (long long)group * all >= s_pref[b + 1]) return;
  const int first = s_pref[b] + group * all, split = flat_cta_of(first, T, S);
  const int parts = flat_cta_of(first + all - 1, T, S) - split + 1;
  const RowRange rows = row_range(p, b, false);
  const int c = group * cols + cl;
  if (parts == 1 || c >= rows.n * p.g) return;
  float M = kMInit, l = 0.f;
  float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](float2 ml, float4 o) {
    const float n = fmaxf(M, ml.x), fa = fast_exp2(M - n), fb = fast_exp2(ml.x - n);
    O.x = O.x * fa + o.x * fb, O.y = O.y * fa + o.y * fb, O.z = O.z * fa + o.z * fb, O.w = O.w * fa + o.w * fb;
    l = l * fa + ml.y * fb;
    M = n;
  };
  for (int i0 = warp; i0 < parts; i0 += U * CW_WARPS) {
    float2 ml[U];
    float4 o[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i0 + u * CW_WARPS < parts) {
        const float4* at = cross_partial(p, kvh, split, i0 + u * CW_WARPS, cols);
        ml[u] = __ldcg(reinterpret_cast<const float2*>(at + 32 * cols) + cl);
        o[u] = __ldcg(at + lane * cols + cl);
      }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i0 + u * CW_WARPS < parts) add(ml[u], o[u]);
  }
  s_o[warp][lane] = O;
  if (lane == 0) s_ml[warp] = make_float2(M, l);
  __syncthreads();
  if (warp != 0) return;
#pragma unroll
  for (int w = 1; w < CW_WARPS; ++w) add(s_ml[w], s_o[w][lane]);
  const float inv = l > 0.f ? 1.f / l : 0.f;
  store_four(p, p.out + cross_out_row(p, rows.first, kvh, c) + 4 * lane, make_float4(O.x * inv, O.y * inv, O.z * inv, O.w * inv));
}

using CrossKernel = void (*)(DecodeParams, const unsigned long long*, const uint4*);
template <int MODE, bool PAGED>
CrossKernel cross_of(int layout) {
  if (layout == kPairs) return decode_tree_kernel<MODE, PAGED, 1, true, kCrossPairs>;
  return decode_tree_kernel<MODE, PAGED, 1, false, kCrossParts>;
}
template <int MODE>
CrossKernel cross_of(bool paged, int layout) {
  return paged ? cross_of<MODE, true>(layout) : cross_of<MODE, false>(layout);
}
CrossKernel cross_kernel(int mode, bool paged, int layout) {
  return mode == VQKV_MODE_VQ2    ? cross_of<VQKV_MODE_VQ2>(paged, layout)
         : mode == VQKV_MODE_VQ4  ? cross_of<VQKV_MODE_VQ4>(paged, layout)
         : mode == VQKV_MODE_VQ3  ? cross_of<VQKV_MODE_VQ3>(paged, layout)
         : mode == VQKV_MODE_VQ15 ? cross_of<VQKV_MODE_VQ15>(paged, layout)
                                  : cross_of<VQKV_MODE_VQ125>(paged, layout);
}
int cross_smem(int mode) {
  return mode == VQKV_MODE_VQ15 || mode == VQKV_MODE_VQ125 ? tr::Geo<VQKV_MODE_VQ15>::SMEM : tr::Geo<VQKV_MODE_VQ2>::SMEM;
}

}  // namespace

int cross_cols(int layout) { return layout == kPairs ? 64 : tr::ROWS; }
int cross_shares(int layout) { return layout == kPairs ? 2 : 1; }

cudaError_t cross_prepare(int mode) {
  cudaError_t e = cudaSuccess;
  for (int i = 0; i < 4 && e == cudaSuccess; ++i)
    e = prepare_split_kernel(cross_kernel(mode, (i & 1) != 0, i < 2 ? kPairs : kBothParts), tr::THREADS, tr::SPLIT_REGS, cross_smem(mode));
  return e;
}

size_t cross_query_bytes(int B, int Hq, int Hkv, int n_rows, int layout) {
  return (size_t)Hkv * (cross_query_slot(n_rows, B, Hq / Hkv, layout == kPairs ? 16 : 32) + 1) *
         (layout == kPairs ? 1 : 2) * 32 * kHeadDim * 2;
}

cudaError_t launch_cross(int mode, const DecodeParams& p, int layout, int groups_max, void* qx, cudaStream_t stream) {
  uint4* q = static_cast<uint4*>(qx);
  const dim3 grid((unsigned)(((long long)p.n_rows * p.g + 31) / 32), p.Hkv);
  cudaError_t e = launch_pdl(layout == kPairs ? cross_query_kernel<true> : cross_query_kernel<false>, grid, dim3(128), 0, stream,
                             p, q);
  if (e == cudaSuccess)
    e = launch_pdl(cross_kernel(mode, p.block_table != nullptr, layout),
                   dim3((p.n_splits + cross_shares(layout) - 1) / cross_shares(layout), p.Hkv), dim3(tr::THREADS),
                   (size_t)cross_smem(mode), stream, p, static_cast<const unsigned long long*>(nullptr),
                   static_cast<const uint4*>(qx));
  if (e == cudaSuccess && p.n_splits > 1) {
    const int cols = cross_cols(layout);
    const int wide_items = p.n_splits > 4LL * p.B * groups_max ? p.B * groups_max : 0;   // few items, many partials
    if (wide_items > 0)
      e = launch_pdl(cross_combine_wide_kernel, dim3(wide_items, p.Hkv, p.ncols), dim3(CW_WARPS * 32), 0, stream, p, cols,
                     groups_max);
    else
      e = launch_pdl(cross_combine_kernel, dim3(p.n_splits, p.Hkv, (p.ncols + 31) / 32), dim3(256), 0, stream, p, cols);
  }
  return e;
}

}  // namespace vqkv
