// Cross attention over a packed cache (vqkv_cross_attn): ragged queries, each of
// which sees all cached tokens of its sequence.  The kernel is that of the draft
// trees (decode_tree.cu) with other work units: an item is a group of up to 64,
// 128 or 256 of a sequence's columns (query, head of the KV head), its units the
// tiles of 64 tokens.  All items' units in order are cut into equal shares; a CTA of
// a KV head takes one share, or two side by side (items of up to 128 columns:
// STREAMS in tile_attn.cuh).  A share has a piece of an item that began before it and
// one that ends behind it at most, so two partials per share hold whatever the
// cut leaves for cross_combine_kernel.
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "tile_attn.cuh"

namespace vqkv {
namespace {

// q' of every column, as the attention kernel's threads load it (tree_query_kernel's
// image): sequence b's groups of 32 columns (PAIR: 16) start at cross_query_slot.
// Columns past a sequence's last are not written: they reach only rows of the
// products that are not stored.  Four threads per column.
template <bool PAIR>
__global__ void __launch_bounds__(128) cross_query_kernel(const __grid_constant__ DecodeParams p, uint4* qx) {
  constexpr int W = PAIR ? 16 : 32;
  __shared__ int s_start[kFlatMaxB];
  grid_dependency_wait();
  grid_dependents_launch();
  for (int i = threadIdx.x; i < p.B; i += 128) s_start[i] = __ldg(p.row_start + i);
  const int kvh = blockIdx.y, part = threadIdx.x & 3;
  const long long col = (long long)blockIdx.x * 32 + (threadIdx.x >> 2);
  const bool any = col < (long long)p.n_rows * p.g;
  const int row = any ? (int)(col / p.g) : 0, h = any ? (int)(col - (long long)row * p.g) : 0;
  __syncthreads();
  const int lo = sequence_of(s_start, p.B, row);   // the last sequence that starts at or before the row
  const RowRange rows = row_range(p, lo, false);
  const bool in = any && row >= rows.first && row - rows.first < rows.n;   // both in [0, n_rows]
  float v[32];
  if (in) {
    const float4* s4 = reinterpret_cast<const float4*>(p.s + (size_t)kvh * kHeadDim + 32 * part);
    const uint2* q = reinterpret_cast<const uint2*>(p.q + (long long)row * p.q_row + (kvh * p.g + h) * kHeadDim + 32 * part);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint2 x = q[i];
      const float4 f = s4[i];
      float2 a, b;
      if (p.bf16) {   // the upper halves of the fp32 values
        a = make_float2(__uint_as_float(x.x << 16), __uint_as_float(x.x & 0xffff0000u));
        b = make_float2(__uint_as_float(x.y << 16), __uint_as_float(x.y & 0xffff0000u));
      } else {
        a = __half22float2(*reinterpret_cast<const __half2*>(&x.x));
        b = __half22float2(*reinterpret_cast<const __half2*>(&x.y));
      }
      v[4 * i] = a.x * f.x, v[4 * i + 1] = a.y * f.y, v[4 * i + 2] = b.x * f.z, v[4 * i + 3] = b.y * f.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = 0.f;
  }
  fwht_column(v, part, p.qscale);
  if (!in) return;
  const int c = (row - rows.first) * p.g + h;
  const size_t slot = (size_t)kvh * (cross_query_slot(p.n_rows, p.B, p.g, W) + 1) + cross_query_slot(rows.first, lo, p.g, W) + c / W;
  uint4* dst = qx + (slot * 16 + 4 * part) * 32 + (c & (W - 1));
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
    if (PAIR) dst[32 * j + 16] = make_uint4(low[0], low[1], low[2], low[3]);
  }
}

// Merges the partials of the item that share blockIdx.x begins and does not end,
// if there is one.  CC_COLS columns per block, one after another per warp; WIDE
// (many partials per item): one column per block, blockIdx.x = item.  Lane = 4 channels, eight
// partials in flight.
constexpr int CC_WARPS = 8, CC_COLS = 32;
template <bool WIDE>
__global__ void __launch_bounds__(CC_WARPS * 32) cross_combine_kernel(const __grid_constant__ DecodeParams p, int cols, int groups_max) {
  constexpr int U = 8;
  __shared__ int s_pref[kFlatMaxB + 1];
  __shared__ float4 s_o[CC_WARPS][32];
  __shared__ float2 s_ml[CC_WARPS];
  const int kvh = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_dependency_wait();
  grid_dependents_launch();
  item_prefix<tr::TOK>(p, cols, s_pref, false);
  const int T = s_pref[p.B], S = min(p.n_splits, T);
  int split, b, group, all;
  if (WIDE) {   // item blockIdx.x of groups_max per sequence
    b = blockIdx.x / groups_max, group = blockIdx.x - b * groups_max;
    all = (clamped_len(p, b) + tr::TOK - 1) / tr::TOK;
    if (s_pref[b] + (long long)group * all >= s_pref[b + 1]) return;
    split = flat_cta_of(s_pref[b] + group * all, T, S);
  } else {      // that of the last unit of share blockIdx.x
    split = blockIdx.x;
    if (split >= S) return;
    const int unit = (int)((long long)T * (split + 1) / S) - 1;
    b = sequence_of(s_pref, p.B, unit);
    all = (clamped_len(p, b) + tr::TOK - 1) / tr::TOK, group = (unit - s_pref[b]) / all;
  }
  const int r0 = (int)((long long)T * split / S), r1 = (int)((long long)T * (split + 1) / S);
  const int first = s_pref[b] + group * all, last = first + all;   // the item's units
  if (first < r0 || last <= r1) return;
  const RowRange rows = row_range(p, b, false);
  const int live = min(cols, rows.n * p.g - group * cols);
  const int parts = flat_cta_of(last - 1, T, S) - split + 1;
  const size_t stride = (size_t)2 * cols * kPartialStride;   // from share to share
  constexpr int STEP = WIDE ? CC_WARPS : 1;
  const int cl0 = WIDE ? blockIdx.z : blockIdx.z * CC_COLS, cl1 = min(live, cl0 + (WIDE ? 1 : CC_COLS));
  for (int cl = WIDE ? cl0 : cl0 + warp; cl < cl1; cl += CC_WARPS) {
    // the first part is its share's second partial, the others the first
    const float* base = p.partials + (((size_t)kvh * p.n_splits + split) * 2 * cols + cl) * kPartialStride;
    float M = kMInit, l = 0.f;
    float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](float2 ml, float4 o) {
      const float n = fmaxf(M, ml.x), fa = fast_exp2(M - n), fb = fast_exp2(ml.x - n);
      O.x = O.x * fa + o.x * fb, O.y = O.y * fa + o.y * fb, O.z = O.z * fa + o.z * fb, O.w = O.w * fa + o.w * fb;
      l = l * fa + ml.y * fb;
      M = n;
    };
    for (int i0 = WIDE ? warp : 0; i0 < parts; i0 += U * STEP) {
      float2 ml[U];
      float4 o[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + u * STEP;
        if (i < parts) {
          const float* at = base + i * stride + (i == 0 ? (size_t)cols * kPartialStride : 0);
          ml[u] = __ldcg(reinterpret_cast<const float2*>(at + 128));
          o[u] = __ldcg(reinterpret_cast<const float4*>(at) + lane);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i0 + u * STEP < parts) add(ml[u], o[u]);
    }
    if (WIDE) {   // the block's warps meet in shared memory
      s_o[warp][lane] = O;
      if (lane == 0) s_ml[warp] = make_float2(M, l);
      __syncthreads();
      if (warp != 0) return;
#pragma unroll
      for (int w = 1; w < CC_WARPS; ++w) add(s_ml[w], s_o[w][lane]);
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    __half* dst = p.out + cross_out_row(p, rows.first, kvh, group * cols + cl) + 4 * lane;
    const float4 w = make_float4(O.x * inv, O.y * inv, O.z * inv, O.w * inv);
    if (p.bf16) store_out4<true>(dst, w); else store_out4<false>(dst, w);
  }
}

using CrossKernel = void (*)(DecodeParams, const unsigned long long*, const uint4*);
template <int MODE, bool PAGED>
CrossKernel cross_of(int layout) {
  if (layout == kPairs) return decode_tree_kernel<MODE, PAGED, 1, true, true>;
  if (layout == kTwoTiles) return decode_tree_kernel<MODE, PAGED, 2, false, true>;
  return decode_tree_kernel<MODE, PAGED, 1, false, true>;
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

int cross_cols(int layout) { return layout == kPairs ? 64 : layout == kTwoTiles ? 2 * tr::ROWS : tr::ROWS; }

cudaError_t cross_prepare(int mode) {
  cudaError_t e = cudaSuccess;
  for (int i = 0; i < 6 && e == cudaSuccess; ++i)
    e = prepare_split_kernel(cross_kernel(mode, (i & 1) != 0, i >> 1), tr::THREADS, tr::SPLIT_REGS, cross_smem(mode));
  return e;
}

size_t cross_query_bytes(int B, int Hq, int Hkv, int n_rows, int layout) {
  return (size_t)Hkv * (cross_query_slot(n_rows, B, Hq / Hkv, layout == kPairs ? 16 : 32) + 1) * 32 * kHeadDim * 2;
}

cudaError_t launch_cross(int mode, const DecodeParams& p, int layout, int groups_max, void* qx, cudaStream_t stream) {
  uint4* q = static_cast<uint4*>(qx);
  const dim3 grid((unsigned)(((long long)p.n_rows * p.g + 31) / 32), p.Hkv);
  cudaError_t e = layout == kPairs ? launch_pdl(cross_query_kernel<true>, grid, dim3(128), 0, stream, p, q)
                                   : launch_pdl(cross_query_kernel<false>, grid, dim3(128), 0, stream, p, q);
  if (e == cudaSuccess)
    e = launch_pdl(cross_kernel(mode, p.block_table != nullptr, layout), dim3(layout == kTwoTiles ? p.n_splits : (p.n_splits + 1) / 2, p.Hkv), dim3(tr::THREADS),
                   (size_t)cross_smem(mode), stream, p, static_cast<const unsigned long long*>(nullptr),
                   static_cast<const uint4*>(qx));
  if (e == cudaSuccess && p.n_splits > 1) {
    const int cols = cross_cols(layout);
    const int wide_items = p.n_splits > 4LL * p.B * groups_max ? p.B * groups_max : 0;   // few items, many partials
    if (wide_items > 0)
      e = launch_pdl(cross_combine_kernel<true>, dim3(wide_items, p.Hkv, p.ncols), dim3(CC_WARPS * 32), 0, stream, p, cols,
                     wide_items / p.B);
    else
      e = launch_pdl(cross_combine_kernel<false>, dim3(p.n_splits, p.Hkv, (p.ncols + CC_COLS - 1) / CC_COLS),
                     dim3(CC_WARPS * 32), 0, stream, p, cols, 0);
  }
  return e;
}

}  // namespace vqkv
