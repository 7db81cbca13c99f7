// Attention of a tree of drafted tokens over a packed cache (sm_103a, tcgen05).
//
// M drafts x g query heads give up to 512 softmax columns per KV head, so the
// two products are matrix products worth the tensor cores.  A CTA takes up to
// 128 or 256 columns (MMA rows) of one KV head and walks its share of the
// batch's tokens in tiles of 64:
//   dequantise  K' and V tiles into shared memory, each centroid gathered
//               once per tile and CTA (16 warps: 8 for K, 8 for V)
//   S = Q' K'^T 128 x 64 x 128, Q' in tensor memory (A), K' rows in shared
//               memory (B, K-major), S in tensor memory
//   softmax     one thread per column: running max and sum in fp32, P =
//               exp2(S - m) as fp16 back to tensor memory; O is rescaled only
//               when a score exceeds the running max by 2^8
//   O += P V    128 x 128 x 64, P in tensor memory (A), V rows in shared
//               memory (B, channel-major), O stays in tensor memory
// There are two softmax warpgroups with an S, P, O, max and sum each.  Up to
// 128 columns (NQ = 1) they take the tiles in turn (one warpgroup alone spends
// more time on a tile's 64 exponentials per thread than everything else
// takes), and their states are merged at the end; a
// warpgroup's next score product is issued as soon as it has read its last
// scores.  Above 128 columns (NQ = 2) each warpgroup takes 128 columns of
// every tile, so one dequantisation serves 256; P then overlays S (tensor
// memory is full).
//
// Work: all sequences' tiles in order are cut into equal shares, one CTA per
// share, KV head and column group (the flat plan of the single-query decode).
// A share that holds a whole sequence writes its O, other overlaps leave
// partials (m, l, O) that tree_combine_kernel merges.
//
// The query transform is that of the single-query decode: q' = (q * s) . Hn,
// scaled by softmax_scale * log2 e.  q' and P are rounded to fp16 (2^-12
// relative, as in the other decode kernels) for the fp16 tensor-core product;
// centroids are fp16 already, sums are fp32.
//
// PAIR (at most 64 columns; for the attention weights, whose softmax sums have to
// match the key pass's scores, and for short trees, which the host bounds):
// q' = hi + lo in two fp16 parts, off by at most max(2^-22 |q'|, 2^-25) per channel.
// The unused half of the MMA rows takes the low parts, 16 columns to a warp: lanes
// 0..15 the high parts, lanes 16..31 the low parts of the same columns, whose scores
// one shuffle adds; both lanes then carry the column.  (Not for long trees: 64
// shuffles more per thread and tile.)
//
// Measured: 64 columns over 196,608 tokens and 8 KV heads at 2 bit take 98 us for the
// call (525 TFLOP/s of the two products; plain torch 11.4 ms).  A 64-token
// tile takes 1,050 cycles.  Bound: shared memory (each token's 512 bytes are
// gathered, stored and read by the MMAs; about three quarters of the time)
// and the hand-offs between the roles.  A 256-column tile (NQ = 2) takes 2,180
// cycles at 2 bit, as much per column as two CTAs of 128, and less at 1.5 bit,
// where the gathers conflict, and it halves the partials: hence the border at 128.
// 135 columns of 8 ragged sequences at 1.5 bit take 173 us, 256 columns of
// 32,768 tokens at 4 bit 53 us, 18 of them for queries, prologue and merge.
//
// Visibility: tokens t < L - M for every column, draft j for the columns
// whose mask has bit j; only tiles that reach past L - M test it.  Without
// masks the M queries are causal.  p.stats, where given, receives each column's
// max and 1 / sum.
#include <type_traits>

#include "common.cuh"
#include "decode_common.cuh"
#include "dequant_tile.cuh"
#include "gather.cuh"
#include "internal.h"
#include "tile_attn.cuh"
#include "umma.cuh"

namespace vqkv {
namespace {

// q' of every softmax column as fp16, in the order the attention kernel's
// threads load it: [B][Hkv][groups of 32 columns][16 pieces of 8 channels][32
// columns], zeros past the last column.  A kernel of its own because every
// share of a sequence needs the same rows (19 of them at 8 KV heads): doing it
// per share took 2.2 us of each CTA at 64 columns and 6.4 us at 256.  It runs
// while the attention kernel fills its codebooks.
// PAIR: groups of 16 columns, rows 0..15 the high and 16..31 the low parts.
// grid (groups, Hkv, B), four threads per column.
template <bool PAIR>
__global__ void __launch_bounds__(PAIR ? 64 : 128) tree_query_kernel(const DecodeParams p, uint4* qx) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int kvh = blockIdx.y, b = blockIdx.z, part = threadIdx.x & 3;
  const int r = threadIdx.x >> 2, c = (PAIR ? 16 : 32) * blockIdx.x + r;
  float v[32];
  transform_column(p, b, kvh, c, part, v);
  uint4* dst = qx + ((((size_t)b * p.Hkv + kvh) * gridDim.x + blockIdx.x) * 16 + 4 * part) * 32 + r;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t w[4], lo[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x = v[8 * j + 2 * i], y = v[8 * j + 2 * i + 1];
      const __half2 h = __floats2half2_rn(x, y);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
      lo[i] = pack_half2(x - __low2float(h), y - __high2float(h));
    }
    dst[32 * j] = make_uint4(w[0], w[1], w[2], w[3]);
    if (PAIR) dst[32 * j + 16] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  }
}

// Merges the partials of the softmax columns of (sequence blockIdx.y, all KV
// heads) that several shares overlap.  One column per warp, or per block (WIDE:
// many partials per sequence); lane = 4 channels, eight partials in flight.
constexpr int TC_WARPS = 4;
template <bool WIDE>
__global__ void __launch_bounds__(TC_WARPS * 32) tree_combine_kernel(const DecodeParams p) {
  constexpr int U = 8;
  __shared__ int s_sum[2][TC_WARPS];
  __shared__ float4 s_o[TC_WARPS][32];
  __shared__ float2 s_ml[TC_WARPS];
  const int b = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int col = WIDE ? blockIdx.x : blockIdx.x * TC_WARPS + warp;
  const int kvh = col / p.ncols, c = col - kvh * p.ncols;
  grid_dependency_wait();
  grid_dependents_launch();
  int before = 0, total = 0;   // tiles of the sequences before b, of all
  for (int i = threadIdx.x; i < p.B; i += TC_WARPS * 32) {
    const int t = (clamped_len(p, i) + tr::TOK - 1) / tr::TOK;
    total += t;
    if (i < b) before += t;
  }
  const int mine = (clamped_len(p, b) + tr::TOK - 1) / tr::TOK;
  before = __reduce_add_sync(0xffffffffu, before);
  total = __reduce_add_sync(0xffffffffu, total);
  if (lane == 0) s_sum[0][warp] = before, s_sum[1][warp] = total;
  __syncthreads();
  before = total = 0;
#pragma unroll
  for (int w = 0; w < TC_WARPS; ++w) before += s_sum[0][w], total += s_sum[1][w];
  if (mine == 0) return;
  const int S = min(p.n_splits, total);
  const int s0 = flat_cta_of(before, total, S), parts = flat_cta_of(before + mine - 1, total, S) - s0 + 1;
  if (parts == 1 || kvh >= p.Hkv) return;   // one share wrote O, or no such column
  const size_t stride = (size_t)p.ncols * kPartialStride;
  const float* base = p.partials + (((size_t)kvh * (p.n_splits + p.B - 1) + s0 + b) * p.ncols + c) * kPartialStride;
  constexpr int STEP = WIDE ? TC_WARPS : 1;
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
        ml[u] = __ldcg(reinterpret_cast<const float2*>(base + i * stride + 128));
        o[u] = __ldcg(reinterpret_cast<const float4*>(base + i * stride) + lane);
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
    for (int w = 1; w < TC_WARPS; ++w) add(s_ml[w], s_o[w][lane]);
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  if (p.stats != nullptr && lane == 0) p.stats[((size_t)b * p.Hkv + kvh) * p.ncols + c] = make_float2(M, inv);
  __half* dst = p.out + out_row(p, b, kvh, c) + 4 * lane;   // out needs only 2-byte alignment
  dst[0] = __float2half_rn(O.x * inv), dst[1] = __float2half_rn(O.y * inv);
  dst[2] = __float2half_rn(O.z * inv), dst[3] = __float2half_rn(O.w * inv);
}

using TreeKernel = void (*)(DecodeParams, const unsigned long long*, const uint4*);
template <int MODE>
TreeKernel tree_of(bool paged, int layout) {
  if (layout == kPairs)
    return paged ? (TreeKernel)decode_tree_kernel<MODE, true, 1, true> : (TreeKernel)decode_tree_kernel<MODE, false, 1, true>;
  if (layout == kTwoTiles)
    return paged ? (TreeKernel)decode_tree_kernel<MODE, true, 2> : (TreeKernel)decode_tree_kernel<MODE, false, 2>;
  return paged ? (TreeKernel)decode_tree_kernel<MODE, true, 1> : (TreeKernel)decode_tree_kernel<MODE, false, 1>;
}
TreeKernel tree_kernel(int mode, bool paged, int layout) {
  return mode == VQKV_MODE_VQ2    ? tree_of<VQKV_MODE_VQ2>(paged, layout)
         : mode == VQKV_MODE_VQ4  ? tree_of<VQKV_MODE_VQ4>(paged, layout)
         : mode == VQKV_MODE_VQ3  ? tree_of<VQKV_MODE_VQ3>(paged, layout)
         : mode == VQKV_MODE_VQ15 ? tree_of<VQKV_MODE_VQ15>(paged, layout)
                                  : tree_of<VQKV_MODE_VQ125>(paged, layout);
}
int tree_smem(int mode) {
  return mode == VQKV_MODE_VQ15 || mode == VQKV_MODE_VQ125 ? tr::Geo<VQKV_MODE_VQ15>::SMEM : tr::Geo<VQKV_MODE_VQ2>::SMEM;
}

}  // namespace

int decode_tree_cols(int ncols) { return ncols > tr::ROWS ? 2 * tr::ROWS : tr::ROWS; }

cudaError_t decode_tree_prepare(int mode) {
  cudaError_t e = cudaSuccess;
  for (int i = 0; i < 6 && e == cudaSuccess; ++i)
    e = prepare_split_kernel(tree_kernel(mode, (i & 1) != 0, i >> 1), tr::THREADS, tr::SPLIT_REGS, tree_smem(mode));
  return e;
}

size_t decode_tree_query_bytes(int B, int Hkv, int ncols, bool pairs) {
  const int w = pairs ? 16 : 32;
  return (size_t)B * Hkv * ((ncols + w - 1) / w) * 32 * kHeadDim * 2;
}

cudaError_t launch_decode_tree(int mode, const DecodeParams& p, const unsigned long long* tree_mask, bool pairs, void* qx,
                               cudaStream_t stream) {
  const int layout = pairs ? kPairs : p.ncols > tr::ROWS ? kTwoTiles : kOneTile;
  cudaError_t e = pairs ? launch_pdl(tree_query_kernel<true>, dim3((p.ncols + 15) / 16, p.Hkv, p.B), dim3(64), 0, stream, p,
                                     static_cast<uint4*>(qx))
                        : launch_pdl(tree_query_kernel<false>, dim3((p.ncols + 31) / 32, p.Hkv, p.B), dim3(128), 0, stream,
                                     p, static_cast<uint4*>(qx));
  if (e == cudaSuccess)
    e = launch_pdl(tree_kernel(mode, p.block_table != nullptr, layout), dim3(p.n_splits, p.Hkv, p.cgroups),
                   dim3(tr::THREADS), (size_t)tree_smem(mode), stream, p, tree_mask, static_cast<const uint4*>(qx));
  if (e == cudaSuccess && p.n_splits > 1) {
    const int cols = p.Hkv * p.ncols;
    if (p.n_splits > TC_WARPS * p.B)
      e = launch_pdl(tree_combine_kernel<true>, dim3(cols, p.B), dim3(TC_WARPS * 32), 0, stream, p);
    else
      e = launch_pdl(tree_combine_kernel<false>, dim3((cols + TC_WARPS - 1) / TC_WARPS, p.B), dim3(TC_WARPS * 32), 0, stream, p);
  }
  return e;
}

}  // namespace vqkv
