// The kernel of attention with many softmax columns over a packed cache (sm_103a,
// tcgen05): draft trees, windows of causal queries (decode_tree.cu) and cross
// attention (cross_attn.cu).  How it works and what bounds it: decode_tree.cu; what
// CROSS changes: cross_attn.cu.
#pragma once

#include <cuda_bf16.h>

#include <type_traits>

#include "common.cuh"
#include "decode_common.cuh"
#include "dequant_tile.cuh"
#include "gather.cuh"
#include "internal.h"
#include "umma.cuh"

namespace vqkv {
namespace {

namespace tr {
constexpr int ROWS = 128;                 // MMA rows: softmax columns of one query tile
constexpr int TOK = 64;                   // tokens per tile
constexpr int SM_WARPS = 8, DQ_WARPS = 16; // two softmax warpgroups, four dequantising ones
constexpr int MMA_WARP = SM_WARPS + DQ_WARPS;
constexpr int THREADS = (MMA_WARP + 4) * 32;   // whole warpgroups, for the register split
// Registers per thread: 72 at launch (896 threads), then 120 for the softmax
// warpgroups (64 scores and 16 packed weights are live), 56 for the dequantising
// ones (32 hold gathered centroids), 40 for the last.  Two sets of code words beside
// the centroids do not fit in 56: 44 to 136 bytes per thread spill.  At 4 bit, with
// twice the words, it would be 216 to 480: there 112, 64 and 24 (120 to 190 spill;
// ragged prompts over paged states 100 -> 93 us, 64 drafts over 32,768 tokens 51.3 ->
// 50.7; at 1.5 bit, where the softmax warps wait for conflicting gathers, a tree of 135
// columns would go from 192 to 212).  Either way 256, 512 and 128 threads hold 64,512 =
// 896 x 72.
template <int MODE>
struct Regs {
  static constexpr int SM = MODE == VQKV_MODE_VQ4 ? 112 : 120, DQ = MODE == VQKV_MODE_VQ4 ? 64 : 56, MMA = MODE == VQKV_MODE_VQ4 ? 24 : 40;
  static_assert(32 * (SM_WARPS * SM + DQ_WARPS * DQ + 4 * MMA) == THREADS * 72, "the launch's registers");
};
constexpr int SPLIT_REGS = THREADS * 72;
constexpr int TILE_SMEM = TOK * 256;      // one dequantised K or V tile: two 64-channel halves of 64 x 128 bytes
constexpr int HALF = TOK * 128;
// tensor memory columns: O, S and P of each softmax warpgroup, then q' (CROSS with
// both parts: one O, q's low parts, then the same)
constexpr uint32_t T_O = 0, T_Q_LOW = 128, T_S = 256, T_COLS = 512;
template <int NQ>
struct Tmem {
  __device__ static constexpr uint32_t p(uint32_t wg) { return NQ == 1 ? 384 + TOK / 2 * wg : T_S + TOK * wg; }
  __device__ static constexpr uint32_t q(uint32_t tile) { return NQ == 1 ? 448 : 384 + 64 * tile; }
};
template <int MODE>
struct Geo {
  static constexpr int CB_BYTES = MODE == VQKV_MODE_VQ15 || MODE == VQKV_MODE_VQ125 ? 131072 : 65536;
  // ring stages of K and of V: what fits beside the codebooks (tile k is in
  // stage k % STAGES and belongs to softmax warpgroup k % 2)
  static constexpr int STAGES = CB_BYTES == 65536 ? 4 : 2;
  static constexpr int K_OFF = CB_BYTES, V_OFF = K_OFF + STAGES * TILE_SMEM;
  static constexpr int BOX_OFF = V_OFF + STAGES * TILE_SMEM;   // 2 KB per softmax warp, for the epilogue
  static constexpr int BAR_OFF = BOX_OFF + SM_WARPS * 2048;
  static constexpr int ML_OFF = BAR_OFF + 256;             // the warpgroups' max and sum per column, for the merge
  static constexpr int PREF_OFF = ML_OFF + 2 * ROWS * 8;       // tiles of the sequences before each
  static constexpr int SMEM = PREF_OFF + (kFlatMaxB + 1) * 4;
  static_assert(SMEM <= 226 * 1024, "shared memory");
};
}  // namespace tr

// One warp of softmax warpgroup wg over a piece's tiles: thread = column.
// Returns false when a wait gave up.  m, l: the column's running max and sum.
// ONE_O: the warpgroups' tiles add to one O, so the running max goes from tile to
// tile: s_ml[warpgroup][column].x holds that after the warpgroup's last one, m_done
// (+ 32 wg + 8 warp) completes per tile.  l stays this warpgroup's own.
template <int NQ, int STAGES, bool PAIR, bool ONE_O, typename Work>
__device__ __forceinline__ bool softmax_tiles_of(const DecodeParams& p, const Work& pc, uint32_t done, int wg, uint32_t t_lane,
                                                 unsigned long long mask, int prefix, uint32_t s_full, uint32_t s_ready,
                                                 uint32_t p_ready, uint32_t o_done, uint32_t m_done, float2* s_ml,
                                                 volatile int* abort_flag, float& m, float& l) {
  using namespace tr;
  const int lane = threadIdx.x & 31, row = threadIdx.x & (ROWS - 1), w = row >> 5;
  const uint32_t t_s = t_lane + T_S + TOK * wg, t_p = t_lane + Tmem<NQ>::p(wg), t_o = t_lane + T_O + (ONE_O ? 0 : kHeadDim * wg);
  bool first = true;   // of this warpgroup
  // NQ 1: tiles whose number (counted over the CTA's pieces) has this parity; NQ 2: every tile
  for (int t = NQ == 1 ? (int)((done + wg) & 1) : 0; t < pc.n; t += NQ == 1 ? 2 : 1) {
    const uint32_t use = NQ == 1 ? (uint32_t)(done + t) >> 1 : (uint32_t)(done + t);
    if (!tr_wait(p, s_full + 8 * wg, use & 1, abort_flag)) return false;
    tcgen05_after_sync();
    float x[2][32], top0 = neg_inf(), top1 = neg_inf();
    if constexpr (PAIR) {
      tmem_ld32(t_s, x[0]);
      tmem_ld32(t_s + 32, x[1]);
      tmem_wait_ld();
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        x[0][i] += __shfl_xor_sync(0xffffffffu, x[0][i], 16);
        x[1][i] += __shfl_xor_sync(0xffffffffu, x[1][i], 16);
        top0 = fmaxf(top0, x[0][i]);
        top1 = fmaxf(top1, x[1][i]);
      }
    } else {
      tmem_ld32_max(t_s, x[0], top0);
      tmem_ld32_max(t_s + 32, x[1], top1);
      tmem_wait_ld();
    }
    if (NQ == 1) {   // the next score product may overwrite S
      tcgen05_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(s_ready + 8 * ((done + t + 2) % STAGES));
    }
    float top = fmaxf(top0, top1);
    const int d = prefix - (pc.tile0 + t) * TOK;
    if (d < TOK) {   // bit i of vis: token i of the tile is visible
      const unsigned long long vis = d >= 0 ? (mask << d) | ((1ull << d) - 1) : d > -64 ? mask >> -d : 0ull;
      top = neg_inf();
#pragma unroll
      for (int i = 0; i < 64; ++i) {
        if (!((vis >> i) & 1)) x[i >> 5][i & 31] = neg_inf();
        top = fmaxf(top, x[i >> 5][i & 31]);
      }
    }
    if (NQ == 1 && !first) {   // O and P of this warpgroup's previous tile are no longer in use
      if (!tr_wait(p, o_done + 8 * wg, (use - 1) & 1, abort_flag)) return false;
      tcgen05_after_sync();
    }                          // (NQ 2: this tile's score product came after that P.V product)
    if (ONE_O && t > 0) {   // the max after the tile before this one
      if (!tr_wait(p, m_done + 32 * (wg ^ 1) + 8 * w, ((done + t - 1) >> 1) & 1, abort_flag)) return false;
      const float mo = s_ml[(wg ^ 1) * ROWS + row].x;
      l *= fast_exp2(m - mo);
      m = mo;
    }
    const bool raise = __any_sync(0xffffffffu, top > m + kSoftmaxSlack);
    const float f = raise ? fast_exp2(m - fmaxf(m, top)) : 1.f;
    if (raise) m = fmaxf(m, top), l *= f;
    if constexpr (ONE_O) {
      s_ml[wg * ROWS + row].x = m;
      __syncwarp();
      if (lane == 0) mbar_arrive(m_done + 32 * wg + 8 * w);
    }
    if (raise) {
      if (ONE_O && t > 0) {   // O has every tile before this one
        if (!tr_wait(p, o_done + 8 * (wg ^ 1), ((done + t - 1) >> 1) & 1, abort_flag)) return false;
        tcgen05_after_sync();
      }
      if (ONE_O ? t > 0 : !first) {
#pragma unroll 1
        for (int q = 0; q < kHeadDim / 16; ++q) {
          uint32_t r[16];
          tmem_ld16(t_o + 16 * q, r);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * f);
          tmem_st16(t_o + 16 * q, r);
        }
      }
    }
    float2 sum = make_float2(0.f, 0.f);
    const float2 minus_m = make_float2(-m, -m);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t r[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float2 e = add_f32x2(make_float2(x[h][2 * i], x[h][2 * i + 1]), minus_m);
        e = make_float2(fast_exp2(e.x), fast_exp2(e.y));
        sum = add_f32x2(sum, e);
        r[i] = pack_half2(e.x, e.y);
      }
      tmem_st16(t_p + 16 * h, r);
    }
    l += sum.x + sum.y;
    tmem_wait_st();
    tcgen05_before_sync();
    __syncwarp();
    if (lane == 0) mbar_arrive(p_ready + 8 * (NQ == 1 ? (done + t) % STAGES : wg));
    first = false;
  }
  return true;
}

// Four consecutive values of an output row, whose address is a multiple of 2 bytes.
__device__ __forceinline__ void store_out4(__half* dst, float4 w) {
  const uint2 h = make_uint2(pack_half2(w.x, w.y), pack_half2(w.z, w.w));
  if ((reinterpret_cast<uintptr_t>(dst) & 7) == 0) {
    *reinterpret_cast<uint2*>(dst) = h;
  } else {
    dst[0] = __ushort_as_half((unsigned short)h.x), dst[1] = __ushort_as_half((unsigned short)(h.x >> 16));
    dst[2] = __ushort_as_half((unsigned short)h.y), dst[3] = __ushort_as_half((unsigned short)(h.y >> 16));
  }
}

// Cross attention: the first of the 32-column (PAIR: 16-column) groups of a sequence's
// queries in qx.
__host__ __device__ __forceinline__ long long cross_query_slot(int row0, int b, int g, int width) {
  return (long long)row0 * g / width + b;
}

// Cross attention: what a softmax warp does with its columns of a piece's O (row =
// column of the item in the lane's tensor memory from t_o on).  The output takes 32
// channels at a time, packed, through the warp's own 2 KB of shared memory (16-byte
// pieces permuted by the row), so that a row's stores are whole sectors; a partial
// goes out as [32 pieces of 4 channels][cols columns], neighbours as they are in the
// warp.  Quarters q0 .. q1 - 1 of the channels.  (Eight rounds of 16 channels with a
// row's address computed in each took 5.5 us of a piece.)
template <int WCOLS>
__device__ __forceinline__ void cross_finish(const DecodeParams& p, bool whole, uint32_t t_o, float m, float l, int q0, int q1,
                                             uint4* box, float4* part, int cols, int cl, int nloc, int col0, int row0, int kvh) {
  const int lane = threadIdx.x & 31, cl0 = cl & ~(WCOLS - 1);
  const bool mine = cl < nloc && lane < WCOLS;
  if (cl0 >= nloc) return;   // the same for the whole warp
  if (!whole) {
#pragma unroll 1
    for (int q = q0; q < q1; ++q) {
      float v[32];
      tmem_ld32(t_o + 32 * q, v);
      tmem_wait_ld();
      if (mine) {
#pragma unroll
        for (int i = 0; i < 8; ++i) part[(8 * q + i) * cols + cl] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
      }
    }
    if (mine && q0 == 0) reinterpret_cast<float2*>(part + 32 * cols)[cl] = make_float2(m, l);
    return;
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  const int x = lane & 3;   // 16-byte piece of the rows 8 i + lane / 4
  const bool wide = (reinterpret_cast<uintptr_t>(p.out) & 15) == 0;   // out needs only 2-byte alignment
  __half* dst[WCOLS / 8];
#pragma unroll
  for (int i = 0; i < WCOLS / 8; ++i) {
    const int c = cl0 + 8 * i + (lane >> 2);
    dst[i] = c < nloc ? p.out + cross_out_row(p, row0, kvh, col0 + c) + 8 * x : nullptr;
  }
#pragma unroll 1
  for (int q = q0; q < q1; ++q) {
    float v[32];
    tmem_ld32(t_o + 32 * q, v);
    tmem_wait_ld();
    uint32_t w[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if (p.bf16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i] * inv, v[2 * i + 1] * inv);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      } else {
        w[i] = pack_half2(v[2 * i] * inv, v[2 * i + 1] * inv);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      box[lane * 4 + (i ^ ((lane >> 1) & 3))] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < WCOLS / 8; ++i) {
      const int r = 8 * i + (lane >> 2);
      const uint4 h = box[r * 4 + (x ^ ((r >> 1) & 3))];
      if (dst[i] == nullptr) continue;
      if (wide) {
        *reinterpret_cast<uint4*>(dst[i] + 32 * q) = h;
      } else {
        const uint32_t e[4] = {h.x, h.y, h.z, h.w};
#pragma unroll
        for (int k = 0; k < 8; ++k) dst[i][32 * q + k] = __ushort_as_half((unsigned short)(e[k >> 1] >> (16 * (k & 1))));
      }
    }
    __syncwarp();
  }
}

// What the kernel attends: a tree or causal queries; a cross attention, whose scores
// take both fp16 parts of q', with items of 64 columns (pairs) or of 128.
enum CrossKind : int { kNoCross = 0, kCrossPairs = 1, kCrossParts = 2 };

// grid (shares, Hkv, column groups of 128 NQ; CROSS: 1).
template <int MODE, bool PAGED, int NQ, bool PAIR = false, int CROSS = kNoCross>
__global__ void __launch_bounds__(tr::THREADS, 1) decode_tree_kernel(const DecodeParams p,
                                                                     const unsigned long long* tree_mask,
                                                                     const uint4* qx) {
  using namespace tr;
  using G = Geo<MODE>;
  // Cross attention of items of 64 columns: the softmax warpgroups work on two
  // shares, each with items, tiles and half of the ring's stages of its own, so that
  // one's passage to its next item (q', first tile, O) hides behind the other's
  // products.  Tensor memory is dealt out as for two query tiles (P overlays S).
  constexpr bool STREAMS = CROSS == kCrossPairs;
  // Both fp16 parts of q': the low ones take the place of the second O, and the two
  // warpgroups' tiles add to one O.  (With two of them and P over S, so that a
  // warpgroup's next scores wait for its P V, a tile took 1,520 cycles, not 1,330.)
  constexpr bool ONE_O = CROSS == kCrossParts;
  static_assert(!CROSS || (NQ == 1 && PAIR == STREAMS), "cross attention: pairs, or one query tile of both parts of q'");
  constexpr int TQ = STREAMS ? 2 : NQ;
  using TM = Tmem<TQ>;
  extern __shared__ __align__(1024) unsigned char smem[];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  const int split = blockIdx.x, kvh = blockIdx.y;
  constexpr int COLS = PAIR ? 64 : NQ * ROWS;   // CROSS: columns of an item
  const int grp0 = CROSS ? 0 : NQ * ROWS * (int)blockIdx.z, width = min(NQ * ROWS, p.ncols - grp0);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // warps with columns in each softmax warpgroup (NQ 1: the same 128 columns)
  static_assert(!PAIR || NQ == 1, "pairs take one query tile");
  constexpr int WCOLS = PAIR ? 16 : 32;   // columns of a warp
  const int active0 = (min(width, ROWS) + WCOLS - 1) / WCOLS;
  const int active1 = NQ == 1 ? active0 : (max(width - ROWS, 0) + 31) >> 5;
  const int jobs = active1 > 0 ? 2 : 1;     // NQ 2: query tiles with columns
  const uint32_t bar = smem_u32(smem + G::BAR_OFF);
  // Per ring stage.  NQ 1: s_ready = K tile in place and the warpgroup's last
  // scores read, pv_ready = V tile and P in place (a tile's warpgroup follows
  // from its stage; one barrier each keeps the issuing warp at two waits per
  // tile).  NQ 2: s_ready = K tile, pv_ready = V tile.  Per softmax warpgroup:
  // s_full, o_done, and for NQ 2 p_ready.  (STREAMS: as NQ 2, stage 2 i + h is stream
  // h's i-th.)  ONE_O: m_done, per softmax warp.
  constexpr uint32_t ST = G::STAGES;
  const uint32_t s_ready = bar, k_empty = bar + 32, pv_ready = bar + 64, v_empty = bar + 96;
  const uint32_t s_full = bar + 128, o_done = bar + 144, p_ready = bar + 160, all_done = bar + 176;
  const uint32_t m_done = bar + 192;
  volatile int* abort_flag = &s_abort;
  int* s_pref = reinterpret_cast<int*>(smem + G::PREF_OFF);
  float2* s_ml = reinterpret_cast<float2*>(smem + G::ML_OFF);
  if (threadIdx.x == 0) {
    for (uint32_t i = 0; i < ST; ++i) {
      mbar_init(s_ready + 8 * i, (TQ == 1 ? 4 + active0 : 4) + ((int)i == p.withhold_stage));
      mbar_init(k_empty + 8 * i, NQ == 1 ? 1 : jobs);
      mbar_init(pv_ready + 8 * i, TQ == 1 ? 4 + active0 : 4);
      mbar_init(v_empty + 8 * i, NQ == 1 ? 1 : jobs);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(s_full + 8 * i, 1);
      mbar_init(o_done + 8 * i, 1);
      mbar_init(p_ready + 8 * i, max(i ? active1 : active0, 1));
    }
    mbar_init(all_done, 1);
    mbar_init(all_done + 8, 1);
    if (ONE_O)
      for (int i = 0; i < SM_WARPS; ++i) mbar_init(m_done + 8 * i, 1);
    s_abort = 0;
    mbar_init_fence();
  }
  if (warp == MMA_WARP) tmem_alloc(smem_u32(&s_tmem), T_COLS);
  // The query kernel right before this one lets it start only when everything
  // before that has completed, and writes nothing but qx: the codebooks and
  // lengths may be read now, qx (and any output written) after the wait.
  fill_codebooks<MODE, THREADS, true>(p, kvh, smem);
  if constexpr (CROSS)
    item_prefix<TOK>(p, COLS, s_pref, blockIdx.x == 0 && blockIdx.y == 0);
  else
    flat_prefix<TOK / 16>(p, s_pref);
  // CROSS: this warp's share.  STREAMS: that of a softmax or dequantising warpgroup, or of an issuing warp
  const int share = STREAMS ? 2 * split + (warp < MMA_WARP ? (warp >> 2) & 1 : warp & 1) : split;
  auto pc = [&] {
    if constexpr (CROSS)
      return ItemPieces<TOK, COLS>(p, s_pref, share, p.n_splits);
    else
      return Pieces(s_pref, p.B, split, p.n_splits);
  }();
  grid_dependency_wait();
  grid_dependents_launch();
  for (int bb = split; bb < p.B; bb += gridDim.x)   // sequences without tokens
    if (s_pref[bb + 1] == s_pref[bb]) {
      if constexpr (CROSS) {   // (or without queries)
        const RowRange rows = row_range(p, bb, false);
        for (long long i = threadIdx.x; i < (long long)rows.n * p.g * kHeadDim; i += THREADS)
          p.out[cross_out_row(p, rows.first, kvh, (int)(i / kHeadDim)) + (i & (kHeadDim - 1))] = __float2half_rn(0.f);
      } else {
        for (int i = threadIdx.x; i < width * kHeadDim; i += THREADS)
          p.out[out_row(p, bb, kvh, grp0 + i / kHeadDim) + (i & (kHeadDim - 1))] = __float2half_rn(0.f);
      }
    }
  tcgen05_before_sync();
  __syncthreads();
  tcgen05_after_sync();
  const uint32_t tmem = s_tmem;
  uint32_t done = 0;   // tiles of earlier pieces
  // Per piece the softmax warps and the issuing ones meet once: q' in tensor
  // memory, and the last piece's state read out of it.  (With the dequantising
  // warps meeting there as well, which waits out a memory latency per piece, 64
  // sequences of up to 512 tokens took 54 us, not 49.)
  constexpr int MEET = STREAMS ? (SM_WARPS / 2 + 1) * 32 : (SM_WARPS + 2) * 32;
  if (warp < SM_WARPS) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Regs<MODE>::SM));
    // ---------------- softmax warpgroup wg: thread = column c
    const int wg = warp >> 2, row = threadIdx.x & (ROWS - 1);
    const int cl = PAIR ? 16 * (warp & 3) + (lane & 15) : NQ == 1 ? row : wg * ROWS + row;
    const bool live = (warp & 3) < (wg ? active1 : active0);
    const uint32_t t_lane = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    if (TQ == 1 && live && lane == 0) mbar_arrive(s_ready + 8 * wg);   // no scores to read yet
    bool ok = live;   // no wait has given up
    for (int piece = 0; pc.next(); ++piece) {
      int col0 = grp0, nloc = width, row0 = 0;   // the piece's first column, its columns; CROSS: its sequence's first row
      size_t qrow;                               // of this warp's columns in qx
      if constexpr (CROSS) {
        const RowRange rows = row_range(p, pc.b, false);
        row0 = rows.first;
        col0 = pc.group * COLS;
        nloc = min(COLS, rows.n * p.g - col0);
        qrow = (size_t)kvh * (cross_query_slot(p.n_rows, p.B, p.g, WCOLS) + 1) + cross_query_slot(row0, pc.b, p.g, WCOLS) +
               (col0 + cl) / WCOLS;
      } else {
        qrow = ((size_t)pc.b * p.Hkv + kvh) * ((p.ncols + WCOLS - 1) / WCOLS) + (col0 + cl) / WCOLS;
      }
      const int c = col0 + cl;
      // q' into tensor memory: lane = column (ONE_O: warpgroup 0 the high parts, 1 the low
      // ones).  CROSS: zeros for the columns past the last, which share a warp, and with it
      // the decision to raise the running max, but have nothing in qx: what an earlier call
      // left there would move the others' roundings.
      if (live && (cl & ~(WCOLS - 1)) < nloc && (TQ == 2 || wg == 0 || ONE_O)) {
        const uint4* q = qx + (ONE_O ? 2 * qrow + wg : qrow) * 16 * 32 + lane;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t r[32];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint4 x = !CROSS || cl < nloc ? __ldcg(q + 32 * (8 * h + i)) : make_uint4(0u, 0u, 0u, 0u);
            r[4 * i] = x.x, r[4 * i + 1] = x.y, r[4 * i + 2] = x.z, r[4 * i + 3] = x.w;
          }
          tmem_st32(t_lane + (ONE_O && wg ? T_Q_LOW : TM::q(wg)) + 32 * h, r);
        }
        tmem_wait_st();
      }
      tcgen05_before_sync();
      named_barrier_sync(STREAMS ? 2 + wg : 2, MEET);
      tcgen05_after_sync();
      float m = kMInit, l = 0.f;
      const int prefix = clamped_len(p, pc.b) - (CROSS ? 0 : p.M);   // tokens below it are visible to every column
      if (ok) {
        unsigned long long mask = 0;
        if (!CROSS && cl < nloc) {
          const int q = c / p.g;   // no masks: causal queries
          mask = tree_mask != nullptr ? tree_mask[(size_t)pc.b * p.M + q] : (2ull << q) - 1;
          if (p.M < 64) mask &= (1ull << p.M) - 1;
        }
        ok = softmax_tiles_of<TQ, G::STAGES, PAIR, ONE_O>(p, pc, done, wg, t_lane, mask, prefix, s_full, s_ready,
                                                          TQ == 1 ? pv_ready : p_ready, o_done, m_done, s_ml, abort_flag, m, l);
        if (TQ == 1) {   // this warpgroup's last tile of the piece, if it has one
          const int last = pc.n - 1 - (int)((done + pc.n - 1 + wg) & 1);
          if (ok && last >= 0) ok = tr_wait(p, o_done + 8 * wg, ((done + last) >> 1) & 1, abort_flag);
        } else if (ok) {
          ok = tr_wait(p, o_done + 8 * wg, piece & 1, abort_flag);
        }
        tcgen05_after_sync();
      }
      // NQ 1: the two warpgroups' states are merged.  Both O's rows are in the
      // same tensor-memory lanes, so each warp reads both and takes half of the
      // channels; the maxima and sums pass through shared memory.
      const bool both = TQ == 1 && !ONE_O && pc.n > 1;             // both warpgroups had tiles, and an O each
      const uint32_t own = TQ == 1 ? done & 1 : (uint32_t)wg;      // the O of the piece's first tile
      float fa = 1.f, fb = 0.f;
      if constexpr (TQ == 1) {
        s_ml[wg * ROWS + row] = make_float2(m, l);
        tcgen05_before_sync();
        named_barrier_sync(1, SM_WARPS * 32);   // both warpgroups' last products are done, too
        tcgen05_after_sync();
        const float2 a = s_ml[own * ROWS + row], z = s_ml[(own ^ 1) * ROWS + row];
        m = fmaxf(a.x, z.x);
        fa = fast_exp2(a.x - m), fb = fast_exp2(z.x - m);
        l = a.y * fa + z.y * fb;
        if (ONE_O) fa = 1.f;   // O is relative to the last tile's max, the larger one
      }
      if constexpr (CROSS) {
        // a share has a piece that began before it, and one that ends behind it, at most
        if (ok && !*abort_flag)
          cross_finish<WCOLS>(p, pc.n == pc.all, t_lane + T_O + (STREAMS || NQ == 2 ? kHeadDim * wg : 0), m, l,
                              ONE_O ? 2 * wg : 0, ONE_O ? 2 * wg + 2 : 4, reinterpret_cast<uint4*>(smem + G::BOX_OFF) + warp * 128,
                              reinterpret_cast<float4*>(p.partials) +
                                  (((size_t)kvh * p.n_splits + share) * 2 + (pc.tile0 == 0)) * (COLS * kPartialStride / 4),
                              COLS, cl, nloc, col0, row0, kvh);
      } else if (ok && !*abort_flag) {
        const bool whole = pc.n == pc.all;
        if (whole) {
          const float inv = l > 0.f ? 1.f / l : 0.f;
          fa *= inv, fb *= inv;
        }
        // 16 channels at a time, transposed through the warp's own shared memory so
        // that a row's stores are neighbours; 16-byte pieces permuted by the row
        const int c0 = c - (lane & (WCOLS - 1));   // the warp's first column
        float* box = reinterpret_cast<float*>(smem + G::BOX_OFF) + warp * (32 * 16);
        float* part = p.partials + (((size_t)kvh * (p.n_splits + p.B - 1) + split + pc.b) * p.ncols + c0) * kPartialStride;
#pragma unroll 1
        for (int q = TQ == 1 ? 4 * wg : 0; q < (TQ == 1 ? 4 * wg + 4 : 8); ++q) {
          uint32_t o[16], z[16];
          tmem_ld16(t_lane + T_O + kHeadDim * own + 16 * q, o);
          if (both) tmem_ld16(t_lane + T_O + kHeadDim * (own ^ 1) + 16 * q, z);
          tmem_wait_ld();
          float v[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(o[i]) * fa;
          if (both) {
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] += __uint_as_float(z[i]) * fb;
          }
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *reinterpret_cast<float4*>(box + lane * 16 + ((i ^ ((lane >> 1) & 3)) << 2)) =
                make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
          __syncwarp();
          const int x = lane & 3;   // 16-byte piece of the rows 8 i + lane / 4
          if (!whole) {
            float* dst = part + (lane >> 2) * kPartialStride + 16 * q + 4 * x;
#pragma unroll
            for (int i = 0; i < WCOLS / 8; ++i) {
              const int r = 8 * i + (lane >> 2);
              if (c0 - col0 + r < nloc)
                *reinterpret_cast<float4*>(dst + 8 * i * kPartialStride) =
                    *reinterpret_cast<const float4*>(box + r * 16 + ((x ^ ((r >> 1) & 3)) << 2));
            }
          } else {
#pragma unroll
            for (int i = 0; i < WCOLS / 8; ++i) {
              const int r = 8 * i + (lane >> 2);
              if (c0 - col0 + r < nloc) {
                const float4 w = *reinterpret_cast<const float4*>(box + r * 16 + ((x ^ ((r >> 1) & 3)) << 2));
                store_out4(p.out + out_row(p, pc.b, kvh, c0 + r) + 16 * q + 4 * x, w);
              }
            }
          }
          __syncwarp();
        }
        if (cl < nloc && lane < WCOLS && (TQ == 2 || wg == 0)) {
          if (!whole)
            *reinterpret_cast<float2*>(part + lane * kPartialStride + 128) = make_float2(m, l);
          else if (p.stats != nullptr)
            p.stats[((size_t)pc.b * p.Hkv + kvh) * p.ncols + c] = make_float2(m, l > 0.f ? 1.f / l : 0.f);
        }
      }
      done += pc.n;
    }
    if constexpr (CROSS) {   // the item that this share begins and does not end, for the merge
      if (kvh == 0 && (threadIdx.x & (ROWS - 1)) == 0 && (STREAMS || wg == 0) && share < p.n_splits)
        reinterpret_cast<int4*>(p.tickets)[share] = pc.split_item(share, p.n_splits);
    }
  } else if (warp < MMA_WARP) {
    // ---------------- dequantisation
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Regs<MODE>::DQ));
    const int dw = warp - SM_WARPS, u = dw & 3, half = (dw >> 2) & 1;
    for (bool ok = true; ok && pc.next();) {
      const int L = clamped_len(p, pc.b);
      if (dw < 8)
        ok = dequant_piece<MODE, VQKV_ROLE_K, PAGED, TOK, G::STAGES, STREAMS>(p, pc.b, kvh, pc.tile0, pc.n, L, done, smem, smem + G::K_OFF,
                                                                     s_ready, k_empty, u, half, lane, abort_flag);
      else
        ok = dequant_piece<MODE, VQKV_ROLE_V, PAGED, TOK, G::STAGES, STREAMS>(p, pc.b, kvh, pc.tile0, pc.n, L, done, smem, smem + G::V_OFF,
                                                                     pv_ready, v_empty, u, half, lane, abort_flag);
      done += pc.n;
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Regs<MODE>::MMA));
    // ---------------- the products.  An issuing warp waits and computes the
    // operands' addresses as one, so they stay in uniform registers, and an
    // elected lane issues.  Issue blocks while the tensor cores are busy, so
    // two warps share it, one waiting while the other's products run: NQ 1,
    // score products and P.V products; NQ 2, query tile 0 and query tile 1 (a
    // tile's score product must follow its last P.V product: same warp, in
    // order).
    constexpr uint32_t idesc_s = umma_idesc_f16_f32(ROWS, TOK);
    constexpr uint32_t idesc_o = umma_idesc_f16_f32(ROWS, kHeadDim) | kIdescBMnMajor;
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    const uint64_t k_desc = umma_desc_sw128(smem_u32(smem + G::K_OFF), 1024, 16);
    const uint64_t v_desc = umma_desc_sw128(smem_u32(smem + G::V_OFF), 1024, HALF);
    const uint32_t k_lo = (uint32_t)k_desc, k_hi = (uint32_t)(k_desc >> 32);
    const uint32_t v_lo = (uint32_t)v_desc, v_hi = (uint32_t)(v_desc >> 32);
    const bool issuer = elect_one();
    // S of warpgroup wg (query tile qt) from the K tile in stage st: 16
    // channels a step, 32 bytes of a 128-byte row, four per 64-channel half
    auto scores = [&](uint32_t st, uint32_t wg, uint32_t qt) {
      const uint32_t lo = k_lo + st * (TILE_SMEM / 16), ds = tm + T_S + TOK * wg, aq = tm + TM::q(qt);
#pragma unroll
      for (int k = 0; k < 8; ++k)
        umma_f16_ts(ds, aq + 8 * k, lo + ((k >> 2) * HALF + (k & 3) * 32) / 16, k_hi, idesc_s, k > 0);
      if constexpr (ONE_O) {   // the low parts of q'
#pragma unroll
        for (int k = 0; k < 8; ++k)
          umma_f16_ts(ds, tm + T_Q_LOW + 8 * k, lo + ((k >> 2) * HALF + (k & 3) * 32) / 16, k_hi, idesc_s, true);
      }
      umma_commit(s_full + 8 * wg);
    };
    // O of warpgroup wg += P V: 16 tokens a step, two 8-token groups
    auto values = [&](uint32_t st, uint32_t wg, bool fresh) {
      const uint32_t lo = v_lo + st * (TILE_SMEM / 16), dv = tm + T_O + (ONE_O ? 0 : kHeadDim * wg), ap = tm + TM::p(wg);
#pragma unroll
      for (int k = 0; k < 4; ++k) umma_f16_ts(dv, ap + 8 * k, lo + k * (2048 / 16), v_hi, idesc_o, !fresh || k > 0);
    };
    bool ok = true;
    while (warp < MMA_WARP + 2 && pc.next()) {
      const int job = warp - MMA_WARP;
      const int n = pc.n;
      tcgen05_before_sync();
      named_barrier_sync(STREAMS ? 2 + job : 2, MEET);
      tcgen05_after_sync();
      if (TQ == 1 && job == 0) {
        for (int t = 0; ok && t < n; ++t) {
          const uint32_t k = done + t, st = k % ST;
          if (!(ok = tr_wait(p, s_ready + 8 * st, (k / ST) & 1, abort_flag))) break;
          tcgen05_after_sync();
          if (issuer) {
            scores(st, k & 1, 0);
            umma_commit(k_empty + 8 * st);
          }
          __syncwarp();
        }
      } else if (TQ == 1 && job == 1) {
        for (int t = 0; ok && t < n; ++t) {
          const uint32_t k = done + t, st = k % ST;
          if (!(ok = tr_wait(p, pv_ready + 8 * st, (k / ST) & 1, abort_flag))) break;
          tcgen05_after_sync();
          if (issuer) {
            values(st, k & 1, ONE_O ? t == 0 : t < 2);
            umma_commit(v_empty + 8 * st);
            umma_commit(o_done + 8 * (k & 1));
          }
          __syncwarp();
        }
      } else if (TQ == 2 && job < jobs) {
        // stage and use of it of tile j
        auto stage = [&](uint32_t j) { return STREAMS ? 2 * (j % (ST / 2)) + job : j % ST; };
        auto round = [&](uint32_t j) { return STREAMS ? j / (ST / 2) : j / ST; };
        for (int t = 0; ok && t <= n; ++t) {   // P.V of tile t - 1, then S of tile t
          const uint32_t k = done + t;
          if (t > 0) {
            const uint32_t j = k - 1, st = stage(j);
            ok = tr_wait(p, pv_ready + 8 * st, round(j) & 1, abort_flag) &&
                 tr_wait(p, p_ready + 8 * job, j & 1, abort_flag);
            if (!ok) break;
            tcgen05_after_sync();
            if (issuer) {
              values(st, job, t == 1);
              umma_commit(v_empty + 8 * st);
              if (t == n) umma_commit(o_done + 8 * job);
            }
            __syncwarp();
          }
          if (t < n) {
            const uint32_t st = stage(k);
            if (!(ok = tr_wait(p, s_ready + 8 * st, round(k) & 1, abort_flag))) break;
            tcgen05_after_sync();
            if (issuer) {
              scores(st, job, job);
              umma_commit(k_empty + 8 * st);
            }
            __syncwarp();
          }
        }
      }
      done += n;
    }
    if (warp < MMA_WARP + 2) drain_products(p, issuer, all_done + 8 * (warp - MMA_WARP));
  }
  __syncwarp();
  tcgen05_before_sync();
  __syncthreads();
  tcgen05_after_sync();
  if (warp == MMA_WARP) tmem_dealloc(tmem, T_COLS);
}

}  // namespace
}  // namespace vqkv
