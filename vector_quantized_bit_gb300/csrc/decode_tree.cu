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
// warpgroups (64 scores and 16 packed weights are live), 56 for the
// dequantising ones (32 hold gathered centroids), 40 for the last:
// 256 x 120 + 512 x 56 + 128 x 40 = 64,512 = 896 x 72.  Two sets of code words
// beside the centroids do not fit in 56: 44 to 136 bytes per thread spill, 216 to
// 384 at 4 bit.
constexpr int REGS_SM = 120, REGS_DQ = 56, REGS_MMA = 40;
constexpr int SPLIT_REGS = 32 * (SM_WARPS * REGS_SM + DQ_WARPS * REGS_DQ + 4 * REGS_MMA);
constexpr int TILE_SMEM = TOK * 256;      // one dequantised K or V tile: two 64-channel halves of 64 x 128 bytes
constexpr int HALF = TOK * 128;
// tensor memory columns: O, S and P of each softmax warpgroup, then q'
constexpr uint32_t T_O = 0, T_S = 256, T_COLS = 512;
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
template <int NQ, int STAGES, bool PAIR>
__device__ __forceinline__ bool softmax_tiles_of(const DecodeParams& p, const Pieces& pc, uint32_t done, int wg, uint32_t t_lane,
                                                 unsigned long long mask, int prefix, uint32_t s_full, uint32_t s_ready,
                                                 uint32_t p_ready, uint32_t o_done, volatile int* abort_flag, float& m,
                                                 float& l) {
  using namespace tr;
  const int lane = threadIdx.x & 31;
  const uint32_t t_s = t_lane + T_S + TOK * wg, t_p = t_lane + Tmem<NQ>::p(wg), t_o = t_lane + T_O + kHeadDim * wg;
  bool first = true;
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
    if (__any_sync(0xffffffffu, top > m + kSoftmaxSlack)) {
      const float mn = fmaxf(m, top), f = fast_exp2(m - mn);
      m = mn;
      l *= f;
      if (!first) {
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

// grid (shares, Hkv, column groups of 128 NQ).
template <int MODE, bool PAGED, int NQ, bool PAIR = false>
__global__ void __launch_bounds__(tr::THREADS, 1) decode_tree_kernel(const DecodeParams p,
                                                                     const unsigned long long* tree_mask,
                                                                     const uint4* qx) {
  using namespace tr;
  using G = Geo<MODE>;
  using TM = Tmem<NQ>;
  extern __shared__ __align__(1024) unsigned char smem[];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  const int split = blockIdx.x, kvh = blockIdx.y;
  const int col0 = NQ * ROWS * (int)blockIdx.z, nloc = min(NQ * ROWS, p.ncols - col0);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // warps with columns in each softmax warpgroup (NQ 1: the same 128 columns)
  static_assert(!PAIR || NQ == 1, "pairs take one query tile");
  constexpr int WCOLS = PAIR ? 16 : 32;   // columns of a warp
  const int active0 = (min(nloc, ROWS) + WCOLS - 1) / WCOLS;
  const int active1 = NQ == 1 ? active0 : (max(nloc - ROWS, 0) + 31) >> 5;
  const int jobs = active1 > 0 ? 2 : 1;     // NQ 2: query tiles with columns
  const uint32_t bar = smem_u32(smem + G::BAR_OFF);
  // Per ring stage.  NQ 1: s_ready = K tile in place and the warpgroup's last
  // scores read, pv_ready = V tile and P in place (a tile's warpgroup follows
  // from its stage; one barrier each keeps the issuing warp at two waits per
  // tile).  NQ 2: s_ready = K tile, pv_ready = V tile.  Per softmax warpgroup:
  // s_full, o_done, and for NQ 2 p_ready.
  constexpr uint32_t ST = G::STAGES;
  const uint32_t s_ready = bar, k_empty = bar + 32, pv_ready = bar + 64, v_empty = bar + 96;
  const uint32_t s_full = bar + 128, o_done = bar + 144, p_ready = bar + 160, all_done = bar + 176;
  volatile int* abort_flag = &s_abort;
  int* s_pref = reinterpret_cast<int*>(smem + G::PREF_OFF);
  if (threadIdx.x == 0) {
    for (uint32_t i = 0; i < ST; ++i) {
      mbar_init(s_ready + 8 * i, (NQ == 1 ? 4 + active0 : 4) + ((int)i == p.withhold_stage));
      mbar_init(k_empty + 8 * i, NQ == 1 ? 1 : jobs);
      mbar_init(pv_ready + 8 * i, NQ == 1 ? 4 + active0 : 4);
      mbar_init(v_empty + 8 * i, NQ == 1 ? 1 : jobs);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(s_full + 8 * i, 1);
      mbar_init(o_done + 8 * i, 1);
      mbar_init(p_ready + 8 * i, max(i ? active1 : active0, 1));
    }
    mbar_init(all_done, 1);
    mbar_init(all_done + 8, 1);
    s_abort = 0;
    mbar_init_fence();
  }
  if (warp == MMA_WARP) tmem_alloc(smem_u32(&s_tmem), T_COLS);
  // The query kernel right before this one lets it start only when everything
  // before that has completed, and writes nothing but qx: the codebooks and
  // lengths may be read now, qx (and any output written) after the wait.
  fill_codebooks<MODE, THREADS, true>(p, kvh, smem);
  flat_prefix<TOK / 16>(p, s_pref);
  Pieces pc(s_pref, p.B, split, p.n_splits);
  grid_dependency_wait();
  grid_dependents_launch();
  for (int bb = split; bb < p.B; bb += gridDim.x)   // sequences without tokens
    if (s_pref[bb + 1] == s_pref[bb])
      for (int i = threadIdx.x; i < nloc * kHeadDim; i += THREADS)
        p.out[out_row(p, bb, kvh, col0 + i / kHeadDim) + (i & (kHeadDim - 1))] = __float2half_rn(0.f);
  tcgen05_before_sync();
  __syncthreads();
  tcgen05_after_sync();
  const uint32_t tmem = s_tmem;
  uint32_t done = 0;   // tiles of earlier pieces
  // Per piece the softmax warps and the issuing ones meet once: q' in tensor
  // memory, and the last piece's state read out of it.  (With the dequantising
  // warps meeting there as well, which waits out a memory latency per piece, 64
  // sequences of up to 512 tokens took 54 us, not 49.)
  constexpr int MEET = (SM_WARPS + 2) * 32;
  if (warp < SM_WARPS) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_SM));
    // ---------------- softmax warpgroup wg: thread = column c
    const int wg = warp >> 2, row = threadIdx.x & (ROWS - 1);
    const int cl = PAIR ? 16 * (warp & 3) + (lane & 15) : NQ == 1 ? row : wg * ROWS + row, c = col0 + cl;
    const bool live = (warp & 3) < (wg ? active1 : active0);
    const uint32_t t_lane = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    if (NQ == 1 && live && lane == 0) mbar_arrive(s_ready + 8 * wg);   // no scores to read yet
    bool ok = live;   // no wait has given up
    for (int piece = 0; pc.next(); ++piece) {
      if (live && (NQ == 2 || wg == 0)) {   // q' into tensor memory: lane = column
        const uint4* q = qx + ((((size_t)pc.b * p.Hkv + kvh) * ((p.ncols + WCOLS - 1) / WCOLS) + c / WCOLS) * 16) * 32 + lane;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t r[32];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint4 x = __ldcg(q + 32 * (8 * h + i));
            r[4 * i] = x.x, r[4 * i + 1] = x.y, r[4 * i + 2] = x.z, r[4 * i + 3] = x.w;
          }
          tmem_st32(t_lane + TM::q(wg) + 32 * h, r);
        }
        tmem_wait_st();
      }
      tcgen05_before_sync();
      named_barrier_sync(2, MEET);
      tcgen05_after_sync();
      float m = kMInit, l = 0.f;
      const int prefix = clamped_len(p, pc.b) - p.M;   // tokens below it are visible to every column
      if (ok) {
        unsigned long long mask = 0;
        if (cl < nloc) {
          const int q = c / p.g;   // no masks: causal queries
          mask = tree_mask != nullptr ? tree_mask[(size_t)pc.b * p.M + q] : (2ull << q) - 1;
          if (p.M < 64) mask &= (1ull << p.M) - 1;
        }
        ok = softmax_tiles_of<NQ, G::STAGES, PAIR>(p, pc, done, wg, t_lane, mask, prefix, s_full, s_ready, NQ == 1 ? pv_ready : p_ready,
                                  o_done, abort_flag, m, l);
        if (NQ == 1) {   // this warpgroup's last tile of the piece, if it has one
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
      const bool both = NQ == 1 && pc.n > 1;                        // both warpgroups had tiles
      const uint32_t own = NQ == 1 ? done & 1 : (uint32_t)wg;       // the O of the piece's first tile
      float fa = 1.f, fb = 0.f;
      if constexpr (NQ == 1) {
        float2* s_ml = reinterpret_cast<float2*>(smem + G::ML_OFF);
        s_ml[wg * ROWS + row] = make_float2(m, l);
        tcgen05_before_sync();
        named_barrier_sync(1, SM_WARPS * 32);   // both warpgroups' last products are done, too
        tcgen05_after_sync();
        const float2 a = s_ml[own * ROWS + row], z = s_ml[(own ^ 1) * ROWS + row];
        m = fmaxf(a.x, z.x);
        fa = fast_exp2(a.x - m), fb = fast_exp2(z.x - m);
        l = a.y * fa + z.y * fb;
      }
      if (ok && !*abort_flag) {
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
        for (int q = NQ == 1 ? 4 * wg : 0; q < (NQ == 1 ? 4 * wg + 4 : 8); ++q) {
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
                __half* dst = p.out + out_row(p, pc.b, kvh, c0 + r) + 16 * q + 4 * x;
                const uint2 h = make_uint2(pack_half2(w.x, w.y), pack_half2(w.z, w.w));
                if ((reinterpret_cast<uintptr_t>(dst) & 7) == 0) {
                  *reinterpret_cast<uint2*>(dst) = h;
                } else {   // out needs only 2-byte alignment
                  dst[0] = __ushort_as_half((unsigned short)h.x), dst[1] = __ushort_as_half((unsigned short)(h.x >> 16));
                  dst[2] = __ushort_as_half((unsigned short)h.y), dst[3] = __ushort_as_half((unsigned short)(h.y >> 16));
                }
              }
            }
          }
          __syncwarp();
        }
        if (cl < nloc && lane < WCOLS && (NQ == 2 || wg == 0)) {
          if (!whole)
            *reinterpret_cast<float2*>(part + lane * kPartialStride + 128) = make_float2(m, l);
          else if (p.stats != nullptr)
            p.stats[((size_t)pc.b * p.Hkv + kvh) * p.ncols + c] = make_float2(m, l > 0.f ? 1.f / l : 0.f);
        }
      }
      done += pc.n;
    }
  } else if (warp < MMA_WARP) {
    // ---------------- dequantisation
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_DQ));
    const int dw = warp - SM_WARPS, u = dw & 3, half = (dw >> 2) & 1;
    for (bool ok = true; ok && pc.next();) {
      const int L = clamped_len(p, pc.b);
      if (dw < 8)
        ok = dequant_piece<MODE, VQKV_ROLE_K, PAGED, TOK, G::STAGES>(p, pc.b, kvh, pc.tile0, pc.n, L, done, smem, smem + G::K_OFF,
                                                                     s_ready, k_empty, u, half, lane, abort_flag);
      else
        ok = dequant_piece<MODE, VQKV_ROLE_V, PAGED, TOK, G::STAGES>(p, pc.b, kvh, pc.tile0, pc.n, L, done, smem, smem + G::V_OFF,
                                                                     pv_ready, v_empty, u, half, lane, abort_flag);
      done += pc.n;
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_MMA));
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
      umma_commit(s_full + 8 * wg);
    };
    // O of warpgroup wg += P V: 16 tokens a step, two 8-token groups
    auto values = [&](uint32_t st, uint32_t wg, bool fresh) {
      const uint32_t lo = v_lo + st * (TILE_SMEM / 16), dv = tm + T_O + kHeadDim * wg, ap = tm + TM::p(wg);
#pragma unroll
      for (int k = 0; k < 4; ++k) umma_f16_ts(dv, ap + 8 * k, lo + k * (2048 / 16), v_hi, idesc_o, !fresh || k > 0);
    };
    bool ok = true;
    while (warp < MMA_WARP + 2 && pc.next()) {
      tcgen05_before_sync();
      named_barrier_sync(2, MEET);
      tcgen05_after_sync();
      const int n = pc.n;
      const int job = warp - MMA_WARP;
      if (NQ == 1 && job == 0) {
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
      } else if (NQ == 1 && job == 1) {
        for (int t = 0; ok && t < n; ++t) {
          const uint32_t k = done + t, st = k % ST;
          if (!(ok = tr_wait(p, pv_ready + 8 * st, (k / ST) & 1, abort_flag))) break;
          tcgen05_after_sync();
          if (issuer) {
            values(st, k & 1, t < 2);
            umma_commit(v_empty + 8 * st);
            umma_commit(o_done + 8 * (k & 1));
          }
          __syncwarp();
        }
      } else if (NQ == 2 && job < jobs) {
        for (int t = 0; ok && t <= n; ++t) {   // P.V of tile t - 1, then S of tile t
          const uint32_t k = done + t;
          if (t > 0) {
            const uint32_t j = k - 1, st = j % ST;
            ok = tr_wait(p, pv_ready + 8 * st, (j / ST) & 1, abort_flag) &&
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
            const uint32_t st = k % ST;
            if (!(ok = tr_wait(p, s_ready + 8 * st, (k / ST) & 1, abort_flag))) break;
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
enum TreeLayout : int { kOneTile = 0, kTwoTiles = 1, kPairs = 2 };   // columns on the MMA rows
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
