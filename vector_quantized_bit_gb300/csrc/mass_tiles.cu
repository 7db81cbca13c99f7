// Attention weights of many softmax columns (vqkv_decode_attn_mass beyond a
// few columns per KV head): tokens as MMA rows, columns as MMA columns.
//
// The decode kernels behind vqkv_decode_attn_mass carry 4 columns per CTA and
// gather every centroid again for each group of 4.  Here one dequantisation
// serves all (up to 64) columns.  The draft-tree attention (paired q' parts) has
// written O and left each column's max m_c and 1 / l_c; one pass over the keys
// alone follows:
//   mass_t += sum_c exp2(s_tc - m_c) / l_c
// It recomputes the scores S = K' [Q'hi Q'lo]^T (128 tokens x 2 columns x 128
// channels) with q' = hi + lo split into two fp16 parts, off by at most
// max(2^-22 |q'|, 2^-25) per channel: near what fp32 keeps of q' down to 2^-3, an
// absolute 2^-25 below.  A thread owns a token (tensor-memory lane): the sum over
// columns is in one thread, in order.
// The alternative, storing the scores, would move 512 bytes per token and KV
// head at 64 columns; the second pass moves its key codes (32 bytes at 2 bit).
//
// What bounds the pass: shared memory (a K' tile is gathered, stored and read
// by the tensor cores, 256 bytes a token each) next to the exponentials: 1,480
// cycles per 128 tokens of 64 columns at 3 bit, 32 us for 4 sequences of up to
// 16,384 tokens and 8 KV heads (the attention before it takes 51 us).
#include "dequant_tile.cuh"

namespace vqkv {
namespace {

namespace mt {
constexpr int TOK = 128;                   // tokens per tile (MMA rows)
constexpr int EP_WARPS = 8, DQ_WARPS = 16; // two epilogue warpgroups; K groups of 16 tokens x 2 tiles in flight
constexpr int MMA_WARP = EP_WARPS + DQ_WARPS;
constexpr int THREADS = (MMA_WARP + 4) * 32;
// As in the draft-tree attention: 256 x 120 + 512 x 56 + 128 x 40 = 896 x 72.  The
// dequantising warps spill 44 to 92 bytes per thread, 112 to 220 at 4 bit.
constexpr int REGS_EP = 120, REGS_DQ = 56, REGS_MMA = 40;
constexpr int SPLIT_REGS = 32 * (EP_WARPS * REGS_EP + DQ_WARPS * REGS_DQ + 4 * REGS_MMA);
constexpr int STAGES = 3;
constexpr int TILE_SMEM = TOK * 256, HALF = TOK * 128;
constexpr int MAX_COLS = 64;
constexpr int CB_BYTES = 65536;            // K codebook at the places of the decode (its V half unused)
constexpr int K_OFF = CB_BYTES, Q_OFF = K_OFF + STAGES * TILE_SMEM;
constexpr int Q_BYTES = 2 * MAX_COLS * 256;
constexpr int COL_OFF = Q_OFF + Q_BYTES;   // per column: m, 1 / l (float2), then the visible length (int)
constexpr int BAR_OFF = COL_OFF + MAX_COLS * 12;
constexpr int PREF_OFF = BAR_OFF + 128;
constexpr int SMEM = PREF_OFF + (kFlatMaxB + 1) * 4;
static_assert(SMEM <= 226 * 1024, "shared memory");
constexpr uint32_t T_COLS = 256;           // two score accumulators of up to 128 columns
}  // namespace mt

// B operand of the score product, one image per (sequence, KV head) in the
// layout it has in shared memory: NC rows of q' hi, NC rows of q' lo (zeros past
// the last column), two 64-channel halves of 128-byte rows, 16-byte pieces
// swizzled by the row.  grid (NC / 32, Hkv, B), 128 threads.
template <int NC>
__global__ void __launch_bounds__(128) mass_query_kernel(const DecodeParams p, unsigned char* image) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int kvh = blockIdx.y, b = blockIdx.z, part = threadIdx.x & 3, c = 32 * blockIdx.x + (threadIdx.x >> 2);
  float v[32];
  transform_column(p, b, kvh, c, part, v);
  unsigned char* img = image + ((size_t)b * p.Hkv + kvh) * (2 * NC * 256) + (part >> 1) * (2 * NC * 128);
#pragma unroll
  for (int j = 0; j < 4; ++j) {   // pieces 4 (part % 2) + j of the half
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = v[8 * j + 2 * i], z = v[8 * j + 2 * i + 1];
      const __half2 h = __floats2half2_rn(a, z);
      hi[i] = *reinterpret_cast<const uint32_t*>(&h);
      lo[i] = pack_half2(a - __low2float(h), z - __high2float(h));
    }
    const int piece = 4 * (part & 1) + j;
    *reinterpret_cast<uint4*>(img + c * 128 + ((piece ^ (c & 7)) << 4)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    const int r = NC + c;
    *reinterpret_cast<uint4*>(img + r * 128 + ((piece ^ (r & 7)) << 4)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  }
}

// The weights of every token, added to p.mass.  grid (shares, Hkv); the shares
// cut all sequences' 128-token tiles.
template <int MODE, bool PAGED, int NC>
__global__ void __launch_bounds__(mt::THREADS, 1) mass_tile_kernel(const DecodeParams p, const unsigned char* image) {
  using namespace mt;
  extern __shared__ __align__(1024) unsigned char smem[];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort, s_skip;
  const int split = blockIdx.x, kvh = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t bar = smem_u32(smem + BAR_OFF);
  const uint32_t k_full = bar, k_empty = bar + 24, d_full = bar + 48, d_empty = bar + 64, all_done = bar + 80;
  volatile int* abort_flag = &s_abort;
  int* s_pref = reinterpret_cast<int*>(smem + PREF_OFF);
  float2* s_col = reinterpret_cast<float2*>(smem + COL_OFF);
  int* s_lim = reinterpret_cast<int*>(smem + COL_OFF + MAX_COLS * 8);
  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(k_full + 8 * i, 8 + (i == p.withhold_key_stage));
      mbar_init(k_empty + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(d_full + 8 * i, 1);
      mbar_init(d_empty + 8 * i, 4);
    }
    mbar_init(all_done, 1);
    s_abort = 0;
    mbar_init_fence();
  }
  if (warp == MMA_WARP) tmem_alloc(smem_u32(&s_tmem), T_COLS);
  // codebooks and lengths are inputs that no kernel of this call writes, and the
  // attention's last kernel started only when everything before the call had completed
  fill_codebooks<MODE, THREADS, false>(p, kvh, smem);
  flat_prefix<TOK / 16>(p, s_pref);
  Pieces pc(s_pref, p.B, split, p.n_splits);
  grid_dependency_wait();
  grid_dependents_launch();
  if (threadIdx.x == 0) s_skip = timed_out(p);   // one answer for all roles
  tcgen05_before_sync();
  __syncthreads();
  tcgen05_after_sync();
  if (s_skip) pc.r1 = pc.r0;   // statistics may be missing: no weights are added
  const uint32_t tmem = s_tmem;
  uint32_t done = 0;   // tiles of earlier pieces

  // Per piece the epilogue warps and the issuing one meet twice: q' and the
  // columns' values in place; the piece done.
  constexpr int MEET = (EP_WARPS + 1) * 32;
  if (warp < EP_WARPS) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_EP));
    // ---------------- epilogue: warpgroup wg takes every other tile, thread = token
    const int wg = warp >> 2, row = threadIdx.x & 127;
    const uint32_t t_d = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + 128 * wg;
    bool ok = true;   // no wait has given up
    while (pc.next()) {
      const int L = clamped_len(p, pc.b);
      const size_t pair = (size_t)pc.b * p.Hkv + kvh;
      {   // q' image, and the columns' max, 1 / sum and visible length
        const uint4* src = reinterpret_cast<const uint4*>(image + pair * (2 * NC * 256));
#pragma unroll 4
        for (int i = threadIdx.x; i < 2 * NC * 16; i += EP_WARPS * 32) reinterpret_cast<uint4*>(smem + Q_OFF)[i] = __ldcg(src + i);
        const int c = threadIdx.x;
        if (c < NC) {
          float2 v = make_float2(__int_as_float(0x7f800000), 0.f);   // columns past the last: exp2(-inf)
          int lim = L;
          if (c < p.ncols) {
            v = p.stats[pair * p.ncols + c];
            lim = L - p.M + c / p.g + 1;
          }
          s_col[c] = v;
          s_lim[c] = lim;
        }
      }
      fence_proxy_async_smem();   // q' is read by the tensor cores
      named_barrier_sync(1, MEET);
      float* mass = p.mass + pair * p.cap_len;
      for (int t = (int)((done + wg) & 1); ok && t < pc.n; t += 2) {
        const int tok0 = (pc.tile0 + t) * TOK, tok = tok0 + row;
        float old = 0.f;
        if (tok < L) old = mass[tok];
        if (!(ok = tr_wait(p, d_full + 8 * wg, ((done + t) >> 1) & 1, abort_flag))) break;
        tcgen05_after_sync();
        const bool tail = tok0 + TOK > L - p.M + 1;   // some token is hidden from some column
        float w = 0.f;
#pragma unroll
        for (int cc = 0; cc < NC; cc += 16) {
          uint32_t hi[16], lo[16];
          tmem_ld16(t_d + cc, hi);
          tmem_ld16(t_d + NC + cc, lo);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float2 col = s_col[cc + i];
            float s = __uint_as_float(hi[i]) + __uint_as_float(lo[i]);
            if (tail && tok >= s_lim[cc + i]) s = neg_inf();
            w = __fmaf_rn(fast_exp2(s - col.x), col.y, w);
          }
        }
        tcgen05_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(d_empty + 8 * wg);
        if (tok < L) mass[tok] = old + w;
      }
      done += pc.n;
      named_barrier_sync(1, MEET);
    }
  } else if (warp < MMA_WARP) {
    // ---------------- dequantisation of the keys
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_DQ));
    const int dw = warp - EP_WARPS;
    for (bool ok = true; ok && pc.next();) {
      ok = dequant_piece<MODE, VQKV_ROLE_K, PAGED, TOK, STAGES>(p, pc.b, kvh, pc.tile0, pc.n, clamped_len(p, pc.b), done, smem,
                                                               smem + K_OFF, k_full, k_empty, dw & 7, dw >> 3, lane,
                                                               abort_flag);
      done += pc.n;
    }
  } else {
    // ---------------- score products: one warp, an elected lane issues
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_MMA));
    constexpr uint32_t idesc = umma_idesc_f16_f32(TOK, 2 * NC);
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    const uint64_t k_desc = umma_desc_sw128(smem_u32(smem + K_OFF), 1024, 16);
    const uint64_t q_desc = umma_desc_sw128(smem_u32(smem + Q_OFF), 1024, 16);
    const bool issuer = elect_one();
    bool ok = true;
    while (warp == MMA_WARP && pc.next()) {
      named_barrier_sync(1, MEET);
      for (int t = 0; ok && t < pc.n; ++t) {
        const uint32_t k = done + t, st = k % STAGES, wg = k & 1;
        ok = tr_wait(p, k_full + 8 * st, (k / STAGES) & 1, abort_flag) &&
             tr_wait(p, d_empty + 8 * wg, ((k >> 1) & 1) ^ 1, abort_flag);
        if (!ok) break;
        tcgen05_after_sync();
        if (issuer) {
#pragma unroll
          for (int i = 0; i < 8; ++i)   // 16 channels: 32 bytes of a 128-byte row, four per 64-channel half
            umma_f16(tm + 128 * wg, k_desc + (st * TILE_SMEM + (i >> 2) * HALF + (i & 3) * 32) / 16,
                     q_desc + ((i >> 2) * (2 * NC * 128) + (i & 3) * 32) / 16, idesc, i > 0);
          umma_commit(k_empty + 8 * st);
          umma_commit(d_full + 8 * wg);
        }
        __syncwarp();
      }
      done += pc.n;
      named_barrier_sync(1, MEET);
    }
    if (warp == MMA_WARP) drain_products(p, issuer, all_done);
  }
  __syncwarp();
  tcgen05_before_sync();
  __syncthreads();
  tcgen05_after_sync();
  if (warp == MMA_WARP) tmem_dealloc(tmem, T_COLS);
}

using TileKernel = void (*)(DecodeParams, const unsigned char*);
template <int MODE>
TileKernel tile_of(bool paged, bool wide) {
  return wide ? (paged ? (TileKernel)mass_tile_kernel<MODE, true, 64> : (TileKernel)mass_tile_kernel<MODE, false, 64>)
              : (paged ? (TileKernel)mass_tile_kernel<MODE, true, 32> : (TileKernel)mass_tile_kernel<MODE, false, 32>);
}
TileKernel tile_kernel(int mode, bool paged, bool wide) {
  switch (mode) {
    case VQKV_MODE_VQ2: return tile_of<VQKV_MODE_VQ2>(paged, wide);
    case VQKV_MODE_VQ4: return tile_of<VQKV_MODE_VQ4>(paged, wide);
    case VQKV_MODE_VQ3: return tile_of<VQKV_MODE_VQ3>(paged, wide);
    case VQKV_MODE_VQ15: return tile_of<VQKV_MODE_VQ15>(paged, wide);
    default: return tile_of<VQKV_MODE_VQ125>(paged, wide);
  }
}

}  // namespace

cudaError_t mass_tiles_prepare(int mode) {
  cudaError_t e = cudaSuccess;
  for (int i = 0; i < 4 && e == cudaSuccess; ++i)
    e = prepare_split_kernel(tile_kernel(mode, (i & 1) != 0, (i & 2) != 0), mt::THREADS, mt::SPLIT_REGS, mt::SMEM);
  return e;
}

size_t mass_tiles_image_bytes(int B, int Hkv, int ncols) { return (size_t)B * Hkv * 2 * (ncols <= 32 ? 32 : 64) * 256; }

cudaError_t launch_mass_queries(const DecodeParams& p, void* image, cudaStream_t stream) {
  const bool wide = p.ncols > 32;
  const dim3 grid(wide ? 2 : 1, p.Hkv, p.B);
  unsigned char* img = static_cast<unsigned char*>(image);
  return launch_pdl(wide ? mass_query_kernel<64> : mass_query_kernel<32>, grid, dim3(128), 0, stream, p, img);
}

cudaError_t launch_mass_tiles(int mode, const DecodeParams& p, const void* image, cudaStream_t stream) {
  return launch_pdl(tile_kernel(mode, p.block_table != nullptr, p.ncols > 32), dim3(p.n_splits, p.Hkv), dim3(mt::THREADS),
                    (size_t)mt::SMEM, stream, p, static_cast<const unsigned char*>(image));
}

}  // namespace vqkv
