// Attention of a tree of drafted tokens over a packed cache (sm_103a, tcgen05).
//
// M drafts x g query heads give up to 512 softmax columns per KV head, so the
// two products are matrix products worth the tensor cores: a CTA takes up to
// 128 columns (the MMA rows) and one token range ("split") of a sequence and
// walks it in tiles of 64 tokens:
//   dequantise  K' and V tiles into shared memory, each centroid gathered
//               once per tile and CTA (8 warps: 4 for K, 4 for V)
//   S = Q' K'^T 128 x 64 x 128, Q' in tensor memory (A), K' rows in shared
//               memory (B, K-major), S in tensor memory
//   softmax     one thread per column (4 warps): running max and sum in fp32,
//               P = exp2(S - m) as fp16 back to tensor memory; O is rescaled
//               only when a score exceeds the running max by 2^8
//   O += P V    128 x 128 x 64, P in tensor memory (A), V rows in shared
//               memory (B, channel-major), O stays in tensor memory
// K and V tiles have a two-stage ring each; S and P are double buffered, and
// the score product of tile t + 1 is issued before the P.V product of tile t,
// so the tensor cores, the softmax warps and the dequantisation overlap.
//
// The query transform is that of the single-query decode: q' = (q * s) . Hn,
// scaled by softmax_scale * log2 e.  q' and P are rounded to fp16 (2^-12
// relative, as in the other decode kernels) for the fp16 tensor-core product;
// centroids are fp16 already, sums are fp32.
//
// Visibility: tokens t < L - M for every column, draft j for the columns
// whose mask has bit j; only tiles that reach past L - M test it.
#include <type_traits>

#include "common.cuh"
#include "decode_common.cuh"
#include "gather.cuh"
#include "internal.h"
#include "umma.cuh"

namespace vqkv {
namespace {

namespace tr {
constexpr int COLS = 128;                 // softmax columns per CTA (MMA rows)
constexpr int TOK = 64;                   // tokens per tile
constexpr int SM_WARPS = 4, DQ_WARPS = 8;
constexpr int MMA_WARP = SM_WARPS + DQ_WARPS;
constexpr int THREADS = (MMA_WARP + 1) * 32;
constexpr int TILE_SMEM = TOK * 256;      // one dequantised K or V tile: two 64-channel halves of 64 x 128 bytes
constexpr int HALF = TOK * 128;
constexpr int STAGES = 2;
constexpr int PREFETCH = 4;               // tiles whose codes a dequantising warp holds in registers
constexpr int Q_PITCH = 272;              // staged q' row (fp16), padded against bank conflicts
// tensor memory columns
constexpr uint32_t T_O = 0, T_S = 128, T_P = 256, T_Q = 320, T_COLS = 512;
constexpr uint32_t MAX_POLLS = 1u << 20;

template <int MODE>
struct Geo {
  static constexpr int CB_BYTES = MODE == VQKV_MODE_VQ15 || MODE == VQKV_MODE_VQ125 ? 131072 : 65536;
  static constexpr int K_OFF = CB_BYTES, V_OFF = K_OFF + STAGES * TILE_SMEM;
  static constexpr int BAR_OFF = V_OFF + STAGES * TILE_SMEM;
  static constexpr int SMEM = BAR_OFF + 256;
  static constexpr int LAYOUT_TOK = MODE == VQKV_MODE_VQ15 ? 64 : 16;
  static constexpr int TILE_BYTES = MODE == VQKV_MODE_VQ2    ? 512
                                    : MODE == VQKV_MODE_VQ4  ? 1024
                                    : MODE == VQKV_MODE_VQ3  ? 768
                                    : MODE == VQKV_MODE_VQ15 ? 1536
                                                             : 320;
  // 32-bit words of a lane's codes of 16 tokens
  static constexpr int KW = MODE == VQKV_MODE_VQ2 ? 4 : MODE == VQKV_MODE_VQ4 ? 8 : MODE == VQKV_MODE_VQ3 ? 6 : 3;
  static constexpr int VW = MODE == VQKV_MODE_VQ125 ? 5 : KW;
  static constexpr int W = VW;
  static_assert(COLS * Q_PITCH <= 2 * STAGES * TILE_SMEM, "staged q' uses the K and V rings before the loop");
  static_assert(SMEM <= 227 * 1024, "shared memory");
};
}  // namespace tr

// Codebooks into shared memory, in the layouts of the single-query decode: 256
// entries: row c of 256 bytes, K replicas then V replicas (16 of 8 bytes or 32
// of 4); 4096 x 4 (3 bit): K then V, once; 4096 x 8 (1.5 bit): K then V, once;
// 1024 x 8 (1.25 bit): four interleaved copies (cb10_offset).
template <int MODE>
__device__ __forceinline__ void fill_codebooks(const DecodeParams& p, int kvh, unsigned char* smem) {
  constexpr int N = tr::THREADS;
  if constexpr (MODE == VQKV_MODE_VQ2 || MODE == VQKV_MODE_VQ4) {
    using Entry = typename std::conditional<MODE == VQKV_MODE_VQ2, uint2, uint32_t>::type;
    constexpr int REPL = 128 / (int)sizeof(Entry);
    for (int i = threadIdx.x; i < 512; i += N) {
      const int c = i & 255, role = i >> 8;
      const Entry e = __ldg(reinterpret_cast<const Entry*>(role ? p.vcb : p.kcb) + (size_t)kvh * 256 + c);
      Entry* row = reinterpret_cast<Entry*>(smem + c * 256 + role * 128);
#pragma unroll 4
      for (int k = 0; k < REPL; ++k) row[(k + threadIdx.x) & (REPL - 1)] = e;
    }
  } else if constexpr (MODE == VQKV_MODE_VQ125) {
#pragma unroll 2
    for (int i = threadIdx.x; i < 2048; i += N) {
      const uint32_t c = i & 1023;
      const uint4 e = __ldg(reinterpret_cast<const uint4*>(i >> 10 ? p.vcb : p.kcb) + (size_t)kvh * 1024 + c);
      unsigned char* row = smem + (i >> 10) * 65536 + cb10_offset(c);
#pragma unroll
      for (int k = 0; k < 4; ++k) *reinterpret_cast<uint4*>(row + 32 * ((k + (c >> 1)) & 3)) = e;
    }
  } else {
    constexpr int PER = MODE == VQKV_MODE_VQ3 ? 2048 : 4096;   // 16-byte pieces per role
#pragma unroll 4
    for (int i = threadIdx.x; i < 2 * PER; i += N) {
      const int role = i / PER, c = i - role * PER;
      reinterpret_cast<uint4*>(smem)[i] =
          __ldg(reinterpret_cast<const uint4*>(role ? p.vcb : p.kcb) + (size_t)kvh * PER + c);
    }
  }
}

// The lane's code words of 16-token group u of a tile (off: byte offset of the
// layout tile that holds it).
template <int MODE, int ROLE>
__device__ __forceinline__ void load_words(const uint8_t* codes, long long off, int u, int lane,
                                           uint32_t (&w)[tr::Geo<MODE>::W]) {
  const uint8_t* t = codes + off;
  if constexpr (MODE == VQKV_MODE_VQ2) {
    const uint4 a = ldg_stream(t + 16 * lane);
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
  } else if constexpr (MODE == VQKV_MODE_VQ4) {
    const uint4 a = ldg_stream(t + 16 * lane), c = ldg_stream(t + 512 + 16 * lane);
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = c.x, w[5] = c.y, w[6] = c.z, w[7] = c.w;
  } else if constexpr (MODE == VQKV_MODE_VQ3) {
    const uint4 a = ldg_stream(t + 16 * lane);
    const uint2 c = __ldg(reinterpret_cast<const uint2*>(t + 512 + 8 * lane));
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = c.x, w[5] = c.y;
  } else if constexpr (MODE == VQKV_MODE_VQ15) {
    const uint32_t* q = reinterpret_cast<const uint32_t*>(t + 48 * lane + 12 * u);
    w[0] = __ldg(q), w[1] = __ldg(q + 1), w[2] = __ldg(q + 2);
  } else if constexpr (ROLE == VQKV_ROLE_K) {
    const uint2 a = __ldg(reinterpret_cast<const uint2*>(t + 8 * lane));
    w[0] = a.x, w[1] = a.y, w[2] = __ldg(reinterpret_cast<const unsigned short*>(t + 256 + 2 * lane));
  } else {
    const int run = 4 * (lane >> 3) + (lane & 3);
    const uint4 a = ldg_stream(t + 16 * run);
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
    w[4] = __ldg(reinterpret_cast<const uint32_t*>(t + 256 + 4 * run));
  }
}

// Writes 4, 8 or 16 bytes (T) at byte `at` of token row `row` of a tile: two
// 64-channel halves, 128-byte rows, 16-byte pieces swizzled by the row.
template <typename T>
__device__ __forceinline__ void put_tile(unsigned char* tile, int row, int at, T v) {
  *reinterpret_cast<T*>(tile + (at >> 7) * tr::HALF + row * 128 + ((((at >> 4) & 7) ^ (row & 7)) << 4) + (at & 15)) = v;
}

// Dequantises the lane's share of 16 key tokens (rows 16u ..) into a tile.
// Lane (gid, tig) holds the codes of tokens gid, gid + 8 for every fourth
// subvector; the stores of a warp cover the banks evenly.
template <int MODE>
__device__ __forceinline__ void dequant_k(const unsigned char* s_cb, unsigned char* tile, int u, int lane,
                                          const uint32_t (&w)[tr::Geo<MODE>::W]) {
  const int gid = lane >> 2, tig = lane & 3;
  const int r0 = 16 * u + gid, r1 = r0 + 8;
  if constexpr (MODE == VQKV_MODE_VQ2) {
    const uint32_t kb = (uint32_t)(lane & 15) << 3;
#define VQKV_K_STEP(S)                                                                                  \
  {                                                                                                     \
    const uint2 c = lds_at<uint2>(s_cb, cb_offset<(S)&3>((S) < 4 ? w[0] : w[1], kb));                     \
    const uint2 d = lds_at<uint2>(s_cb, cb_offset<(S)&3>((S) < 4 ? w[2] : w[3], kb));                     \
    put_tile(tile, r0, 32 * (S) + 8 * tig, c);                                                            \
    put_tile(tile, r1, 32 * (S) + 8 * tig, d);                                                            \
  }
    VQKV_K_STEP(0) VQKV_K_STEP(1) VQKV_K_STEP(2) VQKV_K_STEP(3)
    VQKV_K_STEP(4) VQKV_K_STEP(5) VQKV_K_STEP(6) VQKV_K_STEP(7)
#undef VQKV_K_STEP
  } else if constexpr (MODE == VQKV_MODE_VQ4) {
    const uint32_t kb = (uint32_t)lane << 2;
#define VQKV_K_STEP(S)                                                                                       \
  {                                                                                                          \
    const uint32_t wg = w[(S) >> 1], wh = w[4 + ((S) >> 1)];                                                   \
    put_tile(tile, r0, 32 * (S) + 4 * tig, lds_at<uint32_t>(s_cb, cb_offset<((S)&1) * 2>(wg, kb)));            \
    put_tile(tile, r0, 32 * (S) + 16 + 4 * tig, lds_at<uint32_t>(s_cb, cb_offset<((S)&1) * 2 + 1>(wg, kb)));   \
    put_tile(tile, r1, 32 * (S) + 4 * tig, lds_at<uint32_t>(s_cb, cb_offset<((S)&1) * 2>(wh, kb)));            \
    put_tile(tile, r1, 32 * (S) + 16 + 4 * tig, lds_at<uint32_t>(s_cb, cb_offset<((S)&1) * 2 + 1>(wh, kb)));   \
  }
    VQKV_K_STEP(0) VQKV_K_STEP(1) VQKV_K_STEP(2) VQKV_K_STEP(3)
    VQKV_K_STEP(4) VQKV_K_STEP(5) VQKV_K_STEP(6) VQKV_K_STEP(7)
#undef VQKV_K_STEP
  } else if constexpr (MODE == VQKV_MODE_VQ3) {
#pragma unroll
    for (int S = 0; S < 8; ++S) {
      const uint32_t pg = pair_at(w, 3 * (S & 3)), ph = pair_at(w, 12 + 3 * (S & 3));
      const uint32_t cg = S < 4 ? (pg & 0xfffu) : (pg >> 12), ch = S < 4 ? (ph & 0xfffu) : (ph >> 12);
      put_tile(tile, r0, 32 * S + 8 * tig, lds_at<uint2>(s_cb, cg << 3));
      put_tile(tile, r1, 32 * S + 8 * tig, lds_at<uint2>(s_cb, ch << 3));
    }
  } else if constexpr (MODE == VQKV_MODE_VQ15) {
    // pairs tig, tig + 4 of token gid, then of token gid + 8
#pragma unroll
    for (int s2 = 0; s2 < 4; ++s2) {
      const uint32_t pa = pair24(w[0], w[1], w[2], s2 & 1), pb = pair24(w[0], w[1], w[2], 2 + (s2 & 1));
      const uint32_t ca = s2 < 2 ? (pa & 0xfffu) : (pa >> 12), cb = s2 < 2 ? (pb & 0xfffu) : (pb >> 12);
      put_tile(tile, r0, 64 * s2 + 16 * tig, lds_at<uint4>(s_cb, ca << 4));
      put_tile(tile, r1, 64 * s2 + 16 * tig, lds_at<uint4>(s_cb, cb << 4));
    }
  } else {
    const uint32_t kb = (uint32_t)tig << 5;
#pragma unroll
    for (int s2 = 0; s2 < 4; ++s2) {
      put_tile(tile, r0, 64 * s2 + 16 * tig, lds_at<uint4>(s_cb, kb + cb10_offset(bits10(w, 10 * s2))));
      put_tile(tile, r1, 64 * s2 + 16 * tig, lds_at<uint4>(s_cb, kb + cb10_offset(bits10(w, 40 + 10 * s2))));
    }
  }
}

// The same for 16 value tokens: lane (gid, tig) holds the codes of tokens 2tig,
// 2tig + 1, 2tig + 8, 2tig + 9 for the subvectors j with j % 8 == gid.
template <int MODE>
__device__ __forceinline__ void dequant_v(const unsigned char* s_cb, unsigned char* tile, int u, int lane,
                                          const uint32_t (&w)[tr::Geo<MODE>::W]) {
  const int gid = lane >> 2, tig = lane & 3;
  const int r0 = 16 * u + 2 * tig;
  if constexpr (MODE == VQKV_MODE_VQ2) {
    const uint32_t vb = 128u | ((uint32_t)(lane & 15) << 3);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      put_tile(tile, r0, 64 * i + 8 * gid, lds_at<uint2>(s_cb, cb_offset<0>(w[i], vb)));
      put_tile(tile, r0 + 1, 64 * i + 8 * gid, lds_at<uint2>(s_cb, cb_offset<1>(w[i], vb)));
      put_tile(tile, r0 + 8, 64 * i + 8 * gid, lds_at<uint2>(s_cb, cb_offset<2>(w[i], vb)));
      put_tile(tile, r0 + 9, 64 * i + 8 * gid, lds_at<uint2>(s_cb, cb_offset<3>(w[i], vb)));
    }
  } else if constexpr (MODE == VQKV_MODE_VQ4) {
    const uint32_t vb = 128u | ((uint32_t)lane << 2);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      put_tile(tile, r0, 32 * i + 4 * gid, lds_at<uint32_t>(s_cb, cb_offset<0>(w[i], vb)));
      put_tile(tile, r0 + 1, 32 * i + 4 * gid, lds_at<uint32_t>(s_cb, cb_offset<1>(w[i], vb)));
      put_tile(tile, r0 + 8, 32 * i + 4 * gid, lds_at<uint32_t>(s_cb, cb_offset<2>(w[i], vb)));
      put_tile(tile, r0 + 9, 32 * i + 4 * gid, lds_at<uint32_t>(s_cb, cb_offset<3>(w[i], vb)));
    }
  } else if constexpr (MODE == VQKV_MODE_VQ3) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) {   // token slot k: pair gid + 8 (i % 2), low code for i < 2
        const uint32_t pr = pair_at(w, 6 * k + 3 * (i & 1));
        put_tile(tile, r0 + (k & 1) + 8 * (k >> 1), 64 * i + 8 * gid,
                 lds_at<uint2>(s_cb, 32768u + ((i < 2 ? (pr & 0xfffu) : (pr >> 12)) << 3)));
      }
  } else if constexpr (MODE == VQKV_MODE_VQ15) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t pr = pair24(w[0], w[1], w[2], k);
      const int row = r0 + (k & 1) + 8 * (k >> 1);
      put_tile(tile, row, 16 * gid, lds_at<uint4>(s_cb, 65536u + ((pr & 0xfffu) << 4)));
      put_tile(tile, row, 128 + 16 * gid, lds_at<uint4>(s_cb, 65536u + ((pr >> 12) << 4)));
    }
  } else {
    const uint32_t vb = 65536u + ((uint32_t)tig << 5), sh = 10u * (gid & 1);
    uint32_t v[5];
#pragma unroll
    for (int m = 0; m < 4; ++m) v[m] = __funnelshift_r(w[m], w[m + 1], sh);
    v[4] = w[4] >> sh;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        put_tile(tile, r0 + (k & 1) + 8 * (k >> 1), 128 * i + 16 * gid,
                 lds_at<uint4>(s_cb, vb + cb10_offset(bits10(v, 40 * k + 20 * i))));
  }
}

// Bounded wait by every lane in `mask`: false, with the abort flag and the
// device error bit set, when it runs out or another role gave up.
__device__ __forceinline__ bool tr_wait(uint32_t mbar, uint32_t parity, volatile int* abort_flag, unsigned* err,
                                        unsigned mask) {
  bool ok = false;
  for (uint32_t i = 0; i < tr::MAX_POLLS; ++i) {
    if (mbar_try_wait(mbar, parity)) {
      ok = true;
      break;
    }
    if ((i & 31) == 31 && *abort_flag) break;
  }
  ok = __all_sync(mask, ok);
  if (!ok && !*abort_flag) {
    *abort_flag = 1;
    atomicOr(err, VQKV_DEVERR_TIMEOUT);
  }
  return ok;
}

// The dequantising warp of (role, 16-token group u of each tile): codes are
// loaded PREFETCH tiles ahead into registers, block ids one tile further.
template <int MODE, int ROLE, bool PAGED>
__device__ __forceinline__ void dequant_loop(const DecodeParams& p, int b, int kvh, int tile0, int n, int L,
                                             unsigned char* smem, uint32_t full, uint32_t empty, int u, int lane,
                                             volatile int* abort_flag) {
  using G = tr::Geo<MODE>;
  const uint8_t* codes = ROLE == VQKV_ROLE_K ? p.kc : p.vc;
  const int last_group = (L + 15) >> 4;   // 16-token groups that hold tokens
  uint32_t w[tr::PREFETCH][G::W];
  bool bad = false;
  // byte offset of the layout tile of this warp's group of tile t, -1 past the sequence
  auto place = [&](int t) -> long long {
    const int grp = (tile0 + t) * (tr::TOK / 16) + u;
    if (t >= n || grp >= last_group) return -1;
    return tile_offset<PAGED>(p, b, kvh, G::LAYOUT_TOK == 64 ? tile0 + t : grp, G::TILE_BYTES, &bad);
  };
  auto fetch = [&](long long off, uint32_t (&x)[G::W]) {
    if (off >= 0) {
      load_words<MODE, ROLE>(codes, off, u, lane, x);
    } else {
#pragma unroll
      for (int i = 0; i < G::W; ++i) x[i] = 0u;
    }
  };
#pragma unroll
  for (int d = 0; d < tr::PREFETCH; ++d) fetch(place(d), w[d]);
  long long next = place(tr::PREFETCH);
  for (int t0 = 0; t0 < n; t0 += tr::PREFETCH) {
#pragma unroll
    for (int d = 0; d < tr::PREFETCH; ++d) {
      const int t = t0 + d;
      if (t >= n) break;
      const int st = t & 1;
      if (!tr_wait(empty + 8 * st, ((t >> 1) & 1) ^ 1, abort_flag, p.err, 0xffffffffu)) return;
      unsigned char* tile = smem + (ROLE == VQKV_ROLE_K ? G::K_OFF : G::V_OFF) + st * tr::TILE_SMEM;
      if constexpr (ROLE == VQKV_ROLE_K)
        dequant_k<MODE>(smem, tile, u, lane, w[d]);
      else
        dequant_v<MODE>(smem, tile, u, lane, w[d]);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(full + 8 * st);
      fetch(next, w[d]);
      next = place(t + tr::PREFETCH + 1);
    }
  }
  if (PAGED && bad && lane == 0) atomicOr(p.err, VQKV_DEVERR_BLOCK);
}

// grid (splits, Hkv, B x column groups).
template <int MODE, bool PAGED>
__global__ void __launch_bounds__(tr::THREADS, 1) decode_tree_kernel(const DecodeParams p,
                                                                     const unsigned long long* tree_mask) {
  using namespace tr;
  using G = Geo<MODE>;
  extern __shared__ __align__(1024) unsigned char smem[];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  const int split = blockIdx.x, kvh = blockIdx.y, b = blockIdx.z / p.cgroups;
  const int col0 = COLS * (int)(blockIdx.z % p.cgroups), nloc = min(COLS, p.ncols - col0);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int active = (nloc + 31) >> 5;      // softmax warps with columns
  const uint32_t bar = smem_u32(smem + G::BAR_OFF);
  const uint32_t k_full = bar, k_empty = bar + 16, v_full = bar + 32, v_empty = bar + 48;
  const uint32_t s_full = bar + 64, p_full = bar + 80, o_done = bar + 96, all_done = bar + 112;
  volatile int* abort_flag = &s_abort;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(k_full + 8 * i, 4);
      mbar_init(k_empty + 8 * i, 1);
      mbar_init(v_full + 8 * i, 4);
      mbar_init(v_empty + 8 * i, 1);
      mbar_init(s_full + 8 * i, 1);
      mbar_init(p_full + 8 * i, active);
      mbar_init(o_done + 8 * i, 1);
    }
    mbar_init(all_done, 1);
    s_abort = 0;
    mbar_init_fence();
  }
  if (warp == MMA_WARP) tmem_alloc(smem_u32(&s_tmem), T_COLS);
  grid_dependency_wait();
  grid_dependents_launch();

  int L = p.seq_lens[b];
  if (L < 0 || L > p.max_seq_len) {
    if (split == 0 && kvh == 0 && threadIdx.x == 0) atomicOr(p.err, VQKV_DEVERR_SEQ_LEN);
    L = L < 0 ? 0 : p.max_seq_len;
  }
  const int tiles = (L + TOK - 1) / TOK;
  const int tile0 = split * p.tps, n = min(p.tps, tiles - tile0);   // this CTA's tiles (n <= 0: none)

  // q' of the CTA's columns as fp16 rows in the (still unused) tile rings
  unsigned char* s_q = smem + G::K_OFF;
  if (n > 0) {
    fill_codebooks<MODE>(p, kvh, smem);
    for (int c = warp; c < 32 * active; c += THREADS / 32) {
      const QueryLoad r = load_query(p, b, kvh, c, lane, col0, nloc);   // zeros past the last column
      const __half2 q01 = *reinterpret_cast<const __half2*>(&r.q.x), q23 = *reinterpret_cast<const __half2*>(&r.q.y);
      float v[4] = {__low2float(q01) * r.s.x, __high2float(q01) * r.s.y, __low2float(q23) * r.s.z,
                    __high2float(q23) * r.s.w};
      fwht128_f32(v, lane);
      *reinterpret_cast<uint2*>(s_q + c * Q_PITCH + 8 * lane) =
          make_uint2(pack_half2(v[0] * p.qscale, v[1] * p.qscale), pack_half2(v[2] * p.qscale, v[3] * p.qscale));
    }
  }
  tcgen05_before_sync();
  __syncthreads();
  tcgen05_after_sync();
  const uint32_t tmem = s_tmem;
  const uint32_t t_lane = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
  if (n > 0 && warp < active) {   // q' into tensor memory: lane = column
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t r[32];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint4 x = *reinterpret_cast<const uint4*>(s_q + threadIdx.x * Q_PITCH + 128 * h + 16 * i);
        r[4 * i] = x.x, r[4 * i + 1] = x.y, r[4 * i + 2] = x.z, r[4 * i + 3] = x.w;
      }
      tmem_st32(t_lane + T_Q + 32 * h, r);
    }
    tmem_wait_st();
  }
  tcgen05_before_sync();
  __syncthreads();
  tcgen05_after_sync();

  if (warp < SM_WARPS) {
    // ---------------- softmax: thread = column col0 + threadIdx.x
    const int cl = threadIdx.x, c = col0 + cl;
    float m = kMInit, l = 0.f;
    bool ok = warp < active;
    if (ok && n > 0) {
      const int prefix = L - p.M;            // tokens below it are visible to every column
      unsigned long long mask = 0;
      if (cl < nloc) {
        mask = tree_mask[(size_t)b * p.M + c / p.g];
        if (p.M < 64) mask &= (1ull << p.M) - 1;
      }
      for (int t = 0; t < n; ++t) {
        const int st = t & 1;
        if (!(ok = tr_wait(s_full + 8 * st, (t >> 1) & 1, abort_flag, p.err, 0xffffffffu))) break;
        tcgen05_after_sync();
        float x[2][32];
        tmem_ld32(t_lane + T_S + 64 * st, x[0]);
        tmem_ld32(t_lane + T_S + 64 * st + 32, x[1]);
        tmem_wait_ld();
        const int tok0 = (tile0 + t) * TOK, d = prefix - tok0;
        if (d < TOK) {                       // bit i of vis: token tok0 + i is visible
          unsigned long long vis = d >= 0 ? (mask << d) | ((1ull << d) - 1) : d > -64 ? mask >> -d : 0ull;
#pragma unroll
          for (int i = 0; i < 64; ++i)
            if (!((vis >> i) & 1)) x[i >> 5][i & 31] = neg_inf();
        }
        float top = fmaxf(x[0][0], x[1][0]);
#pragma unroll
        for (int i = 1; i < 32; ++i) top = fmaxf(top, fmaxf(x[0][i], x[1][i]));
        if (__any_sync(0xffffffffu, top > m + kSoftmaxSlack)) {
          const float mn = fmaxf(m, top), f = fast_exp2(m - mn);
          m = mn;
          l *= f;
          if (t > 0) {   // O holds tiles 0 .. t - 1 once P.V of t - 1 is done
            if (!(ok = tr_wait(o_done + 8 * (st ^ 1), ((t - 1) >> 1) & 1, abort_flag, p.err, 0xffffffffu))) break;
            tcgen05_after_sync();
#pragma unroll 1
            for (int q = 0; q < 4; ++q) {
              float o[32];
              tmem_ld32(t_lane + T_O + 32 * q, o);
              tmem_wait_ld();
              uint32_t r[32];
#pragma unroll
              for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(o[i] * f);
              tmem_st32(t_lane + T_O + 32 * q, r);
            }
          }
        }
        uint32_t r[32];
        float l0 = 0.f, l1 = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const float p0 = fast_exp2(x[i >> 4][(2 * i) & 31] - m), p1 = fast_exp2(x[i >> 4][(2 * i + 1) & 31] - m);
          l0 += p0;
          l1 += p1;
          r[i] = pack_half2(p0, p1);
        }
        l += l0 + l1;
        tmem_st32(t_lane + T_P + 32 * st, r);
        tmem_wait_st();
        tcgen05_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full + 8 * st);
      }
      if (ok) ok = tr_wait(o_done + 8 * ((n - 1) & 1), ((n - 1) >> 1) & 1, abort_flag, p.err, 0xffffffffu);
      tcgen05_after_sync();
    }
    if (ok) {
      const float inv = l > 0.f ? 1.f / l : 0.f;
      const bool whole = p.n_splits == 1;
      float* part = p.partials + (((size_t)(b * p.Hkv + kvh) * p.n_splits + split) * p.ncols + c) * kPartialStride;
#pragma unroll 1
      for (int q = 0; q < 4; ++q) {
        float o[32];
        if (n > 0) {
          tmem_ld32(t_lane + T_O + 32 * q, o);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = 0.f;
        }
        if (cl < nloc && !whole) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            *reinterpret_cast<float4*>(part + 32 * q + 4 * i) =
                make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
        } else if (cl < nloc) {
          __half* dst = p.out + out_row(p, b, kvh, c) + 32 * q;
          if ((reinterpret_cast<uintptr_t>(dst) & 15) == 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              *reinterpret_cast<uint4*>(dst + 8 * i) =
                  make_uint4(pack_half2(o[8 * i] * inv, o[8 * i + 1] * inv), pack_half2(o[8 * i + 2] * inv, o[8 * i + 3] * inv),
                             pack_half2(o[8 * i + 4] * inv, o[8 * i + 5] * inv), pack_half2(o[8 * i + 6] * inv, o[8 * i + 7] * inv));
          } else {   // out needs only 2-byte alignment
#pragma unroll
            for (int i = 0; i < 32; ++i) dst[i] = __float2half_rn(o[i] * inv);
          }
        }
      }
      if (!whole && cl < nloc) *reinterpret_cast<float2*>(part + 128) = make_float2(m, l);
    }
  } else if (warp < MMA_WARP) {
    // ---------------- dequantisation
    const int dw = warp - SM_WARPS, u = dw & 3;
    if (n > 0) {
      if (dw < 4)
        dequant_loop<MODE, VQKV_ROLE_K, PAGED>(p, b, kvh, tile0, n, L, smem, k_full, k_empty, u, lane, abort_flag);
      else
        dequant_loop<MODE, VQKV_ROLE_V, PAGED>(p, b, kvh, tile0, n, L, smem, v_full, v_empty, u, lane, abort_flag);
    }
  } else if (lane == 0 && n > 0) {
    // ---------------- one thread issues the products
    constexpr uint32_t idesc_s = umma_idesc_f16_f32(COLS, TOK);
    constexpr uint32_t idesc_o = umma_idesc_f16_f32(COLS, kHeadDim) | kIdescBMnMajor;
    const uint32_t k_smem = smem_u32(smem + G::K_OFF), v_smem = smem_u32(smem + G::V_OFF);
    auto scores = [&](int t) -> bool {
      const int st = t & 1;
      if (!tr_wait(k_full + 8 * st, (t >> 1) & 1, abort_flag, p.err, 1u)) return false;
      tcgen05_after_sync();
#pragma unroll
      for (int k = 0; k < 8; ++k)   // 16 channels each: 32 bytes of a 128-byte row, four per 64-channel half
        umma_f16_ts(tmem + T_S + 64 * st, tmem + T_Q + 8 * k,
                    umma_desc_sw128(k_smem + st * TILE_SMEM + (k >> 2) * HALF + (k & 3) * 32, 1024, 16), idesc_s, k > 0);
      umma_commit(s_full + 8 * st);
      umma_commit(k_empty + 8 * st);
      return true;
    };
    bool ok = scores(0);
    for (int t = 0; ok && t < n; ++t) {
      const int st = t & 1;
      if (t + 1 < n) ok = scores(t + 1);
      ok = ok && tr_wait(v_full + 8 * st, (t >> 1) & 1, abort_flag, p.err, 1u);
      ok = ok && tr_wait(p_full + 8 * st, (t >> 1) & 1, abort_flag, p.err, 1u);
      if (!ok) break;
      tcgen05_after_sync();
#pragma unroll
      for (int k = 0; k < 4; ++k)   // 16 tokens each: two 8-token groups
        umma_f16_ts(tmem + T_O, tmem + T_P + 32 * st + 8 * k,
                    umma_desc_sw128(v_smem + st * TILE_SMEM + k * 2048, 1024, HALF), idesc_o, t > 0 || k > 0);
      umma_commit(v_empty + 8 * st);
      umma_commit(o_done + 8 * st);
    }
    // every product issued has completed before the tensor memory is freed
    umma_commit(all_done);
    tr_wait(all_done, 0, abort_flag, p.err, 1u);
  }
  __syncwarp();
  tcgen05_before_sync();
  __syncthreads();
  tcgen05_after_sync();
  if (warp == MMA_WARP) tmem_dealloc(tmem, T_COLS);
}

using TreeKernel = void (*)(DecodeParams, const unsigned long long*);
template <int MODE>
TreeKernel tree_of(bool paged) {
  return paged ? (TreeKernel)decode_tree_kernel<MODE, true> : (TreeKernel)decode_tree_kernel<MODE, false>;
}
TreeKernel tree_kernel(int mode, bool paged) {
  return mode == VQKV_MODE_VQ2    ? tree_of<VQKV_MODE_VQ2>(paged)
         : mode == VQKV_MODE_VQ4  ? tree_of<VQKV_MODE_VQ4>(paged)
         : mode == VQKV_MODE_VQ3  ? tree_of<VQKV_MODE_VQ3>(paged)
         : mode == VQKV_MODE_VQ15 ? tree_of<VQKV_MODE_VQ15>(paged)
                                  : tree_of<VQKV_MODE_VQ125>(paged);
}
int tree_smem(int mode) {
  return mode == VQKV_MODE_VQ15 || mode == VQKV_MODE_VQ125 ? tr::Geo<VQKV_MODE_VQ15>::SMEM : tr::Geo<VQKV_MODE_VQ2>::SMEM;
}

}  // namespace

int decode_tree_cols() { return tr::COLS; }
int decode_tree_tile() { return tr::TOK; }

cudaError_t decode_tree_prepare(int mode) {
  cudaError_t e = cudaSuccess;
  for (int paged = 0; paged < 2 && e == cudaSuccess; ++paged)
    e = cudaFuncSetAttribute(tree_kernel(mode, paged != 0), cudaFuncAttributeMaxDynamicSharedMemorySize, tree_smem(mode));
  return e;
}

cudaError_t launch_decode_tree(int mode, const DecodeParams& p, const unsigned long long* tree_mask, dim3 grid,
                               cudaStream_t stream) {
  return launch_pdl(tree_kernel(mode, p.block_table != nullptr), grid, dim3(tr::THREADS), (size_t)tree_smem(mode), stream, p,
                    tree_mask);
}

}  // namespace vqkv
