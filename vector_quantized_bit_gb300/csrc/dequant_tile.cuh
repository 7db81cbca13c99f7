// Dequantised tiles of packed codes in shared memory, as tensor-core operands:
// codebooks, code loads, centroid gathers, swizzled tile stores, the loop of a
// dequantising warp, and the shares of a ragged batch.  Used by the kernels
// that run many softmax columns on tcgen05 (decode_tree.cu, cross_attn.cu,
// mass_tiles.cu).
#pragma once

#include <type_traits>

#include "common.cuh"
#include "decode_common.cuh"
#include "gather.cuh"
#include "internal.h"
#include "umma.cuh"

namespace vqkv {
namespace {

template <int MODE>
struct CodeGeo {
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
};

// Codebooks into shared memory, in the layouts of the single-query decode: 256
// entries: row c of 256 bytes, K replicas then V replicas (16 of 8 bytes or 32
// of 4); 4096 x 4 (3 bit): K then V, once; 4096 x 8 (1.5 bit): K then V, once;
// 1024 x 8 (1.25 bit): four interleaved copies (cb10_offset).
// VALUES: K and V, else K only (the same places).  All N threads.
template <int MODE, int N, bool VALUES>
__device__ __forceinline__ void fill_codebooks(const DecodeParams& p, int kvh, unsigned char* smem) {
  constexpr int ROLES = VALUES ? 2 : 1;
  if constexpr (MODE == VQKV_MODE_VQ2 || MODE == VQKV_MODE_VQ4) {
    using Entry = typename std::conditional<MODE == VQKV_MODE_VQ2, uint2, uint32_t>::type;
    constexpr int REPL = 128 / (int)sizeof(Entry);
    for (int i = threadIdx.x; i < 256 * ROLES; i += N) {
      const int c = i & 255, role = i >> 8;
      const Entry e = __ldg(reinterpret_cast<const Entry*>(role ? p.vcb : p.kcb) + (size_t)kvh * 256 + c);
      Entry* row = reinterpret_cast<Entry*>(smem + c * 256 + role * 128);
#pragma unroll 4
      for (int k = 0; k < REPL; ++k) row[(k + threadIdx.x) & (REPL - 1)] = e;
    }
  } else if constexpr (MODE == VQKV_MODE_VQ125) {
#pragma unroll 2
    for (int i = threadIdx.x; i < 1024 * ROLES; i += N) {
      const uint32_t c = i & 1023;
      const uint4 e = __ldg(reinterpret_cast<const uint4*>(i >> 10 ? p.vcb : p.kcb) + (size_t)kvh * 1024 + c);
      unsigned char* row = smem + (i >> 10) * 65536 + cb10_offset(c);
#pragma unroll
      for (int k = 0; k < 4; ++k) *reinterpret_cast<uint4*>(row + 32 * ((k + (c >> 1)) & 3)) = e;
    }
  } else {
    constexpr int PER = MODE == VQKV_MODE_VQ3 ? 2048 : 4096;   // 16-byte pieces per role
#pragma unroll 4
    for (int i = threadIdx.x; i < ROLES * PER; i += N) {
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
                                           uint32_t (&w)[CodeGeo<MODE>::W]) {
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

// Writes 4, 8 or 16 bytes (T) at byte `at` of token row `row` of a tile of TOK
// tokens: two 64-channel halves, 128-byte rows, 16-byte pieces swizzled by the row.
template <int TOK, typename T>
__device__ __forceinline__ void put_tile(unsigned char* tile, int row, int at, T v) {
  *reinterpret_cast<T*>(tile + (at >> 7) * (TOK * 128) + row * 128 + ((((at >> 4) & 7) ^ (row & 7)) << 4) + (at & 15)) = v;
}

// A lane's share of 16 dequantised tokens: 128 bytes, gathered into registers
// before the ring stage it goes to is known to be free.
struct Centroids {
  uint32_t r[32];
  __device__ __forceinline__ void set(int i, uint32_t v) { r[i] = v; }
  __device__ __forceinline__ void set(int i, uint2 v) { r[2 * i] = v.x, r[2 * i + 1] = v.y; }
  __device__ __forceinline__ void set(int i, uint4 v) {
    r[4 * i] = v.x, r[4 * i + 1] = v.y, r[4 * i + 2] = v.z, r[4 * i + 3] = v.w;
  }
  template <typename T>
  __device__ __forceinline__ T get(int i) const;
};
template <>
__device__ __forceinline__ uint32_t Centroids::get<uint32_t>(int i) const {
  return r[i];
}
template <>
__device__ __forceinline__ uint2 Centroids::get<uint2>(int i) const {
  return make_uint2(r[2 * i], r[2 * i + 1]);
}
template <>
__device__ __forceinline__ uint4 Centroids::get<uint4>(int i) const {
  return make_uint4(r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
}

// Gathers the lane's share of 16 key tokens: lane (gid, tig) holds the codes
// of tokens gid, gid + 8 for every fourth subvector; entry 2S (token gid) and
// 2S + 1 (gid + 8) of step S.  Lanes of odd gid take the subvectors two (8-byte
// centroids) or one (16-byte) steps apart from those of even gid: with the
// rows' swizzle the lanes of a store phase then fall on distinct banks.
template <int MODE>
__device__ __forceinline__ void gather_k(const unsigned char* s_cb, int lane, const uint32_t (&w)[CodeGeo<MODE>::W],
                                         Centroids& c) {
  const int gid = lane >> 2, tig = lane & 3;
  const uint32_t odd = gid & 1;
  if constexpr (MODE == VQKV_MODE_VQ2) {
    const uint32_t kb = (uint32_t)(lane & 15) << 3, rot = odd ? 0x1032u : 0x3210u;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t g = __byte_perm(w[i], 0u, rot), h = __byte_perm(w[2 + i], 0u, rot);
      c.set(8 * i, lds_at<uint2>(s_cb, cb_offset<0>(g, kb)));
      c.set(8 * i + 1, lds_at<uint2>(s_cb, cb_offset<0>(h, kb)));
      c.set(8 * i + 2, lds_at<uint2>(s_cb, cb_offset<1>(g, kb)));
      c.set(8 * i + 3, lds_at<uint2>(s_cb, cb_offset<1>(h, kb)));
      c.set(8 * i + 4, lds_at<uint2>(s_cb, cb_offset<2>(g, kb)));
      c.set(8 * i + 5, lds_at<uint2>(s_cb, cb_offset<2>(h, kb)));
      c.set(8 * i + 6, lds_at<uint2>(s_cb, cb_offset<3>(g, kb)));
      c.set(8 * i + 7, lds_at<uint2>(s_cb, cb_offset<3>(h, kb)));
    }
  } else if constexpr (MODE == VQKV_MODE_VQ4) {
    const uint32_t kb = (uint32_t)lane << 2;
#pragma unroll
    for (int i = 0; i < 4; ++i) {   // steps 4i .. 4i + 3: bytes 0..3 of the tokens' words i
      const uint32_t g = w[i], h = w[4 + i];
      c.set(8 * i, lds_at<uint32_t>(s_cb, cb_offset<0>(g, kb)));
      c.set(8 * i + 1, lds_at<uint32_t>(s_cb, cb_offset<0>(h, kb)));
      c.set(8 * i + 2, lds_at<uint32_t>(s_cb, cb_offset<1>(g, kb)));
      c.set(8 * i + 3, lds_at<uint32_t>(s_cb, cb_offset<1>(h, kb)));
      c.set(8 * i + 4, lds_at<uint32_t>(s_cb, cb_offset<2>(g, kb)));
      c.set(8 * i + 5, lds_at<uint32_t>(s_cb, cb_offset<2>(h, kb)));
      c.set(8 * i + 6, lds_at<uint32_t>(s_cb, cb_offset<3>(g, kb)));
      c.set(8 * i + 7, lds_at<uint32_t>(s_cb, cb_offset<3>(h, kb)));
    }
  } else if constexpr (MODE == VQKV_MODE_VQ3) {
#pragma unroll
    for (int P = 0; P < 2; ++P) {   // pairs P and P + 2 of each token, in the lane's order
      const uint32_t a0 = pair_at(w, 3 * P), a2 = pair_at(w, 3 * P + 6);
      const uint32_t b0 = pair_at(w, 12 + 3 * P), b2 = pair_at(w, 18 + 3 * P);
      const uint32_t pg[2] = {odd ? a2 : a0, odd ? a0 : a2}, ph[2] = {odd ? b2 : b0, odd ? b0 : b2};
#pragma unroll
      for (int q = 0; q < 4; ++q) {   // step S = P + 2 (q & 1) + 4 (q >> 1): low code for S < 4
        const int S = P + 2 * (q & 1) + 4 * (q >> 1);
        c.set(2 * S, lds_at<uint2>(s_cb, (q < 2 ? (pg[q & 1] & 0xfffu) : (pg[q & 1] >> 12)) << 3));
        c.set(2 * S + 1, lds_at<uint2>(s_cb, (q < 2 ? (ph[q & 1] & 0xfffu) : (ph[q & 1] >> 12)) << 3));
      }
    }
  } else if constexpr (MODE == VQKV_MODE_VQ15) {
    // pairs tig, tig + 4 of token gid, then of token gid + 8; low code for s2 < 2
    const uint32_t a0 = pair24(w[0], w[1], w[2], 0), a1 = pair24(w[0], w[1], w[2], 1);
    const uint32_t b0 = pair24(w[0], w[1], w[2], 2), b1 = pair24(w[0], w[1], w[2], 3);
    const uint32_t pa[2] = {odd ? a1 : a0, odd ? a0 : a1}, pb[2] = {odd ? b1 : b0, odd ? b0 : b1};
#pragma unroll
    for (int s2 = 0; s2 < 4; ++s2) {
      c.set(2 * s2, lds_at<uint4>(s_cb, (s2 < 2 ? (pa[s2 & 1] & 0xfffu) : (pa[s2 & 1] >> 12)) << 4));
      c.set(2 * s2 + 1, lds_at<uint4>(s_cb, (s2 < 2 ? (pb[s2 & 1] & 0xfffu) : (pb[s2 & 1] >> 12)) << 4));
    }
  } else {
    const uint32_t kb = (uint32_t)tig << 5;
#pragma unroll
    for (int s2 = 0; s2 < 4; ++s2) {
      const uint32_t a0 = bits10(w, 10 * s2), a1 = bits10(w, 10 * (s2 ^ 1));
      const uint32_t b0 = bits10(w, 40 + 10 * s2), b1 = bits10(w, 40 + 10 * (s2 ^ 1));
      c.set(2 * s2, lds_at<uint4>(s_cb, kb + cb10_offset(odd ? a1 : a0)));
      c.set(2 * s2 + 1, lds_at<uint4>(s_cb, kb + cb10_offset(odd ? b1 : b0)));
    }
  }
}

// Writes them as rows 16u + gid, 16u + gid + 8 of a tile.
template <int MODE, int TOK>
__device__ __forceinline__ void put_k(unsigned char* tile, int u, int lane, const Centroids& c) {
  using T = typename std::conditional<MODE == VQKV_MODE_VQ4, uint32_t,
                                      typename std::conditional<MODE == VQKV_MODE_VQ2 || MODE == VQKV_MODE_VQ3, uint2,
                                                                uint4>::type>::type;
  constexpr int STEP = 4 * (int)sizeof(T);   // the four lanes of a step are neighbours
  const int gid = lane >> 2, tig = lane & 3, r0 = 16 * u + gid;
  const int at = (int)sizeof(T) * tig + (MODE == VQKV_MODE_VQ4 ? 0 : 64 * (gid & 1));   // byte (STEP S) ^ at
#pragma unroll
  for (int S = 0; S < 256 / STEP; ++S) {
    put_tile<TOK>(tile, r0, (STEP * S) ^ at, c.get<T>(2 * S));
    put_tile<TOK>(tile, r0 + 8, (STEP * S) ^ at, c.get<T>(2 * S + 1));
  }
}

// The same for 16 value tokens: lane (gid, tig) holds the codes of tokens 2tig,
// 2tig + 1, 2tig + 8, 2tig + 9 (slots k) for the subvectors j with j % 8 ==
// gid; entry 4i + k is subvector gid + 8i of slot k.
template <int MODE>
__device__ __forceinline__ void gather_v(const unsigned char* s_cb, int lane, const uint32_t (&w)[CodeGeo<MODE>::W],
                                         Centroids& c) {
  const int gid = lane >> 2, tig = lane & 3;
  if constexpr (MODE == VQKV_MODE_VQ2 || MODE == VQKV_MODE_VQ4) {
    using T = typename std::conditional<MODE == VQKV_MODE_VQ2, uint2, uint32_t>::type;
    const uint32_t vb = 128u | (MODE == VQKV_MODE_VQ2 ? (uint32_t)(lane & 15) << 3 : (uint32_t)lane << 2);
#pragma unroll
    for (int i = 0; i < (MODE == VQKV_MODE_VQ2 ? 4 : 8); ++i) {
      c.set(4 * i, lds_at<T>(s_cb, cb_offset<0>(w[i], vb)));
      c.set(4 * i + 1, lds_at<T>(s_cb, cb_offset<1>(w[i], vb)));
      c.set(4 * i + 2, lds_at<T>(s_cb, cb_offset<2>(w[i], vb)));
      c.set(4 * i + 3, lds_at<T>(s_cb, cb_offset<3>(w[i], vb)));
    }
  } else if constexpr (MODE == VQKV_MODE_VQ3) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int k = 0; k < 4; ++k) {   // pair gid + 8h of slot k: subvectors gid + 8h, gid + 8h + 16
        const uint32_t pr = pair_at(w, 6 * k + 3 * h);
        c.set(4 * h + k, lds_at<uint2>(s_cb, 32768u + ((pr & 0xfffu) << 3)));
        c.set(4 * (h + 2) + k, lds_at<uint2>(s_cb, 32768u + ((pr >> 12) << 3)));
      }
  } else if constexpr (MODE == VQKV_MODE_VQ15) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t pr = pair24(w[0], w[1], w[2], k);
      c.set(k, lds_at<uint4>(s_cb, 65536u + ((pr & 0xfffu) << 4)));
      c.set(4 + k, lds_at<uint4>(s_cb, 65536u + ((pr >> 12) << 4)));
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
      for (int k = 0; k < 4; ++k) c.set(4 * i + k, lds_at<uint4>(s_cb, vb + cb10_offset(bits10(v, 40 * k + 20 * i))));
  }
}

template <int MODE, int TOK>
__device__ __forceinline__ void put_v(unsigned char* tile, int u, int lane, const Centroids& c) {
  using T = typename std::conditional<MODE == VQKV_MODE_VQ4, uint32_t,
                                      typename std::conditional<MODE == VQKV_MODE_VQ2 || MODE == VQKV_MODE_VQ3, uint2,
                                                                uint4>::type>::type;
  const int gid = lane >> 2, r0 = 16 * u + 2 * (lane & 3);
#pragma unroll
  for (int i = 0; i < 32 / (int)sizeof(T); ++i)
#pragma unroll
    for (int k = 0; k < 4; ++k)
      put_tile<TOK>(tile, r0 + (k & 1) + 8 * (k >> 1), (int)sizeof(T) * (8 * i + gid), c.get<T>(4 * i + k));
}

// Two fp32 additions in one instruction.
__device__ __forceinline__ float2 add_f32x2(float2 a, float2 b) {
  float2 r;
  asm("{ .reg .b64 a, b, r; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5}; add.rn.f32x2 r, a, b; mov.b64 {%0, %1}, r; }"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}

// Bounded wait by a whole warp: false, with the abort flag and the device
// error bit set, when it runs out or another role gave up.  A warp that gave up
// waits for nothing more, in later pieces either: a wait's parity only tells
// neighbouring phases apart.
__device__ __forceinline__ bool tr_wait_long(const DecodeParams& p, uint32_t mbar, uint32_t parity, volatile int* abort_flag) {
  bool ok = false;
  for (uint32_t i = 0; i < p.max_polls; ++i) {
    if (mbar_try_wait(mbar, parity)) {
      ok = true;
      break;
    }
    if ((i & 31) == 31 && *abort_flag) break;
  }
  ok = __all_sync(0xffffffffu, ok);
  if (!ok && !*abort_flag) {
    *abort_flag = 1;
    atomicOr(p.err, VQKV_DEVERR_TIMEOUT);
  }
  return ok;
}
__device__ __forceinline__ bool tr_wait(const DecodeParams& p, uint32_t mbar, uint32_t parity, volatile int* abort_flag) {
  if (__all_sync(0xffffffffu, mbar_try_wait(mbar, parity))) return true;
  return tr_wait_long(p, mbar, parity, abort_flag);
}

// Waits for every product that the issuing warp (lane `issuer`) started, before
// the tiles and the tensor memory they use are given back: bounded by itself,
// whether or not a wait gave up.
__device__ __forceinline__ void drain_products(const DecodeParams& p, bool issuer, uint32_t mbar) {
  if (issuer) umma_commit(mbar);
  __syncwarp();
  bool ok = false;
  for (uint32_t i = 0; i < kTilePolls && !ok; ++i) ok = __all_sync(0xffffffffu, mbar_try_wait(mbar, 0));
  if (!ok) atomicOr(p.err, VQKV_DEVERR_TIMEOUT);
}

// The dequantising warp of (role, 16-token group u of each tile) over every
// other tile of a piece: n tiles of TOK tokens of sequence b from tile0 on,
// those whose number, counted over the CTA's pieces, has parity `half` (done:
// tiles of earlier pieces; tile k goes to stage k % STAGES of `ring`).  Codes are
// loaded PREFETCH of its tiles ahead into registers, block ids one further.
// These warps meet the others only through the ring's barriers, so they run
// ahead into the next piece while the others finish one.  False: a wait gave up.
// STREAM: every tile of the piece; it goes to one of the stages of parity `half`.
template <int MODE, int ROLE, bool PAGED, int TOK, int STAGES, bool STREAM = false>
__device__ __forceinline__ bool dequant_piece(const DecodeParams& p, int b, int kvh, int tile0, int n, int L, uint32_t done,
                                              const unsigned char* s_cb, unsigned char* ring, uint32_t full, uint32_t empty,
                                              int u, int half, int lane, volatile int* abort_flag) {
  using G = CodeGeo<MODE>;
  constexpr int PREFETCH = 2, GROUPS = TOK / 16;
  const uint8_t* codes = ROLE == VQKV_ROLE_K ? p.kc : p.vc;
  const int last_group = (L + 15) >> 4;   // 16-token groups that hold tokens
  uint32_t w[PREFETCH][G::W];
  bool bad = false;
  constexpr int NEXT = STREAM ? 1 : 2;
  const int mine = STREAM ? 0 : (int)((done + half) & 1);   // its first tile
  // byte offset of the layout tile of this warp's group of tile t, -1 past the sequence
  const int t_end = min(n, (last_group - u + GROUPS - 1) / GROUPS - tile0);   // tiles whose group u holds tokens
  constexpr int STEP = TOK / G::LAYOUT_TOK * G::TILE_BYTES;
  auto layout_tile = [&](int t) { return (GROUPS * (tile0 + t) + u) / (G::LAYOUT_TOK / 16); };
  const long long first = PAGED ? 0 : tile_offset<false>(p, b, kvh, layout_tile(0), G::TILE_BYTES, &bad);
  auto place = [&](int t) -> long long {
    if (t >= t_end) return -1;
    if (!PAGED) return first + (long long)t * STEP;
    return tile_offset<PAGED>(p, b, kvh, layout_tile(t), G::TILE_BYTES, &bad);
  };
  auto fetch = [&](long long off, uint32_t (&x)[G::W]) {
    if (off >= 0) {
      load_words<MODE, ROLE>(codes, off, u & 3, lane, x);
    } else {
#pragma unroll
      for (int i = 0; i < G::W; ++i) x[i] = 0u;
    }
  };
#pragma unroll
  for (int d = 0; d < PREFETCH; ++d) fetch(place(mine + NEXT * d), w[d]);
  long long next = place(mine + NEXT * PREFETCH);
  for (int t0 = mine; t0 < n; t0 += NEXT * PREFETCH) {
#pragma unroll
    for (int d = 0; d < PREFETCH; ++d) {
      const int t = t0 + NEXT * d;
      if (t >= n) break;
      const uint32_t k = done + t, st = STREAM ? 2 * (k % (STAGES / 2)) + half : k % STAGES;
      const uint32_t round = STREAM ? k / (STAGES / 2) : k / STAGES;
      Centroids c;   // the gathers need no free stage: their latency overlaps the wait
      if constexpr (ROLE == VQKV_ROLE_K)
        gather_k<MODE>(s_cb, lane, w[d], c);
      else
        gather_v<MODE>(s_cb, lane, w[d], c);
      fetch(next, w[d]);
      next = place(t + NEXT * (PREFETCH + 1));
      if (!tr_wait(p, empty + 8 * st, (round & 1) ^ 1, abort_flag)) return false;
      unsigned char* tile = ring + st * (TOK * 256);
      if constexpr (ROLE == VQKV_ROLE_K)
        put_k<MODE, TOK>(tile, u, lane, c);
      else
        put_v<MODE, TOK>(tile, u, lane, c);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(full + 8 * st);
    }
  }
  if (PAGED && bad && lane == 0) atomicOr(p.err, VQKV_DEVERR_BLOCK);
  return true;
}

// A CTA's pieces: the overlaps of its share with the sequences, in order.
struct Pieces {
  const int* pref;   // tiles of the sequences before each
  int B, r0, r1;     // the share: tiles [r0, r1) of all sequences' tiles
  int b, tile0, n;   // the current piece: n tiles of sequence b from tile0 on
  int all;           // tiles of sequence b

  __device__ __forceinline__ Pieces(const int* pref_, int B_, int split, int n_splits) : pref(pref_), B(B_), b(-1) {
    const int T = pref[B], S = min(n_splits, T);
    r0 = split < S ? (int)((long long)T * split / S) : 0;
    r1 = split < S ? (int)((long long)T * (split + 1) / S) : 0;
    if (r1 > r0) {   // the last sequence that starts at or before r0
      int lo = 0, hi = B - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (pref[mid] <= r0) lo = mid; else hi = mid - 1;
      }
      b = lo - 1;
    }
  }
  __device__ __forceinline__ bool empty() const { return r1 <= r0; }
  __device__ __forceinline__ bool next() {
    if (empty()) return false;
    while (++b < B) {
      const int lo = pref[b], hi = pref[b + 1];
      if (lo >= r1) return false;
      if (hi == lo) continue;
      all = hi - lo;
      tile0 = max(r0, lo) - lo;
      n = min(r1, hi) - lo - tile0;
      return true;
    }
    return false;
  }
};
__device__ __forceinline__ int clamped_len(const DecodeParams& p, int b) {
  return min(max(p.seq_lens[b], 0), p.max_seq_len);
}


// The Walsh-Hadamard transform of a column whose channels 32 part .. 32 part +
// 31 this lane holds, part = lane % 4, times scale.  Five stages are in
// registers, two across the column's four lanes (a lane with 4 channels would
// need five across lanes: 20 shuffles per column and lane instead of 8).  Whole
// warps.
__device__ __forceinline__ void fwht_column(float (&v)[32], int part, float scale) {
#pragma unroll
  for (int h = 1; h < 32; h <<= 1)
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (!(i & h)) {
        const float x = v[i], y = v[i + h];
        v[i] = x + y, v[i + h] = x - y;
      }
#pragma unroll
  for (int h = 1; h < 4; h <<= 1) {
    const float sign = (part & h) ? -1.f : 1.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __fmaf_rn(v[i], sign, __shfl_xor_sync(0xffffffffu, v[i], h));
  }
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] *= scale;
}

// Units of a cross attention's items (a group of up to COLS columns of one
// sequence over a tile of TOK tokens): s_pref[b] = units of sequences 0 .. b - 1.
// All threads.
template <int TOK>
__device__ __forceinline__ void item_prefix(const DecodeParams& p, int cols, int* s_pref, bool report) {
  const int lane = threadIdx.x & 31;
  for (int b = threadIdx.x; b < p.B; b += blockDim.x) {
    const int raw = p.seq_lens[b], L = min(max(raw, 0), p.max_seq_len);
    if (report && raw != L) atomicOr(p.err, VQKV_DEVERR_SEQ_LEN);
    s_pref[b + 1] = (row_range(p, b, report).n * p.g + cols - 1) / cols * ((L + TOK - 1) / TOK);
  }
  if (threadIdx.x == 0) s_pref[0] = 0;
  __syncthreads();
  if (threadIdx.x < 32) {   // inclusive scan, 32 entries per step
    int carry = 0;
    for (int base = 0; base < p.B; base += 32) {
      const int i = base + lane;
      int v = i < p.B ? s_pref[i + 1] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += t;
      }
      if (i < p.B) s_pref[i + 1] = v + carry;
      carry += __shfl_sync(0xffffffffu, v, 31);
    }
  }
  __syncthreads();
}

// The last sequence that starts at or before unit x (x below the total).
__device__ __forceinline__ int sequence_of(const int* pref, int B, int x) {
  int lo = 0, hi = B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (pref[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// A CTA's pieces of a cross attention: the overlaps of its share with the items.
template <int TOK, int COLS>
struct ItemPieces {
  const DecodeParams& p;
  const int* pref;
  int at, r1;        // the share's units not yet taken: [at, r1)
  int b, tile0, n;   // the current piece: n tiles of sequence b from tile0 on
  int all, group;    // tiles of sequence b, the item's group of columns

  __device__ __forceinline__ ItemPieces(const DecodeParams& p_, const int* pref_, int split, int n_splits) : p(p_), pref(pref_) {
    const int T = pref[p.B], S = min(n_splits, T);
    at = split < S ? (int)((long long)T * split / S) : 0;
    r1 = split < S ? (int)((long long)T * (split + 1) / S) : 0;
    b = at < r1 ? sequence_of(pref, p.B, at) : 0;
    n = 0;
  }
  __device__ __forceinline__ bool next() {
    if (at >= r1) return false;
    while (pref[b + 1] <= at) ++b;   // at < r1 <= pref[B]
    all = (min(max(__ldg(p.seq_lens + b), 0), p.max_seq_len) + TOK - 1) / TOK;
    const int local = at - pref[b];
    group = local / all;
    tile0 = local - group * all;
    n = min(all - tile0, r1 - at);
    at += n;
    return true;
  }
  // After the last piece: (sequence, group, parts of its item, 0) if the item began in
  // this share and ends in another, else no parts.
  __device__ __forceinline__ int4 split_item(int split, int n_splits) const {
    const int T = pref[p.B], S = min(n_splits, T);
    if (split >= S || n == 0 || tile0 != 0 || n == all) return make_int4(0, 0, 0, 0);
    return make_int4(b, group, flat_cta_of(pref[b] + (group + 1) * all - 1, T, S) - split + 1, 0);
  }
};

// q' (scaled) of softmax column c of (sequence b, KV head kvh), zeros past the
// last column: channels 32 part .. 32 part + 31 in this lane, part = lane % 4.
// Whole warps.
__device__ __forceinline__ void transform_column(const DecodeParams& p, int b, int kvh, int c, int part, float (&v)[32]) {
  if (c < p.ncols) {
    const int m = c / p.g, hq = kvh * p.g + c - m * p.g;
    const float4* s4 = reinterpret_cast<const float4*>(p.s + (size_t)kvh * kHeadDim + 32 * part);
    const uint2* q = reinterpret_cast<const uint2*>(p.q + (((size_t)b * p.M + m) * p.Hq + hq) * kHeadDim + 32 * part);
#pragma unroll
    for (int i = 0; i < 8; ++i) {   // q is 8-byte aligned
      const uint2 x = q[i];
      const float4 f = s4[i];
      const float2 lo = __half22float2(*reinterpret_cast<const __half2*>(&x.x));
      const float2 hi = __half22float2(*reinterpret_cast<const __half2*>(&x.y));
      v[4 * i] = lo.x * f.x, v[4 * i + 1] = lo.y * f.y, v[4 * i + 2] = hi.x * f.z, v[4 * i + 3] = hi.y * f.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = 0.f;
  }
  fwht_column(v, part, p.qscale);
}

}  // namespace
}  // namespace vqkv
