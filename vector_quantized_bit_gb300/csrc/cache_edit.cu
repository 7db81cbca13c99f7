// Editing a packed cache under a running model: which tokens a sequence keeps
// (vqkv_evict_select) and the in-place move of chosen tokens
// (vqkv_cache_compact).
#include "common.cuh"
#include "internal.h"

namespace vqkv {
namespace {

// ------------------------------------------------------------------ clusters
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync() {
  cluster_arrive();
  cluster_wait();
}
// Shared address of the same variable in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t cluster_addr(uint32_t saddr, uint32_t rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(saddr), "r"(rank));
  return a;
}
__device__ __forceinline__ void cluster_add(uint32_t a, uint32_t v) {
  asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t cluster_ld(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void cluster_st(uint32_t a, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}

template <typename... Args>
cudaError_t launch_cluster(void (*kernel)(Args...), dim3 grid, int cluster, int threads, size_t smem, cudaStream_t stream,
                           const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// ------------------------------------------------------------------ compaction
//
// Token d = start + i of a stream takes the bytes of token src[i] >= d.  In
// place this is safe when every read of a source happens before the write of
// that position.  A cluster of CTAs owns one stream and walks it in rounds of
// consecutive destination tokens; a round's sources are >= its destinations,
// so its writes can only hit sources of the same or an earlier round.  Hence:
// read a round into registers, arrive at the cluster barrier (this CTA's reads
// of this and of earlier rounds are done), issue the reads of the next round,
// wait for the cluster, write the round.
//
// Bound: latency of the dependent loads (source index, then the source's
// bytes): the indices are loaded two rounds ahead, the bytes one.  65,536 kept
// tokens of 196,608 (8 KV heads, 2 bit, weights): 42 us; a token's V bytes lie in
// eight sectors of its group, so 99 MB are read for 36 MB moved.
//
// The layouts keep every token's bytes to itself, spread over the 32 lanes'
// runs of a 16-token group (include/vqkv.h).  A lane of the destination group
// gathers its run: a K run holds SLOTS = 2 tokens (gid, gid + 8), a V run 4
// (2tig, 2tig + 1, 2tig + 8, 2tig + 9), each SB bytes, and only the run of
// the source token's own lane position is read.

constexpr int CP_WARPS = 16;
constexpr int CP_THREADS = CP_WARPS * 32;

template <int BYTES>
struct Bytes {
  uint32_t w[(BYTES + 3) / 4];
};

__device__ __forceinline__ uint32_t ld16(const uint8_t* p) {
  uint16_t v;
  asm volatile("ld.global.u16 %0, [%1];" : "=h"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t ld32(const uint8_t* p) {
  uint32_t v;
  asm volatile("ld.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ uint2 ld64(const uint8_t* p) {
  uint2 v;
  asm volatile("ld.global.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ uint4 ld128(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
  return v;
}

// Bytes a token has in one lane's run, and the run's words.
template <int MODE, int ROLE>
struct RunGeo {
  static constexpr int SLOTS = ROLE == VQKV_ROLE_K ? 2 : 4;
  static constexpr int W = MODE == VQKV_MODE_VQ2    ? 4
                           : MODE == VQKV_MODE_VQ4  ? 8
                           : MODE == VQKV_MODE_VQ3  ? 6
                           : MODE == VQKV_MODE_VQ15 ? 3
                                                    : (ROLE == VQKV_ROLE_K ? 3 : 5);
  static constexpr int SB = MODE == VQKV_MODE_VQ125 ? 5 : W * 4 / SLOTS;
  // V runs of the byte codes interleave their tokens: byte k of every word is slot k
  static constexpr bool INTERLEAVED = ROLE == VQKV_ROLE_V && (MODE == VQKV_MODE_VQ2 || MODE == VQKV_MODE_VQ4);
};

// The SB bytes of token r (0..15) of a 16-token group in the run of lane
// position x (K: x = tig, V: x = gid); p: the group's tile, u: the group
// within it (1.5 bit).
template <int MODE, int ROLE>
__device__ __forceinline__ Bytes<RunGeo<MODE, ROLE>::SB> load_slot(const uint8_t* p, int r, int u, int x) {
  Bytes<RunGeo<MODE, ROLE>::SB> o;
  const int L = ROLE == VQKV_ROLE_K ? 4 * (r & 7) + x : 4 * x + ((r & 7) >> 1);
  const int slot = ROLE == VQKV_ROLE_K ? r >> 3 : (r & 1) + 2 * (r >> 3);
  if constexpr (RunGeo<MODE, ROLE>::INTERLEAVED) {
    const uint32_t sel = 0x0040u + (uint32_t)slot * 0x0011u;   // byte `slot` of two words
#pragma unroll
    for (int h = 0; h < RunGeo<MODE, ROLE>::W / 4; ++h) {
      const uint4 a = ld128(p + 512 * h + 16 * L);
      o.w[h] = __byte_perm(__byte_perm(a.x, a.y, sel), __byte_perm(a.z, a.w, sel), 0x5410);
    }
  } else if constexpr (MODE == VQKV_MODE_VQ2) {
    const uint2 a = ld64(p + 16 * L + 8 * slot);
    o.w[0] = a.x, o.w[1] = a.y;
  } else if constexpr (MODE == VQKV_MODE_VQ4) {
    const uint4 a = ld128(p + 512 * slot + 16 * L);
    o.w[0] = a.x, o.w[1] = a.y, o.w[2] = a.z, o.w[3] = a.w;
  } else if constexpr (MODE == VQKV_MODE_VQ3 && ROLE == VQKV_ROLE_K) {
    o.w[0] = ld32(p + 16 * L + 12 * slot);   // run bytes 0..11 or 12..23 (plane 1 from byte 16)
    const uint2 a = ld64(slot ? p + 512 + 8 * L : p + 16 * L + 8);
    const uint32_t mid = slot ? a.x : ld32(p + 16 * L + 4);
    o.w[1] = mid, o.w[2] = slot ? a.y : a.x;
  } else if constexpr (MODE == VQKV_MODE_VQ3) {
    // run bytes 6 slot .. + 5 of the words (6 slot) / 4 and the next (plane 1 from word 4)
    const int i = (6 * slot) >> 2, sh = 16 * (slot & 1);
    auto word = [&](int n) { return ld32(n < 4 ? p + 16 * L + 4 * n : p + 512 + 8 * L + 4 * (n - 4)); };
    const uint32_t a = word(i), b = word(i + 1);
    o.w[0] = __funnelshift_r(a, b, sh), o.w[1] = b >> sh;
  } else if constexpr (MODE == VQKV_MODE_VQ15 && ROLE == VQKV_ROLE_K) {
    const uint8_t* q = p + 48 * L + 12 * u + 4 * slot;   // words slot, slot + 1 of the lane's 12 bytes
    const uint32_t a = ld32(q), b = ld32(q + 4);
    o.w[0] = __funnelshift_r(a, b, 16 * slot), o.w[1] = b >> (16 * slot);
  } else if constexpr (MODE == VQKV_MODE_VQ15) {
    // bytes 3 slot .. + 2: words (3 slot) / 4 (at most the second) and the next
    const int i = slot < 3 ? (3 * slot) >> 2 : 1;
    const uint8_t* q = p + 48 * L + 12 * u + 4 * i;
    const uint32_t a = ld32(q), b = ld32(q + 4);
    o.w[0] = slot < 3 ? __funnelshift_r(a, b, 24 * slot - 32 * i) : b >> 8;
  } else if constexpr (ROLE == VQKV_ROLE_K) {   // 80-bit run: 8 bytes, then 2 in plane 1
    const uint2 a = ld64(p + 8 * L);
    const uint32_t c = ld16(p + 256 + 2 * L);
    o.w[0] = slot ? __funnelshift_r(a.y, c, 8) : a.x;   // bytes 5 .. 8 or 0 .. 3
    o.w[1] = slot ? c >> 8 : a.y;                       // byte 9 or 4
  } else {   // 160-bit run: words (5 slot) / 4 and the next (the fifth in plane 1)
    const uint32_t a = ld32(p + 16 * L + 4 * slot);
    const uint32_t b = ld32(slot < 3 ? p + 16 * L + 4 * slot + 4 : p + 256 + 4 * L);
    o.w[0] = __funnelshift_r(a, b, 8 * slot), o.w[1] = b >> (8 * slot);
  }
  return o;
}

// Slot k's bytes into the run (k is a constant after unrolling).
template <int MODE, int ROLE>
__device__ __forceinline__ void put_slot(uint32_t (&run)[RunGeo<MODE, ROLE>::W], int k,
                                         const Bytes<RunGeo<MODE, ROLE>::SB>& v) {
  using G = RunGeo<MODE, ROLE>;
  if constexpr (G::INTERLEAVED) {
#pragma unroll
    for (int i = 0; i < G::W; ++i) run[i] |= ((v.w[i >> 2] >> (8 * (i & 3))) & 0xffu) << (8 * k);
  } else {
#pragma unroll
    for (int n = 0; n < G::SB; ++n) {
      const uint32_t byte = (v.w[n >> 2] >> (8 * (n & 3))) & 0xffu;
      const int at = G::SB * k + n;
      run[at >> 2] |= byte << (8 * (at & 3));
    }
  }
}

// The lane's run of a 16-token group.
template <int MODE, int ROLE>
__device__ __forceinline__ void store_run(uint8_t* p, int u, int lane, const uint32_t (&w)[RunGeo<MODE, ROLE>::W]) {
  if constexpr (MODE == VQKV_MODE_VQ2) {
    *reinterpret_cast<uint4*>(p + 16 * lane) = make_uint4(w[0], w[1], w[2], w[3]);
  } else if constexpr (MODE == VQKV_MODE_VQ4) {
    *reinterpret_cast<uint4*>(p + 16 * lane) = make_uint4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<uint4*>(p + 512 + 16 * lane) = make_uint4(w[4], w[5], w[6], w[7]);
  } else if constexpr (MODE == VQKV_MODE_VQ3) {
    *reinterpret_cast<uint4*>(p + 16 * lane) = make_uint4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<uint2*>(p + 512 + 8 * lane) = make_uint2(w[4], w[5]);
  } else if constexpr (MODE == VQKV_MODE_VQ15) {
    uint32_t* q = reinterpret_cast<uint32_t*>(p + 48 * lane + 12 * u);
    q[0] = w[0], q[1] = w[1], q[2] = w[2];
  } else if constexpr (ROLE == VQKV_ROLE_K) {
    *reinterpret_cast<uint2*>(p + 8 * lane) = make_uint2(w[0], w[1]);
    *reinterpret_cast<uint16_t*>(p + 256 + 2 * lane) = (uint16_t)w[2];
  } else if (lane < 16) {   // 16 runs, each with the four tokens of two lane columns
    *reinterpret_cast<uint4*>(p + 16 * lane) = make_uint4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<uint32_t*>(p + 256 + 4 * lane) = w[4];
  }
}

// The call's view of one (sequence, KV head): destinations start .. start + n - 1.
struct Move {
  int b, kvh, L, start, n;
  const int32_t* src;

  __device__ __forceinline__ Move(const CompactParams& p, int b_, int kvh_, bool report) : b(b_), kvh(kvh_) {
    const int raw = p.seq_lens[b];
    L = min(max(raw, 0), p.cap_len);
    start = p.start != nullptr ? p.start[b] : 0;
    const int c = min(max(p.counts[b], 0), p.n_src);
    const bool outside = start < 0 || start > p.cap_len;   // nothing moves, nothing is cleared
    if (outside) start = L;
    n = outside ? 0 : min(c, p.cap_len - start);
    if (report && p.err != nullptr) {
      if (raw != L) atomicOr(p.err, VQKV_DEVERR_SEQ_LEN);
      if (outside || n < c) atomicOr(p.err, VQKV_DEVERR_POSITION);
    }
    src = p.src + ((size_t)b * p.src_heads + (p.src_heads > 1 ? kvh : 0)) * p.n_src;
  }
  // The token whose bytes token d takes (d itself where it stays).
  __device__ __forceinline__ int source(const CompactParams& p, int d, bool report) const {
    const int i = d - start;
    if (i < 0 || i >= n) return d;
    const int s = src[i];
    if (s >= d && s < L) return s;
    if (report && p.err != nullptr) atomicOr(p.err, VQKV_DEVERR_POSITION);
    return d;
  }
};

template <int MODE, int ROLE, bool PAGED>
__device__ __forceinline__ void move_codes(const CompactParams& p, const Move& mv, int rank, int cluster) {
  using G = RunGeo<MODE, ROLE>;
  constexpr int TT = MODE == VQKV_MODE_VQ15 ? 64 : 16;
  constexpr int TILE_BYTES = MODE == VQKV_MODE_VQ2    ? 512
                             : MODE == VQKV_MODE_VQ4  ? 1024
                             : MODE == VQKV_MODE_VQ3  ? 768
                             : MODE == VQKV_MODE_VQ15 ? 1536
                                                      : 320;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gid = lane >> 2, tig = lane & 3;
  uint8_t* codes = p.codes[ROLE];
  const int first = mv.start >> 4, last = mv.n > 0 ? (mv.start + mv.n + 15) >> 4 : first;   // 16-token groups
  constexpr int U = G::W <= 4 ? 4 : 2;   // groups per warp and round (16 words of runs at most)
  const int per = cluster * CP_WARPS * U;
  const int rounds = (last - first + per - 1) / per;
  // the warp's groups of round k are neighbours; lane l looks up token l % 16
  // of group 2 i + l / 16 (pair i of groups)
  auto first_group = [&](int k) { return first + k * per + (rank * CP_WARPS + warp) * U; };
  auto lookup = [&](int k, int (&s)[U / 2]) {
#pragma unroll
    for (int i = 0; i < U / 2; ++i) {
      const int grp = first_group(k) + 2 * i + (lane >> 4);
      s[i] = grp < last ? mv.source(p, (grp << 4) + (lane & 15), ROLE == VQKV_ROLE_K) : -1;
    }
  };
  int src[U / 2];                          // sources of the round whose bytes are loaded next
  Bytes<G::SB> v[U][G::SLOTS];             // its bytes, in flight
  long long dst[U / 2];                    // lane: tile offset of its group of pair i
  unsigned moves[U / 2];                   // tokens of pair i that move
  auto fetch = [&](int k) {
#pragma unroll
    for (int i = 0; i < U / 2; ++i) {
      // where each of the pair's 32 tokens comes from: tile offset | position within the tile
      const int grp = first_group(k) + 2 * i + (lane >> 4), d = (grp << 4) + (lane & 15);
      bool bad = false, sbad = false;
      long long from = 0;
      dst[i] = 0;
      if (grp < last) {
        dst[i] = tile_offset<PAGED>(p, mv.b, mv.kvh, d / TT, TILE_BYTES, &bad);
        from = tile_offset<PAGED>(p, mv.b, mv.kvh, src[i] / TT, TILE_BYTES, &sbad);
        if (sbad) from = dst[i], src[i] = d;
        if (PAGED && (bad || sbad) && p.err != nullptr) atomicOr(p.err, VQKV_DEVERR_BLOCK);
      }
      from |= src[i] & 63;   // tile offsets are multiples of 64
      moves[i] = __ballot_sync(0xffffffffu, grp < last && !bad && src[i] != d);
      if (moves[i] == 0) continue;   // nothing moves: leave the groups as they are
      // (a group of the pair that does not move, or lies past the last, reads
      // some token of the cache for nothing)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int q = 0; q < G::SLOTS; ++q) {
          const int r = ROLE == VQKV_ROLE_K ? gid + 8 * q : 2 * tig + (q & 1) + 8 * (q >> 1);
          const long long f = __shfl_sync(0xffffffffu, from, 16 * h + r);
          const int pos = (int)(f & 63);
          // (1.25-bit V: 16 runs, lanes 16 .. 31 repeat those of 0 .. 15)
          const int x = ROLE == VQKV_ROLE_K ? tig : MODE == VQKV_MODE_VQ125 ? gid & 3 : gid;
          v[2 * i + h][q] = load_slot<MODE, ROLE>(codes + (f & ~63LL), pos & 15, (pos >> 4) & 3, x);
        }
    }
  };
  if (rounds > 0) {
    lookup(0, src);
    fetch(0);
    if (rounds > 1) lookup(1, src);
  }
  for (int k = 0; k < rounds; ++k) {
    uint32_t w[U][G::W];
    long long place[U];   // tile offset | 16 x (group within the tile), -1: nothing to write
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const long long at = __shfl_sync(0xffffffffu, dst[j >> 1], 16 * (j & 1));
      place[j] = ((moves[j >> 1] >> (16 * (j & 1))) & 0xffffu) ? at | (((first_group(k) + j) & 3) << 4) : -1;
#pragma unroll
      for (int q = 0; q < G::W; ++q) w[j][q] = 0u;
#pragma unroll
      for (int q = 0; q < G::SLOTS; ++q) put_slot<MODE, ROLE>(w[j], q, v[j][q]);
    }
    cluster_arrive();
    if (k + 1 < rounds) {
      fetch(k + 1);
      if (k + 2 < rounds) lookup(k + 2, src);
    }
    cluster_wait();
#pragma unroll
    for (int j = 0; j < U; ++j)
      if (place[j] >= 0) store_run<MODE, ROLE>(codes + (place[j] & ~63LL), (int)((place[j] >> 4) & 3), lane, w[j]);
  }
}

// Whether the table entry of the block that holds token t is one of the pool's.
template <int TT>
__device__ __forceinline__ bool block_held(const CompactParams& p, int b, int t) {
  return (unsigned)__ldg(p.block_table + (size_t)b * p.max_blocks + ((t / TT) >> p.block_shift)) < (unsigned)p.num_blocks;
}

template <int MODE, bool PAGED>
__device__ __forceinline__ void move_mass(const CompactParams& p, const Move& mv, int rank, int cluster) {
  constexpr int U = 8, TT = MODE == VQKV_MODE_VQ15 ? 64 : 16;
  float* row = p.mass + ((size_t)mv.b * p.Hkv + mv.kvh) * p.cap_len;
  const int per = cluster * CP_THREADS * U;
  const int rounds = (mv.n + per - 1) / per;
  for (int k = 0; k < rounds; ++k) {
    float v[U];
    int s[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = k * per + (rank * U + u) * CP_THREADS + (int)threadIdx.x;
      s[u] = i < mv.n ? mv.source(p, mv.start + i, false) : -1;
      // a weight goes where its token's codes go: not into or out of a block that is not there
      if (PAGED && i < mv.n && !(block_held<TT>(p, mv.b, mv.start + i) && block_held<TT>(p, mv.b, s[u]))) s[u] = mv.start + i;
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (s[u] >= 0) v[u] = __uint_as_float(ld32(reinterpret_cast<const uint8_t*>(row + s[u])));
    cluster_sync();
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (s[u] >= 0) row[mv.start + k * per + (rank * U + u) * CP_THREADS + (int)threadIdx.x] = v[u];
  }
  // every source has been read: clear what the sequence no longer holds
  for (int t = mv.start + mv.n + rank * CP_THREADS + (int)threadIdx.x; t < mv.L; t += cluster * CP_THREADS) row[t] = 0.f;
}

// grid (cluster, Hkv x streams, B): stream 0 = K codes, 1 = V codes, 2 = mass.
template <int MODE, bool PAGED>
__global__ void __launch_bounds__(CP_THREADS, 2) compact_kernel(const CompactParams p) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int streams = p.mass != nullptr ? 3 : 2;
  const int kvh = blockIdx.y / streams, stream = blockIdx.y - kvh * streams, b = blockIdx.z;
  const Move mv(p, b, kvh, stream == 0 && kvh == 0 && blockIdx.x == 0 && threadIdx.x == 0);
  if (stream == 0)
    move_codes<MODE, VQKV_ROLE_K, PAGED>(p, mv, blockIdx.x, gridDim.x);
  else if (stream == 1)
    move_codes<MODE, VQKV_ROLE_V, PAGED>(p, mv, blockIdx.x, gridDim.x);
  else
    move_mass<MODE, PAGED>(p, mv, blockIdx.x, gridDim.x);
}

// ------------------------------------------------------------------ selection
//
// The K largest of a row of n fp32 weights, in position order.  A row belongs
// to one CTA or to a cluster, each CTA a contiguous part of it, each warp a
// contiguous piece of that.  Radix select on order-preserving 32-bit keys:
//   1. counts of the top 12 bits, added over the cluster through distributed
//      shared memory, give the bin of the K-th largest key;
//   2. each warp counts the keys above that bin and lists those inside it
//      (about 1 %: a bin is an eighth of an octave) in its own segment;
//   3. two more digits of 10 bits over the listed keys alone.  Every CTA of a
//      cluster reads all segments, so these steps exchange nothing;
//   4. the pieces are read again and the kept positions written by ballot
//      ranks: larger keys all, keys equal to the K-th while some are still
//      needed, lowest position first.
// A segment that overflows (long rows of many equal weights) sends the row
// through the digits over all its keys instead.  Steps 2 and 4 compare the
// weights as they are with the bounds' weights where 128 tokens hold nothing
// special, and come to the keys only elsewhere.
//
// Few rows: 1024 threads per CTA, one CTA per SM, the part's weights kept in
// shared memory.  More CTAs than SMs: 512 threads, two CTAs per SM, the weights
// read again from L2, which overlaps the steps of two rows (256 rows of 16,384
// to 32,768 tokens: 30.8 us, 32.6 with 1024 threads; 512 rows of 8,192: 22 and
// 30).  Bound there: a row takes 38,000 cycles beside another one, 10,000 of them
// in step 1 (memory bandwidth), 9,000 each in steps 2 and 4 (issue), the rest
// the digits' scans and barriers; issue slots are busy 55 % of the whole time.  8 rows of 196,608 in clusters of 8: 20 us, of
// which the exchange of step 1 and the remote reads of step 3 take 7.

constexpr int SEL_TOP = 12;        // bits of the first digit; the others have 10
constexpr int SEL_BINS = 1 << SEL_TOP;
constexpr int SEL_LIST = 8192;     // listed keys of a CTA, in one segment per warp
constexpr int SEL_MAX_CLUSTER = 8;
constexpr int SEL_CACHE = 36864;   // weights of a CTA's part kept in shared memory (144 KB)

// Larger weight <=> larger key; NaN below everything, -0 as +0.
__device__ __forceinline__ uint32_t weight_key(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);   // -0 + 0 = +0
  return x != x ? 0u : u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
// The weight of a key from -FLT_MAX's up (keys above +inf's give a NaN, which no weight reaches).
__device__ __forceinline__ float key_weight(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k ^ 0x80000000u : ~k);
}
constexpr uint32_t SEL_KEY_FINITE = 0x00800000u;   // key of -FLT_MAX

template <int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) evict_select_kernel(const SelectParams p) {
  constexpr int WARPS = THREADS / 32, PER = SEL_BINS / THREADS, SEG = SEL_LIST / WARPS;   // PER: bins per thread
  constexpr int U = THREADS == 512 ? 4 : 2;   // 16-byte loads in flight per thread
  extern __shared__ uint4 s_dyn[];
  uint32_t* s_hist = reinterpret_cast<uint32_t*>(s_dyn);             // [SEL_BINS]
  uint32_t* s_total = s_hist + SEL_BINS;                             // [SEL_BINS]
  uint32_t* s_list = s_total + SEL_BINS;                             // [WARPS][SEG]
  float4* s_x = reinterpret_cast<float4*>(s_list + SEL_LIST);        // [p.cache_keys / 4]
  __shared__ uint32_t s_warp[WARPS], s_warp2[WARPS];
  __shared__ uint32_t s_digit, s_above;
  __shared__ uint32_t s_listed[WARPS];                // this CTA's segments
  __shared__ uint32_t s_all[SEL_MAX_CLUSTER * WARPS];   // all CTAs'
  __shared__ uint32_t s_cta[2 * SEL_MAX_CLUSTER];       // per CTA: larger, equal
  const int CL = gridDim.x, rank = blockIdx.x, kvh = blockIdx.y, b = blockIdx.z;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_dependency_wait();
  grid_dependents_launch();
  const int raw = p.seq_lens[b], L = min(max(raw, 0), p.max_seq_len);
  if (threadIdx.x == 0 && rank == 0 && kvh == 0) {
    if (raw != L && p.err != nullptr) atomicOr(p.err, VQKV_DEVERR_SEQ_LEN);
    p.keep_lens[b] = min(L, p.n_keep);
  }
  int32_t* keep = p.keep + ((size_t)b * p.Hkv + kvh) * p.n_keep;
  if (L <= p.n_keep) {   // everything stays
    for (int t = rank * THREADS + (int)threadIdx.x; t < L; t += CL * THREADS) keep[t] = t;
    return;
  }
  // parts of WARPS pieces of whole 128-token strides: a warp walks a
  // contiguous piece, four tokens per lane
  const int piece = ((L + CL * WARPS - 1) / (CL * WARPS) + 127) & ~127;
  const int c0 = min(rank * WARPS * piece, L), c1 = min(c0 + WARPS * piece, L);
  const float* mass = p.mass + ((size_t)b * p.Hkv + kvh) * p.cap_len;
  const bool cached = WARPS * piece <= p.cache_keys;
  const bool aligned16 = (reinterpret_cast<uintptr_t>(mass) & 15) == 0;
  // weights of tokens t .. t + 3 (t a multiple of 4), 0 past the part's end
  auto load4 = [&](int t) -> float4 {
    if (aligned16 && t + 3 < c1) return *reinterpret_cast<const float4*>(mass + t);
    return make_float4(t < c1 ? mass[t] : 0.f, t + 1 < c1 ? mass[t + 1] : 0.f, t + 2 < c1 ? mass[t + 2] : 0.f,
                       t + 3 < c1 ? mass[t + 3] : 0.f);
  };
  auto x4_at = [&](int t) -> float4 { return cached ? s_x[(t - c0) >> 2] : load4(t); };
  // protected tokens rank above +inf
  const int tail = L - p.n_recent;
  auto key_of = [&](float x, int t) -> uint32_t { return t < p.n_sink || t >= tail ? 0xffffffffu : weight_key(x); };
  // 128 tokens from t on of which none is protected or past the part's end
  auto inner = [&](int t) { return t >= p.n_sink && t + 128 <= min(tail, c1); };

  uint32_t prefix = 0;                 // key bits found so far
  uint32_t need = (uint32_t)p.n_keep;  // tokens still to take among keys with that prefix
  auto clear_bins = [&] {
#pragma unroll
    for (int i = 0; i < PER; i += 4) {
      *reinterpret_cast<uint4*>(&s_hist[PER * threadIdx.x + i]) = make_uint4(0u, 0u, 0u, 0u);
      if (CL > 1) *reinterpret_cast<uint4*>(&s_total[PER * threadIdx.x + i]) = make_uint4(0u, 0u, 0u, 0u);
    }
    __syncthreads();
  };
  // The digit of the K-th largest key from the counts in s_hist (summed over the
  // cluster first, if `exchange`).
  auto next_digit = [&](int bits, bool exchange) {
    __syncthreads();
    // bins from the top: thread i holds PER of them from SEL_BINS - 1 - PER i down
    const int hi = SEL_BINS - 1 - PER * (int)threadIdx.x;
    if (exchange) {   // every CTA adds its counts (few bins have any) to every CTA's sums
      cluster_sync();   // all sums are cleared
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const uint32_t n = s_hist[threadIdx.x + i * THREADS];
        if (n != 0)
          for (int r = 0; r < CL; ++r) cluster_add(cluster_addr(smem_u32(&s_total[threadIdx.x + i * THREADS]), r), n);
      }
      cluster_sync();
    }
    uint32_t down[PER], own = 0;
#pragma unroll
    for (int i = 0; i < PER; i += 4) {
      const uint4 x = *reinterpret_cast<const uint4*>(&(exchange ? s_total : s_hist)[hi - 3 - i]);
      down[i] = x.w, down[i + 1] = x.z, down[i + 2] = x.y, down[i + 3] = x.x;
      own += x.x + x.y + x.z + x.w;
    }
    uint32_t inc = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    if (lane == 31) s_warp[warp] = inc;
    __syncthreads();
    // tokens in the bins of the warps before this one
    uint32_t before = inc - own + __reduce_add_sync(0xffffffffu, lane < warp ? s_warp[lane] : 0u);
    if (before < need && need <= before + own) {   // this thread's bins hold the digit
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        if (before < need && need <= before + down[i]) s_digit = hi - i, s_above = before;
        before += down[i];
      }
    }
    __syncthreads();
    prefix = (prefix << bits) | s_digit;
    need -= s_above;
  };

  const int w0 = min(c0 + warp * piece, c1), w1 = min(w0 + piece, c1);   // this warp's tokens
  clear_bins();
  for (int t0 = w0; t0 < w1; t0 += 128 * U) {
    float4 x[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (t0 + 128 * u < w1) x[u] = load4(t0 + 128 * u + 4 * lane);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = t0 + 128 * u + 4 * lane;
      if (t0 + 128 * u >= w1) break;
      if (cached) s_x[(t - c0) >> 2] = x[u];
      const float v[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
      if (inner(t0 + 128 * u)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) atomicAdd(&s_hist[weight_key(v[i]) >> (32 - SEL_TOP)], 1u);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (t + i < w1) atomicAdd(&s_hist[key_of(v[i], t + i) >> (32 - SEL_TOP)], 1u);
      }
    }
  }
  next_digit(SEL_TOP, CL > 1);

  const float* row = cached ? reinterpret_cast<const float*>(s_x) - c0 : mass;
  // Keys above the bin are counted, those inside listed.  Where no token is
  // special the weights are compared with the bin's bounds as they are.
  const uint32_t lt = (1u << lane) - 1u;
  uint32_t* seg = s_list + warp * SEG;
  uint32_t larger = 0, equal = 0, listed = 0;
  {
    const float lo = key_weight(prefix << (32 - SEL_TOP)), hi = key_weight((prefix + 1) << (32 - SEL_TOP));
    const bool finite = (prefix << (32 - SEL_TOP)) >= SEL_KEY_FINITE && prefix < SEL_BINS - 1;
    for (int t0 = w0; t0 < w1; t0 += 128 * U) {
      float4 x[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (t0 + 128 * u < w1) x[u] = x4_at(t0 + 128 * u + 4 * lane);
      uint32_t in = 0;   // bit 4 u + i: token t0 + 128 u + 4 lane + i is listed
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (t0 + 128 * u >= w1) break;
        const float v[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
        if (finite && inner(t0 + 128 * u)) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            larger += v[i] >= hi;
            in |= (uint32_t)(v[i] >= lo && !(v[i] >= hi)) << (4 * u + i);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int t = t0 + 128 * u + 4 * lane + i;
            const uint32_t bin = key_of(v[i], t) >> (32 - SEL_TOP);
            larger += t < w1 && bin > prefix;
            in |= (uint32_t)(t < w1 && bin == prefix) << (4 * u + i);
          }
        }
      }
      // one listed key of each lane per turn
      for (uint32_t who; (who = __ballot_sync(0xffffffffu, in != 0)) != 0; in &= in - 1) {
        const uint32_t at = listed + __popc(who & lt);
        if (in != 0 && at < SEG) {
          const int i = __ffs(in) - 1, t = t0 + 128 * (i >> 2) + 4 * lane + (i & 3);
          seg[at] = key_of(row[t], t);
        }
        listed += __popc(who);
      }
    }
  }
  if (lane == 0) s_listed[warp] = listed;
  if (CL > 1)
    cluster_sync();
  else
    __syncthreads();
  uint32_t n = 0;
  if ((int)threadIdx.x < CL * WARPS) {
    n = CL == 1 ? s_listed[lane % WARPS]
                : cluster_ld(cluster_addr(smem_u32(&s_listed[lane % WARPS]), threadIdx.x / WARPS));
    s_all[threadIdx.x] = n;
  }
  if (__syncthreads_or(n > SEG) == 0) {
    for (int pass = 1; pass < 3; ++pass) {
      clear_bins();
      auto count = [&](uint32_t k) {
        if (pass == 1)
          atomicAdd(&s_hist[(k >> 10) & 1023u], 1u);
        else if ((k >> 10) == prefix)
          atomicAdd(&s_hist[k & 1023u], 1u);
      };
      if (CL == 1) {
        for (uint32_t i = lane; i < listed; i += 32) count(seg[i]);
      } else {   // a warp reads the segments of its number in every CTA, all CTAs' loads in flight
        const uint32_t most = __reduce_max_sync(0xffffffffu, lane < CL ? s_all[lane * WARPS + warp] : 0u);
        for (uint32_t i = lane; i < ((most + 31) & ~31u); i += 32) {
          uint32_t k[SEL_MAX_CLUSTER];
          uint32_t have = 0;
#pragma unroll
          for (int r = 0; r < SEL_MAX_CLUSTER; ++r)
            if (r < CL && i < s_all[r * WARPS + warp]) {
              k[r] = cluster_ld(cluster_addr(smem_u32(seg + i), r));
              have |= 1u << r;
            }
#pragma unroll
          for (int r = 0; r < SEL_MAX_CLUSTER; ++r)
            if ((have >> r) & 1u) count(k[r]);
        }
      }
      next_digit(10, false);
    }
    for (uint32_t i = lane; i < listed; i += 32) {
      larger += (seg[i] > prefix);
      equal += (seg[i] == prefix);
    }
  } else {
    for (int pass = 1; pass < 3; ++pass) {
      const int shift = pass == 1 ? 10 : 0;
      clear_bins();
      for (int t = c0 + 4 * (int)threadIdx.x; t < c1; t += 4 * THREADS) {
        const float4 x = x4_at(t);
        const float v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t k = key_of(v[i], t + i);
          if (t + i < c1 && (k >> (shift + 10)) == prefix) atomicAdd(&s_hist[(k >> shift) & 1023u], 1u);
        }
      }
      next_digit(10, CL > 1);
    }
    larger = 0;
    for (int t = w0 + 4 * lane; t < w1; t += 128) {
      const float4 x = x4_at(t);
      const float v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t k = key_of(v[i], t + i);
        larger += t + i < w1 && k > prefix;
        equal += t + i < w1 && k == prefix;
      }
    }
  }
  // prefix is the K-th largest key; `need` of the keys equal to it are kept
  larger = __reduce_add_sync(0xffffffffu, larger);
  equal = __reduce_add_sync(0xffffffffu, equal);
  __syncthreads();
  if (lane == 0) s_warp[warp] = larger, s_warp2[warp] = equal;
  __syncthreads();
  uint32_t cl = lane < WARPS ? s_warp[lane] : 0u, ce = lane < WARPS ? s_warp2[lane] : 0u;
  uint32_t gl = __reduce_add_sync(0xffffffffu, lane < warp ? cl : 0u);
  uint32_t ge = __reduce_add_sync(0xffffffffu, lane < warp ? ce : 0u);
  if (CL > 1) {
    cl = __reduce_add_sync(0xffffffffu, cl);
    ce = __reduce_add_sync(0xffffffffu, ce);
    if ((int)threadIdx.x < CL) {
      cluster_st(cluster_addr(smem_u32(&s_cta[2 * rank]), threadIdx.x), cl);
      cluster_st(cluster_addr(smem_u32(&s_cta[2 * rank + 1]), threadIdx.x), ce);
    }
    cluster_sync();
    for (int r = 0; r < rank; ++r) gl += s_cta[2 * r], ge += s_cta[2 * r + 1];
  }
  uint32_t at = gl + min(ge, need), seen = ge;   // kept / equal tokens before this warp's piece
  const float limit = key_weight(prefix);
  const bool plain = equal == 0 && prefix >= SEL_KEY_FINITE;   // nothing of this piece ties with the K-th key
  float ahead[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) ahead[i] = w0 + 32 * i + lane < w1 ? row[w0 + 32 * i + lane] : 0.f;
  for (int t0 = w0; t0 < w1; t0 += 128) {
    float x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = t0 + 128 + 32 * i + lane;
      x[i] = ahead[i];
      if (t < w1) ahead[i] = row[t];
    }
    if (plain && inner(t0)) {
      uint32_t all[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) all[i] = __ballot_sync(0xffffffffu, x[i] > limit);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (x[i] > limit) keep[at + __popc(all[i] & lt)] = t0 + 32 * i + lane;
        at += __popc(all[i]);
      }
    } else {
#pragma unroll 1
      for (int i = 0; i < 4; ++i) {
        const int t = t0 + 32 * i + lane;
        const uint32_t k = key_of(i == 0 ? x[0] : i == 1 ? x[1] : i == 2 ? x[2] : x[3], t);
        const uint32_t eq = __ballot_sync(0xffffffffu, k == prefix && t < w1);
        const bool kept = (k > prefix && t < w1) || (((eq >> lane) & 1u) && seen + __popc(eq & lt) < need);
        seen += __popc(eq);
        const uint32_t all = __ballot_sync(0xffffffffu, kept);
        if (kept) keep[at + __popc(all & lt)] = t;
        at += __popc(all);
      }
    }
  }
}

using CompactKernel = void (*)(CompactParams);
template <int MODE>
constexpr CompactKernel compact_of(bool paged) {
  return paged ? (CompactKernel)compact_kernel<MODE, true> : (CompactKernel)compact_kernel<MODE, false>;
}

}  // namespace

static CompactKernel compact_kernel_of(int mode, bool paged) {
  return mode == VQKV_MODE_VQ2    ? compact_of<VQKV_MODE_VQ2>(paged)
         : mode == VQKV_MODE_VQ4  ? compact_of<VQKV_MODE_VQ4>(paged)
         : mode == VQKV_MODE_VQ3  ? compact_of<VQKV_MODE_VQ3>(paged)
         : mode == VQKV_MODE_VQ15 ? compact_of<VQKV_MODE_VQ15>(paged)
                                  : compact_of<VQKV_MODE_VQ125>(paged);
}

// Whether the device places clusters of 16 CTAs, beyond the portable 8, of this kernel.
template <typename K>
static bool places_clusters_of_16(K kernel, int threads, size_t smem) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(16, 1, 1);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 16;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
    cudaGetLastError();   // not an error of the call: the portable size is used
    n = 0;
  }
  return n > 0;
}

// Largest cluster the device can place: 16 CTAs where it can (beyond the
// portable 8), so that the few streams of one sequence still cover the GPU.
cudaError_t compact_prepare(int mode, int* max_cluster) {
  cudaError_t e = cudaSuccess;
  for (int paged = 0; paged < 2 && e == cudaSuccess; ++paged)
    e = cudaFuncSetAttribute(compact_kernel_of(mode, paged != 0), cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  *max_cluster = places_clusters_of_16(compact_kernel_of(mode, true), CP_THREADS, 0) ? 16 : 8;
  return cudaSuccess;
}

cudaError_t launch_compact(int mode, const CompactParams& p, int sms, int max_cluster, cudaStream_t stream) {
  const CompactKernel k = compact_kernel_of(mode, p.block_table != nullptr);
  // CTAs per stream: what moves its tokens in one round (24 streams of 4,096 kept
  // tokens at 2 bit: 15.9 us at 1, 4.8 at 4, 6.5 at 8, 9.6 at 16), up to 8 while all
  // CTAs are fewer than eight per SM (384 streams of a paged 1.25-bit batch: 113 us
  // at 1 CTA each, 88 at 4, 99 at 8).  Sixteen, beyond the portable size, only for
  // so few streams that eight would leave SMs idle: 24 streams of 65,536 kept
  // tokens 55 -> 42 us, but 96 streams of 8,192 22 -> 39 us, because few clusters
  // of 16 are placed at a time.
  const long long streams = (long long)p.B * p.Hkv * (p.mass != nullptr ? 3 : 2);
  const long long groups = ((long long)p.n_src + (p.start != nullptr ? 30 : 15)) / 16;   // a start may lie inside a group
  // groups per CTA and round (where K and V runs differ, those of K)
  const long long round = CP_WARPS * (mode == VQKV_MODE_VQ3 || mode == VQKV_MODE_VQ4 ? 2 : 4);
  int cluster = 1;
  while (cluster < 8 && cluster * round < groups && streams * cluster < 8LL * sms) cluster *= 2;
  if (cluster == 8 && max_cluster == 16 && 8 * round < groups && streams * 8 < 2LL * sms) cluster = 16;
  return launch_cluster(k, dim3(cluster, p.Hkv * (p.mass != nullptr ? 3 : 2), p.B), cluster, CP_THREADS, 0, stream, p);
}

static int select_smem(int keys) { return (2 * SEL_BINS + SEL_LIST + keys) * 4; }

cudaError_t evict_select_prepare() {
  const cudaFuncAttribute a = cudaFuncAttributeMaxDynamicSharedMemorySize;
  const cudaError_t e = cudaFuncSetAttribute(evict_select_kernel<1024>, a, select_smem(SEL_CACHE));
  return e != cudaSuccess ? e : cudaFuncSetAttribute(evict_select_kernel<512>, a, select_smem(0));
}

cudaError_t launch_evict_select(SelectParams p, int sms, cudaStream_t stream) {
  // CTAs per row: spread few rows over the GPU, but at least 4096 tokens each
  const long long rows = (long long)p.B * p.Hkv;
  int cluster = 1;
  while (cluster < SEL_MAX_CLUSTER && rows * cluster * 2 <= sms && p.max_seq_len > 4096 * cluster) cluster *= 2;
  const dim3 grid(cluster, p.Hkv, p.B);
  p.cache_keys = 0;
  if (rows * cluster > sms) return launch_cluster(evict_select_kernel<512>, grid, cluster, 512, select_smem(0), stream, p);
  // one CTA per SM
  const long long part = ((long long)p.max_seq_len + cluster * 32 - 1) / (cluster * 32);
  const long long keys = (part + 127) / 128 * 128 * 32;
  if (keys <= SEL_CACHE) p.cache_keys = (int)keys;
  return launch_cluster(evict_select_kernel<1024>, grid, cluster, 1024, (size_t)select_smem(p.cache_keys), stream, p);
}

}  // namespace vqkv
