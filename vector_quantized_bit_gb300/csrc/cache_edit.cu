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
// bytes): the indices are loaded two rounds ahead, the bytes one.
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

__device__ __forceinline__ void move_mass(const CompactParams& p, const Move& mv, int rank, int cluster) {
  constexpr int U = 8;
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
    move_mass(p, mv, blockIdx.x, gridDim.x);
}

// ------------------------------------------------------------------ selection
//
// The K largest of a row of n fp32 weights, in position order.  A cluster
// owns one (sequence, KV head) row, each CTA a contiguous part of it (kept in
// shared memory as order-preserving 32-bit keys while it fits).  Radix select
// from the top: three passes over 11, 11 and 10 key bits find the K-th
// largest key; per pass the CTAs' 2048-bin counts are added through
// distributed shared memory.  Then the kept positions are counted per warp
// and CTA, and written by ballot ranks: larger keys all, keys equal to the
// K-th while some are still needed, lowest position first.
//
// Bound: instruction issue and, in the first pass, shared-memory atomics on
// equal bins (weights share their leading bits).  So lanes take four
// neighbouring keys at a time, and four copies of the counts, one per lane % 4,
// keep equal bins of a warp apart.

constexpr int SEL_THREADS = 1024;
constexpr int SEL_WARPS = SEL_THREADS / 32;
constexpr int SEL_U = 2;           // 16-byte loads in flight per thread in the first pass
constexpr int SEL_BINS = 2048;
constexpr int SEL_COPIES = 4;
constexpr int SEL_MAX_CLUSTER = 8;
constexpr int SEL_CACHE = 40960;   // keys of a CTA's part kept in shared memory (160 KB)

// Larger weight <=> larger key; NaN below everything, -0 as +0.
__device__ __forceinline__ uint32_t weight_key(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x + 0.f);   // -0 + 0 = +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__global__ void __launch_bounds__(SEL_THREADS, 1) evict_select_kernel(const SelectParams p) {
  extern __shared__ uint4 s_dyn[];
  uint32_t* s_hist = reinterpret_cast<uint32_t*>(s_dyn);             // [SEL_COPIES][SEL_BINS]
  uint32_t* s_total = s_hist + SEL_COPIES * SEL_BINS;                // [SEL_BINS]
  uint4* s_keys = reinterpret_cast<uint4*>(s_total + SEL_BINS);      // [p.cache_keys / 4]
  __shared__ uint32_t s_warp[SEL_WARPS], s_warp2[SEL_WARPS];
  __shared__ uint32_t s_digit, s_above;
  __shared__ uint32_t s_cta[2 * SEL_MAX_CLUSTER];   // per CTA: larger, equal
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
    for (int t = rank * SEL_THREADS + (int)threadIdx.x; t < L; t += CL * SEL_THREADS) keep[t] = t;
    return;
  }
  // parts of SEL_WARPS pieces of whole 128-token strides: a warp walks a
  // contiguous piece, four tokens per lane
  const int piece = ((L + CL * SEL_WARPS - 1) / (CL * SEL_WARPS) + 127) & ~127;
  const int c0 = min(rank * SEL_WARPS * piece, L), c1 = min(c0 + SEL_WARPS * piece, L);
  const float* mass = p.mass + ((size_t)b * p.Hkv + kvh) * p.cap_len;
  const bool cached = SEL_WARPS * piece <= p.cache_keys;
  const bool aligned16 = (reinterpret_cast<uintptr_t>(mass) & 15) == 0;
  // the keys of tokens t .. t + 3 (t a multiple of 4), 0 past the part's end;
  // protected tokens rank above +inf
  auto load_keys = [&](int t) -> uint4 {
    float x[4] = {0.f, 0.f, 0.f, 0.f};
    if (aligned16 && t + 3 < c1) {
      const float4 v = *reinterpret_cast<const float4*>(mass + t);
      x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (t + i < c1) x[i] = mass[t + i];
    }
    uint32_t k[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      k[i] = t + i < p.n_sink || t + i >= L - p.n_recent ? 0xffffffffu : weight_key(x[i]);
      if (t + i >= c1) k[i] = 0u;
    }
    return make_uint4(k[0], k[1], k[2], k[3]);
  };
  auto keys_at = [&](int t) -> uint4 { return cached ? s_keys[(t - c0) >> 2] : load_keys(t); };

  uint32_t prefix = 0;                 // key bits found so far
  uint32_t need = (uint32_t)p.n_keep;  // tokens still to take among keys with that prefix
  uint32_t* hist = s_hist + (lane % SEL_COPIES) * SEL_BINS;
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const int bits = pass == 2 ? 10 : 11;
    for (int i = threadIdx.x; i < SEL_COPIES * SEL_BINS; i += SEL_THREADS) s_hist[i] = 0u;
    __syncthreads();
    const uint32_t mask = (1u << bits) - 1u;
    if (pass == 0) {
      for (int t0 = c0 + 4 * (int)threadIdx.x; t0 < c1; t0 += 4 * SEL_U * SEL_THREADS) {
        uint4 k[SEL_U];
#pragma unroll
        for (int i = 0; i < SEL_U; ++i) {
          const int t = t0 + 4 * i * SEL_THREADS;
          if (t < c1) k[i] = load_keys(t);
        }
#pragma unroll
        for (int i = 0; i < SEL_U; ++i) {
          const int t = t0 + 4 * i * SEL_THREADS;
          if (t >= c1) break;
          if (cached) s_keys[(t - c0) >> 2] = k[i];
          atomicAdd(&hist[k[i].x >> 21], 1u);
          if (t + 1 < c1) atomicAdd(&hist[k[i].y >> 21], 1u);
          if (t + 2 < c1) atomicAdd(&hist[k[i].z >> 21], 1u);
          if (t + 3 < c1) atomicAdd(&hist[k[i].w >> 21], 1u);
        }
      }
    } else {
      // (keys past the part's end are 0: with prefix 0 they would count, so the
      // bound is tested there)
      auto count = [&](uint32_t k, int t) {
        if ((k >> (shift + bits)) == prefix && t < c1) atomicAdd(&hist[(k >> shift) & mask], 1u);
      };
      for (int t = c0 + 4 * (int)threadIdx.x; t < c1; t += 4 * SEL_THREADS) {
        const uint4 k = keys_at(t);
        count(k.x, t), count(k.y, t + 1), count(k.z, t + 2), count(k.w, t + 3);
      }
    }
    __syncthreads();
    // fold the copies: bins from the top, thread i holds 2047 - 2i and 2046 - 2i
    const int hi = SEL_BINS - 1 - 2 * (int)threadIdx.x;
    uint32_t x0 = 0, x1 = 0;
#pragma unroll
    for (int c = 0; c < SEL_COPIES; ++c) {
      const uint2 v = *reinterpret_cast<const uint2*>(&s_hist[c * SEL_BINS + hi - 1]);
      x0 += v.y, x1 += v.x;
    }
    if (CL > 1) {   // this CTA adds a share of the bins over the cluster and gives every CTA the sums
      *reinterpret_cast<uint2*>(&s_hist[hi - 1]) = make_uint2(x1, x0);   // own bins of copy 0 only
      cluster_sync();
      const int share = SEL_BINS / CL;
      if ((int)threadIdx.x < share) {
        const int bin = rank * share + threadIdx.x;
        const uint32_t h = smem_u32(&s_hist[bin]), o = smem_u32(&s_total[bin]);
        uint32_t sum = 0;
        for (int r = 0; r < CL; ++r) sum += cluster_ld(cluster_addr(h, r));
        for (int r = 0; r < CL; ++r) cluster_st(cluster_addr(o, r), sum);
      }
      cluster_sync();
      x0 = s_total[hi], x1 = s_total[hi - 1];
    }
    uint32_t inc = x0 + x1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    if (lane == 31) s_warp[warp] = inc;
    __syncthreads();
    // tokens in the bins of the warps before this one (SEL_WARPS == 32)
    const uint32_t prior = __reduce_add_sync(0xffffffffu, lane < warp ? s_warp[lane] : 0u);
    const uint32_t before = inc - x0 - x1 + prior;   // tokens in higher bins
    if (before < need && need <= before + x0) {
      s_digit = hi, s_above = before;
    } else if (before + x0 < need && need <= before + x0 + x1) {
      s_digit = hi - 1, s_above = before + x0;
    }
    __syncthreads();
    prefix = (prefix << bits) | s_digit;
    need -= s_above;
  }
  // prefix is the K-th largest key; `need` of the keys equal to it are kept
  const int w0 = min(c0 + warp * piece, c1), w1 = min(w0 + piece, c1);
  uint32_t larger = 0, equal = 0;
  for (int t = w0 + 4 * lane; t < w1; t += 128) {
    const uint4 k = keys_at(t);
    larger += (k.x > prefix) + (k.y > prefix) + (k.z > prefix) + (k.w > prefix);   // 0 past the end: never larger
    equal += (k.x == prefix) + (k.y == prefix && t + 1 < c1) + (k.z == prefix && t + 2 < c1) + (k.w == prefix && t + 3 < c1);
  }
  larger = __reduce_add_sync(0xffffffffu, larger);
  equal = __reduce_add_sync(0xffffffffu, equal);
  __syncthreads();
  if (lane == 0) s_warp[warp] = larger, s_warp2[warp] = equal;
  __syncthreads();
  uint32_t cl = s_warp[lane], ce = s_warp2[lane];
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
  const uint32_t lt = (1u << lane) - 1u;
  for (int t0 = w0; t0 < w1; t0 += 128) {
    const int t = t0 + 4 * lane;
    const uint4 kk = t < w1 ? keys_at(t) : make_uint4(0u, 0u, 0u, 0u);
    const uint32_t k[4] = {kk.x, kk.y, kk.z, kk.w};
    uint32_t kept = 0, eq = 0;   // bit i: token t + i
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      kept |= (uint32_t)(k[i] > prefix) << i;
      eq |= (uint32_t)(k[i] == prefix && t + i < w1) << i;
    }
    if (__any_sync(0xffffffffu, eq != 0)) {
      const uint32_t n = __popc(eq);
      uint32_t rank_eq = seen;   // equal tokens before this lane's
#pragma unroll
      for (int q = 0; q < 3; ++q) rank_eq += __popc(__ballot_sync(0xffffffffu, (n >> q) & 1u) & lt) << q;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if ((eq >> i) & 1u) {
          if (rank_eq < need) kept |= 1u << i;
          ++rank_eq;
        }
      seen += __reduce_add_sync(0xffffffffu, n);
    }
    const uint32_t n = __popc(kept);
    uint32_t pos = at, all = 0;
#pragma unroll
    for (int q = 0; q < 3; ++q) {
      const uint32_t bal = __ballot_sync(0xffffffffu, (n >> q) & 1u);
      pos += __popc(bal & lt) << q;
      all += __popc(bal) << q;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if ((kept >> i) & 1u) keep[pos++] = t + i;
    at += all;
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

// Largest cluster the device can place: 16 CTAs where it can (beyond the
// portable 8), so that the few streams of one sequence still cover the GPU.
cudaError_t compact_prepare(int mode, int* max_cluster) {
  cudaError_t e = cudaSuccess;
  for (int paged = 0; paged < 2 && e == cudaSuccess; ++paged)
    e = cudaFuncSetAttribute(compact_kernel_of(mode, paged != 0), cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(16, 1, 1);
  cfg.blockDim = dim3(CP_THREADS);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 16;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, compact_kernel_of(mode, true), &cfg) != cudaSuccess) {
    cudaGetLastError();   // not an error of the call: the portable size is used
    n = 0;
  }
  *max_cluster = n > 0 ? 16 : 8;
  return cudaSuccess;
}

cudaError_t launch_compact(int mode, const CompactParams& p, int sms, int max_cluster, cudaStream_t stream) {
  const CompactKernel k = compact_kernel_of(mode, p.block_table != nullptr);
  // CTAs per stream: at most what one round of its destinations needs, and up to
  // 8 while all CTAs are fewer than eight per SM (384 streams of a paged
  // 1.25-bit batch: 113 us at 1 CTA each, 88 at 4, 99 at 8).  Sixteen, beyond the
  // portable size, only for so few streams that eight would leave SMs idle: 24
  // streams of 196,608 tokens 46 -> 42 us, but 96 streams of 16,384 19 -> 36 us,
  // because few clusters of 16 are placed at a time.
  const long long streams = (long long)p.B * p.Hkv * (p.mass != nullptr ? 3 : 2);
  const long long groups = ((long long)p.n_src + 30) / 16;
  int cluster = 1;
  while (cluster < 8 && (long long)cluster * CP_WARPS < groups && streams * cluster < 8LL * sms) cluster *= 2;
  if (cluster == 8 && max_cluster == 16 && 8LL * CP_WARPS < groups && streams * 8 < 2LL * sms) cluster = 16;
  return launch_cluster(k, dim3(cluster, p.Hkv * (p.mass != nullptr ? 3 : 2), p.B), cluster, CP_THREADS, 0, stream, p);
}

static int select_smem(int keys) { return ((SEL_COPIES + 1) * SEL_BINS + keys) * 4; }

cudaError_t evict_select_prepare() {
  return cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, select_smem(SEL_CACHE));
}

cudaError_t launch_evict_select(SelectParams p, int sms, cudaStream_t stream) {
  // CTAs per row: spread the rows over the GPU, but at least 4096 tokens each
  const long long rows = (long long)p.B * p.Hkv;
  int cluster = 1;
  while (cluster < SEL_MAX_CLUSTER && rows * cluster * 2 <= sms && p.max_seq_len > 4096 * cluster) cluster *= 2;
  const long long part = ((long long)p.max_seq_len + cluster * SEL_WARPS - 1) / (cluster * SEL_WARPS);
  const long long keys = (part + 127) / 128 * 128 * SEL_WARPS;
  p.cache_keys = keys <= SEL_CACHE ? (int)keys : 0;
  return launch_cluster(evict_select_kernel, dim3(cluster, p.Hkv, p.B), cluster, SEL_THREADS,
                        (size_t)select_smem(p.cache_keys), stream, p);
}

}  // namespace vqkv
