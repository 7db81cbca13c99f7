// Host side of the C ABI declared in include/vqkv.h: argument validation,
// the split-KV plan, workspace layout and kernel launches.  Nothing here
// allocates device memory or synchronises the host.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <limits>
#include <mutex>

#include "internal.h"
#include "vqkv.h"

namespace vqkv {
namespace {

constexpr int kMaxDevices = 64;
constexpr size_t kWsHeader = 256;   // word 0: device error flags
constexpr int kMaxGridYZ = 65535;   // CUDA's limit on gridDim.y and gridDim.z
constexpr int kMaxTokens = 1 << 30; // longest row of the cache-editing calls (positions plus a stride stay in 32 bits)

// Kernels that are prepared (attributes set, checks made) only when a call that
// uses them is first planned, so that no other call loads them or fails with them.
enum LazyKernels : int {
  kTreeKernels, kMassKernels, kMassTileKernels, kCompactKernels, kSelectKernels, kEncodeTileKernels, kAppendKernels,
  kAppendTileKernels, kCrossKernels, kCrossRowsKernels, kLazyKernels
};

struct DeviceInfo {
  bool ready = false;
  bool prepared[kLazyKernels][kCodeModes] = {};
  int sms = 0;
  int decode_bpsm[kCodeModes + 1] = {};   // resident decode CTAs per SM: each code mode, then fp16
  int compact_cluster[kCodeModes] = {};   // largest cluster of the compaction
};

std::mutex g_mu;
DeviceInfo g_dev[kMaxDevices];

// Per-device attributes, queried once (kernel attributes set here too).
vqkv_status device_info(DeviceInfo* out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return VQKV_ERR_NO_DEVICE;
  std::lock_guard<std::mutex> lk(g_mu);
  DeviceInfo& d = g_dev[dev];
  if (!d.ready) {
    if (cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return VQKV_ERR_NO_DEVICE;
    for (int m = 0; m < kCodeModes; ++m) {
      if (decode_prepare(m) != cudaSuccess || encode_prepare(m) != cudaSuccess) return VQKV_ERR_CUDA;
      if (decode_occupancy(m, &d.decode_bpsm[m]) != cudaSuccess) return VQKV_ERR_CUDA;
      if (d.decode_bpsm[m] < 1) d.decode_bpsm[m] = 1;
    }
    if (decode_fp16_prepare() != cudaSuccess || decode_fp16_occupancy(&d.decode_bpsm[kModeFp16]) != cudaSuccess)
      return VQKV_ERR_CUDA;
    if (d.decode_bpsm[kModeFp16] < 1) d.decode_bpsm[kModeFp16] = 1;
    d.ready = true;
  }
  *out = d;
  return VQKV_OK;
}

// device_info, and the kernels `what` of a mode ready to launch (kSelectKernels: mode 0).
vqkv_status device_info(LazyKernels what, int mode, DeviceInfo* out) {
  const vqkv_status st = device_info(out);
  if (st != VQKV_OK || out->prepared[what][mode]) return st;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return VQKV_ERR_NO_DEVICE;
  std::lock_guard<std::mutex> lk(g_mu);
  DeviceInfo& d = g_dev[dev];
  const cudaError_t e = what == kTreeKernels       ? decode_tree_prepare(mode)
                        : what == kMassKernels     ? decode_mass_prepare(mode)
                        : what == kMassTileKernels ? mass_tiles_prepare(mode)
                        : what == kCompactKernels  ? compact_prepare(mode, &d.compact_cluster[mode])
                        : what == kEncodeTileKernels ? encode_tiles_prepare(mode)
                        : what == kAppendKernels     ? append_prepare(mode, true)
                        : what == kAppendTileKernels ? append_prepare(mode, false)
                        : what == kCrossKernels    ? cross_prepare(mode)
                        : what == kCrossRowsKernels ? cross_rows_prepare(mode)
                                                   : evict_select_prepare();
  if (e != cudaSuccess) return VQKV_ERR_CUDA;
  d.prepared[what][mode] = true;
  *out = d;
  return VQKV_OK;
}

bool is_code_mode(int m) {
  return m == VQKV_MODE_VQ2 || m == VQKV_MODE_VQ15 || m == VQKV_MODE_VQ4 || m == VQKV_MODE_VQ3 ||
         m == VQKV_MODE_VQ125;
}
bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool overlap(const void* a, size_t a_bytes, const void* b, size_t b_bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y ? y - x < a_bytes : x - y < b_bytes;
}
size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// Sizes only (what the split plan and the workspace size depend on).
vqkv_status validate_decode_sizes(const vqkv_decode_args* a) {
  if (a == nullptr) return VQKV_ERR_INVALID_ARG;
  if (!is_code_mode(a->mode)) return VQKV_ERR_UNSUPPORTED;
  if (a->head_dim != 128) return VQKV_ERR_UNSUPPORTED;
  if (a->B < 0 || a->Hq < 1 || a->Hkv < 1 || a->cap_len < 1) return VQKV_ERR_INVALID_ARG;
  if (a->Hq % a->Hkv != 0) return VQKV_ERR_INVALID_ARG;
  if (a->Hq / a->Hkv > 8) return VQKV_ERR_UNSUPPORTED;
  if (a->max_seq_len < 0 || a->max_seq_len > a->cap_len) return VQKV_ERR_INVALID_ARG;
  if (a->num_splits < 0) return VQKV_ERR_INVALID_ARG;
  return VQKV_OK;
}

vqkv_status validate_decode(const vqkv_decode_args* a) {
  if (a == nullptr) return VQKV_ERR_INVALID_ARG;
  if (!is_code_mode(a->mode)) return VQKV_ERR_UNSUPPORTED;
  if (a->head_dim != 128) return VQKV_ERR_UNSUPPORTED;
  if (a->B < 0 || a->Hq < 1 || a->Hkv < 1 || a->cap_len < 1) return VQKV_ERR_INVALID_ARG;
  if (a->Hq % a->Hkv != 0) return VQKV_ERR_INVALID_ARG;
  if (a->Hq / a->Hkv > 8) return VQKV_ERR_UNSUPPORTED;
  if (a->max_seq_len < 0 || a->max_seq_len > a->cap_len) return VQKV_ERR_INVALID_ARG;
  if (a->num_splits < 0) return VQKV_ERR_INVALID_ARG;
  if (!(std::isfinite(a->softmax_scale))) return VQKV_ERR_INVALID_ARG;
  if (a->B == 0) return VQKV_OK;
  if (!a->q || !a->k_codes || !a->v_codes || !a->seq_lens || !a->k_codebook || !a->v_codebook || !a->s ||
      !a->out)
    return VQKV_ERR_INVALID_ARG;
  if (!aligned(a->q, 8) || !aligned(a->k_codes, 16) || !aligned(a->v_codes, 16) || !aligned(a->k_codebook, 16) ||
      !aligned(a->v_codebook, 16) || !aligned(a->s, 16) || !aligned(a->seq_lens, 4) || !aligned(a->out, 2))
    return VQKV_ERR_INVALID_ARG;
  return VQKV_OK;
}

// Block-table arguments of the paged calls: sizes and alignment only.
vqkv_status validate_paging(const vqkv_paging* pg, int mode, int cap_len) {
  if (pg == nullptr) return VQKV_ERR_INVALID_ARG;
  if (pg->max_blocks < 1 || pg->num_blocks < 1 || pg->block_tokens < 64 ||
      (pg->block_tokens & (pg->block_tokens - 1)) != 0)
    return VQKV_ERR_INVALID_ARG;
  if ((long long)pg->max_blocks * pg->block_tokens < cap_len) return VQKV_ERR_INVALID_ARG;
  if ((long long)pg->num_blocks * vqkv_code_bytes(mode, pg->block_tokens) > (1LL << 46)) return VQKV_ERR_INVALID_ARG;
  return VQKV_OK;
}

template <typename P>
void set_paging(P& p, const vqkv_paging* pg, int mode) {
  if (pg == nullptr) return;
  p.block_table = pg->block_table;
  p.max_blocks = pg->max_blocks;
  p.block_tiles = pg->block_tokens / decode_tile_tokens(mode);
  p.block_shift = 0;
  while ((1 << p.block_shift) < p.block_tiles) ++p.block_shift;
  p.num_blocks = pg->num_blocks;
  p.block_bytes = (long long)vqkv_code_bytes(mode, pg->block_tokens);
}

}  // namespace
size_t decode_ticket_region_bytes(int B, int Hkv);
namespace {

struct DecodePlan {
  int n_splits = 1, tps = 1, bpg = 1, n_bgroups = 1, cgroups = 1, flat = 0;
  size_t tickets_off = 0, partials_off = 0, ws_bytes = 0;
};

// Split-KV plan.  Work is (sequence group, KV head, split); every CTA of a
// split processes `tps` tiles of each sequence in its group.  The plan picks
// the split count that minimises (waves of CTAs) x (tiles per CTA + a fixed
// per-CTA setup cost), assuming full-length sequences; short sequences make
// some CTAs finish early, which the hardware scheduler backfills.
struct PlanInput {
  int mode;   // a code mode or kModeFp16
  int B, Hq, Hkv, max_seq_len, num_splits;
  int M = 1;  // queries per sequence
  // Tiles' worth of extra work in the CTA whose split holds a sequence's
  // last token (the fused append encodes the new rows there first).  When
  // every CTA of the plan runs at once, the splits are sized for
  // max_seq_len + credit_tiles, so that split comes out this much shorter.
  int credit_tiles = 0;
  int width = 8;   // softmax columns per CTA
  bool rows = false;   // packed rows (cross attention of one query per sequence)
};

vqkv_status plan_decode(const PlanInput* a, DecodePlan* pl) {
  DeviceInfo di;
  vqkv_status st = device_info(&di);
  if (st != VQKV_OK) return st;
  const int T = a->mode == kModeFp16 ? 16 : decode_tile_tokens(a->mode);
  const int unit_tiles = a->mode == kModeFp16 ? 1 : decode_tiles_per_step(a->mode);
  const int g = a->Hq / a->Hkv;
  const long long tiles_max = std::max(1, (a->max_seq_len + T - 1) / T);
  const long long slots = (long long)di.sms * di.decode_bpsm[a->mode];
  const int B = std::max(a->B, 1);
  // 1.5-bit CTAs load 128 KB of codebooks: keep one CTA per KV head and split
  // across sequences only when the batch alone cannot fill the GPU.  Not over packed
  // rows: one query of 16 sequences x 8 heads over 700 to 1,500 tokens takes 17 us with
  // a CTA each, 79 with shared ones; of 4 x 8 over 20,000 to 60,000 106 and 118.
  int bpg = 1;
  if (a->mode == VQKV_MODE_VQ15 && (long long)B * a->Hkv < slots && !a->rows) bpg = B;
  const int cgroups = (g * a->M + a->width - 1) / a->width;   // CTAs per (sequence group, KV head, split)
  const long long S = std::max<long long>(1, slots / ((long long)a->Hkv * cgroups));
  // Flat plan for batches on the tile-ring decode: one wave of CTAs per (KV
  // head, column group), each taking an equal share of all sequences' tiles,
  // balanced by the actual lengths on the device (ragged batches leave no CTA
  // idle).  Explicit split counts keep the split plan.
  const bool ring = a->mode == VQKV_MODE_VQ2 || a->mode == VQKV_MODE_VQ4 || a->mode == VQKV_MODE_VQ3 ||
                    a->mode == VQKV_MODE_VQ125;
  const long long super_max = (tiles_max + unit_tiles - 1) / unit_tiles;
  // Packed rows of short sequences: a CTA per sequence, in waves.  A share's passage from
  // sequence to sequence (prologue, merge of its warps, partial) costs as much as some
  // 175 tiles, a wave's 120; the lengths are the host's bound, of which ragged batches may
  // fill a quarter.  16 sequences x 16 heads at 2 bit: 700 to 1,500 tokens 17 us against
  // 27 in shares, 100 to 300 tokens 11 against 22; 3,000 to 8,000 (shares) 49 against 50.
  bool whole = false;
  if (ring && a->rows && a->num_splits == 0 && a->B > 1) {
    const long long waves = ((long long)B * a->Hkv * cgroups + slots - 1) / slots;
    const double tiles = (a->mode == VQKV_MODE_VQ3 ? 2.0 : 1.0) * tiles_max;   // in time: its gathers conflict
    whole = waves * (tiles + 120) <= 75 + 175.0 * (B + S) / S + 0.25 * tiles * B / S;
  }
  if (ring && !whole && a->num_splits == 0 && a->B > 1 && a->B <= kFlatMaxB && (long long)a->B * super_max < (1LL << 30)) {
    pl->flat = 1;
    pl->n_splits = (int)S;
    pl->tps = 0;
    pl->bpg = 1;
    pl->n_bgroups = 1;
    pl->cgroups = cgroups;
    pl->tickets_off = kWsHeader;
    pl->partials_off = decode_ticket_region_bytes(B, a->Hkv * cgroups);
    pl->ws_bytes = pl->partials_off +
                   sizeof(float) * (size_t)a->Hkv * (S + a->B - 1) * g * a->M * kPartialStride;
    return VQKV_OK;
  }
  const long long pairs = (long long)a->Hkv * ((B + bpg - 1) / bpg) * cgroups;
  // per-CTA prologue + merge in tile units
  const double setup_tiles = (a->mode == VQKV_MODE_VQ15) ? 24.0 : (a->mode == kModeFp16) ? 4.0 : 12.0;
  long long best_n = 1;
  double best_cost = 1e300;
  if (a->num_splits > 0) {
    best_n = std::min<long long>(a->num_splits, tiles_max);
  } else if (!whole) {
    const long long n_hi = std::min<long long>(tiles_max, 4 * ((slots + pairs - 1) / pairs) + 64);
    for (long long n = 1; n <= n_hi; ++n) {
      const long long tps = (tiles_max + n - 1) / n;
      const long long waves = (pairs * n + slots - 1) / slots;
      const double cost = (double)waves * ((double)tps * bpg + setup_tiles);
      if (cost < best_cost - 1e-9) {
        best_cost = cost;
        best_n = n;
      }
    }
  }
  const long long unit = unit_tiles;
  const bool one_wave = pairs * best_n <= slots;
  const long long credit = (a->num_splits == 0 && one_wave) ? a->credit_tiles : 0;
  const long long tps = ((tiles_max + credit + best_n - 1) / best_n + unit - 1) / unit * unit;
  pl->tps = (int)tps;
  pl->n_splits = (int)((tiles_max + tps - 1) / tps);
  pl->bpg = bpg;
  pl->n_bgroups = (B + bpg - 1) / bpg;
  pl->cgroups = cgroups;
  pl->tickets_off = kWsHeader;
  pl->partials_off = decode_ticket_region_bytes(B, a->Hkv * cgroups);
  pl->ws_bytes = pl->partials_off +
                 sizeof(float) * (size_t)B * a->Hkv * pl->n_splits * g * a->M * kPartialStride;
  return VQKV_OK;
}

vqkv_status validate_encode(const vqkv_encode_args* a) {
  if (a == nullptr) return VQKV_ERR_INVALID_ARG;
  if (!is_code_mode(a->mode)) return VQKV_ERR_UNSUPPORTED;
  if (a->role != VQKV_ROLE_K && a->role != VQKV_ROLE_V) return VQKV_ERR_INVALID_ARG;
  if (a->head_dim != 128) return VQKV_ERR_UNSUPPORTED;
  if (a->B < 0 || a->Hkv < 1 || a->n_rows < 0 || a->cap_len < 1) return VQKV_ERR_INVALID_ARG;
  if (a->B == 0 || a->n_rows == 0) return VQKV_OK;
  if (!a->x || !a->pos || !a->codebook || !a->codes) return VQKV_ERR_INVALID_ARG;
  if (a->role == VQKV_ROLE_K && !a->s) return VQKV_ERR_INVALID_ARG;
  if (!aligned(a->x, 8) || !aligned(a->codebook, 16) || !aligned(a->pos, 4) ||
      (a->role == VQKV_ROLE_K && !aligned(a->s, 16)) || (a->near_tie_count && !aligned(a->near_tie_count, 8)) ||
      (a->error_flags && !aligned(a->error_flags, 4)))
    return VQKV_ERR_INVALID_ARG;
  if ((long long)a->B * a->n_rows > 0x7fffffffLL) return VQKV_ERR_INVALID_ARG;
  return VQKV_OK;
}

PlanInput plan_input(const vqkv_decode_args* a) {
  return PlanInput{a->mode, a->B, a->Hq, a->Hkv, a->max_seq_len, a->num_splits};
}

// The fields of a decode over packed codes that do not depend on its plan.
DecodeParams packed_params(const vqkv_decode_args* a, int M, const vqkv_paging* pg) {
  DecodeParams p{};
  p.q = reinterpret_cast<const __half*>(a->q);
  p.kc = a->k_codes;
  p.vc = a->v_codes;
  p.seq_lens = a->seq_lens;
  p.kcb = reinterpret_cast<const __half*>(a->k_codebook);
  p.vcb = reinterpret_cast<const __half*>(a->v_codebook);
  p.s = a->s;
  p.out = reinterpret_cast<__half*>(a->out);
  p.err = static_cast<unsigned*>(a->workspace);
  p.stream_bytes = (long long)vqkv_code_bytes(a->mode, a->cap_len);
  p.B = a->B;
  p.Hq = a->Hq;
  p.Hkv = a->Hkv;
  p.g = a->Hq / a->Hkv;
  p.M = M;
  p.ncols = M * p.g;
  p.max_seq_len = a->max_seq_len;
  const float scale = a->softmax_scale > 0.f ? a->softmax_scale : 1.0f / std::sqrt(128.0f);
  p.qscale = scale * 1.4426950408889634f / std::sqrt(128.0f);
  set_paging(p, pg, a->mode);
  return p;
}

// Sequences b0 .. b0 + kFlatMaxB - 1 (at most) of a call's B.
DecodeParams batch_part(const DecodeParams& p, int b0, int B) {
  DecodeParams c = p;
  c.B = std::min(B - b0, kFlatMaxB);
  const size_t rows = (size_t)b0 * p.M * p.Hq * 128;
  c.q = p.q + rows;
  c.out = p.out + rows;
  c.seq_lens = p.seq_lens + b0;
  if (p.row_start != nullptr) {   // packed rows: the starts say where
    c.q = p.q, c.out = p.out;
    c.row_start = p.row_start + b0;
  }
  if (p.mass != nullptr) c.mass = p.mass + (size_t)b0 * p.Hkv * p.cap_len;
  if (p.block_table != nullptr) {
    c.block_table = p.block_table + (size_t)b0 * p.max_blocks;
  } else {
    c.kc = p.kc + (size_t)b0 * p.Hkv * p.stream_bytes;
    c.vc = p.vc + (size_t)b0 * p.Hkv * p.stream_bytes;
  }
  return c;
}

// Draft-tree attention: one CTA per SM (its shared memory), all of them in one
// wave over (share, KV head, column group); a share is an equal part of all
// sequences' tiles, cut on the device.  Batches beyond the flat plan's limit
// run as several launches of up to kFlatMaxB sequences.
struct TreePlan {
  int n_splits = 1, cgroups = 1;
  bool pairs = false;   // scores of q' in two fp16 parts
  size_t query_off = 0, partials_off = 0, ws_bytes = 0;   // transformed queries, partials
};
// Column groups of the decode calls, at most (64 columns in groups of 8).  The tree's
// scratch begins behind the tickets of all of them, so that a serving loop's draft
// and plain decode steps can share a workspace: it leaves the tickets zero.
constexpr int kTicketGroups = 8;

vqkv_status validate_tree_sizes(const vqkv_decode_tree_args* at) {
  if (at == nullptr) return VQKV_ERR_INVALID_ARG;
  const vqkv_status st = validate_decode_sizes(&at->decode);
  if (st != VQKV_OK) return st;
  if (at->n_queries < 1) return VQKV_ERR_INVALID_ARG;
  if (at->n_queries > 64) return VQKV_ERR_UNSUPPORTED;   // one mask word per query
  if (at->decode.Hkv > kMaxGridYZ || at->decode.cap_len > kMaxTokens ||
      (long long)std::min(at->decode.B, kFlatMaxB) * ((at->decode.max_seq_len + 63) / 64) > kMaxTokens)
    return VQKV_ERR_UNSUPPORTED;
  return VQKV_OK;
}

// weights: the plan of the attention weights, whose scores always take both parts
// of q'.  A draft tree of up to 64 columns takes them while a share has two tiles at
// most: such a call is bound by the host (15 us), and the parts cost 0.2 to 0.4 us of
// 11 to 13 on the GPU (519 tokens, 32 columns: 10.7 and 11.0; 2,000 tokens, 64
// columns: 13.3 and 13.7).  Long ones would pay for them in every tile (196,608
// tokens, 64 columns: 96 and 126 us; 8 sequences of 500: 23 and 25).
vqkv_status plan_tree(const vqkv_decode_tree_args* at, bool weights, TreePlan* pl) {
  const vqkv_decode_args* a = &at->decode;
  DeviceInfo di;
  const vqkv_status st = device_info(kTreeKernels, a->mode, &di);
  if (st != VQKV_OK) return st;
  const int cols = at->n_queries * (a->Hq / a->Hkv);
  pl->cgroups = (cols + decode_tree_cols(cols) - 1) / decode_tree_cols(cols);
  const int B = std::max(std::min(a->B, kFlatMaxB), 1);
  // a share has at least one tile when the sequences are full
  const long long tiles = std::max<long long>(1, (long long)B * ((a->max_seq_len + 63) / 64));
  const long long want = a->num_splits > 0 ? std::min(a->num_splits, 1024) : di.sms / ((long long)a->Hkv * pl->cgroups);
  pl->n_splits = (int)std::max<long long>(1, std::min(want, tiles));
  pl->pairs = weights || (cols <= 64 && tiles <= 2 * pl->n_splits);
  pl->query_off = decode_ticket_region_bytes(a->B, a->Hkv * kTicketGroups);   // Hkv <= kMaxGridYZ
  pl->partials_off = pl->query_off + round_up(decode_tree_query_bytes(B, a->Hkv, cols, pl->pairs), 256);
  pl->ws_bytes = pl->partials_off;
  if (pl->n_splits > 1)
    pl->ws_bytes += sizeof(float) * (size_t)a->Hkv * (pl->n_splits + B - 1) * cols * kPartialStride;
  return VQKV_OK;
}

// Decode with attention weights.  Few columns: the decode's plan at 4 columns
// per CTA, then the columns' statistics and the scores behind its workspace.
// Many: the draft-tree attention, then statistics and query images of the
// key-only pass.  A group of 4 columns costs one decode, the other path about
// the same for any number: at 196,608 tokens and 8 KV heads 12 / 16 columns take
// 127 / 169 us at 2 bit, 151 / 200 at 4, 190 / 252 at 1.25 and 261, 240 (12 columns)
// at 3 and 1.5 on the first path; 181, 257, 213, 260 and 250 on the second.  At
// 1.25 bit 16 columns cross where the work does: 37 and 39 us at 16,384 tokens, 63
// and 55 at 32,768, 28 and 36 for 8 sequences of 1,000, 94 and 66 for 32.  Short
// sequences favour the first path further: 16 columns of 4,096 tokens 14 and 26 us
// at 2 bit.
int mass_few_cols(const vqkv_decode_args& a) {
  if (a.mode == VQKV_MODE_VQ3 || a.mode == VQKV_MODE_VQ15) return 12;
  const bool much = (long long)a.B * a.Hkv * a.max_seq_len > 196608;
  return a.mode == VQKV_MODE_VQ125 && much ? 12 : 16;
}

struct MassPlan {
  bool tiles = false;
  DecodePlan d;
  TreePlan t;
  size_t stats_off = 0, scores_off = 0, image_off = 0, ws_bytes = 0;
  int score_row = 0;
};

vqkv_status validate_mass_sizes(const vqkv_decode_mass_args* am) {
  if (am == nullptr) return VQKV_ERR_INVALID_ARG;
  const vqkv_status st = validate_decode_sizes(&am->decode);
  if (st != VQKV_OK) return st;
  const vqkv_decode_args& a = am->decode;
  if (am->n_queries < 1) return VQKV_ERR_INVALID_ARG;
  if (am->n_queries > 64 || am->n_queries * (a.Hq / a.Hkv) > 64) return VQKV_ERR_UNSUPPORTED;
  const int cols = am->n_queries * (a.Hq / a.Hkv);
  if (a.Hkv > kMaxGridYZ || a.cap_len > kMaxTokens) return VQKV_ERR_UNSUPPORTED;
  if (cols <= mass_few_cols(a) && (long long)a.B * ((cols + 3) / 4) > kMaxGridYZ) return VQKV_ERR_UNSUPPORTED;
  if (cols > mass_few_cols(a) && (long long)std::min(a.B, kFlatMaxB) * ((a.max_seq_len + 63) / 64) > kMaxTokens)
    return VQKV_ERR_UNSUPPORTED;
  return VQKV_OK;
}

vqkv_status plan_mass(const vqkv_decode_mass_args* am, MassPlan* pl) {
  const vqkv_decode_args& a = am->decode;
  const int ncols = am->n_queries * (a.Hq / a.Hkv);
  const bool tiles = ncols > mass_few_cols(a);
  DeviceInfo di;
  const vqkv_status ready = device_info(tiles ? kMassTileKernels : kMassKernels, a.mode, &di);
  if (ready != VQKV_OK) return ready;
  if (tiles) {
    pl->tiles = true;
    vqkv_decode_tree_args at{};
    at.decode = a;
    at.n_queries = am->n_queries;
    const vqkv_status st = plan_tree(&at, true, &pl->t);
    if (st != VQKV_OK) return st;
    const int B = std::max(std::min(a.B, kFlatMaxB), 1);
    pl->stats_off = round_up(pl->t.ws_bytes, 256);
    pl->image_off = round_up(pl->stats_off + (size_t)B * a.Hkv * ncols * sizeof(float2), 256);
    pl->ws_bytes = pl->image_off + mass_tiles_image_bytes(B, a.Hkv, ncols);
    return VQKV_OK;
  }
  PlanInput in = plan_input(&a);
  in.M = am->n_queries;
  in.width = 4;
  const vqkv_status st = plan_decode(&in, &pl->d);
  if (st != VQKV_OK) return st;
  const size_t pairs = (size_t)std::max(a.B, 1) * a.Hkv;
  const size_t cols = (size_t)am->n_queries * (a.Hq / a.Hkv);
  // rows to the end of the last step: whole 16-token tiles, up to three of them
  pl->score_row = (a.max_seq_len + 15) / 16 * 16 + 48;
  pl->stats_off = round_up(pl->d.ws_bytes, 256);
  pl->scores_off = round_up(pl->stats_off + pairs * cols * sizeof(float2), 256);
  pl->ws_bytes = pl->scores_off + pairs * pl->d.cgroups * pl->score_row * 4 * sizeof(float);
  return VQKV_OK;
}

// What a timeout test changes in the tile kernels: each wait's polls (0: no
// test), and the ring stage that lacks an arrival in one of the two kernels.
struct TestWaits {
  unsigned polls = 0;
  int stage = -1, key_stage = -1;
  bool set(uint32_t max_polls, bool key_pass, int st) {   // every ring has two stages at least
    if (max_polls < 1 || max_polls > 4096 || st < 0 || st > 1) return false;
    polls = max_polls;
    (key_pass ? key_stage : stage) = st;
    return true;
  }
};

vqkv_status validate_fp16(const vqkv_fp16_decode_args* a, bool sizes_only) {
  if (a == nullptr) return VQKV_ERR_INVALID_ARG;
  if (a->head_dim != 128) return VQKV_ERR_UNSUPPORTED;
  if (a->B < 0 || a->Hq < 1 || a->Hkv < 1 || a->cap_len < 1) return VQKV_ERR_INVALID_ARG;
  if (a->Hq % a->Hkv != 0) return VQKV_ERR_INVALID_ARG;
  if (a->Hq / a->Hkv > 8) return VQKV_ERR_UNSUPPORTED;
  if (a->max_seq_len < 0 || a->max_seq_len > a->cap_len) return VQKV_ERR_INVALID_ARG;
  if (a->num_splits < 0 || !std::isfinite(a->softmax_scale)) return VQKV_ERR_INVALID_ARG;
  if (sizes_only || a->B == 0) return VQKV_OK;
  if (!a->q || !a->k || !a->v || !a->seq_lens || !a->out) return VQKV_ERR_INVALID_ARG;
  if (!aligned(a->q, 4) || !aligned(a->k, 16) || !aligned(a->v, 16) || !aligned(a->seq_lens, 4) ||
      !aligned(a->out, 2))
    return VQKV_ERR_INVALID_ARG;
  return VQKV_OK;
}

PlanInput plan_input(const vqkv_fp16_decode_args* a) {
  return PlanInput{kModeFp16, a->B, a->Hq, a->Hkv, a->max_seq_len, a->num_splits};
}

}  // namespace

vqkv_status decode_validate(const vqkv_decode_args* a) { return validate_decode(a); }

namespace {
// Both decode entry points: ap == nullptr for vqkv_decode_attn.
vqkv_status decode_launch(const vqkv_decode_args* a, const vqkv_decode_append_args* ap, int M, void* stream,
                          const vqkv_paging* pg = nullptr, unsigned test_polls = 0);
vqkv_status encode_launch(const vqkv_encode_args* a, void* stream, const vqkv_paging* pg = nullptr);
}  // namespace

size_t decode_ticket_region_bytes(int B, int Hkv) {
  return round_up(kWsHeader + sizeof(unsigned) * (size_t)std::max(B, 1) * Hkv, 256);
}

}  // namespace vqkv

using namespace vqkv;

extern "C" {

size_t vqkv_code_bytes(int32_t mode, int32_t cap_len) {
  if (cap_len < 0) return 0;
  if (mode == VQKV_MODE_VQ2) return (size_t)((cap_len + 15) / 16) * 512;
  if (mode == VQKV_MODE_VQ15) return (size_t)((cap_len + 63) / 64) * 1536;
  if (mode == VQKV_MODE_VQ4) return (size_t)((cap_len + 15) / 16) * 1024;
  if (mode == VQKV_MODE_VQ3) return (size_t)((cap_len + 15) / 16) * 768;
  if (mode == VQKV_MODE_VQ125) return (size_t)((cap_len + 15) / 16) * 320;
  return 0;
}

size_t vqkv_decode_workspace_bytes(const vqkv_decode_args* a) {
  if (validate_decode_sizes(a) != VQKV_OK) return 0;
  DecodePlan pl;
  const PlanInput in = plan_input(a);
  if (plan_decode(&in, &pl) != VQKV_OK) return 0;
  return pl.ws_bytes;
}

int32_t vqkv_decode_num_splits(const vqkv_decode_args* a) {
  if (validate_decode_sizes(a) != VQKV_OK) return -1;
  DecodePlan pl;
  const PlanInput in = plan_input(a);
  if (plan_decode(&in, &pl) != VQKV_OK) return -1;
  return pl.n_splits;
}

int32_t vqkv_decode_kernel_count(const vqkv_decode_args* a) {
  if (validate_decode_sizes(a) != VQKV_OK) return -1;
  if (a->B == 0) return 0;
  DecodePlan pl;
  const PlanInput in = plan_input(a);
  if (plan_decode(&in, &pl) != VQKV_OK) return -1;
  return (pl.bpg > 1 && pl.n_splits > 1) ? 2 : 1;
}

vqkv_status vqkv_decode_attn(const vqkv_decode_args* a, void* stream) { return decode_launch(a, nullptr, 1, stream); }

vqkv_status vqkv_decode_attn_multi(const vqkv_decode_multi_args* am, void* stream) {
  if (am == nullptr || am->n_queries < 1) return VQKV_ERR_INVALID_ARG;
  return decode_launch(&am->decode, nullptr, am->n_queries, stream);
}

vqkv_status vqkv_decode_append(const vqkv_decode_append_args* ap, void* stream) {
  if (ap == nullptr) return VQKV_ERR_INVALID_ARG;
  return decode_launch(&ap->decode, ap, 1, stream);
}

}  // extern "C"

namespace vqkv {
namespace {

vqkv_status decode_launch(const vqkv_decode_args* a, const vqkv_decode_append_args* ap, int M, void* stream,
                          const vqkv_paging* pg, unsigned test_polls) {
  if (ap != nullptr && a->mode != VQKV_MODE_VQ2 && a->mode != VQKV_MODE_VQ4) return VQKV_ERR_UNSUPPORTED;
  vqkv_status st = validate_decode(a);
  if (st != VQKV_OK) return st;
  if (pg != nullptr) {
    st = validate_paging(pg, a->mode, a->cap_len);
    if (st != VQKV_OK) return st;
    if (a->B > 0 && (!pg->block_table || !aligned(pg->block_table, 4))) return VQKV_ERR_INVALID_ARG;
  }
  if (M > 64 || (long long)M * (a->Hq / a->Hkv) > 64) return VQKV_ERR_UNSUPPORTED;   // <= 8 column groups
  if (ap != nullptr) {
    if (a->B > 0 && (!ap->k_new || !ap->v_new || !aligned(ap->k_new, 8) || !aligned(ap->v_new, 8) ||
                     (ap->near_tie_count && !aligned(ap->near_tie_count, 8))))
      return VQKV_ERR_INVALID_ARG;
  }
  if (a->B == 0) return VQKV_OK;
  DecodePlan pl;
  PlanInput in = plan_input(a);
  in.M = M;
  // the fused append costs its CTA about 60 tiles of streaming (2-bit, one
  // CTA per SM); a split of at most the plain plan's size, so the workspace
  // of vqkv_decode_workspace_bytes still covers it
  if (ap != nullptr) in.credit_tiles = 60;
  st = plan_decode(&in, &pl);
  if (st != VQKV_OK) return st;
  if (a->workspace == nullptr || a->workspace_bytes < pl.ws_bytes) return VQKV_ERR_WORKSPACE;
  if (!aligned(a->workspace, 256)) return VQKV_ERR_INVALID_ARG;
  DecodeParams p;
  unsigned char* ws = static_cast<unsigned char*>(a->workspace);
  p.q = reinterpret_cast<const __half*>(a->q);
  p.kc = a->k_codes;
  p.vc = a->v_codes;
  p.seq_lens = a->seq_lens;
  p.kcb = reinterpret_cast<const __half*>(a->k_codebook);
  p.vcb = reinterpret_cast<const __half*>(a->v_codebook);
  p.s = a->s;
  p.out = reinterpret_cast<__half*>(a->out);
  p.err = reinterpret_cast<unsigned*>(ws);
  p.tickets = reinterpret_cast<unsigned*>(ws + pl.tickets_off);
  p.partials = reinterpret_cast<float*>(ws + pl.partials_off);
  p.stream_bytes = (long long)vqkv_code_bytes(a->mode, a->cap_len);
  p.B = a->B;
  p.Hq = a->Hq;
  p.Hkv = a->Hkv;
  p.g = a->Hq / a->Hkv;
  p.M = M;
  p.ncols = M * p.g;
  p.max_seq_len = a->max_seq_len;
  p.n_splits = pl.n_splits;
  p.tps = pl.tps;
  p.bpg = pl.bpg;
  p.defer_merge = pl.bpg > 1 ? 1 : 0;
  p.flat = pl.flat;
  const float scale = a->softmax_scale > 0.f ? a->softmax_scale : 1.0f / std::sqrt(128.0f);
  p.qscale = scale * 1.4426950408889634f / std::sqrt(128.0f);
  if (ap != nullptr) {
    p.k_new = reinterpret_cast<const __half*>(ap->k_new);
    p.v_new = reinterpret_cast<const __half*>(ap->v_new);
    p.kc_w = const_cast<uint8_t*>(a->k_codes);
    p.vc_w = const_cast<uint8_t*>(a->v_codes);
    p.near_tie = ap->near_tie_count;
  }
  set_paging(p, pg, a->mode);
  if (test_polls > 0) {
    p.max_polls = test_polls;
    p.withhold_first_copy = 1;
  }
  p.cgroups = pl.cgroups;
  const dim3 grid(pl.n_splits, a->Hkv, pl.n_bgroups * pl.cgroups);
  if (launch_decode(a->mode, p, grid, static_cast<cudaStream_t>(stream)) != cudaSuccess) return VQKV_ERR_CUDA;
  if (p.defer_merge && p.n_splits > 1 && launch_combine(p, static_cast<cudaStream_t>(stream)) != cudaSuccess)
    return VQKV_ERR_CUDA;
  return VQKV_OK;
}

}  // namespace
}  // namespace vqkv

extern "C" {

vqkv_status vqkv_encode(const vqkv_encode_args* a, void* stream) { return encode_launch(a, stream); }

vqkv_status vqkv_encode_paged(const vqkv_encode_args* a, const vqkv_paging* pg, void* stream) {
  if (pg == nullptr) return VQKV_ERR_INVALID_ARG;
  return encode_launch(a, stream, pg);
}

vqkv_status vqkv_test_decode_ring_timeout(const vqkv_decode_args* a, uint32_t max_polls, void* stream) {
  if (a == nullptr || a->mode != VQKV_MODE_VQ2) return a == nullptr ? VQKV_ERR_INVALID_ARG : VQKV_ERR_UNSUPPORTED;
  if (max_polls < 1 || max_polls > 4096) return VQKV_ERR_INVALID_ARG;
  return decode_launch(a, nullptr, 1, stream, nullptr, max_polls);
}

vqkv_status vqkv_decode_attn_paged(const vqkv_decode_args* a, const vqkv_paging* pg, void* stream) {
  if (pg == nullptr) return VQKV_ERR_INVALID_ARG;
  return decode_launch(a, nullptr, 1, stream, pg);
}

}  // extern "C"

namespace vqkv {
namespace {

vqkv_status encode_launch(const vqkv_encode_args* a, void* stream, const vqkv_paging* pg) {
  vqkv_status st = validate_encode(a);
  if (st != VQKV_OK) return st;
  if (pg != nullptr) {
    st = validate_paging(pg, a->mode, a->cap_len);
    if (st != VQKV_OK) return st;
    if (a->B > 0 && a->n_rows > 0 && (!pg->block_table || !aligned(pg->block_table, 4))) return VQKV_ERR_INVALID_ARG;
  }
  if (a->B == 0 || a->n_rows == 0) return st;
  DeviceInfo di;
  st = device_info(&di);
  if (st != VQKV_OK) return st;
  EncodeParams p;
  p.x = reinterpret_cast<const __half*>(a->x);
  p.pos = a->pos;
  p.s = a->s;
  p.cb = reinterpret_cast<const __half*>(a->codebook);
  p.codes = a->codes;
  p.near_tie = a->near_tie_count;
  p.err = a->error_flags;
  p.stream_bytes = (long long)vqkv_code_bytes(a->mode, a->cap_len);
  p.B = a->B;
  p.Hkv = a->Hkv;
  p.n_rows = a->n_rows;
  p.cap_len = a->cap_len;
  p.role = a->role;
  const long long rows = (long long)a->B * a->n_rows;   // per KV head
  // Few rows (a decode-step append): one row per CTA, its candidates split
  // over the CTA's warps, for latency.
  const bool split_rows = rows * a->Hkv <= di.sms;
  int blocks_x;
  if (split_rows) {
    blocks_x = (int)rows;
  } else {
    const vqkv_status ready = device_info(kEncodeTileKernels, a->mode, &di);
    if (ready != VQKV_OK) return ready;
    // Persistent tensor-memory CTAs over tiles of 8, 4 or 2 rows, one per SM, in one wave
    // (a few CTAs more would run after the others: 1,000 key rows of 5 heads at 4 bit
    // 33 us with 31 CTAs a head, 21 with 30).
    const long long tiles = (rows + encode_tile_rows(a->mode) - 1) / encode_tile_rows(a->mode);
    blocks_x = (int)std::min<long long>(tiles, std::max(1, di.sms / a->Hkv));
  }
  set_paging(p, pg, a->mode);
  if (launch_encode(a->mode, p, blocks_x, split_rows, static_cast<cudaStream_t>(stream)) != cudaSuccess)
    return VQKV_ERR_CUDA;
  return VQKV_OK;
}

}  // namespace
}  // namespace vqkv

extern "C" {

size_t vqkv_fp16_decode_workspace_bytes(const vqkv_fp16_decode_args* a) {
  if (validate_fp16(a, true) != VQKV_OK) return 0;
  DecodePlan pl;
  const PlanInput in = plan_input(a);
  if (plan_decode(&in, &pl) != VQKV_OK) return 0;
  return pl.ws_bytes;
}

vqkv_status vqkv_decode_attn_fp16(const vqkv_fp16_decode_args* a, void* stream) {
  vqkv_status st = validate_fp16(a, false);
  if (st != VQKV_OK || a->B == 0) return st;
  DecodePlan pl;
  const PlanInput in = plan_input(a);
  st = plan_decode(&in, &pl);
  if (st != VQKV_OK) return st;
  if (a->workspace == nullptr || a->workspace_bytes < pl.ws_bytes) return VQKV_ERR_WORKSPACE;
  if (!aligned(a->workspace, 256)) return VQKV_ERR_INVALID_ARG;
  unsigned char* ws = static_cast<unsigned char*>(a->workspace);
  DecodeParams p{};
  p.q = reinterpret_cast<const __half*>(a->q);
  p.kc = reinterpret_cast<const uint8_t*>(a->k);
  p.vc = reinterpret_cast<const uint8_t*>(a->v);
  p.seq_lens = a->seq_lens;
  p.out = reinterpret_cast<__half*>(a->out);
  p.err = reinterpret_cast<unsigned*>(ws);
  p.tickets = reinterpret_cast<unsigned*>(ws + pl.tickets_off);
  p.partials = reinterpret_cast<float*>(ws + pl.partials_off);
  p.stream_bytes = (long long)a->cap_len * 256;
  p.B = a->B;
  p.Hq = a->Hq;
  p.Hkv = a->Hkv;
  p.g = a->Hq / a->Hkv;
  p.M = 1;
  p.ncols = p.g;
  p.max_seq_len = a->max_seq_len;
  p.n_splits = pl.n_splits;
  p.tps = pl.tps;
  p.bpg = pl.bpg;
  p.defer_merge = pl.bpg > 1 ? 1 : 0;
  const float scale = a->softmax_scale > 0.f ? a->softmax_scale : 1.0f / std::sqrt(128.0f);
  p.qscale = scale * 1.4426950408889634f;
  const dim3 grid(pl.n_splits, a->Hkv, pl.n_bgroups);
  if (launch_decode_fp16(p, grid, static_cast<cudaStream_t>(stream)) != cudaSuccess) return VQKV_ERR_CUDA;
  if (p.defer_merge && p.n_splits > 1 && launch_combine(p, static_cast<cudaStream_t>(stream)) != cudaSuccess)
    return VQKV_ERR_CUDA;
  return VQKV_OK;
}

size_t vqkv_decode_mass_workspace_bytes(const vqkv_decode_mass_args* a) {
  MassPlan pl;
  if (validate_mass_sizes(a) != VQKV_OK || plan_mass(a, &pl) != VQKV_OK) return 0;
  return pl.ws_bytes;
}

}  // extern "C"

namespace vqkv {
namespace {

vqkv_status mass_launch(const vqkv_decode_mass_args* am, const vqkv_paging* pg, void* stream,
                        const TestWaits& test = TestWaits()) {
  vqkv_status st = validate_mass_sizes(am);
  if (st != VQKV_OK) return st;
  const vqkv_decode_args* a = &am->decode;
  st = validate_decode(a);
  if (st != VQKV_OK) return st;
  if (pg != nullptr) {
    st = validate_paging(pg, a->mode, a->cap_len);
    if (st != VQKV_OK) return st;
    if (a->B > 0 && (!pg->block_table || !aligned(pg->block_table, 4))) return VQKV_ERR_INVALID_ARG;
  }
  if (a->B == 0) return VQKV_OK;
  if (!am->mass || !aligned(am->mass, 4)) return VQKV_ERR_INVALID_ARG;
  MassPlan pl;
  st = plan_mass(am, &pl);
  if (st != VQKV_OK) return st;
  if (a->workspace == nullptr || a->workspace_bytes < pl.ws_bytes) return VQKV_ERR_WORKSPACE;
  if (!aligned(a->workspace, 256)) return VQKV_ERR_INVALID_ARG;
  unsigned char* ws = static_cast<unsigned char*>(a->workspace);
  DecodeParams p = packed_params(a, am->n_queries, pg);
  p.mass = am->mass;
  p.cap_len = a->cap_len;
  p.stats = reinterpret_cast<float2*>(ws + pl.stats_off);
  if (test.polls > 0 && !pl.tiles && (a->mode != VQKV_MODE_VQ2 || test.key_stage >= 0)) return VQKV_ERR_UNSUPPORTED;
  if (pl.tiles) {
    p.max_polls = test.polls > 0 ? test.polls : kTilePolls;
    p.withhold_stage = test.stage;
    p.withhold_key_stage = test.key_stage;
    p.partials = reinterpret_cast<float*>(ws + pl.t.partials_off);
    p.cgroups = pl.t.cgroups;
    p.n_splits = pl.t.n_splits;
    for (int b0 = 0; b0 < a->B; b0 += kFlatMaxB) {
      const DecodeParams c = batch_part(p, b0, a->B);
      cudaStream_t s = static_cast<cudaStream_t>(stream);
      if (launch_mass_queries(c, ws + pl.image_off, s) != cudaSuccess ||
          launch_decode_tree(a->mode, c, nullptr, true, ws + pl.t.query_off, s) != cudaSuccess ||
          launch_mass_tiles(a->mode, c, ws + pl.image_off, s) != cudaSuccess)
        return VQKV_ERR_CUDA;
    }
    return VQKV_OK;
  }
  p.tickets = reinterpret_cast<unsigned*>(ws + pl.d.tickets_off);
  p.partials = reinterpret_cast<float*>(ws + pl.d.partials_off);
  if (test.polls > 0) {   // the ring's hook
    p.max_polls = test.polls;
    p.withhold_first_copy = 1;
  }
  p.scores = reinterpret_cast<float*>(ws + pl.scores_off);
  p.score_row = pl.score_row;
  p.n_splits = pl.d.n_splits;
  p.tps = pl.d.tps;
  p.bpg = pl.d.bpg;
  p.defer_merge = pl.d.bpg > 1 ? 1 : 0;
  p.flat = pl.d.flat;
  p.cgroups = pl.d.cgroups;
  const dim3 grid(pl.d.n_splits, a->Hkv, pl.d.n_bgroups * pl.d.cgroups);
  return launch_decode_mass(a->mode, p, grid, static_cast<cudaStream_t>(stream)) == cudaSuccess ? VQKV_OK : VQKV_ERR_CUDA;
}

}  // namespace
}  // namespace vqkv

extern "C" {

vqkv_status vqkv_decode_attn_mass(const vqkv_decode_mass_args* am, const vqkv_paging* pg, void* stream) {
  return mass_launch(am, pg, stream);
}

vqkv_status vqkv_test_decode_mass_timeout(const vqkv_decode_mass_args* am, int32_t key_pass, int32_t stage, uint32_t max_polls,
                                          void* stream) {
  TestWaits test;
  if (!test.set(max_polls, key_pass != 0, stage)) return VQKV_ERR_INVALID_ARG;
  return mass_launch(am, nullptr, stream, test);
}

size_t vqkv_decode_tree_workspace_bytes(const vqkv_decode_tree_args* a) {
  TreePlan pl;
  if (validate_tree_sizes(a) != VQKV_OK || plan_tree(a, false, &pl) != VQKV_OK) return 0;
  return pl.ws_bytes;
}

}  // extern "C"

namespace vqkv {
namespace {

vqkv_status tree_launch(const vqkv_decode_tree_args* at, const vqkv_paging* pg, void* stream,
                        const TestWaits& test = TestWaits()) {
  vqkv_status st = validate_tree_sizes(at);
  if (st != VQKV_OK) return st;
  const vqkv_decode_args* a = &at->decode;
  st = validate_decode(a);
  if (st != VQKV_OK) return st;
  if (pg != nullptr) {
    st = validate_paging(pg, a->mode, a->cap_len);
    if (st != VQKV_OK) return st;
    if (a->B > 0 && (!pg->block_table || !aligned(pg->block_table, 4))) return VQKV_ERR_INVALID_ARG;
  }
  if (a->B == 0) return VQKV_OK;
  if (!at->tree_mask || !aligned(at->tree_mask, 8)) return VQKV_ERR_INVALID_ARG;
  TreePlan pl;
  st = plan_tree(at, false, &pl);
  if (st != VQKV_OK) return st;
  if (a->workspace == nullptr || a->workspace_bytes < pl.ws_bytes) return VQKV_ERR_WORKSPACE;
  if (!aligned(a->workspace, 256)) return VQKV_ERR_INVALID_ARG;
  unsigned char* ws = static_cast<unsigned char*>(a->workspace);
  DecodeParams p = packed_params(a, at->n_queries, pg);
  p.partials = reinterpret_cast<float*>(ws + pl.partials_off);
  p.cgroups = pl.cgroups;
  p.n_splits = pl.n_splits;
  p.max_polls = test.polls > 0 ? test.polls : kTilePolls;
  p.withhold_stage = test.stage;
  const unsigned long long* mask = reinterpret_cast<const unsigned long long*>(at->tree_mask);
  for (int b0 = 0; b0 < a->B; b0 += kFlatMaxB) {
    const DecodeParams c = batch_part(p, b0, a->B);
    if (launch_decode_tree(a->mode, c, mask + (size_t)b0 * p.M, pl.pairs, ws + pl.query_off, static_cast<cudaStream_t>(stream)) !=
        cudaSuccess)
      return VQKV_ERR_CUDA;
  }
  return VQKV_OK;
}

}  // namespace
}  // namespace vqkv

extern "C" {

vqkv_status vqkv_decode_attn_tree(const vqkv_decode_tree_args* at, const vqkv_paging* pg, void* stream) {
  return tree_launch(at, pg, stream);
}

vqkv_status vqkv_test_decode_tree_timeout(const vqkv_decode_tree_args* at, int32_t stage, uint32_t max_polls, void* stream) {
  TestWaits test;
  if (!test.set(max_polls, false, stage)) return VQKV_ERR_INVALID_ARG;
  return tree_launch(at, nullptr, stream, test);
}

vqkv_status vqkv_evict_select(const vqkv_evict_select_args* a, void* stream) {
  if (a == nullptr) return VQKV_ERR_INVALID_ARG;
  if (a->B < 0 || a->Hkv < 1 || a->cap_len < 1 || a->max_seq_len < 0 || a->max_seq_len > a->cap_len || a->n_keep < 1 ||
      a->n_sink < 0 || a->n_recent < 0 || (long long)a->n_sink + a->n_recent > a->n_keep)
    return VQKV_ERR_INVALID_ARG;
  if (a->B > kMaxGridYZ || a->Hkv > kMaxGridYZ || a->cap_len > kMaxTokens) return VQKV_ERR_UNSUPPORTED;
  if (a->B == 0) return VQKV_OK;
  if (!a->mass || !a->seq_lens || !a->keep || !a->keep_lens) return VQKV_ERR_INVALID_ARG;
  if (!aligned(a->mass, 4) || !aligned(a->seq_lens, 4) || !aligned(a->keep, 4) || !aligned(a->keep_lens, 4) ||
      !aligned(a->error_flags, 4))
    return VQKV_ERR_INVALID_ARG;
  // the lengths are read by every CTA of a sequence, the kept ones written by the first
  if (overlap(a->keep_lens, 4 * (size_t)a->B, a->seq_lens, 4 * (size_t)a->B)) return VQKV_ERR_INVALID_ARG;
  DeviceInfo di;
  const vqkv_status st = device_info(kSelectKernels, 0, &di);
  if (st != VQKV_OK) return st;
  SelectParams p;
  p.mass = a->mass;
  p.seq_lens = a->seq_lens;
  p.keep = a->keep;
  p.keep_lens = a->keep_lens;
  p.err = a->error_flags;
  p.B = a->B;
  p.Hkv = a->Hkv;
  p.cap_len = a->cap_len;
  p.max_seq_len = a->max_seq_len;
  p.n_keep = a->n_keep;
  p.n_sink = a->n_sink;
  p.n_recent = a->n_recent;
  return launch_evict_select(p, di.sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? VQKV_OK : VQKV_ERR_CUDA;
}

vqkv_status vqkv_cache_compact(const vqkv_cache_compact_args* a, const vqkv_paging* pg, void* stream) {
  if (a == nullptr) return VQKV_ERR_INVALID_ARG;
  if (!is_code_mode(a->mode)) return VQKV_ERR_UNSUPPORTED;
  if (a->B < 0 || a->Hkv < 1 || a->cap_len < 1 || a->n_src < 0) return VQKV_ERR_INVALID_ARG;
  if (a->src_heads != 1 && a->src_heads != a->Hkv) return VQKV_ERR_INVALID_ARG;
  if (a->B > kMaxGridYZ || 3LL * a->Hkv > kMaxGridYZ || a->cap_len > kMaxTokens) return VQKV_ERR_UNSUPPORTED;
  if (pg != nullptr) {
    const vqkv_status st = validate_paging(pg, a->mode, a->cap_len);
    if (st != VQKV_OK) return st;
    if (a->B > 0 && (!pg->block_table || !aligned(pg->block_table, 4))) return VQKV_ERR_INVALID_ARG;
  }
  if (a->B == 0) return VQKV_OK;
  if (!a->k_codes || !a->v_codes || !a->seq_lens || !a->counts || (!a->src && a->n_src > 0)) return VQKV_ERR_INVALID_ARG;
  if (!aligned(a->k_codes, 16) || !aligned(a->v_codes, 16) || !aligned(a->seq_lens, 4) || !aligned(a->src, 4) ||
      !aligned(a->counts, 4) || !aligned(a->start, 4) || !aligned(a->mass, 4) || !aligned(a->error_flags, 4))
    return VQKV_ERR_INVALID_ARG;
  if (a->n_src == 0 && a->mass == nullptr) return VQKV_OK;
  DeviceInfo di;
  const vqkv_status st = device_info(kCompactKernels, a->mode, &di);
  if (st != VQKV_OK) return st;
  CompactParams p;
  p.codes[VQKV_ROLE_K] = a->k_codes;
  p.codes[VQKV_ROLE_V] = a->v_codes;
  p.seq_lens = a->seq_lens;
  p.src = a->src;
  p.counts = a->counts;
  p.start = a->start;
  p.mass = a->mass;
  p.err = a->error_flags;
  p.stream_bytes = (long long)vqkv_code_bytes(a->mode, a->cap_len);
  p.B = a->B;
  p.Hkv = a->Hkv;
  p.src_heads = a->src_heads;
  p.n_src = a->n_src;
  p.cap_len = a->cap_len;
  set_paging(p, pg, a->mode);
  return launch_compact(a->mode, p, di.sms, di.compact_cluster[a->mode], static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? VQKV_OK
             : VQKV_ERR_CUDA;
}

}  // extern "C"

namespace vqkv {
namespace {

bool is_dtype(int t) { return t == VQKV_DTYPE_F16 || t == VQKV_DTYPE_F32 || t == VQKV_DTYPE_BF16; }
int dtype_bytes(int t) { return t == VQKV_DTYPE_F32 ? 4 : 2; }
bool is_rot_dim(int r) { return r >= 8 && r <= 128 && r % 8 == 0; }
// Below: no byte offset inside a strided array overflows.
constexpr long long kMaxStride = 1LL << 40;

// Rows [T][H][128] by strides, in elements; a single token's or head's stride counts as 0.
struct StridedRows {
  const void* base;
  int T, H, bytes;   // bytes of an element
  long long token, head;
  StridedRows(const void* x, int dtype, int T_, int H_, long long t, long long h)
      : base(x), T(T_), H(H_), bytes(dtype_bytes(dtype)), token(T_ > 1 ? t : 0), head(H_ > 1 ? h : 0) {}
  bool valid() const {
    return base != nullptr && aligned(base, 4 * bytes) && token >= 0 && head >= 0 && token % 4 == 0 && head % 4 == 0 &&
           token <= kMaxStride / T && head <= kMaxStride / H;
  }
  long long token_span() const { return (H - 1) * head + 128; }   // elements from a token's first to behind its last
  long long extent() const { return (T - 1) * token + token_span(); }
  bool rows_apart() const {   // tokens outside heads, or heads outside tokens
    const bool heads = H == 1 || head >= 128, tokens = T == 1 || token >= 128;
    return (heads && (T == 1 || token >= token_span())) || (tokens && (H == 1 || head >= (T - 1) * token + 128));
  }
  bool same(const StridedRows& o) const { return base == o.base && token == o.token && head == o.head; }
  // Known to share no element: apart as a whole, or interleaved token by token.
  bool apart(const StridedRows& o) const {
    if (!overlap(base, (size_t)extent() * bytes, o.base, (size_t)o.extent() * bytes)) return true;
    if (token != o.token || token < token_span() || token < o.token_span()) return false;
    const long long step = token * bytes;
    const long long d = (long long)(reinterpret_cast<uintptr_t>(o.base) - reinterpret_cast<uintptr_t>(base));
    const long long r = ((d % step) + step) % step;   // where o's tokens begin in this one's
    return r >= token_span() * bytes && step - r >= o.token_span() * bytes;
  }
};

// Cross attention: shares of all items' units per KV head, one CTA per SM in one wave.
struct CrossPlan {
  bool rows = false;    // one query per sequence: the decode's kernels and plan
  DecodePlan d;
  int n_splits = 1, layout = kBothParts;
  int groups_max = 1;   // items of a sequence, at most
  size_t query_off = 0, items_off = 0, partials_off = 0, ws_bytes = 0;
};

vqkv_status validate_cross_sizes(const vqkv_cross_args* ac) {
  if (ac == nullptr) return VQKV_ERR_INVALID_ARG;
  const vqkv_decode_args& a = ac->decode;
  const vqkv_status st = validate_decode_sizes(&a);
  if (st != VQKV_OK) return st;
  if (ac->dtype != VQKV_DTYPE_F16 && ac->dtype != VQKV_DTYPE_BF16) return VQKV_ERR_UNSUPPORTED;
  if (ac->n_rows < 0 || ac->max_queries < 1) return VQKV_ERR_INVALID_ARG;
  const long long units = (long long)std::min(a.B, kFlatMaxB) * ((a.max_seq_len + 63) / 64);
  if (a.Hkv > kMaxGridYZ || a.cap_len > kMaxTokens || ac->n_rows > (1 << 27) || ac->max_queries > (1 << 27) || units > kMaxTokens ||
      units * ((ac->max_queries * (long long)(a.Hq / a.Hkv) + 63) / 64) > kMaxTokens)
    return VQKV_ERR_UNSUPPORTED;
  return VQKV_OK;
}

vqkv_status plan_cross(const vqkv_cross_args* ac, CrossPlan* pl) {
  const vqkv_decode_args& a = ac->decode;
  DeviceInfo di;
  if (ac->max_queries == 1 && (long long)a.B * ((a.Hq / a.Hkv + 3) / 4) <= kMaxGridYZ) {
    pl->rows = true;
    const vqkv_status ready = device_info(kCrossRowsKernels, a.mode, &di);
    if (ready != VQKV_OK) return ready;
    PlanInput in = plan_input(&a);
    in.width = 4;
    in.rows = true;
    in.num_splits = std::min(in.num_splits, kRowsMaxSplits);
    const vqkv_status st = plan_decode(&in, &pl->d);
    // partials behind the tickets of all decode calls, which stay zero
    const size_t partials_off = decode_ticket_region_bytes(a.B, a.Hkv * kTicketGroups);
    pl->ws_bytes = pl->d.ws_bytes + (partials_off - pl->d.partials_off);
    pl->d.partials_off = partials_off;
    return st;
  }
  const vqkv_status st = device_info(kCrossKernels, a.mode, &di);
  if (st != VQKV_OK) return st;
  const long long g = a.Hq / a.Hkv, cols = ac->max_queries * g;
  pl->layout = cols <= 64 ? kPairs : kBothParts;
  const int width = cross_cols(pl->layout), B = std::max(std::min(a.B, kFlatMaxB), 1);
  // items, and tiles of full sequences, at most
  const long long items = std::max<long long>(1, std::min(B * ((cols + width - 1) / width), ac->n_rows * g / width + B));
  const long long units = items * std::max(1, (a.max_seq_len + 63) / 64);
  const long long want = a.num_splits > 0 ? std::min(a.num_splits, 1024) : cross_shares(pl->layout) * (di.sms / a.Hkv);
  pl->n_splits = (int)std::max<long long>(1, std::min(want, units));
  pl->groups_max = (int)((cols + width - 1) / width);
  pl->query_off = decode_ticket_region_bytes(a.B, a.Hkv * kTicketGroups);
  pl->items_off = pl->query_off + round_up(cross_query_bytes(B, a.Hq, a.Hkv, ac->n_rows, pl->layout), 256);
  pl->partials_off = pl->items_off + round_up(sizeof(int4) * pl->n_splits, 256);
  pl->ws_bytes = pl->partials_off;
  if (pl->n_splits > 1) pl->ws_bytes += sizeof(float) * (size_t)a.Hkv * pl->n_splits * 2 * width * kPartialStride;
  return VQKV_OK;
}

// Frequencies of the pairs, radians per position; false for arguments out of range.
bool rope_frequencies(const vqkv_rope_table_args* a, double (&f)[64]) {
  const double r = a->rot_dim, pi = 3.14159265358979323846;
  if (!(a->base > 1.0) || !std::isfinite(a->base) || !(std::fabs(a->amplitude) <= std::numeric_limits<float>::max())) return false;
  const bool scaled = a->scaling != VQKV_ROPE_NONE;
  const bool turns = a->scaling == VQKV_ROPE_WAVELENGTH || a->scaling == VQKV_ROPE_RAMP;
  if (scaled && (!(a->factor > 0.0) || !std::isfinite(a->factor))) return false;
  if (turns && (!(a->low_turns > 0.0) || !(a->high_turns > a->low_turns) || !std::isfinite(a->high_turns) || a->original_len < 1))
    return false;
  const double base = a->scaling == VQKV_ROPE_BASE ? a->base * std::pow(a->factor, r / (r - 2)) : a->base;
  if (!(base > 1.0) || !std::isfinite(base)) return false;
  double first = 0, last = 0;
  if (a->scaling == VQKV_ROPE_RAMP) {
    auto pair_of = [&](double n) { return r * std::log(a->original_len / (2 * pi * n)) / (2 * std::log(base)); };
    first = std::max(std::floor(pair_of(a->high_turns)), 0.0);
    last = std::min(std::ceil(pair_of(a->low_turns)), r - 1);
    if (!(last > first)) last = first + 0.001;
  }
  for (int i = 0; i < a->rot_dim / 2; ++i) {
    double g = std::pow(base, -2.0 * i / r);
    if (a->scaling == VQKV_ROPE_LINEAR) {
      g /= a->factor;
    } else if (a->scaling == VQKV_ROPE_WAVELENGTH) {
      const double n = a->original_len * g / (2 * pi);
      const double k = std::min(std::max((n - a->low_turns) / (a->high_turns - a->low_turns), 0.0), 1.0);
      g *= k + (1 - k) / a->factor;
    } else if (a->scaling == VQKV_ROPE_RAMP) {
      const double k = std::min(std::max((i - first) / (last - first), 0.0), 1.0);
      g *= 1 - k + k / a->factor;
    }
    if (!std::isfinite(g)) return false;
    f[i] = g;
  }
  return true;
}

}  // namespace
}  // namespace vqkv

extern "C" {

vqkv_status vqkv_rope_table(const vqkv_rope_table_args* a, void* stream) {
  if (a == nullptr) return VQKV_ERR_INVALID_ARG;
  if (!is_rot_dim(a->rot_dim) || a->scaling < VQKV_ROPE_NONE || a->scaling > VQKV_ROPE_RAMP) return VQKV_ERR_UNSUPPORTED;
  double f[64];
  if (a->n_pos < 0 || !rope_frequencies(a, f)) return VQKV_ERR_INVALID_ARG;
  if (a->n_pos == 0) return VQKV_OK;
  if (!a->table || !aligned(a->table, 16)) return VQKV_ERR_INVALID_ARG;
  DeviceInfo di;
  const vqkv_status st = device_info(&di);
  if (st != VQKV_OK) return st;
  RopeTableParams p{};
  for (int i = 0; i < a->rot_dim / 2; ++i) {
    const double turns = f[i] / (2 * 3.14159265358979323846);
    // 53 bits of the fraction; one that rounds up to a whole turn is none
    const double part = std::ldexp(turns - std::floor(turns), 64);
    p.step[i] = part < 18446744073709551616.0 ? (unsigned long long)part : 0ull;
  }
  p.table = a->table;
  p.n_pos = a->n_pos;
  p.rot = a->rot_dim;
  p.amplitude = (float)a->amplitude;
  return launch_rope_table(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? VQKV_OK : VQKV_ERR_CUDA;
}

vqkv_status vqkv_rope(const vqkv_rope_args* a, void* stream) {
  if (a == nullptr) return VQKV_ERR_INVALID_ARG;
  if (!is_dtype(a->dtype) || a->head_dim != 128 || !is_rot_dim(a->rot_dim) || a->n_heads > kMaxGridYZ) return VQKV_ERR_UNSUPPORTED;
  if (a->n_tokens < 0 || a->n_heads < 1 || a->n_pos < 1) return VQKV_ERR_INVALID_ARG;
  if (a->n_tokens == 0) return VQKV_OK;
  const StridedRows x(a->x, a->dtype, a->n_tokens, a->n_heads, a->x_token_stride, a->x_head_stride);
  const StridedRows out(a->out, a->dtype, a->n_tokens, a->n_heads, a->out_token_stride, a->out_head_stride);
  if (!x.valid() || !out.valid() || !out.rows_apart() || !(out.same(x) || out.apart(x))) return VQKV_ERR_INVALID_ARG;
  if (!a->positions || !a->table || !aligned(a->positions, 4) || !aligned(a->table, 16) || !aligned(a->error_flags, 4))
    return VQKV_ERR_INVALID_ARG;
  DeviceInfo di;
  const vqkv_status st = device_info(&di);
  if (st != VQKV_OK) return st;
  RopeParams p{};
  p.x = a->x, p.out = a->out;
  p.x_token = x.token, p.x_head = x.head, p.out_token = out.token, p.out_head = out.head;
  p.pos = a->positions, p.table = a->table, p.err = a->error_flags;
  p.T = a->n_tokens, p.H = a->n_heads, p.n_pos = a->n_pos, p.rot = a->rot_dim;
  p.dtype = a->dtype, p.interleaved = a->interleaved != 0, p.transpose = a->transpose != 0;
  return launch_rope(p, di.sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? VQKV_OK : VQKV_ERR_CUDA;
}

vqkv_status vqkv_append(const vqkv_append_args* a, const vqkv_paging* pg, void* stream) {
  if (a == nullptr) return VQKV_ERR_INVALID_ARG;
  if (!is_code_mode(a->mode) || !is_dtype(a->dtype) || a->head_dim != 128 || 2LL * a->Hkv > kMaxGridYZ) return VQKV_ERR_UNSUPPORTED;
  if (a->B < 0 || a->Hkv < 1 || a->n_tokens < 0 || a->cap_len < 1) return VQKV_ERR_INVALID_ARG;
  if ((long long)a->B * a->Hkv > 0x7fffffffLL || a->n_tokens > kMaxTokens || a->cap_len > kMaxTokens) return VQKV_ERR_UNSUPPORTED;
  if (a->rope_table != nullptr) {
    if (!is_rot_dim(a->rot_dim)) return VQKV_ERR_UNSUPPORTED;
    if (a->n_pos < 1 || !aligned(a->rope_table, 16)) return VQKV_ERR_INVALID_ARG;
  }
  if (pg != nullptr) {
    const vqkv_status st = validate_paging(pg, a->mode, a->cap_len);
    if (st != VQKV_OK) return st;
    if (a->B > 0 && a->n_tokens > 0 && (!pg->block_table || !aligned(pg->block_table, 4))) return VQKV_ERR_INVALID_ARG;
  }
  if (a->B == 0 || a->n_tokens == 0) return VQKV_OK;
  const StridedRows k(a->k, a->dtype, a->n_tokens, a->Hkv, a->k_token_stride, a->k_head_stride);
  const StridedRows v(a->v, a->dtype, a->n_tokens, a->Hkv, a->v_token_stride, a->v_head_stride);
  if (!k.valid() || !v.valid()) return VQKV_ERR_INVALID_ARG;
  if (!a->row_start || !a->pos || !a->s || !a->k_codebook || !a->v_codebook || !a->k_codes || !a->v_codes)
    return VQKV_ERR_INVALID_ARG;
  if (!aligned(a->row_start, 4) || !aligned(a->pos, 4) || !aligned(a->rope_pos, 4) || !aligned(a->s, 16) ||
      !aligned(a->k_codebook, 16) || !aligned(a->v_codebook, 16) || !aligned(a->near_tie_count, 8) || !aligned(a->error_flags, 4))
    return VQKV_ERR_INVALID_ARG;
  DeviceInfo di;
  vqkv_status st = device_info(&di);
  if (st != VQKV_OK) return st;
  st = device_info(append_few_rows(a->n_tokens, a->Hkv, di.sms) ? kAppendKernels : kAppendTileKernels, a->mode, &di);
  if (st != VQKV_OK) return st;
  AppendParams p{};
  EncodeParams& e = p.both;
  e.s = a->s;
  e.near_tie = a->near_tie_count;
  e.err = a->error_flags;
  e.stream_bytes = (long long)vqkv_code_bytes(a->mode, a->cap_len);
  e.B = a->B, e.Hkv = a->Hkv, e.cap_len = a->cap_len;
  set_paging(e, pg, a->mode);
  p.cb[VQKV_ROLE_K] = reinterpret_cast<const __half*>(a->k_codebook), p.cb[VQKV_ROLE_V] = reinterpret_cast<const __half*>(a->v_codebook);
  p.codes[VQKV_ROLE_K] = a->k_codes, p.codes[VQKV_ROLE_V] = a->v_codes;
  p.x[VQKV_ROLE_K] = k.base, p.token_stride[VQKV_ROLE_K] = k.token, p.head_stride[VQKV_ROLE_K] = k.head;
  p.x[VQKV_ROLE_V] = v.base, p.token_stride[VQKV_ROLE_V] = v.token, p.head_stride[VQKV_ROLE_V] = v.head;
  p.dtype = a->dtype, p.n_tokens = a->n_tokens;
  p.row_start = a->row_start, p.pos = a->pos;
  p.table = a->rope_table, p.rope_pos = a->rope_pos;
  p.n_table = a->n_pos, p.rot = a->rot_dim, p.interleaved = a->interleaved != 0;
  return launch_append(a->mode, p, di.sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? VQKV_OK : VQKV_ERR_CUDA;
}

size_t vqkv_cross_attn_workspace_bytes(const vqkv_cross_args* a) {
  CrossPlan pl;
  if (validate_cross_sizes(a) != VQKV_OK || plan_cross(a, &pl) != VQKV_OK) return 0;
  return pl.ws_bytes;
}

vqkv_status vqkv_cross_attn(const vqkv_cross_args* ac, const vqkv_paging* pg, void* stream) {
  vqkv_status st = validate_cross_sizes(ac);
  if (st != VQKV_OK) return st;
  const vqkv_decode_args* a = &ac->decode;
  if (ac->n_rows > 0) {
    st = validate_decode(a);
    if (st != VQKV_OK) return st;
  }
  if (pg != nullptr) {
    st = validate_paging(pg, a->mode, a->cap_len);
    if (st != VQKV_OK) return st;
    if (a->B > 0 && ac->n_rows > 0 && (!pg->block_table || !aligned(pg->block_table, 4))) return VQKV_ERR_INVALID_ARG;
  }
  if (a->B == 0 || ac->n_rows == 0) return VQKV_OK;
  if (!ac->row_start || !aligned(ac->row_start, 4)) return VQKV_ERR_INVALID_ARG;
  const long long row = a->Hq * 128LL, q_row = ac->n_rows > 1 ? ac->q_row_stride : row;
  if (q_row < row || q_row % 4 != 0 || q_row > kMaxStride / ac->n_rows) return VQKV_ERR_INVALID_ARG;
  if (!(a->q == a->out && q_row == row) &&
      overlap(a->q, 2 * (size_t)((ac->n_rows - 1) * q_row + row), a->out, 2 * (size_t)ac->n_rows * row))
    return VQKV_ERR_INVALID_ARG;
  CrossPlan pl;
  st = plan_cross(ac, &pl);
  if (st != VQKV_OK) return st;
  if (a->workspace == nullptr || a->workspace_bytes < pl.ws_bytes) return VQKV_ERR_WORKSPACE;
  if (!aligned(a->workspace, 256)) return VQKV_ERR_INVALID_ARG;
  unsigned char* ws = static_cast<unsigned char*>(a->workspace);
  DecodeParams p = packed_params(a, 1, pg);
  p.row_start = ac->row_start;
  p.n_rows = ac->n_rows;
  p.max_queries = ac->max_queries;
  p.bf16 = ac->dtype == VQKV_DTYPE_BF16;
  p.q_row = q_row;
  if (pl.rows) {
    p.tickets = reinterpret_cast<unsigned*>(ws + pl.d.tickets_off);
    p.partials = reinterpret_cast<float*>(ws + pl.d.partials_off);
    p.n_splits = pl.d.n_splits;
    p.tps = pl.d.tps;
    p.bpg = 1;   // plan_decode, rows
    p.flat = pl.d.flat;
    p.cgroups = pl.d.cgroups;
    const dim3 grid(pl.d.n_splits, a->Hkv, pl.d.n_bgroups * pl.d.cgroups);
    return launch_cross_rows(a->mode, p, grid, static_cast<cudaStream_t>(stream)) == cudaSuccess ? VQKV_OK : VQKV_ERR_CUDA;
  }
  p.tickets = reinterpret_cast<unsigned*>(ws + pl.items_off);
  p.ncols = (int)std::min<long long>(ac->max_queries * (long long)p.g, cross_cols(pl.layout));
  p.partials = reinterpret_cast<float*>(ws + pl.partials_off);
  p.n_splits = pl.n_splits;
  p.max_polls = kTilePolls;
  for (int b0 = 0; b0 < a->B; b0 += kFlatMaxB)
    if (launch_cross(a->mode, batch_part(p, b0, a->B), pl.layout, pl.groups_max, ws + pl.query_off,
                     static_cast<cudaStream_t>(stream)) != cudaSuccess)
      return VQKV_ERR_CUDA;
  return VQKV_OK;
}

const char* vqkv_status_string(vqkv_status s) {
  switch (s) {
    case VQKV_OK: return "ok";
    case VQKV_ERR_INVALID_ARG: return "invalid argument";
    case VQKV_ERR_UNSUPPORTED: return "unsupported configuration";
    case VQKV_ERR_WORKSPACE: return "workspace missing or too small";
    case VQKV_ERR_CUDA: return "CUDA error";
    case VQKV_ERR_NO_DEVICE: return "no usable CUDA device";
  }
  return "unknown status";
}

}  // extern "C"
