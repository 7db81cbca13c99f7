// Decode attention that also accumulates each cached token's attention weight
// (vqkv_decode_attn_mass).
//
// The weight of token t is sum over columns of exp2(s_t - m) / l, and a
// column's m and l are known only when every split has been merged.  The
// decode kernels (decode_kernels.cuh, MASS) therefore store the scores as
// they pass through the softmax, 16 bytes per token and KV head for 4
// columns, and the merge leaves (m, 1 / l) per column; a second, streaming
// kernel adds the weights.  The alternative, a second pass over the key codes,
// would gather every key centroid again, which is what bounds the decode.
// 4 columns of 196,608 tokens and 8 KV heads at 2 bit: 45.3 us for both kernels
// (the decode alone 35.7), 113 MB at 2.5 TB/s; the second kernel's 6 us are bound
// by memory (16 bytes of scores and 8 of weights per token, partly from L2).
#include "decode_kernels.cuh"

namespace vqkv {
namespace {

constexpr int MS_THREADS = 256, MS_TOKENS = 4;   // tokens per thread

// mass[b][h][t] += sum over columns c of exp2(score_c - m_c) / l_c, one thread
// per token, columns in order.
__global__ void __launch_bounds__(MS_THREADS) decode_mass_kernel(const DecodeParams p) {
  const int kvh = blockIdx.y, b = blockIdx.z;
  grid_dependency_wait();
  grid_dependents_launch();
  const bool skip = timed_out(p);   // scores or statistics may be missing; needed only at the end
  const int L = min(max(p.seq_lens[b], 0), p.max_seq_len);
  const int t0 = blockIdx.x * (MS_THREADS * MS_TOKENS) + threadIdx.x;
  if (t0 >= L) return;
  const size_t pair = (size_t)b * p.Hkv + kvh;
  const float* scores = p.scores + pair * p.cgroups * p.score_row * 4;
  const float2* stats = p.stats + pair * p.ncols;
  float* mass = p.mass + pair * p.cap_len;
  float w[MS_TOKENS], old[MS_TOKENS];
#pragma unroll
  for (int i = 0; i < MS_TOKENS; ++i) {
    w[i] = 0.f;
    const int t = t0 + i * MS_THREADS;
    old[i] = t < L ? mass[t] : 0.f;
  }
  for (int cg = 0; cg < p.cgroups; ++cg) {
    float4 sc[MS_TOKENS];
#pragma unroll
    for (int i = 0; i < MS_TOKENS; ++i) {
      const int t = t0 + i * MS_THREADS;
      if (t < L) sc[i] = __ldcg(reinterpret_cast<const float4*>(scores + ((size_t)cg * p.score_row + t) * 4));
    }
    const int n = min(4, p.ncols - 4 * cg);
    float2 st[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) st[c] = c < n ? stats[4 * cg + c] : make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < MS_TOKENS; ++i) {
      if (t0 + i * MS_THREADS >= L) break;
      w[i] += fast_exp2(sc[i].x - st[0].x) * st[0].y;
      if (n > 1) w[i] += fast_exp2(sc[i].y - st[1].x) * st[1].y;
      if (n > 2) w[i] += fast_exp2(sc[i].z - st[2].x) * st[2].y;
      if (n > 3) w[i] += fast_exp2(sc[i].w - st[3].x) * st[3].y;
    }
  }
#pragma unroll
  for (int i = 0; i < MS_TOKENS; ++i) {
    const int t = t0 + i * MS_THREADS;
    if (t < L && !skip) mass[t] = old[i] + w[i];
  }
}

__global__ void __launch_bounds__(kHeadDim) mass_combine_kernel(const DecodeParams p) {
  grid_dependency_wait();
  grid_dependents_launch();
  combine_splits<true>(p);
}

using DecodeKernel = void (*)(DecodeParams);
template <int MODE>
DecodeKernel ring_of(bool flat, bool paged) {
  return flat ? (paged ? (DecodeKernel)decode_vq2_kernel<kQueryGroups, true, MODE, true, true>
                       : (DecodeKernel)decode_vq2_kernel<kQueryGroups, false, MODE, true, true>)
              : (paged ? (DecodeKernel)decode_vq2_kernel<kQueryGroups, true, MODE, false, true>
                       : (DecodeKernel)decode_vq2_kernel<kQueryGroups, false, MODE, false, true>);
}
DecodeKernel mass_kernel_of(int mode, bool flat, bool paged) {
  switch (mode) {
    case VQKV_MODE_VQ2: return ring_of<VQKV_MODE_VQ2>(flat, paged);
    case VQKV_MODE_VQ4: return ring_of<VQKV_MODE_VQ4>(flat, paged);
    case VQKV_MODE_VQ3: return ring_of<VQKV_MODE_VQ3>(flat, paged);
    case VQKV_MODE_VQ125: return ring_of<VQKV_MODE_VQ125>(flat, paged);
    default:   // 1.5 bit has no flat plan
      return paged ? (DecodeKernel)decode_vq15_kernel<kQueryGroups, true, true>
                   : (DecodeKernel)decode_vq15_kernel<kQueryGroups, false, true>;
  }
}

}  // namespace

cudaError_t decode_mass_prepare(int mode) {
  cudaError_t e = cudaSuccess;
  for (int fl = 0; fl < (mode == VQKV_MODE_VQ15 ? 1 : 2); ++fl)
    for (int pg = 0; pg < 2; ++pg)
      if (e == cudaSuccess)
        e = cudaFuncSetAttribute(mass_kernel_of(mode, fl != 0, pg != 0), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)decode_smem_bytes(mode));
  return e;
}

cudaError_t launch_decode_mass(int mode, const DecodeParams& p, dim3 grid, cudaStream_t stream) {
  cudaError_t e = launch_pdl(mass_kernel_of(mode, p.flat != 0, p.block_table != nullptr), grid, dim3(decode_threads(mode)),
                             decode_smem_bytes(mode), stream, p);
  if (e == cudaSuccess && p.defer_merge && p.n_splits > 1)
    e = launch_pdl(mass_combine_kernel, dim3(p.Hkv * p.ncols, p.B), dim3(kHeadDim), 0, stream, p);
  if (e == cudaSuccess && p.max_seq_len > 0)
    e = launch_pdl(decode_mass_kernel, dim3((p.max_seq_len + MS_THREADS * MS_TOKENS - 1) / (MS_THREADS * MS_TOKENS), p.Hkv, p.B),
                   dim3(MS_THREADS), 0, stream, p);
  return e;
}

}  // namespace vqkv
