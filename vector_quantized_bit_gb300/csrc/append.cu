// Ragged append (vqkv_append): the encode kernels over both roles' rows of a
// batch's new tokens, keys rotated on the way.  A grid row per KV head, its CTAs
// divided among the roles, so one launch writes the whole step.
//
// What a row is and where it goes: rows.cuh.  The search and its bound: encode_kernels.cuh
// (128 dimensions against 256 to 4,096 centroids a subvector; the screening products
// are the least of it, ranking their results the most).  The rotation, the strides and
// the lookup of a row's sequence run in warps that wait for the search anyway: 17,450
// ragged bf16 tokens of 8 heads into a paged 2-bit cache take 405 us, the two encodes of
// as many plain rows 377.
#include <algorithm>

#include "common.cuh"
#include "encode_kernels.cuh"
#include "internal.h"

namespace vqkv {
namespace {

using AppendKernel = void (*)(AppendParams);
struct AppendVariant {
  AppendKernel kernel;
  int threads;
  size_t smem;
  int rows;     // rows a CTA takes at a time
};

// Few rows: one row per CTA, its candidates split over the CTA's warps.  Many:
// the tensor-memory search, one persistent CTA per SM.
AppendVariant variant(int mode, bool few) {
  switch (mode) {
    case VQKV_MODE_VQ2:
      if (few) return {encode_vq2_kernel<ENC_WARPS, 4, true>, ENC_THREADS, 0, 1};
      return {encode_umma_kernel<VQKV_MODE_VQ2, true>, um::THREADS, UmGeo<VQKV_MODE_VQ2>::SMEM, UmGeo<VQKV_MODE_VQ2>::ROWS};
    case VQKV_MODE_VQ4:
      if (few) return {encode_vq2_kernel<ENC_WARPS, 2, true>, ENC_THREADS, 0, 1};
      return {encode_umma_kernel<VQKV_MODE_VQ4, true>, um::THREADS, UmGeo<VQKV_MODE_VQ4>::SMEM, UmGeo<VQKV_MODE_VQ4>::ROWS};
    case VQKV_MODE_VQ3:
      if (few) return {encode_vq3_kernel<ENC3_SPLIT, true>, ENC3_SPLIT * 32, kEnc3Smem, 1};
      return {encode_umma_kernel<VQKV_MODE_VQ3, true>, um::THREADS, UmGeo<VQKV_MODE_VQ3>::SMEM, UmGeo<VQKV_MODE_VQ3>::ROWS};
    case VQKV_MODE_VQ125:
      if (few) return {encode_vq125_kernel<ENC_WARPS, true>, ENC_THREADS, 0, 1};
      return {encode_umma_kernel<VQKV_MODE_VQ125, true>, um::THREADS, UmGeo<VQKV_MODE_VQ125>::SMEM,
              UmGeo<VQKV_MODE_VQ125>::ROWS};
    default:
      if (few) return {encode_vq15_tc_split_kernel<true>, TC_THREADS, kTcSplitSmem, 1};
      return {encode_umma_kernel<VQKV_MODE_VQ15, true>, um::THREADS, UmGeo<VQKV_MODE_VQ15>::SMEM,
              UmGeo<VQKV_MODE_VQ15>::ROWS};
  }
}

}  // namespace

bool append_few_rows(int n_tokens, int Hkv, int sms) { return (long long)n_tokens * 2 * Hkv <= sms; }

cudaError_t append_prepare(int mode, bool few) {
  const AppendVariant v = variant(mode, few);
  if (!few) return prepare_split_kernel(v.kernel, v.threads, um::SPLIT_REGS, (int)v.smem);
  return v.smem > 0 ? cudaFuncSetAttribute(v.kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)v.smem) : cudaSuccess;
}

cudaError_t launch_append(int mode, AppendParams p, int sms, cudaStream_t stream) {
  const int Hkv = p.both.Hkv;
  const AppendVariant v = variant(mode, append_few_rows(p.n_tokens, Hkv, sms));
  const int want = (p.n_tokens + v.rows - 1) / v.rows;   // CTAs of a KV head and role with work
  int keys = want, values = want;
  if (v.rows > 1) {
    // whole waves: with one CTA per SM a few CTAs more would double the time
    const int most = std::max(2, sms / Hkv);
    keys = std::min(want, (most + 1) / 2);
    values = std::min(want, most - keys);
  }
  p.key_ctas = keys;
  return launch_pdl(v.kernel, dim3(keys + values, Hkv), dim3(v.threads), v.smem, stream, p);
}

}  // namespace vqkv
