// Host side of the VQ encode (kernels in encode_kernels.cuh): preparation and
// launches.
#include "common.cuh"
#include "encode_kernels.cuh"
#include "internal.h"

namespace vqkv {

int encode_tile_rows(int mode) {
  return mode == VQKV_MODE_VQ2    ? UmGeo<VQKV_MODE_VQ2>::ROWS
         : mode == VQKV_MODE_VQ4  ? UmGeo<VQKV_MODE_VQ4>::ROWS
         : mode == VQKV_MODE_VQ3  ? UmGeo<VQKV_MODE_VQ3>::ROWS
         : mode == VQKV_MODE_VQ15 ? UmGeo<VQKV_MODE_VQ15>::ROWS
                                  : UmGeo<VQKV_MODE_VQ125>::ROWS;
}

cudaError_t encode_prepare(int mode) {
  const cudaFuncAttribute smem_attr = cudaFuncAttributeMaxDynamicSharedMemorySize;
  if (mode == VQKV_MODE_VQ3) return cudaFuncSetAttribute(encode_vq3_kernel<ENC3_SPLIT>, smem_attr, (int)kEnc3Smem);
  if (mode == VQKV_MODE_VQ15) return cudaFuncSetAttribute(encode_vq15_tc_split_kernel<>, smem_attr, (int)kTcSplitSmem);
  return cudaSuccess;
}

template <int MODE>
cudaError_t prepare_tiles() {
  return prepare_split_kernel(encode_umma_kernel<MODE>, um::THREADS, um::SPLIT_REGS, (int)UmGeo<MODE>::SMEM);
}
cudaError_t encode_tiles_prepare(int mode) {
  return mode == VQKV_MODE_VQ2    ? prepare_tiles<VQKV_MODE_VQ2>()
         : mode == VQKV_MODE_VQ4  ? prepare_tiles<VQKV_MODE_VQ4>()
         : mode == VQKV_MODE_VQ3  ? prepare_tiles<VQKV_MODE_VQ3>()
         : mode == VQKV_MODE_VQ15 ? prepare_tiles<VQKV_MODE_VQ15>()
                                  : prepare_tiles<VQKV_MODE_VQ125>();
}

// split_rows: one row per CTA, candidates split over the CTA's warps.
cudaError_t launch_encode(int mode, const EncodeParams& p, int blocks_x, bool split_rows, cudaStream_t stream) {
  const dim3 grid(blocks_x, p.Hkv);
  if (mode == VQKV_MODE_VQ2) {
    if (split_rows) return launch_pdl(encode_vq2_kernel<ENC_WARPS, 4>, grid, dim3(ENC_THREADS), 0, stream, p);
    return launch_pdl(encode_umma_kernel<VQKV_MODE_VQ2>, grid, dim3(um::THREADS), UmGeo<VQKV_MODE_VQ2>::SMEM,
                      stream, p);
  }
  if (mode == VQKV_MODE_VQ4) {
    if (split_rows) return launch_pdl(encode_vq2_kernel<ENC_WARPS, 2>, grid, dim3(ENC_THREADS), 0, stream, p);
    return launch_pdl(encode_umma_kernel<VQKV_MODE_VQ4>, grid, dim3(um::THREADS), UmGeo<VQKV_MODE_VQ4>::SMEM,
                      stream, p);
  }
  if (mode == VQKV_MODE_VQ125) {
    if (split_rows) return launch_pdl(encode_vq125_kernel<ENC_WARPS>, grid, dim3(ENC_THREADS), 0, stream, p);
    return launch_pdl(encode_umma_kernel<VQKV_MODE_VQ125>, grid, dim3(um::THREADS), UmGeo<VQKV_MODE_VQ125>::SMEM,
                      stream, p);
  }
  if (mode == VQKV_MODE_VQ3) {
    if (split_rows)
      return launch_pdl(encode_vq3_kernel<ENC3_SPLIT>, grid, dim3(ENC3_SPLIT * 32), kEnc3Smem, stream, p);
    return launch_pdl(encode_umma_kernel<VQKV_MODE_VQ3>, grid, dim3(um::THREADS), UmGeo<VQKV_MODE_VQ3>::SMEM,
                      stream, p);
  }
  if (split_rows) return launch_pdl(encode_vq15_tc_split_kernel<>, grid, dim3(TC_THREADS), kTcSplitSmem, stream, p);
  return launch_pdl(encode_umma_kernel<VQKV_MODE_VQ15>, grid, dim3(um::THREADS), UmGeo<VQKV_MODE_VQ15>::SMEM,
                    stream, p);
}

}  // namespace vqkv
