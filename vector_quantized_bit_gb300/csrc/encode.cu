// Host side of the VQ encode (kernels in encode_kernels.cuh): preparation,
// occupancy and launches.
#include "common.cuh"
#include "encode_kernels.cuh"
#include "internal.h"

namespace vqkv {

int encode_warps_per_cta() { return ENC_WARPS; }

cudaError_t encode_prepare(int mode) {
  const cudaFuncAttribute smem_attr = cudaFuncAttributeMaxDynamicSharedMemorySize;
  if (mode == VQKV_MODE_VQ3) {
    cudaError_t e = cudaFuncSetAttribute(encode_vq3_kernel<ENC3_SPLIT>, smem_attr, (int)kEnc3Smem);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(encode_umma_kernel<VQKV_MODE_VQ3>, smem_attr, (int)UmGeo<VQKV_MODE_VQ3>::SMEM);
    return e;
  }
  if (mode == VQKV_MODE_VQ125)
    return cudaFuncSetAttribute(encode_umma_kernel<VQKV_MODE_VQ125>, smem_attr, (int)UmGeo<VQKV_MODE_VQ125>::SMEM);
  if (mode == VQKV_MODE_VQ2)
    return cudaFuncSetAttribute(encode_umma_kernel<VQKV_MODE_VQ2>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)UmGeo<VQKV_MODE_VQ2>::SMEM);
  if (mode == VQKV_MODE_VQ4)
    return cudaFuncSetAttribute(encode_umma_kernel<VQKV_MODE_VQ4>, smem_attr, (int)UmGeo<VQKV_MODE_VQ4>::SMEM);
  if (mode != VQKV_MODE_VQ15) return cudaSuccess;
  {
    const cudaError_t e0 = cudaFuncSetAttribute(encode_umma_kernel<VQKV_MODE_VQ15>,
                                                cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                (int)UmGeo<VQKV_MODE_VQ15>::SMEM);
    if (e0 != cudaSuccess) return e0;
    const cudaError_t e1 = cudaFuncSetAttribute(encode_vq15_tc_split_kernel<>,
                                                cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kTcSplitSmem);
    if (e1 != cudaSuccess) return e1;
  }
  return cudaSuccess;
}

cudaError_t encode_occupancy(int mode, int* blocks_per_sm) {
  if (mode == VQKV_MODE_VQ2)
    return cudaOccupancyMaxActiveBlocksPerMultiprocessor(blocks_per_sm, encode_umma_kernel<VQKV_MODE_VQ2>,
                                                         um::THREADS, UmGeo<VQKV_MODE_VQ2>::SMEM);
  if (mode == VQKV_MODE_VQ4)
    return cudaOccupancyMaxActiveBlocksPerMultiprocessor(blocks_per_sm, encode_umma_kernel<VQKV_MODE_VQ4>,
                                                         um::THREADS, UmGeo<VQKV_MODE_VQ4>::SMEM);
  if (mode == VQKV_MODE_VQ3)
    return cudaOccupancyMaxActiveBlocksPerMultiprocessor(blocks_per_sm, encode_umma_kernel<VQKV_MODE_VQ3>,
                                                         um::THREADS, UmGeo<VQKV_MODE_VQ3>::SMEM);
  if (mode == VQKV_MODE_VQ125)
    return cudaOccupancyMaxActiveBlocksPerMultiprocessor(blocks_per_sm, encode_umma_kernel<VQKV_MODE_VQ125>,
                                                         um::THREADS, UmGeo<VQKV_MODE_VQ125>::SMEM);
  return cudaOccupancyMaxActiveBlocksPerMultiprocessor(blocks_per_sm, encode_umma_kernel<VQKV_MODE_VQ15>,
                                                       um::THREADS, UmGeo<VQKV_MODE_VQ15>::SMEM);
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
