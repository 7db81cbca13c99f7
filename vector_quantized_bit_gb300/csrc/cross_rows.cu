// Cross attention of one query per sequence at most (vqkv_cross_attn with
// max_queries = 1): the single-query decode's kernels on packed rows, four columns
// of two fp16 parts of q' per CTA, a CTA per sequence where they are short
// (plan_decode).  One column of 16 sequences of 700 to 1,500 tokens and 16 heads at 2
// bit takes 17 us here, 27 in equal shares of all tokens, and 39 us on the tile kernel,
// whose products have 128 rows and whose softmax then hangs on one warp.
#include "decode_kernels.cuh"

namespace vqkv {
namespace {

using DecodeKernel = void (*)(DecodeParams);
template <int MODE>
DecodeKernel ring_of(bool flat, bool paged) {
  return flat ? (paged ? (DecodeKernel)decode_vq2_kernel<kQueryGroups, true, MODE, true, kRows>
                       : (DecodeKernel)decode_vq2_kernel<kQueryGroups, false, MODE, true, kRows>)
              : (paged ? (DecodeKernel)decode_vq2_kernel<kQueryGroups, true, MODE, false, kRows>
                       : (DecodeKernel)decode_vq2_kernel<kQueryGroups, false, MODE, false, kRows>);
}
DecodeKernel rows_kernel_of(int mode, bool flat, bool paged) {
  switch (mode) {
    case VQKV_MODE_VQ2: return ring_of<VQKV_MODE_VQ2>(flat, paged);
    case VQKV_MODE_VQ4: return ring_of<VQKV_MODE_VQ4>(flat, paged);
    case VQKV_MODE_VQ3: return ring_of<VQKV_MODE_VQ3>(flat, paged);
    case VQKV_MODE_VQ125: return ring_of<VQKV_MODE_VQ125>(flat, paged);
    default:   // 1.5 bit has no flat plan
      return paged ? (DecodeKernel)decode_vq15_kernel<kQueryGroups, true, kRows>
                   : (DecodeKernel)decode_vq15_kernel<kQueryGroups, false, kRows>;
  }
}

}  // namespace

cudaError_t cross_rows_prepare(int mode) {
  cudaError_t e = cudaSuccess;
  for (int fl = 0; fl < (mode == VQKV_MODE_VQ15 ? 1 : 2); ++fl)
    for (int pg = 0; pg < 2; ++pg)
      if (e == cudaSuccess)
        e = cudaFuncSetAttribute(rows_kernel_of(mode, fl != 0, pg != 0), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)decode_smem_bytes(mode));
  return e;
}

cudaError_t launch_cross_rows(int mode, const DecodeParams& p, dim3 grid, cudaStream_t stream) {
  return launch_pdl(rows_kernel_of(mode, p.flat != 0, p.block_table != nullptr), grid, dim3(decode_threads(mode)),
                    decode_smem_bytes(mode), stream, p);
}

}  // namespace vqkv
