// Single- and multi-query decode over packed codes: kernel tables and
// launches (the kernels are in decode_kernels.cuh).
#include "decode_kernels.cuh"

namespace vqkv {
namespace {

// One CTA per (query head, sequence), one thread per channel.
__global__ void __launch_bounds__(kHeadDim) decode_combine_kernel(const DecodeParams p) {
  grid_dependency_wait();
  grid_dependents_launch();
  combine_splits(p);
}

}  // namespace

cudaError_t launch_combine(const DecodeParams& p, cudaStream_t stream) {
  return launch_pdl(decode_combine_kernel, dim3(p.Hkv * p.ncols, p.B), dim3(kHeadDim), 0, stream, p);
}

int decode_tile_tokens(int mode) { return mode == VQKV_MODE_VQ15 ? V15_TILE : V2_TILE; }
int decode_tiles_per_step(int mode) {
  return mode == VQKV_MODE_VQ2   ? V2Geo<VQKV_MODE_VQ2>::TPI
         : mode == VQKV_MODE_VQ4 ? V2Geo<VQKV_MODE_VQ4>::TPI
         : mode == VQKV_MODE_VQ3 ? V2Geo<VQKV_MODE_VQ3>::TPI
         : mode == VQKV_MODE_VQ125 ? V2Geo<VQKV_MODE_VQ125>::TPI
                                 : 1;
}
size_t decode_smem_bytes(int mode) {
  return mode == VQKV_MODE_VQ2     ? kV2Smem
         : mode == VQKV_MODE_VQ4   ? kV4Smem
         : mode == VQKV_MODE_VQ3   ? kV3Smem
         : mode == VQKV_MODE_VQ125 ? kV125Smem
                                   : kV15Smem;
}
int decode_threads(int mode) { return mode == VQKV_MODE_VQ15 ? V15_THREADS : V2_THREADS; }

namespace {
using DecodeKernel = void (*)(DecodeParams);

// [flat][paged][query layout] instantiations of one mode's decode kernel.
template <int MODE>
struct ByteCodeKernels {
  static constexpr DecodeKernel k[2][2][3] = {
      {{decode_vq2_kernel<kOneQuery, false, MODE, false>, decode_vq2_kernel<kQueries, false, MODE, false>,
        decode_vq2_kernel<kQueryGroups, false, MODE, false>},
       {decode_vq2_kernel<kOneQuery, true, MODE, false>, decode_vq2_kernel<kQueries, true, MODE, false>,
        decode_vq2_kernel<kQueryGroups, true, MODE, false>}},
      {{decode_vq2_kernel<kOneQuery, false, MODE, true>, decode_vq2_kernel<kQueries, false, MODE, true>,
        decode_vq2_kernel<kQueryGroups, false, MODE, true>},
       {decode_vq2_kernel<kOneQuery, true, MODE, true>, decode_vq2_kernel<kQueries, true, MODE, true>,
        decode_vq2_kernel<kQueryGroups, true, MODE, true>}}};
};
struct Vq15Kernels {
  static constexpr DecodeKernel k[2][2][3] = {
      {{decode_vq15_kernel<kOneQuery, false>, decode_vq15_kernel<kQueries, false>,
        decode_vq15_kernel<kQueryGroups, false>},
       {decode_vq15_kernel<kOneQuery, true>, decode_vq15_kernel<kQueries, true>,
        decode_vq15_kernel<kQueryGroups, true>}},
      {{nullptr, nullptr, nullptr}, {nullptr, nullptr, nullptr}}};   // no flat plan at 1.5 bit
};

const DecodeKernel (*kernels_of(int mode))[2][3] {
  return mode == VQKV_MODE_VQ2   ? ByteCodeKernels<VQKV_MODE_VQ2>::k
         : mode == VQKV_MODE_VQ4 ? ByteCodeKernels<VQKV_MODE_VQ4>::k
         : mode == VQKV_MODE_VQ3 ? ByteCodeKernels<VQKV_MODE_VQ3>::k
         : mode == VQKV_MODE_VQ125 ? ByteCodeKernels<VQKV_MODE_VQ125>::k
                                 : Vq15Kernels::k;
}
}  // namespace

cudaError_t decode_prepare(int mode) {
  const cudaFuncAttribute a = cudaFuncAttributeMaxDynamicSharedMemorySize;
  const auto ks = kernels_of(mode);
  cudaError_t e = cudaSuccess;
  for (int fl = 0; fl < 2; ++fl)
    for (int pg = 0; pg < 2; ++pg)
      for (int q = 0; q < 3; ++q)
        if (e == cudaSuccess && ks[fl][pg][q] != nullptr)
          e = cudaFuncSetAttribute(ks[fl][pg][q], a, (int)decode_smem_bytes(mode));
  return e;
}

cudaError_t decode_occupancy(int mode, int* blocks_per_sm) {
  return cudaOccupancyMaxActiveBlocksPerMultiprocessor(blocks_per_sm, kernels_of(mode)[0][0][kOneQuery],
                                                       decode_threads(mode), decode_smem_bytes(mode));
}

cudaError_t launch_decode(int mode, const DecodeParams& p, dim3 grid, cudaStream_t stream) {
  const int q = p.M == 1 ? kOneQuery : p.cgroups == 1 ? kQueries : kQueryGroups;
  const bool paged = p.block_table != nullptr;
  const DecodeKernel k = kernels_of(mode)[p.flat ? 1 : 0][paged][q];
  if (k == nullptr) return cudaErrorInvalidValue;
  return launch_pdl(k, grid, dim3(decode_threads(mode)), decode_smem_bytes(mode), stream, p);
}

}  // namespace vqkv
