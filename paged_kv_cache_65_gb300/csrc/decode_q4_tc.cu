// Instantiations of the tcgen05 split pass over q4_0 K/V, D_h = 128.
#include "decode_q4_tc.cuh"
#include "decode_launch.cuh"

namespace pkv {

cudaError_t launch_decode_q4_tc(const DecodeArgs& a_in, int sm_count, int max_grid, int* grid_io,
                                cudaStream_t st, bool pdl) {
  constexpr int smem = decode_q4_tc_smem_bytes();
  static_assert(smem <= 227 * 1024, "shared memory of a CTA");
  const int v = a_in.segs ? 1 : 0;
  auto kern = v ? decode_q4_tc_kernel<true> : decode_q4_tc_kernel<false>;
  // the dynamic shared-memory limit is a per-function, per-device attribute
  static bool attr_set[2][64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_set[v][dev]) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    // the warpgroups' register split assumes the launch count
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, kern);
    if (e != cudaSuccess) return e;
    if (fa.numRegs != kQ4TcRegsLaunch) return cudaErrorInvalidConfiguration;
    attr_set[v][dev] = true;
  }
  if (*grid_io <= 0) *grid_io = sm_count < max_grid ? sm_count : max_grid;
  DecodeArgs a = a_in;
  a.grid = *grid_io;
  return launch_kernel(pdl, kern, dim3(a.grid), dim3(kQ4TcThreads), smem, st, a);
}

}  // namespace pkv
