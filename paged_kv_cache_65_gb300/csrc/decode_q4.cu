// Instantiations of the split pass over q4_0 K/V (4-bit codes, one fp16 scale
// per 32 values).
#include "decode_q4.cuh"
#include "decode_launch.cuh"

namespace pkv {

namespace {
template <int D, int UR>
cudaError_t launch_q4(DecodeArgs a, int sm_count, int max_grid, int* grid_io, cudaStream_t st,
                      bool pdl) {
  constexpr int smem = decode_q4_smem_bytes<D>();
  const int v = a.segs ? 1 : 0;
  auto kern = v ? decode_q4_kernel<D, UR, true> : decode_q4_kernel<D, UR, false>;
  // the dynamic shared-memory limit is a per-function, per-device attribute
  static bool attr_set[2][64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_set[v][dev]) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    attr_set[v][dev] = true;
  }
  if (*grid_io <= 0) {
    const int g = kQ4CtasPerSm * sm_count;
    *grid_io = g > max_grid ? max_grid : g;
  }
  a.grid = *grid_io;
  return launch_kernel(pdl, kern, dim3(a.grid), dim3(kQ4Threads), smem, st, a);
}

template <int D>
cudaError_t launch_q4_units(const DecodeArgs& a, int sm_count, int max_grid, int* grid_io,
                            cudaStream_t st, bool pdl) {
  switch (q4_unit_rows(a.block_size)) {
    case 8: return launch_q4<D, 8>(a, sm_count, max_grid, grid_io, st, pdl);
    case 16: return launch_q4<D, 16>(a, sm_count, max_grid, grid_io, st, pdl);
    case 32: return launch_q4<D, 32>(a, sm_count, max_grid, grid_io, st, pdl);
    case 64: return launch_q4<D, 64>(a, sm_count, max_grid, grid_io, st, pdl);
    default: return cudaErrorInvalidValue;  // not a tensor-core shape
  }
}
}  // namespace

cudaError_t launch_decode_q4(int D, const DecodeArgs& a, int sm_count, int max_grid, int* grid_io,
                             cudaStream_t st, bool pdl, bool* supported) {
  *supported = true;
  if (D == 128) return launch_q4_units<128>(a, sm_count, max_grid, grid_io, st, pdl);
  if (D == 64) return launch_q4_units<64>(a, sm_count, max_grid, grid_io, st, pdl);
  *supported = false;
  return cudaSuccess;
}

}  // namespace pkv
