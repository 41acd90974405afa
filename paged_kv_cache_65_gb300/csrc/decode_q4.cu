// Instantiations of the split pass over q4_0 K/V (4-bit codes, one fp16 scale
// per 32 values).
#include "decode_q4.cuh"
#include "decode_launch.cuh"

namespace pkv {

namespace {
template <int D, int UR, bool WIDE>
cudaError_t launch_q4(DecodeArgs a, int sm_count, int max_grid, int* grid_io, cudaStream_t st,
                      bool pdl) {
  using T = Q4Team<WIDE>;
  constexpr int smem = T::TEAMS * decode_q4_team_bytes<D, WIDE>();
  static_assert(smem <= 227 * 1024, "shared memory of a CTA");
  const int v = a.segs ? 1 : 0;
  auto kern = v ? decode_q4_kernel<D, UR, true, WIDE> : decode_q4_kernel<D, UR, false, WIDE>;
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
    if (fa.numRegs != T::REGS) return cudaErrorInvalidConfiguration;
    attr_set[v][dev] = true;
  }
  // the split counts teams
  if (*grid_io <= 0) {
    const int g = T::TEAMS * sm_count;
    *grid_io = (g > max_grid ? max_grid : g) / T::TEAMS * T::TEAMS;
  }
  a.grid = *grid_io;
  return launch_kernel(pdl, kern, dim3(a.grid / T::TEAMS), dim3(T::THREADS), smem, st, a);
}

template <int D>
cudaError_t launch_q4_units(const DecodeArgs& a, bool wide, int sm_count, int max_grid,
                            int* grid_io, cudaStream_t st, bool pdl) {
  auto go = [&](auto narrow_fn, auto wide_fn) {
    return wide ? wide_fn(a, sm_count, max_grid, grid_io, st, pdl)
                : narrow_fn(a, sm_count, max_grid, grid_io, st, pdl);
  };
  switch (q4_unit_rows(a.block_size)) {
    case 8: return go(launch_q4<D, 8, false>, launch_q4<D, 8, true>);
    case 16: return go(launch_q4<D, 16, false>, launch_q4<D, 16, true>);
    case 32: return go(launch_q4<D, 32, false>, launch_q4<D, 32, true>);
    case 64: return go(launch_q4<D, 64, false>, launch_q4<D, 64, true>);
    default: return cudaErrorInvalidValue;  // not a tensor-core shape
  }
}
}  // namespace

cudaError_t launch_decode_q4(int D, const DecodeArgs& a, bool wide, int sm_count, int max_grid,
                             int* grid_io, cudaStream_t st, bool pdl, bool* supported) {
  *supported = true;
  if (D == 128) return launch_q4_units<128>(a, wide, sm_count, max_grid, grid_io, st, pdl);
  if (D == 64) return launch_q4_units<64>(a, wide, sm_count, max_grid, grid_io, st, pdl);
  *supported = false;
  return cudaSuccess;
}

}  // namespace pkv
