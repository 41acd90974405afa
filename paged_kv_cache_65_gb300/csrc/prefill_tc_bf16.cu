// The tcgen05 chunked-prefill attention over bfloat16 K/V, D_h = 128.
#include "prefill_tc_launch.cuh"

namespace pkv {

cudaError_t launch_prefill_tc(const CUtensorMap& tk, const CUtensorMap& tv, const PrefillArgs& a,
                              int max_chunk, int n_items, cudaStream_t st, bool pdl) {
  return launch_prefill<false>(tk, tv, a, max_chunk, n_items, st, pdl);
}

}  // namespace pkv
