// Row writes into a q4_0 pool and row reads from any pool (rows.cu).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "pool.h"

namespace pkv {

// Slot write into a q4_0 pool (layer -1: every layer).
cudaError_t launch_slot_write_q4(const kvPool* p, int layer, const void* k_new, const void* v_new,
                                 const int64_t* slots, int n_tokens, cudaStream_t st);

// Rows at `slots` as float32 or bfloat16 (layer -1: every layer).
cudaError_t launch_gather_rows(const kvPool* p, int layer, const int64_t* slots, int n_tokens,
                               void* k_out, void* v_out, int out_dtype, cudaStream_t st);

}  // namespace pkv
