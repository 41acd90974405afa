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

// fp16 copy of the blocks a staged prefill of a q4_0 pool reads: first the
// (sequence, K/V head) powers of two (seq_scale), then the copy.
struct StageQ4 {
  const int32_t* table;  // [n_seq][max_blocks]
  const int32_t* ctx;    // [n_seq]
  int n_seq, max_blocks, layer;
  void* k_stage;         // fp16 rows (copy block i * max_blocks + j, slot) of H_kv * D_h
  void* v_stage;
  int32_t* stage_table;  // [n_seq][max_blocks]: i * max_blocks + j
  float2* seq_scale;     // [n_seq][H_kv]
};
cudaError_t launch_prefill_stage_q4(const kvPool* p, const StageQ4& g, cudaStream_t st);

}  // namespace pkv
