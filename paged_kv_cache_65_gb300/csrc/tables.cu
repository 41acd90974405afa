// Block tables and slot maps built on the device from the requests' token
// counts, and the return of a request's blocks (paged_tables_append,
// paged_tables_release).
//
// Both run as two kernels.  The first (one CTA) checks the whole batch, scans
// the listed rows' new blocks and tokens, and commits lengths and the free
// ring's state, or refuses the batch and changes nothing.  The second fills
// what each listed row and token gets, spread over the device.
//
// What bounds them is latency: the scan's loads (row, then its length), two
// scans over the CTA and the second kernel's start make 5.6 us for 37 rows of
// 256 entries, whatever the bytes.  1,000 rows of 2,050 entries, 12 MB in and
// out, take 9.2 us: the fill moves them with eight loads in flight a thread and
// 32-bit divisions (four loads and 64-bit ones: 11.3 us).  Reading the rows
// ahead of the wait for the scan gained nothing, nor did 16-byte vectors, which
// rows of 2,050 entries do not allow.
#include <cuda_runtime.h>

#include <cstdint>

#include "launch.cuh"
#include "pool.h"
#include "ptx.cuh"

namespace pkv {
namespace {

constexpr int kScanThreads = 1024;
constexpr int kFillThreads = 256, kFillAhead = 8;
constexpr int kMaxRows = 1 << 20;  // rows of a table set: one bit each in shared memory

// Workspace: the batch's verdict and the ring position it starts at, then one
// record per listed row.
struct BatchHead {
  int64_t head;    // ring position of the batch's first block
  int32_t ok;      // 0: refused, outputs describe an empty batch
  int32_t n_tok;   // tokens of the batch
  int32_t pad[4];
};
struct RowPlan {
  int32_t old_len;  // tokens before the batch
  int32_t n;        // new tokens (append); blocks (release)
  int32_t blk0;     // blocks of the batch before this row's
  int32_t tok0;     // tokens of the batch before this row's
};

struct TablesArgs {
  int32_t* tables;
  int32_t* lens;
  int32_t* free_ids;
  int64_t* free_state;
  int n_rows, max_blocks, free_cap;
  const int32_t* rows;
  const int32_t* counts;
  int n_seq, max_tokens, B, n_blocks;
  int64_t* slots;
  int32_t* positions;
  int32_t* chunk_start;
  int32_t* block_table;
  int32_t* context_lens;
  int32_t* lens_out;
  int64_t* free_state_out;
  BatchHead* head;
  RowPlan* plan;
  int32_t* status;
};

// Inclusive scan of two 64-bit values over the CTA's threads; returns the
// thread's exclusive values and the totals.
__device__ void block_scan2(int64_t& a, int64_t& b, int64_t* sh, int64_t& ta, int64_t& tb) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t a0 = a, b0 = b;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, a, o), y = __shfl_up_sync(0xffffffffu, b, o);
    if (lane >= o) {
      a += x;
      b += y;
    }
  }
  if (lane == 31) {
    sh[warp] = a;
    sh[32 + warp] = b;
  }
  __syncthreads();
  if (warp == 0) {
    int64_t x = sh[lane], y = sh[32 + lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t u = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) {
        x += u;
        y += v;
      }
    }
    sh[lane] = x;
    sh[32 + lane] = y;
  }
  __syncthreads();
  a += (warp ? sh[warp - 1] : 0) - a0;
  b += (warp ? sh[32 + warp - 1] : 0) - b0;
  ta = sh[31];
  tb = sh[63];
  __syncthreads();
}

// Row i of the batch: -1 = a padding entry, -2 = out of range.
__device__ __forceinline__ int batch_row(const TablesArgs& a, int i) {
  const int r = a.rows ? a.rows[i] : i;
  return r >= -1 && r < a.n_rows ? r : -2;
}

template <bool RELEASE>
__global__ void __launch_bounds__(kScanThreads, 1) tables_scan_kernel(const TablesArgs a) {
  extern __shared__ uint32_t seen[];  // one bit per row
  __shared__ int64_t sh[64];
  __shared__ int bad;
  griddep_wait();
  griddep_launch_dependents();
  // everything the first 1024 rows need is on its way before the bits are clear
  const int64_t head = a.free_state[0], count = a.free_state[1];
  int r = -1, old = 0, cnt = 0;
  auto load_row = [&](int i) {
    r = -1;
    old = cnt = 0;
    if (i >= a.n_seq) return;
    if (!RELEASE) cnt = a.counts ? a.counts[i] : 1;
    r = batch_row(a, i);
    if (r >= 0) old = a.lens[r];
  };
  load_row(threadIdx.x);
  const int words = (a.n_rows + 31) / 32;
  for (int i = threadIdx.x; i < words; i += kScanThreads) seen[i] = 0;
  if (threadIdx.x == 0) bad = 0;
  __syncthreads();
  const int64_t room = static_cast<int64_t>(a.max_blocks) * a.B;
  int64_t blocks = 0, tokens = 0;
  for (int base = 0; base < a.n_seq; base += kScanThreads) {
    const int i = base + threadIdx.x;
    int64_t nb = 0, nt = 0;
    if (i < a.n_seq) {
      if (r >= 0) {
        const bool dup = (atomicOr(&seen[r >> 5], 1u << (r & 31)) >> (r & 31)) & 1u;
        if (dup || old < 0 || old > room || cnt < 0 || static_cast<int64_t>(old) + cnt > room) {
          bad = 1;
        } else if (RELEASE) {
          nb = (old + a.B - 1) / a.B;
        } else {
          nt = cnt;
          nb = (static_cast<int64_t>(old) + cnt + a.B - 1) / a.B - (old + a.B - 1) / a.B;
        }
      } else if (r == -2) {
        bad = 1;
      }
    }
    const int64_t mine_b = nb, mine_t = nt;
    int64_t tb, tt;
    block_scan2(nb, nt, sh, tb, tt);
    if (i < a.n_seq)
      a.plan[i] = RowPlan{old, static_cast<int32_t>(RELEASE ? mine_b : mine_t),
                          static_cast<int32_t>(blocks + nb), static_cast<int32_t>(tokens + nt)};
    blocks += tb;
    tokens += tt;
    if (base + kScanThreads < a.n_seq) load_row(i + kScanThreads);
  }
  __syncthreads();
  int why = bad ? KV_DEV_BAD_TABLE_ROW : 0;
  if (head < 0 || head >= a.free_cap || count < 0 || count > a.free_cap)
    why |= KV_DEV_BAD_TABLE_ROW;
  else if (RELEASE ? count + blocks > a.free_cap : blocks > count)
    why |= RELEASE ? KV_DEV_BAD_TABLE_ROW : KV_DEV_NO_FREE_BLOCK;
  if (!RELEASE && tokens > a.max_tokens) why |= KV_DEV_BAD_TABLE_ROW;
  const bool ok = why == 0;
  __syncthreads();  // every thread has read the state before it is written
  if (threadIdx.x == 0) {
    if (!ok) record_status(a.status, why);
    // release: the ring position behind the last free block
    a.head[0] = BatchHead{RELEASE ? (head + count) % a.free_cap : head, ok ? 1 : 0,
                          static_cast<int32_t>(ok ? tokens : 0), {0, 0, 0, 0}};
    if (RELEASE) {
      if (ok) a.free_state[1] = count + blocks;
    } else {
      const bool take = ok && blocks > 0;
      a.free_state_out[0] = take ? (head + blocks) % a.free_cap : head;
      a.free_state_out[1] = take ? count - blocks : count;
    }
    if (!RELEASE && a.chunk_start) a.chunk_start[a.n_seq] = ok ? static_cast<int32_t>(tokens) : 0;
  }
  if (!RELEASE && a.lens_out != a.lens) {
    for (int r = threadIdx.x; r < a.n_rows; r += kScanThreads) a.lens_out[r] = a.lens[r];
    __syncthreads();
  }
  for (int i = threadIdx.x; i < a.n_seq; i += kScanThreads) {
    const int r = batch_row(a, i);
    if (RELEASE) {
      if (ok && r >= 0) a.lens[r] = 0;
      continue;
    }
    const RowPlan p = a.plan[i];  // written by this thread
    if (ok && r >= 0) a.lens_out[r] = p.old_len + p.n;
    if (a.chunk_start) a.chunk_start[i] = ok ? p.tok0 : 0;
    if (a.context_lens) a.context_lens[i] = ok && r >= 0 ? p.old_len + p.n : 0;
  }
}

// The k-th block the batch takes.
__device__ __forceinline__ int taken(const TablesArgs& a, int64_t head, int k) {
  int64_t at = head + k;
  if (at >= a.free_cap) at -= a.free_cap;
  return a.free_ids[at];
}

// Append, second kernel.  CTAs below n_tok_ctas: one token a thread, its row
// found by bisection of the rows' first tokens.  The others: table entries,
// gridDim.y parts of a listed row.
__global__ void __launch_bounds__(kFillThreads) tables_fill_kernel(const TablesArgs a,
                                                                   int n_tok_ctas, int parts) {
  griddep_wait();
  griddep_launch_dependents();
  const BatchHead h = a.head[0];
  if (static_cast<int>(blockIdx.x) < n_tok_ctas) {
    const int t = blockIdx.x * kFillThreads + threadIdx.x;
    if (t >= a.max_tokens) return;
    int64_t slot = -1;
    int pos = -1;
    if (t < h.n_tok) {
      int lo = 0, hi = a.n_seq;  // plan[lo].tok0 <= t < plan[hi].tok0
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.plan[mid].tok0 <= t)
          lo = mid;
        else
          hi = mid;
      }
      const RowPlan p = a.plan[lo];
      const int r = batch_row(a, lo);
      pos = p.old_len + t - p.tok0;
      const int j = pos / a.B, ob = (p.old_len + a.B - 1) / a.B;
      const int id = j < ob ? a.tables[static_cast<int64_t>(r) * a.max_blocks + j]
                            : taken(a, h.head, p.blk0 + j - ob);
      if (id < 0 || id >= a.n_blocks)
        record_status(a.status, KV_DEV_BAD_BLOCK_ID);  // the slot stays -1: not written
      else
        slot = static_cast<int64_t>(id) * a.B + (pos - j * a.B);
    }
    if (a.slots) a.slots[t] = slot;
    if (a.positions) a.positions[t] = pos;
    return;
  }
  const unsigned w = blockIdx.x - n_tok_ctas;
  const int i = w / static_cast<unsigned>(parts), part = w - i * parts;
  const RowPlan p = a.plan[i];
  const int r = batch_row(a, i);
  const bool live = h.ok && r >= 0;
  // below 2^32: a row's room is below 2^31 tokens
  const unsigned uB = a.B, end = static_cast<unsigned>(p.old_len) + p.n;
  const int ob = live ? static_cast<int>((p.old_len + uB - 1) / uB) : 0;
  const int nb = live ? static_cast<int>((end + uB - 1) / uB) : 0;
  int32_t* row = live ? a.tables + static_cast<int64_t>(r) * a.max_blocks : nullptr;
  int32_t* out = a.block_table ? a.block_table + static_cast<int64_t>(i) * a.max_blocks : nullptr;
  const int j0 = out ? 0 : ob, j1 = out ? a.max_blocks : nb;
  // kFillAhead entries a thread, their loads in flight together
  for (int jb = j0 + part * kFillThreads * kFillAhead + threadIdx.x; jb < j1;
       jb += parts * kFillThreads * kFillAhead) {
    int id[kFillAhead];
#pragma unroll
    for (int u = 0; u < kFillAhead; ++u) {
      const int j = jb + u * kFillThreads;
      id[u] = j < ob ? row[j] : (j < nb ? taken(a, h.head, p.blk0 + j - ob) : -1);
    }
#pragma unroll
    for (int u = 0; u < kFillAhead; ++u) {
      const int j = jb + u * kFillThreads;
      if (j >= j1) continue;
      if (j >= ob && j < nb) row[j] = id[u];
      if (out) out[j] = id[u];
    }
  }
}

// Release, second kernel: a row's blocks go to the ring's end in table order,
// and its entries become -1.
__global__ void __launch_bounds__(kFillThreads) tables_release_kernel(const TablesArgs a,
                                                                      int parts) {
  griddep_wait();
  griddep_launch_dependents();
  const BatchHead h = a.head[0];
  const int i = blockIdx.x / parts, part = blockIdx.x - i * parts;
  const RowPlan p = a.plan[i];
  const int r = batch_row(a, i);
  if (!h.ok || r < 0) return;
  int32_t* row = a.tables + static_cast<int64_t>(r) * a.max_blocks;
  for (int j = part * kFillThreads + threadIdx.x; j < p.n; j += parts * kFillThreads) {
    int64_t at = h.head + p.blk0 + j;
    if (at >= a.free_cap) at -= a.free_cap;
    a.free_ids[at] = row[j];
    row[j] = -1;
  }
}

size_t workspace_bytes(int n_seq) {
  return sizeof(BatchHead) + static_cast<size_t>(n_seq) * sizeof(RowPlan);
}

kvStatus check_tables(const kvPool* p, const kvTables* t, const int32_t* d_rows, int n_seq,
                      const void* ws, size_t ws_bytes) {
  if (!p || !p->k || !t || n_seq < 0) return KV_ERR_INVALID_ARG;
  if (t->n_rows <= 0 || t->n_rows > kMaxRows || t->max_blocks <= 0 || t->free_cap <= 0)
    return KV_ERR_INVALID_ARG;
  if (static_cast<int64_t>(t->max_blocks) * p->B >= (int64_t(1) << 31)) return KV_ERR_INVALID_ARG;
  if (!t->tables || !t->lens || !t->free_ids || !t->free_state) return KV_ERR_INVALID_ARG;
  if (!d_rows && n_seq > t->n_rows) return KV_ERR_INVALID_ARG;
  if (!pool_on_current_device(p)) return KV_ERR_INVALID_ARG;
  if (n_seq > 0 && (!ws || (reinterpret_cast<uintptr_t>(ws) & 15) != 0 ||
                    ws_bytes < workspace_bytes(n_seq)))
    return KV_ERR_INVALID_ARG;
  return KV_OK;
}

TablesArgs base_args(const kvPool* p, const kvTables* t, const int32_t* d_rows, int n_seq,
                     void* ws) {
  TablesArgs a = {};
  a.tables = t->tables;
  a.lens = t->lens;
  a.free_ids = t->free_ids;
  a.free_state = t->free_state;
  a.n_rows = t->n_rows;
  a.max_blocks = t->max_blocks;
  a.free_cap = t->free_cap;
  a.rows = d_rows;
  a.n_seq = n_seq;
  a.B = p->B;
  a.n_blocks = p->N;
  a.head = static_cast<BatchHead*>(ws);
  a.plan = reinterpret_cast<RowPlan*>(static_cast<unsigned char*>(ws) + sizeof(BatchHead));
  a.status = p->d_status;
  return a;
}

template <bool RELEASE>
cudaError_t launch_scan(bool pdl, const TablesArgs& a, cudaStream_t st) {
  const size_t smem = static_cast<size_t>((a.n_rows + 31) / 32) * 4;
  if (smem > 40 * 1024) {  // with the static part past the default limit
    const cudaError_t e = cudaFuncSetAttribute(
        tables_scan_kernel<RELEASE>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxRows / 8);
    if (e != cudaSuccess) return e;
  }
  return launch_kernel(pdl, tables_scan_kernel<RELEASE>, dim3(1), dim3(kScanThreads), smem, st, a);
}

// CTAs per row: one for each kFillAhead * kFillThreads entries (to the nearest:
// a CTA goes round for what is left), at most eight.
int row_parts(int max_blocks) {
  const int per = kFillAhead * kFillThreads;
  const int want = max_blocks / per + (max_blocks % per > per / 2);
  return want < 1 ? 1 : (want > 8 ? 8 : want);
}

}  // namespace
}  // namespace pkv

extern "C" {

size_t paged_tables_workspace_bytes(const kvPool* p, int n_seq) {
  return !p || n_seq < 0 ? 0 : pkv::workspace_bytes(n_seq);
}

kvStatus paged_tables_append(kvPool* p, const kvTables* t, const int32_t* d_rows,
                             const int32_t* d_counts, int n_seq, int max_tokens, int64_t* d_slots,
                             int32_t* d_positions, int32_t* d_chunk_start, int32_t* d_block_table,
                             int32_t* d_context_lens, int32_t* d_lens_out,
                             int64_t* d_free_state_out, void* d_workspace, size_t workspace_bytes,
                             void* stream) {
  using namespace pkv;
  kvStatus s = check_tables(p, t, d_rows, n_seq, d_workspace, workspace_bytes);
  if (s != KV_OK) return s;
  if (max_tokens < 0 || d_block_table == t->tables) return KV_ERR_INVALID_ARG;
  if (n_seq == 0) return KV_OK;
  TablesArgs a = base_args(p, t, d_rows, n_seq, d_workspace);
  a.counts = d_counts;
  a.max_tokens = max_tokens;
  a.slots = d_slots;
  a.positions = d_positions;
  a.chunk_start = d_chunk_start;
  a.block_table = d_block_table;
  a.context_lens = d_context_lens;
  a.lens_out = d_lens_out ? d_lens_out : t->lens;
  a.free_state_out = d_free_state_out ? d_free_state_out : t->free_state;
  const int n_tok_ctas =
      d_slots || d_positions ? (max_tokens + kFillThreads - 1) / kFillThreads : 0;
  const int parts = row_parts(t->max_blocks);
  if (static_cast<int64_t>(n_tok_ctas) + static_cast<int64_t>(n_seq) * parts > 0x7fffffffLL)
    return KV_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (launch_scan<false>(p->pdl, a, st) != cudaSuccess) return KV_ERR_CUDA;
  p->device_tables = true;
  const cudaError_t e = launch_kernel(p->pdl, tables_fill_kernel, dim3(n_tok_ctas + n_seq * parts),
                                      dim3(kFillThreads), 0, st, a, n_tok_ctas, parts);
  return e == cudaSuccess ? KV_OK : KV_ERR_CUDA;
}

kvStatus paged_tables_release(kvPool* p, const kvTables* t, const int32_t* d_rows, int n_seq,
                              void* d_workspace, size_t workspace_bytes, void* stream) {
  using namespace pkv;
  kvStatus s = check_tables(p, t, d_rows, n_seq, d_workspace, workspace_bytes);
  if (s != KV_OK) return s;
  if (n_seq == 0) return KV_OK;
  TablesArgs a = base_args(p, t, d_rows, n_seq, d_workspace);
  const int parts = row_parts(t->max_blocks);
  if (static_cast<int64_t>(n_seq) * parts > 0x7fffffffLL) return KV_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (launch_scan<true>(p->pdl, a, st) != cudaSuccess) return KV_ERR_CUDA;
  p->device_tables = true;
  const cudaError_t e = launch_kernel(p->pdl, tables_release_kernel, dim3(n_seq * parts),
                                      dim3(kFillThreads), 0, st, a, parts);
  return e == cudaSuccess ? KV_OK : KV_ERR_CUDA;
}

}  // extern "C"
