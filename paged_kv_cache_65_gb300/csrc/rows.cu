// Row writes into a q4_0 pool and row reads from any pool.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "launch.cuh"
#include "ptx.cuh"
#include "rows.h"

namespace pkv {

namespace {

// Codes of eight values as one 32-bit word of nibbles c + 8.  The format asks
// for x / d rounded to float32 (IEEE) and then to the nearest integer, ties to
// even.  r = x * inv is within 2^-21 |x / d| of that quotient, and |x / d| <=
// 10.5 by the choice of d (a subnormal scale may be rounded down by a third),
// so both round to the same integer unless r lies within 1e-5 of a half: only
// then are the eight divided out.  Rounding is the addition of 1.5 * 2^23,
// whose sum holds the integer in its low bits; four nibbles are joined by
// multiply-adds (exact below 2^24), so no conversion instruction is needed.
__device__ __forceinline__ uint32_t q4_codes8(const float (&f)[8], float d, float inv) {
  constexpr float kRound = 12582912.f;  // 1.5 * 2^23
  float c[8];
  float off = 0.f;  // largest distance from the integer taken
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float r = f[k] * inv;
    c[k] = __fadd_rn(r, kRound) - kRound;
    off = fmaxf(off, fabsf(r - c[k]));
  }
  if (!(off < 0.49999f)) {
#pragma unroll
    for (int k = 0; k < 8; ++k) c[k] = d > 0.f ? rintf(__fdiv_rn(f[k], d)) : 0.f;
  }
  float lo = 0.f, hi = 0.f;
#pragma unroll
  for (int k = 3; k >= 0; --k) {
    lo = fmaf(lo, 16.f, fminf(fmaxf(c[k], -7.f), 7.f) + 8.f);
    hi = fmaf(hi, 16.f, fminf(fmaxf(c[k + 4], -7.f), 7.f) + 8.f);
  }
  // 2^23 + n holds n < 2^16 in its low half
  return __byte_perm(__float_as_uint(lo + 8388608.f), __float_as_uint(hi + 8388608.f), 0x5410);
}

// Slot write into a q4_0 pool.  Four lanes share a group of 32 bfloat16
// values, eight each (one 16-byte load): the group's largest |x| by two
// shuffles, d = the fp16 nearest to it over 7 (float32 IEEE division), codes =
// the integers nearest to x / d clamped to [-7, 7], stored as c + 8, zero when
// d is 0.  A lane's eight nibbles are one 32-bit word, a group's four words its
// 16 bytes of the chunk's code plane.  What bounds it is latency: slot, values
// and stores depend on each other, so a CTA takes up to kWriteTokens tokens of
// a layer and every lane has the loads of all of them in flight at once, and
// instructions, 270 a vector: 128 tokens into 36 layers, 8 heads of 128, take 15
// us, 19 MB in and 5 MB out (17 us with one token a CTA; a whole group a lane
// saved a fifth of the instructions, the same time, and made one step's 37
// tokens 4.7 us instead of 3.7 with the read-back).
constexpr int kWriteTokens = 2;

__global__ void __launch_bounds__(256)
    slot_write_q4_kernel(const uint4* __restrict__ k_new, const uint4* __restrict__ v_new,
                         const int64_t* __restrict__ slots, int n_tok, int per_cta,
                         unsigned char* kc, unsigned char* vc, int layer, int n_blocks, int B,
                         int H, int GR, int32_t* status) {
  griddep_wait();
  griddep_launch_dependents();
  const int i0 = blockIdx.x * per_cta;
  const int ly = layer >= 0 ? layer : blockIdx.y;
  const int row = H * GR * 4;  // lanes (8-value vectors) of a token row
  const long long src = ((layer >= 0 ? 0LL : (long long)blockIdx.y * n_tok) + i0) * row;
  const int64_t n_slots = static_cast<int64_t>(n_blocks) * B;
  const long long chunk_bytes = static_cast<long long>(B) * GR * 18;
  const unsigned quad = 0xfu << (threadIdx.x & 28);
  // K lanes, then V lanes: both multiples of 4, so a group's lanes run together
  for (int v = threadIdx.x; v < 2 * row; v += blockDim.x) {
    const bool is_k = v < row;
    const int vv = is_k ? v : v - row;
    const uint4* in = (is_k ? k_new : v_new) + src + vv;
    uint4 x[kWriteTokens];
    int64_t slot[kWriteTokens];
#pragma unroll
    for (int u = 0; u < kWriteTokens; ++u) {
      if (u >= per_cta || i0 + u >= n_tok) continue;
      slot[u] = slots[i0 + u];
      x[u] = in[static_cast<long long>(u) * row];
    }
    const int gi = vv >> 2;  // group of the token row
    const int h = gi / GR, q = gi - h * GR;
#pragma unroll
    for (int u = 0; u < kWriteTokens; ++u) {
      if (u >= per_cta || i0 + u >= n_tok || slot[u] < 0) continue;
      if (slot[u] >= n_slots) {
        if (threadIdx.x == 0) record_status(status, KV_DEV_BAD_SLOT);
        continue;
      }
      const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
      float f[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        f[2 * k] = __uint_as_float(w[k] << 16);
        f[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
      }
      float amax = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) amax = fmaxf(amax, fabsf(f[k]));
      amax = fmaxf(amax, __shfl_xor_sync(quad, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(quad, amax, 2));
      const __half d16 = __float2half_rn(__fdiv_rn(amax, 7.f));
      const float d = __half2float(d16);
      const uint32_t word = d > 0.f ? q4_codes8(f, d, __fdividef(1.f, d)) : 0x88888888u;
      const uint32_t blk = static_cast<uint32_t>(slot[u]) / static_cast<uint32_t>(B);
      const int o = static_cast<int>(static_cast<uint32_t>(slot[u]) - blk * B);
      unsigned char* chunk =
          (is_k ? kc : vc) + ((static_cast<long long>(ly) * n_blocks + blk) * H + h) * chunk_bytes;
      reinterpret_cast<uint32_t*>(chunk + (static_cast<long long>(q) * B + o) * 16)[vv & 3] = word;
      if ((vv & 3) == 0) {
        __half* sc = reinterpret_cast<__half*>(chunk + static_cast<long long>(GR) * B * 16);
        sc[is_k ? o * GR + q : q * B + o] = d16;
      }
    }
  }
}

// Eight (float32 pools: four) consecutive values of a row as float32.
template <int DT>
struct RowSource {
  static constexpr int VEC = DT == KV_DTYPE_F32 ? 4 : 8;
  const unsigned char* cache;   // K or V
  const unsigned char* scales;  // q8_0
  float scale;                  // FP8
  int B, H, D, GR;
  bool is_k;

  // vector v of the row [H][D] at (block index incl. layer, offset)
  __device__ __forceinline__ void load(long long blk, int o, int v, float (&f)[VEC]) const {
    const long long row = (blk * B + o) * H * D / VEC + v;
    if constexpr (DT == KV_DTYPE_F32) {
      const float4 x = reinterpret_cast<const float4*>(cache)[row];
      f[0] = x.x;
      f[1] = x.y;
      f[2] = x.z;
      f[3] = x.w;
    } else if constexpr (DT == KV_DTYPE_BF16) {
      const uint4 x = reinterpret_cast<const uint4*>(cache)[row];
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        f[2 * k] = __uint_as_float(w[k] << 16);
        f[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
      }
    } else if constexpr (DT == KV_DTYPE_FP8_E4M3) {
      const uint2 x = reinterpret_cast<const uint2*>(cache)[row];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t h2;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;"
            : "=r"(h2)
            : "h"(static_cast<uint16_t>((k < 2 ? x.x : x.y) >> (16 * (k & 1)))));
        f[2 * k] = scale * __half2float(__ushort_as_half(static_cast<unsigned short>(h2 & 0xffffu)));
        f[2 * k + 1] = scale * __half2float(__ushort_as_half(static_cast<unsigned short>(h2 >> 16)));
      }
    } else if constexpr (DT == KV_DTYPE_Q8_0) {
      const uint2 x = reinterpret_cast<const uint2*>(cache)[row];
      const int gi = v >> 2, h = gi / GR, q = gi - h * GR;
      const float d = __half2float(
          reinterpret_cast<const __half*>(scales)[((blk * H + h) * B + o) * GR + q]);
#pragma unroll
      for (int k = 0; k < 8; ++k)
        f[k] = d * static_cast<float>(static_cast<int8_t>(((k < 4 ? x.x : x.y) >> (8 * (k & 3))) & 0xffu));
    } else {
      const int gi = v >> 2, h = gi / GR, q = gi - h * GR;
      const unsigned char* chunk = cache + (blk * H + h) * (static_cast<long long>(B) * GR * 18);
      const uint32_t x = reinterpret_cast<const uint32_t*>(
          chunk + (static_cast<long long>(q) * B + o) * 16)[v & 3];
      const float d = __half2float(reinterpret_cast<const __half*>(
          chunk + static_cast<long long>(GR) * B * 16)[is_k ? o * GR + q : q * B + o]);
#pragma unroll
      for (int k = 0; k < 8; ++k)
        // 2^23 + n - (2^23 + 8) = c without a conversion
        f[k] = d * (__uint_as_float(0x4b000000u | ((x >> (4 * k)) & 15u)) - 8388616.f);
    }
  }
};

// Rows at the listed slots: one token of a layer a CTA, one vector of its K or
// V row a thread.  Bound by the sectors it touches: a q4_0 row of one head is
// D / 32 pieces of 16 bytes and its scales, B * 16 bytes apart, so that 128
// tokens of 36 layers at scattered slots read 44 MB for 5 MB of codes and write
// 19 MB in 13 us, 4.7 TB/s.
template <int DT, bool BF16>
__global__ void __launch_bounds__(256)
    gather_rows_kernel(RowSource<DT> ks, RowSource<DT> vs, const int64_t* __restrict__ slots,
                       int n_tok, int layer, int n_blocks, void* k_out, void* v_out,
                       int32_t* status) {
  constexpr int VEC = RowSource<DT>::VEC;
  griddep_wait();
  griddep_launch_dependents();
  const int i = blockIdx.x;
  const int ly = layer >= 0 ? layer : blockIdx.y;
  const int64_t slot = slots[i];
  if (slot < 0) return;
  if (slot >= static_cast<int64_t>(n_blocks) * ks.B) {
    if (threadIdx.x == 0) record_status(status, KV_DEV_BAD_SLOT);
    return;
  }
  // a pool has fewer than 2^31 slots
  const uint32_t blk = static_cast<uint32_t>(slot) / static_cast<uint32_t>(ks.B);
  const int o = static_cast<int>(static_cast<uint32_t>(slot) - blk * ks.B);
  const int row = ks.H * ks.D / VEC;
  const long long dst = ((layer >= 0 ? 0LL : (long long)blockIdx.y * n_tok) + i) * row;
  for (int v = threadIdx.x; v < 2 * row; v += blockDim.x) {
    const bool is_k = v < row;
    const int vv = is_k ? v : v - row;
    float f[VEC];
    (is_k ? ks : vs).load(static_cast<long long>(ly) * n_blocks + blk, o, vv, f);
    void* out = is_k ? k_out : v_out;
    if constexpr (BF16) {
      uint32_t w[VEC / 2];
#pragma unroll
      for (int k = 0; k < VEC / 2; ++k) {
        const __nv_bfloat162 a = __floats2bfloat162_rn(f[2 * k], f[2 * k + 1]);
        w[k] = *reinterpret_cast<const uint32_t*>(&a);
      }
      if constexpr (VEC == 8)
        reinterpret_cast<uint4*>(out)[dst + vv] = make_uint4(w[0], w[1], w[2], w[3]);
      else
        reinterpret_cast<uint2*>(out)[dst + vv] = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
      for (int k = 0; k < VEC / 4; ++k)
        reinterpret_cast<float4*>(out)[(dst + vv) * (VEC / 4) + k] =
            make_float4(f[4 * k], f[4 * k + 1], f[4 * k + 2], f[4 * k + 3]);
    }
  }
}

// Tokens per CTA: several where that still leaves the SMs two CTAs each.
int tokens_per_cta(const kvPool* p, int n_tokens, int layer, int most) {
  const long long rows = static_cast<long long>(n_tokens) * (layer >= 0 ? 1 : p->L);
  const int sms = p->sm_count > 0 ? p->sm_count : 1;
  int n = most;
  while (n > 1 && rows < 2LL * sms * n) n >>= 1;
  return n;
}

template <int DT>
cudaError_t launch_gather(const kvPool* p, int layer, const int64_t* slots, int n_tokens,
                          void* k_out, void* v_out, int out_dtype, cudaStream_t st) {
  RowSource<DT> ks{static_cast<const unsigned char*>(p->k),
                   static_cast<const unsigned char*>(p->k_sc), p->k_scale, p->B, p->H, p->D,
                   p->D / 32, true};
  RowSource<DT> vs{static_cast<const unsigned char*>(p->v),
                   static_cast<const unsigned char*>(p->v_sc), p->v_scale, p->B, p->H, p->D,
                   p->D / 32, false};
  const int lanes = 2 * p->H * p->D / RowSource<DT>::VEC;
  const int threads = lanes >= 256 ? 256 : (lanes + 31) / 32 * 32;
  const dim3 grid(n_tokens, layer >= 0 ? 1 : p->L);
  return launch_kernel(p->pdl,
                       out_dtype == KV_DTYPE_BF16 ? gather_rows_kernel<DT, true>
                                                  : gather_rows_kernel<DT, false>,
                       grid, dim3(threads), 0, st, ks, vs, slots, n_tokens, layer, p->N, k_out, v_out,
                       p->d_status);
}

// Staged chunked prefill of a q4_0 pool, first kernel: one CTA per (K/V head,
// sequence) finds the largest K and V scale inside the sequence's context and
// from it the power of two 2^e that the copies are divided by: with
// d < 2^(floor(log2 d) + 1), |c d| < 2^(floor(log2 d) + 4), so e =
// floor(log2 d) - 11 keeps every copied value below 2^15 and the values down
// to 2^-29 of that normal in fp16, whatever the magnitude of K and V.  Reads
// the scales alone (a ninth of the blocks' bytes); latency: table entries, then
// scales, eight of each in flight a thread (one at a time took 20 us for eight
// sequences of up to 8,192 tokens, this 6).
constexpr int kScaleThreads = 512, kScaleAhead = 8;

__global__ void __launch_bounds__(kScaleThreads)
    prefill_scale_q4_kernel(const unsigned char* __restrict__ kc,
                            const unsigned char* __restrict__ vc, StageQ4 g, int n_blocks, int B,
                            int H, int GR) {
  __shared__ uint32_t red[2][kScaleThreads / 32];
  const int h = blockIdx.x, i = blockIdx.y;
  griddep_wait();
  griddep_launch_dependents();
  const int len = g.ctx[i];
  const long long chunk_bytes = static_cast<long long>(B) * GR * 18;
  const int vecs = B * GR / 8;  // 16-byte vectors of a chunk's scales
  int nb = len > 0 ? (len + B - 1) / B : 0;
  if (nb > g.max_blocks) nb = g.max_blocks;
  uint32_t mk = 0, mv = 0;
  const long long total = static_cast<long long>(nb) * vecs;
  // kScaleAhead vectors of K and of V in flight a thread
  const int32_t* row = g.table + static_cast<long long>(i) * g.max_blocks;
  for (long long w0 = threadIdx.x; w0 < total; w0 += kScaleThreads * kScaleAhead) {
    int pid[kScaleAhead], j[kScaleAhead], v[kScaleAhead];
    uint4 xk[kScaleAhead], xv[kScaleAhead];
#pragma unroll
    for (int u = 0; u < kScaleAhead; ++u) {
      const long long w = w0 + static_cast<long long>(u) * kScaleThreads;
      j[u] = static_cast<int>(w / vecs);
      v[u] = static_cast<int>(w - static_cast<long long>(j[u]) * vecs);
      pid[u] = w < total ? row[j[u]] : -1;
    }
#pragma unroll
    for (int u = 0; u < kScaleAhead; ++u) {
      if (pid[u] < 0 || pid[u] >= n_blocks) continue;  // flagged by the copy
      const long long off =
          ((static_cast<long long>(g.layer) * n_blocks + pid[u]) * H + h) * chunk_bytes +
          static_cast<long long>(GR) * B * 16;
      xk[u] = reinterpret_cast<const uint4*>(kc + off)[v[u]];
      xv[u] = reinterpret_cast<const uint4*>(vc + off)[v[u]];
    }
#pragma unroll
    for (int u = 0; u < kScaleAhead; ++u) {
      if (pid[u] < 0 || pid[u] >= n_blocks) continue;
      const uint32_t wk[4] = {xk[u].x, xk[u].y, xk[u].z, xk[u].w};
      const uint32_t wv[4] = {xv[u].x, xv[u].y, xv[u].z, xv[u].w};
      const int rows = len - j[u] * B;  // slots of this block inside the context
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int o = v[u] * 8 + e;
        const uint32_t bk = (wk[e >> 1] >> (16 * (e & 1))) & 0x7fffu;
        const uint32_t bv = (wv[e >> 1] >> (16 * (e & 1))) & 0x7fffu;
        if (o / GR < rows) mk = max(mk, bk);  // K: [B][GR]
        if (o % B < rows) mv = max(mv, bv);   // V: [GR][B]
      }
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    mk = max(mk, __shfl_xor_sync(0xffffffffu, mk, o));
    mv = max(mv, __shfl_xor_sync(0xffffffffu, mv, o));
  }
  if ((threadIdx.x & 31) == 0) {
    red[0][threadIdx.x >> 5] = mk;
    red[1][threadIdx.x >> 5] = mv;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 0; w < kScaleThreads / 32; ++w) {
      mk = max(mk, red[0][w]);
      mv = max(mv, red[1][w]);
    }
    auto pow2 = [](uint32_t bits) {
      const float d = __half2float(__ushort_as_half(static_cast<unsigned short>(bits)));
      const int e = static_cast<int>(__float_as_uint(d) >> 23) - 127;  // floor(log2 d)
      return bits == 0 ? 1.f : __uint_as_float(static_cast<uint32_t>(e - 11 + 127) << 23);
    };
    g.seq_scale[i * H + h] = make_float2(pow2(mk), pow2(mv));
  }
}

// Second kernel: the codes of every block a listed sequence reads become fp16
// values c d / 2^e: d / 2^e as fp16 (exact while normal, so for every scale
// within 2^-25 of the largest) times c, one rounding (2^-11 relative).  Logical
// block j of sequence i goes to copy block i * max_blocks + j; slots past the
// context are zeros.  One CTA per (logical block, sequence); a lane takes one
// word of eight codes, neighbours adjacent ones here and in the copy, four words
// in flight.  Bound by memory: 30,208 tokens of 8 heads, 35 MB in and 124 MB
// out, take 35 us, 4.6 TB/s (a group a lane, whose 64 bytes wrote half sectors:
// 42 us).  A pair of nibbles becomes c without a conversion: n beside the
// exponent of 1024, less 1032.
constexpr int kStageThreads = 256, kStageAhead = 4;

__global__ void __launch_bounds__(kStageThreads)
    prefill_stage_q4_kernel(const unsigned char* __restrict__ kc,
                            const unsigned char* __restrict__ vc, StageQ4 g, int n_blocks, int B,
                            int H, int GR, int32_t* status) {
  const int j = blockIdx.x, i = blockIdx.y;
  const long long sb = static_cast<long long>(i) * g.max_blocks + j;
  griddep_wait();
  griddep_launch_dependents();
  if (threadIdx.x == 0) g.stage_table[sb] = static_cast<int32_t>(sb);
  const int len = g.ctx[i];
  if (len <= 0 || j >= (len + B - 1) / B) return;
  const int pid = g.table[sb];
  const bool ok = pid >= 0 && pid < n_blocks;
  if (!ok && threadIdx.x == 0) record_status(status, KV_DEV_BAD_BLOCK_ID);
  const int rows = len - j * B < B ? len - j * B : B;
  const long long chunk_bytes = static_cast<long long>(B) * GR * 18;
  const long long blk = (static_cast<long long>(g.layer) * n_blocks + (ok ? pid : 0)) * H;
  const int lgr = GR == 4 ? 2 : 1;
  const int n = B * H << (lgr + 2);  // words (8 codes, 16 bytes out) of one of K, V
  const __half2 off = __float2half2_rn(1032.f);
  for (int base = threadIdx.x; base < 2 * n; base += kStageAhead * kStageThreads) {
    uint32_t w[kStageAhead];
    __half sc[kStageAhead];
    float2 e[kStageAhead];
#pragma unroll
    for (int u = 0; u < kStageAhead; ++u) {
      const int idx = base + u * kStageThreads;
      const bool is_k = idx < n;
      const int x = is_k ? idx : idx - n;
      const unsigned t = static_cast<unsigned>(x) >> (lgr + 2);  // head of a slot
      const int q = (x >> 2) & (GR - 1), o = t / static_cast<unsigned>(H), h = t - o * H;
      w[u] = 0x88888888u;  // zeros
      sc[u] = __half();
      e[u] = make_float2(1.f, 1.f);
      if (idx < 2 * n && ok && o < rows) {
        const unsigned char* chunk = (is_k ? kc : vc) + (blk + h) * chunk_bytes;
        w[u] = reinterpret_cast<const uint32_t*>(chunk + (q * B + o) * 16)[x & 3];
        sc[u] = reinterpret_cast<const __half*>(chunk + GR * B * 16)[is_k ? o * GR + q : q * B + o];
        e[u] = g.seq_scale[i * H + h];
      }
    }
#pragma unroll
    for (int u = 0; u < kStageAhead; ++u) {
      const int idx = base + u * kStageThreads;
      if (idx >= 2 * n) break;
      const bool is_k = idx < n;
      const int x = is_k ? idx : idx - n;
      // 1 / 2^e from the exponent's bits
      const float inv = __uint_as_float(0x7f000000u - __float_as_uint(is_k ? e[u].x : e[u].y));
      const __half2 d = __float2half2_rn(__half2float(sc[u]) * inv);
      const uint32_t hi = w[u] >> 4;
      uint32_t h2[4];
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        // byte b's low nibble in the low half, its high nibble in the upper
        const uint32_t n2 = (__byte_perm(w[u], hi, b | (b + 4) << 8) & 0x000f000fu) | 0x64006400u;
        const __half2 p = __hmul2(__hsub2(*reinterpret_cast<const __half2*>(&n2), off), d);
        h2[b] = *reinterpret_cast<const uint32_t*>(&p);
      }
      // words of a (slot, head) are its row's 16-byte vectors in order
      (static_cast<uint4*>(is_k ? g.k_stage : g.v_stage) + sb * n)[x] =
          make_uint4(h2[0], h2[1], h2[2], h2[3]);
    }
  }
}

}  // namespace

cudaError_t launch_prefill_stage_q4(const kvPool* p, const StageQ4& g, cudaStream_t st) {
  const unsigned char* kc = static_cast<const unsigned char*>(p->k);
  const unsigned char* vc = static_cast<const unsigned char*>(p->v);
  const cudaError_t e =
      launch_kernel(p->pdl, prefill_scale_q4_kernel, dim3(p->H, g.n_seq), dim3(kScaleThreads), 0,
                    st, kc, vc, g, p->N, p->B, p->H, p->D / 32);
  if (e != cudaSuccess) return e;
  return launch_kernel(p->pdl, prefill_stage_q4_kernel, dim3(g.max_blocks, g.n_seq),
                       dim3(kStageThreads), 0, st, kc, vc, g, p->N, p->B, p->H, p->D / 32,
                       p->d_status);
}

cudaError_t launch_slot_write_q4(const kvPool* p, int layer, const void* k_new, const void* v_new,
                                 const int64_t* slots, int n_tokens, cudaStream_t st) {
  const int lanes = 2 * p->H * p->D / 8;
  const int threads = lanes >= 256 ? 256 : (lanes + 31) / 32 * 32;
  const int per_cta = tokens_per_cta(p, n_tokens, layer, kWriteTokens);
  const dim3 grid((n_tokens + per_cta - 1) / per_cta, layer >= 0 ? 1 : p->L);
  return launch_kernel(p->pdl, slot_write_q4_kernel, grid, dim3(threads), 0, st,
                       static_cast<const uint4*>(k_new), static_cast<const uint4*>(v_new), slots,
                       n_tokens, per_cta, static_cast<unsigned char*>(p->k),
                       static_cast<unsigned char*>(p->v), layer, p->N, p->B, p->H, p->D / 32,
                       p->d_status);
}

cudaError_t launch_gather_rows(const kvPool* p, int layer, const int64_t* slots, int n_tokens,
                               void* k_out, void* v_out, int out_dtype, cudaStream_t st) {
  switch (p->dtype) {
    case KV_DTYPE_F32:
      return launch_gather<KV_DTYPE_F32>(p, layer, slots, n_tokens, k_out, v_out, out_dtype, st);
    case KV_DTYPE_BF16:
      return launch_gather<KV_DTYPE_BF16>(p, layer, slots, n_tokens, k_out, v_out, out_dtype, st);
    case KV_DTYPE_FP8_E4M3:
      return launch_gather<KV_DTYPE_FP8_E4M3>(p, layer, slots, n_tokens, k_out, v_out, out_dtype,
                                              st);
    case KV_DTYPE_Q8_0:
      return launch_gather<KV_DTYPE_Q8_0>(p, layer, slots, n_tokens, k_out, v_out, out_dtype, st);
    default:
      return launch_gather<KV_DTYPE_Q4_0>(p, layer, slots, n_tokens, k_out, v_out, out_dtype, st);
  }
}

}  // namespace pkv
