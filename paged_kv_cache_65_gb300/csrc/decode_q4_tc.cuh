// Split-K paged decode attention, partial pass, over a q4_0 pool on the
// fifth-generation tensor cores (tcgen05), D_h = 128.
//
// Same contract, work split, pieces and workspace as decode_mma.cuh.  Per
// stage of 128 token rows of one K/V head:
//     S^T [128 tokens x N] = K' [128 x 128] . Q^T [128 x N]        (8 MMAs, K = 16)
//     O^T [128 dims  x N] += V'^T [128 x 128] . P'^T [128 x N]      (8 MMAs)
// N = 16 for pieces of up to 16 query columns, 32 otherwise.  The MMAs cost
// the warps no issue slots, whatever N is, so a segment shared by four
// branches of eight query heads each costs little more than one of eight
// columns; what remains is turning nibbles into operands, once per stage.
//
// Operands.  A token row's stored values are (n - 8) d_q, n the nibble and d_q
// the scale of group q.  Let 2^E be the power of two below the row's largest
// scale (1 <= d_max / 2^E < 2).  Rows are converted to fp16 as
//     (n - 8) (d_q / 2^E) 2^-10,
// one AND and one fused multiply-add a pair: the bit pattern n of an fp16 is
// the subnormal n 2^-24 (n << 4: n 2^-20), and with A = d_q 2^(14-E) (2^(10-E))
// and B = -d_q 2^(-7-E), both exact, fma(n 2^-24, A, B) is that value rounded
// once (2^-11 relative; a group whose scale is below d_max / 16 loses bits
// below 2^-15 d_max).  The row's 2^E joins the score scale of its row (K) and
// the weight of its token (V).  Four words of eight nibbles come unpacked in
// the order 0 4 1 5 2 6 3 7 of each eight dimensions; Q is staged in the same
// order, and O's rows are written back through it.
//
// Q of a piece is scaled by the power of two that brings its largest |q| into
// [2^14, 2^15) and turned into fp16: bf16's 8 bits stay exact over 2^21 of
// range.  P' = p 2^(E - e) in fp16: p <= 2^8 by the lazy reference m (moved
// when a score passes it by more than 2^8), and e, a running reference of V's
// exponents, is moved when a row's E passes it by more than 4, both with a
// rescale of O^T; p is one rounding to 11 bits.
//
// Warps (one CTA of 20 per SM): 0-3 and 4-7 softmax, each group half of the
// columns (thread r owns token row r of a stage and, at a piece's end, row r of
// O^T; a column's references are its group's own, so the groups never meet);
// 8-11 turn K rows into fp16 in tensor memory, 12-15 V rows into fp16 in shared
// memory (M-major, 128-byte swizzle); 16 copies the codes (a whole block of one
// head is one bulk copy), 17 stages Q, 18 issues the S MMAs, 19 the P.V MMAs.  The codes' ring is
// free again as soon as they are converted, so its five stages (92 KB) are
// all in flight while the converted stages (three of K, two of V and P) are
// worked on.
//
// Every mbarrier wait is bounded, as in decode_tc.cuh; a role that gave up
// runs the rest of its loops without waiting or issuing.
#pragma once

#include "decode_q4.cuh"
#include "decode_tc.cuh"

namespace pkv {

struct Q4Tc {
  static constexpr int D = 128;
  static constexpr int TS = 128;                // tokens per stage
  static constexpr int ROW = D / 2 + D / 16;    // bytes of a token row of codes and scales
  static constexpr int CODES = TS * ROW;        // K (or V) codes of a stage
  static constexpr int NC = 5;                  // stages of codes in the ring
  static constexpr int NK = 3;                  // converted K stages (tensor memory)
  static constexpr int NV = 2;                  // converted V stages (shared memory)
  static constexpr int NP = 4;                  // stages of weights
  static constexpr int NKP = 8;                 // rows' powers: the converters may be NK + 2 ahead
  static constexpr int HALF = TS * 128;         // 64 dimensions of a converted V stage
  static constexpr int VBUF = 2 * HALF;
  static constexpr int PBUF = TS * 64;          // 32 columns a token
  static constexpr int QHALF = 32 * 128;
  static constexpr int QTILE = 2 * QHALF;
  static constexpr int QBUF = 2;
  static constexpr int TM_S = 0;                // S^T buffers at columns 0 and 32
  static constexpr int TM_O = 64;
  static constexpr int TM_K = 128;              // 64 columns a stage
  static constexpr int TM_COLS = 512;
  static constexpr float TAU = 8.f;             // base-2 headroom of the scores' reference
  static constexpr int ETAU = 4;                // and of V's exponents
  static constexpr int WARPS = 20;
  static constexpr int NBARS = 2 * NC + 2 * NK + NV + 4 + 2 * NP + 2 * QBUF + 2;
};
static_assert(Q4Tc::TM_K + Q4Tc::NK * 64 <= Q4Tc::TM_COLS, "TMEM columns");
constexpr int kQ4TcThreads = Q4Tc::WARPS * 32;
// registers a thread per warpgroup (two softmax, K and V converters, helpers)
// against the 96 that 20 warps are launched with (the launcher checks it)
constexpr int kQ4TcRegsLaunch = 96;
constexpr int kQ4TcRegsSoftmax = 120, kQ4TcRegsCvt = 96, kQ4TcRegsHelper = 48;
static_assert(2 * kQ4TcRegsSoftmax + 2 * kQ4TcRegsCvt + kQ4TcRegsHelper <= 5 * kQ4TcRegsLaunch,
              "register split");

constexpr int decode_q4_tc_smem_bytes() {
  using C = Q4Tc;
  return C::NV * C::VBUF + C::NP * C::PBUF + C::QBUF * C::QTILE  // 1 KiB aligned operands
         + 2 * C::NC * C::CODES                            // codes
         + 2 * C::NKP * C::TS * 4                            // rows' powers of two: K, V
         + 2 * 4 * 128 * 4                                 // per softmax group: maxima, sums
         + 64                                              // Q factors, exponent maxima
         + C::NBARS * 8 + 4 * 8 + 16                       // mbarriers, walk state, TMEM address
         + kTableCache * 4 + 128                           // table cache, start record
         + 1024;                                           // alignment
}

// Dimension of converted element i (rows of O^T, k-slots of K and Q).
__device__ __forceinline__ int q4_dim(int i) {
  return (i & ~7) | ((i >> 1) & 3) | ((i & 1) << 2);
}

// 2^e as a float, -126 <= e <= 127
__device__ __forceinline__ float q4_pow2(int e) {
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

__device__ __forceinline__ float q4_max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// E of a row with these scales (fp16 bits): floor(log2) of the largest, -24 for
// zeros.
__device__ __forceinline__ int q4_row_exp(const uint32_t (&sc)[2]) {
  const float mx = fmaxf(fmaxf(half_lo(sc[0]), half_hi(sc[0])), fmaxf(half_lo(sc[1]), half_hi(sc[1])));
  const int E = static_cast<int>(__float_as_uint(mx) >> 23) - 127;
  return E < -24 ? -24 : E;
}

// Multipliers of one token row from its four scales (fp16 bits): E, and per
// pair of groups A = d 2^(14-E).  live = false: all zero, so that whatever the
// row holds becomes zeros.
__device__ __forceinline__ int q4_row_scales(const uint32_t (&sc)[2], bool live, __half2 (&A)[2]) {
  float d[4];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    d[2 * i] = half_lo(sc[i]);
    d[2 * i + 1] = half_hi(sc[i]);
  }
  const int E = q4_row_exp(sc);
  const float f = live ? q4_pow2(14 - E) : 0.f;
#pragma unroll
  for (int i = 0; i < 2; ++i)
    A[i] = live ? __floats2half2_rn(d[2 * i] * f, d[2 * i + 1] * f) : __half2(__ushort_as_half(0), __ushort_as_half(0));
  return E;
}

// The words of one group (16 bytes) to 32 fp16 values.
__device__ __forceinline__ void q4_convert(const uint32_t (&w)[4], __half2 a_lo, uint32_t* h) {
  const __half2 a_hi = __hmul2(a_lo, __half2(__ushort_as_half(0x2c00), __ushort_as_half(0x2c00)));   // 2^-4
  const __half2 b = __hmul2(a_lo, __half2(__ushort_as_half(0x8008), __ushort_as_half(0x8008)));      // -2^-21
  auto cv = [&](uint32_t x, __half2 m) -> uint32_t {
    const __half2 r = __hfma2(*reinterpret_cast<const __half2*>(&x), m, b);
    return *reinterpret_cast<const uint32_t*>(&r);
  };
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t x = w[i], x8 = w[i] >> 8;
    h[4 * i] = cv(x & kNibLo, a_lo);
    h[4 * i + 1] = cv(x & kNibHi, a_hi);
    h[4 * i + 2] = cv(x8 & kNibLo, a_lo);
    h[4 * i + 3] = cv(x8 & kNibHi, a_hi);
  }
}

// 16 columns of tensor memory, without the wait for it
__device__ __forceinline__ void tmem_st16_nowait(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
      "%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// State of the softmax warps for one CTA.
struct Q4TcSoftmax {
  const DecodeArgs* a;
  unsigned char* p_st;
  const float* k_pow;   // [NKP][128] 2^(E + 10) of the K rows
  const float* v_exp;   // [NKP][128] E of the V rows
  const float* q_fac;   // [QBUF] score factor of the piece
  float *red, *cmx, *lsum;
  float* emx;           // [4] exponent maxima per warp
  uint64_t *s_full, *s_empty, *p_full, *pv_done, *o_free, *q_full, *q_empty;
  uint32_t tmem;
  int cstride;
  int grp;              // softmax group: warps 4 grp .. 4 grp + 3
  bool alive;
  int stage, npiece;

  // Lane 0 of the warp waits, the others follow it: fewer polls in the way of
  // the warps that work.
  __device__ void wait(uint64_t* bar, uint32_t parity) {
    bool ok = alive;
    if (ok && (threadIdx.x & 31) == 0 && !q4_wait(bar, parity)) {
      ok = false;
      record_status(a->status, 8);
    }
    alive = __all_sync(0xffffffffu, ok);
  }

  // A piece without columns for this group: it keeps its place in the stages.
  __device__ void idle(int n_st) {
    using C = Q4Tc;
    const bool first = (threadIdx.x & 31) == 0;
    wait(&q_full[npiece % C::QBUF], (npiece / C::QBUF) & 1);
    if (first) mbar_arrive(&q_empty[npiece % C::QBUF]);
    for (int i = 0; i < n_st; ++i, ++stage) {
      wait(&s_full[stage & 1], (stage >> 1) & 1);
      if (first) {
        mbar_arrive(&s_empty[stage & 1]);
        mbar_arrive(&p_full[stage % C::NP]);
      }
    }
    // O^T is given back only after the piece's last MMAs, so that this group
    // never stands in for the other one at a later piece
    wait(&pv_done[(stage - 1) % C::NP], ((stage - 1) / C::NP) & 1);
    if (first) mbar_arrive(o_free);
    ++npiece;
  }

  // Columns c_first .. c_first + NCP - 1 of one piece.
  template <int NCP>
  __device__ void run(const Piece& p, int n_st, int tok_first, int c_first) {
    using C = Q4Tc;
    const int t = threadIdx.x & 127;  // token row of a stage / row of O^T
    const int warp = t >> 5, lane = t & 31;
    const int bar = 1 + grp;
    const uint32_t tl = (static_cast<uint32_t>(warp * 32) << 16) + c_first;
    const int ncols = min(p.ncols - c_first, NCP);
    float m_ref[NCP], l_part[NCP];
#pragma unroll
    for (int c = 0; c < NCP; ++c) {
      m_ref[c] = -INFINITY;
      l_part[c] = 0.f;
    }
    float e_ref = -1000.f;  // no V row seen
    wait(&q_full[npiece % C::QBUF], (npiece / C::QBUF) & 1);
    __syncwarp();
    const float qs = q_fac[npiece % C::QBUF];
    __syncwarp();
    if (lane == 0) mbar_arrive(&q_empty[npiece % C::QBUF]);
    for (int i = 0; i < n_st; ++i, ++stage) {
      const int nvalid = min(p.tok_end - (tok_first + i * C::TS), C::TS);
      const bool valid = t < nvalid;
      wait(&s_full[stage & 1], (stage >> 1) & 1);
      __syncwarp();
      tc_fence_after();
      uint32_t sr[NCP];
      tmem_ld<NCP>(tmem + C::TM_S + (stage & 1) * 32 + tl, sr);
      const float kf = qs * k_pow[(stage % C::NKP) * C::TS + t];
      const float ve = v_exp[(stage % C::NKP) * C::TS + t];
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s_empty[stage & 1]);
      float x[NCP], top = -INFINITY;
#pragma unroll
      for (int c = 0; c < NCP; ++c) x[c] = fmaf(__uint_as_float(sr[c]), kf, -m_ref[c]);
#pragma unroll
      for (int c = 0; c < NCP; c += 2) top = q4_max3(top, x[c], x[c + 1]);
      if (bar_or_sync(bar, 128, valid && (top > C::TAU || ve > e_ref + C::ETAU))) {
        // ---- a reference moves: exact column maxima (and the largest V
        // exponent) of this stage
        float v[NCP];
#pragma unroll
        for (int c = 0; c < NCP; ++c) v[c] = valid ? __uint_as_float(sr[c]) * kf : -INFINITY;
        const float wm = warp_column_reduce<NCP, true>(v);
        if (lane < NCP) red[warp * 32 + lane] = wm;
        float em = valid ? ve : -1000.f;
#pragma unroll
        for (int off = 16; off; off >>= 1) em = fmaxf(em, __shfl_xor_sync(0xffffffffu, em, off));
        if (lane == 0) emx[warp] = em;
        named_bar_sync(bar, 128);
        float cm = -INFINITY;
        if (lane < NCP) {
#pragma unroll
          for (int w = 0; w < 4; ++w) cm = fmaxf(cm, red[w * 32 + lane]);
        }
        cmx[warp * 32 + lane] = cm;
        const float e_new = fmaxf(e_ref, fmaxf(fmaxf(emx[0], emx[1]), fmaxf(emx[2], emx[3])));
        const float ef = exp2_approx(e_ref - e_new);  // exact: integers (0 at the first move)
        e_ref = e_new;
        __syncwarp();
        float al[NCP];
#pragma unroll
        for (int c = 0; c < NCP; ++c) {
          const float mn = fmaxf(m_ref[c], cmx[warp * 32 + c]);
          al[c] = exp2_approx(m_ref[c] - mn);
          m_ref[c] = mn;
          l_part[c] *= al[c];
          x[c] = fmaf(__uint_as_float(sr[c]), kf, -mn);
        }
        if (i > 0) {
          // rescale O^T once the previous stage's MMAs are done with it
          wait(&pv_done[(stage - 1) % C::NP], ((stage - 1) / C::NP) & 1);
          __syncwarp();
          tc_fence_after();
          uint32_t o[NCP];
          tmem_ld<NCP>(tmem + C::TM_O + tl, o);
#pragma unroll
          for (int c = 0; c < NCP; ++c)
            o[c] = __float_as_uint(__uint_as_float(o[c]) * (al[c] * ef));
          tmem_st<NCP>(tmem + C::TM_O + tl, o);
        }
      }
      // ---- weights: row t of P' (N-major, 64-byte swizzle: 16-byte chunk c at
      // c ^ (t / 2 mod 4)), into the buffer that the MMAs of four stages before
      // have read
      if (stage >= C::NP) wait(&pv_done[stage % C::NP], ((stage / C::NP) - 1) & 1);
      // a power of two; 0 for a row past the context, whose exponent may be any
      const __half2 pe = __float2half2_rn(valid ? exp2_approx(ve - e_ref) : 0.f);
      const uint32_t pb = smem_u32(p_st + (stage % C::NP) * C::PBUF) + t * 64;
#pragma unroll
      for (int c8 = 0; c8 < NCP / 8; ++c8) {
        uint32_t hi[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int c = c8 * 8 + 2 * k;
          const float p0 = valid ? exp2_approx(x[c]) : 0.f;
          const float p1 = valid ? exp2_approx(x[c + 1]) : 0.f;
          l_part[c] += p0;
          l_part[c + 1] += p1;
          const __half2 ph = __hmul2(__floats2half2_rn(p0, p1), pe);
          hi[k] = *reinterpret_cast<const uint32_t*>(&ph);
        }
        sts128(pb + (((c_first / 8 + c8) ^ ((t >> 1) & 3)) << 4), hi[0], hi[1], hi[2], hi[3]);
      }
      fence_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[stage % C::NP]);
    }

    // ---- end of the piece: O^T from TMEM once the last stage's MMAs are
    // done, l reduced over the 128 rows
    wait(&pv_done[(stage - 1) % C::NP], ((stage - 1) / C::NP) & 1);
    __syncwarp();
    tc_fence_after();
    const long long slot_id = (long long)blockIdx.x + p.seg;
    const float of = exp2_approx(e_ref + 10.f);
    float* dst = a->ws_o + (slot_id * cstride + c_first) * C::D + q4_dim(t);
#pragma unroll
    for (int c0 = 0; c0 < NCP; c0 += 8) {
      uint32_t o[8];
      tmem_ld8(tmem + C::TM_O + c0 + tl, o);
#pragma unroll
      for (int c = 0; c < 8; ++c)
        if (c0 + c < ncols) dst[(c0 + c) * C::D] = __uint_as_float(o[c]) * of;
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(o_free);
    const float ls = warp_column_reduce<NCP, false>(l_part);
    if (lane < NCP) lsum[warp * 32 + lane] = ls;
    named_bar_sync(bar, 128);
    if (warp == 0 && lane < ncols) {
      float mc = m_ref[0];
#pragma unroll
      for (int c = 1; c < NCP; ++c) mc = lane == c ? m_ref[c] : mc;
      float L = 0.f;
#pragma unroll
      for (int w = 0; w < 4; ++w) L += lsum[w * 32 + lane];
      a->ws_ml[(slot_id * cstride + c_first + lane) * 2] = mc;
      a->ws_ml[(slot_id * cstride + c_first + lane) * 2 + 1] = L;
    }
    ++npiece;
  }
};

template <bool PLAN>
__global__ void __launch_bounds__(kQ4TcThreads, 1) decode_q4_tc_kernel(const DecodeArgs a) {
  using C = Q4Tc;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  unsigned char* v_st = smem;
  unsigned char* p_st = v_st + C::NV * C::VBUF;
  unsigned char* q_s = p_st + C::NP * C::PBUF;
  unsigned char* k_code = q_s + C::QBUF * C::QTILE;
  unsigned char* v_code = k_code + C::NC * C::CODES;
  float* k_pow = reinterpret_cast<float*>(v_code + C::NC * C::CODES);
  float* v_exp = k_pow + C::NKP * C::TS;
  float* red = v_exp + C::NKP * C::TS;
  float* cmx = red + 2 * 128;  // these three [group][4][32]
  float* lsum = cmx + 2 * 128;
  float* q_fac = lsum + 4 * 128;  // [QBUF]
  float* emx = q_fac + 8;         // [group][4]
  uint64_t* full = reinterpret_cast<uint64_t*>(emx + 8);  // [NC] codes in
  uint64_t* empty = full + C::NC;                         // [NC] codes converted
  uint64_t* k_full = empty + C::NC;                       // [NK] K rows in TMEM
  uint64_t* k_empty = k_full + C::NK;                     // [NK] S MMAs done
  uint64_t* v_full = k_empty + C::NK;                     // [NV] V rows converted
  uint64_t* pv_done = v_full + C::NV;                     // [NP] P.V MMAs done
  uint64_t* s_full = pv_done + C::NP;                     // [2]
  uint64_t* s_empty = s_full + 2;                         // [2]
  uint64_t* p_full = s_empty + 2;                         // [NP]
  uint64_t* q_full = p_full + C::NP;                      // [QBUF]
  uint64_t* q_empty = q_full + C::QBUF;                   // [QBUF]
  uint64_t* o_free = q_empty + C::QBUF;
  uint64_t* fin = o_free + 1;
  long long* walk = reinterpret_cast<long long*>(full + C::NBARS);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(walk + 4);
  int32_t* tcache = reinterpret_cast<int32_t*>(tmem_slot + 4);
  PlanStart* rec_s = reinterpret_cast<PlanStart*>(tcache + kTableCache);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int B = a.block_size;
  const int H = a.n_kv_heads;
  const int G = a.n_q_heads / H;
  const int UR = q4_unit_rows(B);  // tokens per copied unit
  const int lur = 31 - __clz(UR);
  const int KU = B / UR;           // units per block
  const uint32_t unit_bytes = static_cast<uint32_t>(UR) * C::ROW;

  // self-check: swizzled buffers must sit on 1 KiB boundaries
  if ((smem_u32(v_st) & 1023u) != 0u) {
    if (threadIdx.x == 0) record_status(a.status, 32);
    return;
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::NC; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 8);  // K and V converter warps
    }
    for (int i = 0; i < C::NK; ++i) {
      mbar_init(&k_full[i], 4);
      mbar_init(&k_empty[i], 1);
    }
    for (int i = 0; i < C::NV; ++i) mbar_init(&v_full[i], 4);
    for (int i = 0; i < C::NP; ++i) {
      mbar_init(&pv_done[i], 1);
      mbar_init(&p_full[i], 8);  // softmax warps
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], 8);
    }
    for (int i = 0; i < C::QBUF; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 9);  // the S MMAs done, the factor read by eight warps
    }
    mbar_init(o_free, 8);
    mbar_init(fin, 2);
    fence_barrier_init();
  }
  if (warp == 0) {
    tmem_alloc(tmem_slot, C::TM_COLS);
    tmem_relinquish();
  }
  // tables and lengths that kernels before this one write are read only after
  // them (decode_q4.cuh)
  if (a.meta_wait) griddep_wait();
  const bool use_rec = PLAN && a.starts != nullptr && a.start_grid == a.grid;
  if (warp == 16) {
    if constexpr (PLAN) {
      const long long W = a.plan_W;
      long long chunk = (W + a.grid - 1) / a.grid;
      if (chunk == 0) chunk = 1;
      int s0 = 0;
      if (use_rec) {
        reinterpret_cast<int32_t*>(rec_s)[lane] =
            reinterpret_cast<const int32_t*>(a.starts + blockIdx.x)[lane];
      } else {
        const long long r0 = (long long)blockIdx.x * chunk;
        s0 = r0 < W ? plan_find(a.segs, a.n_segs, r0) : a.n_segs;
      }
      if (lane == 0) {
        walk[0] = s0;
        walk[1] = 0;
        walk[2] = W;
        walk[3] = chunk;
      }
    } else {
      WalkStart w = find_start(a.ctx, a.n_seq, B, H, a.max_blocks, a.grid, blockIdx.x, a.status);
      if (lane == 0) {
        walk[0] = w.s;
        walk[1] = w.pre;
        walk[2] = w.W;
        walk[3] = w.chunk;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  const long long W = walk[2], chunk = walk[3];
  const long long r_begin = (long long)blockIdx.x * chunk;
  const long long r_end = r_begin + chunk < W ? r_begin + chunk : W;
  PieceWalker pw;
  PlanWalker plw;
  if constexpr (PLAN) {
    plw.segs = a.segs;
    plw.n_segs = a.n_segs;
    plw.B = B;
    plw.s = (int)walk[0];
    plw.r = r_begin;
    plw.r1 = r_end;
  } else {
    pw.ctx = a.ctx;
    pw.n_seq = a.n_seq;
    pw.B = B;
    pw.H = H;
    pw.max_blocks = a.max_blocks;
    pw.s = (int)walk[0];
    pw.pre = walk[1];
    pw.r = r_begin;
    pw.r1 = r_end;
  }
  bool rec_first = use_rec;  // the first piece comes from the start record
  auto next_piece = [&](Piece& p) -> bool {
    if constexpr (PLAN) {
      if (rec_first) {
        rec_first = false;
        const PlanStart& R = *rec_s;
        if (R.seg < 0) {
          plw.s = plw.n_segs;
          return false;
        }
        p.rep = R.rep;
        p.head = R.head;
        p.b0 = R.b0;
        p.b1 = R.b1;
        p.tok_end = R.tok_end;
        p.ncols = R.ncols;
        p.mem = R.mem;
        p.seg = R.seg;
        p.last = R.last;
        plw.s = R.seg;
        plw.r = R.r_after;
        return true;
      }
      return plw.next(p);
    } else {
      if (!pw.next()) return false;
      p.rep = pw.seq;
      p.head = pw.head;
      p.b0 = pw.b0;
      p.b1 = pw.b1;
      p.tok_end = pw.b1 * B < pw.ctx_len ? pw.b1 * B : pw.ctx_len;
      p.ncols = G;
      p.mem = -1;
      p.seg = pw.seq * H + pw.head;
      p.last = 0;
      return true;
    }
  };
  auto wait_previous_grid = [&]() {
    griddep_wait();
    griddep_launch_dependents();
    if constexpr (!PLAN) {
      if (blockIdx.x == 0 && warp == 16)
        write_prefix(a.ctx, a.n_seq, B, H, a.max_blocks, a.ws_pre);
    }
  };
  auto stages_of = [&](const Piece& p) -> int {
    const int n = p.tok_end - p.b0 * B;
    return n > 0 ? (n + C::TS - 1) / C::TS : 0;
  };
  bool alive = true;
  // whole warps: lane 0 waits, the others follow it
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    bool ok = alive;
    if (ok && lane == 0 && !q4_wait(bar, parity)) {
      ok = false;
      record_status(a.status, 8);
    }
    alive = __all_sync(0xffffffffu, ok);
  };

  if (warp < 8) {
    // ------------------------------------------------------ softmax warps
    reg_alloc<kQ4TcRegsSoftmax>();
    wait_previous_grid();
    Q4TcSoftmax sm;
    sm.a = &a;
    sm.p_st = p_st;
    sm.k_pow = k_pow;
    sm.v_exp = v_exp;
    sm.q_fac = q_fac;
    sm.grp = warp >> 2;
    sm.red = red + sm.grp * 128;
    sm.cmx = cmx + sm.grp * 128;
    sm.lsum = lsum + sm.grp * 128;
    sm.emx = emx + sm.grp * 4;
    sm.s_full = s_full;
    sm.s_empty = s_empty;
    sm.p_full = p_full;
    sm.pv_done = pv_done;
    sm.o_free = o_free;
    sm.q_full = q_full;
    sm.q_empty = q_empty;
    sm.tmem = tmem;
    sm.cstride = PLAN ? a.c_max : G;
    sm.alive = true;
    sm.stage = 0;
    sm.npiece = 0;
    Piece p;
    while (next_piece(p)) {
      const int n_st = stages_of(p);
      if (n_st == 0) {
        // no block of this piece: an empty partial that the merge skips
        const long long slot_id = (long long)blockIdx.x + p.seg;
        if (sm.grp == 0) {
          for (int c = 0; c < p.ncols; ++c)
            a.ws_o[(slot_id * sm.cstride + c) * C::D + threadIdx.x] = 0.f;
          if (threadIdx.x < p.ncols) {
            a.ws_ml[(slot_id * sm.cstride + threadIdx.x) * 2] = -INFINITY;
            a.ws_ml[(slot_id * sm.cstride + threadIdx.x) * 2 + 1] = 0.f;
          }
        }
        continue;
      }
      // the columns in two halves; up to eight are one group's
      const int half = p.ncols <= 16 ? 8 : 16, c_first = sm.grp * half;
      if (c_first >= p.ncols)
        sm.idle(n_st);
      else if (half == 8)
        sm.template run<8>(p, n_st, p.b0 * B, c_first);
      else
        sm.template run<16>(p, n_st, p.b0 * B, c_first);
    }
  } else if (warp < 16) {
    // ------------------------------------------ converters (K 8-11, V 12-15)
    wait_previous_grid();
    const bool kp = warp < 12;
    const int r = threadIdx.x & 127;  // token row of a stage
    const uint32_t tl = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const int ro = r & (UR - 1);
    const uint32_t unit = (r >> lur) * unit_bytes;
    const uint32_t code_off = smem_u32(kp ? k_code : v_code) + unit + ro * 16;
    const uint32_t ks_off = smem_u32(k_code) + unit + UR * 64 + ro * 8;
    const uint32_t vs_off = smem_u32(v_code) + unit + UR * 64 + ro * 2;
    // 16-byte chunk ch of a converted V row at ch ^ (r mod 8) in its half
    const uint32_t v_row = smem_u32(v_st) + r * 128 + ((r & 7) << 4);
    int stage = 0, slot = 0;
    uint32_t slot_par = 0;
    Piece p;
    while (next_piece(p)) {
      for (int left = p.tok_end - p.b0 * B; left > 0; left -= C::TS, ++stage) {
        wait(&full[slot], slot_par);
        const uint32_t sb = slot * C::CODES;
        const bool live = r < left;
        // V's scales of the row (both kinds of warps: the K warps, which run
        // ahead, publish the exponents the softmax needs)
        uint32_t vsc[2];
        {
          uint16_t s4[4];
#pragma unroll
          for (int q = 0; q < 4; ++q)
            asm volatile("ld.shared.u16 %0, [%1];" : "=h"(s4[q]) : "r"(vs_off + sb + q * UR * 2));
          vsc[0] = s4[0] | (static_cast<uint32_t>(s4[1]) << 16);
          vsc[1] = s4[2] | (static_cast<uint32_t>(s4[3]) << 16);
        }
        __half2 A[2];
        if (kp) {
          uint32_t ksc[2];
          lds_scales<4>(ks_off + sb, ksc);
          k_pow[(stage % C::NKP) * C::TS + r] = q4_pow2(q4_row_scales(ksc, live, A) + 10);
          v_exp[(stage % C::NKP) * C::TS + r] = static_cast<float>(q4_row_exp(vsc));
          if (stage >= C::NK) wait(&k_empty[stage % C::NK], ((stage / C::NK) - 1) & 1);
        } else {
          q4_row_scales(vsc, live, A);
          if (stage >= C::NV)
            wait(&pv_done[(stage - C::NV) % C::NP], ((stage - C::NV) / C::NP) & 1);
        }
        if (!alive) continue;
        tc_fence_after();
        // one group at a time, the loop not unrolled: five kinds of warps share
        // an SM sub-partition's instruction fetch, and short loops stay in it
        const uint32_t out = kp ? tmem + tl + C::TM_K + (stage % C::NK) * 64
                                : v_row + (stage % C::NV) * C::VBUF;
        uint32_t a01 = *reinterpret_cast<const uint32_t*>(&A[0]);
        uint32_t a23 = *reinterpret_cast<const uint32_t*>(&A[1]);
#pragma unroll 1
        for (int q = 0; q < 4; ++q) {
          uint32_t w[4], h[16];
          lds128(code_off + sb + q * UR * 16, w[0], w[1], w[2], w[3]);
          const uint32_t aa = __byte_perm(a01, a01, 0x1010);
          a01 = __byte_perm(a01, a23, 0x5432);  // the next group's scale
          a23 >>= 16;
          q4_convert(w, *reinterpret_cast<const __half2*>(&aa), h);
          if (kp) {
            tmem_st16_nowait(out + q * 16, h);
          } else {
            // chunks 4 q .. 4 q + 3 of the row: half q / 2
#pragma unroll
            for (int k = 0; k < 4; ++k)
              sts128((out + (q >> 1) * C::HALF) ^ ((4 * (q & 1) + k) << 4), h[4 * k], h[4 * k + 1],
                     h[4 * k + 2], h[4 * k + 3]);
          }
        }
        // the codes have been read: their stage may be copied over
        if (kp) {
          tmem_wait_st();
          tc_fence_before();
        } else {
          fence_async_smem();
        }
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&empty[slot]);
          mbar_arrive(kp ? &k_full[stage % C::NK] : &v_full[stage % C::NV]);
        }
        if (++slot == C::NC) {
          slot = 0;
          slot_par ^= 1;
        }
      }
    }
  } else {
    reg_dealloc<kQ4TcRegsHelper>();
    if (warp == 16) {
      // --------------------------------------------------------- code copies
      TableCache tc;
      tc.ent = tcache;
      const unsigned char* pool = static_cast<const unsigned char*>(lane < 16 ? a.k_pool : a.v_pool);
      unsigned char* st = lane < 16 ? k_code : v_code;
      const long long pool_row = (long long)a.layer * a.n_blocks * H;  // chunks before the layer
      const int ups = C::TS >> lur;                                   // units per stage
      Piece p;
      bool have = next_piece(p);
      if (have && !use_rec) tc.ensure(a.table, a.max_blocks, p.rep, p.b0, p.b0, lane);
      wait_previous_grid();
      int stage = 0;
      for (; have; have = next_piece(p)) {
        const int n_st = stages_of(p);
        const int u_first = p.b0 * KU;
        const int u_end = u_first + ((p.tok_end - p.b0 * B + UR - 1) >> lur);
        for (int i = 0; i < n_st; ++i, ++stage) {
          // lanes 0 .. 15 bring the K units of a stage, lanes 16 .. 31 the V units
          const int u0 = u_first + i * ups, u = u0 + (lane & 15);
          const int n_units = min(u_end - u0, ups);
          const bool mine = (lane & 15) < n_units;
          const int j0 = KU == 1 ? u0 : u0 / KU;
          const int jl = KU == 1 ? u0 + n_units - 1 : (u0 + n_units - 1) / KU;
          const int j = KU == 1 ? u : u / KU;
          const int row = KU == 1 ? 0 : (u - j * KU) * UR;
          // the first stage of the record's piece takes the record's block ids
          const bool from_rec = use_rec && stage == 0 && p.seg == rec_s->seg && j0 >= rec_s->b0 &&
                                jl - rec_s->b0 < rec_s->n_pid;
          if (!from_rec) tc.ensure(a.table, a.max_blocks, p.rep, j0, jl, lane);
          int pid = 0;
          if (mine) pid = from_rec ? rec_s->pid[j - rec_s->b0] : tc.ent[j - tc.base];
          if (pid < 0 || pid >= a.n_blocks) {
            record_status(a.status, 1);
            pid = 0;  // stay in bounds; the result is flagged as invalid
          }
          const unsigned char* src = pool + (pool_row + static_cast<long long>(pid) * H + p.head) *
                                                static_cast<long long>(B * C::ROW);
          const int slot = stage % C::NC;
          unsigned char* dst = st + slot * C::CODES + (lane & 15) * unit_bytes;
          if (stage >= C::NC) wait(&empty[slot], ((stage / C::NC) & 1) ^ 1);
          if (!alive) continue;
          if (lane == 0) mbar_arrive_expect_tx(&full[slot], 2u * n_units * unit_bytes);
          __syncwarp();
          if (mine) {
            if (KU == 1) {
              bulk_load(dst, src, unit_bytes, &full[slot]);
            } else {  // part of a larger block: plane by plane
              for (int q = 0; q < 4; ++q) {
                bulk_load(dst + q * UR * 16, src + (q * B + row) * 16, UR * 16, &full[slot]);
                if (lane >= 16)
                  bulk_load(dst + UR * 64 + q * UR * 2, src + B * 64 + (q * B + row) * 2, UR * 2,
                            &full[slot]);
              }
              if (lane < 16) bulk_load(dst + UR * 64, src + B * 64 + row * 8, UR * 8, &full[slot]);
            }
          }
        }
      }
      // copies still in flight land before the CTA may exit
      const int first = stage > C::NC ? stage - C::NC : 0;
      for (int k = first; k < stage && alive; ++k)
        alive = q4_wait(&full[k % C::NC], (k / C::NC) & 1);
    } else if (warp == 17) {
      // ------------------------------------------------------------ Q tiles
      wait_previous_grid();
      int np = 0;
      Piece p;
      while (next_piece(p)) {
        if (stages_of(p) == 0) continue;
        const int qb = np % C::QBUF;
        if (np >= C::QBUF) wait(&q_empty[qb], ((np / C::QBUF) - 1) & 1);
        // 16-byte chunk (column, eight dimensions) k * 32 + lane: two columns
        // a step, the columns past the piece's zero
        const int cols = p.ncols <= 16 ? 16 : 32;  // N of its S MMAs
        auto chunk_at = [&](int k) -> uint4 {
          const int col = k * 2 + (lane >> 4), cg = lane & 15;
          if (col >= p.ncols) return make_uint4(0u, 0u, 0u, 0u);
          int seqm = p.rep, gi = col;
          if constexpr (PLAN) {
            const int mi = col / G;
            gi = col - mi * G;
            seqm = a.members[p.mem + mi];
          }
          return *reinterpret_cast<const uint4*>(
              static_cast<const unsigned char*>(a.q) +
              (((long long)seqm * a.n_q_heads + (long long)p.head * G + gi) * C::D + cg * 8) * 2);
        };
        uint32_t am = 0;
#pragma unroll 4
        for (int k = 0; k < cols / 2; ++k) {
          const uint4 v = chunk_at(k);
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) am = max(am, max((w[i] << 16) & 0x7fffffffu, w[i] & 0x7fff0000u));
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) am = max(am, __shfl_xor_sync(0xffffffffu, am, o));
        int E = static_cast<int>(am >> 23);  // biased exponent of the largest |q|
        E = E < 14 ? 14 : E;
        const float sc = __uint_as_float(static_cast<uint32_t>(268 - E) << 23);  // 2^(141 - E)
        const uint32_t qs = smem_u32(q_s + qb * C::QTILE);
#pragma unroll 4
        for (int k = 0; k < cols / 2; ++k) {
          const uint4 v = chunk_at(k);  // from the L1 this time
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
          float x[8];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16) * sc;
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u) * sc;
          }
          const int col = k * 2 + (lane >> 4), cg = lane & 15;
          if (alive)  // element order of the converted K rows: 0 4 1 5 2 6 3 7
            sts128(qs + (cg >> 3) * C::QHALF + col * 128 + (((cg & 7) ^ (col & 7)) << 4),
                   pack_f16(x[0], x[4]), pack_f16(x[1], x[5]), pack_f16(x[2], x[6]),
                   pack_f16(x[3], x[7]));
        }
        // S = 2^(E - 141) * accumulator (K rows' powers of two apart)
        if (lane == 0 && alive)
          q_fac[qb] = a.qscale * __uint_as_float(static_cast<uint32_t>(E) << 23) * 0x1p-14f;
        fence_async_smem();
        __syncwarp();
        if (lane == 0 && alive) mbar_arrive(&q_full[qb]);
        ++np;
      }
    } else {
      // ----------------------------------- MMA issuers: 18 for S, 19 for P.V.
      // The whole warp walks and waits, so that descriptors are the warp's
      // (uniform) values, and one lane issues.
      wait_previous_grid();
      const bool one = lane == 0;
      int stage = 0, np = 0;
      Piece p;
      if (warp == 18) {
        constexpr uint32_t idS16 = idesc_f16(128, 16, false, false);
        constexpr uint32_t idS32 = idesc_f16(128, 32, false, false);
        while (next_piece(p)) {
          const int n_st = stages_of(p);
          if (n_st == 0) continue;
          const uint32_t id = p.ncols <= 16 ? idS16 : idS32;
          const int qb = np % C::QBUF;
          const uint64_t q_desc = smem_desc(smem_u32(q_s + qb * C::QTILE), 16, 1024, kSwizzle128);
          wait(&q_full[qb], (np / C::QBUF) & 1);
          for (int i = 0; i < n_st; ++i, ++stage) {
            if (stage >= 2) wait(&s_empty[stage & 1], ((stage >> 1) - 1) & 1);
            wait(&k_full[stage % C::NK], (stage / C::NK) & 1);
            if (!alive) continue;
            tc_fence_after();
            const uint32_t d = tmem + C::TM_S + (stage & 1) * 32;
            const uint32_t k0 = tmem + C::TM_K + (stage % C::NK) * 64;
            if (one) {
#pragma unroll
              for (int k = 0; k < 8; ++k)
                tc_mma_ts(d, k0 + k * 8, q_desc + (((k >> 2) * C::QHALF + (k & 3) * 32) >> 4), id,
                          k > 0);
              tc_commit(&k_empty[stage % C::NK]);
              tc_commit(&s_full[stage & 1]);
            }
            __syncwarp();
          }
          if (one) tc_commit(&q_empty[qb]);
          ++np;
        }
      } else {
        constexpr uint32_t idP16 = idesc_f16(128, 16, true, true);
        constexpr uint32_t idP32 = idesc_f16(128, 32, true, true);
        const uint64_t v_desc = smem_desc(smem_u32(v_st), C::HALF, 1024, kSwizzle128);
        const uint64_t p_desc = smem_desc(smem_u32(p_st), C::PBUF, 512, kSwizzle64);
        while (next_piece(p)) {
          const int n_st = stages_of(p);
          if (n_st == 0) continue;
          const uint32_t id = p.ncols <= 16 ? idP16 : idP32;
          if (np > 0) wait(o_free, (np - 1) & 1);
          for (int i = 0; i < n_st; ++i, ++stage) {
            const int b = stage % C::NV, pb = stage % C::NP;
            wait(&v_full[b], (stage / C::NV) & 1);
            wait(&p_full[pb], (stage / C::NP) & 1);
            if (!alive) continue;
            tc_fence_after();
            const uint64_t vd = v_desc + ((b * C::VBUF) >> 4), pd = p_desc + ((pb * C::PBUF) >> 4);
            const int nvalid = p.tok_end - (p.b0 * B + i * C::TS);
            if (one) {
              // a stage's 16-token steps; those past the context are left out
#pragma unroll
              for (int k = 0; k < 8; ++k)
                if (k * 16 < nvalid)
                  tc_mma(tmem + C::TM_O, vd + k * (2048 >> 4), pd + k * (1024 >> 4), id,
                         (i > 0 || k > 0) ? 1u : 0u);
              tc_commit(&pv_done[pb]);
            }
            __syncwarp();
          }
          ++np;
        }
      }
      // every MMA either warp issued has completed before TMEM is released
      if (one) {
        tc_commit(fin);
        q4_wait(fin, 0);
      }
      __syncwarp();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TM_COLS);
  }
}

}  // namespace pkv
