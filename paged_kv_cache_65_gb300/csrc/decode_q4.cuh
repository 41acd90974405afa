// Split-K paged decode attention, partial pass, over a q4_0 pool (4-bit codes,
// one fp16 scale per 32 values).
//
// Same contract, work split and workspace as decode.cuh and decode_mma.cuh
// (see there): per piece of a segment it emits the base-2 online-softmax
// statistics m, l and the unnormalised O of every query column.
//
// The stored value of dimension d of token t is (n - 8) * ks, n the nibble
// (0 .. 15) and ks the scale of (token, group of 32 dimensions).  With the
// groups q = 0 .. D/32 - 1:
//     S[t]  = sum_q ks[t][q] * (sum_{d in q} n[t][d] Q[d] - 8 sum_{d in q} Q[d])
//     O[d]  = sum_t n[t][d] P'[t][q] - 8 sum_t P'[t][q],  P'[t][q] = p[t] vs[t][q]
// so both products run on the nibbles themselves and the offset 8 costs one
// constant per group (the MMA's initial accumulator) in S and one more MMA per
// group in O.
//
// Nibbles become fp16 MMA operands with one AND each: the fp16 bit pattern n
// (n < 16, exponent bits zero) is the subnormal n * 2^-24, and n << 4 is
// n * 2^-20, both exact MMA inputs.  A 32-bit word of eight nibbles gives four
// operand registers in five instructions (four ANDs, one shift); the factors
// 2^-24 and 16 go into Q (scaled per column by a power of two, so that any
// magnitude of q stays inside fp16) and into the final scale of O.
//
// MMAs are m16n8k16 (fp16 in, f32 accumulate) per 16-token tile:
//     S^T [16 tokens x 8 cols] = K [16 x 32] . Q^T [32 x 8]   two per group
//     O^T [32 x 8 cols]       += V^T [32 x 16] . P'^T [16 x 8] two per group
// A group's 32 dimensions of one token are 16 consecutive bytes, so the
// 16-bit ldmatrix hands lane (g, t) word t of token row g: nibbles of
// dimensions 8t .. 8t + 7.  The sum over dimensions does not depend on their
// order, so Q's fragments just follow the order the words unpack in.  V^T
// comes from the 8-bit transposing ldmatrix (ldsm8_t): bytes of four tokens in
// byte column g = dimensions 2g (low nibbles) and 2g + 1 (high nibbles), which
// an MMA takes as its rows g and g + 8.
//
// Shared memory: a stage holds TS tokens of K and of V of one K/V head as
// units of UR = min(B, TS) tokens, each unit laid out like a pool chunk of UR
// tokens: D/32 code planes [UR][16 bytes], then the scales.  Rows of a plane
// are adjacent 16-byte vectors, so every 8-row phase of both ldmatrix forms
// reads 8 different bank groups without a swizzle, and a block that is a
// whole unit arrives in one bulk copy.
#pragma once

#include <cuda_fp16.h>

#include "decode_mma.cuh"

namespace pkv {

constexpr int kQ4Warps = 4;                        // consumer warps
constexpr int kQ4Threads = (kQ4Warps + 1) * 32;    // and the producer
constexpr int kQ4CtasPerSm = 3;

template <int D>
struct Q4Cfg {
  static constexpr int GR = D / 32;                // groups of 32 dimensions
  static constexpr int TS = 128;                   // tokens per stage
  static constexpr int ROW = D / 2 + D / 16;       // bytes per token row: codes and scales
  static constexpr int STAGE_BYTES = TS * ROW;     // K (or V) per stage
  static constexpr int NST = 3;                    // stages in the ring
  static constexpr int MT = D / 16;                // m-tiles of O^T
  static constexpr int CC = 4;                     // columns per combine pass
  static_assert(D == 64 || D == 128, "head dim");
};

// Tokens per unit for block size B: a block when it divides the stage, the
// stage when that divides the block, else 64 (B = 192).  A power of two.
__host__ __device__ constexpr int q4_unit_rows(int B) {
  return B <= 128 ? B : (B % 128 == 0 ? 128 : 64);
}

// Token order inside a 16-token tile: row k of S^T (and k-slot k of P'^T)
// stands for token q4_srow(k); lane i of ldsm8_t addresses token q4_vrow(i).
// ldsm8_t hands lane (g, t) the tokens of lanes 4t .. 4t + 3 as bytes 0 .. 3;
// bytes 0 and 2 become k-slots 2t and 2t + 1, bytes 1 and 3 k-slots 2t + 8 and
// 2t + 9.  The rotation of the upper eight keeps each 8-lane phase on eight
// different 16-byte bank groups.
__device__ __forceinline__ int q4_srow(int k) { return k < 8 ? k : 8 + ((k + 4) & 7); }
__device__ __forceinline__ int q4_vrow(int i) {
  return q4_srow(2 * (i >> 2) + ((i >> 1) & 1) + 8 * (i & 1));
}

constexpr uint32_t kNibLo = 0x000f000fu;  // n * 2^-24
constexpr uint32_t kNibHi = 0x00f000f0u;  // n * 2^-20
constexpr uint32_t kNibOff = 0x80088008u; // -8 * 2^-24 twice

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t r;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(r) : "r"(addr));
  return r;
}

template <int D>
constexpr int decode_q4_smem_bytes() {
  using C = Q4Cfg<D>;
  return 2 * C::NST * C::STAGE_BYTES        // K and V stages
         + kQ4Warps * C::CC * D * 4         // combine: O per warp, CC columns at a time
         + kQ4Warps * 8 * 2 * 4             // combine: m, l per warp and column
         + 2 * C::NST * 8                   // mbarriers
         + kTableCache * 4                  // producer table cache
         + kPieceRing * (48 + 16)           // piece descriptors and their mbarriers
         + 64 + 128 + 16;                   // walk state, start record, alignment
}

template <int D, bool PLAN>
__global__ void __launch_bounds__(kQ4Threads, kQ4CtasPerSm) decode_q4_kernel(const DecodeArgs a) {
  using C = Q4Cfg<D>;
  constexpr int NST = C::NST, GR = C::GR;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  unsigned char* k_st = smem_raw;
  unsigned char* v_st = k_st + NST * C::STAGE_BYTES;
  float* cmb_o = reinterpret_cast<float*>(v_st + NST * C::STAGE_BYTES);
  float* cmb_ml = cmb_o + kQ4Warps * C::CC * D;
  uint64_t* full = reinterpret_cast<uint64_t*>(cmb_ml + kQ4Warps * 8 * 2);
  uint64_t* empty = full + NST;
  long long* walk = reinterpret_cast<long long*>(empty + NST);
  int32_t* tcache = reinterpret_cast<int32_t*>(walk + 4);
  PlanStart* rec_s = reinterpret_cast<PlanStart*>(tcache + kTableCache);
  Piece* ring = reinterpret_cast<Piece*>(rec_s + 1);
  uint64_t* dfull = reinterpret_cast<uint64_t*>(ring + kPieceRing);
  uint64_t* dempty = dfull + kPieceRing;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int B = a.block_size;
  const int H = a.n_kv_heads, G = a.n_q_heads / H;
  const int UR = q4_unit_rows(B);
  const int lur = 31 - __clz(UR);
  const uint32_t unit_bytes = static_cast<uint32_t>(UR) * C::ROW;

  if (threadIdx.x == 0) {
    for (int i = 0; i < NST; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], kQ4Warps);
    }
    for (int i = 0; i < kPieceRing; ++i) {
      mbar_init(&dfull[i], 1);
      mbar_init(&dempty[i], kQ4Warps);
    }
    fence_barrier_init();
  }
  // tables and lengths that kernels before this one write (a pool with device
  // tables) are read only after them; host-written ones before the wait, as in
  // decode_mma.cuh
  if (a.meta_wait) griddep_wait();
  const bool use_rec = PLAN && a.starts != nullptr && a.start_grid == a.grid;
  if (warp == 0) {
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
  __syncthreads();

  const long long W = walk[2], chunk = walk[3];
  const long long r_begin = (long long)blockIdx.x * chunk;
  const long long r_end = r_begin + chunk < W ? r_begin + chunk : W;
  auto wait_previous_grid = [&]() {
    griddep_wait();
    griddep_launch_dependents();
    if constexpr (!PLAN) {
      if (blockIdx.x == 0 && warp == 0)
        write_prefix(a.ctx, a.n_seq, B, H, a.max_blocks, a.ws_pre);
    }
  };

  if (warp == kQ4Warps) {
    // ------------------------------------------------------------ producer
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
    bool alive = true;
    int stage = 0;
    TableCache tc;
    tc.ent = tcache;
    // pieces go to the consumers as descriptors, published one piece ahead of
    // their copies (see decode_mma.cuh); rep = -1 ends the list
    int npub = 0;
    auto publish = [&](const Piece& x, bool valid) {
      const int di = npub % kPieceRing;
      if (npub >= kPieceRing && alive) {
        if (!mbar_wait_bounded(&dempty[di], ((npub / kPieceRing) - 1) & 1, kWaitLimitNs)) {
          alive = false;
          if (lane == 0) record_status(a.status, 8);
        }
      }
      if (lane == 0) {
        Piece y = x;
        if (!valid) y.rep = -1;
        ring[di] = y;
        mbar_arrive(&dfull[di]);
      }
      __syncwarp();
      ++npub;
    };
    Piece p, pn;
    bool have = next_piece(p);
    if (have && !use_rec) tc.ensure(a.table, a.max_blocks, p.rep, p.b0, p.b0, lane);
    wait_previous_grid();
    publish(p, have);
    while (have) {
      const bool have_next = next_piece(pn);
      publish(pn, have_next);
      for (int tok0 = p.b0 * B; tok0 < p.tok_end; tok0 += C::TS) {
        const int slot = stage % NST;
        if (stage >= NST && alive) {
          if (!mbar_wait_bounded(&empty[slot], ((stage / NST) & 1) ^ 1, kWaitLimitNs)) {
            alive = false;
            if (lane == 0) record_status(a.status, 8);
          }
        }
        const int nvalid = p.tok_end - tok0 < C::TS ? p.tok_end - tok0 : C::TS;
        const int nunits = (nvalid + UR - 1) >> lur;
        const int jl = (tok0 + (nunits - 1) * UR) / B;
        // the first stage of the record's piece takes the record's block ids
        const bool from_rec = use_rec && stage == 0 && p.seg == rec_s->seg &&
                              tok0 / B >= rec_s->b0 && jl - rec_s->b0 < rec_s->n_pid;
        if (!from_rec) tc.ensure(a.table, a.max_blocks, p.rep, tok0 / B, jl, lane);
        if (lane == 0) mbar_arrive_expect_tx(&full[slot], 2u * nunits * unit_bytes);
        __syncwarp();
        for (int u = lane; u < nunits; u += 32) {
          const int t = tok0 + u * UR;
          const int j = t / B;
          const int row = t - j * B;
          int pid = from_rec ? rec_s->pid[j - rec_s->b0] : tc.ent[j - tc.base];
          if (pid < 0 || pid >= a.n_blocks) {
            record_status(a.status, 1);
            pid = 0;  // stay in bounds; the result is flagged as invalid
          }
          const long long chunk_off =
              (((long long)a.layer * a.n_blocks + pid) * H + p.head) * B * C::ROW;
          const unsigned char* kg = static_cast<const unsigned char*>(a.k_pool) + chunk_off;
          const unsigned char* vg = static_cast<const unsigned char*>(a.v_pool) + chunk_off;
          unsigned char* ks = k_st + slot * C::STAGE_BYTES + u * unit_bytes;
          unsigned char* vs = v_st + slot * C::STAGE_BYTES + u * unit_bytes;
          if (UR == B) {
            bulk_load(ks, kg, unit_bytes, &full[slot]);
            bulk_load(vs, vg, unit_bytes, &full[slot]);
          } else {  // part of a larger block: plane by plane
#pragma unroll
            for (int q = 0; q < GR; ++q) {
              bulk_load(ks + q * UR * 16, kg + (q * B + row) * 16, UR * 16, &full[slot]);
              bulk_load(vs + q * UR * 16, vg + (q * B + row) * 16, UR * 16, &full[slot]);
              bulk_load(vs + GR * UR * 16 + q * UR * 2, vg + GR * B * 16 + (q * B + row) * 2,
                        UR * 2, &full[slot]);
            }
            bulk_load(ks + GR * UR * 16, kg + GR * B * 16 + row * GR * 2, UR * GR * 2,
                      &full[slot]);
          }
        }
        ++stage;
      }
      p = pn;
      have = have_next;
    }
    const int first = stage > NST ? stage - NST : 0;
    for (int k = first; k < stage; ++k)
      mbar_wait_bounded(&full[k % NST], (k / NST) & 1, kWaitLimitNs);
    return;
  }

  // -------------------------------------------------------------- consumers
  wait_previous_grid();
  const int g = lane >> 2;  // groupID: row of A / C, column of B
  const int t = lane & 3;   // thread in group
  const uint32_t k_base = smem_u32(k_st);
  const uint32_t v_base = smem_u32(v_st);
  const int cstride = PLAN ? a.c_max : G;  // columns per workspace slot
  bool alive = true;
  int stage = 0;
  // q of this warp's column of a piece (column wn * 8 + g): dimensions
  // 32 q + 8 t .. + 7 of each group, raw bf16, loaded one piece ahead
  auto load_q = [&](const Piece& pc, uint4 (&qr)[GR]) {
    const int NTc = pc.ncols <= 8 ? 1 : (pc.ncols <= 16 ? 2 : 4);
    const int col = (warp % NTc) * 8 + g;
    const bool colv = col < pc.ncols;
    int seqm = pc.rep, gi = col;
    if constexpr (PLAN) {
      const int mi = col / G;
      gi = col - mi * G;
      seqm = colv ? a.members[pc.mem + mi] : 0;
    }
    const uint4* qw = reinterpret_cast<const uint4*>(
        static_cast<const unsigned char*>(a.q) +
        ((long long)seqm * a.n_q_heads + (long long)pc.head * G + (colv ? gi : 0)) * D * 2);
#pragma unroll
    for (int q = 0; q < GR; ++q) qr[q] = colv ? qw[q * 4 + t] : make_uint4(0u, 0u, 0u, 0u);
  };
  int nread = 0;
  auto read_piece = [&](Piece& x) -> bool {
    const int di = nread % kPieceRing;
    if (alive && !mbar_wait_bounded(&dfull[di], (nread / kPieceRing) & 1, kWaitLimitNs)) {
      alive = false;
      if (lane == 0) record_status(a.status, 8);
    }
    alive = __all_sync(0xffffffffu, alive);
    if (!alive) return false;
    x = ring[di];
    __syncwarp();
    if (lane == 0) mbar_arrive(&dempty[di]);
    ++nread;
    return x.rep >= 0;
  };
  Piece p, pn;
  uint4 qn[GR];
  bool have = read_piece(p), have_next = false;
  if (have) load_q(p, qn);
  for (; have; p = pn, have = have_next) {
    const int NT = p.ncols <= 8 ? 1 : (p.ncols <= 16 ? 2 : 4);  // n-tiles of the piece
    const int WT = kQ4Warps / NT;                                 // warps per n-tile
    const int wt = warp / NT;
    // Q fragments.  Column g is scaled by the power of two that brings its
    // largest |q| into [2^11, 2^12): bf16's 8 bits then stay exact in fp16
    // over 2^25 of range.  MMA 0 of a group takes dimensions 8t + {0, 4} and
    // {2, 6}, MMA 1 (the nibbles times 16) 8t + {1, 5} and {3, 7} over 16.
    uint32_t qf[GR][4];
    float ccol[GR][2], fcol[2];  // columns 2t and 2t + 1
    {
      uint32_t am = 0;
#pragma unroll
      for (int q = 0; q < GR; ++q) {
        const uint32_t w[4] = {qn[q].x, qn[q].y, qn[q].z, qn[q].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          am = max(am, (w[i] << 16) & 0x7fffffffu);
          am = max(am, w[i] & 0x7fff0000u);
        }
      }
      am = max(am, __shfl_xor_sync(0xffffffffu, am, 1));
      am = max(am, __shfl_xor_sync(0xffffffffu, am, 2));
      int E = static_cast<int>(am >> 23);  // biased exponent of the largest |q|
      E = E < 12 ? 12 : E;
      const float sc = __uint_as_float(static_cast<uint32_t>(265 - E) << 23);  // 2^(138 - E)
      // S = 2^24 * 2^(E - 138) * accumulator, times the score scale
      const float f = a.qscale * __uint_as_float(static_cast<uint32_t>(E) << 23) * 0x1p13f;
      fcol[0] = __shfl_sync(0xffffffffu, f, 8 * t);
      fcol[1] = __shfl_sync(0xffffffffu, f, 8 * t + 4);
#pragma unroll
      for (int q = 0; q < GR; ++q) {
        const uint32_t w[4] = {qn[q].x, qn[q].y, qn[q].z, qn[q].w};
        float x[8];
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[2 * i] = __uint_as_float(w[i] << 16) * sc;
          x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u) * sc * 0.0625f;
        }
        qf[q][0] = pack_f16(x[0], x[4]);
        qf[q][1] = pack_f16(x[2], x[6]);
        qf[q][2] = pack_f16(x[1], x[5]);
        qf[q][3] = pack_f16(x[3], x[7]);
        // the offset's sum takes the values the MMAs take (as rounded)
        sum = (half_lo(qf[q][0]) + half_hi(qf[q][0])) + (half_lo(qf[q][1]) + half_hi(qf[q][1]));
        sum += 16.f * ((half_lo(qf[q][2]) + half_hi(qf[q][2])) +
                       (half_lo(qf[q][3]) + half_hi(qf[q][3])));
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        sum *= -8.f * 0x1p-24f;
        ccol[q][0] = __shfl_sync(0xffffffffu, sum, 8 * t);
        ccol[q][1] = __shfl_sync(0xffffffffu, sum, 8 * t + 4);
      }
    }
    have_next = read_piece(pn);
    if (have_next) load_q(pn, qn);
    float m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f};
    float o[C::MT][4], oc[GR][4];
#pragma unroll
    for (int mt = 0; mt < C::MT; ++mt) o[mt][0] = o[mt][1] = o[mt][2] = o[mt][3] = 0.f;
#pragma unroll
    for (int q = 0; q < GR; ++q) oc[q][0] = oc[q][1] = oc[q][2] = oc[q][3] = 0.f;

    for (int tok0 = p.b0 * B; tok0 < p.tok_end; tok0 += C::TS, ++stage) {
      const int slot = stage % NST;
      if (alive && !mbar_wait_bounded(&full[slot], (stage / NST) & 1, kWaitLimitNs)) {
        alive = false;
        if (lane == 0) record_status(a.status, 8);
      }
      alive = __all_sync(0xffffffffu, alive);  // reconverge before ldmatrix / mma.sync
      const int nvalid = p.tok_end - tok0 < C::TS ? p.tok_end - tok0 : C::TS;
      const uint32_t kb = k_base + slot * C::STAGE_BYTES;
      const uint32_t vb = v_base + slot * C::STAGE_BYTES;
      // shared offset of token r's unit and of its row inside the unit
      auto unit_of = [&](int r) -> uint32_t { return (r >> lur) * unit_bytes; };
      auto row_of = [&](int r) -> uint32_t { return r & (UR - 1); };
#pragma unroll 1
      for (int tb = wt * 16; tb < nvalid; tb += WT * 16) {
        const int nv = nvalid - tb;  // tokens of the tile inside the context (>= 1)
        const int rlo = tb + q4_srow(g), rhi = tb + q4_srow(g + 8);
        // ---- S^T = K . Q^T, one accumulator per group
        float s[4] = {0.f, 0.f, 0.f, 0.f};
        {
          // matrices: rows 0-7 and 8-15 of group q, then of group q + 1
          const int r = tb + q4_srow(((lane >> 3) & 1) * 8 + (lane & 7));
          const uint32_t ka = kb + unit_of(r) + row_of(r) * 16 + (lane >> 4) * UR * 16;
          const uint32_t sb = kb + GR * UR * 16;
          const uint32_t slo = sb + unit_of(rlo) + row_of(rlo) * GR * 2;
          const uint32_t shi = sb + unit_of(rhi) + row_of(rhi) * GR * 2;
#pragma unroll
          for (int q = 0; q < GR; q += 2) {
            uint32_t w[4];
            ldsm_x4(ka + q * UR * 16, w[0], w[1], w[2], w[3]);
            const uint32_t kl = lds32(slo + q * 2), kh = lds32(shi + q * 2);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint32_t wa = w[2 * i], wb = w[2 * i + 1];
              const uint32_t wa8 = wa >> 8, wb8 = wb >> 8;
              float acc[4] = {ccol[q + i][0], ccol[q + i][1], ccol[q + i][0], ccol[q + i][1]};
              mma_f16(acc, wa & kNibLo, wb & kNibLo, wa8 & kNibLo, wb8 & kNibLo, qf[q + i][0],
                      qf[q + i][1]);
              mma_f16(acc, wa & kNibHi, wb & kNibHi, wa8 & kNibHi, wb8 & kNibHi, qf[q + i][2],
                      qf[q + i][3]);
              const float fl = i ? half_hi(kl) : half_lo(kl), fh = i ? half_hi(kh) : half_lo(kh);
              s[0] = fmaf(fl, acc[0], s[0]);
              s[1] = fmaf(fl, acc[1], s[1]);
              s[2] = fmaf(fh, acc[2], s[2]);
              s[3] = fmaf(fh, acc[3], s[3]);
            }
          }
        }
        // ---- scale, mask (rows past the context, whatever their bytes hold),
        // tile maximum per column
        const bool v0 = rlo < nvalid, v1 = rhi < nvalid;
        s[0] = v0 ? s[0] * fcol[0] : -INFINITY;
        s[1] = v0 ? s[1] * fcol[1] : -INFINITY;
        s[2] = v1 ? s[2] * fcol[0] : -INFINITY;
        s[3] = v1 ? s[3] * fcol[1] : -INFINITY;
        float mx0 = fmaxf(s[0], s[2]), mx1 = fmaxf(s[1], s[3]);
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
          mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, off));
          mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, off));
        }
        const float mn0 = fmaxf(m_run[0], mx0), mn1 = fmaxf(m_run[1], mx1);
        const float al0 = exp2_approx(m_run[0] - mn0), al1 = exp2_approx(m_run[1] - mn1);
        m_run[0] = mn0;
        m_run[1] = mn1;
        const float p0 = exp2_approx(s[0] - mn0), p1 = exp2_approx(s[1] - mn1);
        const float p2 = exp2_approx(s[2] - mn0), p3 = exp2_approx(s[3] - mn1);
        l_run[0] = l_run[0] * al0 + (p0 + p2);
        l_run[1] = l_run[1] * al1 + (p1 + p3);
        // the rescale is skipped when no running maximum of the warp moved
        if (__any_sync(0xffffffffu, (al0 != 1.f) | (al1 != 1.f))) {
#pragma unroll
          for (int mt = 0; mt < C::MT; ++mt) {
            o[mt][0] *= al0;
            o[mt][1] *= al1;
            o[mt][2] *= al0;
            o[mt][3] *= al1;
          }
#pragma unroll
          for (int q = 0; q < GR; ++q) {
            oc[q][0] *= al0;
            oc[q][1] *= al1;
            oc[q][2] *= al0;
            oc[q][3] *= al1;
          }
        }
        // ---- P^T in fp16 (p <= 1; 11 bits), transposed: b0 holds tokens
        // srow(2t), srow(2t + 1) of column g, b1 srow(2t + 8), srow(2t + 9)
        const uint32_t b0 = movm_t(pack_f16(p0, p1)), b1 = movm_t(pack_f16(p2, p3));
        // ---- O^T += V^T . (P vs)^T per group.  The V scales of a token pair
        // are adjacent, so P' is one fp16 product per register (a second
        // rounding to 11 bits; |p| <= 1 and the scale is a finite fp16, so it
        // never overflows); scales past the context count as zero.
        {
          const int k0 = 2 * t, k1 = q4_srow(2 * t + 8);  // even: a pair never crosses a unit
          const uint32_t m0 = (k0 < nv ? 0x0000ffffu : 0u) | (k0 + 1 < nv ? 0xffff0000u : 0u);
          const uint32_t m1 = (k1 < nv ? 0x0000ffffu : 0u) | (k1 + 1 < nv ? 0xffff0000u : 0u);
          const uint32_t sb = vb + GR * UR * 16;
          const uint32_t s0 = sb + unit_of(tb + k0) + row_of(tb + k0) * 2;
          const uint32_t s1 = sb + unit_of(tb + k1) + row_of(tb + k1) * 2;
          const int r = tb + q4_vrow(lane & 15);
          const uint32_t va = vb + unit_of(r) + row_of(r) * 16;
#pragma unroll
          for (int q = 0; q < GR; ++q) {
            const uint32_t c0 = hmul2(b0, lds32(s0 + q * UR * 2) & m0);
            const uint32_t c1 = hmul2(b1, lds32(s1 + q * UR * 2) & m1);
            uint32_t r0, r1;
            ldsm8_t(va + q * UR * 16, r0, r1);
            const uint32_t r08 = r0 >> 8, r18 = r1 >> 8;
            mma_f16(o[2 * q], r0 & kNibLo, r0 & kNibHi, r08 & kNibLo, r08 & kNibHi, c0, c1);
            mma_f16(o[2 * q + 1], r1 & kNibLo, r1 & kNibHi, r18 & kNibLo, r18 & kNibHi, c0, c1);
            mma_f16(oc[q], kNibOff, kNibOff, kNibOff, kNibOff, c0, c1);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[slot]);
    }
    // row g of m-tile 2q + h is dimension 32 q + 16 h + 2 g, row g + 8 the next
    // one (nibbles times 16)
#pragma unroll
    for (int mt = 0; mt < C::MT; ++mt)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        o[mt][i] = (o[mt][i] * (i < 2 ? 1.f : 0.0625f) + oc[mt >> 1][i]) * 0x1p24f;

    // ---- combine the states of the warps that share an n-tile
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
      l_run[0] += __shfl_xor_sync(0xffffffffu, l_run[0], off);
      l_run[1] += __shfl_xor_sync(0xffffffffu, l_run[1], off);
    }
    if (g == 0) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        cmb_ml[(warp * 8 + 2 * t + k) * 2] = m_run[k];
        cmb_ml[(warp * 8 + 2 * t + k) * 2 + 1] = l_run[k];
      }
    }
    const long long slot_id = (long long)blockIdx.x + p.seg;
    for (int pc = 0; pc < 8; pc += C::CC) {
      if (pc >= p.ncols) break;  // no column of any n-tile in this pass
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int c8 = 2 * t + k;
        if (c8 >= pc && c8 < pc + C::CC) {
#pragma unroll
          for (int mt = 0; mt < C::MT; ++mt)
            *reinterpret_cast<float2*>(&cmb_o[(warp * C::CC + c8 - pc) * D + mt * 16 + 2 * g]) =
                make_float2(o[mt][k], o[mt][2 + k]);
        }
      }
      named_bar_sync(1, kQ4Warps * 32);
      constexpr int D4 = D / 4;
      for (int idx = threadIdx.x; idx < NT * C::CC * D4; idx += kQ4Warps * 32) {
        const int wni = idx / (C::CC * D4);
        const int rem = idx - wni * C::CC * D4;
        const int cc = rem / D4, d = (rem - cc * D4) * 4;
        const int col = wni * 8 + pc + cc;
        if (col >= p.ncols) continue;
        float M = -INFINITY;
        for (int j = 0; j < WT; ++j) M = fmaxf(M, cmb_ml[((wni + j * NT) * 8 + pc + cc) * 2]);
        float L = 0.f;
        float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int j = 0; j < WT; ++j) {
          const int w = wni + j * NT;
          const float mw = cmb_ml[(w * 8 + pc + cc) * 2];
          const float f = mw == -INFINITY ? 0.f : exp2_approx(mw - M);
          L += f * cmb_ml[(w * 8 + pc + cc) * 2 + 1];
          const float4 v = *reinterpret_cast<const float4*>(&cmb_o[(w * C::CC + cc) * D + d]);
          O.x += f * v.x;
          O.y += f * v.y;
          O.z += f * v.z;
          O.w += f * v.w;
        }
        *reinterpret_cast<float4*>(&a.ws_o[(slot_id * cstride + col) * D + d]) = O;
        if (d == 0) {
          a.ws_ml[(slot_id * cstride + col) * 2] = M;
          a.ws_ml[(slot_id * cstride + col) * 2 + 1] = L;
        }
      }
      named_bar_sync(1, kQ4Warps * 32);
    }
  }
}

}  // namespace pkv
