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
// so both products run on the nibbles themselves.  The offset 8 costs S one MMA
// per tile (the scales times the groups' sums of Q); for O every MMA of
// nibbles is followed by one whose A operand is -8 throughout, into the same
// accumulator, which so never holds more than a tile's offset beside the
// signed sum (summed apart over a long piece the two would cancel to a small
// rest of large sums: 1.8x the error at 32,771 tokens).
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
constexpr int kQ4CtasPerSm = 2;

template <int D>
struct Q4Cfg {
  static constexpr int GR = D / 32;                // groups of 32 dimensions
  static constexpr int TS = 64;                    // tokens per slot
  static constexpr int ROW = D / 2 + D / 16;       // bytes per token row: codes and scales
  static constexpr int SLOT_BYTES = TS * ROW;      // K (or V) per slot
  static constexpr int NS = 10;                    // slots in the ring
  static constexpr int PT = 4;                     // 16-token tiles per pass
  static constexpr int MT = D / 16;                // m-tiles of O^T
  static constexpr int CC = 4;                     // columns per combine pass
  static_assert(D == 64 || D == 128, "head dim");
};

// Tokens per unit: a block when it divides the slot, else the slot (blocks of
// 128, 192 and 256).  A power of two.
__host__ __device__ constexpr int q4_unit_rows(int B) { return B < 64 ? B : 64; }

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
constexpr uint32_t kNibOffLo = 0x80088008u;  // -8 * 2^-24 twice
constexpr uint32_t kNibOffHi = 0x80808080u;  // -8 * 2^-20 twice

// Headroom of a column's reference over the maximum that moved it, in base-2
// units: weights are at most 1 and those of the moving maximum 2^-2.
constexpr float kQ4Head = 2.f;

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

// The fp16 MMA of decode_mma.cuh and its transpose of a fragment as pure
// operations: the two tiles of a pass are independent, and the compiler
// interleaves their chains only where nothing pins the order.
__device__ __forceinline__ void q4_mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                       uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// without an addend: D = A . B
__device__ __forceinline__ void q4_mma_z(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t q4_movm(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// The fp16 scales of one row's groups (K): GR / 2 words.
template <int GR>
__device__ __forceinline__ void lds_scales(uint32_t addr, uint32_t (&r)[GR / 2]) {
  if constexpr (GR == 4)
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(addr));
  else
    r[0] = lds32(addr);
}

// ldsm8_t of two 16 x 16 byte tiles: lanes 0-15 address the first one's rows,
// lanes 16-31 the second's; r0, r1 and r2, r3 as ldsm8_t gives them.
__device__ __forceinline__ void ldsm8_x2_t(uint32_t addr, uint32_t& r0, uint32_t& r1, uint32_t& r2,
                                           uint32_t& r3) {
  asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0, %1, %2, %3}, [%4];"
               : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
               : "r"(addr));
}

// mbar_wait_bounded for roles that wait most of their time: a failed try
// suspends the warp for up to the hinted time (it resumes when the phase
// completes) instead of polling, which takes issue slots from the warps that
// work; the clock is read between tries only.
__device__ __forceinline__ bool q4_try_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity), "r"(100000u)  // ns
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool q4_wait(uint64_t* bar, uint32_t parity) {
  if (q4_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  while (!q4_try_wait(bar, parity))
    if (globaltimer_ns() - t0 > kWaitLimitNs) return false;
  return true;
}

// Arrive `n` times.
__device__ __forceinline__ void mbar_arrive_n(uint64_t* bar, uint32_t n) {
  asm volatile(
      "{\n\t.reg .b64 st;\n\t"
      "mbarrier.arrive.release.cta.shared::cta.b64 st, [%0], %1;\n\t}" ::"r"(smem_u32(bar)),
      "r"(n)
      : "memory");
}

template <int D>
constexpr int decode_q4_smem_bytes() {
  using C = Q4Cfg<D>;
  return 2 * C::NS * C::SLOT_BYTES        // K and V stages
         + kQ4Warps * C::CC * D * 4         // combine: O per warp, CC columns at a time
         + kQ4Warps * 8 * 2 * 4             // combine: m, l per warp and column
         + 2 * C::NS * 8                    // mbarriers
         + kTableCache * 4                  // producer table cache
         + kPieceRing * (48 + 16)           // piece descriptors and their mbarriers
         + 64 + 128 + 16;                   // walk state, start record, alignment
}

// UR: q4_unit_rows of the pool's block size.
template <int D, int UR, bool PLAN>
__global__ void __launch_bounds__(kQ4Threads, kQ4CtasPerSm) decode_q4_kernel(const DecodeArgs a) {
  using C = Q4Cfg<D>;
  constexpr int NS = C::NS, GR = C::GR, PT = C::PT;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  unsigned char* k_st = smem_raw;
  unsigned char* v_st = k_st + NS * C::SLOT_BYTES;
  float* cmb_o = reinterpret_cast<float*>(v_st + NS * C::SLOT_BYTES);
  float* cmb_ml = cmb_o + kQ4Warps * C::CC * D;
  uint64_t* full = reinterpret_cast<uint64_t*>(cmb_ml + kQ4Warps * 8 * 2);
  uint64_t* empty = full + NS;
  long long* walk = reinterpret_cast<long long*>(empty + NS);
  int32_t* tcache = reinterpret_cast<int32_t*>(walk + 4);
  PlanStart* rec_s = reinterpret_cast<PlanStart*>(tcache + kTableCache);
  Piece* ring = reinterpret_cast<Piece*>(rec_s + 1);
  uint64_t* dfull = reinterpret_cast<uint64_t*>(ring + kPieceRing);
  uint64_t* dempty = dfull + kPieceRing;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int B = a.block_size;
  const int H = a.n_kv_heads, G = a.n_q_heads / H;
  constexpr int lur = ilog2(UR);
  constexpr uint32_t unit_bytes = static_cast<uint32_t>(UR) * C::ROW;

  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; ++i) {
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
        if (!q4_wait(&dempty[di], ((npub / kPieceRing) - 1) & 1)) {
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
    constexpr int UPS = C::TS / UR;  // units per slot
    const int KU = B / UR;           // units per block
    const unsigned char* pool = static_cast<const unsigned char*>(lane < 16 ? a.k_pool : a.v_pool);
    unsigned char* st = lane < 16 ? k_st : v_st;
    const long long pool_row = (long long)a.layer * a.n_blocks * H;  // chunks before the layer
    Piece p, pn;
    bool have = next_piece(p);
    if (have && !use_rec) tc.ensure(a.table, a.max_blocks, p.rep, p.b0, p.b0, lane);
    wait_previous_grid();
    publish(p, have);
    while (have) {
      const bool have_next = next_piece(pn);
      publish(pn, have_next);
      // lanes 0 .. 15 bring the K units of a slot, lanes 16 .. 31 the V units;
      // where a unit is goes before the wait for the slot, and no division by
      // the block size is on the way (KU = 1 for blocks of up to 64 tokens)
      const int u_first = p.b0 * KU;
      const int u_last = u_first + ((p.tok_end - p.b0 * B + UR - 1) >> lur) - 1;
      for (int u0 = u_first; u0 <= u_last; u0 += UPS) {
        const int u = u0 + (lane & 15);
        const int n_units = min(u_last + 1 - u0, UPS);
        const bool mine = (lane & 15) < n_units;
        const int j0 = KU == 1 ? u0 : u0 / KU, jl = KU == 1 ? u0 + n_units - 1 : (u0 + n_units - 1) / KU;
        const int j = KU == 1 ? u : u / KU;
        const int row = KU == 1 ? 0 : (u - j * KU) * UR;
        // the first slot of the record's piece takes the record's block ids
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
        const int slot = stage % NS;
        unsigned char* dst = st + slot * C::SLOT_BYTES + (lane & 15) * unit_bytes;
        if (stage >= NS && alive) {
          if (!q4_wait(&empty[slot], ((stage / NS) & 1) ^ 1)) {
            alive = false;
            if (lane == 0) record_status(a.status, 8);
          }
        }
        if (lane == 0) mbar_arrive_expect_tx(&full[slot], 2u * n_units * unit_bytes);
        __syncwarp();
        if (mine) {
          if (KU == 1) {
            bulk_load(dst, src, unit_bytes, &full[slot]);
          } else {  // part of a larger block: plane by plane
#pragma unroll
            for (int q = 0; q < GR; ++q) {
              bulk_load(dst + q * UR * 16, src + (q * B + row) * 16, UR * 16, &full[slot]);
              if (lane >= 16)
                bulk_load(dst + GR * UR * 16 + q * UR * 2, src + GR * B * 16 + (q * B + row) * 2,
                          UR * 2, &full[slot]);
            }
            if (lane < 16)
              bulk_load(dst + GR * UR * 16, src + GR * B * 16 + row * GR * 2, UR * GR * 2,
                        &full[slot]);
          }
        }
        ++stage;
      }
      p = pn;
      have = have_next;
    }
    const int first = stage > NS ? stage - NS : 0;
    for (int k = first; k < stage; ++k)
      q4_wait(&full[k % NS], (k / NS) & 1);
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
  int base = 0;  // slots before the piece
  // q of this warp's column of a piece (column wn * 8 + g): dimensions
  // 32 q + 8 t .. + 7 of each group, raw bf16
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
  // offsets inside a slot of what this lane reads of the first two tiles, and
  // the step to the next two
  auto unit_of = [](int r) -> uint32_t { return (r >> lur) * unit_bytes; };
  auto row_of = [](int r) -> uint32_t { return r & (UR - 1); };
  const int rk = (lane >> 4) * 16 + q4_srow(((lane >> 3) & 1) * 8 + (lane & 7));
  const int rv = (lane >> 4) * 16 + q4_vrow(lane & 15);
  const uint32_t at_kc = unit_of(rk) + row_of(rk) * 16, at_vc = unit_of(rv) + row_of(rv) * 16;
  uint32_t at_ks[2], at_vs[2];  // scales of K rows g, g + 8 and of V's token pairs
#pragma unroll
  for (int hi = 0; hi < 2; ++hi) {
    const int r = q4_srow(g + 8 * hi);
    at_ks[hi] = unit_of(r) + GR * UR * 16 + row_of(r) * GR * 2;
    const int rp = q4_srow(2 * t + 8 * hi);  // even: a pair never crosses a unit
    at_vs[hi] = unit_of(rp) + GR * UR * 16 + row_of(rp) * 2;
  }
  constexpr uint32_t tile_ks = UR >= 32 ? 16u * GR * 2 : (16u >> lur) * unit_bytes;
  constexpr uint32_t tile_vs = UR >= 32 ? 16u * 2 : (16u >> lur) * unit_bytes;
  constexpr uint32_t pair_c = UR >= 64 ? 32u * 16 : (32u >> lur) * unit_bytes;
  constexpr uint32_t pair_ks = UR >= 64 ? 32u * GR * 2 : (32u >> lur) * unit_bytes;
  constexpr uint32_t pair_vs = UR >= 64 ? 32u * 2 : (32u >> lur) * unit_bytes;
  int nread = 0;
  auto read_piece = [&](Piece& x) -> bool {
    const int di = nread % kPieceRing;
    if (alive && !q4_wait(&dfull[di], (nread / kPieceRing) & 1)) {
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
  Piece p;
  while (read_piece(p)) {
    uint4 qn[GR];
    load_q(p, qn);
    const int NT = p.ncols <= 8 ? 1 : (p.ncols <= 16 ? 2 : 4);  // n-tiles of the piece
    const int WT = kQ4Warps / NT;                                 // warps per n-tile
    const int wt = warp / NT;
    // Q fragments.  Column g is scaled by the power of two that brings its
    // largest |q| into [2^14, 2^15): bf16's 8 bits then stay exact in fp16
    // over 2^28 of range.  MMA 0 of a group takes dimensions 8t + {0, 4} and
    // {2, 6}, MMA 1 (the nibbles times 16) 8t + {1, 5} and {3, 7} over 16.
    uint32_t qf[GR][4];
    uint32_t qoff;   // offset fragment, see below
    float fcol[2];   // score factors of columns 2t and 2t + 1
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
      E = E < 14 ? 14 : E;
      const float sc = __uint_as_float(static_cast<uint32_t>(268 - E) << 23);  // 2^(141 - E)
      // S = 2^24 * 2^(E - 141) * accumulator, times the score scale
      const float f = a.qscale * __uint_as_float(static_cast<uint32_t>(E) << 23) * 0x1p10f;
      fcol[0] = __shfl_sync(0xffffffffu, f, 8 * t);
      fcol[1] = __shfl_sync(0xffffffffu, f, 8 * t + 4);
      float off[GR];
#pragma unroll
      for (int q = 0; q < GR; ++q) {
        const uint32_t w[4] = {qn[q].x, qn[q].y, qn[q].z, qn[q].w};
        float x[8];
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
        float sum = (half_lo(qf[q][0]) + half_hi(qf[q][0])) + (half_lo(qf[q][1]) + half_hi(qf[q][1]));
        sum += 16.f * ((half_lo(qf[q][2]) + half_hi(qf[q][2])) +
                       (half_lo(qf[q][3]) + half_hi(qf[q][3])));
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        off[q] = sum * (-8.f * 0x1p-24f);  // below 1: |q| < 2^15
      }
      // The offset of S is a product of its own, ks [16 x GR] . off [GR x 8],
      // one MMA: k-slots 2t, 2t + 1 take groups 2 (t & 1) and the next one, of
      // off's fp16 high part for t < 2 and of the rest (22 bits together)
      // above
      const float u0 = GR == 4 && (t & 1) ? off[GR - 2] : (t & 1) ? 0.f : off[0];
      const float u1 = GR == 4 && (t & 1) ? off[GR - 1] : (t & 1) ? 0.f : off[1];
      qoff = pack_f16(u0, u1);
      if (t >= 2) qoff = pack_f16(u0 - half_lo(qoff), u1 - half_hi(qoff));
    }
    float m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f};
    float o[C::MT][4];
#pragma unroll
    for (int mt = 0; mt < C::MT; ++mt) o[mt][0] = o[mt][1] = o[mt][2] = o[mt][3] = 0.f;

    // slot r of the ring goes to the warps with wt = r mod WT (one per n-tile)
    const int tok_first = p.b0 * B;
    const int n_slots = (p.tok_end - tok_first + C::TS - 1) / C::TS;
    for (int r = base + ((wt - base) & (WT - 1)); r < base + n_slots; r += WT) {
      const int slot = r % NS;
      if (alive && !q4_wait(&full[slot], (r / NS) & 1)) {
        alive = false;
        if (lane == 0) record_status(a.status, 8);
      }
      alive = __all_sync(0xffffffffu, alive);  // reconverge before ldmatrix / mma.sync
      const int nv = min(p.tok_end - (tok_first + (r - base) * C::TS), C::TS);
      const uint32_t kb = k_base + slot * C::SLOT_BYTES;
      const uint32_t vb = v_base + slot * C::SLOT_BYTES;
      // ---- S^T = K . Q^T, one accumulator per tile and group, weighted by
      // its rows' K scales
      float s[PT][4];
#pragma unroll
      for (int j = 0; j < PT / 2; ++j) {
        uint32_t sc[2][2][GR / 2];  // scales of rows g and g + 8 of each tile
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          lds_scales<GR>(kb + at_ks[0] + j * pair_ks + i * tile_ks, sc[i][0]);
          lds_scales<GR>(kb + at_ks[1] + j * pair_ks + i * tile_ks, sc[i][1]);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
          q4_mma_z(s[2 * j + i], GR == 4 && (t & 1) ? sc[i][0][GR / 2 - 1] : sc[i][0][0],
                   GR == 4 && (t & 1) ? sc[i][1][GR / 2 - 1] : sc[i][1][0], 0u, 0u, qoff, 0u);
#pragma unroll
        for (int q = 0; q < GR; ++q) {
          // ldmatrix: rows 0-7 and 8-15 of the first tile, then of the second
          uint32_t w[4];
          ldsm_x4(kb + at_kc + j * pair_c + q * UR * 16, w[0], w[1], w[2], w[3]);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t wa = w[2 * i], wb = w[2 * i + 1];
            const uint32_t wa8 = wa >> 8, wb8 = wb >> 8;
            float acc[4];
            q4_mma_z(acc, wa & kNibLo, wb & kNibLo, wa8 & kNibLo, wb8 & kNibLo, qf[q][0],
                     qf[q][1]);
            q4_mma(acc, wa & kNibHi, wb & kNibHi, wa8 & kNibHi, wb8 & kNibHi, qf[q][2], qf[q][3]);
            const float fl = q & 1 ? half_hi(sc[i][0][q / 2]) : half_lo(sc[i][0][q / 2]);
            const float fh = q & 1 ? half_hi(sc[i][1][q / 2]) : half_lo(sc[i][1][q / 2]);
            float(&x)[4] = s[2 * j + i];
            x[0] = fmaf(fl, acc[0], x[0]);
            x[1] = fmaf(fl, acc[1], x[1]);
            x[2] = fmaf(fh, acc[2], x[2]);
            x[3] = fmaf(fh, acc[3], x[3]);
          }
        }
      }
      // ---- mask: rows past the context, whatever their bytes hold
      if (nv < C::TS) {
#pragma unroll
        for (int i = 0; i < PT; ++i) {
          if (i * 16 + q4_srow(g) >= nv) s[i][0] = s[i][1] = -INFINITY;
          if (i * 16 + q4_srow(g + 8) >= nv) s[i][2] = s[i][3] = -INFINITY;
        }
        // and their V scales zero (a NaN times a zero weight would reach the
        // sum): every warp that reads the slot writes the same zeros, the fence
        // orders them before the copy that refills it
#pragma unroll
        for (int r0 = 0; r0 < C::TS; r0 += 32) {
          const int rr = r0 + lane;
          if (rr >= nv) {
            const uint32_t sa = vb + unit_of(rr) + GR * UR * 16 + row_of(rr) * 2;
#pragma unroll
            for (int q = 0; q < GR; ++q)
              asm volatile("st.shared.b16 [%0], %1;" ::"r"(sa + q * UR * 2), "h"(
                               static_cast<uint16_t>(0))
                           : "memory");
          }
        }
        fence_async_smem();
        __syncwarp();
      }
      // ---- reference of the weights, per column: p = 2^(s - m) with m the
      // maximum at its last move plus kQ4Head, moved when a score passes it.
      // So p <= 1 always (p times a scale stays inside fp16), the check is
      // one vote, and moves are rare once the first tokens have set it.
      float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
      for (int i = 0; i < PT; ++i) {
        mx0 = fmaxf(mx0, fmaxf(s[i][0], s[i][2]));
        mx1 = fmaxf(mx1, fmaxf(s[i][1], s[i][3]));
      }
      mx0 *= fcol[0];
      mx1 *= fcol[1];
      if (__any_sync(0xffffffffu, (mx0 > m_run[0]) | (mx1 > m_run[1]))) {
        float n0 = mx0, n1 = mx1;
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
          n0 = fmaxf(n0, __shfl_xor_sync(0xffffffffu, n0, off));
          n1 = fmaxf(n1, __shfl_xor_sync(0xffffffffu, n1, off));
        }
        n0 = n0 > m_run[0] ? n0 + kQ4Head : m_run[0];
        n1 = n1 > m_run[1] ? n1 + kQ4Head : m_run[1];
        const float al0 = exp2_approx(m_run[0] - n0), al1 = exp2_approx(m_run[1] - n1);
        m_run[0] = n0;
        m_run[1] = n1;
        l_run[0] *= al0;
        l_run[1] *= al1;
#pragma unroll
        for (int mt = 0; mt < C::MT; ++mt) {
          o[mt][0] *= al0;
          o[mt][1] *= al1;
          o[mt][2] *= al0;
          o[mt][3] *= al1;
        }
      }
      // ---- P^T in fp16 (11 bits), transposed: b[i][0] holds tokens
      // srow(2t), srow(2t + 1) of column g, b[i][1] srow(2t + 8), + 1
      uint32_t b[PT][2];
#pragma unroll
      for (int i = 0; i < PT; ++i) {
        const float p0 = exp2_approx(fmaf(s[i][0], fcol[0], -m_run[0]));
        const float p1 = exp2_approx(fmaf(s[i][1], fcol[1], -m_run[1]));
        const float p2 = exp2_approx(fmaf(s[i][2], fcol[0], -m_run[0]));
        const float p3 = exp2_approx(fmaf(s[i][3], fcol[1], -m_run[1]));
        l_run[0] += p0 + p2;
        l_run[1] += p1 + p3;
        b[i][0] = q4_movm(pack_f16(p0, p1));
        b[i][1] = q4_movm(pack_f16(p2, p3));
      }
      // ---- O^T += V^T . (P vs)^T per group.  The V scales of a token pair
      // are adjacent, so P' is one fp16 product per register (a second
      // rounding to 11 bits; p <= 1 and the scale is a finite fp16, so it
      // never overflows).
#pragma unroll
      for (int j = 0; j < PT / 2; ++j) {
#pragma unroll
        for (int q = 0; q < GR; ++q) {
          uint32_t w[4];
          ldsm8_x2_t(vb + at_vc + j * pair_c + q * UR * 16, w[0], w[1], w[2], w[3]);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t sa = vb + j * pair_vs + i * tile_vs + q * UR * 2;
            const uint32_t c0 = hmul2(b[2 * j + i][0], lds32(sa + at_vs[0]));
            const uint32_t c1 = hmul2(b[2 * j + i][1], lds32(sa + at_vs[1]));
            const uint32_t r0 = w[2 * i], r1 = w[2 * i + 1], r08 = r0 >> 8, r18 = r1 >> 8;
            q4_mma(o[2 * q], r0 & kNibLo, r0 & kNibHi, r08 & kNibLo, r08 & kNibHi, c0, c1);
            q4_mma(o[2 * q + 1], r1 & kNibLo, r1 & kNibHi, r18 & kNibLo, r18 & kNibHi, c0, c1);
            q4_mma(o[2 * q], kNibOffLo, kNibOffHi, kNibOffLo, kNibOffHi, c0, c1);
            q4_mma(o[2 * q + 1], kNibOffLo, kNibOffHi, kNibOffLo, kNibOffHi, c0, c1);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive_n(&empty[slot], WT);  // WT x NT = kQ4Warps
    }
    base += n_slots;
    // row g of m-tile 2q + h is dimension 32 q + 16 h + 2 g, row g + 8 the next
    // one (nibbles times 16)
#pragma unroll
    for (int mt = 0; mt < C::MT; ++mt)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        o[mt][i] *= i < 2 ? 0x1p24f : 0x1p20f;

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
