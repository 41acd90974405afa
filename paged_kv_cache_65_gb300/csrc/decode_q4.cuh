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
// so both products run on the nibbles themselves, and the offset 8 is a small
// product of the scales apart from them: for S the scales times the groups'
// sums of Q, one MMA per tile and n-tile; for O the scales' transpose times p,
// likewise, for all groups at once, beside the sum of p itself.
//
// Nibbles become fp16 MMA operands with one AND each: the fp16 bit pattern n
// (n < 16, exponent bits zero) is the subnormal n * 2^-24, and n << 4 is
// n * 2^-20, both exact MMA inputs.  The factors 2^-24 and 16 go into Q (scaled
// per column by a power of two, so that any magnitude of q stays inside fp16)
// and into the final scale of O.
//
// MMAs are m16n8k16 (fp16 in, f32 accumulate) per 16-token tile:
//     S^T [16 tokens x 8 cols] = K [16 x 32] . Q^T [32 x 8]   two per group
//     O^T [32 x 8 cols]       += V^T [32 x 16] . P'^T [16 x 8] two per group
// (e4m3 operands would take the nibbles with half the masks, but mma.sync of
// e4m3 converts them to fp16 here and ran slower: 49 against 43 us for the
// 131,071 tokens below.)
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
//
// What bounds it.  Narrow form (segments of up to 8 columns, three teams an
// SM): memory.  A longer context adds time at 6.8 TB/s of codes and scales (a
// pass that only copies: 7.0), and what is left of a call is its start, the
// pieces' ends and the merge pass, 8.6 us at 333 tokens.  37 sequences of 2K
// tokens, 8 K/V heads of 4 query heads: 27.0 us, 24 without any arithmetic;
// 131,071 tokens, 8 heads of 8: 39.6 us, 36 without arithmetic.  It took 30 and 43
// us with CTAs of 5 warps instead of teams: 128 registers a thread spilled, and
// the compiler could not overlap the tile's chains.
// Wide form (up to 32 columns, two teams an SM): instruction issue.  A pass of
// 32 tokens by 16 columns is 72 MMAs and about 420 other instructions, 1,250
// cycles with two warps a scheduler, the tensor pipe busy 46% of them.  12
// prefixes of 32,771 tokens by 32 columns: 209 us; with one n-tile a warp (the
// narrow form, unpacking everything four times) 298 us, with K and V converted
// to fp16 for tcgen05 (tensor and shared memory traffic for every value, roles
// waiting for one another) 276 us.
#pragma once

#include <cuda_fp16.h>

#include "decode_mma.cuh"

namespace pkv {

constexpr int kQ4Warps = 4;  // consumer warps of a team

// A CTA is several teams, each a CTA of the split by itself: four consumer
// warps (a warpgroup), a producer warp, its own stages and work.  The producers
// share the last warpgroup and pass their registers to the consumers.  NTW:
// 8-column tiles a consumer warp holds at once: two in the wide form, so that a
// tile of K and V is read and unpacked half as often; its O then takes 64
// registers, which leaves room for two teams (three spill and take as long).
template <bool WIDE>
struct Q4Team {
  static constexpr int TEAMS = WIDE ? 2 : 3;
  static constexpr int NTW = WIDE ? 2 : 1;
  static constexpr int NST = WIDE ? 5 : 3;                // stages in a team's ring
  static constexpr int THREADS = (TEAMS + 1) * 128;
  // registers a thread: at launch, consumers, producers
  static constexpr int REGS = WIDE ? 168 : 128, REGS_C = WIDE ? 216 : 144, REGS_P = WIDE ? 72 : 80;
  static_assert(TEAMS * REGS_C + REGS_P <= (TEAMS + 1) * REGS, "setmaxnreg waits for registers");
};

template <int D>
struct Q4Cfg {
  static constexpr int GR = D / 32;                // groups of 32 dimensions
  static constexpr int TS = 128;                   // tokens per stage
  static constexpr int ROW = D / 2 + D / 16;       // bytes per token row: codes and scales
  static constexpr int STAGE_BYTES = TS * ROW;     // K (or V) per stage
  static constexpr int MT = D / 16;                // m-tiles of O^T
  static constexpr int CC = 4;                     // columns per combine pass
  static_assert(D == 64 || D == 128, "head dim");
};

// Tokens per unit: a block when it has at most 64, else 64 (blocks of
// 128, 192 and 256).  A power of two.
__host__ __device__ constexpr int q4_unit_rows(int B) { return B < 64 ? B : 64; }

// Token order inside a 16-token tile: row k of S^T (and k-slot k of P'^T)
// stands for token q4_srow(k); lane i of ldsm8_t addresses token q4_vrow(i).
// ldsm8_t hands lane (g, t) the tokens of lanes 4t .. 4t + 3 as bytes 0 .. 3;
// bytes 0 and 2 become k-slots 2t and 2t + 1, bytes 1 and 3 k-slots 2t + 8 and
// 2t + 9: tokens 4t .. 4t + 3, whose four V scales are one 8-byte load.
__device__ __forceinline__ int q4_srow(int k) { return 4 * ((k >> 1) & 3) + 2 * (k >> 3) + (k & 1); }
__device__ __forceinline__ int q4_vrow(int i) { return (i & ~3) + 2 * (i & 1) + ((i >> 1) & 1); }

constexpr uint32_t kNibLo = 0x000f000fu;  // n * 2^-24
constexpr uint32_t kNibHi = 0x00f000f0u;  // n * 2^-20
constexpr uint32_t kByte = 0x00ff00ffu;   // (16 n' + n) * 2^-24, n' the high nibble

// Headroom of a column's largest weight over the maximum that set it, in
// base-2 units: the weights of a moved maximum are 2^(e - kQ4Head), e below.
constexpr float kQ4Head = 2.f;
// Weights go up to 2^e: 14 while every V scale seen is below 2 (bit 14 of an
// fp16), so that a weight times a scale stays in fp16's normal range far below
// the maximum however small the scales are; 0 from the first larger scale on.
constexpr float kQ4Exp = 14.f;

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 r;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(addr));
  return r;
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 r;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "r"(addr));
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
// Bytes 1 and 3 of a word as halves: the fp16 operands 16 n' + n of them.
__device__ __forceinline__ uint32_t q4_odd_bytes(uint32_t w) { return __byte_perm(w, 0, 0x4341); }
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

// q4_wait for the producer, whose ring gives it time: it sleeps between tries
__device__ __forceinline__ bool q4_wait_idle(uint64_t* bar, uint32_t parity) {
  const uint64_t t0 = globaltimer_ns();
  for (;;) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    if (ok) return true;
    if (globaltimer_ns() - t0 > kWaitLimitNs) return false;
    __nanosleep(300);
  }
}
// named_bar_sync that tells every thread whether `ok` holds for all of them.
__device__ __forceinline__ bool named_bar_all(int id, int n, bool ok) {
  uint32_t all;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %3, 0;\n\t"
      "barrier.cta.red.and.aligned.pred q, %1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(all)
      : "r"(id), "r"(n), "r"(static_cast<uint32_t>(ok))
      : "memory");
  return all != 0;
}

template <int D, bool WIDE>
constexpr int decode_q4_team_bytes() {
  using C = Q4Cfg<D>;
  using T = Q4Team<WIDE>;
  constexpr int n = 2 * T::NST * C::STAGE_BYTES       // K and V stages
                    + kQ4Warps * C::CC * D * 4        // combine: O per warp, CC columns at a time
                    + kQ4Warps * T::NTW * 8 * 2 * 4   // combine: m, l per warp and column
                    + (WIDE ? 2 * T::NTW * C::GR * 512 : 0)  // Q fragments of two sets
                    + 2 * T::NST * 8                  // mbarriers
                    + kTableCache * 4                 // producer table cache
                    + kPieceRing * (48 + 16)          // piece descriptors and their mbarriers
                    + 128;                            // start record
  return (n + 127) / 128 * 128;
}

// UR: q4_unit_rows of the pool's block size.
template <int D, int UR, bool PLAN, bool WIDE>
__global__ void __launch_bounds__(Q4Team<WIDE>::THREADS, 1) decode_q4_kernel(const DecodeArgs a) {
  using C = Q4Cfg<D>;
  using T = Q4Team<WIDE>;
  constexpr int NST = T::NST, GR = C::GR, NTW = T::NTW;
  extern __shared__ __align__(128) unsigned char smem_q4[];
  const int warp_cta = threadIdx.x >> 5;
  const bool is_producer = warp_cta >= T::TEAMS * 4;
  const int team = is_producer ? warp_cta - T::TEAMS * 4 : warp_cta >> 2;
  const int warp = warp_cta & 3;  // consumer warp of its team
  const int lane = threadIdx.x & 31;
  const int cta = blockIdx.x * T::TEAMS + team;  // of the split's a.grid
  unsigned char* k_st = smem_q4 + team * decode_q4_team_bytes<D, WIDE>();
  unsigned char* v_st = k_st + NST * C::STAGE_BYTES;
  float* cmb_o = reinterpret_cast<float*>(v_st + NST * C::STAGE_BYTES);
  float* cmb_ml = cmb_o + kQ4Warps * C::CC * D;
  uint4* q_frag = reinterpret_cast<uint4*>(cmb_ml + kQ4Warps * NTW * 8 * 2);
  uint64_t* full = reinterpret_cast<uint64_t*>(q_frag + (WIDE ? 2 * NTW * GR * 32 : 0));
  uint64_t* empty = full + NST;
  uint64_t* dfull = empty + NST;
  uint64_t* dempty = dfull + kPieceRing;
  PlanStart* rec_s = reinterpret_cast<PlanStart*>(dempty + kPieceRing);
  Piece* ring = reinterpret_cast<Piece*>(rec_s + 1);
  int32_t* tcache = reinterpret_cast<int32_t*>(ring + kPieceRing);

  const int B = a.block_size;
  const int H = a.n_kv_heads, G = a.n_q_heads / H;
  constexpr int lur = ilog2(UR);
  constexpr uint32_t unit_bytes = static_cast<uint32_t>(UR) * C::ROW;

  const bool use_rec = PLAN && a.starts != nullptr && a.start_grid == a.grid;
  if (is_producer) {
    // tables and lengths that kernels before this one write (a pool with device
    // tables) are read only after them; host-written ones before the wait, as in
    // decode_mma.cuh
    if (a.meta_wait) griddep_wait();
    if (use_rec && team < T::TEAMS)
      reinterpret_cast<int32_t*>(rec_s)[lane] =
          reinterpret_cast<const int32_t*>(a.starts + cta)[lane];
  }
  if (is_producer && team < T::TEAMS && lane == 0) {
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
  __syncthreads();

  auto wait_previous_grid = [&]() {
    griddep_wait();
    griddep_launch_dependents();
    if constexpr (!PLAN) {
      if (cta == 0 && !is_producer && warp == 0)
        write_prefix(a.ctx, a.n_seq, B, H, a.max_blocks, a.ws_pre);
    }
  };

  if (is_producer) {
    // ------------------------------------------------------------ producer
    reg_dealloc<T::REGS_P>();
    if (team >= T::TEAMS) return;  // a warp without a team
    PieceWalker pw;
    PlanWalker plw;
    if constexpr (PLAN) {
      const long long W = a.plan_W;
      long long chunk = (W + a.grid - 1) / a.grid;
      if (chunk < a.min_chunk) chunk = a.min_chunk;
      const long long r0 = (long long)cta * chunk;
      plw.segs = a.segs;
      plw.n_segs = a.n_segs;
      plw.B = B;
      plw.r = r0;
      plw.r1 = r0 + chunk < W ? r0 + chunk : W;
      plw.s = 0;
      if (!use_rec) plw.s = r0 < W ? plan_find(a.segs, a.n_segs, r0) : a.n_segs;
    } else {
      const WalkStart w = find_start<true>(a.ctx, a.n_seq, B, H, a.max_blocks, a.grid, cta, a.status);
      const long long r0 = (long long)cta * w.chunk;
      pw.ctx = a.ctx;
      pw.n_seq = a.n_seq;
      pw.B = B;
      pw.H = H;
      pw.max_blocks = a.max_blocks;
      pw.s = w.s;
      pw.pre = w.pre;
      pw.r = r0;
      pw.r1 = r0 + w.chunk < w.W ? r0 + w.chunk : w.W;
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
    // pieces go to the consumers as descriptors, published after the first
    // copies of the piece before (finding one reads the plan or the lengths);
    // rep = -1 ends the list
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
    // lanes 0 .. 15 bring the K units of a slot, lanes 16 .. 31 the V units;
    // where a unit is goes before the wait for the slot, and no division by the
    // block size is on the way (KU = 1 for blocks of up to 64 tokens)
    auto copy_slot = [&](int u0, int u_last) {
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
      const int slot = stage % NST;
      unsigned char* dst = st + slot * C::STAGE_BYTES + (lane & 15) * unit_bytes;
      if (stage >= NST && alive) {
        if (!q4_wait_idle(&empty[slot], ((stage / NST) & 1) ^ 1)) {
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
    };
    bool have = next_piece(p);
    if (have && !use_rec) tc.ensure(a.table, a.max_blocks, p.rep, p.b0, p.b0, lane);
    wait_previous_grid();
    publish(p, have);
    while (have) {
      bool have_next = false;
      const int u_first = p.b0 * KU;
      const int u_last = u_first + ((p.tok_end - p.b0 * B + UR - 1) >> lur) - 1;
      // (a piece may hold no block: work units are finer)
      for (int u0 = u_first; u0 <= u_last || u0 == u_first; u0 += UPS) {
        if (u0 <= u_last) copy_slot(u0, u_last);
        if (u0 == u_first) {
          have_next = next_piece(pn);
          publish(pn, have_next);
        }
      }
      p = pn;
      have = have_next;
    }
    const int first = stage > NST ? stage - NST : 0;
    for (int k = first; k < stage; ++k)
      q4_wait(&full[k % NST], (k / NST) & 1);
    return;
  }

  // -------------------------------------------------------------- consumers
  reg_alloc<T::REGS_C>();
  wait_previous_grid();
  const int g = lane >> 2;  // groupID: row of A / C, column of B
  const int t = lane & 3;   // thread in group
  const uint32_t k_base = smem_u32(k_st);
  const int cstride = PLAN ? a.c_max : G;  // columns per workspace slot
  bool alive = true;
  int slot = 0;        // stage being read
  uint32_t phase = 0;  // and the parity of its full barrier
  // n-tiles are dealt to the warps NTW at a time (a set); warps that share a set
  // split its tokens.  q of this warp's column g of the set's tile j: dimensions
  // 32 q + 8 t .. + 7 of each group, raw bf16
  auto n_sets = [&](const Piece& pc) {
    const int nt = pc.ncols <= 8 ? 1 : (pc.ncols <= 16 ? 2 : 4);
    return nt <= NTW ? 1 : nt / NTW;
  };
  auto load_q = [&](const Piece& pc, int j, uint4 (&qr)[GR]) {
    const int col = ((warp % n_sets(pc)) * NTW + j) * 8 + g;
    const bool colv = col < pc.ncols;
    int seqm = pc.rep, gi = col;
    if constexpr (PLAN) {
      const int mi = col / G;
      gi = col - mi * G;
      // the first member is the piece's own row
      if (mi > 0) seqm = colv ? a.members[pc.mem + mi] : 0;
    }
    const uint4* qw = reinterpret_cast<const uint4*>(
        static_cast<const unsigned char*>(a.q) +
        ((long long)seqm * a.n_q_heads + (long long)pc.head * G + (colv ? gi : 0)) * D * 2);
#pragma unroll
    for (int q = 0; q < GR; ++q) qr[q] = colv ? qw[q * 4 + t] : make_uint4(0u, 0u, 0u, 0u);
  };
  // shared offset of token r's unit and its row inside the unit
  auto unit_of = [&](int r) -> uint32_t { return (r >> lur) * unit_bytes; };
  auto row_of = [&](int r) -> uint32_t { return r & (UR - 1); };
  // offsets inside a stage of what this lane reads of the pass at token tb;
  // those of a warp's first pass are kept (a narrow piece has no other)
  struct Offsets {
    int tb;
    uint32_t kc, vc;        // K and V codes (lane's row of the matrix loads)
    uint32_t ks, vs;        // scales of K row g (g + 8: two tokens on), of V's four tokens
    uint32_t vo;            // V scales of group g & 3 (rows of the offset's MMA)
  };
  auto offsets = [&](int tb) -> Offsets {
    Offsets x;
    x.tb = tb;
    const int rk = tb + (lane >> 4) * 16 + q4_srow(((lane >> 3) & 1) * 8 + (lane & 7));
    const int rv = tb + (lane >> 4) * 16 + q4_vrow(lane & 15);
    x.kc = unit_of(rk) + row_of(rk) * 16;
    x.vc = unit_of(rv) + row_of(rv) * 16;
    const int rs = tb + q4_srow(g);
    x.ks = unit_of(rs) + GR * UR * 16 + row_of(rs) * GR * 2;
    const int rp = tb + 4 * t;  // four tokens never cross a unit
    x.vs = unit_of(rp) + GR * UR * 16 + row_of(rp) * 2;
    x.vo = x.vs + (g & (GR - 1)) * UR * 2;
    return x;
  };
  // from a pass's first tile to its second
  constexpr uint32_t tile_ks = UR >= 32 ? 16u * GR * 2 : (16u >> lur) * unit_bytes;
  constexpr uint32_t tile_vs = UR >= 32 ? 16u * 2 : (16u >> lur) * unit_bytes;
  int nread = 0;
  auto read_piece = [&](Piece& x) -> bool {
    const int di = nread % kPieceRing;
    if (alive && !q4_wait(&dfull[di], (nread / kPieceRing) & 1)) {
      alive = false;
      if (lane == 0) record_status(a.status, 8);
    }
    // a wait that gave up ends the team as a whole, between pieces: its warps
    // meet in barriers inside one
    __syncwarp();
    alive = named_bar_all(1 + team, kQ4Warps * 32, alive);
    if (!alive) return false;
    x = ring[di];
    __syncwarp();
    if (lane == 0) mbar_arrive(&dempty[di]);
    ++nread;
    return x.rep >= 0;
  };
  Piece p;
  while (read_piece(p)) {
    uint4 qn[NTW][GR];
#pragma unroll
    for (int j = 0; j < NTW; ++j) load_q(p, j, qn[j]);
    const int NP = n_sets(p);       // sets of n-tiles of the piece
    const int WT = kQ4Warps / NP;   // warps per set
    const int wt = warp / NP;
    // Q fragments.  Column g is scaled by the power of two that brings its
    // largest |q| into [2^14, 2^15): bf16's 8 bits then stay exact in fp16
    // over 2^28 of range.  MMA 0 of a group takes dimensions 8t + {0, 4} and
    // {2, 6}, MMA 1 (the nibbles times 16) 8t + {1, 5} and {3, 7} over 16.
    uint32_t qf[NTW][GR][4];
    uint32_t qoff[NTW];   // offset fragment, see below
    float fcol[NTW][2];   // score factors of columns 2t and 2t + 1
#pragma unroll
    for (int j = 0; j < NTW; ++j) {
      uint32_t am = 0;
#pragma unroll
      for (int q = 0; q < GR; ++q) {
        const uint32_t w[4] = {qn[j][q].x, qn[j][q].y, qn[j][q].z, qn[j][q].w};
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
      fcol[j][0] = __shfl_sync(0xffffffffu, f, 8 * t);
      fcol[j][1] = __shfl_sync(0xffffffffu, f, 8 * t + 4);
      float off[GR];
#pragma unroll
      for (int q = 0; q < GR; ++q) {
        const uint32_t w[4] = {qn[j][q].x, qn[j][q].y, qn[j][q].z, qn[j][q].w};
        uint32_t(&qx)[4] = qf[j][q];
        float x[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u) * sc * 0.0625f;
          x[2 * i] = __uint_as_float(w[i] << 16) * sc;
        }
        qx[0] = pack_f16(x[0], x[4]);
        qx[1] = pack_f16(x[2], x[6]);
        qx[2] = pack_f16(x[1], x[5]);
        qx[3] = pack_f16(x[3], x[7]);
        // the offset's sum takes the values the MMAs take (as rounded)
        float sum = (half_lo(qx[0]) + half_hi(qx[0])) + (half_lo(qx[1]) + half_hi(qx[1]));
        sum += 16.f * ((half_lo(qx[2]) + half_hi(qx[2])) + (half_lo(qx[3]) + half_hi(qx[3])));
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
      qoff[j] = pack_f16(u0, u1);
      if (t >= 2) qoff[j] = pack_f16(u0 - half_lo(qoff[j]), u1 - half_hi(qoff[j]));
    }
    Offsets at = offsets((wt & 1) * 32);
    // WIDE: the fragments go through shared memory, which leaves the registers to
    // O; the warps of a set hold the same ones
    const uint32_t q_addr = smem_u32(q_frag) + ((warp % NP) * NTW * GR * 32 + lane) * 16;
    if constexpr (WIDE) {
      if (wt == 0) {
#pragma unroll
        for (int j = 0; j < NTW; ++j)
#pragma unroll
          for (int q = 0; q < GR; ++q)
            q_frag[((warp % NP) * NTW * GR + j * GR + q) * 32 + lane] =
                make_uint4(qf[j][q][0], qf[j][q][1], qf[j][q][2], qf[j][q][3]);
      }
      named_bar_sync(1 + team, kQ4Warps * 32);
    }
    float m_run[NTW][2];
    float e_run = kQ4Exp;  // weights are at most 2^e_run
    float o[NTW][C::MT][4];
#pragma unroll
    for (int j = 0; j < NTW; ++j) {
      m_run[j][0] = m_run[j][1] = -INFINITY;
#pragma unroll
      for (int mt = 0; mt < C::MT; ++mt) o[j][mt][0] = o[j][mt][1] = o[j][mt][2] = o[j][mt][3] = 0.f;
    }
    // The offset's part of O, -8 sum_t vs[t][q] p[t], is the same for every
    // dimension of a group: an MMA with the V scales as its rows, one for all
    // groups (rows 0 .. 3, row q & (GR - 1)); its row 4 is ones and sums the
    // weights.  The offset is kept apart from O and added every few stages: summed
    // apart over a long piece the two would cancel to a small rest of large sums
    // (1.8x the error at 32,771 tokens).
    const uint32_t one = g == 4 ? 0x3c003c00u : 0u, gm = g < 4 ? 0xffffffffu : 0u;
    float ov[NTW][4];  // rows 8 .. 15, the upper half, repeat and are not used
#pragma unroll
    for (int j = 0; j < NTW; ++j) ov[j][0] = ov[j][1] = ov[j][2] = ov[j][3] = 0.f;
    auto fold = [&]() {
#pragma unroll
      for (int j = 0; j < NTW; ++j)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
#pragma unroll
          for (int q = 0; q < GR; ++q) {
            const float x = __shfl_sync(0xffffffffu, ov[j][k], 4 * q + t);
            o[j][2 * q][k] = fmaf(x, -8.f * 0x1p-24f, o[j][2 * q][k]);
            o[j][2 * q + 1][k] = fmaf(x, -8.f * 0x1p-24f, o[j][2 * q + 1][k]);
            o[j][2 * q][2 + k] = fmaf(x, -136.f * 0x1p-24f, o[j][2 * q][2 + k]);
            o[j][2 * q + 1][2 + k] = fmaf(x, -136.f * 0x1p-24f, o[j][2 * q + 1][2 + k]);
          }
          if (g < 4) ov[j][k] = 0.f;
        }
    };

    for (int tok0 = p.b0 * B; tok0 < p.tok_end; tok0 += C::TS) {
      if (alive && !q4_wait(&full[slot], phase)) {
        alive = false;
        if (lane == 0) record_status(a.status, 8);
      }
      alive = __all_sync(0xffffffffu, alive);  // reconverge before ldmatrix / mma.sync
      const int nvalid = p.tok_end - tok0 < C::TS ? p.tok_end - tok0 : C::TS;
      // two 16-token tiles a pass: their chains of MMAs interleave, and one
      // check of the running maximum covers both
#pragma unroll 1
      for (int tb = wt * 32; tb < nvalid; tb += WT * 32) {
        const int nv = nvalid - tb;  // tokens of the pass inside the context (>= 1)
        // 64 tokens on are whole units on: only a warp that takes every pass (WT =
        // 1) meets other offsets
        if ((tb & 32) != at.tb) at = offsets(tb & 32);
        const uint32_t kb =
            k_base + slot * C::STAGE_BYTES + (tb >> 6) * ((64 >> lur) * unit_bytes);
        const uint32_t vb = kb + NST * C::STAGE_BYTES;
        // past the context: V scales zero, whatever the bytes hold (a NaN times
        // a zero weight would reach the sum).  This warp alone reads them, the
        // fence orders the writes before the copy that refills the stage.
        if (nv < 32) {
          if (lane >= nv) {
            const int r = (tb & 32) + lane;
            const uint32_t sa = vb + unit_of(r) + GR * UR * 16 + row_of(r) * 2;
#pragma unroll
            for (int q = 0; q < GR; ++q)
              asm volatile("st.shared.b16 [%0], %1;" ::"r"(sa + q * UR * 2), "h"(
                               static_cast<uint16_t>(0))
                           : "memory");
          }
          fence_async_smem();
          __syncwarp();
        }
        // V scales of group g & 3 and four tokens of each tile: over the lanes all
        // of the pass
        uint2 so[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) so[i] = lds64(vb + at.vo + i * tile_vs);
        // ---- S^T = K . Q^T per tile: one accumulator per group, weighted by
        // its rows' K scales
        float s[NTW][2][4];
        {
          // ldmatrix: rows 0-7 and 8-15 of the first tile, then of the second
          const uint32_t ka = kb + at.kc;
          uint32_t sc[2][2][GR / 2];  // scales of rows g and g + 8 of each tile
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            lds_scales<GR>(kb + at.ks + i * tile_ks, sc[i][0]);
            lds_scales<GR>(kb + at.ks + i * tile_ks + 4 * GR, sc[i][1]);
          }
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < NTW; ++j)
              q4_mma_z(s[j][i], GR == 4 && (t & 1) ? sc[i][0][GR / 2 - 1] : sc[i][0][0],
                       GR == 4 && (t & 1) ? sc[i][1][GR / 2 - 1] : sc[i][1][0], 0u, 0u, qoff[j],
                       0u);
#pragma unroll
          for (int q = 0; q < GR; ++q) {
            uint32_t w[4];
            ldsm_x4(ka + q * UR * 16, w[0], w[1], w[2], w[3]);
            uint4 fq[NTW];
#pragma unroll
            for (int j = 0; j < NTW; ++j)
              fq[j] = WIDE ? lds128(q_addr + (j * GR + q) * 512)
                           : make_uint4(qf[j][q][0], qf[j][q][1], qf[j][q][2], qf[j][q][3]);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint32_t wa = w[2 * i], wb = w[2 * i + 1];
              const uint32_t wa8 = wa >> 8, wb8 = wb >> 8;
              const float fl = q & 1 ? half_hi(sc[i][0][q / 2]) : half_lo(sc[i][0][q / 2]);
              const float fh = q & 1 ? half_hi(sc[i][1][q / 2]) : half_lo(sc[i][1][q / 2]);
#pragma unroll
              for (int j = 0; j < NTW; ++j) {
                float acc[4];
                q4_mma_z(acc, wa & kNibLo, wb & kNibLo, wa8 & kNibLo, wb8 & kNibLo, fq[j].x,
                         fq[j].y);
                q4_mma(acc, wa & kNibHi, wb & kNibHi, wa8 & kNibHi, wb8 & kNibHi, fq[j].z, fq[j].w);
                s[j][i][0] = fmaf(fl, acc[0], s[j][i][0]);
                s[j][i][1] = fmaf(fl, acc[1], s[j][i][1]);
                s[j][i][2] = fmaf(fh, acc[2], s[j][i][2]);
                s[j][i][3] = fmaf(fh, acc[3], s[j][i][3]);
              }
            }
          }
        }
        if (nv < 32) {  // rows past the context
#pragma unroll
          for (int j = 0; j < NTW; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              if (i * 16 + q4_srow(g) >= nv) s[j][i][0] = s[j][i][1] = -INFINITY;
              if (i * 16 + q4_srow(g + 8) >= nv) s[j][i][2] = s[j][i][3] = -INFINITY;
            }
        }
        // ---- reference of the weights, per column: p = 2^(s - m), m the
        // maximum at its last move plus kQ4Head less e_run, moved when a score
        // passes m + e_run or e_run changes.  So p <= 2^e_run always, the check
        // is one vote, and moves are rare once the first tokens have set it.
        float mx[NTW][2];
        const bool big =
            ((so[0].x | so[0].y | so[1].x | so[1].y) & 0x40004000u) != 0 && e_run > 0.f;
        bool move = big;
#pragma unroll
        for (int j = 0; j < NTW; ++j)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            mx[j][k] = fmaxf(fmaxf(s[j][0][k], s[j][0][2 + k]), fmaxf(s[j][1][k], s[j][1][2 + k])) *
                       fcol[j][k];
            move |= mx[j][k] > m_run[j][k] + e_run;
          }
        if (__any_sync(0xffffffffu, move)) {
          const float e_old = e_run;
          if (__any_sync(0xffffffffu, big)) e_run = 0.f;
          fold();
#pragma unroll
          for (int j = 0; j < NTW; ++j)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              float n = mx[j][k];
#pragma unroll
              for (int off = 4; off < 32; off <<= 1)
                n = fmaxf(n, __shfl_xor_sync(0xffffffffu, n, off));
              n = (n > m_run[j][k] + e_old ? n + kQ4Head : m_run[j][k] + e_old) - e_run;
              const float al = exp2_approx(m_run[j][k] - n);
              m_run[j][k] = n;
              ov[j][k] *= al;  // the sum of weights
#pragma unroll
              for (int mt = 0; mt < C::MT; ++mt) {
                o[j][mt][k] *= al;
                o[j][mt][2 + k] *= al;
              }
            }
        }
        // ---- P^T in fp16 (11 bits), transposed: b[.][i][0] holds tokens
        // srow(2t), srow(2t + 1) of column g, b[.][i][1] srow(2t + 8), + 1
        uint32_t b[NTW][2][2];
#pragma unroll
        for (int j = 0; j < NTW; ++j)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float p0 = exp2_approx(fmaf(s[j][i][0], fcol[j][0], -m_run[j][0]));
            const float p1 = exp2_approx(fmaf(s[j][i][1], fcol[j][1], -m_run[j][1]));
            const float p2 = exp2_approx(fmaf(s[j][i][2], fcol[j][0], -m_run[j][0]));
            const float p3 = exp2_approx(fmaf(s[j][i][3], fcol[j][1], -m_run[j][1]));
            b[j][i][0] = q4_movm(pack_f16(p0, p1));
            b[j][i][1] = q4_movm(pack_f16(p2, p3));
          }
        // ---- O^T += V^T . (P vs)^T per group.  The V scales of a lane's four
        // tokens are adjacent, so P' is one fp16 product per register (a second
        // rounding to 11 bits; p times a scale stays inside fp16).  Row g of a
        // tile takes the low nibbles, row g + 8 the whole bytes 16 n' + n: four
        // operations a word of eight nibbles, and the low ones are taken off
        // again at the end.
        {
          const uint32_t va = vb + at.vc;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t a0 = (so[i].x & gm) | one, a2 = (so[i].y & gm) | one;
#pragma unroll
            for (int j = 0; j < NTW; ++j) q4_mma(ov[j], a0, a0, a2, a2, b[j][i][0], b[j][i][1]);
          }
#pragma unroll
          for (int q = 0; q < GR; ++q) {
            uint32_t w[4];
            ldsm8_x2_t(va + q * UR * 16, w[0], w[1], w[2], w[3]);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint2 sv = lds64(vb + at.vs + i * tile_vs + q * UR * 2);
              const uint32_t r0 = w[2 * i], r1 = w[2 * i + 1];
              const uint32_t r08 = q4_odd_bytes(r0), r18 = q4_odd_bytes(r1);
#pragma unroll
              for (int j = 0; j < NTW; ++j) {
                const uint32_t c0 = hmul2(b[j][i][0], sv.x), c1 = hmul2(b[j][i][1], sv.y);
                q4_mma(o[j][2 * q], r0 & kNibLo, r0 & kByte, r08 & kNibLo, r08, c0, c1);
                q4_mma(o[j][2 * q + 1], r1 & kNibLo, r1 & kByte, r18 & kNibLo, r18, c0, c1);
              }
            }
          }
        }
      }
      if ((tok0 / C::TS & 7) == 7) fold();
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[slot]);
      if (++slot == NST) {
        slot = 0;
        phase ^= 1;
      }
    }
    // row g of m-tile 2q + h is dimension 32 q + 16 h + 2 g, row g + 8, less
    // row g, the next one times 16
    fold();
#pragma unroll
    for (int j = 0; j < NTW; ++j)
#pragma unroll
      for (int mt = 0; mt < C::MT; ++mt)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          o[j][mt][2 + k] = (o[j][mt][2 + k] - o[j][mt][k]) * 0x1p20f;
          o[j][mt][k] *= 0x1p24f;
        }

    // ---- combine the states of the warps that share a set
#pragma unroll
    for (int j = 0; j < NTW; ++j)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if (g == 4) {
          cmb_ml[((warp * NTW + j) * 8 + 2 * t + k) * 2] = m_run[j][k];
          cmb_ml[((warp * NTW + j) * 8 + 2 * t + k) * 2 + 1] = ov[j][k];
        }
      }
    const long long slot_id = (long long)cta + p.seg;
#pragma unroll
    for (int j = 0; j < NTW; ++j) {
      for (int pc = 0; pc < 8; pc += C::CC) {
        if (j * 8 + pc >= p.ncols) break;  // no column of any set in this pass
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int c8 = 2 * t + k;
          if (c8 >= pc && c8 < pc + C::CC) {
#pragma unroll
            for (int mt = 0; mt < C::MT; ++mt)
              *reinterpret_cast<float2*>(&cmb_o[(warp * C::CC + c8 - pc) * D + mt * 16 + 2 * g]) =
                  make_float2(o[j][mt][k], o[j][mt][2 + k]);
          }
        }
        named_bar_sync(1 + team, kQ4Warps * 32);
        constexpr int D4 = D / 4;
        for (int idx = threadIdx.x & (kQ4Warps * 32 - 1); idx < NP * C::CC * D4;
             idx += kQ4Warps * 32) {
          const int set = idx / (C::CC * D4);
          const int rem = idx - set * C::CC * D4;
          const int cc = rem / D4, d = (rem - cc * D4) * 4;
          const int col = (set * NTW + j) * 8 + pc + cc;
          if (col >= p.ncols) continue;
          float M = -INFINITY;
          for (int i = 0; i < WT; ++i)
            M = fmaxf(M, cmb_ml[(((set + i * NP) * NTW + j) * 8 + pc + cc) * 2]);
          float L = 0.f;
          float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int i = 0; i < WT; ++i) {
            const int w = set + i * NP;
            const float* ml = &cmb_ml[((w * NTW + j) * 8 + pc + cc) * 2];
            const float f = ml[0] == -INFINITY ? 0.f : exp2_approx(ml[0] - M);
            L += f * ml[1];
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
        named_bar_sync(1 + team, kQ4Warps * 32);
      }
    }
  }
}

}  // namespace pkv
