// Attention of drafted tokens over a paged latent cache on tcgen05 (bf16 in,
// fp32 accumulate): for token t of sequence b and head h, over the cached rows
// and the drafted rows that t sees,
//   x_s = scale q[t,h].k_s,  out = sum_s exp(x_s - m) k_s[:512] / l.
// The heads of all drafted tokens of a sequence share the sequence's keys, so
// its T * H query rows are cut into tiles of 128 and each tile runs over the
// keys in blocks of 112 slots, cached blocks first, then drafted ones.
//
// Work split.  One CTA pair per two SMs; the (tile, block) pairs of the whole
// batch form one list, cut into equal runs, one per CTA pair, whatever the
// lengths are (the lengths live on the device: every pair finds its run by
// itself).  A run covers whole tiles and, at its ends, parts of a tile, whose
// unnormalised O, running maximum and sum go to the workspace and are joined
// by tree_join_kernel.  The order of every sum follows from the lengths alone.
//
// MMA layout (two-CTA MMAs, M = 128 = 64 rows per CTA, issued by CTA 0).  B is
// split by N between the CTAs' shared memories, and each CTA's accumulator
// keeps its 64 rows twice over the 128 TMEM lanes: lanes 0..63 pair with CTA
// 0's half of B, lanes 64..127 with CTA 1's.  CTA c holds columns D_c of every
// key: value columns [256c, 256c+256) and rope columns [512+32c, 512+32c+32),
// so a key row crosses from L2 into shared memory once per pair:
//   logits: A in TMEM, lanes h / 64+h hold row h's columns D_0 / D_1; lane h
//     ends with the partial logit over D_0, lane 64+h with the one over D_1;
//     the softmax warps add the two through shared memory;
//   O += P V: N = 256 value columns, CTA 0's half of B in lanes 0..63, CTA 1's
//     in lanes 64..127; 2 MMAs per 16 slots cover the 512 columns in 256 TMEM
//     columns.
// TMEM: O 256 + logits 112 + query 144 columns.  Three key stages, two P
// buffers; the logits of block j+1 run during the softmax of block j.  112 slots:
// what 512 TMEM columns leave for the logits, and N = 2 x 112 runs at full rate.
//
// Keys arrive by TMA straight from the pages (which hold a multiple of 16
// rows): one copy brings 16 or 32 rows x 256 value columns, already as the
// tensor cores read them, [8-row group][64 columns][8 rows], one more their
// rope columns.  Few large copies matter: issuing one holds the issuing thread
// for about 180 cycles whatever its size (measured without any other work: 32
// rows from one thread 55 bytes per cycle and SM, with the rope columns from a
// second warp 69; 16 rows 34; 16 x 64 pieces 21, which bounded the whole loop).
// What a masked place holds never reaches the sums.  Its logit is masked; and
// where a 16-slot step of P V has a slot past the last row, on an unusable
// page, or seen by no token of the tile, the slot's value columns are zeroed in
// shared memory before the tensor cores read them (steps without any seen slot
// are not run).  A drafted row with an infinity or NaN that only some of the
// tile's tokens see is zeroed too, and the tokens that see it get NaN.
//
// A tile's query takes a slot of the key ring ahead of its keys: 448 of its value
// columns come by TMA, and the fix warps move them into TMEM, with the other 64
// and the rope columns from registers, once the last logits of the tile before
// have read the old query (per-row loads of the softmax warps took 4,200 cycles
// between two tiles).
//
// Bound.  A block's MMAs take 1,956 cycles back to back (logits 1,008, P V 896);
// the loop takes about 2,800 per block (keys from L2) to 3,050 (from HBM), a tile
// change some 5,500 more.  The loop is the softmax warps' chain of waits: logits
// out of TMEM, the exchange through shared memory (whose bandwidth the operands'
// reads, the copies and the exchange use to two thirds), P back, and the signals
// between the CTAs.  Measured, each call on other inputs than the last: 16 trees of 48
// tokens over 2K-6K rows, 128 heads, 714 us = 1,230 TFLOP/s (the same inputs again and
// again: 673 us); 64 single tokens over 1K-16K rows 152 us = 4.3 TB/s and 1,010 TFLOP/s
// (12 us of it the join; tensor pipes 53 % and DRAM 61 % busy); one token over 1K rows
// 15 us (the two launches, one tile, the join); 1,024 tokens after 16K rows 3,220 us =
// 1,500 TFLOP/s.  A prompt's first 2,048 tokens take 1,080 us, 540 TFLOP/s: their blocks
// are drafted ones, whose copies are of 8 rows and pass the fix warps.
//
// A wait tests the parity of a barrier's phase: no barrier may complete two phases ahead
// of a waiting thread.  tests/test_tree_ring.py models the roles' order of waits and
// arrivals for that; a change of either belongs in both.
//
// Roles per CTA: warp 0 = TMEM allocation, MMA issuer of the logits (CTA 0);
// warps 1..4 = query into TMEM, passing on of key stages (with the zeroing
// above); warps 5..20 = softmax and epilogue; warp 21 = MMA issuer of P V (CTA
// 0); warps 22, 23 = loads (value columns and query; rope columns and schedule).
#include <math.h>
#include <stddef.h>

#include "tree_attn.cuh"

namespace dsa {
namespace tree {

constexpr int kHC = 64, kTile = 128, kDQK = 576, kDV = 512;
constexpr int kBlk = 112, kGroups = kBlk / 16;
constexpr int kStages = 3;
constexpr int kAtom = 8 * 128;                     // 8 slots x 64 value columns (SW128 rows)
constexpr int kOct = 4 * kAtom;                    // 8 slots x the CTA's 256 value columns
constexpr int kValue = kBlk / 8 * kOct;            // value part of a stage: [8-slot group][64 columns][8 slots]
constexpr int kRope = kBlk * 64;                   // 112 slots x 32 rope columns (SW64 rows)
constexpr int kStageBytes = kValue + kRope;
constexpr int kPBytes = 2 * kHC * 128;
constexpr int kPvSteps = kBlk / 16;
constexpr int kQTile = kHC * 128, kQTiles = 7;     // query through a stage: tiles of 64 rows x 64 columns (SW128 rows)
constexpr int kUnit = 4 * kHC * 16;                // one float4 of every (column part, row): exchange unit
constexpr int kFixWarps = 4, kSoftWarps = 16, kLoadWarps = 2, kSoftThreads = 32 * kSoftWarps;
constexpr int kWarpFix0 = 1, kWarpSoft0 = kWarpFix0 + kFixWarps;
constexpr int kWarpPv = kWarpSoft0 + kSoftWarps, kWarpLoad = kWarpPv + 1;
constexpr int kThreads = 32 * (kWarpLoad + kLoadWarps);
static_assert(kQTiles * kQTile <= kStageBytes, "the query's slot");
static_assert(kBlk <= 32 * kFixWarps && kBlk % 16 == 0, "a fix warp takes two 16-slot steps");
constexpr int kTmemCols = 512;
constexpr uint32_t kColO = 0, kColS = 256, kColQ = kColS + kBlk;
constexpr uint32_t kIdescS = idesc_bf16(128, 2 * kBlk, false, false);
constexpr uint32_t kIdescPV = idesc_bf16(128, 256, false, true);
constexpr float kRescaleThreshold = 8.0f;          // log2 units
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
static_assert(kColQ + 144 == kTmemCols, "TMEM columns");
static_assert(kValue % 1024 == 0 && kRope % 512 == 0 && kStageBytes % 1024 == 0, "operand alignment");

// one part of one tile, as the schedule hands it to the other roles
struct Seg {
  int b, tile, j0, j1, nc, len, t0, T;               // blocks [j0, j1) of the tile; nc = cached blocks
  int part;                                        // workspace slot of a partial result, -1: whole tile
  int end;                                         // no further segment
};

// workspace: partial O [slot][128 column quads][128 rows] float4, then
// [slot][128 rows] float4 (running max, sum, true max), then the join list
struct Join {
  long long row0;                                  // first query row (token * H + head)
  int nrows, nparts;                               // rows of the tile; 0 parts: nothing to join
};
constexpr size_t kPartBytes = (size_t)kTile * kDV * 4, kStatBytes = (size_t)kTile * 16;

struct __align__(1024) Smem {
  uint8_t stage[kStages][kStageBytes];             // value columns | rope columns
  uint8_t p[2][kPBytes];                           // P of even / odd blocks (and the exchange)
  Seg seg[2];
  alignas(16) unsigned long long valid[kStages][2];            // slots that hold a row
  uint32_t bad[kStages][kFixWarps];                // 32 slots each: zeroed for an infinity or NaN
  uint8_t plain[kStages];                          // the block needs no fix
  alignas(4) uint8_t live[kStages][kFixWarps];     // 2 steps of 16 slots each: some token sees some slot
  alignas(16) uint8_t spare[kUnit];                // of the logit exchange; row maxima and sums between exchanges
  uint64_t st_full[kStages], st_empty[kStages], ready[kStages], fixed[kStages];
  uint64_t s_full, s_free, p_full[2];
  uint64_t q_tm[2], q_free[2], mma_done[2], sc_full[2], sc_empty[2], fin[2];
  uint32_t tmem_base;
  int abort, no_abort;
};
static_assert(offsetof(Smem, p) % 1024 == 0 && offsetof(Smem, spare) % 16 == 0 && offsetof(Smem, live) % 4 == 0 &&
                  offsetof(Smem, valid) % 16 == 0 && offsetof(Smem, st_full) % 8 == 0 && kPBytes % 1024 == 0,
              "vector accesses and operands");
static_assert(sizeof(Smem) <= 232448, "shared memory budget");

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Partial results lie in L2 from a run's first tile to the join, while the keys
// stream past: they are written with the wish to stay (32 of 40 MB were gone and
// the join read them from HBM), and read for the last time without it.
__device__ __forceinline__ uint64_t policy_stay() {
  uint64_t p;
  asm("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ uint64_t policy_go() {
  uint64_t p;
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ void st_part(float4* p, float a, float b, float c, float d, uint64_t policy) {
  asm volatile("st.global.L2::cache_hint.v4.f32 [%0], {%1, %2, %3, %4}, %5;" ::"l"(p), "f"(a), "f"(b), "f"(c), "f"(d),
               "l"(policy)
               : "memory");
}
__device__ __forceinline__ float4 ld_part(const float4* p, uint64_t policy) {
  float4 v;
  asm volatile("ld.global.L2::cache_hint.v4.f32 {%0, %1, %2, %3}, [%4], %5;"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "l"(p), "l"(policy));
  return v;
}

// ---- two-CTA tcgen05 forms ----
__device__ __forceinline__ void tmem_alloc2(uint32_t dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(ncols)
               : "memory");
}
__device__ __forceinline__ void tmem_relinquish2() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc2(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
// The issuing thread shares its scheduler with the softmax warps, so each
// instruction of it takes several cycles: an operand descriptor is one low word
// that moves by a constant from MMA to MMA, and a constant high word (18 MMAs
// with whole descriptors computed for each took 1,350 cycles to issue, against
// the 1,010 that they run).
constexpr uint32_t desc_hi(uint32_t sbo, uint32_t layout) { return (sbo >> 4) | (1u << 14) | (layout << 29); }
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) { return (saddr >> 4) | ((lbo >> 4) << 16); }
__device__ __forceinline__ void mma2_ss(uint32_t d, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo, uint32_t b_hi,
                                        uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 a, b;\n setp.ne.b32 p, %6, 0;\n mov.b64 a, {%1, %2};\n mov.b64 b, {%3, %4};\n"
      " tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %5, p;\n}\n" ::"r"(d),
      "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma2_ts(uint32_t d, uint32_t a_tmem, uint32_t b_lo, uint32_t b_hi, uint32_t idesc,
                                        uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 b;\n setp.ne.b32 p, %5, 0;\n mov.b64 b, {%2, %3};\n"
      " tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], b, %4, p;\n}\n" ::"r"(d),
      "r"(a_tmem), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(acc)
      : "memory");
}
// arrive once on the barrier at the same offset in both CTAs of the pair when
// every tcgen05 operation issued so far by this thread has completed
__device__ __forceinline__ void commit2(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
      " [%0], %1;" ::"r"(bar),
      "h"((uint16_t)3)
      : "memory");
}
// true if any of the `n` threads of named barrier `id` passed true
__device__ __forceinline__ bool named_bar_or(uint32_t id, uint32_t n, bool v) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 q, %1, 0;\n bar.red.or.pred p, %2, %3, q;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(r)
      : "r"((uint32_t)v), "r"(id), "r"(n)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* tm, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          dst),
      "l"(tm), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap* tm, int x0, int x1, int x2, int x3, int x4,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
      "l"(tm), "r"(x0), "r"(x1), "r"(x2), "r"(x3), "r"(x4), "r"(bar)
      : "memory");
}
// the same, into this CTA, completing on a barrier of either CTA of the pair (cluster address)
__device__ __forceinline__ void tma_load2_3d(uint32_t dst, const CUtensorMap* tm, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(tm), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_load2_5d(uint32_t dst, const CUtensorMap* tm, int x0, int x1, int x2, int x3,
                                             int x4, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
      "l"(tm), "r"(x0), "r"(x1), "r"(x2), "r"(x3), "r"(x4), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void mbar_arrive_n(uint32_t bar, uint32_t n) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(n) : "memory");
}
__device__ __forceinline__ void st_zero16(uint32_t addr) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(addr), "r"(0u) : "memory");
}
// 32 bytes to global memory (32-byte aligned)
__device__ __forceinline__ void st_global32(void* p, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
               "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
// lane = thread's TMEM lane, 4 consecutive 32-bit columns
__device__ __forceinline__ void tmem_st4(uint32_t taddr, const uint4& v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(v.x), "r"(v.y),
               "r"(v.z), "r"(v.w)
               : "memory");
}
__device__ __forceinline__ long long warp_sum(long long v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// a / b for a >= 0, b > 0 (a 64-bit division takes one thread some 600 cycles)
__device__ __forceinline__ long long div_pos(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

// ---- schedule: tiles and blocks of a sequence ----
struct Plan {
  int tiles, nc, nd;                               // query tiles; cached / drafted blocks (all tokens)
  int T, H;
  bool chain;
};
__device__ __forceinline__ Plan make_plan(const TreeArgs& a, const TreeSeq& s) {
  Plan p;
  p.T = s.T;
  p.H = a.H;
  p.chain = a.mask == nullptr;
  p.tiles = (int)(((long long)s.T * a.H + kTile - 1) / kTile);
  p.nc = (s.len + kBlk - 1) / kBlk;
  p.nd = (s.T + kBlk - 1) / kBlk;
  return p;
}
// blocks of one tile: a chain's tokens see no drafted row behind themselves
__device__ __forceinline__ int tile_blocks(const Plan& p, int tile) {
  if (!p.chain) return p.nc + p.nd;
  const int last = (int)((128u * (uint32_t)tile + 127u) / (uint32_t)p.H);
  return p.nc + (last < p.T - 1 ? last : p.T - 1) / kBlk + 1;
}
// blocks of the first r tiles.  Chain: tile r' runs over drafted block k iff
// (128 r' + 127) / H >= 112 k, i.e. r' >= 112 k H / 128 (both rounded down).
__device__ __forceinline__ long long chain_term(const Plan& p, long long r, int k) {
  const long long from = 112ll * k * p.H / 128;
  return r > from ? r - from : 0;
}
__device__ __forceinline__ long long tiles_cost(const Plan& p, long long r) {  // one thread
  if (p.T == 0) return 0;
  if (!p.chain) return r * (p.nc + p.nd);
  long long c = r * (p.nc + 1);
  for (int k = 1; k <= (p.T - 1) / kBlk; ++k) c += chain_term(p, r, k);
  return c;
}
__device__ __forceinline__ long long tiles_cost_warp(const Plan& p, long long r) {  // chain, one warp
  long long c = 0;
  for (int k = 1 + (threadIdx.x & 31); k <= (p.T - 1) / kBlk; k += 32) c += chain_term(p, r, k);
  return warp_sum(c) + r * (p.nc + 1);
}

// A pair's run of the list of all (tile, block): an even share, segment by segment
// (one warp, the same state in every lane).
struct Schedule {
  long long x, x1, run;                            // list positions: next, end; length of every run
  TreeSeq s;
  Plan p;
  int b, tile, j;
  Join join;                                       // the tile that starts in this run and goes on in the next ones

  __device__ __forceinline__ void start(const TreeArgs& a, int pair, int npairs, const DevCtx& c) {
    const int lane = threadIdx.x & 31;
    bool wrong = false;
    long long total = 0, cost = 0;                 // cost: of the last 32 sequences
    for (int b0 = 0; b0 < a.n_seqs; b0 += 32) {
      cost = 0;
      if (b0 + lane < a.n_seqs) {
        const Plan q = make_plan(a, tree_seq(a, b0 + lane, &wrong));
        cost = tiles_cost(q, q.tiles);
      }
      total += cost;
    }
    total = warp_sum(total);
    if (__any_sync(0xffffffffu, wrong) && lane == 0) set_status(c, DSA_ERR_INDEX);
    run = div_pos(total + npairs - 1, npairs);
    x = run * pair;
    x1 = x + run < total ? x + run : total;
    join = {0, 0, 0};
    if (x >= x1) return;
    // the sequence, tile and block where this pair's run starts
    b = 0;
    long long off = x;
    for (int b0 = 0; b0 < a.n_seqs; b0 += 32) {
      if (a.n_seqs > 32) {
        cost = 0;
        if (b0 + lane < a.n_seqs) {
          const Plan q = make_plan(a, tree_seq(a, b0 + lane, &wrong));
          cost = tiles_cost(q, q.tiles);
        }
      }
      long long incl = cost;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += y;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, incl > off);
      if (past) {
        const int l = __ffs(past) - 1;
        off -= __shfl_sync(0xffffffffu, incl - cost, l);
        b = b0 + l;
        break;
      }
      off -= __shfl_sync(0xffffffffu, incl, 31);
    }
    s = tree_seq(a, b, &wrong);
    p = make_plan(a, s);
    if (!p.chain) {
      tile = (int)div_pos(off, p.nc + p.nd);
      j = (int)(off - (long long)tile * (p.nc + p.nd));
    } else {
      int lo = 0, hi = p.tiles;                    // cost(lo) <= off < cost(hi)
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (tiles_cost_warp(p, mid) <= off) lo = mid;
        else hi = mid;
      }
      tile = lo;
      j = (int)(off - tiles_cost_warp(p, lo));
    }
  }

  __device__ __forceinline__ Seg next(const TreeArgs& a, int pair) {
    Seg g;
    g.end = x >= x1;
    if (g.end) return g;
    if (tile == p.tiles) {                         // on to the next sequence with tokens (there is one: x < x1)
      bool wrong = false;
      do {
        ++b;
        s = tree_seq(a, b, &wrong);
      } while (s.T == 0);
      p = make_plan(a, s);
      tile = 0;
    }
    const int nb = tile_blocks(p, tile);
    const long long left = x1 - x;
    const int j1 = nb - j < left ? nb : (int)(j + left);
    const bool whole = j == 0 && j1 == nb;
    g.b = b;
    g.tile = tile;
    g.j0 = j;
    g.j1 = j1;
    g.nc = p.nc;
    g.len = s.len;
    g.t0 = s.t0;
    g.T = s.T;
    g.part = whole ? -1 : 2 * pair + (j == 0 ? 1 : 0);
    if (!whole && j == 0) {
      const long long rows = (long long)s.T * a.H - 128ll * tile;
      join.row0 = (long long)s.t0 * a.H + 128ll * tile;
      join.nrows = rows < kTile ? (int)rows : kTile;
      join.nparts = (int)div_pos(x + nb - 1, run) - pair + 1;
    }
    x += j1 - j;
    j = 0;
    ++tile;
    return g;
  }
};

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    tree_attn_tc_kernel(TreeArgs a, const __nv_bfloat16* __restrict__ qg, const __nv_bfloat16* __restrict__ kvn,
                        __nv_bfloat16* __restrict__ out, float* __restrict__ mx, float* __restrict__ sm_out,
                        float4* __restrict__ parts, float4* __restrict__ stats, Join* __restrict__ joins,
                        DevCtx c, int wide, const __grid_constant__ CUtensorMap tm_page_v,
                        const __grid_constant__ CUtensorMap tm_page_v2, const __grid_constant__ CUtensorMap tm_page_r,
                        const __grid_constant__ CUtensorMap tm_page_r2, const __grid_constant__ CUtensorMap tm_new_v,
                        const __grid_constant__ CUtensorMap tm_new_r, const __grid_constant__ CUtensorMap tm_q) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>(smem_raw);   // the operands' swizzles need the 1024-byte alignment
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t crank = cluster_ctarank();
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  volatile int* abort_flag = &sm.abort;
  if ((smem_u32(smem_raw) & 1023u) != 0) {         // (dynamic shared memory starts at 1 KB: never)
    set_status(c, DSA_ERR_CUDA);
    return;
  }

  if (threadIdx.x == 32 * kWarpFix0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_u32(&sm.st_full[i]), kLoadWarps);
      mbar_init(smem_u32(&sm.st_empty[i]), 1 + kFixWarps);  // the last MMAs, and the fix warps
      mbar_init(smem_u32(&sm.ready[i]), 2 * kFixWarps);
      mbar_init(smem_u32(&sm.fixed[i]), kFixWarps);
    }
    mbar_init(smem_u32(&sm.s_full), 1);
    // ready, s_free, p_full, q_tm (used in CTA 0): the warps of both CTAs arrive
    mbar_init(smem_u32(&sm.s_free), 2 * kSoftWarps);
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&sm.p_full[i]), 2 * 2);   // (row groups)
      mbar_init(smem_u32(&sm.q_tm[i]), 2 * kFixWarps);
      mbar_init(smem_u32(&sm.q_free[i]), 1);
      mbar_init(smem_u32(&sm.mma_done[i]), 1);
      mbar_init(smem_u32(&sm.sc_full[i]), 1);
      // readers of a segment: fix and softmax warps, value loads, and CTA 0's issuers
      mbar_init(smem_u32(&sm.sc_empty[i]), kFixWarps + kSoftWarps + 1 + (crank == 0 ? 2 : 0));
      mbar_init(smem_u32(&sm.fin[i]), 1);
    }
    sm.abort = 0;
    sm.no_abort = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc2(smem_u32(&sm.tmem_base), kTmemCols);
    tmem_relinquish2();
    tc_fence_before();
  }
  __syncthreads();
  cluster_sync_all();  // both CTAs' barriers initialised before any remote arrive
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  let_next_launch();
  wait_for_earlier();

  if (warp >= kWarpLoad) {
    // ------------------------------- key loads -------------------------------
    // Groups of 16 slots; one copy takes two of them where they lie in one page
    // (`wide`: pages of a multiple of 32 rows).  A drafted group starts at any
    // row: value copies of 8 rows.
    const bool rope = warp != kWarpLoad;
    int G = 0;                                     // ring slots so far
    uint32_t ready_par = 0, direct = 0;            // a bit per stage: phase of its `ready`, last use plain
    bool ok = true;
    Schedule sched;                                // the rope warp's
    if (rope) sched.start(a, pair, npairs, c);
    for (int i = 0; ok; ++i) {
      Seg g;
      if (rope) {
        // makes the segment out for everyone, once the last but one is read
        if (!mbar_wait_warp(smem_u32(&sm.sc_empty[i & 1]), ((i >> 1) & 1) ^ 1, c, abort_flag)) break;
        g = sched.next(a, pair);
        if (lane == 0) {
          sm.seg[i & 1] = g;
          mbar_arrive(smem_u32(&sm.sc_full[i & 1]));
        }
        __syncwarp();
      } else {
        if (!mbar_wait_warp(smem_u32(&sm.sc_full[i & 1]), (i >> 1) & 1, c, abort_flag)) break;
        g = sm.seg[i & 1];
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.sc_empty[i & 1]));
      }
      if (g.end) break;
      const int32_t* trow = a.table + (long long)g.b * a.max_pages;
      {
        // the query's slot: 64 rows x 448 value columns (rows behind the tile's last
        // come along; nothing of theirs is written)
        const int st = G % kStages;
        if (!mbar_wait_warp(smem_u32(&sm.st_empty[st]), ((G / kStages) & 1) ^ 1, c, abort_flag)) break;
        if (lane == 0) {
          const uint32_t bar = smem_u32(&sm.st_full[st]);
          if (rope) {
            mbar_arrive(bar);
          } else {
            mbar_arrive_expect_tx(bar, kQTiles * kQTile);
            const int y = (int)((long long)g.t0 * a.H + 128ll * g.tile) + kHC * (int)crank;
#pragma unroll 1
            for (int k = 0; k < kQTiles; ++k) tma_load_2d(smem_u32(sm.stage[st]) + k * kQTile, &tm_q, 64 * k, y, bar);
          }
        }
        __syncwarp();
        direct &= ~(1u << st);
        ++G;
      }
      for (int j = g.j0; j < g.j1; ++j, ++G) {
        const int st = G % kStages;
        const bool drafted = j >= g.nc;
        // lane l < 7: group l
        int cnt = 0, x = 0, page = 0;              // rows of the group, first row (in the page / drafted), page
        if (lane < kGroups) {
          const int pos = (drafted ? j - g.nc : j) * kBlk + 16 * lane;
          const int left = (drafted ? g.T : g.len) - pos;
          cnt = left <= 0 ? 0 : (left < 16 ? left : 16);
          if (drafted) {
            x = g.t0 + pos;
          } else if (cnt > 0) {
            page = trow[pos / a.R];
            x = pos % a.R;
            if (page < 0 || page >= a.n_pages) {
              cnt = 0;
              set_status(c, DSA_ERR_INDEX);
            }
          }
        }
        const uint32_t loaded = __ballot_sync(0xffffffffu, cnt > 0);
        const uint32_t bar = smem_u32(&sm.st_full[st]), base = smem_u32(sm.stage[st]);
        const uint32_t even = (j & 1) ? 0x2Au : 0x15u;  // groups at a multiple of 32 rows: 7 j + k even
        if (wide && !drafted && loaded == 0x7Fu) {
          // The usual block: three copies of 32 rows and one of 16, the 16 first (j
          // odd) or last, from coordinates that are ready before the wait.
          const int k0 = j & 1;
          int gx[4], gp[4];
#pragma unroll
          for (int t = 0; t < 4; ++t) {            // t < 3: groups k0 + 2t and the next; t = 3: the single one
            const int k = t < 3 ? k0 + 2 * t : (k0 ? 0 : 6);
            gx[t] = __shfl_sync(0xffffffffu, x, k);
            gp[t] = __shfl_sync(0xffffffffu, page, k);
          }
          const int last = __shfl_sync(0xffffffffu, cnt, kGroups - 1);
          const uint32_t d0 = base + (rope ? kValue + k0 * 1024 : k0 * 2 * kOct);
          const uint32_t d3 = base + (rope ? kValue + (k0 ? 0 : 6 * 1024) : (k0 ? 0 : 12 * kOct));
          if (!mbar_wait_warp(smem_u32(&sm.st_empty[st]), ((G / kStages) & 1) ^ 1, c, abort_flag)) {
            ok = false;
            break;
          }
          // A block without an empty slot is plain: its copies complete on the
          // issuer's barrier, past the fix warps (450 cycles, and the signals from
          // the other CTA another 500)
          const bool plain = last == 16;
          if (lane == 0) {
            const uint32_t full = plain ? mapa_shared(smem_u32(&sm.ready[st]), 0) : mapa_shared(bar, crank);
            if (rope) {
              if (plain) mbar_arrive(bar);
              else mbar_arrive_expect_tx(bar, kRope);
              const int col = kDV + 32 * (int)crank;
#pragma unroll
              for (int t = 0; t < 3; ++t) tma_load2_3d(d0 + t * 2048, &tm_page_r2, col, gx[t], gp[t], full);
              tma_load2_3d(d3, &tm_page_r, col, gx[3], gp[3], full);
            } else {
              sm.valid[st][0] = ~0ull;
              sm.valid[st][1] = 0xFFFFFFFFull | ((unsigned long long)((1u << last) - 1u) << 32);
              sm.plain[st] = plain;
              if (plain) {
                *reinterpret_cast<uint32_t*>(sm.live[st]) = 0x01030303u;
                mbar_arrive(bar);
                if (crank == 0) {                  // in the fix warps' stead, for the copies of both CTAs
                  const uint32_t rd = smem_u32(&sm.ready[st]);
                  mbar_arrive_expect_tx(rd, 2 * kStageBytes);
                  mbar_arrive_n(rd, 2 * kFixWarps - 1);
                }
              } else {
                mbar_arrive_expect_tx(bar, kValue);
              }
#pragma unroll
              for (int t = 0; t < 3; ++t)
                tma_load2_5d(d0 + t * 4 * kOct, &tm_page_v2, 0, 0, 4 * (int)crank, gx[t] >> 3, gp[t], full);
              tma_load2_5d(d3, &tm_page_v, 0, 0, 4 * (int)crank, gx[3] >> 3, gp[3], full);
            }
          }
          direct = plain ? direct | (1u << st) : direct & ~(1u << st);
          ready_par ^= 1u << st;
          __syncwarp();
          continue;
        }
        unsigned long long v0 = 0, v1 = 0;
#pragma unroll
        for (int k = 0; k < kGroups; ++k) {
          const unsigned long long bits = (1u << __shfl_sync(0xffffffffu, cnt, k)) - 1u;
          if (k < 4) v0 |= bits << (16 * k);
          else v1 |= bits << (16 * (k - 4));
        }
        if (!mbar_wait_warp(smem_u32(&sm.st_empty[st]), ((G / kStages) & 1) ^ 1, c, abort_flag)) {
          ok = false;
          break;
        }
        direct &= ~(1u << st);
        ready_par ^= 1u << st;
        // the second group of a pair goes with the first
        uint32_t first = loaded, pairs = 0;
        if (wide && !drafted) {
          pairs = loaded & even & 0x3Fu;           // (group 6 has no second one in this block)
          first = loaded & ~(pairs << 1);
        }
        if (lane == 0) {
          if (!rope) {
            sm.valid[st][0] = v0;
            sm.valid[st][1] = v1;
            sm.plain[st] = 0;
          }
          // a pair brings both its groups, the second past the last row or not
          const int left = g.T - (j - g.nc) * kBlk, n8 = ((left < kBlk ? left : kBlk) + 7) / 8;
          const int groups = __popc(first) + __popc(pairs);
          mbar_arrive_expect_tx(bar, rope ? groups * 1024u : drafted ? n8 * (uint32_t)kOct : groups * 2u * kOct);
        }
        __syncwarp();
#pragma unroll 1
        for (uint32_t m = first; m; m &= m - 1) {
          const int k = __ffs(m) - 1;
          const int gx = __shfl_sync(0xffffffffu, x, k), gp = __shfl_sync(0xffffffffu, page, k);
          const int gn = __shfl_sync(0xffffffffu, cnt, k);
          const bool two = (pairs >> k) & 1u;
          if (lane == 0) {
            if (rope) {
              const uint32_t dr = base + kValue + k * 1024;
              const int col = kDV + 32 * (int)crank;
              if (drafted) tma_load_2d(dr, &tm_new_r, col, gx, bar);
              else tma_load_3d(dr, two ? &tm_page_r2 : &tm_page_r, col, gx, gp, bar);
            } else {
              const uint32_t dv = base + 2 * k * kOct;
              if (drafted) {
                tma_load_3d(dv, &tm_new_v, 0, gx, 4 * (int)crank, bar);
                if (gn > 8) tma_load_3d(dv + kOct, &tm_new_v, 0, gx + 8, 4 * (int)crank, bar);
              } else {
                tma_load_5d(dv, two ? &tm_page_v2 : &tm_page_v, 0, 0, 4 * (int)crank, gx >> 3, gp, bar);
              }
            }
          }
        }
        __syncwarp();
      }
    }
    if (rope && crank == 0 && lane == 0) joins[pair] = sched.join;
    // no copy may still be in flight when the CTA exits (bounded, whatever the others do)
    for (int k = G - kStages < 0 ? 0 : G - kStages; k < G; ++k) {
      const int st = k % kStages;
      mbar_wait_warp(smem_u32(&sm.st_full[st]), (k / kStages) & 1, c, &sm.no_abort);
      // (CTA 1's plain copies, too: it does not exit before CTA 0)
      if (crank == 0 && ((direct >> st) & 1u))
        mbar_wait_warp(smem_u32(&sm.ready[st]), ((ready_par >> st) & 1u) ^ 1u, c, &sm.no_abort);
    }
  } else if (warp >= kWarpFix0 && warp < kWarpSoft0) {
    // ------------------------- key stages passed on -------------------------
    const int fw = warp - kWarpFix0;
    const int s0 = 32 * fw;                        // this warp's slots: [s0, s0 + 32) of the block
    const uint32_t kAll = kBlk - s0 >= 32 ? 0xffffffffu : (1u << ((kBlk - s0) & 31)) - 1u;
    int G = 0;
    bool ok = true;
    for (int i = 0; ok; ++i) {
      if (!mbar_wait_warp(smem_u32(&sm.sc_full[i & 1]), (i >> 1) & 1, c, abort_flag)) break;
      const Seg g = sm.seg[i & 1];
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sm.sc_empty[i & 1]));
      if (g.end) break;
      {
        // thread = TMEM lane l of this warp's quadrant: row l & 63, column half l >> 6
        const int st = G % kStages, l = (warp & 3) * 32 + lane, rl = l & 63, half = l >> 6;
        const long long qrow = (long long)g.t0 * a.H + 128ll * g.tile + kHC * (int)crank + rl;
        const bool there = qrow < (long long)a.n_tok * a.H;
        const __nv_bfloat16* qh = qg + (there ? qrow : 0) * kDQK;
        uint4 r[4];                                // rope columns [32 half, +32)
#pragma unroll
        for (int t = 0; t < 4; ++t)
          r[t] = there ? __ldg(reinterpret_cast<const uint4*>(qh + kDV + 32 * half) + t) : make_uint4(0, 0, 0, 0);
        uint32_t x[32];                            // half 1: value columns 448..511
        auto put = [&](int t, uint4 v) { x[4 * t] = v.x, x[4 * t + 1] = v.y, x[4 * t + 2] = v.z, x[4 * t + 3] = v.w; };
        if (half == 1) {
#pragma unroll
          for (int t = 0; t < 8; ++t)
            put(t, there ? __ldg(reinterpret_cast<const uint4*>(qh + 448) + t) : make_uint4(0, 0, 0, 0));
        }
        ok = mbar_wait_warp(smem_u32(&sm.st_full[st]), (G / kStages) & 1, c, abort_flag) &&
             (i == 0 || mbar_wait_warp(smem_u32(&sm.q_free[(i - 1) & 1]), ((i - 1) >> 1) & 1, c, abort_flag));
        if (!ok) break;
        tc_fence_after();
        const uint32_t dst = tmem + ((uint32_t)((warp & 3) * 32) << 16) + kColQ;
        const uint8_t* src = sm.stage[st] + rl * 128;
#pragma unroll 1
        for (int p = 3; p >= 0; --p) {             // 64 value columns -> 32 TMEM columns
          if (p < 3 || half == 0) {
#pragma unroll
            for (int t = 0; t < 8; ++t)
              put(t, *reinterpret_cast<const uint4*>(src + (4 * half + p) * kQTile + ((t ^ (rl & 7)) << 4)));
          }
          __syncwarp();
          tmem_st32(dst + 32 * p, x);
          tmem_st_wait();
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) tmem_st4(dst + 128 + 4 * t, r[t]);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_u32(&sm.st_empty[st]));
          mbar_arrive(smem_u32(&sm.fixed[st]));    // (its phases are those of the slots)
          arrive_leader(&sm.q_tm[i & 1], crank);
        }
        __syncwarp();
        ++G;
      }
      // the tokens of the tile
      const int ta = (int)(128u * (uint32_t)g.tile / (uint32_t)a.H);  // (rows of all tokens: below 2^31)
      const int last = (int)((128u * (uint32_t)g.tile + 127u) / (uint32_t)a.H);
      const int tb = last < g.T - 1 ? last : g.T - 1;
      for (int j = g.j0; j < g.j1; ++j, ++G) {
        const int st = G % kStages;
        // slots that any / every token of the tile sees
        uint32_t any = kAll, every = kAll;
        if (j >= g.nc) {
          const int first = (j - g.nc) * kBlk + s0;
          if (a.mask == nullptr) {
            const int na = ta - first + 1, nb = tb - first + 1;  // slots that the first / last token sees
            every = na <= 0 ? 0u : na >= 32 ? kAll : (1u << na) - 1u;
            any = nb <= 0 ? 0u : nb >= 32 ? kAll : (1u << nb) - 1u;
          } else {
            const int w = first >> 6, sh = first & 63;
            uint32_t o = 0u, n = kAll;
            for (int t = ta + lane; t <= tb; t += 32) {
              const unsigned long long* mrow = a.mask + (long long)(g.t0 + t) * a.mask_words;
              unsigned long long m = w < a.mask_words ? mrow[w] >> sh : 0ull;
              if (sh && w + 1 < a.mask_words) m |= mrow[w + 1] << (64 - sh);
              o |= (uint32_t)m & kAll;
              n &= (uint32_t)m;
            }
            any = __reduce_or_sync(0xffffffffu, o);
            every = __reduce_and_sync(0xffffffffu, n);
          }
        }
        if (!mbar_wait_warp(smem_u32(&sm.st_full[st]), (G / kStages) & 1, c, abort_flag)) {
          ok = false;
          break;
        }
        if (sm.plain[st]) {
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(smem_u32(&sm.st_empty[st]));
            mbar_arrive(smem_u32(&sm.fixed[st]));
          }
          continue;
        }
        const uint32_t valid = (uint32_t)(sm.valid[st][fw >> 1] >> (32 * (fw & 1))) & kAll;
        const uint32_t seen = valid & any;
        uint32_t bad = 0;
        for (uint32_t mixed = seen & ~every; mixed; mixed &= mixed - 1) {
          const int k = __ffs(mixed) - 1;
          const uint4* src =
              reinterpret_cast<const uint4*>(kvn + (long long)(g.t0 + (j - g.nc) * kBlk + s0 + k) * kDQK);
          bool inf = false;
#pragma unroll
          for (int u = 0; u < 3; ++u) {
            const int e = 32 * u + lane;
            if (e < kDQK / 8) {
              const uint4 v = __ldg(src + e);
              const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
              for (int q = 0; q < 4; ++q)
                inf |= (w[q] & 0x7F80u) == 0x7F80u || (w[q] & 0x7F800000u) == 0x7F800000u;
            }
          }
          if (__any_sync(0xffffffffu, inf)) bad |= 1u << k;
        }
        const uint32_t live = ((seen & 0xffffu) ? 1u : 0u) | ((seen >> 16) ? 2u : 0u);
        if (lane == 0) {
          sm.bad[st][fw] = bad;
          sm.live[st][fw] = (uint8_t)live;
        }
        // zero rows of the steps that run (step 0 always counts: a block without a
        // seen slot may have to start O)
        const uint32_t runs = ((live & 1u) || fw == 0 ? 0xffffu : 0u) | ((live & 2u) ? 0xffff0000u : 0u);
        const uint32_t clear = (~seen | bad) & runs & kAll;
        if (clear) {
          const uint32_t pv = smem_u32(sm.stage[st]) + fw * 4 * kOct + (lane >> 3) * kAtom + (lane & 7) * 16;
#pragma unroll
          for (int o = 0; o < 4; ++o) {            // 8 rows x 512 bytes each
            if (((clear >> (8 * o)) & 0xffu) == 0) continue;
#pragma unroll
            for (int k = 0; k < 8; ++k)
              if ((clear >> (8 * o + k)) & 1u) st_zero16(pv + o * kOct + k * 128);
          }
          fence_proxy_async_smem();                // these writes -> the tensor cores' reads
        }
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_u32(&sm.st_empty[st]));
          mbar_arrive(smem_u32(&sm.fixed[st]));
          arrive_leader_shared(&sm.ready[st], crank);
        }
      }
    }
  } else if (warp == 0) {
    if (crank == 0 && lane == 0) {
      // -------------------------- MMA issuer: logits --------------------------
      // Two issuers: a thread's barrier tests wait behind its own queued MMAs (some
      // 430 cycles), so while the MMAs of one run, the other has its answers.
      int G = 0;                                   // blocks so far
      uint32_t st = 0, slot = 0;                   // stage, ring slot
      uint32_t ready_par = 0;                      // parity of each stage's next `ready` phase, a bit each
      bool ok = true;
      for (int i = 0; ok; ++i) {
        const int bi = i & 1;
        if (!mbar_wait(smem_u32(&sm.sc_full[bi]), (i >> 1) & 1, c, abort_flag)) break;
        const int nblk = sm.seg[bi].j1 - sm.seg[bi].j0, end = sm.seg[bi].end;
        mbar_arrive(smem_u32(&sm.sc_empty[bi]));
        if (end) break;
        if (!mbar_wait<true>(smem_u32(&sm.q_tm[bi]), (i >> 1) & 1, c, abort_flag)) break;
        tc_fence_after();
        const uint32_t query = smem_u32(&sm.st_empty[0]) + 8 * st;
        if (++st == kStages) st = 0;
        ++slot;
        for (int j = 0; j < nblk; ++j, ++G, ++slot) {
          // the keys; the last logits read; PV(G-2) done, whose P buffer the softmax
          // of this block exchanges logits through (with the tile before: mma_done)
          ok = mbar_wait<true>(smem_u32(&sm.ready[0]) + 8 * st, (ready_par >> st) & 1u, c, abort_flag) &&
               (G == 0 || mbar_wait<true>(smem_u32(&sm.s_free), (G - 1) & 1, c, abort_flag)) &&
               (j < 2 || mbar_wait(smem_u32(&sm.st_empty[0]) + 8 * ((slot - 2) % kStages), ((slot - 2) / kStages) & 1, c,
                                   abort_flag));
          if (!ok) break;
          tc_fence_after();
          // The query's slot is free only now, although q_tm said that it is read: s_free
          // says that every softmax warp is past the last block but one of the tile
          // before, whose wait for its P V (to rescale O) is on this slot's st_empty.
          // Released at once, that barrier could complete two phases ahead of a late warp.
          if (j == 0) commit2(query);
          const uint32_t sb = smem_u32(sm.stage[0]) + st * kStageBytes;
          const uint32_t v = desc_lo(sb, 16), r = desc_lo(sb + kValue, 16);
#pragma unroll
          for (int kk = 0; kk < 16; ++kk)
            mma2_ts(tmem + kColS, tmem + kColQ + kk * 8, v + ((kk >> 2) * kAtom + (kk & 3) * 32) / 16,
                    desc_hi(kOct, kSw128), kIdescS, kk > 0 ? 1u : 0u);
#pragma unroll
          for (int k = 0; k < 2; ++k)
            mma2_ts(tmem + kColS, tmem + kColQ + 128 + k * 8, r + 2 * k, desc_hi(512, kSw64), kIdescS, 1u);
          commit2(smem_u32(&sm.s_full));
          ready_par ^= 1u << st;
          if (++st == kStages) st = 0;
        }
        if (ok) commit2(smem_u32(&sm.q_free[bi]));
      }
      commit2(smem_u32(&sm.fin[0]));
      mbar_wait(smem_u32(&sm.fin[0]), 0, c, &sm.no_abort);
    }
  } else if (warp == kWarpPv) {
    if (crank == 0 && lane == 0) {
      // --------------------------- MMA issuer: O += P V ---------------------------
      int G = 0;
      uint32_t st = 0;
      bool ok = true;
      for (int i = 0; ok; ++i) {
        const int bi = i & 1;
        if (!mbar_wait(smem_u32(&sm.sc_full[bi]), (i >> 1) & 1, c, abort_flag)) break;
        const int nblk = sm.seg[bi].j1 - sm.seg[bi].j0, end = sm.seg[bi].end;
        mbar_arrive(smem_u32(&sm.sc_empty[bi]));
        if (end) break;
        if (++st == kStages) st = 0;               // the query's slot
        for (int j = 0; j < nblk; ++j, ++G) {
          ok = mbar_wait<true>(smem_u32(&sm.p_full[G & 1]), (G >> 1) & 1, c, abort_flag);
          if (!ok) break;
          tc_fence_after();
          const uint32_t sb = smem_u32(sm.stage[0]) + st * kStageBytes;
          const uint32_t v = desc_lo(sb, kAtom), p = desc_lo(smem_u32(sm.p[0]) + (G & 1) * kPBytes, 16);
          // the 16-slot steps that some token sees (2 bits per byte); one at least
          const uint32_t lv = *reinterpret_cast<const volatile uint32_t*>(sm.live[st]);
          uint32_t steps = (lv & 3u) | ((lv >> 6) & 12u) | ((lv >> 12) & 48u) | ((lv >> 18) & 192u);
          uint32_t acc = j > 0;
          if (steps == 0x7fu) {
#pragma unroll
            for (int kk = 0; kk < kPvSteps; ++kk) {
#pragma unroll
              for (int m = 0; m < 2; ++m)
                mma2_ss(tmem + kColO + 128 * m, p + ((kk >> 2) * (kHC * 128) + (kk & 3) * 32) / 16,
                        desc_hi(1024, kSw128), v + (2 * m * kAtom + kk * 2 * kOct) / 16, desc_hi(kOct, kSw128),
                        kIdescPV, kk > 0 ? 1u : acc);
            }
          } else {
            if (steps == 0) steps = 1;
#pragma unroll 1
            for (; steps; steps &= steps - 1, acc = 1) {
              const int kk = __ffs(steps) - 1;
#pragma unroll
              for (int m = 0; m < 2; ++m)
                mma2_ss(tmem + kColO + 128 * m, p + ((kk >> 2) * (kHC * 128) + (kk & 3) * 32) / 16,
                        desc_hi(1024, kSw128), v + (2 * m * kAtom + kk * 2 * kOct) / 16, desc_hi(kOct, kSw128),
                        kIdescPV, acc);
            }
          }
          commit2(smem_u32(&sm.st_empty[0]) + 8 * st);
          if (++st == kStages) st = 0;
        }
        if (ok) commit2(smem_u32(&sm.mma_done[bi]));  // this segment's O complete
      }
      commit2(smem_u32(&sm.fin[1]));
      mbar_wait(smem_u32(&sm.fin[1]), 0, c, &sm.no_abort);
    }
  } else {
    // --------------------------- softmax / epilogue ---------------------------
    const int quad = warp & 3, ch = (warp - kWarpSoft0) >> 2;
    const int l = quad * 32 + lane;                // TMEM lane
    const int hl = l & 63, half = l >> 6;          // row in the CTA; lane half
    const int rr = kHC * (int)crank + hl;          // row in the tile
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    const float sl2e = a.scale * kLog2e;
    // Column part ch = slots [c0, c0 + 32) (ch even) or [c0, c0 + 24) (ch odd) of
    // the block; thread (lane l, part ch) keeps the first 16 of row hl in lane
    // half 0, the rest in lane half 1 (runs of 8: whole 16-byte pieces of P).
    const int c0 = 56 * (ch >> 1) + 32 * (ch & 1);
    const int kept = half && (ch & 1) ? 8 : 16;
    const int s0 = c0 + 16 * half;
    const uint32_t keep_bits = (1u << kept) - 1u;
    // Row groups: 256 threads each (rows 0..31, 32..63 of the CTA); nothing but the
    // signals to the issuer passes between them inside a block.
    const uint32_t group_bar = 4 + (quad & 1), pair_bar = 6 + 2 * ch + (quad & 1);
    // [ch][half] -> 32 rows of the group, in the spare's 4 x (64 rows x 16 bytes)
    auto red = [&](int c4, int h) -> float& {
      return *reinterpret_cast<float*>(sm.spare + (c4 >> 1) * 1024 + (quad & 1) * 512 + ((c4 & 1) * 2 + h) * 128 + lane * 4);
    };
    // of a row's eight values in red[], the same order in each of its threads
    auto row_max = [&]() {
      float m = -INFINITY;
#pragma unroll
      for (int t = 0; t < 4; ++t)
        m = fmaxf(m, fmaxf(red(t, 0), red(t, 1)));
      return m;
    };
    // this thread's bits of 112 slot bits (s0 is a multiple of 8)
    auto cut = [&](const void* bits) -> uint32_t {
      const uint8_t* b = static_cast<const uint8_t*>(bits) + (s0 >> 3);
      return (b[0] | (uint32_t)b[1] << 8) & keep_bits;
    };
    // Exchange with the lane-pair partner (lane l ^ 64, same ch): half 1 sends the
    // part's slots 0..15 (4 float4), half 0 the others (4, or 2 for ch odd).  The
    // first two lie where their reader's own P goes afterwards (16-byte pieces of
    // its row, swizzled), so that reading and overwriting them needs no barrier;
    // the others in the rope part of this block's stage (its last reader, the
    // logits, is done), in the spare, and in pieces 14 and 15 of a P row, which
    // hold no slots.
    auto piece = [&](int t) { return (uint32_t)((t >> 3) * (kHC * 128) + hl * 128 + (((t & 7) ^ (hl & 7)) << 4)); };
    const int p0 = c0 / 8;
    const uint32_t first0 = piece(p0), first1 = piece(p0 + 1);  // half 0's pieces of P
    const uint32_t last0 = piece(p0 + 2), last1 = piece((ch & 1) ? 14 + (ch >> 1) : p0 + 3);  // half 1's
    const uint32_t own0 = half ? last0 : first0, own1 = half ? last1 : first1;
    const uint32_t his0 = half ? first0 : last0, his1 = half ? first1 : last1;
    const uint32_t spare_at = (ch >> 1) * 2048 + hl * 16, rope_at = kValue + ch * 1024 + hl * 16, pad_at = piece(14);
    // Every warp executes the same sequence of named barriers whatever happens
    // (after a failed wait it goes on through the segment without work, and
    // the vote at the next one makes all of them stop).
    bool ok = true;
    int G = 0, B = 0;                              // ring slots, blocks so far
    for (int i = 0;; ++i) {
      const int bi = i & 1;
      if (ok) ok = mbar_wait_warp(smem_u32(&sm.sc_full[bi]), (i >> 1) & 1, c, abort_flag);
      if (named_bar_or(2, kSoftThreads, !ok)) break;
      const Seg g = sm.seg[bi];
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sm.sc_empty[bi]));
      if (g.end) break;
      const long long rows = (long long)g.T * a.H - 128ll * g.tile;
      const bool live = rr < rows;
      const int tok = live ? (int)((128u * (uint32_t)g.tile + rr) / (uint32_t)a.H) : g.T - 1;
      float m_run = -INFINITY, m_own = -INFINITY, l_run = 0.f;  // m_own: over this thread's slots
      bool poison = false;
      ++G;                                         // the query's slot
      for (int j = g.j0; j < g.j1; ++j, ++G, ++B) {
        const int pb = B & 1, st = G % kStages;
        // fixed: valid and bad of this CTA's load and fix warps are there (long before
        // the logits, and not done again before this block's P V).  s_full: the issuer of
        // the logits took this block after PV(G-2), so P buffer pb is free.
        if (ok) {
          const uint32_t fixed = smem_u32(&sm.fixed[st]), full = smem_u32(&sm.s_full), f = (G / kStages) & 1;
          const bool there = mbar_test(full, B & 1) & mbar_test(fixed, f);  // (both in flight)
          if (!__all_sync(0xffffffffu, there))
            ok = mbar_wait_warp(fixed, f, c, abort_flag) && mbar_wait_warp(full, B & 1, c, abort_flag);
        }
        uint32_t lo[16], hi[16];                   // the part's slots 0..15 and 16..31 (ch odd: 16..23)
        uint32_t vmask = 0;                        // visible ones of the slots that this thread keeps
#pragma unroll
        for (int t = 0; t < 16; ++t) hi[t] = 0u;
        if (ok) {
          tc_fence_after();
          const uint32_t sbuf = tmem + lane_off + kColS + c0;
          tmem_ld16(sbuf, lo);
          tmem_ld16(sbuf + 16, hi);                // (ch odd: 8 columns of the next part or the query, unused)
          vmask = cut(sm.valid[st]);
          tmem_ld_wait16(lo);
          tmem_ld_also16(hi);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive_leader(&sm.s_free, crank);  // the logit buffer is free
        } else {
#pragma unroll
          for (int t = 0; t < 16; ++t) lo[t] = 0u;
        }
        uint8_t *const pbuf = sm.p[pb], *const xs = sm.spare + spare_at, *const xr = sm.stage[st] + rope_at;
        uint8_t* const xr1 = ch < 3 ? xr + kUnit : sm.p[pb ^ 1] + pad_at;
        auto put = [&](uint8_t* dst, const uint32_t* v) {
          *reinterpret_cast<uint4*>(dst) = make_uint4(v[0], v[1], v[2], v[3]);
        };
        float x[16];
        if (half == 0) {
          put(pbuf + his0, hi);
          put(pbuf + his1, hi + 4);
          if ((ch & 1) == 0) {
            put(xs, hi + 8);
            put(xs + 1024, hi + 12);
          }
#pragma unroll
          for (int t = 0; t < 16; ++t) x[t] = __uint_as_float(lo[t]);
        } else {
          put(pbuf + his0, lo);
          put(pbuf + his1, lo + 4);
          put(xr, lo + 8);
          put(xr1, lo + 12);
#pragma unroll
          for (int t = 0; t < 16; ++t) x[t] = __uint_as_float(hi[t]);
        }
        if (j >= g.nc) {
          const int first = (j - g.nc) * kBlk + s0;
          if (a.mask == nullptr) {
            const int n = tok - first + 1;
            vmask &= n <= 0 ? 0u : n >= 16 ? 0xffffu : (1u << n) - 1u;
          } else {
            const unsigned long long* mrow = a.mask + (long long)(g.t0 + tok) * a.mask_words;
            const int w = first >> 6, sh = first & 63;
            unsigned long long m = w < a.mask_words ? __ldg(mrow + w) >> sh : 0ull;
            if (sh && w + 1 < a.mask_words) m |= __ldg(mrow + w + 1) << (64 - sh);
            vmask &= (uint32_t)m;
          }
          if (vmask & cut(sm.bad[st])) poison = true;
        }
        named_bar_sync(pair_bar, 64);
        auto add = [&](int t, const uint8_t* src) {
          const float4 v = *reinterpret_cast<const float4*>(src);
          x[t] += v.x;
          x[t + 1] += v.y;
          x[t + 2] += v.z;
          x[t + 3] += v.w;
        };
        add(0, pbuf + own0);
        add(4, pbuf + own1);
        if (kept == 16) {
          add(8, half ? xs : xr);
          add(12, half ? xs + 1024 : xr1);
        }
        if (vmask != keep_bits || kept != 16) {
#pragma unroll
          for (int t = 0; t < 16; ++t)
            if (((vmask >> t) & 1u) == 0) x[t] = -INFINITY;
        }
        float bm = x[0], bn = x[1];
#pragma unroll
        for (int t = 2; t < 16; t += 2) {
          bm = fmaxf(bm, x[t]);
          bn = fmaxf(bn, x[t + 1]);
        }
        bm = fmaxf(bm, bn);
        bm *= sl2e;                                // log2 units (sl2e > 0)
        m_own = fmaxf(m_own, bm);
        // The maximum that P is taken against moves only when a logit exceeds it
        // by more than 2^8: rescaling O in TMEM is rare, and P stays below 2^8
        // (bf16 and fp32 lose nothing by a power of two).  So P is computed
        // before it is known whether another thread of the row has such a logit.
        float lsum_blk;
        uint32_t pk[8];
        auto weights = [&]() {
          const float mu = (m_run == -INFINITY) ? 0.f : m_run;
          lsum_blk = 0.f;
          float other = 0.f;
#pragma unroll
          for (int t = 0; t < 8; ++t) {
            const float pa = ex2(fmaf(x[2 * t], sl2e, -mu));
            const float pc = ex2(fmaf(x[2 * t + 1], sl2e, -mu));
            lsum_blk += pa;                        // the sum takes P before its rounding
            other += pc;
            pk[t] = pack_bf16x2(pa, pc);           // bf16: the operand type of the PV product
          }
          lsum_blk += other;
        };
        auto store_p = [&]() {
          put(pbuf + own0, pk);
          if (kept == 16) put(pbuf + own1, pk + 4);
          fence_proxy_async_smem();
        };
        const bool start = j == g.j0;              // nothing to compare with yet
        if (!start) {
          weights();
          store_p();
        }
        // (this barrier also ends the reads of the exchange, before the next block's)
        if (named_bar_or(group_bar, kSoftThreads / 2, start || bm > m_run + kRescaleThreshold)) {
          // the row's block max over its eight threads (lane pair x column parts)
          red(ch, half) = bm;
          named_bar_sync(group_bar, kSoftThreads / 2);
          bm = row_max();
          named_bar_sync(group_bar, kSoftThreads / 2);  // red makes room for the next exchange
          const bool need = bm > m_run + kRescaleThreshold;
          if (ok && (start || __any_sync(0xffffffffu, need))) {
            const float m_new = need ? bm : m_run;
            const float alpha = (m_run == -INFINITY || !need) ? (need ? 0.f : 1.f) : ex2(m_run - m_new);
            if (j > g.j0 && __any_sync(0xffffffffu, need && m_run != -INFINITY)) {
              // O must hold PV(G-1) before it is rescaled.  (The stage's next use needs
              // this block's P or, as a query's slot, s_free of the block after this one:
              // its st_empty cannot complete twice ahead of this wait.)
              ok = mbar_wait_warp(smem_u32(&sm.st_empty[(G - 1) % kStages]), ((G - 1) / kStages) & 1, c, abort_flag);
              tc_fence_after();
#pragma unroll 1
              for (int cc = 0; cc < 64 && ok; cc += 16) {
                const uint32_t oa = tmem + lane_off + kColO + 128 * (cc >> 5) + 32 * ch + (cc & 31);
                uint32_t o[16];
                tmem_ld16(oa, o);
                tmem_ld_wait16(o);
#pragma unroll
                for (int t = 0; t < 16; ++t) o[t] = __float_as_uint(__uint_as_float(o[t]) * alpha);
                tmem_st16(oa, o);
                tmem_st_wait();
              }
              tc_fence_before();
            }
            l_run *= alpha;
            m_run = m_new;
            weights();
            store_p();
          }
          named_bar_sync(group_bar, kSoftThreads / 2);
        }
        if (!ok) continue;
        l_run += lsum_blk;
        // after the barrier P of all the group's warps is there
        if (ch == 0 && half == 0 && lane == 0) arrive_leader_shared(&sm.p_full[pb], crank);
      }
      // ------------------------------- epilogue -------------------------------
      // the row's sum and maximum over its eight threads, while the last P V runs
      if (poison) l_run = NAN;
      red(ch, half) = l_run;
      named_bar_sync(group_bar, kSoftThreads / 2);
      float lsum = 0.f;
#pragma unroll
      for (int t = 0; t < 4; ++t) lsum += red(t, 0) + red(t, 1);
      named_bar_sync(group_bar, kSoftThreads / 2);
      red(ch, half) = m_own;
      named_bar_sync(group_bar, kSoftThreads / 2);
      const float m_true = row_max();
      if (ok) ok = mbar_wait_warp(smem_u32(&sm.mma_done[bi]), (i >> 1) & 1, c, abort_flag);
      if (!ok) continue;
      tc_fence_after();
      if (g.part >= 0) {
        // part of a tile: O as it stands, [column quad][row] so that a warp's
        // 32 rows make whole lines.  128 KB for 64 rows at the 32 bytes per cycle that
        // an SM writes (by any kind of store): 4,100 cycles.
        float4* po = parts + (size_t)g.part * (kTile * kDV / 4) + rr;
        const uint64_t stay = policy_stay();
#pragma unroll 1
        for (int m = 0; m < 2; ++m) {
          uint32_t o[32];
          tmem_ld32(tmem + lane_off + kColO + 128 * m + 32 * ch, o);
          tmem_ld_wait(o);
          const int quad0 = (256 * half + 128 * m + 32 * ch) / 4;
          if (!live) continue;
#pragma unroll
          for (int t = 0; t < 8; ++t)
            st_part(po + (size_t)(quad0 + t) * kTile, __uint_as_float(o[4 * t]), __uint_as_float(o[4 * t + 1]),
                    __uint_as_float(o[4 * t + 2]), __uint_as_float(o[4 * t + 3]), stay);
        }
        if (half == 0 && ch == 0 && live) stats[(size_t)g.part * kTile + rr] = make_float4(m_run, lsum, m_true, 0.f);
      } else {
        const float inv = lsum == 0.f ? 0.f : 1.f / lsum;  // no visible key: 0
        const long long row0 = (long long)g.t0 * a.H + 128ll * g.tile + kHC * (int)crank;  // first row of this CTA
        // A thread holds 64 columns of its row, 4 pieces of 32 bytes.  Four lanes
        // transpose theirs, so that a store of the warp fills 8 whole lines instead of
        // touching 32, and nobody waits for the stores.
        uint32_t w[4][8];
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          uint32_t o[32];
          tmem_ld32(tmem + lane_off + kColO + 64 * ch + 32 * m, o);
          tmem_ld_wait(o);
#pragma unroll
          for (int t = 0; t < 16; ++t)
            w[2 * m + (t >> 3)][t & 7] =
                pack_bf16x2(__uint_as_float(o[2 * t]) * inv, __uint_as_float(o[2 * t + 1]) * inv);
        }
#pragma unroll
        for (int d = 1; d < 4; d <<= 1) {
          const bool up = (lane & d) != 0;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (k & d) continue;                   // pieces k and k + d of lanes l and l ^ d
#pragma unroll
            for (int t = 0; t < 8; ++t) {
              const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? w[k][t] : w[k + d][t], d);
              if (up) w[k][t] = got;
              else w[k + d][t] = got;
            }
          }
        }
        const bool wide_out = (reinterpret_cast<uintptr_t>(out) & 31u) == 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {              // row k of the four lanes, this lane's piece
          const int r4 = (hl & ~3) + k;
          __nv_bfloat16* dst = out + (row0 + r4) * kDV + 256 * half + 64 * ch + 16 * (lane & 3);
          if (kHC * (int)crank + r4 >= rows) continue;
          if (wide_out) {
            st_global32(dst, w[k]);
          } else {
            reinterpret_cast<uint4*>(dst)[0] = make_uint4(w[k][0], w[k][1], w[k][2], w[k][3]);
            reinterpret_cast<uint4*>(dst)[1] = make_uint4(w[k][4], w[k][5], w[k][6], w[k][7]);
          }
        }
        if (half == 0 && ch == 0 && live) {
          const bool any = m_true != -INFINITY;
          mx[row0 + hl] = any ? m_true * kLn2 : -INFINITY;
          sm_out[row0 + hl] = lsum == 0.f ? 0.f : lsum * ex2(m_run - m_true);
        }
      }
      tc_fence_before();                           // O is overwritten by the next segment's first PV
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // the peer may still read our shared memory / arrive until here
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc2(tmem, kTmemCols);
  }
}

// Joins the parts of the tiles that several pairs worked on:
//   M = max m_k, w_k = 2^(m_k - M), l = sum w_k l_k, out = sum w_k O_k / l,
// in a fixed order.  A tile may have a part from every pair (one long sequence),
// or the batch a two-part tile from every pair.  Up to 8 parts, one thread takes
// all parts of one row's 8 columns; above, four threads share them.  What counts
// is that many loads are in flight (one thread for 4 columns of all 74 parts of a
// 16K-row sequence: 25 us).  64 sequences, 39 MB of parts: 12 us.
constexpr int kJoinThreads = 256, kJoinGroups = 4, kJoinFew = 8;
constexpr int kJoinPerPair = 6;                    // CTAs: what is resident at once (a CTA's start costs a piece's time)
constexpr int kMaxPairs = 256;

// parts k = g, g + step, ... of one row: running max, sum, true max, and O of two column quads
struct Joined {
  float M, l, true_max;
  float4 o[2];
};
// four parts at a time, all of their loads in flight together
__device__ __forceinline__ Joined join_parts(const float4* __restrict__ parts, const float4* __restrict__ stats,
                                             int pair, int nparts, int g, int step, int row, int q) {
  auto slot = [&](int k) { return (size_t)(k == 0 ? 2 * pair + 1 : 2 * (pair + k)); };
  constexpr int NQ = 2, U = 4;
  const uint64_t go = policy_go();
  Joined j;
  j.M = j.true_max = -INFINITY;
  j.l = 0.f;
#pragma unroll
  for (int t = 0; t < NQ; ++t) j.o[t] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (int k0 = g; k0 < nparts; k0 += U * step) {
    float4 s[U], v[U][NQ];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + u * step;
      const bool in = k < nparts;
      const size_t sl = slot(in ? k : k0);
      s[u] = stats[sl * kTile + row];
      const float4* p = parts + sl * (kTile * kDV / 4) + (size_t)q * kTile + row;
#pragma unroll
      for (int t = 0; t < NQ; ++t) v[u][t] = in ? ld_part(p + t * kTile, go) : make_float4(0.f, 0.f, 0.f, 0.f);
      if (!in) s[u] = make_float4(-INFINITY, 0.f, -INFINITY, 0.f);
    }
    float M = j.M;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      M = fmaxf(M, s[u].x);
      j.true_max = fmaxf(j.true_max, s[u].z);
    }
    const float mu = M == -INFINITY ? 0.f : M, w0 = ex2(j.M - mu);  // nothing so far: 2^-inf = 0
    j.l *= w0;
#pragma unroll
    for (int t = 0; t < NQ; ++t) j.o[t] = make_float4(w0 * j.o[t].x, w0 * j.o[t].y, w0 * j.o[t].z, w0 * j.o[t].w);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float w = ex2(s[u].x - mu);            // a part with no visible key: 0
      j.l = fmaf(w, s[u].y, j.l);
#pragma unroll
      for (int t = 0; t < NQ; ++t) {
        j.o[t].x = fmaf(w, v[u][t].x, j.o[t].x);
        j.o[t].y = fmaf(w, v[u][t].y, j.o[t].y);
        j.o[t].z = fmaf(w, v[u][t].z, j.o[t].z);
        j.o[t].w = fmaf(w, v[u][t].w, j.o[t].w);
      }
    }
    j.M = M;
  }
  return j;
}
__device__ __forceinline__ void join_store(const Joined& j, long long r, int q, __nv_bfloat16* out, float* mx,
                                           float* sm_out) {
  const float inv = j.l == 0.f ? 0.f : 1.f / j.l;
  uint2* dst = reinterpret_cast<uint2*>(out + r * kDV + 4 * q);
#pragma unroll
  for (int t = 0; t < 2; ++t)
    dst[t] = make_uint2(pack_bf16x2(j.o[t].x * inv, j.o[t].y * inv), pack_bf16x2(j.o[t].z * inv, j.o[t].w * inv));
  if (q == 0) {
    mx[r] = j.true_max == -INFINITY ? -INFINITY : j.true_max * kLn2;
    sm_out[r] = j.l == 0.f ? 0.f : j.l * ex2((j.M == -INFINITY ? 0.f : j.M) - j.true_max);
  }
}

// (three CTAs per SM: 93 registers and two took 3 us more for 64 tokens)
__global__ void __launch_bounds__(kJoinThreads, 3)
    tree_join_kernel(const float4* __restrict__ parts, const float4* __restrict__ stats,
                     const Join* __restrict__ joins, int npairs, __nv_bfloat16* __restrict__ out,
                     float* __restrict__ mx, float* __restrict__ sm_out) {
  __shared__ Joined shared[kJoinGroups - 1][64];
  __shared__ Join list[kMaxPairs];
  __shared__ uint16_t list_pair[kMaxPairs];
  __shared__ int below[kMaxPairs / 32];
  let_next_launch();
  wait_for_earlier();
  const int tid = threadIdx.x;
  // the pairs whose tile is to be joined, in order
  Join mine = {0, 0, 0};
  if (tid < npairs) mine = joins[tid];
  const uint32_t bits = __ballot_sync(0xffffffffu, mine.nparts > 0);
  if ((tid & 31) == 0) below[tid >> 5] = __popc(bits);
  __syncthreads();
  int at = __popc(bits & ((1u << (tid & 31)) - 1u)), n = 0;
#pragma unroll
  for (int w = 0; w < kMaxPairs / 32; ++w) {
    if (w < (tid >> 5)) at += below[w];
    n += below[w];
  }
  if (mine.nparts > 0) {
    list[at] = mine;
    list_pair[at] = (uint16_t)tid;
  }
  __syncthreads();
  int i = 0, base = 0;                             // tile, its first piece
  for (int piece = blockIdx.x;; piece += gridDim.x) {
    int pieces = 0;
    for (; i < n; ++i, base += pieces) {
      pieces = list[i].nparts <= kJoinFew ? 32 : 128;
      if (piece < base + pieces) break;
    }
    if (i == n) break;
    const Join jn = list[i];
    const int pair = list_pair[i], k = piece - base;
    if (jn.nparts <= kJoinFew) {                   // 128 rows x 2 x 8 columns
      const int row = tid & 127, q = 4 * k + 2 * (tid >> 7);
      if (row < jn.nrows)
        join_store(join_parts(parts, stats, pair, jn.nparts, 0, 1, row, q), jn.row0 + row, q, out, mx, sm_out);
      continue;
    }
    // 64 rows x 8 columns, four threads each
    const int cell = tid & 63, row = (k & 1) * 64 + cell, q = 2 * (k >> 1), g = tid >> 6;
    Joined j;
    if (row < jn.nrows) j = join_parts(parts, stats, pair, jn.nparts, g, kJoinGroups, row, q);
    __syncthreads();                               // the last piece's sums are read
    if (g > 0) shared[g - 1][cell] = j;
    __syncthreads();
    if (g > 0 || row >= jn.nrows) continue;
    Joined all = j;
#pragma unroll
    for (int t = 0; t < kJoinGroups - 1; ++t) {
      all.M = fmaxf(all.M, shared[t][cell].M);
      all.true_max = fmaxf(all.true_max, shared[t][cell].true_max);
    }
    const float mu = all.M == -INFINITY ? 0.f : all.M;
    auto add = [&](const Joined& p, bool first) {  // (no key in the group: weight 0)
      const float w = ex2(p.M - mu);
      all.l = fmaf(w, p.l, first ? 0.f : all.l);
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        all.o[t].x = fmaf(w, p.o[t].x, first ? 0.f : all.o[t].x);
        all.o[t].y = fmaf(w, p.o[t].y, first ? 0.f : all.o[t].y);
        all.o[t].z = fmaf(w, p.o[t].z, first ? 0.f : all.o[t].z);
        all.o[t].w = fmaf(w, p.o[t].w, first ? 0.f : all.o[t].w);
      }
    };
    add(j, true);
#pragma unroll
    for (int t = 0; t < kJoinGroups - 1; ++t) add(shared[t][cell], false);
    join_store(all, jn.row0 + row, q, out, mx, sm_out);
  }
}

}  // namespace tree

bool make_tmap_bf16(CUtensorMap* tm, const void* base, int rank, const uint64_t* dims, const uint64_t* strides,
                    const uint32_t* box, int swizzle_bytes);

// CTA pairs of the kernel at most: one CTA per SM (152 SMs when there is no device to ask)
static int tree_pairs_bound() {
  int dev = 0, sms = 0;
  if (!cuda_ok(cudaGetDevice(&dev)) || !cuda_ok(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) ||
      sms < 2)
    sms = 152;
  return sms / 2;
}
static size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }
size_t tree_tc_workspace() {
  const size_t n = (size_t)tree_pairs_bound();
  return up256(2 * n * tree::kPartBytes) + up256(2 * n * tree::kStatBytes) + up256(n * sizeof(tree::Join));
}

int launch_tree_attn_tc(const TreeArgs& a, const void* q, const void* pool, long long page_stride, const void* kv_new,
                        void* out, float* mx, float* sm, void* ws, DevCtx c, cudaStream_t st) {
  using namespace tree;
  const size_t smem = sizeof(Smem);
  if (!cuda_ok(cudaFuncSetAttribute(tree_attn_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)))
    return DSA_ERR_CUDA;
  static int pairs_by_device[64] = {0};
  int dev = 0;
  if (!cuda_ok(cudaGetDevice(&dev))) return DSA_ERR_CUDA;
  int pairs = dev < 64 ? pairs_by_device[dev] : 0;
  if (pairs <= 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    if (!cuda_ok(cudaOccupancyMaxActiveClusters(&pairs, tree_attn_tc_kernel, &cfg)) || pairs <= 0)
      pairs = tree_pairs_bound();
    if (dev < 64) pairs_by_device[dev] = pairs;
  }
  const int bound = tree_pairs_bound();
  if (pairs > bound) pairs = bound;
  if (pairs > kMaxPairs) pairs = kMaxPairs;
  const size_t n = (size_t)bound;
  float4* parts = (float4*)ws;
  float4* stats = (float4*)((uint8_t*)ws + up256(2 * n * kPartBytes));
  Join* joins = (Join*)((uint8_t*)ws + up256(2 * n * kPartBytes) + up256(2 * n * kStatBytes));
  CUtensorMap pv, pv2, pr, pr2, nv, nr, pq;
  // cached value columns: 64 columns, 8 rows, 64-column blocks, 8-row groups, pages; drafted ones: any first row
  const uint64_t row = kDQK * 2, R = (uint64_t)a.R, P = (uint64_t)a.n_pages, N = (uint64_t)a.n_tok;
  const uint64_t pv_dim[5] = {64, 8, 8, R / 8, P}, pv_str[4] = {row, 128, 8 * row, (uint64_t)page_stride};
  const uint64_t pr_dim[3] = {kDQK, R, P}, pr_str[2] = {row, (uint64_t)page_stride};
  const uint64_t nv_dim[3] = {64, N, 8}, nv_str[2] = {row, 128};
  const uint64_t nr_dim[2] = {kDQK, N}, nr_str[1] = {row};
  const uint32_t pv_box[5] = {64, 8, 4, 2, 1}, pr_box[3] = {32, 16, 1}, nv_box[3] = {64, 8, 4}, nr_box[2] = {32, 16};
  const uint64_t pq_dim[2] = {kDQK, N * (uint64_t)a.H}, pq_str[1] = {row};
  const uint32_t pq_box[2] = {64, kHC};
  const int wide = a.R % 32 == 0;                  // two groups of 16 rows per copy
  const uint32_t pv2_box[5] = {64, 8, 4, wide ? 4u : 2u, 1}, pr2_box[3] = {32, wide ? 32u : 16u, 1};
  if (!make_tmap_bf16(&pv, pool, 5, pv_dim, pv_str, pv_box, 128) ||
      !make_tmap_bf16(&pv2, pool, 5, pv_dim, pv_str, pv2_box, 128) ||
      !make_tmap_bf16(&pr, pool, 3, pr_dim, pr_str, pr_box, 64) ||
      !make_tmap_bf16(&pr2, pool, 3, pr_dim, pr_str, pr2_box, 64) ||
      !make_tmap_bf16(&nv, kv_new, 3, nv_dim, nv_str, nv_box, 128) ||
      !make_tmap_bf16(&nr, kv_new, 2, nr_dim, nr_str, nr_box, 64) ||
      !make_tmap_bf16(&pq, q, 2, pq_dim, pq_str, pq_box, 128))
    return DSA_ERR_CUDA;
  if (!launch_programmatic(tree_attn_tc_kernel, dim3(2 * pairs), dim3(kThreads), smem, st, 1, a, (const __nv_bfloat16*)q,
                           (const __nv_bfloat16*)kv_new, (__nv_bfloat16*)out, mx, sm, parts, stats, joins, c, wide, pv,
                           pv2, pr, pr2, nv, nr, pq))
    return DSA_ERR_CUDA;
  return launch_programmatic(tree_join_kernel, dim3(kJoinPerPair * pairs), dim3(kJoinThreads), 0, st, 1,
                             (const float4*)parts, (const float4*)stats, (const Join*)joins, pairs,
                             (__nv_bfloat16*)out, mx, sm)
             ? DSA_OK
             : DSA_ERR_CUDA;
}

}  // namespace dsa
