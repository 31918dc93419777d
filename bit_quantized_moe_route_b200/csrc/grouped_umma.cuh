// Grouped products on the 5th-generation tensor cores (sm_100a): TMA loads,
// tcgen05.mma on pairs of SMs, accumulators in tensor memory.
//
// A tile is 256 values of the M side (128 per CTA of the pair) by up to 256 of
// the N side: where that is the rows of an expert, they are cut into equal
// tiles of at most 256 (8-bit: 128), rounded up to 16 (32), so that an expert with
// few rows costs a narrow MMA and not a padded tile.  Steps of the
// contracted dimension are 128 bytes per row: 64 16-bit values or 128 e4m3
// codes, the block of the 8-bit scales.
//
//   kernel      M side (A operand)         N side (B operand)
//   mm          W[e] rows o, K-major       x rows, K-major
//   dx          W[e] columns i, M-major    dy rows, K-major
//   dw          dy columns o, M-major      x columns i, N-major
//   mm, ROWM    x rows, K-major            W[e] rows o, K-major
//
// With the rows on the M side (ROWM: dw, whose output rows are o, and the 8-bit
// product of many rows per expert) a thread has one output row and one row
// scale; with them on the N side the M side is the output's contiguous
// dimension.  Either way the output leaves through shared memory, in whole
// lines (the 8-bit product of aligned rows: from the registers).
//
// MT = 2 (16-bit products with enough tiles): a tile is 512 values of the M
// side, two MMAs of 256 that share the B operand.  Per product that moves three
// quarters of the bytes from L2 to the SMs, and those bytes are what a 1000 W
// card runs out of first: 32,768 rows over 32 experts, in a loop, took 502 us
// with 256 x 256 tiles at an SM clock of 1110 MHz, with the tensor pipe 81 %
// busy at that clock.
//
// One tile step is MT x 16 KB of A and up to 16 KB of B per CTA, in a ring of
// six (MT = 2: four).
// M- and N-major operands are 64-value panels of 64 contracted rows.  For dw
// the contracted rows are the expert's: in its last step only the rows that
// are left are copied, in boxes of 32 rows to one, and the rest of the last 16
// comes from beyond the tensor's end, which TMA fills with zeros, so that no
// value of another expert's rows (a NaN, say) enters a product.
//
// ANY: operands of any alignment and row stride.  TMA takes 16-byte aligned
// rows whose strides are multiples of 16 bytes, and 8 rows (e4m3: 16) are that
// far apart whatever one row's stride is: each operand has 8 (16) tensor maps,
// one for the rows of each number modulo 8, from the aligned block on that
// holds its first row's first byte.  They bring the aligned blocks that hold a
// step's rows to shared memory, three steps at a time on their way; eight more
// warps cut the operands' 16-byte pieces out of two neighbouring blocks each
// and store them where TMA would have put them, for two operand stages.  Bound
// by those warps' shared memory traffic: 32,768 rows over 32 experts with 2,047
// inputs run at 628 TFLOP/s (mm), 558 (dx), 542 (dw) and 429 (8-bit); with
// asynchronous 16-byte copies instead of TMA it was 382, 344, 354 and 422.
//
// The tiles, in the order expert, M tile, row tile, are dealt out to the pairs
// of CTAs in turn, so that pairs that run at the same time read the same
// weights and rows from L2 (with each pair on a run of neighbouring tiles
// instead, 74 pairs stream 148 MB between two uses of an operand tile, more
// than L2 holds: 32,768 rows over 32 experts took 870 us that way, 588 dealt
// out).  All but the last one to two tiles per pair are dealt whole, and as
// many of the rest's halves as there are for all pairs.  What is then left is
// dealt whole too, or cut evenly, a number of pairs to each, or (dw, whose tiles
// differ in length, and few tiles) cut by steps: their steps are one line, cut
// so that every pair has the same cost in all.  Which, is what steps and joins
// cost (gu_plan): one 8-bit token, 4096 -> 2048, is eight tiles in four parts
// each; one token over eight 16-bit experts of that size is 64 tiles dealt
// whole, with ten of the 74 pairs idle.  A tile that a cut goes through is summed by
// the pairs that hold parts of it: each writes its fp32 partial sums to the
// workspace and counts itself in; the last one adds the partials in the
// pieces' order (so the result does not depend on who was last) and writes
// the outputs.  No pair waits for another.  This costs at most two partial
// tiles per pair.
//
// Tensor memory is a ring of eight slots of 64 columns; a sum takes one, two
// or four of them, so that narrow tiles have up to eight sums in flight
// between the MMA and the epilogue.
//
// CHAIN = 0: the tile's whole sum is taken in tensor memory.  CHAIN > 0: every
// CHAIN steps the sum is handed to the epilogue warps, which add it to sums in
// registers with ordinary fp32 additions.  The tensor core truncates as it adds:
// for positive operands a sum of 65,536 products taken whole is 1.0e-5 of its
// size too low and one of 2^20 3.8e-4, chained both are 1.1e-7.  So outputs in
// fp32 are chained, whatever the operands' alignment.
//
// The 8-bit product hands over every step (CHAIN = 1), since its scales change
// there: register sum += scale[row] * step sum, on pairs of columns (packed
// fp32 instructions).  The hand-over costs some 2,000 cycles there and back
// (commit, barriers of two CTAs, TMEM reads) against 512 for the MMA of a
// 256-row tile, so a half of tensor memory holds one step of a wide tile, two
// of a tile of up to 128 rows or four of up to 64, handed over together, and
// is given back when its last values are in registers.  With the rows on the
// M side a thread holds 128 sums and 64 of a step's, of 208 registers: what
// makes the compiler spill four bytes there costs a third (32,768 rows over 32
// experts: 430 us, not 317).
#pragma once

#include <cuda.h>

#include <type_traits>

#include "ffn_umma.cuh"
#include "grouped_plan.cuh"

namespace moe {

constexpr int kGuTile = 16384;            // bytes of 128 operand rows of one step
constexpr int kGuRing = 12 * kGuTile;
// ANY: two stages, and the aligned blocks of three steps
constexpr int kGuRaw = 128 * (128 + 16);  // (64 rows of 256 + 16 are less)
constexpr int kGuRaws = 3;
static_assert(2 * 2 * kGuTile + kGuRaws * 2 * kGuRaw <= kGuRing, "operand ring");
// bytes from the blocks of one class of rows (their number modulo 16 or, for
// 16-bit values, 8) to the next's; `few`: 32 rows, not 128.  TMA wants
// multiples of 128.
template <bool FP8>
constexpr uint32_t gu_raw_class(bool mn, bool few) {
  const int r = FP8 ? 16 : 8;
  return mn ? 64 / r * 272 : few ? (32 / r * 144 + 127) / 128 * 128 : 128 / r * 144;
}
static_assert(gu_raw_class<false>(true, false) % 128 == 0 && gu_raw_class<false>(false, false) % 128 == 0 &&
                  gu_raw_class<true>(false, false) % 128 == 0,
              "TMA's alignment in shared memory");
constexpr int kGuN = 256;                 // output rows per tile
// Warps: 0 loads, 1 MMA, 2 scales, 3 items, 4-11 the epilogue, two for each 32
// TMEM lanes.  (Sixteen epilogue warps were slower: each barrier wait and
// shared-memory access takes some 300 clocks beside the MMA's and TMA's own
// traffic, and twice the warps make twice as many.)
constexpr int kGuEpiWarps = 8;
constexpr int kGuThreads = 128 + 32 * kGuEpiWarps;
constexpr int kGuStageRows = 16;          // output rows that a warp stores together
// Registers per thread at launch and, where the epilogue holds a tile's sums or
// rounded outputs, then of warps 0-3 and of the epilogue.
constexpr bool gu_hand_over(int mt, int chain) { return mt > 1 || chain > 0; }
// ANY: eight more warps; less for each.
constexpr int kGuLoadWarps = 8;
constexpr int gu_threads(bool any) { return kGuThreads + (any ? 32 * kGuLoadWarps : 0); }
constexpr int kGuAnyRegs = 96;
struct GuAnyShare {  // of warps 0-3, the load warps and the epilogue
  int low, load, high;
  constexpr bool fits() const {
    return 128 * low + 32 * kGuLoadWarps * load + 32 * kGuEpiWarps * high <= gu_threads(true) * kGuAnyRegs;
  }
};
// Chained 16-bit sums are 128 in each thread of the epilogue.  (With 64 of them, tiles half as wide, and the other
// split: 32,768 rows over 32 experts with 2,047 inputs took 1,476 / 1,501 / 1,524 us, not 921 / 1,023 / 1,098: mm, dx, dw.)
constexpr GuAnyShare gu_any_share(bool fp8, int chain) {
  return chain > 0 && !fp8 ? GuAnyShare{48, 48, 168} : GuAnyShare{64, 64, 144};
}
static_assert(gu_any_share(true, 1).fits() && gu_any_share(false, 0).fits() && gu_any_share(false, 8).fits(),
              "registers of the block");
constexpr int kGuRegs = 168, kGuRegsLow = 88, kGuRegsHigh = 208;
static_assert(128 * kGuRegsLow + (kGuThreads - 128) * kGuRegsHigh <= kGuThreads * kGuRegs, "registers of the block");
constexpr int gu_launch_regs(bool any) { return any ? kGuAnyRegs : kGuRegs; }
constexpr int kGuScaleSlots = 5;
constexpr int kGuScaleAhead = 4;          // slots whose copies are in flight
constexpr int kGuItems = 4;               // items handed out ahead
constexpr int kGuSegs = 8;                // sums between the MMA and the epilogue; TMEM slots
constexpr int kGuSlotCols = 512 / kGuSegs;
constexpr int kGuPart = 128 * kGuN * 4;   // bytes of one partial tile of one CTA
constexpr int kGuPairsMax = 74;
constexpr long long kGuLinger = 4000000;  // ~2 ms
constexpr size_t kGuCounters = 1024;      // workspace: counters, then the partial tiles
constexpr size_t kGuParts = 4096;
constexpr size_t kGuWsBytes = size_t(40) << 20;
static_assert(kGuPairsMax <= 96, "the plan's threads");
static_assert(kGuCounters + kGuPairsMax * 2 * 4 <= kGuParts, "counters");
static_assert(kGuParts + (size_t)kGuPairsMax * 4 * kGuPart <= kGuWsBytes, "workspace");

struct alignas(64) GuParams {
  CUtensorMap a_map;     // mm, dx: W; dw: dy, 64 rows
  CUtensorMap b_map[4];  // mm, dx: rows in boxes of 16, 32, 64, 128; dw: x, 64 rows
  CUtensorMap a_tail[6], b_tail[6];  // dw: boxes of 32, 16, .. 1 rows
  GmmProblem g;
  int type;              // GmmType of the operands
  int split_most;        // pieces that a tile may be cut into
  unsigned char* ws;
};

// ANY: rows c, c + R, .. of an operand, from the aligned block that holds the
// first byte of row c on (R rows are a multiple of 16 bytes apart).
template <bool FP8>
struct alignas(64) GuAnyParams : GuParams {
  static constexpr int R = FP8 ? 16 : 8;
  CUtensorMap a_rows[R], b_rows[R], b_few[R];  // b_few: of 32 rows, not 128
};
template <bool FP8, bool ANY>
using GuKernelParams = std::conditional_t<ANY, GuAnyParams<FP8>, GuParams>;

// ------------------------------------------------------------ PTX wrappers
// 4-byte copy to shared memory, zero if not `in`
MOE_DEV void gu_cp4(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(in ? 4 : 0) : "memory");
}
MOE_DEV void gu_tma_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  um_tma_2d_pair(dst, map, x, y, bar);
}
MOE_DEV void gu_tma_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, "
      "%4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
template <bool FP8>
MOE_DEV void gu_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  if constexpr (FP8)
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
// 128-byte swizzled operand.  K-major: 8-row groups 1024 bytes apart.  M- or
// N-major: panels of 64 values, 8192 bytes apart, whose contracted rows are
// 128 bytes, in groups of eight 1024 bytes apart.
MOE_DEV uint64_t gu_desc(uint32_t saddr, bool major_mn) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)(major_mn ? 8192u >> 4 : 1u) << 16) |
         ((uint64_t)(1024u >> 4) << 32) | ((uint64_t)1u << 46) | ((uint64_t)2u << 61);
}
// 32 consecutive TMEM columns of this warp's 32 lanes
MOE_DEV void gu_ld32(uint32_t taddr, float (&v)[32]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// the same, without the wait: v is complete after gu_ld_wait
MOE_DEV void gu_ld_issue(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
MOE_DEV void gu_ld_issue(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
// waits for every load issued; r's uses stay behind it
template <int W>
MOE_DEV void gu_ld_wait(uint32_t (&r)[W]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < W; ++i) asm volatile("" : "+r"(r[i]));
}

// two fp32 in one register pair, and the packed instructions on them
MOE_DEV unsigned long long gu_pack(float lo, float hi) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
MOE_DEV void gu_unpack(unsigned long long v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
MOE_DEV void gu_fma2(unsigned long long& c, unsigned long long a, unsigned long long b) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(c) : "l"(a), "l"(b));
}
MOE_DEV ulonglong2 gu_lds_u64x2(uint32_t a) {
  ulonglong2 v;
  asm volatile("ld.shared.v2.u64 {%0,%1}, [%2];" : "=l"(v.x), "=l"(v.y) : "r"(a));
  return v;
}
// W step sums times their columns' scales into register sums c0, c0 + 1, ...
template <int W>
MOE_DEV void gu_scaled(unsigned long long (&acc)[16], const int c0, const uint32_t (&r)[W], uint32_t scales) {
#pragma unroll
  for (int i = 0; i < W; i += 4) {
    const ulonglong2 s = gu_lds_u64x2(scales + 4u * i);
    gu_fma2(acc[(c0 + i) / 2], gu_pack(__uint_as_float(r[i]), __uint_as_float(r[i + 1])), s.x);
    gu_fma2(acc[(c0 + i) / 2 + 1], gu_pack(__uint_as_float(r[i + 2]), __uint_as_float(r[i + 3])), s.y);
  }
}
// 32 step sums times one scale (in both halves of `s`)
MOE_DEV void gu_times(unsigned long long (&acc)[16], const uint32_t (&r)[32], unsigned long long s) {
#pragma unroll
  for (int i = 0; i < 32; i += 2) gu_fma2(acc[i / 2], gu_pack(__uint_as_float(r[i]), __uint_as_float(r[i + 1])), s);
}
MOE_DEV void gu_add2(unsigned long long& c, unsigned long long a) { asm("add.rn.f32x2 %0, %0, %1;" : "+l"(c) : "l"(a)); }
// ANY: the 16 bytes from byte `shift` of two blocks on, to where TMA would put them
MOE_DEV void gu_cut16(uint32_t to, uint4 a, uint4 b, uint32_t shift) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  uint32_t t[6], u[5], o[4];
#pragma unroll
  for (int i = 0; i < 6; ++i) t[i] = shift & 8 ? w[i + 2] : w[i];
#pragma unroll
  for (int i = 0; i < 5; ++i) u[i] = shift & 4 ? t[i + 1] : t[i];
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = __funnelshift_r(u[i], u[i + 1], (shift & 3) * 8);
  tc_sts128(to, o[0], o[1], o[2], o[3]);
}

// ------------------------------------------------------------ work items
// A run of steps of one tile.
struct alignas(16) GuItem {
  int e, m0, n0, nv;       // expert, first M and N value (rows: of the whole input), N values in use
  int np, kb0, kb1, nkb;   // MMA width, steps, the tile's number of steps
  int cost, r0, r1;        // of one step; dw: the expert's rows
  int kind;                // GuKind
  long long pos;           // where the tile begins on the line
  int mv, halves;          // M values in use; MMAs of 256 of them (at most MT)
};
static_assert(sizeof(GuItem) == 64, "four 16-byte pieces");
enum GuKind : int {
  GU_RUN = 0,
  GU_ZEROS = 1,  // dw: an expert without rows; one step that reads nothing, zeros to write
  GU_STOP = 2    // no more items
};

constexpr int kGuTailMost = 2 * 2 * kGuPairsMax;  // two tiles per pair, in halves

// The plan of a launch (shared memory of each CTA; the same in all of them).
struct alignas(16) GuLine {
  long long tail[kGuTailMost + 1];  // the tiles that are split: where each begins on the line of costs
  long long cut[kGuPairsMax + 1];   // where each pair's piece of that line begins
  long long hand[kGuPairsMax];      // cost of the tiles that each pair has whole
  GuItem item[kGuItems];
  int off[kGmmMaxExperts + 1];      // the experts' rows
  int cum[kGmmMaxExperts + 1];      // the experts' tiles
  int chunk[kGmmMaxExperts / 32];
  int steps_most;                   // dw: of a tile
};

// shared memory from the first 1024-byte boundary: operand ring, scales, the
// epilogue's rows on their way out, plan, barriers
constexpr uint32_t kGuScaleOff = kGuRing;
constexpr uint32_t kGuOutOff = kGuScaleOff + kGuScaleSlots * kGuN * 4;
constexpr uint32_t kGuLineOff = kGuOutOff + kGuEpiWarps * kGuStageRows * 128;
constexpr uint32_t kGuBarOff = kGuLineOff + sizeof(GuLine);
constexpr size_t gu_smem() { return 1024 + kGuBarOff + 512; }
static_assert(gu_smem() <= 227 * 1024, "shared memory");

template <int OP, bool FP8, bool ROWM, int MT_, bool ANY>
struct GuTiles {
  static constexpr int MT = MT_;
  static constexpr bool kRowsM = ROWM, kFp8 = FP8, kAny = ANY;
  static constexpr bool kMFast = ROWM && OP != G_DW;            // tiles in turn: along the M side first
  static constexpr int KE = FP8 ? 128 : 64;                     // contracted values per step
  static constexpr int kMost = FP8 && !ROWM ? 128 : kGuN;       // N values per tile
  // N values per MMA in multiples of 16 (8-bit: 32; dw: whole 64-value panels in both CTAs)
  static constexpr int kRound = OP == G_DW ? 128 : FP8 ? 32 : 16;
  MOE_DEV static int m_all(const GmmProblem& p, int rows) {
    return OP == G_DX ? p.n_in : OP == G_MM && ROWM ? rows : p.n_out;
  }
  MOE_DEV static int n_all(const GmmProblem& p, int rows) {
    return OP == G_DW ? p.n_in : OP == G_MM && ROWM ? p.n_out : rows;
  }
  MOE_DEV static int m_count(const GmmProblem& p, int rows) { return (m_all(p, rows) + 256 * MT - 1) / (256 * MT); }
  MOE_DEV static int n_count(int n) { return (n + kMost - 1) / kMost; }
  MOE_DEV static int of_expert(const GmmProblem& p, int rows) { return m_count(p, rows) * n_count(n_all(p, rows)); }
  MOE_DEV static int steps(const GmmProblem& p, int rows) {
    return OP == G_MM ? (p.n_in + KE - 1) / KE : OP == G_DX ? (p.n_out + KE - 1) / KE : max(1, (rows + KE - 1) / KE);
  }
  // N values per tile: n of them are cut into nt equal tiles (8-bit weight rows: into whole scale blocks)
  MOE_DEV static int width(int n, int nt) {
    if (FP8 && ROWM) return kGuN;
    return min(kMost, (int)(((unsigned)n + nt - 1) / (unsigned)nt + kRound - 1) & ~(kRound - 1));
  }
  MOE_DEV static int padded(int nv) { return max(kRound, (nv + kRound - 1) & ~(kRound - 1)); }
  // A step's cost is its operands' bytes (256 rows of A, np of B), between
  // that of reading weights from HBM (the same for every np) and that of the MMA.
  MOE_DEV static int cost(int np, int halves) { return 256 * halves + np; }
  // Tile g whole.  Neighbouring tiles share weights (mm, dx; 8-bit rows on the M
  // side too) or columns of dy: dw's then write neighbouring lines (the tiles of
  // one column in turn instead: 187 us, not 181, for 260 rows over ten experts).
  MOE_DEV static void get(const GmmProblem& p, const GuLine& l, int g, GuItem& it) {
    int lo = 0, hi = p.E;  // cum[lo] <= g < cum[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (l.cum[mid] <= g) lo = mid;
      else hi = mid;
    }
    it.e = lo;
    it.r0 = l.off[lo];
    it.r1 = l.off[lo + 1];
    const int rows = it.r1 - it.r0, n = n_all(p, rows), nt = n_count(n), tn = width(n, nt);
    const unsigned fast = (unsigned)(kMFast ? m_count(p, rows) : nt), tile = (unsigned)(g - l.cum[lo]);
    const int slow = (int)(tile / fast), quick = (int)(tile - (unsigned)slow * fast);
    const int t_m = kMFast ? quick : slow, t_n = kMFast ? slow : quick;
    it.m0 = t_m * 256 * MT;
    it.mv = m_all(p, rows) - it.m0;
    it.halves = MT == 1 || it.mv <= 256 ? 1 : 2;
    it.n0 = t_n * tn;
    it.nv = max(0, min(tn, n - it.n0));
    it.np = padded(it.nv);
    if (OP != G_DW) {
      if (ROWM) it.m0 += it.r0;
      else it.n0 += it.r0;
    }
    it.nkb = steps(p, rows);
    it.kind = OP == G_DW && rows == 0 ? GU_ZEROS : GU_RUN;
    it.cost = cost(it.np, it.halves);
  }
  // Of the tiles that are split, number t after the first `dealt`: halves of 256 M values.
  MOE_DEV static void get_tail(const GmmProblem& p, const GuLine& l, int dealt, int t, GuItem& it) {
    get(p, l, dealt + t / MT, it);
    if (MT > 1) {
      it.m0 += 256 * (t % MT);
      it.mv -= 256 * (t % MT);
      it.halves = 1;
      it.cost = cost(it.np, 1);
      if (it.mv <= 0) it.nkb = 0;  // (the tile has one half)
    }
  }
};

// TMEM slots of sums n wide, in a ring; the MMA and the epilogue walk it alike.
struct GuRing {
  int pos = 0, used = 0;
  MOE_DEV int take(int np) {  // first slot; `used`: how many
    used = np <= kGuSlotCols ? 1 : np <= 2 * kGuSlotCols ? 2 : 4;
    const int at = ((pos + used - 1) & ~(used - 1)) & (kGuSegs - 1);
    pos = at + used;
    return at;
  }
};

// 8-bit product, rows on the N side: columns per step in a half of tensor
// memory, which holds 256 / stride steps.
MOE_DEV int gu_stride(int np) { return np <= 64 ? 64 : 128; }

// Walks a pair's work; every warp that does, and both CTAs of the pair, see the same items.
template <typename Tiles>
struct GuWalk {
  const GmmProblem& p;
  const GuLine& l;
  int pair, cols, n_tiles, whole, halves;  // whole, halves: tiles and half tiles dealt to each pair
  int row;
  long long begin, end;

  MOE_DEV GuWalk(const GmmProblem& p_, const GuLine& l_, int pair_, int cols_, int n_tiles_, int whole_, int halves_)
      : p(p_), l(l_), pair(pair_), cols(cols_), n_tiles(n_tiles_), whole(whole_), halves(halves_), row(0) {
    begin = l.cut[pair];
    end = l.cut[pair + 1];
    if (whole + halves == 0) seek();
  }
  // tiles (halves for MT = 2) on the line
  MOE_DEV int on_line() const { return (n_tiles - whole * cols) * Tiles::MT - halves * cols; }
  // to the piece's first tile: the last one that begins at or before it
  MOE_DEV void seek() {
    if (begin == end) return;
    int lo = 0, hi = on_line();
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (l.tail[mid] <= begin) lo = mid;
      else hi = mid;
    }
    row = whole + halves + lo;
  }
  MOE_DEV bool next(GuItem& it) {
    for (;;) {
      const int t = row - whole - halves;
      if (t >= 0 && (begin >= end || t >= on_line() || l.tail[t] >= end)) return false;
      if (row < whole) Tiles::get(p, l, row * cols + pair, it);
      else Tiles::get_tail(p, l, whole * cols, t < 0 ? (row - whole) * cols + pair : halves * cols + t, it);
      ++row;
      it.kb0 = 0;
      it.kb1 = it.nkb;
      it.pos = 0;
      if (t < 0) {
        if (t == -1) seek();
      } else {
        it.pos = l.tail[t];
        it.kb0 = steps_before(begin, it);
        it.kb1 = steps_before(end, it);
      }
      if (it.kb0 < it.kb1) return true;
    }
  }
  // steps of the tile that begin before `at`
  MOE_DEV static int steps_before(long long at, const GuItem& it) {
    const long long d = at - it.pos;
    if (d <= 0) return 0;
    if (d > (long long)(it.nkb - 1) * it.cost) return it.nkb;
    return d < (1LL << 31) ? (int)(((unsigned)d + it.cost - 1) / (unsigned)it.cost) : (int)((d + it.cost - 1) / it.cost);
  }
};

// Fills the plan; called by NT threads (0 .. NT-1 = tid): the item warp alone,
// or, for dw, whose tiles differ in length by the experts' rows, the block.
// Returns the number of tiles, -1 when the offsets are not valid (they are the
// caller's, and checked before any is used as an index: 0 <= off[0] <= ... <=
// off[E] <= rows).
template <int OP, typename Tiles, int NT>
MOE_DEV int gu_plan(const GmmProblem& p, GuLine& l, int tid, int cols, int split_most, int* whole_out,
                    int* halves_out) {
  const int warp = tid >> 5, lane = tid & 31;
  auto sync = [] {
    if constexpr (NT == 32) __syncwarp();
    else __syncthreads();
  };
#pragma unroll 4
  for (int e = tid; e <= p.E; e += NT) l.off[e] = gmm_off(p, e);
  if (tid == 0) l.steps_most = 0;
  sync();
  int bad = 0;
  const int chunks = (p.E + 31) >> 5;
  for (int k = warp; k < chunks; k += NT / 32) {
    const int e = 32 * k + lane;
    int n = 0;
    if (e < p.E) {
      const int a = l.off[e], b = l.off[e + 1];
      if (a < 0 || b < a || b > p.rows) bad = 1;
      else n = Tiles::of_expert(p, b - a);
      if (OP == G_DW && !bad) atomicMax(&l.steps_most, Tiles::steps(p, b - a));
    }
    int x = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (e < p.E) l.cum[e] = x - n;
    if (lane == 31) l.chunk[k] = x;
  }
  if constexpr (NT == 32) bad = __any_sync(0xffffffffu, bad);
  else bad = __syncthreads_or(bad);
  if (bad) return -1;
  sync();
  int x = lane < chunks ? l.chunk[lane] : 0;  // (at most 32 chunks)
  const int own = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  const int n_tiles = __shfl_sync(0xffffffffu, x, 31);
  for (int k = warp; k < chunks; k += NT / 32) {
    const int before = __shfl_sync(0xffffffffu, x - own, k);
    if (k > 0 && 32 * k + lane < p.E) l.cum[32 * k + lane] += before;
  }
  if (tid == 0) l.cum[p.E] = n_tiles;
  const int whole = max(0, n_tiles / cols - 1), dealt = whole * cols, rest = (n_tiles - dealt) * Tiles::MT;
  if constexpr (OP == G_DW)
    for (int i = tid; i < cols; i += NT) l.hand[i] = 0;
  sync();
  // What each pair's whole tiles cost.  mm, dx: as good as the same for all
  // pairs.  dw: a tile's steps are its expert's rows.
  if constexpr (OP == G_DW) {
    const int q = tid % 96, part = tid / 96;  // (threads beyond a multiple of 96 have no part)
    if (whole > 0 && q < cols && part < NT / 96) {
      long long c = 0;
      for (int e = part; e < p.E; e += NT / 96) {
        const int g0 = min(l.cum[e], dealt), g1 = min(l.cum[e + 1], dealt);
        const int n = (g1 + cols - 1 - q) / cols - (g0 + cols - 1 - q) / cols;  // tiles q, q + cols, ... among them
        c += (long long)n * Tiles::steps(p, l.off[e + 1] - l.off[e]);
      }
      c *= Tiles::cost(Tiles::padded(Tiles::width(p.n_in, Tiles::n_count(p.n_in))), Tiles::MT);
      atomicAdd(reinterpret_cast<unsigned long long*>(&l.hand[q]), (unsigned long long)c);
    }
  }
  // What is left (halves of tiles for MT = 2; at most kGuTailMost - 1): as many
  // as there are for every pair are dealt too, and each of the others is cut
  // evenly, for at most as many pairs as there are, or all of it is the line,
  // whichever costs less.  Measured, in us, for tiles of np columns, with
  // operands in L2 (a step whose weights come from HBM takes longer): a step
  // 0.145 + np / 3000 (8-bit of over 64 columns, which hand over every other
  // step: 0.45; ANY: 0.45 + np / 470); joining k parts 0.4 + np / 62 + k (0.2 +
  // np / 154).  E.g. 128 steps of 32 columns: whole 33.0, in four 18.2, eight
  // 17.2, sixteen 20.1; 19 steps of 240: whole 13.6, in two 20.7.  dw, whose
  // tiles differ in length:
  // dealt if the longest have at most 40 steps, else the line.  Dealt / line, us,
  // for ten experts of 4096 -> 2048: 4 steps 85 / 105, 20 steps 163 / 178, 40 steps
  // 301 / 314, 80 steps 692 / 696, 160 steps 1,340 / 1,289; six of 1024 -> 1024: 4
  // steps 18 / 32, 40 steps 60 / 67, 80 steps 104 / 102, 160 steps 209 / 179.
  int halves = 0, each_in = 0;
  {
    const int q = rest / cols, r = rest - q * cols;
    if constexpr (OP == G_DW) {
      if (l.steps_most <= 40) {
        halves = q;
        each_in = 1;
      }
    } else {
      const float steps = (float)Tiles::steps(p, 0);
      const int rows = l.off[p.E] - l.off[0], m_tiles = max(1, Tiles::m_count(p, rows));
      // columns of a tile, on average
      const float np = Tiles::kRowsM ? (float)min(kGuN, p.n_out)
                                     : fminf((float)kGuN, (float)rows * m_tiles / max(1, n_tiles) + 8.f);
      const float step = Tiles::kAny                ? 0.45f + np * (1.f / 470.f)
                         : Tiles::kFp8 && np > 64.f ? 0.45f
                                                    : 0.145f + np * (1.f / 3000.f);
      const float join = 0.4f + np * (1.f / 62.f), part = 0.2f + np * (1.f / 154.f);
      float best = r ? steps * step : 0.f;
      int k = 1;
      for (int i = 2; r && i <= min(split_most, cols / r); ++i) {
        const float c = steps * step / i + join + i * part;
        if (c < best) {
          best = c;
          k = i;
        }
      }
      const float parts = fmaxf(1.f, (float)cols / max(1, rest)) + 1.5f;  // of a tile on the line
      const float line = steps * step * rest / cols + 1.5f * (join + parts * part);
      if (q * steps * step + best <= line) {
        halves = q;
        each_in = k;
      }
    }
  }
  const int tails = rest - halves * cols;
  for (int i = tid; i < tails; i += NT) {
    GuItem it;
    Tiles::get_tail(p, l, dealt, halves * cols + i, it);
    l.tail[i] = (long long)it.nkb * it.cost;
  }
  sync();
  if (warp == 0) {
    long long sum = 0;
    for (int i0 = 0; i0 < tails; i0 += 32) {
      const long long v = i0 + lane < tails ? l.tail[i0 + lane] : 0;
      long long y = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long z = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o) y += z;
      }
      if (i0 + lane < tails) l.tail[i0 + lane] = sum + y - v;
      sum += __shfl_sync(0xffffffffu, y, 31);
    }
    if (lane == 0) l.tail[tails] = sum;
    __syncwarp();
    if (each_in) {
      for (int i = lane; i <= cols; i += 32) {
        const int t = i / each_in, part = i - t * each_in;
        l.cut[i] = t < tails ? l.tail[t] + (l.tail[t + 1] - l.tail[t]) * part / each_in : sum;
      }
    } else if (OP != G_DW || whole == 0) {
      // Pieces of one length, a tile cut into split_most on average at most.
      const int pieces = max(1, (int)min((long long)cols, (long long)tails * split_most));
      const long long each = sum / pieces;
      const int over = (int)(sum - each * pieces);
      for (int i = lane; i <= cols; i += 32) l.cut[i] = i < pieces ? i * each + i * over / pieces : sum;
    } else {
      // a piece brings its pair up to the mean of all pairs
      long long hands = 0;
      for (int i = lane; i < cols; i += 32) hands += l.hand[i];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) hands += __shfl_xor_sync(0xffffffffu, hands, o);
      const long long mean = (sum + hands + cols - 1) / cols;
      long long before = 0;
      for (int i0 = 0; i0 < cols; i0 += 32) {
        const long long v = i0 + lane < cols ? max(0LL, mean - l.hand[i0 + lane]) : 0;
        long long y = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const long long z = __shfl_up_sync(0xffffffffu, y, o);
          if (lane >= o) y += z;
        }
        if (i0 + lane < cols) l.cut[i0 + lane] = before + y - v;
        before += __shfl_sync(0xffffffffu, y, 31);
      }
      const double scale = (double)sum / (double)max(1LL, before);
      __syncwarp();
      for (int i = lane; i < cols; i += 32) l.cut[i] = min(sum, (long long)((double)l.cut[i] * scale));
      if (lane == 0) l.cut[cols] = sum;
    }
  }
  sync();
  *whole_out = whole;
  *halves_out = halves;
  return n_tiles;
}

// two values as a 16-bit pair, eight as four pairs
MOE_DEV uint32_t gu_pack2(int type, float lo, float hi) {
  if (type == G_BF16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
MOE_DEV uint4 gu_pack8(int type, const float* f) {
  return make_uint4(gu_pack2(type, f[0], f[1]), gu_pack2(type, f[2], f[3]), gu_pack2(type, f[4], f[5]),
                    gu_pack2(type, f[6], f[7]));
}

// Rows on the N side leave through shared memory: a warp has 32 M values
// (lanes) of up to 16 rows as fp32 words [row][lane] in `buf`, and stores them
// as 16-byte pieces where the rows allow it (`vec`: all 32 values there, 16-byte
// aligned rows), else value by value.  `base`: element of the first row's first
// value.
template <int F32>
MOE_DEV void gu_rows_out(void* out, int type, long long base, long long ld, int rows, int vals, bool vec, uint32_t buf) {
  const int lane = threadIdx.x & 31;
  __syncwarp();
  const bool f32 = F32 < 0 ? type == G_FP32 : F32 == 1;
  if (vec && !f32) {
    const int v = (lane & 3) * 8;
    float f[2][8];
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int i = 0; i < 8; i += 4) {
        const uint4 a = tc_lds128(buf + (uint32_t)(((lane >> 2) + 8 * k) * 128 + (v + i) * 4));
        f[k][i] = __uint_as_float(a.x);
        f[k][i + 1] = __uint_as_float(a.y);
        f[k][i + 2] = __uint_as_float(a.z);
        f[k][i + 3] = __uint_as_float(a.w);
      }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int r = (lane >> 2) + 8 * k;
      if (r < rows)
        *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(out) + base + r * ld + v) = gu_pack8(type, f[k]);
    }
  } else if (vec) {
    const int v = (lane & 7) * 4;
#pragma unroll
    for (int r = lane >> 3; r < kGuStageRows; r += 4)
      if (r < rows)
        *reinterpret_cast<uint4*>(reinterpret_cast<float*>(out) + base + r * ld + v) =
            tc_lds128(buf + (uint32_t)(r * 128 + v * 4));
  } else if (lane < vals) {
#pragma unroll 1
    for (int r = 0; r < rows; r += 4) {
      float t[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) t[k] = __uint_as_float(tc_lds32(buf + (uint32_t)((r + k) * 128 + lane * 4)));
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (r + k < rows) gmm_store(out, type, base + (r + k) * ld + lane, t[k]);
    }
  }
  __syncwarp();
}

// The same for values that are rounded already, as 16-bit words [row][lane] in `buf`.
MOE_DEV void gu_rows_out16(void* out, long long base, long long ld, int rows, int vals, bool vec, uint32_t buf) {
  const int lane = threadIdx.x & 31;
  uint16_t* o = reinterpret_cast<uint16_t*>(out) + base;
  __syncwarp();
  if (vec) {
    const int r = lane >> 2, v = (lane & 3) * 8;
    const uint4 a = tc_lds128(buf + 16u * lane), b = tc_lds128(buf + 512 + 16u * lane);
    if (r < rows) *reinterpret_cast<uint4*>(o + r * ld + v) = a;
    if (r + 8 < rows) *reinterpret_cast<uint4*>(o + (r + 8) * ld + v) = b;
  } else if (lane < vals) {
#pragma unroll 1
    for (int r = 0; r < rows; ++r) o[r * ld + lane] = (uint16_t)um_lds16(buf + (uint32_t)(64 * r + 2 * lane));
  }
  __syncwarp();
}
// Rows on the M side: LB bytes (64 or 128) of each lane's row leave through
// shared memory, 2 KB at a time, so that every store is of that many
// neighbouring bytes (with each lane storing to its own row in 32-byte sectors,
// weights' gradients of few rows, which are all stores, ran at 1.4 TB/s).  w:
// the lane's values, from element `base` of the warp's first row on, `left` of
// them in `vals` rows.
template <bool F32, int LB>
MOE_DEV void gu_lines_out(void* out, long long base, long long ld, int left, int vals, int unit, const uint32_t* w,
                          uint32_t buf) {
  constexpr int ES = F32 ? 4 : 2, PER = 16 / ES, CH = LB / 16, ROWS = 2048 / LB;
  const int lane = threadIdx.x & 31;
  char* o = reinterpret_cast<char*>(out) + base * ES;
  auto place = [&](int r, int c) {
    return buf + (uint32_t)(r * LB + ((CH == 8 ? c ^ (r & 7) : c ^ ((r >> 1) & 3)) << 4));
  };
  auto value = [&](char* to, uint32_t from) {
    if (F32) *reinterpret_cast<uint32_t*>(to) = tc_lds32(from);
    else *reinterpret_cast<uint16_t*>(to) = (uint16_t)um_lds16(from);
  };
  // (rolled loops: this is expanded at several places, and the 8-bit products
  // took 358 us instead of 333 with code that the instruction caches do not hold)
#pragma unroll 1
  for (int r0 = 0; r0 < vals; r0 += ROWS) {
    const int rows = min(ROWS, vals - r0);
    __syncwarp();
    if (ROWS == 32 || lane / ROWS == r0 / ROWS) {
#pragma unroll
      for (int c = 0; c < CH; ++c) tc_sts128(place(lane % ROWS, c), w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
    }
    __syncwarp();
    const int c = lane % CH;
    char* to = o + ((long long)(r0 + lane / CH) * ld + PER * c) * ES;
    if (unit >= 16 && left >= PER * CH) {
#pragma unroll
      for (int i = 0; i < ROWS; i += 32 / CH) {
        if (i + lane / CH < rows) *reinterpret_cast<uint4*>(to) = tc_lds128(place(i + lane / CH, c));
        to += (long long)(32 / CH) * ld * ES;
      }
    } else if (unit >= 16) {
      const int n = min(PER, left - PER * c);  // valid values of this lane's 16 bytes
#pragma unroll 1
      for (int r = lane / CH; r < rows; r += 32 / CH, to += (long long)(32 / CH) * ld * ES) {
        const uint32_t from = place(r, c);
        if (n == PER) *reinterpret_cast<uint4*>(to) = tc_lds128(from);
        else
#pragma unroll 1
          for (int k = 0; k < n; ++k) value(to + k * ES, from + k * ES);
      }
    } else {  // rows at any element: 32 neighbouring values per store, eight on their way
      constexpr int VS = LB / ES / 32, RS = 8 / VS;
#pragma unroll 1
      for (int r = 0; r < rows; r += RS) {
        uint32_t t[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int v = lane + 32 * (k % VS);
          const uint32_t from = place(r + k / VS, v * ES >> 4) + (uint32_t)(v * ES & 15);
          t[k] = F32 ? tc_lds32(from) : um_lds16(from);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int v = lane + 32 * (k % VS);
          char* to = o + ((r0 + r + k / VS) * ld + v) * ES;
          if (r + k / VS < rows && v < left) {
            if (F32) *reinterpret_cast<uint32_t*>(to) = t[k];
            else *reinterpret_cast<uint16_t*>(to) = (uint16_t)t[k];
          }
        }
      }
    }
  }
  __syncwarp();
}

// This warp's share, the part-th of `parts`, of `bytes` zeros.
MOE_DEV void gu_zeros_out(char* o, int bytes, int part, int parts) {
  const int lane = threadIdx.x & 31;
  const int head = min(bytes, (int)(-reinterpret_cast<uintptr_t>(o) & 15)), n = (bytes - head) >> 4;
#pragma unroll 4
  for (int i = 32 * part + lane; i < n; i += 32 * parts)
    *reinterpret_cast<uint4*>(o + head + 16 * i) = make_uint4(0, 0, 0, 0);
  if (part == 0 && 2 * lane < head) *reinterpret_cast<uint16_t*>(o + 2 * lane) = 0;
  const int end = head + 16 * n + 2 * lane;
  if (part == 1 && end < bytes) *reinterpret_cast<uint16_t*>(o + end) = 0;
}

// 32 bytes to a 32-byte aligned address: one whole sector per lane and store
// (with 16 the lanes of a warp, each in a row of its own, fill half sectors)
MOE_DEV void gu_st256(void* p, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
               "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// ------------------------------------------------------------ the kernel
// Launched in clusters of two CTAs (gridDim.x even), one CTA per SM.
template <int OP, bool FP8, bool ROWM, int MT, int CHAIN, bool ANY>
__global__ void __launch_bounds__(gu_threads(ANY), 1) grouped_umma_kernel(
    const __grid_constant__ GuKernelParams<FP8, ANY> p) {
  constexpr int EW = kGuEpiWarps, H = EW / 4, SR = kGuStageRows;
  constexpr bool SCALE_RING = FP8 && !ROWM;  // the scales come through shared memory
  static_assert(!FP8 || CHAIN == 1, "the 8-bit product hands over every step");
  static_assert(MT == 1 || (CHAIN == 0 && !ANY), "register sums and loads hold one MMA's");
  // what the kernel knows of the output's type: 1 fp32, 0 16 bits, -1 nothing
  constexpr int F32 = FP8 ? -1 : CHAIN ? 1 : 0;
  constexpr GuAnyShare kShare = gu_any_share(FP8, CHAIN);  // ANY
  constexpr int NS = ANY ? 2 : 12 / (MT + 1);  // stages
  constexpr int kStep = (MT + 1) * kGuTile;   // bytes of one: A (MT x 128 rows), B
  using Tiles = GuTiles<OP, FP8, ROWM, MT, ANY>;
  using Walk = GuWalk<Tiles>;
  constexpr bool A_MN = OP != G_MM, B_MN = OP == G_DW;
  constexpr int KE = Tiles::KE;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw32 = tc_smem(smem_raw);
  const uint32_t base = (raw32 + 1023u) & ~1023u;
  uint8_t* gen = smem_raw + (base - raw32);
  const uint32_t sc0 = base + kGuScaleOff, bar = base + kGuBarOff;
  GuLine& line = *reinterpret_cast<GuLine*>(gen + kGuLineOff);
  // (L): used in the leader CTA only
  auto full = [&](int s) { return bar + 8u * s; };                                      // (L) TMA bytes of both CTAs
  auto empty = [&](int s) { return bar + 8u * (NS + s); };                       // MMA commit
  auto acc_full = [&](int b) { return bar + 8u * (2 * NS + b); };                // MMA commit
  auto acc_empty = [&](int b) { return bar + 8u * (2 * NS + kGuSegs + b); };     // (L) epilogue warps, both CTAs
  constexpr int kBarSc = 2 * NS + 2 * kGuSegs;
  auto sc_full = [&](int s) { return bar + 8u * (kBarSc + s); };                        // scale warp
  auto sc_empty = [&](int s) { return bar + 8u * (kBarSc + kGuScaleSlots + s); };       // epilogue warps
  constexpr int kBarIt = kBarSc + 2 * kGuScaleSlots;
  auto it_full = [&](int s) { return bar + 8u * (kBarIt + s); };                        // item warp
  auto it_empty = [&](int s) { return bar + 8u * (kBarIt + kGuItems + s); };            // this CTA's other warps
  constexpr int kBarRaw = kBarIt + 2 * kGuItems;
  auto raw_full = [&](int s) { return bar + 8u * (kBarRaw + s); };                      // ANY: TMA bytes
  auto raw_empty = [&](int s) { return bar + 8u * (kBarRaw + kGuRaws + s); };           // ANY: load warps
  constexpr int kBars = kBarRaw + (ANY ? 2 * kGuRaws : 0);
  const uint32_t drain = bar + 8u * kBars;                                              // (L)
  const uint32_t join = drain + 8u;                                                     // epilogue warps
  int* tail = reinterpret_cast<int*>(gen + kGuBarOff + 8 * (kBars + 2));
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tail);
  volatile int* abort_flag = tail + 1;
  int* last_flag = tail + 2;
  static_assert(8 * (kBars + 2) + 16 <= 512, "barrier block");

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint32_t rank, pair, npairs;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm("mov.u32 %0, %%clusterid.x;" : "=r"(pair));
  asm("mov.u32 %0, %%nclusterid.x;" : "=r"(npairs));
  const bool leader = rank == 0;
  const GmmProblem& g = p.g;

  if (tid == 0) {
    for (int s = 0; s < NS; ++s) {
      tc_bar_init(full(s), ANY ? 2 * kGuLoadWarps : 1);
      tc_bar_init(empty(s), 1);
    }
    if constexpr (ANY)
      for (int s = 0; s < kGuRaws; ++s) {
        tc_bar_init(raw_full(s), 1);
        tc_bar_init(raw_empty(s), kGuLoadWarps);
      }
    for (int b = 0; b < kGuSegs; ++b) {
      tc_bar_init(acc_full(b), 1);
      tc_bar_init(acc_empty(b), 2 * EW);
    }
    for (int s = 0; s < kGuScaleSlots; ++s) {
      tc_bar_init(sc_full(s), 1);
      tc_bar_init(sc_empty(s), EW);
    }
    for (int s = 0; s < kGuItems; ++s) {
      tc_bar_init(it_full(s), 1);
      tc_bar_init(it_empty(s), (ANY ? 1 + kGuLoadWarps : 1) + (leader ? 1 : 0) + (SCALE_RING ? 1 : 0) + EW);
    }
    tc_bar_init(drain, 1);
    tc_bar_init(join, EW);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(tc_smem(tmem_slot)),
                 "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  const int cols = (int)npairs;
  // Everything above is this CTA's own.  From here on global memory is read:
  // the kernel before in the stream has to be through (launched with
  // programmatic serialization, this one starts on SMs that it has left).
  pdl_wait();
  pdl_trigger();

  // The plan.  Only the item warp works from it (and the epilogue reads the
  // cuts, after an item), so it makes it while the others set up; with many
  // experts it takes the whole block (256 experts: 2.9 us, one warp 6.9).
  int whole = 0, halves = 0, n_tiles = -1;
  const bool by_block = OP == G_DW || MT > 1 || g.E > 64;
  if (by_block) n_tiles = gu_plan<OP, Tiles, gu_threads(ANY)>(g, line, tid, cols, p.split_most, &whole, &halves);
  tc_fence_before();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  if constexpr (OP != G_DW)
    if (!by_block && warp == 3) n_tiles = gu_plan<OP, Tiles, 32>(g, line, lane, cols, p.split_most, &whole, &halves);
  if (warp == 3 && lane == 0 && n_tiles < 0) {
    set_error(g.err, kErrDeviceInput);
    line.cut[pair] = line.cut[pair + 1] = 0;
  }
  // both CTAs' barriers initialised and TMEM allocated before any cross-CTA use
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // The next item, in shared memory until it is given back; NULL after the
  // last.  Called by whole warps, or by lane 0 alone (`alone`).
  int it_at = 0;
  uint32_t it_ph = 0;
  auto next_item = [&](bool alone) -> const GuItem* {
    bool got = tc_bar_wait(it_full(it_at), it_ph, abort_flag);
    if (!alone) got = __all_sync(0xffffffffu, got) != 0;
    if (!got) return nullptr;
    const GuItem* it = &line.item[it_at];
    return it->kind == GU_STOP ? nullptr : it;
  };
  auto give_item = [&](bool alone) {
    if (!alone) __syncwarp();
    if (lane == 0) tc_bar_arrive(it_empty(it_at));
    if (++it_at == kGuItems) it_at = 0, it_ph ^= 1u;
  };
  auto copy_item = [&](GuItem& it, bool alone) {
    const GuItem* src = next_item(alone);
    if (!src) return false;
    it = *src;
    give_item(alone);
    return true;
  };

  if (warp < 4) {
    // the epilogue gets registers of these warps (the host checks that the block has kGuRegs per thread)
    if constexpr (ANY) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kShare.low));
    else if constexpr (gu_hand_over(MT, CHAIN)) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kGuRegsLow));
    if (ANY && warp == 0) {
      if constexpr (ANY) {
        // ================= TMA issuer of the aligned blocks: lanes 0 .. R - 1
        // the rows of A by their number modulo R, lanes 16 .. 16 + R - 1 those of B
        constexpr int R = GuAnyParams<FP8>::R;
        const int c = lane & 15;
        const bool is_b = lane >= 16, mine = c < R;
        const bool mn = is_b ? B_MN : A_MN;
        GuItem it;
        int st = 0, issued = 0;
        uint32_t ph = 0;
        bool ok = true;
        while (ok && copy_item(it, false)) {
          if (OP == G_DW && it.kind == GU_ZEROS) continue;
          const int half = it.np >> 1, m = it.m0 + (int)rank * 128, n = it.n0 + (int)rank * half;
          const bool few = !B_MN && half <= 32;
          const CUtensorMap* map = (!is_b ? p.a_rows : few ? p.b_few : p.b_rows) + (c & (R - 1));
          // the first step's first row (of the whole operand) and value
          const int k0 = it.kb0 * KE, we = it.e * g.n_out;
          int row = OP == G_DW ? it.r0 + k0 : is_b ? n : OP == G_DX ? we + k0 : we + m;
          int x = mn ? (is_b ? n : m) : k0;
          const uint32_t to = (is_b ? (uint32_t)kGuRaw : 0u) + (uint32_t)c * gu_raw_class<FP8>(mn, is_b && few);
          const uint32_t bytes = (A_MN ? 64 * 272 : 128 * 144) + (B_MN ? 64 * 272 : few ? 32 * 144 : 128 * 144);
          for (int kb = it.kb0; kb < it.kb1; ++kb) {
            ok = __all_sync(0xffffffffu, cl_bar_wait(raw_empty(st), ph ^ 1u, abort_flag)) != 0;
            if (!ok) break;
            if (lane == 0) um_expect_tx(raw_full(st), bytes);
            __syncwarp();
            if (mine)
              um_tma_2d(base + (uint32_t)(NS * kStep + st * 2 * kGuRaw) + to, map, x, (row - c + R - 1) / R,
                        raw_full(st));
            if (mn) row += 64;
            else x += KE;
            ++issued;
            if (++st == kGuRaws) st = 0, ph ^= 1u;
          }
        }
        // copies that no load warp will wait for (after a timeout) land before the block ends
        if (!ok || *abort_flag) {
          const long long t0 = clock64();
          for (int i = max(0, issued - kGuRaws); i < issued; ++i)
            while (!cl_bar_try(raw_full(i % kGuRaws), (uint32_t)(i / kGuRaws) & 1u) && clock64() - t0 < kTcWaitCycles) {
            }
        }
      }
    } else if (warp == 0) {
      // ================= TMA issuer of this CTA's halves of both operands
      // (lane 0; all lanes share the many small copies of dw's last steps)
      if (lane == 0) {
        um_prefetch_map(&p.a_map);
        um_prefetch_map(&p.b_map[0]);
      }
      GuItem it;
      int st = 0;
      uint32_t ph = 0;
      bool ok = true;
      while (ok && copy_item(it, false)) {
        if (OP == G_DW && it.kind == GU_ZEROS) continue;
        const int half = it.np >> 1;
        const int m = it.m0 + (int)rank * 128, n = it.n0 + (int)rank * half;
        const int bx = half <= 16 ? 0 : half <= 32 ? 1 : half <= 64 ? 2 : 3;
        const int panels = (half + 63) >> 6, a_panels = 2 * it.halves;  // dw
        for (int kb = it.kb0; kb < it.kb1; ++kb) {
          ok = __all_sync(0xffffffffu, cl_bar_wait(empty(st), ph ^ 1u, abort_flag)) != 0;
          if (!ok) break;
          const uint32_t a = base + (uint32_t)(st * kStep), b = a + MT * kGuTile;
          const uint32_t fb = cl_addr(full(st), 0);
          if constexpr (OP != G_DW) {
            if (lane == 0) {
              if (leader) um_expect_tx(full(st), (uint32_t)(2 * (it.halves * kGuTile + (ROWM ? kGuTile : (16 << bx) * 128))));
              if constexpr (ROWM) {
                gu_tma_2d(a, &p.a_map, kb * KE, m, fb);
                gu_tma_3d(b, &p.b_map[0], kb * KE, n, it.e, fb);
              } else if constexpr (OP == G_MM) {
                gu_tma_3d(a, &p.a_map, kb * KE, m, it.e, fb);
                if (MT > 1 && it.halves > 1) gu_tma_3d(a + kGuTile, &p.a_map, kb * KE, m + 256, it.e, fb);
              } else {
                for (int q = 0; q < 2 * it.halves; ++q)
                  gu_tma_3d(a + q * 8192, &p.a_map, m + 256 * (q >> 1) + 64 * (q & 1), kb * KE, it.e, fb);
              }
              if constexpr (!ROWM) gu_tma_2d(b, &p.b_map[bx], kb * KE, n, fb);
            }
          } else {
            const int y = it.r0 + kb * KE, left = it.r1 - y;
            if (left >= KE) {
              if (lane == 0) {
                if (leader) um_expect_tx(full(st), (uint32_t)(2 * (a_panels + panels) * 8192));
                for (int q = 0; q < a_panels; ++q)
                  gu_tma_2d(a + q * 8192, &p.a_map, m + 256 * (q >> 1) + 64 * (q & 1), y, fb);
                for (int q = 0; q < panels; ++q) gu_tma_2d(b + q * 8192, &p.b_map[0], n + 64 * q, y, fb);
              }
            } else {
              // The rows that are left, and zeros (from beyond the tensor) up
              // to a multiple of 16, each in boxes of their binary digits.
              const int fill = (left + 15) & ~15, zeros = fill - left;
              const int n_left = __popc(left), pieces = n_left + __popc(zeros);
              if (lane == 0 && leader) um_expect_tx(full(st), (uint32_t)(2 * fill * 128 * (a_panels + panels)));
              __syncwarp();
              for (int i = lane; i < pieces * (a_panels + panels); i += 32) {
                const int q = i / pieces, w = i - q * pieces;
                const bool zero = w >= n_left;
                int digits = zero ? zeros : left, r = zero ? left : 0;
                for (int k = zero ? w - n_left : w; k > 0; --k) {  // past the larger digits
                  const int top = 31 - __clz(digits);
                  digits ^= 1 << top;
                  r += 1 << top;
                }
                const int size = 31 - __clz(digits);
                const bool is_a = q < a_panels;
                const uint32_t dst = (is_a ? a + q * 8192 : b + (q - a_panels) * 8192) + (uint32_t)(r * 128);
                const CUtensorMap* maps = is_a ? p.a_tail : p.b_tail;
                const int x = is_a ? m + 256 * (q >> 1) + 64 * (q & 1) : n + 64 * (q - a_panels);
                gu_tma_2d(dst, &maps[5 - size], x, zero ? g.rows : y + r, fb);
              }
              __syncwarp();
            }
          }
          if (++st == NS) st = 0, ph ^= 1u;
        }
      }
      if (!ok) {  // a wait gave up: let the copies in flight land before this CTA's memory is released
        const long long t0 = clock64();
        while (clock64() - t0 < kGuLinger) {
        }
      }
      __syncwarp();
    } else if (warp == 1) {
      // ================= MMA issuer (leader CTA)
      if (leader && lane == 0) {
        GuItem it = {};
        int st = 0, seg = 0;
        uint32_t ph = 0;
        bool ok = true;
        GuRing ring;
        int user[kGuSegs];  // the last sum in each TMEM slot
        int done = -1;      // the latest sum known to be through the epilogue
#pragma unroll
        for (int i = 0; i < kGuSegs; ++i) user[i] = -1;
        const uint32_t idesc0 = (1u << 4) | ((uint32_t)(p.type == G_BF16 ? 1 : 0) * ((1u << 7) | (1u << 10))) |
                                ((A_MN ? 1u : 0u) << 15) | ((B_MN ? 1u : 0u) << 16) | (16u << 24);
        const uint64_t da0 = gu_desc(base, A_MN), db0 = gu_desc(base + MT * kGuTile, B_MN);
        // TMEM slots for the next sum, n wide: its first column.  The sums
        // leave the epilogue in order, so all that used these slots or this
        // barrier (eight sums ago) are through once the latest of them is.
        // One already seen through is not waited for again: its barrier may be
        // phases ahead.
        auto open_sum = [&](int n, uint32_t& d) {
          const int at = ring.take(n);
          int before = seg - kGuSegs;
#pragma unroll
          for (int i = 0; i < kGuSegs; ++i)
            if (i >= at && i < at + ring.used) {
              before = max(before, user[i]);
              user[i] = seg;
            }
          ++seg;
          d = tmem + (uint32_t)at * kGuSlotCols;
          if (before > done) {
            if (!cl_bar_wait(acc_empty(before & (kGuSegs - 1)), (uint32_t)(before / kGuSegs) & 1u, abort_flag)) return false;
            done = before;
          }
          tc_fence_after();
          return true;
        };
        // the MMAs of one step's stage s for the h-th 256 M values
        auto step_mma = [&](int s, int h, int kb, uint32_t d, uint32_t idesc, uint32_t acc) {
          const uint64_t so = (uint64_t)((uint32_t)(s * kStep) >> 4), ao = so + (uint64_t)((uint32_t)(h * kGuTile) >> 4);
          int steps = 4;
          if constexpr (OP == G_DW) steps = min(4, (it.r1 - it.r0 - kb * KE + 15) >> 4);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (OP != G_DW || k < steps) {
              // 16 (e4m3: 32) contracted values: 32 bytes along a K-major row, 16 rows of a panel otherwise
              gu_mma<FP8>(d, da0 + ao + (uint64_t)((A_MN ? 2048 : 32) * k >> 4),
                          db0 + so + (uint64_t)((B_MN ? 2048 : 32) * k >> 4), idesc, acc);
              acc = 1;
            }
        };
        while (ok && copy_item(it, true)) {
          if (OP == G_DW && it.kind == GU_ZEROS) continue;
          const uint32_t idesc = idesc0 | ((uint32_t)(it.np >> 3) << 17);
          if (MT > 1 && it.halves > 1) {
            // Both halves of the tile.  The second half's accumulator is still
            // being read when the first half's is free: the first steps, as
            // many as there are stages, are done for the first half, then for
            // the second.
            uint32_t d0, d1;
            ok = open_sum(it.np, d0);
            const int lead = min(NS, it.nkb);
            int s1 = st;
            for (int kb = 0; ok && kb < lead; ++kb) {
              ok = cl_bar_wait(full(s1), s1 < st ? ph ^ 1u : ph, abort_flag);
              if (!ok) break;
              tc_fence_after();
              step_mma(s1, 0, kb, d0, idesc, kb > 0);
              if (++s1 == NS) s1 = 0;
            }
            if (!ok) break;
            const int seg0 = (seg - 1) & (kGuSegs - 1);
            if (lead == it.nkb) umma2_commit_both(acc_full(seg0));
            ok = open_sum(it.np, d1);
            if (!ok) break;
            for (int kb = 0; kb < it.nkb; ++kb) {
              if (kb >= lead) {
                ok = cl_bar_wait(full(st), ph, abort_flag);
                if (!ok) break;
                tc_fence_after();
                step_mma(st, 0, kb, d0, idesc, 1u);
                if (kb + 1 == it.nkb) umma2_commit_both(acc_full(seg0));
              }
              step_mma(st, 1, kb, d1, idesc, kb > 0);
              umma2_commit_both(empty(st));
              if (++st == NS) st = 0, ph ^= 1u;
            }
            if (!ok) break;
            umma2_commit_both(acc_full((seg - 1) & (kGuSegs - 1)));
            continue;
          }
          for (int kb = it.kb0; kb < it.kb1;) {
            const int stride = SCALE_RING ? gu_stride(it.np) : kGuN;
            const int kend = SCALE_RING ? min(it.kb1, kb + kGuN / stride) : CHAIN ? min(it.kb1, kb + CHAIN) : it.kb1;
            uint32_t d, acc = 0;
            // (the operands are there before a hand-over's accumulator is: waited for first, their wait is hidden)
            if (FP8) ok = cl_bar_wait(full(st), ph, abort_flag);
            ok = ok && open_sum(FP8 ? kGuN : it.np, d);
            for (const int first = kb; ok && kb < kend; ++kb) {
              if (!FP8 || kb > first) ok = cl_bar_wait(full(st), ph, abort_flag);
              if (!ok) break;
              tc_fence_after();
              step_mma(st, 0, kb, d, idesc, acc);
              acc = 1;
              if constexpr (SCALE_RING) {
                acc = 0;
                d += stride;
              }
              umma2_commit_both(empty(st));
              if (++st == NS) st = 0, ph ^= 1u;
            }
            if (!ok) break;
            umma2_commit_both(acc_full((seg - 1) & (kGuSegs - 1)));
          }
        }
        umma2_commit_both(drain);
        const long long t0 = clock64();
        while (!cl_bar_try(drain, 0) && clock64() - t0 < kTcWaitCycles) {
        }
      }
      __syncwarp();
    } else if (warp == 2) {
      // ================= 8-bit product: the scales of each hand-over, row
      // scale times this CTA's weight scale.  The row scales are copied to
      // their slot up to kGuScaleAhead slots ahead; each lane then multiplies
      // those that it copied.
      if constexpr (SCALE_RING) {
        GuItem it;
        int fill = 0, slot = 0;  // the next slot to copy to, and to multiply
        float w = 0.f;           // this lane's of the weight scales of 32 steps
        uint32_t ph = 0;
        bool ok = true;
        const int groups = (g.n_in + 127) >> 7;
        while (ok && copy_item(it, false)) {
          const int ob = (it.m0 >> 7) + (int)rank;
          const float* swp = g.sw + ((long long)it.e * ((g.n_out + 127) >> 7) + ob) * groups;
          const bool live = ob * 128 < g.n_out;
          const int lg = it.np <= 64 ? 6 : 7, per = kGuN >> lg;  // (gu_stride)
          const int overs = (it.kb1 - it.kb0 + per - 1) >> (8 - lg);
          for (int i = 0; i < overs + kGuScaleAhead; ++i) {
            if (i < overs) {
              ok = __all_sync(0xffffffffu, cl_bar_wait(sc_empty(fill), ph ^ 1u, abort_flag)) != 0;
              if (!ok) break;
              const int k0 = it.kb0 + i * per;
              const uint32_t dst = sc0 + (uint32_t)(fill * kGuN + lane) * 4;
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const int kb = k0 + (32 * j >> lg), c = (32 * j + lane) & ((1 << lg) - 1);
                const bool in = kb < it.kb1 && c < it.nv;
                gu_cp4(dst + 128u * j, g.sx + (in ? (long long)kb * g.rows + it.n0 + c : 0), in);
              }
              if (++fill == kGuScaleSlots) fill = 0, ph ^= 1u;
            }
            cp_commit();
            if (i < kGuScaleAhead) continue;
            const int step = (i - kGuScaleAhead) * per;
            if ((step & 31) == 0) w = live && it.kb0 + step + lane < it.kb1 ? __ldg(swp + it.kb0 + step + lane) : 0.f;
            cp_wait<kGuScaleAhead>();
            const uint32_t at = sc0 + (uint32_t)(slot * kGuN + lane) * 4;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float ws = __shfl_sync(0xffffffffu, w, (step & 31) + (32 * j >> lg));
              const float v = __uint_as_float(tc_lds32(at + 128u * j)) * ws;
              asm volatile("st.shared.f32 [%0], %1;" ::"r"(at + 128u * j), "f"(v) : "memory");
            }
            __syncwarp();
            if (lane == 0) tc_bar_arrive(sc_full(slot));
            if (++slot == kGuScaleSlots) slot = 0;
          }
        }
        cp_wait<0>();
      }
    } else {
      // ================= the items of this CTA, a few ahead of the warps that work on them
      if (lane == 0) {
        Walk walk(g, line, (int)pair, cols, max(n_tiles, 0), whole, halves);
        GuItem it;
        int at = 0;
        uint32_t ph = 0;
        for (bool more = true; more;) {
          more = walk.next(it);
          if (!more) it.kind = GU_STOP;
          if (!tc_bar_wait(it_empty(at), ph ^ 1u, abort_flag)) break;
          line.item[at] = it;
          tc_bar_arrive(it_full(at));
          if (++at == kGuItems) at = 0, ph ^= 1u;
        }
      }
      __syncwarp();
    }
  } else if (ANY && warp >= 4 + kGuEpiWarps) {
    if constexpr (ANY) {
      // ================= the operands' pieces out of the aligned blocks: eight
      // neighbouring lanes have one row's 128 bytes (which hit different banks,
      // read and written); M- or N-major: of 64 rows, each of two panels.
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kShare.load));
      constexpr int ES = FP8 ? 1 : 2, R = GuAnyParams<FP8>::R;
      const int lw = warp - 4 - kGuEpiWarps;  // 0 .. 7
      // rows from number `first` on, of which the first is at `low` modulo 16 bytes
      auto cut = [&](auto mn, uint32_t to, uint32_t from, uint32_t low, uint32_t ld, int first, int rows, uint32_t cls) {
        constexpr bool MN = decltype(mn)::value;
        constexpr int C = MN ? 16 : 8, PITCH = MN ? 272 : 144, J = 32 / C;  // pieces of a row, rows at a time
        const int c = lane & (C - 1);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int r = (16 / (C / 8)) * lw + lane / C + J * j;
          if (!MN && r - lane / C >= rows) break;
          const uint32_t at = from + (uint32_t)((first + r) & (R - 1)) * cls + (uint32_t)(r / R * PITCH + 16 * c);
          const uint32_t dst = to + (uint32_t)((c >> 3) * 8192 + r * 128 + (((c & 7) ^ (r & 7)) << 4));
          if (!MN || r < rows) gu_cut16(dst, tc_lds128(at), tc_lds128(at + 16), (low + (uint32_t)r * ld) & 15u);
          else tc_sts128(dst, 0u, 0u, 0u, 0u);
        }
      };
      constexpr std::integral_constant<bool, A_MN> a_mn;
      constexpr std::integral_constant<bool, B_MN> b_mn;
      GuItem it;
      int st = 0, rs = 0;
      uint32_t ph = 0, rph = 0;
      bool ok = true;
      while (ok && copy_item(it, false)) {
        if (OP == G_DW && it.kind == GU_ZEROS) continue;
        const int half = it.np >> 1, m = it.m0 + (int)rank * 128, n = it.n0 + (int)rank * half;
        const bool few = !B_MN && half <= 32;
        const int k0 = it.kb0 * KE, we = it.e * g.n_out;
        // numbers of the rows as the issuer has them, addresses and row strides modulo 16 bytes
        int a_row = OP == G_DW ? it.r0 + k0 : OP == G_DX ? we + k0 : we + m, b_row = OP == G_DW ? it.r0 + k0 : n;
        int left = OP == G_DW ? it.r1 - it.r0 - k0 : g.n_out - k0;  // contracted rows (M- or N-major)
        const uint32_t lda = (uint32_t)(OP == G_DW ? g.ld_rows : g.n_in) * ES;
        const uint32_t ldb = (uint32_t)(OP == G_DW ? g.ld_x : g.ld_rows) * ES;
        const void *a_at = OP == G_DW ? g.rows_in : g.w, *b_at = OP == G_DW ? g.x : g.rows_in;
        const uint32_t a_low = (uint32_t)reinterpret_cast<uintptr_t>(a_at) + (uint32_t)a_row * lda;
        const uint32_t b_low = (uint32_t)reinterpret_cast<uintptr_t>(b_at) + (uint32_t)b_row * ldb;
        const uint32_t a_cls = gu_raw_class<FP8>(A_MN, false), b_cls = gu_raw_class<FP8>(B_MN, few);
        for (int kb = it.kb0; kb < it.kb1; ++kb) {
          ok = __all_sync(0xffffffffu, cl_bar_wait(raw_full(rs), rph, abort_flag) &&
                                           cl_bar_wait(empty(st), ph ^ 1u, abort_flag)) != 0;
          if (!ok) break;
          const uint32_t a = base + (uint32_t)(st * kStep), raw = base + (uint32_t)(NS * kStep + rs * 2 * kGuRaw);
          cut(a_mn, a, raw, a_low, lda, a_row, A_MN ? left : 128, a_cls);
          cut(b_mn, a + kGuTile, raw + kGuRaw, b_low, ldb, b_row, B_MN ? left : half, b_cls);
          if (A_MN) a_row += 64;
          if (B_MN) b_row += 64;
          left -= 64;
          tc_fence_proxy();  // the stores, before the tensor core reads them
          __syncwarp();
          if (lane == 0) {
            cl_arrive(cl_addr(full(st), 0));
            tc_bar_arrive(raw_empty(rs));
          }
          if (++st == NS) st = 0, ph ^= 1u;
          if (++rs == kGuRaws) rs = 0, rph ^= 1u;
        }
      }
    }
  } else {
    if constexpr (ANY) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kShare.high));
    else if constexpr (gu_hand_over(MT, CHAIN)) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kGuRegsHigh));
    // ================= epilogue: 32 TMEM lanes (M values) and every H-th 32 columns (output rows) per warp
    const int q = warp & 3, h = (warp - 4) >> 2;
    const uint32_t buf = base + kGuOutOff + (uint32_t)((warp - 4) * SR * 128);
    const long long ld = OP == G_DW ? g.n_in : g.ld_out;
    const int out_bytes = g.out_type == G_FP32 ? 4 : 2;
    const uintptr_t bits = (uintptr_t)(ld * out_bytes) | reinterpret_cast<uintptr_t>(g.out);
    const int unit = bits % 32 == 0 ? 32 : bits % 16 == 0 ? 16 : 1;  // the output rows' alignment
    GuRing ring;
    int seg = 0, slot = 0, joins = 0;
    uint32_t sph = 0, jph = 0;
    auto epi_sync = [&]() {  // the epilogue warps meet (bounded, unlike a hardware barrier)
      __syncwarp();
      if (lane == 0) tc_bar_arrive(join);
      const bool met = tc_bar_wait(join, jph, abort_flag);
      jph ^= 1u;
      return __all_sync(0xffffffffu, met) != 0;
    };
    const uint32_t lane_addr = tmem + ((uint32_t)(32 * q) << 16);
    unsigned* counters = reinterpret_cast<unsigned*>(p.ws + kGuCounters);
    // a partial tile: four columns (16 bytes) of each M value together
    auto part_of = [&](int piece, int which) {
      return reinterpret_cast<float4*>(p.ws + kGuParts + (size_t)((piece * 2 + (int)rank) * 2 + which) * kGuPart) +
             32 * q + lane;
    };
    bool ok = true;
    while (ok) {
      GuItem it;
      if (!copy_item(it, false)) break;
      const int chunks = (it.np + 31) >> 5;
      // This warp's 32-column ranges: every H-th, or (rows on the M side, for
      // longer stores) neighbours; 8-bit: those of one scale block.
      const int share = FP8 ? 4 : (chunks + 1) >> 1;
      const int c_first = ROWM ? h * share : h, c_end = ROWM && h == 0 ? min(share, chunks) : chunks;
      constexpr int C_STEP = ROWM ? 1 : H;
      const bool all = it.kb0 == 0 && it.kb1 == it.nkb;
      const int m = (int)rank * 128 + 32 * q;       // the warp's first M value in the tile
      int vals = min(32, it.mv - m);                // how many it has
      // the first M and N value's output element
      long long ob = ROWM ? (OP == G_DW ? (long long)it.e * g.n_out + it.m0 + m : (long long)it.m0 + m) * ld + it.n0
                          : (long long)it.n0 * ld + it.m0 + m;
      // N values 32 c .. of the tile to the output
      auto out32 = [&](int c, const float (&v)[32]) {
        const int left = it.nv - 32 * c;
        if (left <= 0 || vals <= 0) return;
        if constexpr (ROWM) {
          const bool f32 = F32 < 0 ? g.out_type == G_FP32 : F32 == 1;
          uint32_t w[32];
          if (f32) {
#pragma unroll
            for (int i = 0; i < 32; ++i) w[i] = __float_as_uint(v[i]);
            if constexpr (F32 != 0) gu_lines_out<true, 128>(g.out, ob + 32 * c, ld, left, vals, unit, w, buf);
          } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) w[i] = gu_pack2(g.out_type, v[2 * i], v[2 * i + 1]);
            if constexpr (F32 != 1) gu_lines_out<false, 64>(g.out, ob + 32 * c, ld, left, vals, unit, w, buf);
          }
        } else {
#pragma unroll
          for (int u = 0; u < 32; u += SR)
            if (left > u) {
#pragma unroll
              for (int i = 0; i < SR; ++i)
                asm volatile("st.shared.f32 [%0], %1;" ::"r"(buf + (uint32_t)(i * 128 + 4 * lane)), "f"(v[u + i]) : "memory");
              gu_rows_out<F32>(g.out, g.out_type, ob + (32 * c + u) * ld, ld, min(SR, left - u), vals,
                               unit >= 16 && vals == 32, buf);
            }
        }
      };
      auto put = [&](int c, const float (&v)[32]) {  // ... or to this pair's part
        if (all) {
          out32(c, v);
        } else {
          float4* part = part_of((int)pair, it.kb0 > 0 ? 0 : 1) + 8 * c * 128;
#pragma unroll
          for (int i = 0; i < 8; ++i)
            __stcg(part + i * 128, make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]));
        }
      };
      // 64 rounded values from 32 c on (rows on the M side)
      auto out64 = [&](int c, const uint32_t* w) {
        const int left = it.nv - 32 * c;
        if (left > 0 && vals > 0) gu_lines_out<false, 128>(g.out, ob + 32 * c, ld, left, vals, unit, w, buf);
      };
      if constexpr (OP == G_DW) {
        if (it.kind == GU_ZEROS) {
          // An expert's matrix has no gaps, and all tiles of 256 of its rows
          // are zeros: each writes its share of those rows as one run, whatever
          // their alignment.
          for (int half = 0; half < it.halves; ++half) {
            const int mv = min(256, it.mv - 256 * half);
            char* o = reinterpret_cast<char*>(g.out) +
                      (((long long)it.e * g.n_out + it.m0 + 256 * half) * g.n_in + (long long)mv * it.n0) * out_bytes;
            if (mv > 0) gu_zeros_out(o, mv * it.nv * out_bytes, (int)rank * EW + warp - 4, 2 * EW);
          }
          continue;
        }
      }
      auto wait_sums = [&]() {
        const bool got = cl_bar_wait(acc_full(seg & (kGuSegs - 1)), (uint32_t)(seg / kGuSegs) & 1u, abort_flag);
        if (!__all_sync(0xffffffffu, got)) return false;
        tc_fence_after();
        return true;
      };
      auto give_back = [&]() {  // the sums are in registers
        tc_fence_before();
        __syncwarp();
        if (lane == 0) cl_arrive(cl_addr(acc_empty(seg & (kGuSegs - 1)), 0));
      };
      if constexpr (CHAIN == 0) {
        if (!ANY && all) {
          // Rounded to the output's 16 bits on the way into registers, both
          // halves, so that the accumulators are free before the first store:
          // the next tile's MMAs wait for 800 clocks of TMEM reads then, and
          // not for 4,800 more of stores.
          uint32_t w[MT][64];
#pragma unroll
          for (int half = 0; half < MT; ++half)
            if (half < it.halves) {
              const int at = ring.take(it.np);
              ok = ok && wait_sums();
              if (ok) {
                const uint32_t ta = lane_addr + (uint32_t)(at * kGuSlotCols);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                  if (c_first + C_STEP * j < c_end) {
                    float v[32];
                    gu_ld32(ta + 32u * (c_first + C_STEP * j), v);
#pragma unroll
                    for (int i = 0; i < 16; ++i) w[half][16 * j + i] = gu_pack2(g.out_type, v[2 * i], v[2 * i + 1]);
                  } else if (ROWM && (j & 1)) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) w[half][16 * j + i] = 0;
                  }
                give_back();
                ++seg;
              }
            }
          if (!ok) break;
#pragma unroll
          for (int half = 0; half < MT; ++half) {
            if (half >= it.halves) break;
            if constexpr (ROWM) {
              // 64 values where this warp has both ranges; a last one alone ends before its neighbour's
#pragma unroll
              for (int j = 0; j < 4; j += 2) {
                const int c = c_first + j;
                if (c + 1 < c_end) out64(c, &w[half][16 * j]);
                else if (c < c_end && it.nv > 32 * c && vals > 0)
                  gu_lines_out<false, 64>(g.out, ob + 32 * c, ld, it.nv - 32 * c, vals, unit, &w[half][16 * j], buf);
              }
            } else {
#pragma unroll
              for (int j = 0; j < 4; ++j)
                if (H * j + h < chunks) {
#pragma unroll
                  for (int u = 0; u < 2; ++u) {
                    const int c = 2 * (H * j + h) + u, left = it.nv - SR * c;
                    if (left <= 0 || vals <= 0) continue;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                      const uint32_t to = buf + (uint32_t)(128 * i + 2 * lane), x = w[half][16 * j + 8 * u + i];
                      asm volatile("st.shared.u16 [%0], %1;" ::"r"(to), "h"((uint16_t)x) : "memory");
                      asm volatile("st.shared.u16 [%0], %1;" ::"r"(to + 64), "h"((uint16_t)(x >> 16)) : "memory");
                    }
                    gu_rows_out16(g.out, ob + SR * c * ld, ld, min(SR, left), vals, unit >= 16 && vals == 32, buf);
                  }
                }
            }
            ob += ROWM ? 256 * ld : 256;  // the second half's M values
            vals = min(32, it.mv - 256 - m);
          }
        } else {
          const int at = ring.take(it.np);
          ok = wait_sums();
          if (!ok) break;
          for (int c = c_first; c < c_end; c += C_STEP) {
            float v[32];
            gu_ld32(lane_addr + (uint32_t)(at * kGuSlotCols + 32 * c), v);
            put(c, v);
          }
          give_back();
          ++seg;
        }
      } else {
        // sums in pairs of columns, for the packed fp32 instructions
        constexpr int NJ = Tiles::kMost / 64;
        unsigned long long acc[NJ][16];
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
          for (int i = 0; i < 16; ++i) acc[j][i] = 0;
        if constexpr (SCALE_RING) {
          const int stride = gu_stride(it.np);
          for (int kb = it.kb0; kb < it.kb1; kb += kGuN / stride) {
            const int at = ring.take(kGuN);
            ok = tc_bar_wait(sc_full(slot), sph, abort_flag);  // (there before the sums are)
            ok = __all_sync(0xffffffffu, ok) && wait_sums();
            if (!ok) break;
            const uint32_t ta = lane_addr + (uint32_t)(at * kGuSlotCols + 32 * h);
            const uint32_t sp = sc0 + (uint32_t)(slot * kGuN + 32 * h) * 4;
            const int ranges = min(kGuN / stride, it.kb1 - kb) * (stride >> 6);  // 64 columns each, 32 for this warp
            if (32 * h < it.np) {
#pragma unroll
              for (int j = 0; j < 4; ++j)
                if (j < ranges) {
                  uint32_t r[32];
                  gu_ld_issue(ta + 64u * j, r);
                  gu_ld_wait(r);
                  if (stride == 128 && (j & 1)) gu_scaled(acc[1], 0, r, sp + 256u * j);
                  else gu_scaled(acc[0], 0, r, sp + 256u * j);
                }
            }
            give_back();
            if (lane == 0) tc_bar_arrive(sc_empty(slot));
            if (++slot == kGuScaleSlots) slot = 0, sph ^= 1u;
            ++seg;
          }
        } else if constexpr (FP8) {
          // one row scale per thread and step, and one weight scale per warp
          // (128 columns); those of the next steps are on their way
          const int groups = (g.n_in + 127) >> 7, blocks = (g.n_out + 127) >> 7;
          const float* sxp = g.sx + it.m0 + m + min(lane, max(vals - 1, 0));
          const float* swp = g.sw + ((long long)it.e * blocks + min((it.n0 >> 7) + h, blocks - 1)) * groups;
          auto scale_of = [&](int kb, float& x, float& a) {
            kb = min(kb, it.kb1 - 1);
            x = vals > 0 ? __ldg(sxp + (long long)kb * g.rows) : 0.f;
            a = __ldg(swp + kb);
          };
          float x0, a0, x1, a1;
          scale_of(it.kb0, x0, a0);
          scale_of(it.kb0 + 1, x1, a1);
          for (int kb = it.kb0; kb < it.kb1; ++kb) {
            const int at = ring.take(kGuN);
            const float sa = x0 * a0;
            const unsigned long long sc = gu_pack(sa, sa);
            x0 = x1, a0 = a1;
            scale_of(kb + 2, x1, a1);
            ok = wait_sums();
            if (!ok) break;
            const uint32_t ta = lane_addr + (uint32_t)(at * kGuSlotCols + 128 * h);
            // (columns beyond the tile's hold what was there before and are not stored)
            uint32_t r0[32], r1[32];
            gu_ld_issue(ta, r0);
            gu_ld_wait(r0);
            gu_ld_issue(ta + 32, r1);
            gu_times(acc[0], r0, sc);
            gu_ld_wait(r1);
            gu_ld_issue(ta + 64, r0);
            gu_times(acc[1], r1, sc);
            gu_ld_wait(r0);
            gu_ld_issue(ta + 96, r1);
            gu_times(acc[2], r0, sc);
            gu_ld_wait(r1);
            give_back();
            gu_times(acc[3], r1, sc);
            ++seg;
          }
        } else {
          constexpr int LW = ANY ? 16 : 32;  // columns at a time; ANY has no registers for 32 beside the sums
          for (int kb = it.kb0; kb < it.kb1; kb += CHAIN) {
            const int at = ring.take(it.np);
            ok = wait_sums();
            if (!ok) break;
            const uint32_t ta = lane_addr + (uint32_t)(at * kGuSlotCols);
#pragma unroll
            for (int j = 0; j < NJ; ++j)
              if (c_first + C_STEP * j < c_end) {
#pragma unroll
                for (int u = 0; u < 32; u += LW) {
                  uint32_t r[LW];
                  gu_ld_issue(ta + 32u * (c_first + C_STEP * j) + u, r);
                  gu_ld_wait(r);
#pragma unroll
                  for (int i = 0; i < LW; i += 2)
                    gu_add2(acc[j][(u + i) / 2], gu_pack(__uint_as_float(r[i]), __uint_as_float(r[i + 1])));
                }
              }
            give_back();
            ++seg;
          }
        }
        if (!ok) break;
        if (FP8 && ROWM && all && g.out_type != G_FP32) {
#pragma unroll
          for (int j = 0; j + 1 < NJ; j += 2) {
            uint32_t w[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              float lo, hi;
              gu_unpack(acc[j + i / 16][i % 16], lo, hi);
              w[i] = gu_pack2(g.out_type, lo, hi);
            }
            const int c = c_first + j, left = it.nv - 32 * c;
            if (left <= 0 || vals <= 0) continue;
            if (left >= 64 && unit == 32) {
              // (straight from the registers: the next sums cannot be taken
              // from tensor memory meanwhile, and this is the shorter way)
              uint16_t* o = reinterpret_cast<uint16_t*>(g.out) + ob + lane * ld + 32 * c;
              if (lane < vals) {
#pragma unroll
                for (int i = 0; i < 32; i += 8) gu_st256(o + 2 * i, w + i);
              }
            } else {
              out64(c, w);
            }
          }
        } else {
#pragma unroll
          for (int j = 0; j < NJ; ++j)
            if (c_first + C_STEP * j < c_end) {
              float v[32];
#pragma unroll
              for (int i = 0; i < 16; ++i) gu_unpack(acc[j][i], v[2 * i], v[2 * i + 1]);
              put(c_first + C_STEP * j, v);
            }
        }
      }
      if (!all) {
        // Count this part in; the last part's CTA adds them all, in the
        // pieces' order.  The parts are those of the pieces from the one that
        // holds the tile's first step to the one that holds its last, less
        // those too short to hold a step.
        auto piece_at = [&](long long u) {
          int lo = 0, hi = cols;  // cut[lo] <= u < cut[hi]
          while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (line.cut[mid] <= u) lo = mid;
            else hi = mid;
          }
          return lo;
        };
        const int first = piece_at(it.pos), last = piece_at(it.pos + (long long)(it.nkb - 1) * it.cost);
        // of 32 pieces from `from` on, those with a part
        auto with_part = [&](int from) {
          const int s = from + lane;
          return __ballot_sync(0xffffffffu, s <= last && Walk::steps_before(line.cut[s], it) <
                                                              Walk::steps_before(line.cut[s + 1], it));
        };
        int parts = 0;
#pragma unroll 1
        for (int from = first; from <= last; from += 32) parts += __popc(with_part(from));
        __threadfence();
        ok = epi_sync();
        if (!ok) break;
        volatile int* flag = last_flag + (joins++ & 1);  // (two: the next join's is not this one's)
        if (tid == 128) {
          unsigned* ctr = counters + first * 2 + rank;
          const unsigned before = atomicAdd(ctr, 1u);
          *flag = before + 1 == (unsigned)parts;
          if (before + 1 == (unsigned)parts) *ctr = 0;
        }
        ok = epi_sync();
        if (!ok) break;
        if (*flag) {
          __threadfence();
          // 32 columns at a time, two parts' loads in flight together
#pragma unroll 1
          for (int c = c_first; c < c_end; c += C_STEP) {
            float v[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = 0.f;
#pragma unroll 1
            for (int from = first; from <= last; from += 32) {
              uint32_t left = with_part(from);
#pragma unroll 1
              while (left) {
                float4 a[2][8];
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                  const int piece = from + __ffs(left) - 1;
                  const float4* src = part_of(max(piece, 0), piece == first ? 1 : 0) + 8 * c * 128;
#pragma unroll
                  for (int i = 0; i < 8; ++i) a[s][i] = left ? __ldcg(src + i * 128) : make_float4(0.f, 0.f, 0.f, 0.f);
                  left &= left - 1;
                }
#pragma unroll
                for (int s = 0; s < 2; ++s)
#pragma unroll
                  for (int i = 0; i < 8; ++i) {
                    v[4 * i] += a[s][i].x;
                    v[4 * i + 1] += a[s][i].y;
                    v[4 * i + 2] += a[s][i].z;
                    v[4 * i + 3] += a[s][i].w;
                  }
              }
            }
            out32(c, v);
          }
        }
      }
    }
  }
  __syncthreads();
  tc_fence_before();
  cluster_sync_all();  // the pair's MMAs have drained; neither CTA's memory is read from now on
  tc_fence_after();
  if (tid == 0 && *abort_flag) set_error(g.err, kErrTimeout);
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
}

// One translation unit per kernel: gu_launch starts `pairs` clusters, gu_pairs
// sets the kernel's attributes on the current device and returns how many
// pairs fit at once, or why it cannot tell (GU_QUERY_FAILED: the runtime's last
// error says).
enum GuNoPairs : int { GU_NO_FIT = 0, GU_QUERY_FAILED = -1, GU_REGISTERS = -2 };
template <int OP, bool FP8, bool ROWM, int MT, int CHAIN, bool ANY>
bool gu_launch(const GuParams& p, int pairs, cudaStream_t s);
template <int OP, bool FP8, bool ROWM, int MT, int CHAIN, bool ANY>
int gu_pairs();
constexpr int kGuChain = 8;  // 16-bit products with fp32 outputs: 512 contracted values per chain
#define MOE_GU_DECL(OP, FP8, ROWM, MT, CHAIN, ANY)                                             \
  template <>                                                                                  \
  bool gu_launch<OP, FP8, ROWM, MT, CHAIN, ANY>(const GuParams& p, int pairs, cudaStream_t s); \
  template <>                                                                                  \
  int gu_pairs<OP, FP8, ROWM, MT, CHAIN, ANY>();
MOE_GU_DECL(G_MM, false, false, 1, 0, false)
MOE_GU_DECL(G_MM, false, false, 2, 0, false)
MOE_GU_DECL(G_MM, false, false, 1, kGuChain, false)
MOE_GU_DECL(G_MM, false, false, 1, 0, true)
MOE_GU_DECL(G_MM, false, false, 1, kGuChain, true)
MOE_GU_DECL(G_DX, false, false, 1, 0, false)
MOE_GU_DECL(G_DX, false, false, 2, 0, false)
MOE_GU_DECL(G_DX, false, false, 1, kGuChain, false)
MOE_GU_DECL(G_DX, false, false, 1, 0, true)
MOE_GU_DECL(G_DX, false, false, 1, kGuChain, true)
MOE_GU_DECL(G_DW, false, true, 1, 0, false)
MOE_GU_DECL(G_DW, false, true, 2, 0, false)
MOE_GU_DECL(G_DW, false, true, 1, kGuChain, false)
MOE_GU_DECL(G_DW, false, true, 1, 0, true)
MOE_GU_DECL(G_DW, false, true, 1, kGuChain, true)
MOE_GU_DECL(G_MM, true, false, 1, 1, false)
MOE_GU_DECL(G_MM, true, true, 1, 1, false)
MOE_GU_DECL(G_MM, true, false, 1, 1, true)
#undef MOE_GU_DECL

}  // namespace moe
