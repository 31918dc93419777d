// Grouped products on the 5th-generation tensor cores (sm_100a): TMA loads,
// tcgen05.mma on pairs of SMs, accumulators in tensor memory.
//
// A tile is 256 values of the output's contiguous dimension (M side, 128 per
// CTA of the pair) by up to 256 output rows (N side): the rows of an expert
// are cut into equal tiles of at most 256, rounded up to 32, so that an
// expert with few rows costs a narrow MMA and not a padded tile.  Steps of the
// contracted dimension are 128 bytes per row: 64 16-bit values or 128 e4m3
// codes, the block of the 8-bit scales.
//
//   op   M side (A operand)                  N side (B operand)
//   mm   W[e] rows o, K-major                x rows, K-major
//   dx   W[e] columns i, M-major             dy rows, K-major
//   dw   x columns i, M-major                dy columns o, N-major
//
// One tile step is 16 KB of A and up to 16 KB of B per CTA in a ring of six.
// M- and N-major operands are 64-value panels of 64 contracted rows.  For dw
// the contracted rows are the expert's: in its last step only the rows that
// are left are copied, in boxes of eight and one, and the rest of the last 16
// comes from beyond the tensor's end, which TMA fills with zeros, so that no
// value of another expert's rows (a NaN, say) enters a product.
//
// Work is split by steps, not by tiles.  The tiles, in the order expert, M
// tile, row tile, are dealt out to the pairs of CTAs in turn, so that pairs
// that run at the same time read the same weights and rows from L2 (with
// each pair on a run of neighbouring tiles instead, 74 pairs stream 148 MB
// between two uses of an operand tile, more than L2 holds: 32,768 rows over 32
// experts took 870 us that way).  The pairs' hands, one after the other, are a
// line, and the line is cut into pieces of equal cost, one per pair.  A tile
// that a cut goes through
// is summed by the pairs that hold parts of it: each writes its fp32 partial
// sums to the workspace and counts itself in; the last one adds the partials
// in the pieces' order (so the result does not depend on who was last) and
// writes the outputs.  No pair waits for another.  This keeps every SM busy
// when there are few tiles (one token over eight experts: 64 tiles for 74
// pairs), and costs at most two partial tiles per pair.
//
// CHAIN = 0: the tile's whole sum is taken in tensor memory.  CHAIN > 0: every
// CHAIN steps the sum is handed to the epilogue warps, which add it to sums in
// registers with ordinary fp32 additions, scaled for the 8-bit product.
#pragma once

#include <cuda.h>

#include "ffn_umma.cuh"
#include "grouped_plan.cuh"

namespace moe {

constexpr int kGuStages = 6;
constexpr int kGuTile = 16384;            // bytes of one operand of one step
constexpr int kGuN = 256;                 // output rows per tile
constexpr int kGuThreads = 384;           // warps: 0 loads, 1 MMA, 2 scales, 4-11 epilogue
constexpr int kGuEpiWarps = 8;
constexpr int kGuScaleSlots = 8;
constexpr int kGuPart = 128 * kGuN * 4;   // bytes of one partial tile of one CTA
constexpr int kGuPairsMax = 74;
constexpr long long kGuLinger = 4000000;  // ~2 ms
constexpr size_t kGuCounters = 1024;      // workspace: counters, then the partial tiles
constexpr size_t kGuParts = 4096;
constexpr size_t kGuWsBytes = size_t(40) << 20;
static_assert(kGuCounters + kGuPairsMax * 2 * 4 <= kGuParts, "counters");
static_assert(kGuParts + (size_t)kGuPairsMax * 4 * kGuPart <= kGuWsBytes, "workspace");

struct alignas(64) GuParams {
  CUtensorMap a_map;     // mm, dx: W; dw: x, 64 rows
  CUtensorMap b_map[4];  // mm, dx: rows in boxes of 16, 32, 64, 128; dw: dy, 64 rows
  CUtensorMap a_tail[2], b_tail[2];  // dw: boxes of eight rows and of one
  GmmProblem g;
  int type;              // GmmType of the operands
  int split_most;        // pieces that a tile may be cut into
  unsigned char* ws;
};

// ------------------------------------------------------------ PTX wrappers
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

// ------------------------------------------------------------ work items
// A run of steps of one tile.
struct GuItem {
  int e, m0, n0, nv, np;   // expert, first M value, first output row (dw: first o), rows in use, MMA width
  int kb0, kb1, nkb;       // steps, and the tile's number of steps
  int cost;                // of one step
  int r0, r1;              // dw: the expert's rows
  bool none;               // dw: no rows; one step that reads nothing, zeros to write
  long long pos;           // where the tile begins on the line
};

// The line of work and this pair's piece of it (shared memory of each CTA).
struct GuLine {
  long long col[kGuPairsMax + 1];  // where each pair's hand begins
  long long cost_most;             // of a step
  long long start_pos;             // the piece's first tile: where it begins, whose hand, which of it
  int start_col, start_row;
  int flag;
};

constexpr size_t gu_smem() {
  return 1024 + (size_t)kGuStages * 2 * kGuTile + kGuScaleSlots * kGuN * 4 + (kGmmMaxExperts + 1) * 8 +
         sizeof(GuLine) + 512;
}
static_assert(gu_smem() <= 227 * 1024, "shared memory");

template <int OP, int KE>
struct GuTiles {
  // (dw: whole 64-value panels in both CTAs)
  static constexpr int kRound = OP == G_DW ? 128 : 32;
  MOE_DEV static int count(int n) { return (n + kGuN - 1) / kGuN; }
  MOE_DEV static int m_count(const GmmProblem& p) { return ((OP == G_MM ? p.n_out : p.n_in) + 255) >> 8; }
  MOE_DEV static int of_expert(const GmmProblem& p, int rows) {
    return m_count(p) * count(OP == G_DW ? p.n_out : rows);
  }
  MOE_DEV static int steps(const GmmProblem& p, int rows) {
    return OP == G_MM ? (p.n_in + KE - 1) / KE : OP == G_DX ? (p.n_out + KE - 1) / KE : max(1, (rows + KE - 1) / KE);
  }
  // Tile g whole: an expert's rows are cut into equal tiles.  A step's cost
  // is its operands' bytes (256 rows of A, np of B), between that of reading
  // weights from HBM (the same for every np) and that of the MMA.
  MOE_DEV static void get(const GmmProblem& p, const long long* cum, int g, GuItem& it) {
    it.e = gmm_expert_of(cum, p.E, g);
    it.r0 = gmm_off(p, it.e);
    it.r1 = gmm_off(p, it.e + 1);
    const int n_all = OP == G_DW ? p.n_out : it.r1 - it.r0;
    const unsigned nt = (unsigned)count(n_all), tile = (unsigned)(g - cum[it.e]);
    const int tn = min(kGuN, (int)(((unsigned)n_all + nt - 1) / nt + kRound - 1) & ~(kRound - 1));
    const int t_m = (int)(tile / nt), n_begin = (int)(tile % nt) * tn;
    it.m0 = t_m * 256;
    it.nv = max(0, min(tn, n_all - n_begin));
    it.np = max(kRound, (it.nv + kRound - 1) & ~(kRound - 1));
    it.n0 = OP == G_DW ? n_begin : it.r0 + n_begin;
    it.nkb = steps(p, it.r1 - it.r0);
    it.none = OP == G_DW && it.r1 == it.r0;
    it.cost = 256 + it.np;
  }
};

// Walks a piece; every warp that does, and both CTAs of the pair, see the same items.
template <int OP, int KE>
struct GuWalk {
  const GmmProblem& p;
  const long long* cum;
  int col, row, cols, n_tiles;
  long long pos, begin, end;

  MOE_DEV GuWalk(const GmmProblem& p_, const long long* cum_, const GuLine& line, int cols_, long long begin_,
                 long long end_)
      : p(p_), cum(cum_), col(line.start_col), row(line.start_row), cols(cols_), n_tiles((int)cum_[p_.E]),
        pos(line.start_pos), begin(begin_), end(end_) {}
  MOE_DEV bool next(GuItem& it) {
    while (pos < end) {
      GuTiles<OP, KE>::get(p, cum, row * cols + col, it);
      it.pos = pos;
      it.kb0 = pos >= begin ? 0 : (int)((begin - pos + it.cost - 1) / it.cost);
      const long long to = (end - pos + it.cost - 1) / it.cost;
      it.kb1 = to < it.nkb ? (int)to : it.nkb;
      pos += (long long)it.nkb * it.cost;
      if (++row * (long long)cols + col >= n_tiles) {
        row = 0;
        ++col;
      }
      if (it.kb0 < it.kb1) return true;
    }
    return false;
  }
};

template <typename T>
MOE_DEV T gu_cast(float v);
template <>
MOE_DEV float gu_cast<float>(float v) { return v; }
template <>
MOE_DEV __nv_bfloat16 gu_cast<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
MOE_DEV __half gu_cast<__half>(float v) { return __float2half_rn(v); }

// 32 columns (output rows n .. n+31) of this lane's M value
template <typename T>
MOE_DEV void gu_store32_t(void* out, long long base, long long ld, int left, const float (&v)[32]) {
  T* o = reinterpret_cast<T*>(out) + base;
#pragma unroll
  for (int i = 0; i < 32; ++i)
    if (i < left) o[i * ld] = gu_cast<T>(v[i]);
}
MOE_DEV void gu_store32(void* out, int type, long long base, long long ld, int left, const float (&v)[32]) {
  if (type == G_BF16) gu_store32_t<__nv_bfloat16>(out, base, ld, left, v);
  else if (type == G_FP16) gu_store32_t<__half>(out, base, ld, left, v);
  else gu_store32_t<float>(out, base, ld, left, v);
}

// ------------------------------------------------------------ the kernel
// Launched in clusters of two CTAs (gridDim.x even), one CTA per SM.
template <int OP, bool FP8, int CHAIN>
__global__ void __launch_bounds__(kGuThreads, 1) grouped_umma_kernel(const __grid_constant__ GuParams p) {
  constexpr bool A_MN = OP != G_MM, B_MN = OP == G_DW;
  constexpr int KE = FP8 ? 128 : 64;  // contracted values per step
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw32 = tc_smem(smem_raw);
  const uint32_t base = (raw32 + 1023u) & ~1023u;
  uint8_t* gen = smem_raw + (base - raw32);
  constexpr uint32_t kScaleOff = kGuStages * 2 * kGuTile, kCumOff = kScaleOff + kGuScaleSlots * kGuN * 4,
                     kLineOff = kCumOff + (kGmmMaxExperts + 1) * 8, kBarOff = kLineOff + sizeof(GuLine);
  const uint32_t sc0 = base + kScaleOff, bar = base + kBarOff;
  long long* cum = reinterpret_cast<long long*>(gen + kCumOff);
  GuLine& line = *reinterpret_cast<GuLine*>(gen + kLineOff);
  // (L): used in the leader CTA only
  auto full = [&](int s) { return bar + 8u * s; };                                   // (L) TMA bytes of both CTAs
  auto empty = [&](int s) { return bar + 8u * (kGuStages + s); };                    // MMA commit
  auto acc_full = [&](int b) { return bar + 8u * (2 * kGuStages + b); };             // MMA commit
  auto acc_empty = [&](int b) { return bar + 8u * (2 * kGuStages + 2 + b); };        // (L) epilogue warps of both CTAs
  auto sc_full = [&](int s) { return bar + 8u * (2 * kGuStages + 4 + s); };          // scale warp
  auto sc_empty = [&](int s) { return bar + 8u * (2 * kGuStages + 4 + kGuScaleSlots + s); };  // epilogue warps
  constexpr int kBars = 2 * kGuStages + 4 + 2 * kGuScaleSlots;
  const uint32_t drain = bar + 8u * kBars;                                           // (L)
  const uint32_t join = drain + 8u;                                                  // epilogue warps
  int* tail = reinterpret_cast<int*>(gen + (bar - base) + 8 * (kBars + 2));
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tail);
  volatile int* abort_flag = tail + 1;
  int* last_flag = tail + 2;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint32_t rank, pair, npairs;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm("mov.u32 %0, %%clusterid.x;" : "=r"(pair));
  asm("mov.u32 %0, %%nclusterid.x;" : "=r"(npairs));
  const bool leader = rank == 0;
  const GmmProblem& g = p.g;

  if (tid == 0) {
    for (int s = 0; s < kGuStages; ++s) {
      tc_bar_init(full(s), 1);
      tc_bar_init(empty(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      tc_bar_init(acc_full(b), 1);
      tc_bar_init(acc_empty(b), 2 * kGuEpiWarps);
    }
    for (int s = 0; s < kGuScaleSlots; ++s) {
      tc_bar_init(sc_full(s), 1);
      tc_bar_init(sc_empty(s), kGuEpiWarps);
    }
    tc_bar_init(drain, 1);
    tc_bar_init(join, kGuEpiWarps);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(tc_smem(tmem_slot)),
                 "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  using Tiles = GuTiles<OP, KE>;
  using Walk = GuWalk<OP, KE>;
  const int m_all = OP == G_MM ? g.n_out : g.n_in;
  const int cols = (int)npairs;
  const bool plan_ok = gmm_plan(
      g, [&](int rows) -> long long { return Tiles::of_expert(g, rows); }, cum, &line.flag);
  const int n_tiles = plan_ok ? (int)cum[g.E] : 0;
  for (int i = tid; i <= cols; i += kGuThreads) line.col[i] = 0;
  if (tid == 0) {
    line.cost_most = 0;
    line.start_pos = 0;
    line.start_col = line.start_row = 0;
  }
  __syncthreads();
  for (int t = tid; t < n_tiles; t += kGuThreads) {  // the cost of each hand
    GuItem it;
    Tiles::get(g, cum, t, it);
    atomicAdd(reinterpret_cast<unsigned long long*>(&line.col[t % cols]), (unsigned long long)it.nkb * it.cost);
    atomicMax(reinterpret_cast<unsigned long long*>(&line.cost_most), (unsigned long long)it.cost);
  }
  __syncthreads();
  if (warp == 0) {  // hands one after the other
    long long sum = 0;
    for (int c0 = 0; c0 < cols; c0 += 32) {
      const long long v = c0 + lane < cols ? line.col[c0 + lane] : 0;
      long long x = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (c0 + lane < cols) line.col[c0 + lane] = sum + x - v;
      sum += __shfl_sync(0xffffffffu, x, 31);
    }
    if (lane == 0) line.col[cols] = sum;
  }
  __syncthreads();
  // Pieces: one per pair, none shorter than a step (each piece that a tile
  // reaches into then holds a step of it), a tile cut into split_most at most.
  const long long total = line.col[cols];
  long long pieces = 0;
  if (total > 0) {
    pieces = min((long long)cols, total / line.cost_most);
    pieces = min(pieces, (long long)n_tiles * p.split_most);
  }
  const long long begin = pair < pieces ? (long long)pair * total / pieces : 0;
  const long long end = pair < pieces ? ((long long)pair + 1) * total / pieces : 0;
  auto piece_of = [&](long long u) { return (int)(((u + 1) * pieces - 1) / total); };
  if (warp == 0 && begin < end) {  // the piece's first tile
    int c = 0;
    for (int c0 = 0; c0 < cols; c0 += 32)
      c += __popc(__ballot_sync(0xffffffffu, c0 + lane < cols && line.col[c0 + lane + 1] <= begin));
    long long at = line.col[c];
    for (int row = 0;; row += 32) {
      const long long t = (long long)(row + lane) * cols + c;
      long long w = 0;
      if (t < n_tiles) {
        GuItem it;
        Tiles::get(g, cum, (int)t, it);
        w = (long long)it.nkb * it.cost;
      }
      long long x = w;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      const uint32_t here = __ballot_sync(0xffffffffu, w > 0 && at + x > begin);
      if (here) {
        if (lane == __ffs(here) - 1) {
          line.start_pos = at + x - w;
          line.start_col = c;
          line.start_row = row + lane;
        }
        break;
      }
      at += __shfl_sync(0xffffffffu, x, 31);
      if ((long long)(row + 32) * cols + c >= n_tiles) break;  // not reached: begin lies in this hand
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // both CTAs' barriers initialised and TMEM allocated before any cross-CTA use
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    // ================= TMA issuer of this CTA's halves of both operands
    if (lane == 0) {
      um_prefetch_map(&p.a_map);
      Walk walk(g, cum, line, cols, begin, end);
      GuItem it;
      int st = 0;
      uint32_t ph = 0;
      bool ok = true;
      while (ok && walk.next(it)) {
        if (it.none) continue;
        const int half = it.np >> 1;
        const int m = it.m0 + (int)rank * 128;
        const int bx = half <= 16 ? 0 : half <= 32 ? 1 : half <= 64 ? 2 : 3;
        const int panels = (half + 63) >> 6;  // dw
        for (int kb = it.kb0; kb < it.kb1; ++kb) {
          if (!cl_bar_wait(empty(st), ph ^ 1u, abort_flag)) {
            ok = false;
            break;
          }
          const uint32_t a = base + (uint32_t)st * 2 * kGuTile, b = a + kGuTile;
          const uint32_t fb = cl_addr(full(st), 0);
          if constexpr (OP != G_DW) {
            if (leader) um_expect_tx(full(st), (uint32_t)(2 * (kGuTile + (16 << bx) * 128)));
            if constexpr (OP == G_MM) {
              gu_tma_3d(a, &p.a_map, kb * KE, m, it.e, fb);
            } else {
              gu_tma_3d(a, &p.a_map, m, kb * KE, it.e, fb);
              gu_tma_3d(a + 8192, &p.a_map, m + 64, kb * KE, it.e, fb);
            }
            gu_tma_2d(b, &p.b_map[bx], kb * KE, it.n0 + (int)rank * half, fb);
          } else {
            const int y = it.r0 + kb * KE, left = it.r1 - y, n = it.n0 + (int)rank * half;
            if (left >= KE) {
              if (leader) um_expect_tx(full(st), (uint32_t)(2 * (kGuTile + panels * 8192)));
              gu_tma_2d(a, &p.a_map, m, y, fb);
              gu_tma_2d(a + 8192, &p.a_map, m + 64, y, fb);
              for (int q = 0; q < panels; ++q) gu_tma_2d(b + q * 8192, &p.b_map[0], n + 64 * q, y, fb);
            } else {
              const int fill = (left + 15) & ~15;
              if (leader) um_expect_tx(full(st), (uint32_t)(2 * fill * 128 * (2 + panels)));
              for (int q = 0; q < 2 + panels; ++q) {
                const bool isa = q < 2;
                const uint32_t dst = isa ? a + q * 8192 : b + (q - 2) * 8192;
                const int x = isa ? m + 64 * q : n + 64 * (q - 2);
                const CUtensorMap* maps = isa ? p.a_tail : p.b_tail;
                int r = 0;
                for (; r + 8 <= left; r += 8) gu_tma_2d(dst + r * 128, &maps[0], x, y + r, fb);
                for (; r & 7 || r < left; ++r)  // rows beyond the expert's: from beyond the tensor, zeros
                  gu_tma_2d(dst + r * 128, &maps[1], x, r < left ? y + r : g.rows, fb);
                if (r < fill) gu_tma_2d(dst + r * 128, &maps[0], x, g.rows, fb);
              }
            }
          }
          if (++st == kGuStages) st = 0, ph ^= 1u;
        }
      }
      if (!ok) {  // a wait gave up: let the copies in flight land before this CTA's memory is released
        const long long t0 = clock64();
        while (clock64() - t0 < kGuLinger) {
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ================= MMA issuer (leader CTA)
    if (leader && lane == 0) {
      Walk walk(g, cum, line, cols, begin, end);
      GuItem it;
      int st = 0, seg = 0;
      uint32_t ph = 0;
      bool ok = true;
      const uint32_t idesc0 = (1u << 4) | ((uint32_t)(p.type == G_BF16 ? 1 : 0) * ((1u << 7) | (1u << 10))) |
                              ((A_MN ? 1u : 0u) << 15) | ((B_MN ? 1u : 0u) << 16) | (16u << 24);
      const uint64_t da0 = gu_desc(base, A_MN), db0 = gu_desc(base + kGuTile, B_MN);
      while (ok && walk.next(it)) {
        if (it.none) continue;
        const uint32_t idesc = idesc0 | ((uint32_t)(it.np >> 3) << 17);
        for (int kb = it.kb0; kb < it.kb1;) {
          const int kend = CHAIN ? min(it.kb1, kb + CHAIN) : it.kb1;
          const int buf = seg & 1;
          if (!cl_bar_wait(acc_empty(buf), ((seg >> 1) & 1) ^ 1u, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d = tmem + (uint32_t)buf * kGuN;
          uint32_t acc = 0;
          for (; kb < kend; ++kb) {
            if (!cl_bar_wait(full(st), ph, abort_flag)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint64_t so = (uint64_t)((uint32_t)st * 2 * kGuTile >> 4);
            int steps = 4;
            if constexpr (OP == G_DW) steps = min(4, (it.r1 - it.r0 - kb * KE + 15) >> 4);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (OP != G_DW || k < steps) {
                // 16 (e4m3: 32) contracted values: 32 bytes along a K-major row, 16 rows of a panel otherwise
                gu_mma<FP8>(d, da0 + so + (uint64_t)((A_MN ? 2048 : 32) * k >> 4),
                            db0 + so + (uint64_t)((B_MN ? 2048 : 32) * k >> 4), idesc, acc);
                acc = 1;
              }
            umma2_commit_both(empty(st));
            if (++st == kGuStages) st = 0, ph ^= 1u;
          }
          if (!ok) break;
          umma2_commit_both(acc_full(buf));
          ++seg;
        }
      }
      umma2_commit_both(drain);
      const long long t0 = clock64();
      while (!cl_bar_try(drain, 0) && clock64() - t0 < kTcWaitCycles) {
      }
    }
    __syncwarp();
  } else if (warp == 2) {
    // ================= 8-bit product: the scales of each step, row scale times this CTA's weight scale
    if constexpr (FP8) {
      Walk walk(g, cum, line, cols, begin, end);
      GuItem it;
      int slot = 0;
      uint32_t ph = 0;
      bool ok = true;
      const int groups = (g.n_in + 127) >> 7;
      constexpr int AHEAD = 4;  // steps whose loads are in flight together
      while (ok && walk.next(it)) {
        const int ob = (it.m0 >> 7) + (int)rank;
        const float* swp = g.sw + ((long long)it.e * ((g.n_out + 127) >> 7) + ob) * groups;
        const bool live = ob * 128 < g.n_out;
        const float* sxp = g.sx + it.n0;
        for (int k0 = it.kb0; k0 < it.kb1 && ok; k0 += AHEAD) {
          float v[AHEAD][8], w[AHEAD];
#pragma unroll
          for (int a = 0; a < AHEAD; ++a) {
            const int kb = min(k0 + a, it.kb1 - 1);
            w[a] = live ? __ldg(swp + kb) : 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const int c = lane + 32 * j;
              v[a][j] = c < it.nv ? __ldg(sxp + (long long)kb * g.rows + c) : 0.f;
            }
          }
#pragma unroll
          for (int a = 0; a < AHEAD; ++a) {
            if (k0 + a >= it.kb1) break;
            ok = cl_bar_wait(sc_empty(slot), ph ^ 1u, abort_flag);
            if (!__all_sync(0xffffffffu, ok)) {
              ok = false;
              break;
            }
            const uint32_t dst = sc0 + (uint32_t)slot * kGuN * 4 + 4u * lane;
#pragma unroll
            for (int j = 0; j < 8; ++j)
              asm volatile("st.shared.f32 [%0], %1;" ::"r"(dst + 128u * j), "f"(v[a][j] * w[a]) : "memory");
            __syncwarp();
            if (lane == 0) tc_bar_arrive(sc_full(slot));
            if (++slot == kGuScaleSlots) slot = 0, ph ^= 1u;
          }
        }
      }
    }
  } else if (warp >= 4) {
    // ================= epilogue: 32 TMEM lanes (M values) and every other 32 columns (output rows) per warp
    const int q = warp & 3, h = (warp - 4) >> 2;
    Walk walk(g, cum, line, cols, begin, end);
    GuItem it;
    int seg = 0, slot = 0;
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
    auto part_of = [&](int piece, int which) {
      return reinterpret_cast<float*>(p.ws + kGuParts + (size_t)((piece * 2 + (int)rank) * 2 + which) * kGuPart) + 32 * q +
             lane;
    };
    bool ok = true;
    while (ok && walk.next(it)) {
      const int chunks = (it.np + 31) >> 5;
      const int m = it.m0 + (int)rank * 128 + 32 * q + lane;
      const long long ld = OP == G_DW ? g.n_in : g.ld_out;
      const long long ob = (OP == G_DW ? ((long long)it.e * g.n_out + it.n0) * g.n_in : (long long)it.n0 * g.ld_out) + m;
      const bool whole = it.kb0 == 0 && it.kb1 == it.nkb;
      float* part = part_of((int)pair, it.kb0 > 0 ? 0 : 1);
      auto put = [&](int c, const float (&v)[32]) {
        if (whole) {
          if (m < m_all) gu_store32(g.out, g.out_type, ob + 32 * c * ld, ld, it.nv - 32 * c, v);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) __stcg(part + (32 * c + i) * 128, v[i]);
        }
      };
      if (it.none) {
        float z[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) z[i] = 0.f;
        for (int c = h; c < chunks; c += 2)
          if (m < m_all) gu_store32(g.out, g.out_type, ob + 32 * c * ld, ld, it.nv - 32 * c, z);
        continue;
      }
      if constexpr (CHAIN == 0) {
        const int buf = seg & 1;
        ok = cl_bar_wait(acc_full(buf), (seg >> 1) & 1, abort_flag);
        if (!__all_sync(0xffffffffu, ok)) break;
        tc_fence_after();
        for (int c = h; c < chunks; c += 2) {
          float v[32];
          gu_ld32(lane_addr + (uint32_t)(buf * kGuN + 32 * c), v);
          put(c, v);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) cl_arrive(cl_addr(acc_empty(buf), 0));
        ++seg;
      } else {
        float acc[4][32];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int i = 0; i < 32; ++i) acc[j][i] = 0.f;
        for (int kb = it.kb0; kb < it.kb1; kb += CHAIN) {
          const int buf = seg & 1;
          ok = cl_bar_wait(acc_full(buf), (seg >> 1) & 1, abort_flag);
          if (FP8) ok = ok && tc_bar_wait(sc_full(slot), sph, abort_flag);
          if (!__all_sync(0xffffffffu, ok)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sp = sc0 + (uint32_t)slot * kGuN * 4;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int c = 2 * j + h;
            if (c < chunks) {
              float v[32];
              gu_ld32(lane_addr + (uint32_t)(buf * kGuN + 32 * c), v);
#pragma unroll
              for (int i = 0; i < 32; i += 4) {
                if constexpr (FP8) {
                  const uint4 s = tc_lds128(sp + (uint32_t)(32 * c + i) * 4);
                  acc[j][i] = fmaf(v[i], __uint_as_float(s.x), acc[j][i]);
                  acc[j][i + 1] = fmaf(v[i + 1], __uint_as_float(s.y), acc[j][i + 1]);
                  acc[j][i + 2] = fmaf(v[i + 2], __uint_as_float(s.z), acc[j][i + 2]);
                  acc[j][i + 3] = fmaf(v[i + 3], __uint_as_float(s.w), acc[j][i + 3]);
                } else {
#pragma unroll
                  for (int k = 0; k < 4; ++k) acc[j][i + k] += v[i + k];
                }
              }
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            cl_arrive(cl_addr(acc_empty(buf), 0));
            if (FP8) tc_bar_arrive(sc_empty(slot));
          }
          ++seg;
          if (FP8 && ++slot == kGuScaleSlots) slot = 0, sph ^= 1u;
        }
        if (!ok) break;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (2 * j + h < chunks) put(2 * j + h, acc[j]);
      }
      if (!whole) {
        // count this part in; the last part's CTA adds them all, in the pieces' order
        const int first = piece_of(it.pos), last = piece_of(it.pos + (long long)(it.nkb - 1) * it.cost);
        __threadfence();
        ok = epi_sync();
        if (!ok) break;
        if (tid == 128) {
          unsigned* ctr = counters + first * 2 + rank;
          const unsigned before = atomicAdd(ctr, 1u);
          *last_flag = before == (unsigned)(last - first);
          if (before == (unsigned)(last - first)) *ctr = 0;
        }
        ok = epi_sync();
        if (!ok) break;
        const bool mine = *reinterpret_cast<volatile int*>(last_flag) != 0;
        ok = epi_sync();  // the flag is read before the next item can write it
        if (!ok) break;
        if (mine) {
          __threadfence();
          for (int c = h; c < chunks; c += 2) {
            float v[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = __ldcg(part_of(first, 1) + (32 * c + i) * 128);
            for (int s = first + 1; s <= last; ++s) {
              const float* src = part_of(s, 0);
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] += __ldcg(src + (32 * c + i) * 128);
            }
            if (m < m_all) gu_store32(g.out, g.out_type, ob + 32 * c * ld, ld, it.nv - 32 * c, v);
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
// pairs fit at once (0: none).
template <int OP, bool FP8, int CHAIN>
bool gu_launch(const GuParams& p, int pairs, cudaStream_t s);
template <int OP, bool FP8, int CHAIN>
int gu_pairs();
constexpr int kGuChain = 8;  // 16-bit products with fp32 outputs: 512 contracted values per chain
#define MOE_GU_DECL(OP, FP8, CHAIN)                                                \
  template <>                                                                      \
  bool gu_launch<OP, FP8, CHAIN>(const GuParams& p, int pairs, cudaStream_t s);    \
  template <>                                                                      \
  int gu_pairs<OP, FP8, CHAIN>();
MOE_GU_DECL(G_MM, false, 0)
MOE_GU_DECL(G_MM, false, kGuChain)
MOE_GU_DECL(G_DX, false, 0)
MOE_GU_DECL(G_DX, false, kGuChain)
MOE_GU_DECL(G_DW, false, 0)
MOE_GU_DECL(G_DW, false, kGuChain)
MOE_GU_DECL(G_MM, true, 1)
#undef MOE_GU_DECL

}  // namespace moe
