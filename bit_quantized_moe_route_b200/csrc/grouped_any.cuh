// Grouped products for operands of any alignment and row stride, on the
// warp-level tensor-core MMA: the layouts that the tensor-memory kernel cannot
// take, whose TMA copies need 16-byte aligned rows.
//
// A block computes 128 (M) x 64 (N) outputs; eight warps 32 x 32 each.  A step
// is 64 bytes of the contracted dimension: 32 16-bit values (m16n8k16) or 64
// e4m3 codes (m16n8k32, whose operand layout is the same in bytes).  Operands
// go through registers: a 16-byte piece at any address is cut out of the two
// aligned 16-byte blocks that hold it (both inside the operand, else byte by
// byte), and the next step's pieces are in flight while this one's are
// multiplied.  K-major operands lie in shared memory as [row][64 bytes], those
// contiguous along M or N as [contracted row][values], read with the
// transposing ldmatrix; 16-byte pieces are permuted by the row so that both
// the stores and the reads touch all banks.
//
// Every 128 contracted values the step sums are added to the block's sums with
// an ordinary fp32 addition (the tensor core truncates as it accumulates); for
// the 8-bit product, whose scales change every 128 inputs, this is where they
// are applied.
//
// Bound by the latency of the loads and the instructions around them (two
// loads, a shift by selects and a store for each 16 bytes), so two blocks share
// an SM, and steps whose pieces are all whole and inside the operand skip every
// check.  Tried and slower: 128 x 128 tiles, one block per SM; raw blocks
// brought in by asynchronous copies three steps ahead and shifted from shared
// memory.
#pragma once

#include <cuda_fp16.h>

#include "grouped_plan.cuh"

namespace moe {

constexpr int kGaM = 128, kGaN = 64, kGaThreads = 256;

template <int IN>
MOE_DEV void ga_mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (IN == G_BF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else if constexpr (IN == G_FP16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <bool TRANS>
MOE_DEV void ga_ldm(uint32_t addr, uint32_t (&r)[4]) {
  if constexpr (TRANS)
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
  else
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}

// One side of a step: ROWS values of M or N.  KFAST: the contracted dimension
// is the contiguous one.  A thread has the same pieces (a shared row and 16
// bytes of it) of every step, so that their addresses advance by a constant.
template <int ROWS, bool KFAST, int ES>
struct GaSide {
  static constexpr int kPieces = ROWS * 4 / kGaThreads;  // per thread
  static constexpr int kChunks = KFAST ? 4 : ROWS / 8;   // pieces per shared row
  const char *lo, *hi;      // the operand's bytes: nothing else is read
  const char* at[kPieces];  // where the next step's pieces begin
  uint4 a[kPieces], b[kPieces];
  long long step;           // bytes to the same piece of the next step
  int n[kPieces];           // valid bytes, 16 at most
  const char *first, *last; // the next step's lowest and highest byte (all ROWS rows)
  bool plain;               // the step loaded: every piece whole, or its row not there

  // p: value (0, 0) of the tile; ld: bytes between shared rows
  MOE_DEV void begin(const char* lo_, const char* hi_, const char* p, long long ld) {
    lo = lo_;
    hi = hi_;
    step = KFAST ? 64 : ld * (64 / ES);
    first = p;
    last = p + ((KFAST ? ROWS : 64 / ES) - 1) * ld + (KFAST ? 64 : ROWS * ES);
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
      const int q = threadIdx.x + kGaThreads * j;
      at[j] = p + (q / kChunks) * ld + 16 * (q % kChunks);
    }
  }
  // loads the next step: rows: shared rows there are; len: bytes in use of each
  MOE_DEV void load(int rows, int len) {
    constexpr int kAll = KFAST ? ROWS : 64 / ES;
    plain = rows == kAll && len >= 16 * kChunks && first - 16 >= lo && last + 32 <= hi;
    first += step;
    last += step;
    if (plain) {
#pragma unroll
      for (int j = 0; j < kPieces; ++j) {
        const uint4* p0 = reinterpret_cast<const uint4*>(reinterpret_cast<uintptr_t>(at[j]) & ~(uintptr_t)15);
        a[j] = __ldg(p0);
        b[j] = __ldg(p0 + 1);
      }
      return;
    }
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
      const int q = threadIdx.x + kGaThreads * j, r = q / kChunks, c = q % kChunks;
      n[j] = r < rows ? min(16, len - 16 * c) : 0;
      if (n[j] > 0) {
        const int shift = (int)(reinterpret_cast<uintptr_t>(at[j]) & 15);
        const char* p0 = at[j] - shift;
        if (p0 >= lo && p0 + 32 <= hi) {
          a[j] = __ldg(reinterpret_cast<const uint4*>(p0));
          if (shift) b[j] = __ldg(reinterpret_cast<const uint4*>(p0) + 1);
        } else {  // at an end of the operand: its bytes one by one, where they lie in the blocks
          uint32_t w[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (p0 + i >= lo && p0 + i < hi)
              w[i >> 2] |= (uint32_t) * reinterpret_cast<const uint8_t*>(p0 + i) << (8 * (i & 3));
          a[j] = make_uint4(w[0], w[1], w[2], w[3]);
          b[j] = make_uint4(w[4], w[5], w[6], w[7]);
        }
      }
    }
  }
  // 16-byte piece c of shared row r
  MOE_DEV static uint32_t place(int r, int c) {
    return (uint32_t)(r * kChunks + (KFAST ? c ^ ((r >> 1) & 3) : c ^ (r & 7))) * 16;
  }
  // the loaded step into the tile; on to the next
  MOE_DEV void put(uint32_t tile) {
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
      const int q = threadIdx.x + kGaThreads * j;
      uint32_t o[4] = {0, 0, 0, 0};
      if (plain || n[j] > 0) {
        const uint32_t w[8] = {a[j].x, a[j].y, a[j].z, a[j].w, b[j].x, b[j].y, b[j].z, b[j].w};
        uint32_t t[6], u[5];
        const int shift = (int)(reinterpret_cast<uintptr_t>(at[j]) & 15), bits = (shift & 3) * 8;
#pragma unroll
        for (int i = 0; i < 6; ++i) t[i] = shift & 8 ? w[i + 2] : w[i];
#pragma unroll
        for (int i = 0; i < 5; ++i) u[i] = shift & 4 ? t[i + 1] : t[i];
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = __funnelshift_r(u[i], u[i + 1], bits);
        if (!plain && n[j] < 16) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int left = n[j] - 4 * i;  // valid bytes of this word
            o[i] = left >= 4 ? o[i] : left <= 0 ? 0u : o[i] & (0xFFFFFFFFu >> (32 - 8 * left));
          }
        }
      }
      asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(tile + place(q / kChunks, q % kChunks)), "r"(o[0]),
                   "r"(o[1]), "r"(o[2]), "r"(o[3])
                   : "memory");
      at[j] += step;
    }
  }
  // The 16 x 32-byte block at (i0, kk-th 32 bytes) as four 8 x 16-byte
  // matrices: rows 0-7 and 8-15 of the first 16 bytes, then of the second.
  MOE_DEV static void frag(uint32_t tile, int i0, int kk, uint32_t (&r)[4]) {
    const int lane = threadIdx.x & 31;
    if constexpr (KFAST) {
      ga_ldm<false>(tile + place(i0 + (lane & 15), 2 * kk + (lane >> 4)), r);
    } else {
      // [contracted row][values]: matrices of 8 contracted rows x 8 values, transposed
      const int k = 16 * kk + (lane & 7) + (lane >> 4) * 8;
      ga_ldm<true>(tile + place(k, (i0 >> 3) + ((lane >> 3) & 1)), r);
    }
  }
};

template <int OP, int IN>
__global__ void __launch_bounds__(kGaThreads, 2) grouped_any_kernel(const GmmProblem p) {
  constexpr int ES = IN == G_E4M3 ? 1 : 2;
  using SideM = GaSide<kGaM, OP == G_MM, ES>;
  using SideN = GaSide<kGaN, OP != G_DW, ES>;
  constexpr int KS = 64 / ES;
  __shared__ long long cum[kGmmMaxExperts + 1];
  __shared__ int flag;
  __shared__ __align__(128) uint8_t sm[2][(kGaM + kGaN) * 64];
  const int m_all = OP == G_MM ? p.n_out : p.n_in;
  const int m_tiles = (m_all + kGaM - 1) / kGaM;
  const int o_tiles = (p.n_out + kGaN - 1) / kGaN;
  const bool ok = gmm_plan(
      p,
      [&](int rows) -> long long { return (long long)m_tiles * (OP == G_DW ? o_tiles : (rows + kGaN - 1) / kGaN); }, cum,
      &flag);
  if (!ok) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int wm = (warp & 3) * 32, wn = (warp >> 2) * 32;
  const uint32_t tile0 = (uint32_t)__cvta_generic_to_shared(&sm[0][0]);
  const char* lo_m = reinterpret_cast<const char*>(OP == G_DW ? p.x : p.w);
  const char* hi_m =
      lo_m + (OP == G_DW ? ((long long)(p.rows - 1) * p.ld_x + p.n_in) : (long long)p.E * p.n_out * p.n_in) * ES;
  const char* lo_n = reinterpret_cast<const char*>(p.rows_in);
  const char* hi_n = lo_n + ((long long)(p.rows - 1) * p.ld_rows + (OP == G_MM ? p.n_in : p.n_out)) * ES;
  for (long long u = blockIdx.x; u < cum[p.E]; u += gridDim.x) {
    const int e = gmm_expert_of(cum, p.E, u);
    const long long v = u - cum[e];
    const int m0 = (int)(v % m_tiles) * kGaM, nt = (int)(v / m_tiles);
    const int r0 = gmm_off(p, e), r1 = gmm_off(p, e + 1);
    const int n0 = OP == G_DW ? nt * kGaN : r0 + nt * kGaN;                // first output row
    const int nn = min(kGaN, (OP == G_DW ? p.n_out : r1) - n0), nm = min(kGaM, m_all - m0);
    const int nc = OP == G_MM ? p.n_in : OP == G_DX ? p.n_out : r1 - r0;   // contracted values
    SideM am;
    SideN an;
    am.begin(lo_m, hi_m,
             lo_m + (OP == G_DW ? (long long)r0 * p.ld_x + m0
                                : (long long)e * p.n_out * p.n_in + (OP == G_MM ? (long long)m0 * p.n_in : m0)) * ES,
             (OP == G_DW ? p.ld_x : p.n_in) * ES);
    an.begin(lo_n, hi_n, lo_n + (OP == G_DW ? (long long)r0 * p.ld_rows + n0 : (long long)n0 * p.ld_rows) * ES,
             p.ld_rows * ES);
    auto load = [&](int c0) {
      const int k = min(KS, nc - c0);
      am.load(OP == G_MM ? nm : k, (OP == G_MM ? k : nm) * ES);
      an.load(OP == G_DW ? k : nn, (OP == G_DW ? nn : k) * ES);
    };
    float acc[2][4][4] = {}, part[2][4][4] = {};
    if (nc > 0) load(0);
    for (int c0 = 0, b = 0; c0 < nc; c0 += KS, b ^= 1) {
      const uint32_t bm = tile0 + (uint32_t)(b * (kGaM + kGaN) * 64), bn = bm + kGaM * 64;
      am.put(bm);
      an.put(bn);
      __syncthreads();  // (the other buffer's readers have been here since)
      if (c0 + KS < nc) load(c0 + KS);
      if (wn < nn) {
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
          uint32_t fa[2][4], fb[2][4];
#pragma unroll
          for (int i = 0; i < 2; ++i) SideM::frag(bm, wm + 16 * i, kk, fa[i]);
#pragma unroll
          for (int j = 0; j < 2; ++j) SideN::frag(bn, wn + 16 * j, kk, fb[j]);
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) ga_mma<IN>(part[i][j], fa[i], fb[j >> 1][j & 1], fb[j >> 1][2 + (j & 1)]);
        }
      }
      if (((c0 + KS) & 127) == 0 || c0 + KS >= nc) {  // 128 contracted values, or the last ones
        const int grp = c0 >> 7;
        float sw = 1.f;
        if constexpr (IN == G_E4M3)
          sw = __ldg(p.sw + ((long long)e * ((p.n_out + 127) >> 7) + (m0 >> 7)) * ((p.n_in + 127) >> 7) + grp);
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float s = 1.f;
            if constexpr (IN == G_E4M3) {
              const int n = wn + 8 * j + 2 * t + h;
              s = n < nn ? sw * __ldg(p.sx + (long long)grp * p.rows + n0 + n) : 0.f;
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              acc[i][j][h] = fmaf(part[i][j][h], s, acc[i][j][h]);
              acc[i][j][2 + h] = fmaf(part[i][j][2 + h], s, acc[i][j][2 + h]);
              part[i][j][h] = part[i][j][2 + h] = 0.f;
            }
          }
      }
    }
    __syncthreads();  // before the next tile's first step
    const long long ob = OP == G_DW ? ((long long)e * p.n_out + n0) * p.n_in + m0 : (long long)n0 * p.ld_out + m0;
    const long long ldo = OP == G_DW ? p.n_in : p.ld_out;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          const int m = wm + 16 * i + g + 8 * (h >> 1), n = wn + 8 * j + 2 * t + (h & 1);
          if (m < nm && n < nn) gmm_store(p.out, p.out_type, ob + n * ldo + m, acc[i][j][h]);
        }
  }
}

}  // namespace moe
