// Grouped products for operands of any alignment and row stride, on the
// warp-level tensor-core MMA (m16n8k16, 16-bit operands, fp32 sums): the
// layouts that the tensor-memory kernel cannot take, whose copies need
// 16-byte aligned rows.  e4m3 operands widen to fp16 on their way into shared
// memory (exact, as are their products in fp32).
//
// A block computes 64 (M) x 64 (N) outputs over steps of 32 of the contracted
// dimension; the next step's values are in registers while this one's are
// multiplied.  Every 128 contracted values the step sums are added to the
// block's sums with an ordinary fp32 addition (the tensor core truncates as it
// accumulates); for the 8-bit product, whose scales change every 128 inputs,
// this is where they are applied.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "grouped_plan.cuh"

namespace moe {

constexpr int kGaTile = 64, kGaK = 32, kGaThreads = 128;
constexpr int kGaPitch = kGaK + 8;  // 16-bit values per shared row: fragment reads hit 32 banks

template <int IN>
MOE_DEV void ga_mma(float (&c)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  if constexpr (IN == G_BF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

// one value as the 16 bits that the MMA reads
template <int IN>
MOE_DEV uint16_t ga_load(const void* base, long long i) {
  if constexpr (IN == G_E4M3) {
    const __half_raw h = __nv_cvt_fp8_to_halfraw(reinterpret_cast<const __nv_fp8_storage_t*>(base)[i], __NV_E4M3);
    return h.x;
  } else {
    return reinterpret_cast<const uint16_t*>(base)[i];
  }
}

// 64 x 32 values of one side.  KFAST: the contracted dimension is the
// contiguous one.  i0/c0: first index and first contracted index; ni/nc: how
// many are left (zeros beyond).
template <int IN, bool KFAST>
struct GaSide {
  uint16_t v[16];
  MOE_DEV void load(const void* base, long long ld, int ni, int nc) {
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const int q = threadIdx.x + kGaThreads * j;
      const int i = KFAST ? q / kGaK : q % kGaTile, c = KFAST ? q % kGaK : q / kGaTile;
      v[j] = i < ni && c < nc ? ga_load<IN>(base, KFAST ? i * ld + c : c * ld + i) : (uint16_t)0;
    }
  }
  MOE_DEV void put(uint16_t* s) const {
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const int q = threadIdx.x + kGaThreads * j;
      const int i = KFAST ? q / kGaK : q % kGaTile, c = KFAST ? q % kGaK : q / kGaTile;
      s[i * kGaPitch + c] = v[j];
    }
  }
};

template <int OP, int IN>
__global__ void __launch_bounds__(kGaThreads) grouped_any_kernel(const GmmProblem p) {
  __shared__ long long cum[kGmmMaxExperts + 1];
  __shared__ int flag;
  __shared__ __align__(16) uint16_t sm[kGaTile * kGaPitch], sn[kGaTile * kGaPitch];
  const int m_all = OP == G_MM ? p.n_out : p.n_in;
  const int m_tiles = (m_all + kGaTile - 1) / kGaTile;
  const int o_tiles = (p.n_out + kGaTile - 1) / kGaTile;
  const bool ok = gmm_plan(
      p,
      [&](int rows) -> long long {
        return (long long)m_tiles * (OP == G_DW ? o_tiles : (rows + kGaTile - 1) / kGaTile);
      },
      cum, &flag);
  if (!ok) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int wm = (warp & 1) * 32, wn = (warp >> 1) * 32;
  constexpr int bytes = IN == G_E4M3 ? 1 : 2;
  for (long long u = blockIdx.x; u < cum[p.E]; u += gridDim.x) {
    const int e = gmm_expert_of(cum, p.E, u);
    const int v = (int)(u - cum[e]);
    const int m0 = v % m_tiles * kGaTile, nt = v / m_tiles;
    const int r0 = gmm_off(p, e), r1 = gmm_off(p, e + 1);
    const int n0 = OP == G_DW ? nt * kGaTile : r0 + nt * kGaTile;          // first output row
    const int nn = min(kGaTile, (OP == G_DW ? p.n_out : r1) - n0), nm = min(kGaTile, m_all - m0);
    const int nc = OP == G_MM ? p.n_in : OP == G_DX ? p.n_out : r1 - r0;   // contracted values
    // the sides at contracted index 0
    const char* mp = OP == G_DW ? reinterpret_cast<const char*>(p.x) + ((long long)r0 * p.ld_x + m0) * bytes
                                : reinterpret_cast<const char*>(p.w) +
                                      ((long long)e * p.n_out * p.n_in + (OP == G_MM ? (long long)m0 * p.n_in : m0)) * bytes;
    const char* np = reinterpret_cast<const char*>(p.rows_in) +
                     (OP == G_DW ? (long long)r0 * p.ld_rows + n0 : (long long)n0 * p.ld_rows) * bytes;
    const long long ld_m = OP == G_DW ? p.ld_x : p.n_in, ld_n = p.ld_rows;
    GaSide<IN, OP == G_MM> am;
    GaSide<IN, OP != G_DW> an;
    float acc[2][4][4] = {}, part[2][4][4] = {};
    am.load(mp, ld_m, nm, nc);
    an.load(np, ld_n, nn, nc);
    for (int c0 = 0; c0 < nc; c0 += kGaK) {
      __syncthreads();
      am.put(sm);
      an.put(sn);
      __syncthreads();
      if (c0 + kGaK < nc) {
        const long long c = c0 + kGaK;
        am.load(mp + (OP == G_MM ? c : c * ld_m) * bytes, ld_m, nm, nc - (int)c);
        an.load(np + (OP == G_DW ? c * ld_n : c) * bytes, ld_n, nn, nc - (int)c);
      }
#pragma unroll
      for (int kk = 0; kk < kGaK; kk += 16) {
        uint32_t a[2][4], b[4][2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint16_t* q = sm + (wm + 16 * i + g) * kGaPitch + kk + 2 * t;
          a[i][0] = *reinterpret_cast<const uint32_t*>(q);
          a[i][1] = *reinterpret_cast<const uint32_t*>(q + 8 * kGaPitch);
          a[i][2] = *reinterpret_cast<const uint32_t*>(q + 8);
          a[i][3] = *reinterpret_cast<const uint32_t*>(q + 8 * kGaPitch + 8);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint16_t* q = sn + (wn + 8 * j + g) * kGaPitch + kk + 2 * t;
          b[j][0] = *reinterpret_cast<const uint32_t*>(q);
          b[j][1] = *reinterpret_cast<const uint32_t*>(q + 8);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) ga_mma<IN>(part[i][j], a[i], b[j]);
      }
      if ((c0 & 96) == 96 || c0 + kGaK >= nc) {  // 128 contracted values, or the last ones
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
