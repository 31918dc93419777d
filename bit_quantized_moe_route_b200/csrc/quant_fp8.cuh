// Rows to 8 bits with one scale for each 128 inputs:
//   a = max |x| over the group (at least 448 * 2^-126, so that the scale is a
//   normal number), s = a / 448, q = e4m3(x * (448 / a)),
// both quotients and the product rounded once to fp32, the code to nearest
// even.  A group that holds an infinity or a NaN becomes NaN codes or an
// infinite or NaN scale, so that what is computed from it is NaN too.
//
// Bound by HBM: 2 bytes read and 1 + 4/128 written per input.  A block takes
// 32 rows x 512 inputs; a warp takes four of the rows with all their loads in
// flight, 16 inputs (32 bytes) per lane, so that a group is eight lanes and
// its maximum three shuffles.  Scales are stored [group][row] and leave
// through shared memory as 128-byte runs.  Rows that are not 16-byte aligned
// take the same path value by value, lanes over consecutive inputs.
#pragma once

#include <cuda_fp16.h>

#include "grouped_plan.cuh"

namespace moe {

constexpr int kQfThreads = 256, kQfRows = 32, kQfCols = 512, kQfPerWarp = 4;

MOE_DEV float qf_value(uint32_t bits16, int type) {
  return type == G_BF16 ? bf16_bits_to_float(bits16) : __half2float(__ushort_as_half((unsigned short)bits16));
}
// |v| as an integer whose order is that of the magnitudes, with infinity and NaN above all
MOE_DEV uint32_t qf_mag(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }
MOE_DEV void qf_scales(uint32_t mag, float* s, float* inv) {
  const float a = __uint_as_float(max(mag, __float_as_uint(448.f * 1.17549435e-38f)));
  *s = __fdiv_rn(a, 448.f);
  *inv = __fdiv_rn(448.f, a);
}
// two values to two codes, the first in the low byte
MOE_DEV uint32_t qf_code2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

template <int TYPE, bool VEC>
__global__ void __launch_bounds__(kQfThreads) quant_fp8_kernel(const uint16_t* __restrict__ x, long long ld, int rows,
                                                               int n, uint8_t* __restrict__ q, float* __restrict__ s) {
  __shared__ float scales[kQfCols / 128][kQfRows + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c0 = blockIdx.y * kQfCols;
  const int groups = (n + 127) >> 7;
  for (long long b = blockIdx.x; b * kQfRows < rows; b += gridDim.x) {
    const int r0 = (int)(b * kQfRows) + warp * kQfPerWarp;
    if constexpr (VEC) {
      const int c = c0 + 16 * lane;  // n is a multiple of 16 here
      uint4 v[kQfPerWarp][2];
#pragma unroll
      for (int i = 0; i < kQfPerWarp; ++i) {
        v[i][0] = v[i][1] = make_uint4(0, 0, 0, 0);
        if (r0 + i < rows && c < n) {
          const uint16_t* src = x + (r0 + i) * ld + c;
          v[i][0] = ldg_stream(src);
          v[i][1] = ldg_stream(src + 8);
        }
      }
#pragma unroll
      for (int i = 0; i < kQfPerWarp; ++i) {
        const uint32_t w[8] = {v[i][0].x, v[i][0].y, v[i][0].z, v[i][0].w, v[i][1].x, v[i][1].y, v[i][1].z, v[i][1].w};
        float f[16];
        uint32_t mag = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          f[2 * j] = qf_value(w[j] & 0xFFFFu, TYPE);
          f[2 * j + 1] = qf_value(w[j] >> 16, TYPE);
          mag = max(mag, max(qf_mag(f[2 * j]), qf_mag(f[2 * j + 1])));
        }
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) mag = max(mag, __shfl_xor_sync(0xffffffffu, mag, o));
        float sc, inv;
        qf_scales(mag, &sc, &inv);
        uint32_t out[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          out[j] = qf_code2(f[4 * j] * inv, f[4 * j + 1] * inv) | qf_code2(f[4 * j + 2] * inv, f[4 * j + 3] * inv) << 16;
        if (r0 + i < rows && c < n)
          __stcs(reinterpret_cast<uint4*>(q + (long long)(r0 + i) * n + c), make_uint4(out[0], out[1], out[2], out[3]));
        if ((lane & 7) == 0) scales[lane >> 3][warp * kQfPerWarp + i] = sc;
      }
    } else {
      for (int i = 0; i < kQfPerWarp; ++i) {
        const long long r = r0 + i;
#pragma unroll
        for (int gr = 0; gr < kQfCols / 128; ++gr) {
          float f[4];
          uint32_t mag = 0;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int c = c0 + 128 * gr + 32 * j + lane;
            f[j] = r < rows && c < n ? qf_value(x[r * ld + c], TYPE) : 0.f;
            mag = max(mag, qf_mag(f[j]));
          }
          mag = __reduce_max_sync(0xffffffffu, mag);
          float sc, inv;
          qf_scales(mag, &sc, &inv);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int c = c0 + 128 * gr + 32 * j + lane;
            if (r < rows && c < n) q[r * n + c] = (uint8_t)(qf_code2(f[j] * inv, 0.f) & 0xFFu);
          }
          if (lane == 0) scales[gr][warp * kQfPerWarp + i] = sc;
        }
      }
    }
    __syncthreads();
    if (threadIdx.x < kQfRows * (kQfCols / 128)) {
      const int gr = threadIdx.x / kQfRows, i = threadIdx.x % kQfRows;
      const long long r = b * kQfRows + i;
      const int grp = (c0 >> 7) + gr;
      if (r < rows && grp < groups) s[(long long)grp * rows + r] = scales[gr][i];
    }
    __syncthreads();
  }
}

}  // namespace moe
