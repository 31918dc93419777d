// What the grouped products share: their parameters.
//
// Rows are in expert order, expert e owning rows [off[e], off[e+1]):
//   mm   y[r, o]     = sum_i W[e, o, i] x[r, i]
//   dx   dx[r, i]    = sum_o W[e, o, i] dy[r, o]
//   dw   dW[e, o, i] = sum_{r of e} dy[r, o] x[r, i]
// Each is a set of matrix products, one per expert, of an M side and an N
// side.  The M side is the output's contiguous dimension (o, i, i), the N side
// its rows (r, r, o), so that one epilogue serves all three and an expert with
// few rows costs a narrow N instead of a padded M.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace moe {

enum GmmOp : int { G_MM = 0, G_DX = 1, G_DW = 2 };
enum GmmType : int { G_BF16 = 0, G_FP16 = 1, G_FP32 = 2, G_E4M3 = 3 };

constexpr int kGmmMaxExperts = 1024;

struct GmmProblem {
  const void* w;         // [E, n_out, n_in] (mm, dx)
  const void* rows_in;   // mm: x [rows, n_in]; dx: dy [rows, n_out]; dw: dy
  const void* x;         // dw: x [rows, n_in]
  long long ld_rows, ld_x;  // elements
  const int* off;        // [E + 1] or NULL: one matrix, every row
  void* out;             // mm: y; dx: dx; dw: dW [E, n_out, n_in]
  long long ld_out;      // elements between output rows (mm, dx)
  const float* sx;       // 8-bit product: row scales [groups][rows]
  const float* sw;       // 8-bit product: weight scales [E][n_out / 128][groups]
  int out_type;          // GmmType
  int E, rows, n_out, n_in;
  int* err;
};

MOE_DEV int gmm_off(const GmmProblem& p, int e) { return p.off ? __ldg(p.off + e) : (e == 0 ? 0 : p.rows); }

MOE_DEV void gmm_store(void* out, int type, long long i, float v) {
  if (type == G_BF16) reinterpret_cast<__nv_bfloat16*>(out)[i] = __float2bfloat16_rn(v);
  else if (type == G_FP16) reinterpret_cast<__half*>(out)[i] = __float2half_rn(v);
  else reinterpret_cast<float*>(out)[i] = v;
}

}  // namespace moe
