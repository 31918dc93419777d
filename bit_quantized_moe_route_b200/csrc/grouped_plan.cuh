// What the grouped products share: their parameters and the walk over the
// experts' row ranges.
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

// Called by every thread of the block: cum[e] = work units of the experts
// before e, for units(rows of the expert) units each, and cum[E] the total.
// The offsets are the caller's, so they are checked here, before any of them
// is used as an index: 0 <= off[0] <= ... <= off[E] <= rows.  Returns false
// (in every thread, with the error recorded) when they are not.
template <typename Units>
MOE_DEV bool gmm_plan(const GmmProblem& p, Units units, long long* cum, int* flag) {
  if (threadIdx.x == 0) *flag = 1;
  __syncthreads();
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    long long base = 0;
    bool ok = true;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      const int e = e0 + lane;
      long long u = 0;
      if (e < p.E) {
        const int a = gmm_off(p, e), b = gmm_off(p, e + 1);
        if (a < 0 || b < a || b > p.rows) ok = false;
        else u = units(b - a);
      }
      long long s = u;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += v;
      }
      if (e < p.E) cum[e] = base + s - u;
      base += __shfl_sync(0xffffffffu, s, 31);
    }
    if (lane == 0) cum[p.E] = base;
    if (!ok) *flag = 0;
  }
  __syncthreads();
  if (!*flag && threadIdx.x == 0) set_error(p.err, kErrDeviceInput);
  return *flag != 0;
}

// The expert whose units hold unit u (0 <= u < cum[E]).
MOE_DEV int gmm_expert_of(const long long* cum, int E, long long u) {
  int lo = 0, hi = E;  // cum[lo] <= u < cum[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cum[mid] <= u) lo = mid;
    else hi = mid;
  }
  return lo;
}

}  // namespace moe
