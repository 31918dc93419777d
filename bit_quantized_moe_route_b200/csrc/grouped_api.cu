// Host side of the grouped products and of the 8-bit row quantiser declared in
// include/moe_lowbit.h: argument validation and kernel launches.
#include <cuda_runtime.h>

#include <algorithm>

#include "api_util.h"
#include "device_cache.h"
#include "grouped_umma.cuh"
#include "quant_fp8.cuh"

using namespace moe;

namespace {

constexpr size_t kGmmWsBytes = kGuWsBytes;

#define GMM_TRY(call)                    \
  do {                                   \
    const moe_status_t st_ = (call);     \
    if (st_ != MOE_OK) return st_;       \
  } while (0)

int sm_count(int* sms) {
  static DeviceCache cached;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 1;
  *sms = cached.get(dev, [dev] {
    int v = 0;
    return cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess ? v : 0;
  });
  return *sms < 1;
}

size_t type_bytes(int t) { return t == G_FP32 ? 4 : t == G_E4M3 ? 1 : 2; }

// Rows of `width` bytes, `pitch` bytes apart.
struct Span {
  const char* name;
  const void* p;
  size_t bytes;  // from the first row's first byte to the last row's last
  size_t pitch, width;
};
Span rows_span(const char* name, const void* p, long long rows, long long ld, long long n, int type) {
  const size_t es = type_bytes(type);
  return {name, p, rows > 0 ? ((size_t)(rows - 1) * ld + n) * es : 0, (size_t)ld * es, (size_t)n * es};
}
Span flat_span(const char* name, const void* p, size_t bytes) { return {name, p, bytes, bytes, bytes}; }

moe_status_t check_apart(const Span& out, const Span* in, int n) {
  const uintptr_t a = (uintptr_t)out.p, b = a + out.bytes;
  for (int i = 0; i < n; ++i) {
    const uintptr_t c = (uintptr_t)in[i].p, d = c + in[i].bytes;
    if (!in[i].p || !out.bytes || !in[i].bytes || b <= c || d <= a) continue;
    // column ranges of one buffer: the same pitch, and neither row reaches into the other
    if (out.pitch == in[i].pitch && out.width < out.pitch && in[i].width < out.pitch) {
      const size_t delta = c >= a ? (c - a) % out.pitch : (out.pitch - (a - c) % out.pitch) % out.pitch;
      if (delta >= out.width && delta + in[i].width <= out.pitch) continue;
    }
    return api_fail(MOE_ERR_INVALID_ARG, "%s overlaps %s", out.name, in[i].name);
  }
  return MOE_OK;
}

moe_status_t check_aligned(const Span& s, size_t unit) {
  if ((uintptr_t)s.p % unit) return api_fail(MOE_ERR_INVALID_ARG, "%s is not aligned to its elements", s.name);
  return MOE_OK;
}

moe_status_t check_gmm_dims(const moe_gmm_dims_t* d, bool fp8, bool have_offsets) {
  if (!d) return api_fail(MOE_ERR_INVALID_ARG, "dims is NULL");
  if (!fp8 && d->dtype != MOE_BF16 && d->dtype != MOE_FP16)
    return api_fail(MOE_ERR_UNSUPPORTED, "dtype=%d not in {0 (bf16), 1 (fp16)}", d->dtype);
  if (d->out_dtype != MOE_BF16 && d->out_dtype != MOE_FP16 && d->out_dtype != MOE_FP32)
    return api_fail(MOE_ERR_UNSUPPORTED, "out_dtype=%d not in {0 (bf16), 1 (fp16), 2 (fp32)}", d->out_dtype);
  if (!fp8 && d->out_dtype != MOE_FP32 && d->out_dtype != d->dtype)
    return api_fail(MOE_ERR_UNSUPPORTED, "out_dtype must be dtype or fp32");
  if (d->n_experts < 1 || d->n_experts > kGmmMaxExperts)
    return api_fail(MOE_ERR_INVALID_ARG, "n_experts=%d outside [1, %d]", d->n_experts, kGmmMaxExperts);
  if (!have_offsets && d->n_experts != 1)
    return api_fail(MOE_ERR_INVALID_ARG, "expert_offsets is NULL with n_experts=%d", d->n_experts);
  if (d->n_out < 1 || d->n_out > 65536 || d->n_in < 1 || d->n_in > 65536)
    return api_fail(MOE_ERR_INVALID_ARG, "n_out=%d or n_in=%d outside [1, 65536]", d->n_out, d->n_in);
  if (d->rows < 0 || d->rows > (1 << 30)) return api_fail(MOE_ERR_INVALID_ARG, "rows=%d outside [0, 2^30]", d->rows);
  if (d->reserved) return api_fail(MOE_ERR_INVALID_ARG, "reserved must be 0");
  return MOE_OK;
}

moe_status_t check_ld(long long ld, int n, const char* name) {
  if (ld < n || ld > (1LL << 31))
    return api_fail(MOE_ERR_INVALID_ARG, "%s=%lld outside [%d, 2^31]", name, ld, n);
  return MOE_OK;
}

moe_status_t check_gmm_ws(void* ws, size_t ws_bytes) {
  if (!ws) return api_fail(MOE_ERR_INVALID_ARG, "workspace is NULL");
  if ((uintptr_t)ws % 256) return api_fail(MOE_ERR_INVALID_ARG, "workspace is not 256-byte aligned");
  if (ws_bytes < kGmmWsBytes)
    return api_fail(MOE_ERR_WORKSPACE, "workspace has %zu bytes, %zu needed", ws_bytes, kGmmWsBytes);
  return api_check_dev_ptr(ws, "workspace");
}

// Resident pairs of a tensor-memory kernel on the current device, or a GuNoPairs.
template <int OP, bool FP8, bool ROWM, int MT, int CHAIN, bool ANY>
int resident_pairs() {
  static DeviceCache cached;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return GU_QUERY_FAILED;
  return cached.get(dev, gu_pairs<OP, FP8, ROWM, MT, CHAIN, ANY>);
}

bool aligned16(const void* p) { return (uintptr_t)p % 16 == 0; }

// TMA's rules: base addresses and row strides in multiples of 16 bytes.
template <int OP>
bool tma_ok(const GmmProblem& p, int es) {
  if (p.rows < 1 || !aligned16(p.rows_in) || p.ld_rows * es % 16) return false;
  return OP == G_DW ? aligned16(p.x) && p.ld_x * es % 16 == 0 : aligned16(p.w) && (long long)p.n_in * es % 16 == 0;
}

// The 8-bit product has its rows on the M side from this mean per expert on.  On
// the N side / M side, us, 32 experts of 4096 -> 2048: 64 rows each 65 / 87, 128
// 85 / 90, 160 (two tiles on the N side) 137 / 90, 384 215 / 149; 64 experts of
// 1024 -> 1024: 64 rows 23 / 32, 128 32 / 37, 160 46 / 38, 384 68 / 60.  Rows are
// seldom even: above the 160 at which even ones cross.
constexpr long long kRowsPerExpertM = 192;

template <int OP, bool FP8, bool ROWM, int MT, int CHAIN, bool ANY>
moe_status_t launch_umma(const GmmProblem& p, int type, void* ws, cudaStream_t s) {
  const int pairs = resident_pairs<OP, FP8, ROWM, MT, CHAIN, ANY>();
  if (pairs == GU_QUERY_FAILED)
    return api_fail(MOE_ERR_CUDA, "grouped_umma_kernel: %s", cudaGetErrorString(cudaGetLastError()));
  if (pairs == GU_REGISTERS)
    return api_fail(MOE_ERR_CUDA, "the grouped kernel was not compiled to the registers that its warps share out");
  if (pairs < 1) return api_fail(MOE_ERR_CUDA, "the grouped kernel does not fit this device");
  GuKernelParams<FP8, ANY> q;
  q.g = p;
  q.type = type;
  q.ws = reinterpret_cast<unsigned char*>(ws);
  q.split_most = 16;
  const uint64_t es = FP8 ? 1 : 2;
  const CUtensorMapDataType dt = FP8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                     : type == G_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  if constexpr (ANY) {
    constexpr int R = GuAnyParams<FP8>::R;
    // (a class that has no rows, as any without rows at all, is one value that may be read and is not used)
    auto classes = [&](CUtensorMap* maps, const void* ptr, long long rows, int cols, long long ld, uint32_t block,
                       uint32_t box_rows) -> moe_status_t {
      if (rows < 1) ptr = ws;
      for (int c = 0; c < R; ++c) {
        const bool any = c < rows;
        const uintptr_t at = (uintptr_t)ptr + (any ? c * ld * es : 0);
        const uint64_t before = (at & 15) / es;
        const uint64_t dims[2] = {before + (any ? cols : 1), any ? (uint64_t)((rows - c + R - 1) / R) : 1u};
        const uint64_t st[1] = {(uint64_t)ld * es * R};
        const uint32_t box[2] = {block / (uint32_t)es, box_rows / R};
        GMM_TRY(api_tensor_map(&maps[c], dt, 2, (const void*)(at & ~(uintptr_t)15), dims, st, box, false));
      }
      return MOE_OK;
    };
    if constexpr (OP == G_DW) {
      GMM_TRY(classes(q.a_rows, p.rows_in, p.rows, p.n_out, p.ld_rows, 272, 64));
      GMM_TRY(classes(q.b_rows, p.x, p.rows, p.n_in, p.ld_x, 272, 64));
    } else {
      const int cols = OP == G_MM ? p.n_in : p.n_out;
      const bool mn = OP == G_DX;
      GMM_TRY(classes(q.a_rows, p.w, (long long)p.E * p.n_out, p.n_in, p.n_in, mn ? 272 : 144, mn ? 64 : 128));
      if (p.rows > 64) GMM_TRY(classes(q.b_rows, p.rows_in, p.rows, cols, p.ld_rows, 144, 128));
      GMM_TRY(classes(q.b_few, p.rows_in, p.rows, cols, p.ld_rows, 144, 32));
    }
  } else {
    const uint32_t inner = 128 / es;
    if constexpr (OP == G_DW) {
      const uint64_t dims_x[2] = {(uint64_t)p.n_in, (uint64_t)p.rows}, st_x[1] = {(uint64_t)p.ld_x * es};
      const uint64_t dims_y[2] = {(uint64_t)p.n_out, (uint64_t)p.rows}, st_y[1] = {(uint64_t)p.ld_rows * es};
      for (int i = 0; i < 7; ++i) {
        const uint32_t box[2] = {inner, 64u >> i};
        GMM_TRY(api_tensor_map(i ? &q.a_tail[i - 1] : &q.a_map, dt, 2, p.rows_in, dims_y, st_y, box));
        GMM_TRY(api_tensor_map(i ? &q.b_tail[i - 1] : &q.b_map[0], dt, 2, p.x, dims_x, st_x, box));
      }
    } else {
      const uint64_t dims_w[3] = {(uint64_t)p.n_in, (uint64_t)p.n_out, (uint64_t)p.E};
      const uint64_t st_w[2] = {(uint64_t)p.n_in * es, (uint64_t)p.n_in * p.n_out * es};
      const uint32_t box_w[3] = {inner, OP == G_MM ? 128u : 64u, 1u};
      GMM_TRY(api_tensor_map(ROWM ? &q.b_map[0] : &q.a_map, dt, 3, p.w, dims_w, st_w, box_w));
      const uint64_t dims_r[2] = {(uint64_t)(OP == G_MM ? p.n_in : p.n_out), (uint64_t)p.rows};
      const uint64_t st_r[1] = {(uint64_t)p.ld_rows * es};
      // no tile has more rows than there are: boxes beyond the first that holds half of them are not used
      for (int i = ROWM ? 3 : 0; i < 4 && (ROWM || i == 0 || p.rows > (32 << (i - 1))); ++i) {
        const uint32_t box[2] = {inner, 16u << i};
        GMM_TRY(api_tensor_map(ROWM ? &q.a_map : &q.b_map[i], dt, 2, p.rows_in, dims_r, st_r, box));
      }
    }
  }
  if (!gu_launch<OP, FP8, ROWM, MT, CHAIN, ANY>(q, pairs, s))
    return api_fail(MOE_ERR_CUDA, "grouped_umma_kernel: %s", cudaGetErrorString(cudaGetLastError()));
  return MOE_OK;
}

// 512-value tiles where there are two or more for each pair of SMs (from the
// host's side: as if every expert had rows).  256 / 512 values, us, calls in a
// loop: 32,768 rows over 256 experts of 4096 -> 2048: mm 845 / 840, dx 866 / 828,
// dw 1,943 / 1,665; over 32: 447 / 458, 455 / 454, 529 / 492; 128 tiles: mm of 8,192
// rows over 8 117 / 133, dw of 16,384 over 4 of 1024 -> 4096 157 / 173.
template <int OP>
bool many_tiles(const GmmProblem& p) {
  const long long m = ((OP == G_DX ? p.n_in : p.n_out) + 511) / 512;
  const long long n = OP == G_DW ? (long long)p.E * ((p.n_in + kGuN - 1) / kGuN)
                                 : std::max<long long>(p.rows / kGuN, std::min(p.E, p.rows));
  return m * n >= 2 * kGuPairsMax;
}

template <int OP>
moe_status_t run_gmm(const GmmProblem& p, int in_type, void* ws, cudaStream_t s) {
  constexpr bool ROWM = OP == G_DW;
  const bool fp8 = in_type == G_E4M3;
  if (!tma_ok<OP>(p, fp8 ? 1 : 2)) {
    if constexpr (OP == G_MM)
      if (fp8) return launch_umma<OP, true, false, 1, 1, true>(p, in_type, ws, s);
    return p.out_type == G_FP32 ? launch_umma<OP, false, ROWM, 1, kGuChain, true>(p, in_type, ws, s)
                                : launch_umma<OP, false, ROWM, 1, 0, true>(p, in_type, ws, s);
  }
  if constexpr (OP == G_MM)
    if (fp8)
      return (long long)p.rows >= kRowsPerExpertM * p.E ? launch_umma<OP, true, true, 1, 1, false>(p, in_type, ws, s)
                                                        : launch_umma<OP, true, false, 1, 1, false>(p, in_type, ws, s);
  if (p.out_type == G_FP32) return launch_umma<OP, false, ROWM, 1, kGuChain, false>(p, in_type, ws, s);
  return many_tiles<OP>(p) ? launch_umma<OP, false, ROWM, 2, 0, false>(p, in_type, ws, s)
                           : launch_umma<OP, false, ROWM, 1, 0, false>(p, in_type, ws, s);
}

// The products over rows: mm (rows_in = x) and dx (rows_in = dy).
template <int OP>
moe_status_t rows_product(const moe_gmm_dims_t* d, const char* in_name, const void* in, int64_t ld_in, const void* w,
                          const int32_t* off, const char* out_name, void* out, int64_t ld_out, const float* sx,
                          const float* sw, bool fp8, void* ws, size_t ws_bytes, void* stream) {
  api_clear_detail();
  GMM_TRY(check_gmm_dims(d, fp8, off != nullptr));
  const int in_cols = OP == G_MM ? d->n_in : d->n_out, out_cols = OP == G_MM ? d->n_out : d->n_in;
  GMM_TRY(check_ld(ld_in, in_cols, OP == G_MM ? "ld_x" : "ld_dy"));
  GMM_TRY(check_ld(ld_out, out_cols, OP == G_MM ? "ld_y" : "ld_dx"));
  if (d->rows == 0) return MOE_OK;
  const int type = fp8 ? G_E4M3 : d->dtype;
  const long long groups = (d->n_in + 127) / 128;
  const Span ins[5] = {
      rows_span(in_name, in, d->rows, ld_in, in_cols, type),
      rows_span("w", w, (long long)d->n_experts * d->n_out, d->n_in, d->n_in, type),
      flat_span("expert_offsets", off, off ? sizeof(int) * (size_t)(d->n_experts + 1) : 0),
      flat_span("x_scales", sx, fp8 ? sizeof(float) * (size_t)(groups * d->rows) : 0),
      flat_span("w_scales", sw, fp8 ? sizeof(float) * (size_t)(groups * d->n_experts * ((d->n_out + 127) / 128)) : 0)};
  const Span o = rows_span(out_name, out, d->rows, ld_out, out_cols, d->out_dtype);
  GMM_TRY(check_gmm_ws(ws, ws_bytes));
  for (const Span& s : ins)
    if (s.p || s.bytes) GMM_TRY(api_check_dev_ptr(s.p, s.name));
  GMM_TRY(api_check_dev_ptr(out, out_name));
  GMM_TRY(check_aligned(ins[0], type_bytes(type)));
  GMM_TRY(check_aligned(ins[1], type_bytes(type)));
  GMM_TRY(check_aligned(ins[2], 4));
  GMM_TRY(check_aligned(ins[3], 4));
  GMM_TRY(check_aligned(ins[4], 4));
  GMM_TRY(check_aligned(o, type_bytes(d->out_dtype)));
  GMM_TRY(check_apart(o, ins, 5));
  const Span wsp = flat_span("ws", ws, kGmmWsBytes);
  GMM_TRY(check_apart(o, &wsp, 1));
  GMM_TRY(check_apart(wsp, ins, 5));
  GmmProblem p{};
  p.w = w;
  p.rows_in = in;
  p.ld_rows = ld_in;
  p.off = off;
  p.out = out;
  p.ld_out = ld_out;
  p.sx = sx;
  p.sw = sw;
  p.out_type = d->out_dtype;
  p.E = d->n_experts;
  p.rows = d->rows;
  p.n_out = d->n_out;
  p.n_in = d->n_in;
  p.err = reinterpret_cast<int*>(ws);
  return run_gmm<OP>(p, type, ws, reinterpret_cast<cudaStream_t>(stream));
}

}  // namespace

extern "C" {

size_t moe_grouped_workspace_size(void) { return kGmmWsBytes; }

moe_status_t moe_grouped_mm(const moe_gmm_dims_t* dims, const void* x, int64_t ld_x, const void* w,
                            const int32_t* expert_offsets, void* y, int64_t ld_y, void* ws, size_t ws_bytes,
                            void* stream) {
  return rows_product<G_MM>(dims, "x", x, ld_x, w, expert_offsets, "y", y, ld_y, nullptr, nullptr, false, ws, ws_bytes,
                            stream);
}

moe_status_t moe_grouped_mm_dx(const moe_gmm_dims_t* dims, const void* dy, int64_t ld_dy, const void* w,
                               const int32_t* expert_offsets, void* dx, int64_t ld_dx, void* ws, size_t ws_bytes,
                               void* stream) {
  return rows_product<G_DX>(dims, "dy", dy, ld_dy, w, expert_offsets, "dx", dx, ld_dx, nullptr, nullptr, false, ws,
                            ws_bytes, stream);
}

moe_status_t moe_grouped_mm_dw(const moe_gmm_dims_t* dims, const void* dy, int64_t ld_dy, const void* x, int64_t ld_x,
                               const int32_t* expert_offsets, void* dw, void* ws, size_t ws_bytes, void* stream) {
  api_clear_detail();
  GMM_TRY(check_gmm_dims(dims, false, expert_offsets != nullptr));
  const moe_gmm_dims_t& d = *dims;
  GMM_TRY(check_ld(ld_dy, d.n_out, "ld_dy"));
  GMM_TRY(check_ld(ld_x, d.n_in, "ld_x"));
  const Span ins[3] = {
      rows_span("dy", dy, d.rows, ld_dy, d.n_out, d.dtype), rows_span("x", x, d.rows, ld_x, d.n_in, d.dtype),
      flat_span("expert_offsets", expert_offsets, expert_offsets ? sizeof(int) * (size_t)(d.n_experts + 1) : 0)};
  const Span o = rows_span("dw", dw, (long long)d.n_experts * d.n_out, d.n_in, d.n_in, d.out_dtype);
  GMM_TRY(check_gmm_ws(ws, ws_bytes));
  for (const Span& s : ins)
    if (s.bytes) GMM_TRY(api_check_dev_ptr(s.p, s.name));
  GMM_TRY(api_check_dev_ptr(dw, "dw"));
  GMM_TRY(check_aligned(ins[0], 2));
  GMM_TRY(check_aligned(ins[1], 2));
  GMM_TRY(check_aligned(ins[2], 4));
  GMM_TRY(check_aligned(o, type_bytes(d.out_dtype)));
  GMM_TRY(check_apart(o, ins, 3));
  const Span wsp = flat_span("ws", ws, kGmmWsBytes);
  GMM_TRY(check_apart(o, &wsp, 1));
  GMM_TRY(check_apart(wsp, ins, 3));
  GmmProblem p{};
  p.rows_in = dy;
  p.x = x;
  p.ld_rows = ld_dy;
  p.ld_x = ld_x;
  p.off = expert_offsets;
  p.out = dw;
  p.out_type = d.out_dtype;
  p.E = d.n_experts;
  p.rows = d.rows;
  p.n_out = d.n_out;
  p.n_in = d.n_in;
  p.err = reinterpret_cast<int*>(ws);
  return run_gmm<G_DW>(p, d.dtype, ws, reinterpret_cast<cudaStream_t>(stream));
}

moe_status_t moe_grouped_mm_fp8(const moe_gmm_dims_t* dims, const void* x, int64_t ld_x, const float* x_scales,
                                const void* w, const float* w_scales, const int32_t* expert_offsets, void* y,
                                int64_t ld_y, void* ws, size_t ws_bytes, void* stream) {
  return rows_product<G_MM>(dims, "x", x, ld_x, w, expert_offsets, "y", y, ld_y, x_scales, w_scales, true, ws, ws_bytes,
                            stream);
}

moe_status_t moe_quant_fp8(int32_t dtype, int32_t rows, int32_t n_in, const void* x, int64_t ld_x, void* codes,
                           float* scales, void* stream) {
  api_clear_detail();
  if (dtype != MOE_BF16 && dtype != MOE_FP16)
    return api_fail(MOE_ERR_UNSUPPORTED, "dtype=%d not in {0 (bf16), 1 (fp16)}", dtype);
  if (n_in < 1 || n_in > 65536) return api_fail(MOE_ERR_INVALID_ARG, "n_in=%d outside [1, 65536]", n_in);
  if (rows < 0 || rows > (1 << 30)) return api_fail(MOE_ERR_INVALID_ARG, "rows=%d outside [0, 2^30]", rows);
  GMM_TRY(check_ld(ld_x, n_in, "ld_x"));
  if (rows == 0) return MOE_OK;
  const Span in = rows_span("x", x, rows, ld_x, n_in, dtype);
  const Span o1 = flat_span("codes", codes, (size_t)rows * n_in);
  const Span o2 = flat_span("scales", scales, (size_t)rows * ((n_in + 127) / 128) * 4);
  GMM_TRY(api_check_dev_ptr(x, "x"));
  GMM_TRY(api_check_dev_ptr(codes, "codes"));
  GMM_TRY(api_check_dev_ptr(scales, "scales"));
  GMM_TRY(check_aligned(in, 2));
  GMM_TRY(check_aligned(o2, 4));
  GMM_TRY(check_apart(o1, &in, 1));
  GMM_TRY(check_apart(o2, &in, 1));
  GMM_TRY(check_apart(o1, &o2, 1));
  int sms = 0;
  if (sm_count(&sms)) return api_fail(MOE_ERR_CUDA, "device query failed");
  const bool vec = n_in % 16 == 0 && ld_x % 8 == 0 && (uintptr_t)x % 16 == 0 && (uintptr_t)codes % 16 == 0;
  const int gy = (n_in + kQfCols - 1) / kQfCols;
  const dim3 grid((unsigned)std::min((rows + kQfRows - 1) / kQfRows, std::max(1, sms * 64 / gy)), (unsigned)gy);
  const uint16_t* xp = reinterpret_cast<const uint16_t*>(x);
  uint8_t* q = reinterpret_cast<uint8_t*>(codes);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == MOE_BF16) {
    if (vec) quant_fp8_kernel<G_BF16, true><<<grid, kQfThreads, 0, s>>>(xp, ld_x, rows, n_in, q, scales);
    else quant_fp8_kernel<G_BF16, false><<<grid, kQfThreads, 0, s>>>(xp, ld_x, rows, n_in, q, scales);
  } else {
    if (vec) quant_fp8_kernel<G_FP16, true><<<grid, kQfThreads, 0, s>>>(xp, ld_x, rows, n_in, q, scales);
    else quant_fp8_kernel<G_FP16, false><<<grid, kQfThreads, 0, s>>>(xp, ld_x, rows, n_in, q, scales);
  }
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return api_fail(MOE_ERR_CUDA, "quant_fp8_kernel: %s", cudaGetErrorString(e));
  return MOE_OK;
}

}  // extern "C"
