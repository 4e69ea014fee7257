// C ABI front end: argument validation on the host, then kernel dispatch.
// Every check runs before any HIP call, so a rejected call touches no
// device state (and can be exercised on a machine without a GPU).
#include <math.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#include "../../include/nvfp4_w4a4.h"
#include "internal.h"

namespace {

bool aligned(const void* p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) % a) == 0;
}

// [lo, lo + len) and [lo2, lo2 + len2) intersect (byte ranges).
bool overlap(const void* a, int64_t alen, const void* b, int64_t blen) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a);
  const uintptr_t y = reinterpret_cast<uintptr_t>(b);
  return x < y + static_cast<uintptr_t>(blen) &&
         y < x + static_cast<uintptr_t>(alen);
}

// Sizes whose byte extents stay far below 2^62.
constexpr int64_t kMaxDim = int64_t(1) << 40;

int status_of(hipError_t e) {
  return e == hipSuccess ? NVFP4_OK : NVFP4_ERR_LAUNCH;
}

// Shared checks of a [rows][k] input tensor x (k % 16 == 0, ldx >= k,
// 16-byte aligned rows).  Returns NVFP4_OK or the status to report.
int check_x(const void* x, int x_dtype, int64_t rows, int64_t k, int64_t ldx) {
  if (!x) return NVFP4_ERR_INVALID_VALUE;
  if (rows < 1 || k < 16 || k % 16 != 0 || ldx < k) return NVFP4_ERR_INVALID_VALUE;
  if (rows > kMaxDim || ldx > kMaxDim || rows > kMaxDim / ldx)
    return NVFP4_ERR_INVALID_VALUE;
  if (rows * (k / 16) > (int64_t(1) << 39)) return NVFP4_ERR_INVALID_VALUE;
  if (x_dtype != NVFP4_DTYPE_F32 && x_dtype != NVFP4_DTYPE_BF16)
    return NVFP4_ERR_UNSUPPORTED;
  const int64_t es = x_dtype == NVFP4_DTYPE_F32 ? 4 : 2;
  if (!aligned(x, 16) || (ldx * es) % 16 != 0) return NVFP4_ERR_MISALIGNED;
  return NVFP4_OK;
}

// Extent in bytes of [token][head][d] rows.
int64_t rows_bytes(int64_t tokens, int64_t ts, int64_t heads, int64_t hs, int64_t d, int64_t es) {
  return tokens < 1 ? 0 : ((tokens - 1) * ts + (heads - 1) * hs + d) * es;
}

// [token][head][d] rows of a caller's tensor: strides that keep rows apart,
// `align` bytes of alignment.
int check_rows(const void* p, int64_t tokens, int64_t ts, int64_t heads, int64_t hs, int64_t d,
               int64_t es, int64_t align) {
  if (!p) return NVFP4_ERR_INVALID_VALUE;
  if (ts < d || hs < d || ts > kMaxDim || hs > kMaxDim || tokens > kMaxDim / ts ||
      heads > kMaxDim / hs)
    return NVFP4_ERR_INVALID_VALUE;
  if (!aligned(p, align) || (ts * es) % align != 0 || (hs * es) % align != 0)
    return NVFP4_ERR_MISALIGNED;
  return NVFP4_OK;
}

// A paged cache as kv_page_write and kv_paged_attention take it.
int check_pool(const nvfp4::KvPool& p, int dtype) {
  if (!p.k || !p.v) return NVFP4_ERR_INVALID_VALUE;
  if (p.n_pages < 1 || p.page_size < 1 || p.n_heads < 1 || p.d < 16 || p.n_pages > 0x7FFFFFFF ||
      p.page_size > (1 << 24) || p.n_heads > (1 << 16))
    return NVFP4_ERR_INVALID_VALUE;
  if (dtype != NVFP4_DTYPE_BF16 && dtype != NVFP4_DTYPE_E4M3) return NVFP4_ERR_UNSUPPORTED;
  if (p.page_size % 16 != 0) return NVFP4_ERR_UNSUPPORTED;
  if (p.page_stride < p.d || p.head_stride < p.d || p.token_stride < p.d ||
      p.page_stride > kMaxDim || p.head_stride > kMaxDim || p.token_stride > kMaxDim ||
      p.n_pages > kMaxDim / p.page_stride || p.n_heads > kMaxDim / p.head_stride ||
      p.page_size > kMaxDim / p.token_stride)
    return NVFP4_ERR_INVALID_VALUE;
  if (p.fp8 && (!p.k_scale || !p.v_scale)) return NVFP4_ERR_INVALID_VALUE;
  const int64_t es = p.fp8 ? 1 : 2;
  if (!aligned(p.k, 16) || !aligned(p.v, 16) || (p.page_stride * es) % 16 != 0 ||
      (p.head_stride * es) % 16 != 0 || (p.token_stride * es) % 16 != 0 ||
      (p.fp8 && (!aligned(p.k_scale, 4) || !aligned(p.v_scale, 4))))
    return NVFP4_ERR_MISALIGNED;
  return NVFP4_OK;
}

int64_t pool_bytes(const nvfp4::KvPool& p) {
  return ((p.n_pages - 1) * p.page_stride + (p.n_heads - 1) * p.head_stride +
          (p.page_size - 1) * p.token_stride + p.d) * (p.fp8 ? 1 : 2);
}

// Sizes and options that both attention calls share.
int check_attention(const nvfp4::AttnCall& c) {
  constexpr int64_t kInt = 0x7FFFFFFF;
  if (c.n_tokens < 0 || c.n_heads < 1 || c.n_kv_heads < 1 || c.n_heads % c.n_kv_heads != 0 ||
      c.n_heads > (1 << 16) || c.n_requests < 1 || c.n_requests > (1 << 24) || c.max_new < 0 ||
      c.max_kv < 0 || c.max_kv > kInt - 65536 || c.max_new > kInt - 65536 || c.window < 0 ||
      c.window > kInt - 65536)
    return NVFP4_ERR_INVALID_VALUE;
  // a launch has fewer than 2^32 threads: 64 a row to join, 256 a tile
  if (c.n_tokens > (int64_t(1) << 25) / c.n_heads ||
      c.n_requests > (int64_t(1) << 20) / c.n_kv_heads)
    return NVFP4_ERR_INVALID_VALUE;
  if (!(c.scale > 0.0f) || isinf(c.scale)) return NVFP4_ERR_INVALID_VALUE;
  if (c.d != 64 && c.d != 128 && c.d != 256) return NVFP4_ERR_UNSUPPORTED;
  return NVFP4_OK;
}

// Workspace and output of an attention call, then the launch.
int run_attention(const nvfp4::AttnCall& c, int64_t workspace_bytes, void* stream) {
  const int64_t need = nvfp4::attention_workspace(c);
  if (need < 0 || workspace_bytes < need || (need > 0 && !c.workspace))
    return NVFP4_ERR_INVALID_VALUE;
  if (need > 0 && !aligned(c.workspace, 16)) return NVFP4_ERR_MISALIGNED;
  const int64_t obytes = rows_bytes(c.n_tokens, c.out_token, c.n_heads, c.out_head, c.d, 2);
  const bool paged = c.table != nullptr;
  struct Range { const void* p; int64_t len; };
  const Range in[] = {
      {c.q.p, rows_bytes(c.n_tokens, c.q.token, c.n_heads, c.q.head, c.d, 2)},
      {paged ? c.pool.k : c.k.p, paged ? pool_bytes(c.pool) : rows_bytes(c.n_tokens, c.k.token, c.n_kv_heads, c.k.head, c.d, 2)},
      {paged ? c.pool.v : c.v.p, paged ? pool_bytes(c.pool) : rows_bytes(c.n_tokens, c.v.token, c.n_kv_heads, c.v.head, c.d, 2)},
      {c.cu, 4 * (c.n_requests + 1)},
      {c.kv_lens, paged ? 4 * c.n_requests : 0},
      {c.table, paged ? ((c.n_requests - 1) * c.ld_table + c.cols) * 4 : 0}};
  for (const Range& r : in) {
    if (r.len < 1) continue;
    if (overlap(c.out, obytes, r.p, r.len)) return NVFP4_ERR_INVALID_VALUE;
    if (need > 0 && overlap(c.workspace, need, r.p, r.len)) return NVFP4_ERR_INVALID_VALUE;
  }
  if (need > 0 && overlap(c.workspace, need, c.out, obytes)) return NVFP4_ERR_INVALID_VALUE;
  return status_of(nvfp4::launch_attention(c, static_cast<hipStream_t>(stream)));
}

// Codes and scales of an MXFP4 tensor [rows][k].
int check_mxfp4(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t k) {
  if (!codes || !scales) return NVFP4_ERR_INVALID_VALUE;
  if (rows < 1 || k < 32 || k % 32 != 0 || k > kMaxDim || rows > kMaxDim / k)
    return NVFP4_ERR_INVALID_VALUE;
  return NVFP4_OK;
}

// A dense [rows][ld] tensor of F32 or BF16 with 16-byte aligned rows.
int check_dense(const void* p, int dtype, int64_t rows, int64_t k, int64_t ld) {
  if (!p || ld < k || ld > kMaxDim || rows > kMaxDim / ld) return NVFP4_ERR_INVALID_VALUE;
  if (dtype != NVFP4_DTYPE_F32 && dtype != NVFP4_DTYPE_BF16) return NVFP4_ERR_UNSUPPORTED;
  if (!aligned(p, 16) || (ld * (dtype == NVFP4_DTYPE_F32 ? 4 : 2)) % 16 != 0)
    return NVFP4_ERR_MISALIGNED;
  return NVFP4_OK;
}

// Sizes of a gdn_attention call.
int check_gdn(const nvfp4::GdnCall& c) {
  constexpr int64_t kInt = 0x7FFFFFFF;
  if (c.n_tokens < 0 || c.n_k_heads < 1 || c.n_heads < 1 || c.n_heads % c.n_k_heads != 0 ||
      c.n_heads > (1 << 16) || c.n_requests < 1 || c.max_len < 0 || c.max_len > kInt || c.dk < 1 ||
      c.dv < 1)
    return NVFP4_ERR_INVALID_VALUE;
  // a launch has fewer than 2^32 threads
  if (c.n_tokens > (int64_t(1) << 27) / c.n_heads || c.n_requests > (int64_t(1) << 20) / c.n_heads)
    return NVFP4_ERR_INVALID_VALUE;
  if ((c.dk != 64 && c.dk != 128) || c.dv % 16 != 0 || c.dv > 512) return NVFP4_ERR_UNSUPPORTED;
  return NVFP4_OK;
}

}  // namespace

extern "C" {

int nvfp4_abi_version(void) { return 3; }

const char* nvfp4_status_string(int status) {
  switch (status) {
    case NVFP4_OK: return "NVFP4_OK";
    case NVFP4_ERR_INVALID_VALUE:
      return "NVFP4_ERR_INVALID_VALUE: null pointer, bad size, k not a "
             "multiple of 16, bad stride or overlapping buffers";
    case NVFP4_ERR_UNSUPPORTED:
      return "NVFP4_ERR_UNSUPPORTED: unknown dtype, global mode or epilogue, "
             "or a shape outside the call's kernels (gate pair: more than 256 "
             "columns or k not a multiple of 128; fused quantise + GEMM: more "
             "than 64 rows or k not a multiple of 128; paged cache: page size "
             "not a multiple of 16; attention: d not 64, 128 or 256; "
             "gdn_attention: dk not 64 or 128, dv not a multiple of 16 or "
             "above 512; mxfp4_gemm: k above 2^22)";
    case NVFP4_ERR_MISALIGNED:
      return "NVFP4_ERR_MISALIGNED: a pointer or row stride breaks the "
             "required alignment";
    case NVFP4_ERR_LAUNCH:
      return "NVFP4_ERR_LAUNCH: the HIP runtime rejected a kernel launch";
    default: return "unknown nvfp4 status";
  }
}

int nvfp4_quantize(const void* x, int x_dtype, int64_t rows, int64_t k,
                   int64_t ldx, uint8_t* codes, uint8_t* scales,
                   float* global, int mode, void* stream) {
  if (!x || !codes || !scales || !global) return NVFP4_ERR_INVALID_VALUE;
  if (rows < 1 || k < 16 || k % 16 != 0 || ldx < k) return NVFP4_ERR_INVALID_VALUE;
  if (rows > kMaxDim || ldx > kMaxDim || rows > kMaxDim / ldx)
    return NVFP4_ERR_INVALID_VALUE;
  if (rows * (k / 16) > (int64_t(1) << 39)) return NVFP4_ERR_INVALID_VALUE;
  if (x_dtype != NVFP4_DTYPE_F32 && x_dtype != NVFP4_DTYPE_BF16)
    return NVFP4_ERR_UNSUPPORTED;
  if (mode != NVFP4_GLOBAL_COMPUTE && mode != NVFP4_GLOBAL_GIVEN)
    return NVFP4_ERR_UNSUPPORTED;
  const int64_t es = x_dtype == NVFP4_DTYPE_F32 ? 4 : 2;
  if (!aligned(x, 16) || (ldx * es) % 16 != 0 || !aligned(codes, 8) ||
      !aligned(global, 4))
    return NVFP4_ERR_MISALIGNED;
  const int64_t xbytes = ((rows - 1) * ldx + k) * es;
  const int64_t cbytes = rows * (k / 2), sbytes = rows * (k / 16);
  if (overlap(x, xbytes, codes, cbytes) || overlap(x, xbytes, scales, sbytes) ||
      overlap(x, xbytes, global, 4) || overlap(codes, cbytes, scales, sbytes) ||
      overlap(codes, cbytes, global, 4) || overlap(scales, sbytes, global, 4))
    return NVFP4_ERR_INVALID_VALUE;
  return status_of(nvfp4::launch_quantize(x, x_dtype, rows, k, ldx, codes,
                                          scales, global, mode,
                                          static_cast<hipStream_t>(stream)));
}

int nvfp4_harmonize_group(uint8_t* scales, int64_t k,
                          const int64_t* row_offsets, int n_modules,
                          const float* module_globals, float* shared_global,
                          void* stream) {
  if (!scales || !row_offsets || !module_globals || !shared_global)
    return NVFP4_ERR_INVALID_VALUE;
  if (k < 16 || k % 16 != 0 || k > kMaxDim) return NVFP4_ERR_INVALID_VALUE;
  if (n_modules < 1 || n_modules > nvfp4::kMaxModules)
    return NVFP4_ERR_INVALID_VALUE;
  if (row_offsets[0] != 0) return NVFP4_ERR_INVALID_VALUE;
  for (int i = 0; i < n_modules; ++i)
    if (row_offsets[i + 1] <= row_offsets[i]) return NVFP4_ERR_INVALID_VALUE;
  const int64_t total_rows = row_offsets[n_modules];
  if (total_rows > kMaxDim || total_rows > (int64_t(1) << 39) / (k / 16))
    return NVFP4_ERR_INVALID_VALUE;
  if (!aligned(scales, 16) || !aligned(module_globals, 4) || !aligned(shared_global, 4))
    return NVFP4_ERR_MISALIGNED;
  const int64_t sbytes = total_rows * (k / 16);
  if (overlap(shared_global, 4, module_globals, 4 * int64_t(n_modules)) ||
      overlap(shared_global, 4, scales, sbytes) ||
      overlap(module_globals, 4 * int64_t(n_modules), scales, sbytes))
    return NVFP4_ERR_INVALID_VALUE;
  return status_of(nvfp4::launch_harmonize(scales, k, row_offsets, n_modules,
                                           module_globals, shared_global,
                                           static_cast<hipStream_t>(stream)));
}

int w4a4_gemm(const uint8_t* a_codes, const uint8_t* a_scales,
              const float* a_global, int64_t m,
              const uint8_t* b_codes, const uint8_t* b_scales,
              const float* b_global, int64_t n, int64_t k,
              void* out, int out_dtype, int64_t ldo, int epilogue,
              void* stream) {
  if (!a_codes || !a_scales || !a_global || !b_codes || !b_scales ||
      !b_global || !out)
    return NVFP4_ERR_INVALID_VALUE;
  if (m < 1 || n < 1 || k < 16 || k % 16 != 0 || ldo < n)
    return NVFP4_ERR_INVALID_VALUE;
  if (m > kMaxDim || n > kMaxDim || k > kMaxDim || ldo > kMaxDim ||
      m > kMaxDim / ldo || m > kMaxDim / k || n > kMaxDim / k)
    return NVFP4_ERR_INVALID_VALUE;
  if (out_dtype != NVFP4_DTYPE_F32 && out_dtype != NVFP4_DTYPE_BF16)
    return NVFP4_ERR_UNSUPPORTED;
  if (epilogue != W4A4_EPI_NONE && epilogue != W4A4_EPI_ALPHA &&
      epilogue != W4A4_EPI_BETA)
    return NVFP4_ERR_UNSUPPORTED;
  const int64_t os = out_dtype == NVFP4_DTYPE_F32 ? 4 : 2;
  if (!aligned(a_codes, 16) || !aligned(b_codes, 16) || !aligned(a_scales, 16) ||
      !aligned(b_scales, 16) || !aligned(out, 4) || !aligned(a_global, 4) ||
      !aligned(b_global, 4))
    return NVFP4_ERR_MISALIGNED;
  const int64_t obytes = ((m - 1) * ldo + n) * os;
  if (overlap(out, obytes, a_codes, m * (k / 2)) ||
      overlap(out, obytes, a_scales, m * (k / 16)) ||
      overlap(out, obytes, b_codes, n * (k / 2)) ||
      overlap(out, obytes, b_scales, n * (k / 16)) ||
      overlap(out, obytes, a_global, 4) || overlap(out, obytes, b_global, 4))
    return NVFP4_ERR_INVALID_VALUE;
  return status_of(nvfp4::launch_gemm(a_codes, a_scales, a_global, m, b_codes,
                                      b_scales, b_global, n, k, out, out_dtype,
                                      ldo, epilogue,
                                      static_cast<hipStream_t>(stream)));
}

int w4a4_gemm_gdn_gates(const uint8_t* x_codes, const uint8_t* x_scales,
                        const float* x_global, int64_t m,
                        const uint8_t* w_codes, const uint8_t* w_scales,
                        const float* w_global, int64_t n_beta, int64_t n_alpha,
                        int64_t k, const float* a_log, const float* dt_bias,
                        float* beta_out, int64_t ld_beta, float* alpha_out,
                        int64_t ld_alpha, void* stream) {
  if (!x_codes || !x_scales || !x_global || !w_codes || !w_scales || !w_global)
    return NVFP4_ERR_INVALID_VALUE;
  if (m < 1 || n_beta < 0 || n_alpha < 0 || n_beta + n_alpha < 1 || k < 16 ||
      k % 16 != 0 || m > kMaxDim || k > kMaxDim || m > kMaxDim / k)
    return NVFP4_ERR_INVALID_VALUE;
  if (n_beta > 0 && (!beta_out || ld_beta < n_beta || m > kMaxDim / ld_beta))
    return NVFP4_ERR_INVALID_VALUE;
  if (n_alpha > 0 && (!alpha_out || !a_log || !dt_bias || ld_alpha < n_alpha ||
                      m > kMaxDim / ld_alpha))
    return NVFP4_ERR_INVALID_VALUE;
  if (n_beta + n_alpha > nvfp4::kMaxGateCols || k % 128 != 0)
    return NVFP4_ERR_UNSUPPORTED;
  if (!aligned(x_codes, 16) || !aligned(w_codes, 16) || !aligned(x_scales, 16) ||
      !aligned(w_scales, 16) || !aligned(x_global, 4) || !aligned(w_global, 4) ||
      (n_beta > 0 && !aligned(beta_out, 4)) ||
      (n_alpha > 0 && (!aligned(alpha_out, 4) || !aligned(a_log, 4) ||
                       !aligned(dt_bias, 4))))
    return NVFP4_ERR_MISALIGNED;
  const int64_t n = n_beta + n_alpha;
  struct Range { const void* p; int64_t len; };
  const Range in[] = {{x_codes, m * (k / 2)}, {x_scales, m * (k / 16)},
                      {x_global, 4}, {w_codes, n * (k / 2)},
                      {w_scales, n * (k / 16)}, {w_global, 4},
                      {a_log, 4 * n_alpha}, {dt_bias, 4 * n_alpha}};
  const Range outs[] = {{beta_out, n_beta ? ((m - 1) * ld_beta + n_beta) * 4 : 0},
                        {alpha_out, n_alpha ? ((m - 1) * ld_alpha + n_alpha) * 4 : 0}};
  for (const Range& o : outs) {
    if (o.len == 0) continue;
    for (const Range& i : in)
      if (i.len > 0 && overlap(o.p, o.len, i.p, i.len)) return NVFP4_ERR_INVALID_VALUE;
  }
  if (outs[0].len && outs[1].len && overlap(outs[0].p, outs[0].len, outs[1].p, outs[1].len))
    return NVFP4_ERR_INVALID_VALUE;
  return status_of(nvfp4::launch_gdn_gates(x_codes, x_scales, x_global, m, w_codes,
                                           w_scales, w_global, n_beta, n_alpha, k,
                                           a_log, dt_bias, beta_out, ld_beta,
                                           alpha_out, ld_alpha,
                                           static_cast<hipStream_t>(stream)));
}

int w4a4_gemm_quantize_a(const void* x, int x_dtype, int64_t m, int64_t k, int64_t ldx,
                         uint8_t* x_codes, uint8_t* x_scales, float* x_global, int mode,
                         const uint8_t* w_codes, const uint8_t* w_scales,
                         const float* w_global, int64_t n, void* out, int out_dtype,
                         int64_t ldo, void* stream) {
  if (!x_codes || !x_scales || !x_global || !w_codes || !w_scales || !w_global || !out)
    return NVFP4_ERR_INVALID_VALUE;
  const int cx = check_x(x, x_dtype, m, k, ldx);
  if (cx != NVFP4_OK) return cx;
  if (n < 1 || ldo < n || n > kMaxDim || k > kMaxDim || ldo > kMaxDim ||
      m > kMaxDim / ldo || n > kMaxDim / k)
    return NVFP4_ERR_INVALID_VALUE;
  if (mode != NVFP4_GLOBAL_COMPUTE && mode != NVFP4_GLOBAL_GIVEN)
    return NVFP4_ERR_UNSUPPORTED;
  if (out_dtype != NVFP4_DTYPE_F32 && out_dtype != NVFP4_DTYPE_BF16)
    return NVFP4_ERR_UNSUPPORTED;
  if (m > nvfp4::kMaxFusedRows || k % 128 != 0) return NVFP4_ERR_UNSUPPORTED;
  if (!aligned(x_codes, 16) || !aligned(x_scales, 16) || !aligned(w_codes, 16) ||
      !aligned(w_scales, 16) || !aligned(x_global, 4) || !aligned(w_global, 4) ||
      !aligned(out, 4))
    return NVFP4_ERR_MISALIGNED;
  const int64_t es = x_dtype == NVFP4_DTYPE_F32 ? 4 : 2;
  const int64_t os = out_dtype == NVFP4_DTYPE_F32 ? 4 : 2;
  struct Range { const void* p; int64_t len; };
  const Range in[] = {{x, ((m - 1) * ldx + k) * es}, {w_codes, n * (k / 2)},
                      {w_scales, n * (k / 16)}, {w_global, 4}};
  const Range outs[] = {{x_codes, m * (k / 2)}, {x_scales, m * (k / 16)},
                        {x_global, 4}, {out, ((m - 1) * ldo + n) * os}};
  for (int i = 0; i < 4; ++i) {
    for (const Range& r : in)
      if (overlap(outs[i].p, outs[i].len, r.p, r.len)) return NVFP4_ERR_INVALID_VALUE;
    for (int j = i + 1; j < 4; ++j)
      if (overlap(outs[i].p, outs[i].len, outs[j].p, outs[j].len))
        return NVFP4_ERR_INVALID_VALUE;
  }
  return status_of(nvfp4::launch_quantize_gemm(x, x_dtype, m, k, ldx, mode, x_codes, x_scales,
                                               x_global, w_codes, w_scales, w_global, n, out,
                                               out_dtype, ldo,
                                               static_cast<hipStream_t>(stream)));
}

int nvfp4_dequantize(const uint8_t* codes, const uint8_t* scales,
                     const float* global, int64_t rows, int64_t k, void* out,
                     int out_dtype, int64_t ldo, void* stream) {
  if (!codes || !scales || !global || !out) return NVFP4_ERR_INVALID_VALUE;
  if (rows < 1 || k < 16 || k % 16 != 0 || ldo < k) return NVFP4_ERR_INVALID_VALUE;
  if (rows > kMaxDim || ldo > kMaxDim || rows > kMaxDim / ldo)
    return NVFP4_ERR_INVALID_VALUE;
  if (rows * (k / 16) > (int64_t(1) << 39)) return NVFP4_ERR_INVALID_VALUE;
  if (out_dtype != NVFP4_DTYPE_F32 && out_dtype != NVFP4_DTYPE_BF16)
    return NVFP4_ERR_UNSUPPORTED;
  const int64_t os = out_dtype == NVFP4_DTYPE_F32 ? 4 : 2;
  if (!aligned(codes, 8) || !aligned(out, 16) || (ldo * os) % 16 != 0 ||
      !aligned(global, 4))
    return NVFP4_ERR_MISALIGNED;
  const int64_t obytes = ((rows - 1) * ldo + k) * os;
  if (overlap(out, obytes, codes, rows * (k / 2)) ||
      overlap(out, obytes, scales, rows * (k / 16)) || overlap(out, obytes, global, 4))
    return NVFP4_ERR_INVALID_VALUE;
  return status_of(nvfp4::launch_dequantize(codes, scales, global, rows, k, out,
                                            out_dtype, ldo,
                                            static_cast<hipStream_t>(stream)));
}

int nvfp4_error_stats(const void* x, int x_dtype, int64_t rows, int64_t k,
                      int64_t ldx, const uint8_t* codes, const uint8_t* scales,
                      const float* global, double* stats, void* stream) {
  if (!x || !codes || !scales || !global || !stats) return NVFP4_ERR_INVALID_VALUE;
  if (rows < 1 || k < 16 || k % 16 != 0 || ldx < k) return NVFP4_ERR_INVALID_VALUE;
  if (rows > kMaxDim || ldx > kMaxDim || rows > kMaxDim / ldx)
    return NVFP4_ERR_INVALID_VALUE;
  if (rows * (k / 16) > (int64_t(1) << 39)) return NVFP4_ERR_INVALID_VALUE;
  if (x_dtype != NVFP4_DTYPE_F32 && x_dtype != NVFP4_DTYPE_BF16)
    return NVFP4_ERR_UNSUPPORTED;
  const int64_t es = x_dtype == NVFP4_DTYPE_F32 ? 4 : 2;
  if (!aligned(x, 16) || (ldx * es) % 16 != 0 || !aligned(codes, 8) ||
      !aligned(global, 4) || !aligned(stats, 8))
    return NVFP4_ERR_MISALIGNED;
  const int64_t sbytes = rows * 3 * 8;
  if (overlap(stats, sbytes, x, ((rows - 1) * ldx + k) * es) ||
      overlap(stats, sbytes, codes, rows * (k / 2)) ||
      overlap(stats, sbytes, scales, rows * (k / 16)) || overlap(stats, sbytes, global, 4))
    return NVFP4_ERR_INVALID_VALUE;
  return status_of(nvfp4::launch_error_stats(x, x_dtype, rows, k, ldx, codes, scales,
                                             global, stats,
                                             static_cast<hipStream_t>(stream)));
}

int fp8_kv_amax_update(const void* x, int x_dtype, int64_t rows, int64_t k,
                       int64_t ldx, float* amax, void* stream) {
  const int st = check_x(x, x_dtype, rows, k, ldx);
  if (st != NVFP4_OK) return st;
  if (!amax) return NVFP4_ERR_INVALID_VALUE;
  if (!aligned(amax, 4)) return NVFP4_ERR_MISALIGNED;
  return status_of(nvfp4::launch_kv_amax_update(x, x_dtype, rows, k, ldx, amax,
                                                static_cast<hipStream_t>(stream)));
}

int fp8_kv_scale_from_amax(const float* amax, float* scale, void* stream) {
  if (!amax || !scale) return NVFP4_ERR_INVALID_VALUE;
  if (!aligned(amax, 4) || !aligned(scale, 4)) return NVFP4_ERR_MISALIGNED;
  return status_of(nvfp4::launch_kv_scale(amax, scale, static_cast<hipStream_t>(stream)));
}

int fp8_kv_cast(const void* x, int x_dtype, int64_t rows, int64_t k, int64_t ldx,
                const float* scale, uint8_t* out, int64_t ldo, void* stream) {
  const int st = check_x(x, x_dtype, rows, k, ldx);
  if (st != NVFP4_OK) return st;
  if (!scale || !out || ldo < k || ldo > kMaxDim || rows > kMaxDim / ldo)
    return NVFP4_ERR_INVALID_VALUE;
  if (!aligned(scale, 4) || !aligned(out, 16) || ldo % 16 != 0)
    return NVFP4_ERR_MISALIGNED;
  const int64_t es = x_dtype == NVFP4_DTYPE_F32 ? 4 : 2;
  const int64_t obytes = (rows - 1) * ldo + k;
  if (overlap(out, obytes, x, ((rows - 1) * ldx + k) * es) || overlap(out, obytes, scale, 4))
    return NVFP4_ERR_INVALID_VALUE;
  return status_of(nvfp4::launch_kv_cast(x, x_dtype, rows, k, ldx, scale, out, ldo,
                                         static_cast<hipStream_t>(stream)));
}

int kv_page_tables(const int32_t* new_lens, const int32_t* cached_lens, int64_t n_requests,
                   int32_t* block_table, int64_t max_blocks, int64_t ld_table,
                   const int32_t* free_pages, int64_t n_free, int64_t page_size,
                   int64_t n_tokens, int32_t* cu_new, int32_t* kv_lens, int32_t* positions,
                   int64_t* slots, int32_t* pages_used, void* stream) {
  if (!new_lens || !cached_lens || !block_table || !cu_new || !kv_lens || !pages_used ||
      (n_free > 0 && !free_pages) || (n_tokens > 0 && (!positions || !slots)))
    return NVFP4_ERR_INVALID_VALUE;
  if (n_requests < 1 || n_requests > (1 << 24) || max_blocks < 1 || ld_table < max_blocks ||
      ld_table > 0x7FFFFFFF || n_free < 0 || n_free > 0x7FFFFFFF || page_size < 1 ||
      page_size > (1 << 24) || n_tokens < 0 || n_tokens > 0x7FFFFFFF)
    return NVFP4_ERR_INVALID_VALUE;
  if (page_size % 16 != 0) return NVFP4_ERR_UNSUPPORTED;
  if (!aligned(new_lens, 4) || !aligned(cached_lens, 4) || !aligned(block_table, 4) ||
      !aligned(free_pages, 4) || !aligned(cu_new, 4) || !aligned(kv_lens, 4) ||
      !aligned(positions, 4) || !aligned(slots, 8) || !aligned(pages_used, 4))
    return NVFP4_ERR_MISALIGNED;
  struct Range { const void* p; int64_t len; };
  const Range in[] = {{new_lens, 4 * n_requests}, {cached_lens, 4 * n_requests},
                      {free_pages, 4 * n_free}};
  const Range outs[] = {{block_table, ((n_requests - 1) * ld_table + max_blocks) * 4},
                        {cu_new, 4 * (n_requests + 1)}, {kv_lens, 4 * n_requests},
                        {positions, 4 * n_tokens}, {slots, 8 * n_tokens}, {pages_used, 4}};
  for (int i = 0; i < 6; ++i) {
    if (outs[i].len < 1) continue;
    for (const Range& r : in)
      if (r.len > 0 && overlap(outs[i].p, outs[i].len, r.p, r.len)) return NVFP4_ERR_INVALID_VALUE;
    for (int j = i + 1; j < 6; ++j)
      if (outs[j].len > 0 && overlap(outs[i].p, outs[i].len, outs[j].p, outs[j].len))
        return NVFP4_ERR_INVALID_VALUE;
  }
  return status_of(nvfp4::launch_page_tables(new_lens, cached_lens, n_requests, block_table,
                                             max_blocks, ld_table, free_pages, n_free, page_size,
                                             n_tokens, cu_new, kv_lens, positions, slots,
                                             pages_used, static_cast<hipStream_t>(stream)));
}

int kv_page_write(const void* k, int64_t k_token_stride, int64_t k_head_stride, const void* v,
                  int64_t v_token_stride, int64_t v_head_stride, int x_dtype, int64_t n_tokens,
                  void* k_cache, void* v_cache, int cache_dtype, int64_t n_pages,
                  int64_t page_size, int64_t n_heads, int64_t d, int64_t page_stride,
                  int64_t head_stride, int64_t token_stride, const float* k_scale,
                  const float* v_scale, const int64_t* slots, void* stream) {
  const nvfp4::KvPool pool = {k_cache, v_cache, cache_dtype == NVFP4_DTYPE_E4M3, n_pages,
                              page_size, n_heads, d, page_stride, head_stride, token_stride,
                              k_scale, v_scale};
  const int cp = check_pool(pool, cache_dtype);
  if (cp != NVFP4_OK) return cp;
  if (n_tokens < 0) return NVFP4_ERR_INVALID_VALUE;
  if (d % 16 != 0 || d > 1024) return NVFP4_ERR_UNSUPPORTED;
  if (x_dtype != NVFP4_DTYPE_F32 && x_dtype != NVFP4_DTYPE_BF16) return NVFP4_ERR_UNSUPPORTED;
  if (n_tokens == 0) return NVFP4_OK;
  const int64_t es = x_dtype == NVFP4_DTYPE_F32 ? 4 : 2;
  int st = check_rows(k, n_tokens, k_token_stride, n_heads, k_head_stride, d, es, 16);
  if (st != NVFP4_OK) return st;
  st = check_rows(v, n_tokens, v_token_stride, n_heads, v_head_stride, d, es, 16);
  if (st != NVFP4_OK) return st;
  if (!slots || n_tokens >= (int64_t(1) << 31) / (n_heads * (d / 16)))
    return NVFP4_ERR_INVALID_VALUE;
  if (!aligned(slots, 8)) return NVFP4_ERR_MISALIGNED;
  struct Range { const void* p; int64_t len; };
  const Range in[] = {{k, rows_bytes(n_tokens, k_token_stride, n_heads, k_head_stride, d, es)},
                      {v, rows_bytes(n_tokens, v_token_stride, n_heads, v_head_stride, d, es)},
                      {slots, 8 * n_tokens}, {k_scale, pool.fp8 ? 4 : 0},
                      {v_scale, pool.fp8 ? 4 : 0}};
  for (const Range& r : in)
    if (r.len > 0 && (overlap(k_cache, pool_bytes(pool), r.p, r.len) ||
                      overlap(v_cache, pool_bytes(pool), r.p, r.len)))
      return NVFP4_ERR_INVALID_VALUE;
  return status_of(nvfp4::launch_page_write({k, k_token_stride, k_head_stride},
                                            {v, v_token_stride, v_head_stride}, x_dtype, n_tokens,
                                            pool, slots, static_cast<hipStream_t>(stream)));
}

int64_t kv_paged_attention_workspace(int64_t n_tokens, int64_t n_heads, int64_t n_kv_heads,
                                     int64_t d, int64_t n_requests, int64_t max_new,
                                     int64_t max_kv, int64_t window) {
  nvfp4::AttnCall c = {};
  static const int32_t paged = 0;      // any non-null table: only its presence counts
  c.table = &paged;
  c.n_tokens = n_tokens; c.n_heads = n_heads; c.n_kv_heads = n_kv_heads; c.d = d;
  c.n_requests = n_requests; c.max_new = max_new; c.max_kv = max_kv; c.window = window;
  c.scale = 1.0f;
  return check_attention(c) == NVFP4_OK ? nvfp4::attention_workspace(c) : -1;
}

int kv_paged_attention(const void* q, int64_t q_token_stride, int64_t q_head_stride,
                       int64_t n_tokens, int64_t n_heads, const void* k_cache,
                       const void* v_cache, int cache_dtype, int64_t n_pages, int64_t page_size,
                       int64_t n_kv_heads, int64_t d, int64_t page_stride, int64_t head_stride,
                       int64_t token_stride, const float* k_scale, const float* v_scale,
                       const int32_t* block_table, int64_t max_blocks, int64_t ld_table,
                       const int32_t* cu_new, const int32_t* kv_lens, int64_t n_requests,
                       int64_t max_new, int64_t max_kv, float scale, int causal, int64_t window,
                       void* out, int64_t out_token_stride, int64_t out_head_stride,
                       void* workspace, int64_t workspace_bytes, void* stream) {
  nvfp4::AttnCall c = {};
  c.q = {q, q_token_stride, q_head_stride};
  c.out = out; c.out_token = out_token_stride; c.out_head = out_head_stride;
  c.n_tokens = n_tokens; c.n_heads = n_heads; c.n_kv_heads = n_kv_heads; c.d = d;
  c.pool = {const_cast<void*>(k_cache), const_cast<void*>(v_cache),
            cache_dtype == NVFP4_DTYPE_E4M3, n_pages, page_size, n_kv_heads, d, page_stride,
            head_stride, token_stride, k_scale, v_scale};
  c.table = block_table; c.cols = max_blocks; c.ld_table = ld_table;
  c.cu = cu_new; c.kv_lens = kv_lens;
  c.n_requests = n_requests; c.max_new = max_new; c.max_kv = max_kv;
  c.scale = scale; c.causal = causal != 0; c.window = window; c.workspace = workspace;
  if (!block_table || !cu_new || !kv_lens) return NVFP4_ERR_INVALID_VALUE;
  int st = check_attention(c);
  if (st != NVFP4_OK) return st;
  st = check_pool(c.pool, cache_dtype);
  if (st != NVFP4_OK) return st;
  if (max_blocks < 1 || ld_table < max_blocks || ld_table > 0x7FFFFFFF ||
      token_stride * (c.pool.fp8 ? 1 : 2) >= (1 << 26))
    return NVFP4_ERR_INVALID_VALUE;
  if (n_tokens == 0) return NVFP4_OK;
  st = check_rows(q, n_tokens, q_token_stride, n_heads, q_head_stride, d, 2, 16);
  if (st != NVFP4_OK) return st;
  st = check_rows(out, n_tokens, out_token_stride, n_heads, out_head_stride, d, 2, 8);
  if (st != NVFP4_OK) return st;
  if (!aligned(block_table, 4) || !aligned(cu_new, 4) || !aligned(kv_lens, 4))
    return NVFP4_ERR_MISALIGNED;
  return run_attention(c, workspace_bytes, stream);
}

int64_t prompt_attention_workspace(int64_t n_tokens, int64_t n_heads, int64_t n_kv_heads,
                                   int64_t d, int64_t n_prompts, int64_t max_len,
                                   int64_t window) {
  nvfp4::AttnCall c = {};
  c.n_tokens = n_tokens; c.n_heads = n_heads; c.n_kv_heads = n_kv_heads; c.d = d;
  c.n_requests = n_prompts; c.max_new = c.max_kv = max_len; c.window = window;
  c.scale = 1.0f;
  return check_attention(c) == NVFP4_OK ? nvfp4::attention_workspace(c) : -1;
}

int prompt_attention(const void* q, int64_t q_token_stride, int64_t q_head_stride, const void* k,
                     int64_t k_token_stride, int64_t k_head_stride, const void* v,
                     int64_t v_token_stride, int64_t v_head_stride, int64_t n_tokens,
                     int64_t n_heads, int64_t n_kv_heads, int64_t d, const int32_t* cu_lens,
                     int64_t n_prompts, int64_t max_len, float scale, int causal, int64_t window,
                     void* out, int64_t out_token_stride, int64_t out_head_stride,
                     void* workspace, int64_t workspace_bytes, void* stream) {
  nvfp4::AttnCall c = {};
  c.q = {q, q_token_stride, q_head_stride};
  c.k = {k, k_token_stride, k_head_stride};
  c.v = {v, v_token_stride, v_head_stride};
  c.out = out; c.out_token = out_token_stride; c.out_head = out_head_stride;
  c.n_tokens = n_tokens; c.n_heads = n_heads; c.n_kv_heads = n_kv_heads; c.d = d;
  c.cu = cu_lens; c.n_requests = n_prompts; c.max_new = c.max_kv = max_len;
  c.scale = scale; c.causal = causal != 0; c.window = window; c.workspace = workspace;
  if (!cu_lens) return NVFP4_ERR_INVALID_VALUE;
  int st = check_attention(c);
  if (st != NVFP4_OK) return st;
  if (n_tokens == 0) return NVFP4_OK;
  st = check_rows(q, n_tokens, q_token_stride, n_heads, q_head_stride, d, 2, 16);
  if (st != NVFP4_OK) return st;
  st = check_rows(k, n_tokens, k_token_stride, n_kv_heads, k_head_stride, d, 2, 16);
  if (st != NVFP4_OK) return st;
  st = check_rows(v, n_tokens, v_token_stride, n_kv_heads, v_head_stride, d, 2, 16);
  if (st != NVFP4_OK) return st;
  if (k_token_stride >= (1 << 25) || v_token_stride >= (1 << 25)) return NVFP4_ERR_INVALID_VALUE;
  st = check_rows(out, n_tokens, out_token_stride, n_heads, out_head_stride, d, 2, 8);
  if (st != NVFP4_OK) return st;
  if (!aligned(cu_lens, 4)) return NVFP4_ERR_MISALIGNED;
  return run_attention(c, workspace_bytes, stream);
}

int mxfp4_quantize(const void* x, int x_dtype, int64_t rows, int64_t k, int64_t ldx,
                   uint8_t* codes, uint8_t* scales, void* stream) {
  int st = check_mxfp4(codes, scales, rows, k);
  if (st != NVFP4_OK) return st;
  st = check_dense(x, x_dtype, rows, k, ldx);
  if (st != NVFP4_OK) return st;
  if (!aligned(codes, 16)) return NVFP4_ERR_MISALIGNED;
  const int64_t xbytes = ((rows - 1) * ldx + k) * (x_dtype == NVFP4_DTYPE_F32 ? 4 : 2);
  const int64_t cbytes = rows * (k / 2), sbytes = rows * (k / 32);
  if (overlap(x, xbytes, codes, cbytes) || overlap(x, xbytes, scales, sbytes) ||
      overlap(codes, cbytes, scales, sbytes))
    return NVFP4_ERR_INVALID_VALUE;
  return status_of(nvfp4::launch_mxfp4_quantize(x, x_dtype, rows, k, ldx, codes, scales,
                                                static_cast<hipStream_t>(stream)));
}

int mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t k,
                     void* out, int out_dtype, int64_t ldo, void* stream) {
  int st = check_mxfp4(codes, scales, rows, k);
  if (st != NVFP4_OK) return st;
  st = check_dense(out, out_dtype, rows, k, ldo);
  if (st != NVFP4_OK) return st;
  if (!aligned(codes, 16)) return NVFP4_ERR_MISALIGNED;
  const int64_t obytes = ((rows - 1) * ldo + k) * (out_dtype == NVFP4_DTYPE_F32 ? 4 : 2);
  if (overlap(out, obytes, codes, rows * (k / 2)) || overlap(out, obytes, scales, rows * (k / 32)))
    return NVFP4_ERR_INVALID_VALUE;
  return status_of(nvfp4::launch_mxfp4_dequantize(codes, scales, rows, k, out, out_dtype, ldo,
                                                  static_cast<hipStream_t>(stream)));
}

int mxfp4_gemm(const uint8_t* a_codes, const uint8_t* a_scales, int64_t m, const uint8_t* b_codes,
               const uint8_t* b_scales, int64_t n, int64_t k, void* out, int out_dtype,
               int64_t ldo, void* stream) {
  int st = check_mxfp4(a_codes, a_scales, m, k);
  if (st != NVFP4_OK) return st;
  st = check_mxfp4(b_codes, b_scales, n, k);
  if (st != NVFP4_OK) return st;
  if (!out || ldo < n || ldo > kMaxDim || m > kMaxDim / ldo) return NVFP4_ERR_INVALID_VALUE;
  if (out_dtype != NVFP4_DTYPE_F32 && out_dtype != NVFP4_DTYPE_BF16) return NVFP4_ERR_UNSUPPORTED;
  if (k > nvfp4::kMaxMxfp4K) return NVFP4_ERR_UNSUPPORTED;
  if (!aligned(a_codes, 16) || !aligned(a_scales, 16) || !aligned(b_codes, 16) ||
      !aligned(b_scales, 16) || !aligned(out, 4))
    return NVFP4_ERR_MISALIGNED;
  const int64_t obytes = ((m - 1) * ldo + n) * (out_dtype == NVFP4_DTYPE_F32 ? 4 : 2);
  if (overlap(out, obytes, a_codes, m * (k / 2)) || overlap(out, obytes, a_scales, m * (k / 32)) ||
      overlap(out, obytes, b_codes, n * (k / 2)) || overlap(out, obytes, b_scales, n * (k / 32)))
    return NVFP4_ERR_INVALID_VALUE;
  return status_of(nvfp4::launch_mxfp4_gemm(a_codes, a_scales, m, b_codes, b_scales, n, k, out,
                                            out_dtype, ldo, static_cast<hipStream_t>(stream)));
}

int64_t gdn_attention_workspace(int64_t n_tokens, int64_t n_k_heads, int64_t n_heads, int64_t dk,
                                int64_t dv, int64_t n_requests, int64_t max_len, int delta) {
  nvfp4::GdnCall c = {};
  static const float given = 0.0f;     // any non-null beta: only its presence counts
  c.n_tokens = n_tokens; c.n_k_heads = n_k_heads; c.n_heads = n_heads; c.dk = dk; c.dv = dv;
  c.n_requests = n_requests; c.max_len = max_len; c.beta = delta ? &given : nullptr;
  return check_gdn(c) == NVFP4_OK ? nvfp4::gdn_workspace(c) : -1;
}

int gdn_attention(const void* q, int64_t q_token_stride, int64_t q_head_stride, const void* k,
                  int64_t k_token_stride, int64_t k_head_stride, const void* v,
                  int64_t v_token_stride, int64_t v_head_stride, int64_t n_tokens,
                  int64_t n_k_heads, int64_t n_heads, int64_t dk, int64_t dv, const float* alpha,
                  int64_t ld_alpha, const float* beta, int64_t ld_beta, float* state,
                  int64_t n_slots, int64_t slot_stride, const int32_t* slots,
                  const int32_t* cu_lens, const int32_t* cached_lens, int64_t n_requests,
                  int64_t max_len, float scale, int normalize, void* out,
                  int64_t out_token_stride, int64_t out_head_stride, void* workspace,
                  int64_t workspace_bytes, void* stream) {
  nvfp4::GdnCall c = {};
  c.q = {q, q_token_stride, q_head_stride};
  c.k = {k, k_token_stride, k_head_stride};
  c.v = {v, v_token_stride, v_head_stride};
  c.alpha = alpha; c.ld_alpha = ld_alpha; c.beta = beta; c.ld_beta = ld_beta;
  c.n_tokens = n_tokens; c.n_k_heads = n_k_heads; c.n_heads = n_heads; c.dk = dk; c.dv = dv;
  c.state = state; c.n_slots = n_slots; c.slot_stride = slot_stride; c.slots = slots;
  c.cu = cu_lens; c.cached = cached_lens; c.n_requests = n_requests; c.max_len = max_len;
  c.scale = scale; c.normalize = normalize != 0;
  c.out = out; c.out_token = out_token_stride; c.out_head = out_head_stride;
  c.workspace = workspace;
  int st = check_gdn(c);
  if (st != NVFP4_OK) return st;
  if (!state || !cu_lens || n_slots < 1 || n_slots > kMaxDim || (!slots && n_slots < n_requests))
    return NVFP4_ERR_INVALID_VALUE;
  const int64_t held = n_heads * dk * dv;
  if (slot_stride < held || slot_stride > kMaxDim || n_slots > kMaxDim / slot_stride)
    return NVFP4_ERR_INVALID_VALUE;
  if (!(scale > 0.0f) || isinf(scale)) return NVFP4_ERR_INVALID_VALUE;
  if (!aligned(state, 16) || slot_stride % 4 != 0 || !aligned(slots, 4) || !aligned(cu_lens, 4) ||
      !aligned(cached_lens, 4))
    return NVFP4_ERR_MISALIGNED;
  if (n_tokens == 0) return NVFP4_OK;
  if (!alpha || ld_alpha < n_heads || ld_alpha > kMaxDim || n_tokens > kMaxDim / ld_alpha ||
      (beta && (ld_beta < n_heads || ld_beta > kMaxDim || n_tokens > kMaxDim / ld_beta)))
    return NVFP4_ERR_INVALID_VALUE;
  if (!aligned(alpha, 4) || !aligned(beta, 4)) return NVFP4_ERR_MISALIGNED;
  st = check_rows(q, n_tokens, q_token_stride, n_k_heads, q_head_stride, dk, 2, 16);
  if (st != NVFP4_OK) return st;
  st = check_rows(k, n_tokens, k_token_stride, n_k_heads, k_head_stride, dk, 2, 16);
  if (st != NVFP4_OK) return st;
  st = check_rows(v, n_tokens, v_token_stride, n_heads, v_head_stride, dv, 2, 16);
  if (st != NVFP4_OK) return st;
  st = check_rows(out, n_tokens, out_token_stride, n_heads, out_head_stride, dv, 2, 8);
  if (st != NVFP4_OK) return st;
  // 32-bit offsets within the 64 rows of a chunk
  constexpr int64_t kStride = int64_t(1) << 24;
  if (q_token_stride >= kStride || k_token_stride >= kStride || v_token_stride >= kStride ||
      out_token_stride >= kStride)
    return NVFP4_ERR_INVALID_VALUE;
  const int64_t need = nvfp4::gdn_workspace(c);
  if (need < 0 || workspace_bytes < need || (need > 0 && !workspace))
    return NVFP4_ERR_INVALID_VALUE;
  if (need > 0 && !aligned(workspace, 16)) return NVFP4_ERR_MISALIGNED;
  struct Range { const void* p; int64_t len; };
  const Range in[] = {
      {q, rows_bytes(n_tokens, q_token_stride, n_k_heads, q_head_stride, dk, 2)},
      {k, rows_bytes(n_tokens, k_token_stride, n_k_heads, k_head_stride, dk, 2)},
      {v, rows_bytes(n_tokens, v_token_stride, n_heads, v_head_stride, dv, 2)},
      {alpha, ((n_tokens - 1) * ld_alpha + n_heads) * 4},
      {beta, beta ? ((n_tokens - 1) * ld_beta + n_heads) * 4 : 0},
      {slots, slots ? 4 * n_requests : 0},
      {cu_lens, 4 * (n_requests + 1)},
      {cached_lens, cached_lens ? 4 * n_requests : 0}};
  const Range outs[] = {
      {out, rows_bytes(n_tokens, out_token_stride, n_heads, out_head_stride, dv, 2)},
      {state, ((n_slots - 1) * slot_stride + held) * 4}, {workspace, need}};
  for (int i = 0; i < 3; ++i) {
    if (outs[i].len < 1) continue;
    for (const Range& r : in)
      if (r.len > 0 && overlap(outs[i].p, outs[i].len, r.p, r.len)) return NVFP4_ERR_INVALID_VALUE;
    for (int j = i + 1; j < 3; ++j)
      if (outs[j].len > 0 && overlap(outs[i].p, outs[i].len, outs[j].p, outs[j].len))
        return NVFP4_ERR_INVALID_VALUE;
  }
  return status_of(nvfp4::launch_gdn(c, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
