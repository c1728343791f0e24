// attention_api.cpp -- the extern "C" entry points of the attention half of a
// decoder layer: argument validation (always before any HIP call) and the
// launches.
#include "api_common.h"
#include "attention.h"

using namespace nvfp4::api;

extern "C" {

static int add_rmsnorm(const void* x, int x_dtype, const void* residual, int residual_dtype, const void* w, int w_dtype,
                       double eps, int64_t M, int64_t K, const float* g_inv, float* row_g, void* residual_out,
                       uint8_t* codes, uint8_t* scales, void* stream) {
  for (int d : {x_dtype, residual_dtype, w_dtype})
    if (d != NVFP4_DTYPE_BF16 && d != NVFP4_DTYPE_F32) return fail(NVFP4_ERR_INVALID_ARG, "dtypes must be BF16 or F32");
  if (!dim_ok(M) || K < 0 || K > kMaxDim || K % 16 != 0)
    return fail(NVFP4_ERR_INVALID_ARG, "need 0 <= M <= 2^24 and 0 <= K <= 2^24 a multiple of 16 (M=%lld K=%lld)",
                (long long)M, (long long)K);
  if (!(eps >= 0.0)) return fail(NVFP4_ERR_INVALID_ARG, "eps must not be negative");
  if (M * K == 0) { g_err[0] = '\0'; return NVFP4_OK; }
  if (!x || !w || !codes || !scales) return fail(NVFP4_ERR_INVALID_ARG, "null pointer argument");
  if (!g_inv && !row_g) return fail(NVFP4_ERR_INVALID_ARG, "null g_inv or row_g");
  if (!aligned16(x) || !aligned16(w) || !aligned16(codes) || !aligned16(residual) || !aligned16(residual_out))
    return fail(NVFP4_ERR_INVALID_ARG, "x, residual, w, residual_out and codes must be 16-byte aligned");
  if (residual_out && (residual ? residual_out == x && residual_dtype != x_dtype : false))
    return fail(NVFP4_ERR_INVALID_ARG, "residual_out may be x only where both have one type");
  int st = check_device();
  if (st) return st;
  nvfp4::NormArgs a{x, residual, w, residual_out, M, K, x_dtype == NVFP4_DTYPE_F32, residual_dtype == NVFP4_DTYPE_F32,
                    w_dtype == NVFP4_DTYPE_F32, eps, g_inv, row_g, codes, scales};
  return hip_status(nvfp4::launch_add_rmsnorm_quant(a, as_stream(stream)), "add_rmsnorm launch");
}

int add_rmsnorm_nvfp4_quant(const void* x, int x_dtype, const void* residual, int residual_dtype, const void* w,
                            int w_dtype, double eps, int64_t M, int64_t K, const float* g_inv, void* residual_out,
                            uint8_t* codes, uint8_t* scales, void* stream) {
  if (M > 0 && K > 0 && !g_inv) return fail(NVFP4_ERR_INVALID_ARG, "null g_inv");
  return add_rmsnorm(x, x_dtype, residual, residual_dtype, w, w_dtype, eps, M, K, g_inv, nullptr, residual_out, codes,
                     scales, stream);
}

int add_rmsnorm_nvfp4_quant_per_token(const void* x, int x_dtype, const void* residual, int residual_dtype,
                                      const void* w, int w_dtype, double eps, int64_t M, int64_t K, void* residual_out,
                                      uint8_t* codes, uint8_t* scales, float* row_g, void* stream) {
  if (M > 0 && K > 0 && !row_g) return fail(NVFP4_ERR_INVALID_ARG, "null row_g");
  return add_rmsnorm(x, x_dtype, residual, residual_dtype, w, w_dtype, eps, M, K, nullptr, row_g, residual_out, codes,
                     scales, stream);
}

int nvfp4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t M, int64_t K, const float* g,
                     const float* row_g, void* out, int out_dtype, void* stream) {
  if (out_dtype != NVFP4_DTYPE_BF16 && out_dtype != NVFP4_DTYPE_F32)
    return fail(NVFP4_ERR_INVALID_ARG, "out_dtype must be BF16 or F32");
  if (!dim_ok(M) || K < 0 || K > kMaxDim || K % 16 != 0)
    return fail(NVFP4_ERR_INVALID_ARG, "need 0 <= M <= 2^24 and 0 <= K <= 2^24 a multiple of 16 (M=%lld K=%lld)",
                (long long)M, (long long)K);
  if (M * K == 0) { g_err[0] = '\0'; return NVFP4_OK; }
  if (!codes || !scales || !out) return fail(NVFP4_ERR_INVALID_ARG, "null pointer argument");
  if (!g == !row_g) return fail(NVFP4_ERR_INVALID_ARG, "give one of g and row_g");
  if (!aligned16(codes) || !aligned16(out)) return fail(NVFP4_ERR_INVALID_ARG, "codes and out must be 16-byte aligned");
  int st = check_device();
  if (st) return st;
  return hip_status(nvfp4::launch_dequantize(codes, scales, M, K, g, row_g, out, out_dtype == NVFP4_DTYPE_F32,
                                             as_stream(stream)), "dequantize launch");
}

// The cache of one layer: checked sizes.
static int cache_sizes(int64_t pages, int64_t page_size, int64_t heads, int64_t dim) {
  if (pages < 1 || pages > INT32_MAX) return fail(NVFP4_ERR_INVALID_ARG, "pages=%lld must be 1 to 2^31 - 1", (long long)pages);
  if (page_size < 16 || page_size > 65536 || page_size % 16 != 0)
    return fail(NVFP4_ERR_INVALID_ARG, "page_size=%lld must be a multiple of 16, at most 65536", (long long)page_size);
  if (pages * (page_size / 16) > INT32_MAX)
    return fail(NVFP4_ERR_INVALID_ARG, "the cache's pages must hold fewer than 2^35 tokens");
  if (heads < 1 || heads > 4096) return fail(NVFP4_ERR_INVALID_ARG, "heads=%lld must be 1 to 4096", (long long)heads);
  if (dim != 64 && dim != 128 && dim != 256)
    return fail(NVFP4_ERR_INVALID_ARG, "head_dim=%lld must be 64, 128 or 256", (long long)dim);
  return NVFP4_OK;
}

size_t nvfp4_kv_cache_bytes(int64_t pages, int64_t page_size, int64_t heads, int64_t head_dim) {
  if (cache_sizes(pages, page_size, heads, head_dim)) return 0;
  return (size_t)pages * heads * (page_size / 16) * 18 * head_dim;
}

int nvfp4_kv_write(const void* k, const void* v, int dtype, int64_t T, int64_t k_stride, int64_t v_stride,
                   const int64_t* slots, const float* k_g_inv, const float* v_g_inv, void* cache, int64_t pages,
                   int64_t page_size, int64_t heads, int64_t head_dim, void* stream) {
  if (dtype != NVFP4_DTYPE_BF16 && dtype != NVFP4_DTYPE_F32) return fail(NVFP4_ERR_INVALID_ARG, "dtype must be BF16 or F32");
  int st = cache_sizes(pages, page_size, heads, head_dim);
  if (st) return st;
  if (!dim_ok(T)) return fail(NVFP4_ERR_INVALID_ARG, "T=%lld out of range", (long long)T);
  if (T == 0) { g_err[0] = '\0'; return NVFP4_OK; }
  if (!k || !v || !slots || !k_g_inv || !v_g_inv || !cache) return fail(NVFP4_ERR_INVALID_ARG, "null pointer argument");
  const int64_t unit = dtype == NVFP4_DTYPE_F32 ? 4 : 8;
  for (int64_t s : {k_stride, v_stride})
    if (s % unit != 0 || s < (T > 1 ? heads * head_dim : 0) || s > (int64_t(1) << 40))
      return fail(NVFP4_ERR_INVALID_ARG, "token strides must be at least heads * head_dim and whole 16-byte units");
  if (!aligned16(k) || !aligned16(v) || !aligned16(cache) || reinterpret_cast<uintptr_t>(slots) % 8)
    return fail(NVFP4_ERR_INVALID_ARG, "k, v and cache must be 16-byte aligned, slots 8-byte");
  st = check_device();
  if (st) return st;
  const nvfp4::CacheArgs c{static_cast<uint8_t*>(cache), pages, (int)page_size, (int)heads, (int)head_dim};
  return hip_status(nvfp4::launch_kv_write(c, k, v, dtype == NVFP4_DTYPE_F32, T, k_stride, v_stride, slots, k_g_inv,
                                           v_g_inv, as_stream(stream)), "kv_write launch");
}

int nvfp4_kv_read(const void* cache, int64_t pages, int64_t page_size, int64_t heads, int64_t head_dim,
                  const int64_t* slots, int64_t T, const float* k_g, const float* v_g, void* k, void* v, int dtype,
                  void* stream) {
  if (dtype != NVFP4_DTYPE_BF16 && dtype != NVFP4_DTYPE_F32) return fail(NVFP4_ERR_INVALID_ARG, "dtype must be BF16 or F32");
  int st = cache_sizes(pages, page_size, heads, head_dim);
  if (st) return st;
  if (!dim_ok(T)) return fail(NVFP4_ERR_INVALID_ARG, "T=%lld out of range", (long long)T);
  if (T == 0) { g_err[0] = '\0'; return NVFP4_OK; }
  if (!k || !v || !slots || !k_g || !v_g || !cache) return fail(NVFP4_ERR_INVALID_ARG, "null pointer argument");
  if (!aligned16(k) || !aligned16(v) || !aligned16(cache) || reinterpret_cast<uintptr_t>(slots) % 8)
    return fail(NVFP4_ERR_INVALID_ARG, "k, v and cache must be 16-byte aligned, slots 8-byte");
  st = check_device();
  if (st) return st;
  const nvfp4::CacheArgs c{static_cast<uint8_t*>(const_cast<void*>(cache)), pages, (int)page_size, (int)heads, (int)head_dim};
  return hip_status(nvfp4::launch_kv_read(c, slots, T, k_g, v_g, k, v, dtype == NVFP4_DTYPE_F32, as_stream(stream)),
                    "kv_read launch");
}

// The arrival counters of split units come first in the workspace, in a
// region of one size for every call, so that calls of other sizes leave them
// zero. Only calls of fewer units than this split.
static constexpr int64_t kAttnCounters = 1024;

static int attn_sizes(int64_t T, int64_t B, int64_t heads_q, int64_t heads, int64_t head_dim, int64_t max_q,
                      int64_t max_len, int64_t window, nvfp4::AttnPlan& p) {
  int st = cache_sizes(1, 16, heads, head_dim);
  if (st) return st;
  if (heads_q < 1 || heads_q > 65536 || heads_q % heads != 0)
    return fail(NVFP4_ERR_INVALID_ARG, "heads_q=%lld must be a multiple of heads=%lld", (long long)heads_q, (long long)heads);
  if (!dim_ok(T) || !dim_ok(B) || !dim_ok(max_q)) return fail(NVFP4_ERR_INVALID_ARG, "T, B or max_q out of range");
  if (max_len < 0 || max_len > (int64_t(1) << 30)) return fail(NVFP4_ERR_INVALID_ARG, "max_len must be 0 to 2^30");
  if (window < 0 || window > (int64_t(1) << 30)) return fail(NVFP4_ERR_INVALID_ARG, "window must be 0 to 2^30");
  p = nvfp4::attn_plan(B, (int)heads_q, (int)heads, (int)head_dim, max_q, max_len, window);
  if (p.units > nvfp4::kAttnMaxUnits) return fail(NVFP4_ERR_INVALID_ARG, "too many sequences, heads and queries for one call");
  return NVFP4_OK;
}

size_t nvfp4_kv_attention_workspace_bytes(int64_t T, int64_t B, int64_t heads_q, int64_t heads, int64_t head_dim,
                                          int64_t max_q, int64_t max_len) {
  nvfp4::AttnPlan p;
  if (attn_sizes(T, B, heads_q, heads, head_dim, max_q, max_len, 0, p)) return 0;
  const int64_t floats = nvfp4::attn_workspace_floats(B, (int)heads_q, (int)heads, (int)head_dim, max_q, max_len);
  return kAttnCounters * sizeof(uint32_t) + align256((size_t)floats * sizeof(float));
}

int nvfp4_kv_attention(const uint16_t* q, int64_t q_stride, int64_t T, int64_t B, int64_t heads_q,
                       const int32_t* q_offsets, int64_t max_q, const void* cache, int64_t pages, int64_t page_size,
                       int64_t heads, int64_t head_dim, const int32_t* block_table, int64_t table_stride,
                       int64_t table_width, const int32_t* seq_lens, int64_t max_len, float scale, int64_t window,
                       const float* k_g, const float* v_g, void* ws, size_t ws_bytes, void* out, int out_dtype,
                       float* lse, void* stream) {
  if (out_dtype != NVFP4_DTYPE_BF16 && out_dtype != NVFP4_DTYPE_F32)
    return fail(NVFP4_ERR_INVALID_ARG, "out_dtype must be BF16 or F32");
  int st = cache_sizes(pages, page_size, heads, head_dim);
  if (st) return st;
  nvfp4::AttnPlan p;
  st = attn_sizes(T, B, heads_q, heads, head_dim, max_q, max_len, window, p);
  if (st) return st;
  if (table_width < 0 || table_width > (int64_t(1) << 26) || (B > 1 && table_stride < table_width))
    return fail(NVFP4_ERR_INVALID_ARG, "bad block table width or stride");
  if (T == 0 || B == 0 || max_q == 0) { g_err[0] = '\0'; return NVFP4_OK; }
  if (!q_offsets && T != B * max_q)
    return fail(NVFP4_ERR_INVALID_ARG, "without q_offsets T=%lld must be B * max_q = %lld", (long long)T, (long long)(B * max_q));
  if (!q || !cache || (!block_table && table_width > 0) || !seq_lens || !k_g || !v_g || !out)
    return fail(NVFP4_ERR_INVALID_ARG, "null pointer argument");
  if (q_stride % 8 != 0 || q_stride < (T > 1 ? heads_q * head_dim : 0) || q_stride > (int64_t(1) << 40))
    return fail(NVFP4_ERR_INVALID_ARG, "q's token stride must be at least heads_q * head_dim and a multiple of 8");
  if (!aligned16(q) || !aligned16(cache) || !aligned16(out))
    return fail(NVFP4_ERR_INVALID_ARG, "q, cache and out must be 16-byte aligned");
  const size_t need = nvfp4_kv_attention_workspace_bytes(T, B, heads_q, heads, head_dim, max_q, max_len);
  if (!ws || ws_bytes < need || !aligned16(ws))
    return fail(NVFP4_ERR_INVALID_ARG, "workspace of %zu bytes needed, 16-byte aligned (have %zu)", need, ws ? ws_bytes : (size_t)0);
  st = check_device();
  if (st) return st;
  nvfp4::AttnArgs a{};
  a.c = {static_cast<uint8_t*>(const_cast<void*>(cache)), pages, (int)page_size, (int)heads, (int)head_dim};
  a.q = q; a.q_stride = q_stride; a.T = T; a.B = B; a.heads_q = (int)heads_q; a.q_offsets = q_offsets; a.max_q = max_q;
  a.table = block_table; a.table_stride = table_stride; a.table_width = table_width; a.seq_lens = seq_lens;
  a.max_len = max_len; a.scale = scale; a.window = window; a.k_g = k_g; a.v_g = v_g; a.out = out;
  a.f32_out = out_dtype == NVFP4_DTYPE_F32; a.lse = lse;
  a.counters = static_cast<uint32_t*>(ws);
  a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kAttnCounters * sizeof(uint32_t));
  return hip_status(nvfp4::launch_kv_attention(a, p, as_stream(stream)), "kv_attention launch");
}

}  // extern "C"
