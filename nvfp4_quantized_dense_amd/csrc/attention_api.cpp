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

// Rows of keys and values on their way into the cache.
static int kv_rows(const void* k, const void* v, int dtype, int64_t T, int64_t k_stride, int64_t v_stride, const int64_t* slots,
                   const float* k_g_inv, const float* v_g_inv, const void* cache, int64_t heads, int64_t head_dim) {
  if (dtype != NVFP4_DTYPE_BF16 && dtype != NVFP4_DTYPE_F32) return fail(NVFP4_ERR_INVALID_ARG, "dtype must be BF16 or F32");
  if (!dim_ok(T)) return fail(NVFP4_ERR_INVALID_ARG, "T=%lld out of range", (long long)T);
  if (T == 0) return NVFP4_OK;
  if (!k || !v || !slots || !k_g_inv || !v_g_inv || !cache) return fail(NVFP4_ERR_INVALID_ARG, "null pointer argument");
  const int64_t unit = dtype == NVFP4_DTYPE_F32 ? 4 : 8;
  for (int64_t s : {k_stride, v_stride})
    if (s % unit != 0 || s < (T > 1 ? heads * head_dim : 0) || s > (int64_t(1) << 40))
      return fail(NVFP4_ERR_INVALID_ARG, "token strides must be at least heads * head_dim and whole 16-byte units");
  if (!aligned16(k) || !aligned16(v) || !aligned16(cache) || reinterpret_cast<uintptr_t>(slots) % 8)
    return fail(NVFP4_ERR_INVALID_ARG, "k, v and cache must be 16-byte aligned, slots 8-byte");
  return NVFP4_OK;
}

int nvfp4_kv_write(const void* k, const void* v, int dtype, int64_t T, int64_t k_stride, int64_t v_stride,
                   const int64_t* slots, const float* k_g_inv, const float* v_g_inv, void* cache, int64_t pages,
                   int64_t page_size, int64_t heads, int64_t head_dim, void* stream) {
  int st = cache_sizes(pages, page_size, heads, head_dim);
  if (st) return st;
  st = kv_rows(k, v, dtype, T, k_stride, v_stride, slots, k_g_inv, v_g_inv, cache, heads, head_dim);
  if (st) return st;
  if (T == 0) { g_err[0] = '\0'; return NVFP4_OK; }
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
                      int64_t max_len, int64_t window, int64_t sinks, bool tree, int64_t rows, nvfp4::AttnPlan& p) {
  int st = cache_sizes(1, 16, heads, head_dim);
  if (st) return st;
  if (heads_q < 1 || heads_q > 65536 || heads_q % heads != 0)
    return fail(NVFP4_ERR_INVALID_ARG, "heads_q=%lld must be a multiple of heads=%lld", (long long)heads_q, (long long)heads);
  if (!dim_ok(T) || !dim_ok(B) || !dim_ok(max_q)) return fail(NVFP4_ERR_INVALID_ARG, "T, B or max_q out of range");
  if (max_len < 0 || max_len > (int64_t(1) << 30)) return fail(NVFP4_ERR_INVALID_ARG, "max_len must be 0 to 2^30");
  if (window < 0 || window > (int64_t(1) << 30)) return fail(NVFP4_ERR_INVALID_ARG, "window must be 0 to 2^30");
  if (sinks < 0 || sinks > (int64_t(1) << 30)) return fail(NVFP4_ERR_INVALID_ARG, "sinks must be 0 to 2^30");
  if (sinks > 0 || tree) {
    p = nvfp4::attn_masked_plan(B, (int)heads_q, (int)heads, (int)head_dim, max_q, max_len, window, sinks, tree, rows);
  } else {
    p = nvfp4::attn_plan(B, (int)heads_q, (int)heads, (int)head_dim, max_q, max_len, window);
  }
  if (p.units > nvfp4::kAttnMaxUnits) return fail(NVFP4_ERR_INVALID_ARG, "too many sequences, heads and queries for one call");
  return NVFP4_OK;
}

size_t nvfp4_kv_attention_workspace_bytes(int64_t T, int64_t B, int64_t heads_q, int64_t heads, int64_t head_dim,
                                          int64_t max_q, int64_t max_len) {
  nvfp4::AttnPlan p;
  if (attn_sizes(T, B, heads_q, heads, head_dim, max_q, max_len, 0, 0, false, 0, p)) return 0;
  const int64_t floats = nvfp4::attn_workspace_floats(B, (int)heads_q, (int)heads, (int)head_dim, max_q, max_len);
  return kAttnCounters * sizeof(uint32_t) + align256((size_t)floats * sizeof(float));
}

int nvfp4_kv_attention(const uint16_t* q, int64_t q_stride, int64_t T, int64_t B, int64_t heads_q,
                       const int32_t* q_offsets, int64_t max_q, const void* cache, int64_t pages, int64_t page_size,
                       int64_t heads, int64_t head_dim, const int32_t* block_table, int64_t table_stride,
                       int64_t table_width, const int32_t* seq_lens, int64_t max_len, float scale, int64_t window,
                       const float* k_g, const float* v_g, void* ws, size_t ws_bytes, void* out, int out_dtype,
                       float* lse, void* stream) {
  return nvfp4_kv_attention_masked(q, q_stride, T, B, heads_q, q_offsets, max_q, cache, pages, page_size, heads, head_dim,
                                   block_table, table_stride, table_width, seq_lens, max_len, scale, window, 0, nullptr, 0,
                                   k_g, v_g, ws, ws_bytes, out, out_dtype, lse, stream);
}

int nvfp4_kv_attention_masked(const uint16_t* q, int64_t q_stride, int64_t T, int64_t B, int64_t heads_q,
                              const int32_t* q_offsets, int64_t max_q, const void* cache, int64_t pages, int64_t page_size,
                              int64_t heads, int64_t head_dim, const int32_t* block_table, int64_t table_stride,
                              int64_t table_width, const int32_t* seq_lens, int64_t max_len, float scale, int64_t window,
                              int64_t sinks, const uint64_t* tree, int64_t tree_words, const float* k_g, const float* v_g,
                              void* ws, size_t ws_bytes, void* out, int out_dtype, float* lse, void* stream) {
  if (out_dtype != NVFP4_DTYPE_BF16 && out_dtype != NVFP4_DTYPE_F32)
    return fail(NVFP4_ERR_INVALID_ARG, "out_dtype must be BF16 or F32");
  int st = cache_sizes(pages, page_size, heads, head_dim);
  if (st) return st;
  if (window == 0 && sinks > 0 && sinks <= (int64_t(1) << 30)) sinks = 0;  // nothing to keep
  nvfp4::AttnPlan p;
  st = attn_sizes(T, B, heads_q, heads, head_dim, max_q, max_len, window, sinks, tree != nullptr, q_offsets ? T : 0, p);
  if (st) return st;
  if (tree) {
    if (max_q > nvfp4::kMaxTree || tree_words < (max_q + 63) / 64 || tree_words > nvfp4::kMaxTree / 64)
      return fail(NVFP4_ERR_INVALID_ARG, "tree needs max_q <= %lld and ceil(max_q / 64) to %lld words a row (max_q=%lld words=%lld)",
                  (long long)nvfp4::kMaxTree, (long long)(nvfp4::kMaxTree / 64), (long long)max_q, (long long)tree_words);
    if (window > 0 && window < max_q)
      return fail(NVFP4_ERR_INVALID_ARG, "with a tree window=%lld must be 0 or at least max_q=%lld", (long long)window, (long long)max_q);
    if (reinterpret_cast<uintptr_t>(tree) % 8) return fail(NVFP4_ERR_INVALID_ARG, "tree must be 8-byte aligned");
  }
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
  a.max_len = max_len; a.scale = scale; a.window = window;
  a.sinks = sinks; a.tree = tree; a.tree_words = (int)tree_words; a.k_g = k_g; a.v_g = v_g; a.out = out;
  a.f32_out = out_dtype == NVFP4_DTYPE_F32; a.lse = lse;
  a.counters = static_cast<uint32_t*>(ws);
  a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kAttnCounters * sizeof(uint32_t));
  return hip_status(nvfp4::launch_kv_attention(a, p, as_stream(stream)), "kv_attention launch");
}

int nvfp4_tree_mask(const int32_t* parents, int64_t T, int64_t B, const int32_t* q_offsets, int64_t max_q, uint64_t* tree,
                    int64_t tree_words, int32_t* positions, void* stream) {
  if (!dim_ok(T) || !dim_ok(B)) return fail(NVFP4_ERR_INVALID_ARG, "T or B out of range");
  if (max_q < 0 || max_q > nvfp4::kMaxTree || tree_words < (max_q + 63) / 64 || tree_words > nvfp4::kMaxTree / 64)
    return fail(NVFP4_ERR_INVALID_ARG, "need max_q <= %lld and ceil(max_q / 64) to %lld words a row (max_q=%lld words=%lld)",
                (long long)nvfp4::kMaxTree, (long long)(nvfp4::kMaxTree / 64), (long long)max_q, (long long)tree_words);
  if (T == 0 || B == 0 || max_q == 0) { g_err[0] = '\0'; return NVFP4_OK; }
  if (!q_offsets && T != B * max_q)
    return fail(NVFP4_ERR_INVALID_ARG, "without q_offsets T=%lld must be B * max_q = %lld", (long long)T, (long long)(B * max_q));
  if (!parents || !tree) return fail(NVFP4_ERR_INVALID_ARG, "null pointer argument");
  if (reinterpret_cast<uintptr_t>(tree) % 8) return fail(NVFP4_ERR_INVALID_ARG, "tree must be 8-byte aligned");
  int st = check_device();
  if (st) return st;
  const nvfp4::TreeArgs a{parents, q_offsets, T, max_q, tree, (int)tree_words, positions};
  return hip_status(nvfp4::launch_tree_mask(a, B, as_stream(stream)), "tree_mask launch");
}

// The part of a rotation's arguments that its two entry points share.
static int rope_args(nvfp4::RopeArgs& r, const void* x, int x_dtype, int64_t x_stride, int64_t T, int64_t heads, int64_t dim,
                     const int32_t* positions, int64_t axis_stride, int64_t axes, const float* inv_freq, const int32_t* axis,
                     int64_t rotary, int pairs, double factor, void* out, int out_dtype, int64_t out_stride) {
  for (int d : {x_dtype, out_dtype})
    if (d != NVFP4_DTYPE_BF16 && d != NVFP4_DTYPE_F32) return fail(NVFP4_ERR_INVALID_ARG, "dtypes must be BF16 or F32");
  if (!dim_ok(T)) return fail(NVFP4_ERR_INVALID_ARG, "T=%lld out of range", (long long)T);
  if (heads < 0 || heads > 65536) return fail(NVFP4_ERR_INVALID_ARG, "heads=%lld must be at most 65536", (long long)heads);
  if (dim < 8 || dim > 1024 || dim % 8 != 0)
    return fail(NVFP4_ERR_INVALID_ARG, "head_dim=%lld must be a multiple of 8, at most 1024", (long long)dim);
  if (rotary < 16 || rotary > dim || rotary > 512 || rotary % 16 != 0)
    return fail(NVFP4_ERR_INVALID_ARG, "rotary=%lld must be a multiple of 16, at most head_dim and 512", (long long)rotary);
  if (axes < 1 || axes > 16) return fail(NVFP4_ERR_INVALID_ARG, "axes=%lld must be 1 to 16", (long long)axes);
  if (pairs != NVFP4_ROPE_HALVES && pairs != NVFP4_ROPE_NEIGHBOURS) return fail(NVFP4_ERR_INVALID_ARG, "bad pairs");
  if (!(factor - factor == 0.0)) return fail(NVFP4_ERR_INVALID_ARG, "factor must be finite");
  if (axis_stride < 0 || axis_stride > (int64_t(1) << 40)) return fail(NVFP4_ERR_INVALID_ARG, "bad axis stride");
  if (T == 0) return NVFP4_OK;
  if ((heads > 0 && (!x || !out)) || !positions || !inv_freq) return fail(NVFP4_ERR_INVALID_ARG, "null pointer argument");
  if (!aligned16(x) || !aligned16(out)) return fail(NVFP4_ERR_INVALID_ARG, "rows must be 16-byte aligned");
  const int64_t unit[2] = {x_dtype == NVFP4_DTYPE_F32 ? 4 : 8, out_dtype == NVFP4_DTYPE_F32 ? 4 : 8}, stride[2] = {x_stride, out_stride};
  for (int i = 0; i < 2; ++i)
    if (stride[i] % unit[i] != 0 || stride[i] < (T > 1 ? heads * dim : 0) || stride[i] > (int64_t(1) << 40))
      return fail(NVFP4_ERR_INVALID_ARG, "token strides must be at least heads * head_dim and whole 16-byte units");
  if (x == out && heads > 0 && (x_dtype != out_dtype || x_stride != out_stride))
    return fail(NVFP4_ERR_INVALID_ARG, "in place, both sides must have one type and stride");
  r = {x, x_stride, x_dtype == NVFP4_DTYPE_F32, out, out_stride, out_dtype == NVFP4_DTYPE_F32, T, (int)heads, (int)dim, positions,
       axis_stride, (int)axes, inv_freq, axis, (int)rotary, pairs == NVFP4_ROPE_NEIGHBOURS, factor};
  return NVFP4_OK;
}

int nvfp4_rope(const void* x, int x_dtype, int64_t x_stride, int64_t T, int64_t heads, int64_t head_dim,
               const int32_t* positions, int64_t axis_stride, int64_t axes, const float* inv_freq, const int32_t* axis,
               int64_t rotary, int pairs, double factor, void* out, int out_dtype, int64_t out_stride, void* stream) {
  nvfp4::RopeArgs r{};
  int st = rope_args(r, x, x_dtype, x_stride, T, heads, head_dim, positions, axis_stride, axes, inv_freq, axis, rotary, pairs,
                     factor, out, out_dtype, out_stride);
  if (st) return st;
  if (T == 0 || heads == 0) { g_err[0] = '\0'; return NVFP4_OK; }
  st = check_device();
  if (st) return st;
  return hip_status(nvfp4::launch_rope(r, as_stream(stream)), "rope launch");
}

int nvfp4_rope_kv_write(const void* q, int64_t q_stride, int64_t heads_q, const void* k, const void* v, int dtype, int64_t T,
                        int64_t k_stride, int64_t v_stride, const int32_t* positions, int64_t axis_stride, int64_t axes,
                        const float* inv_freq, const int32_t* axis, int64_t rotary, int pairs, double factor,
                        const int64_t* slots, const float* k_g_inv, const float* v_g_inv, void* cache, int64_t pages,
                        int64_t page_size, int64_t heads, int64_t head_dim, void* q_out, int q_out_dtype, int64_t q_out_stride,
                        void* stream) {
  int st = cache_sizes(pages, page_size, heads, head_dim);
  if (st) return st;
  nvfp4::RopeArgs r{};
  st = rope_args(r, q, dtype, q_stride, T, heads_q, head_dim, positions, axis_stride, axes, inv_freq, axis, rotary, pairs, factor,
                 q_out, q_out_dtype, q_out_stride);
  if (st) return st;
  st = kv_rows(k, v, dtype, T, k_stride, v_stride, slots, k_g_inv, v_g_inv, cache, heads, head_dim);
  if (st) return st;
  if (T == 0) { g_err[0] = '\0'; return NVFP4_OK; }
  st = check_device();
  if (st) return st;
  const nvfp4::CacheArgs c{static_cast<uint8_t*>(cache), pages, (int)page_size, (int)heads, (int)head_dim};
  return hip_status(nvfp4::launch_rope_kv_write(r, c, k, v, k_stride, v_stride, slots, k_g_inv, v_g_inv, as_stream(stream)),
                    "rope_kv_write launch");
}

static int pool_pages(int64_t pages) {
  if (pages < 1 || pages >= (int64_t(1) << 30)) return fail(NVFP4_ERR_INVALID_ARG, "pages=%lld must be 1 to 2^30 - 1", (long long)pages);
  return NVFP4_OK;
}

size_t nvfp4_kv_pool_bytes(int64_t pages) {
  if (pool_pages(pages)) return 0;
  return ((size_t)pages + nvfp4::kPoolHead) * sizeof(int32_t);
}

int nvfp4_kv_pool_reset(void* pool, int64_t pages, void* stream) {
  int st = pool_pages(pages);
  if (st) return st;
  if (!pool || !aligned16(pool)) return fail(NVFP4_ERR_INVALID_ARG, "pool must not be null, 16-byte aligned");
  st = check_device();
  if (st) return st;
  return hip_status(nvfp4::launch_kv_pool_reset(static_cast<int32_t*>(pool), pages, as_stream(stream)), "kv_pool_reset launch");
}

int nvfp4_kv_advance(const int32_t* counts, int64_t B, int32_t* seq_lens, int32_t* block_table, int64_t table_stride,
                     int64_t table_width, int64_t page_size, void* pool, int64_t pages, int64_t T,
                     const int32_t* position_offsets, int32_t* q_offsets, int64_t* slots, int32_t* positions, void* stream) {
  int st = pool_pages(pages);
  if (st) return st;
  st = cache_sizes(pages, page_size, 1, 64);
  if (st) return st;
  if (B < 0 || B > 65536) return fail(NVFP4_ERR_INVALID_ARG, "B=%lld must be 0 to 65536", (long long)B);
  if (!dim_ok(T)) return fail(NVFP4_ERR_INVALID_ARG, "T=%lld out of range", (long long)T);
  if (table_width < 0 || table_width > (int64_t(1) << 26) || (B > 1 && table_stride < table_width) || table_stride > (int64_t(1) << 40))
    return fail(NVFP4_ERR_INVALID_ARG, "bad block table width or stride");
  if ((B > 0 && (!counts || !seq_lens || (!block_table && table_width > 0))) || !pool)
    return fail(NVFP4_ERR_INVALID_ARG, "null pointer argument");
  if (!aligned16(pool) || reinterpret_cast<uintptr_t>(slots) % 8) return fail(NVFP4_ERR_INVALID_ARG, "pool must be 16-byte aligned, slots 8-byte");
  st = check_device();
  if (st) return st;
  const nvfp4::AdvanceArgs a{counts, B, seq_lens, block_table, table_stride, (int)table_width, (int)page_size,
                             static_cast<int32_t*>(pool), (int)pages, (int)T, position_offsets, q_offsets, slots, positions};
  return hip_status(nvfp4::launch_kv_advance(a, as_stream(stream)), "kv_advance launch");
}

}  // extern "C"
