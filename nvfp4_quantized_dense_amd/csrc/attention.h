// attention.h -- host-side launchers of the attention half of a decoder
// layer: norm + quantize, dequantize, the paged NVFP4 cache and the attention
// that reads it (internal interface, arguments validated by the caller).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kv_attention_plan.h"

namespace nvfp4 {

// norm_quant.hip
struct NormArgs {
  const void* x;           // [M, K], bf16 or f32
  const void* residual;    // [M, K] of res_f32's type, or null
  const void* w;           // [K], bf16 or f32
  void* residual_out;      // [M, K] of the residual's type (x's type without one), or null
  int64_t M, K;
  bool x_f32, res_f32, w_f32;
  double eps;
  const float* g_inv;      // static scale, or null: per token
  float* row_g;            // per token: [M]
  uint8_t* codes;
  uint8_t* scales;
};
hipError_t launch_add_rmsnorm_quant(const NormArgs& a, hipStream_t s);
// out[m, k] = E2M1 * E4M3 * g, g = *g or row_g[m].
hipError_t launch_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t M, int64_t K, const float* g,
                             const float* row_g, void* out, bool f32_out, hipStream_t s);

// The paged cache of one layer: pages x heads x (page_size / 16) records of
// 18 * dim bytes (kv_layout.h).
struct CacheArgs {
  uint8_t* cache;
  int64_t pages;
  int page_size, heads, dim;
};

// kv_cache.hip
hipError_t launch_kv_write(const CacheArgs& c, const void* k, const void* v, bool f32_in, int64_t T, int64_t k_stride,
                           int64_t v_stride, const int64_t* slots, const float* k_g_inv, const float* v_g_inv,
                           hipStream_t s);
hipError_t launch_kv_read(const CacheArgs& c, const int64_t* slots, int64_t T, const float* k_g, const float* v_g,
                          void* k, void* v, bool f32_out, hipStream_t s);

// kv_attention.hip
struct AttnArgs {
  CacheArgs c;
  const uint16_t* q;         // bf16, token stride q_stride, heads and channels dense
  int64_t q_stride;
  int64_t T, B;
  int heads_q;
  const int32_t* q_offsets;  // [B + 1], or null: T / B queries each
  int64_t max_q;
  const int32_t* table;      // [B, table_width], row stride table_stride
  int64_t table_stride, table_width;
  const int32_t* seq_lens;   // [B]
  int64_t max_len;
  float scale;
  int64_t window;            // 0: none
  const float* k_g;
  const float* v_g;
  void* out;                 // [T, heads_q, dim] bf16 or f32
  bool f32_out;
  float* lse;                // [T, heads_q] or null
  float* part;               // split partials
  uint32_t* counters;        // one per (row block, head, sequence), zero
};
hipError_t launch_kv_attention(const AttnArgs& a, const AttnPlan& p, hipStream_t s);
// kv_attention_tile.hip
hipError_t launch_kv_attention_tile(const AttnArgs& a, const AttnPlan& p, hipStream_t s);

}  // namespace nvfp4
