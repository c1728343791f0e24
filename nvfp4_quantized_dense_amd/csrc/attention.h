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

// Turns the pairs of channels of x by angles positions[axis[i]] * inv_freq[i].
struct RopeArgs {
  const void* x;             // [T, heads, dim], token stride in elements
  int64_t x_stride;
  bool x_f32;
  void* out;                 // [T, heads, dim], may be x
  int64_t out_stride;
  bool out_f32;
  int64_t T;
  int heads, dim;
  const int32_t* positions;  // [axes, T], axis stride in elements
  int64_t axis_stride;
  int axes;
  const float* inv_freq;     // [rotary / 2]
  const int32_t* axis;       // [rotary / 2], or null: axis 0
  int rotary;                // channels turned, a multiple of 16
  bool neighbours;           // pairs (2 i, 2 i + 1), else (i, i + rotary / 2)
  double factor;             // of cosine and sine
};
hipError_t launch_rope(const RopeArgs& r, hipStream_t s);
// launch_rope of the queries, and launch_kv_write with the keys turned.
hipError_t launch_rope_kv_write(const RopeArgs& r, const CacheArgs& c, const void* k, const void* v, int64_t k_stride,
                                int64_t v_stride, const int64_t* slots, const float* k_g_inv, const float* v_g_inv,
                                hipStream_t s);

// The pool of free pages: int32 [4 + pages], free pages, status, arrivals, 0,
// then a stack of free pages.
constexpr int kPoolHead = 4;
struct AdvanceArgs {
  const int32_t* counts;     // [B]
  int64_t B;
  int32_t* seq_lens;         // [B]
  int32_t* table;            // [B, table_width], row stride table_stride
  int64_t table_stride;
  int table_width, page_size;
  int32_t* pool;
  int pages;
  int T;                     // rows of slots and positions
  const int32_t* offsets;    // [B] added to positions, or null
  int32_t* q_offsets;        // [B + 1] or null
  int64_t* slots;            // [T] or null
  int32_t* positions;        // [T] or null
};
hipError_t launch_kv_pool_reset(int32_t* pool, int64_t pages, hipStream_t s);
hipError_t launch_kv_advance(const AdvanceArgs& a, hipStream_t s);

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
  int64_t sinks;             // first keys that stay visible behind a window
  const uint64_t* tree;      // [T, tree_words] drafted keys a query sees, or null: causal
  int tree_words;
};
// Whether a call needs the masked kernels.
inline bool attn_masked(const AttnArgs& a) { return a.sinks > 0 || a.tree != nullptr; }
hipError_t launch_kv_attention(const AttnArgs& a, const AttnPlan& p, hipStream_t s);
struct TreeArgs {
  const int32_t* parents;    // [T], by number in the sequence's draft; none below 0 or from the own number on
  const int32_t* q_offsets;  // [B + 1], or null: max_q each
  int64_t T, max_q;
  uint64_t* tree;            // [T, tree_words]
  int tree_words;
  int32_t* positions;        // [T]: become the first row's plus the depth; or null
};
constexpr int64_t kMaxTree = 4096;  // most drafted tokens of a sequence
hipError_t launch_tree_mask(const TreeArgs& a, int64_t B, hipStream_t s);
// kv_attention_tile.hip
hipError_t launch_kv_attention_tile(const AttnArgs& a, const AttnPlan& p, hipStream_t s);

}  // namespace nvfp4
