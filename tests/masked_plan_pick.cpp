// The plan of one call of masked attention, on the host.
#include "../nvfp4_quantized_dense_amd/csrc/kv_attention_plan.h"

// out: tiled, rows of a workgroup, splits, packed, chunk, units.
extern "C" void pick(int64_t B, int heads_q, int heads, int dim, int64_t max_q, int64_t max_len, int64_t window, int64_t sinks,
                     int tree, int64_t T, int64_t* out) {
  const nvfp4::AttnPlan p = nvfp4::attn_masked_plan(B, heads_q, heads, dim, max_q, max_len, window, sinks, tree != 0, T);
  const int64_t v[] = {p.tiled, p.rows, p.splits, p.packed, p.chunk, p.units};
  for (int i = 0; i < 6; ++i) out[i] = v[i];
}
