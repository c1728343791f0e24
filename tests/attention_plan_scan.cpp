// Plans of random sizes against the workspace's bound, on the host.
#include "../nvfp4_quantized_dense_amd/csrc/kv_attention_plan.h"

#include <cmath>
#include <random>

using namespace nvfp4;

// 0, or which check failed (1 the workspace is too small for a plan, 2 for a
// plan of smaller sizes, 3 it shrinks with larger sizes, 4 a plan that counts
// arrivals has more units than counters, 5 splits do not cover the keys) with
// the sizes in `at`: B, heads_q, heads, dim, max_q, max_len, window. `tight`:
// the largest share of a workspace that a plan used.
extern "C" int scan(int seed, int n, int64_t* at, double* tight) {
  std::mt19937_64 rng(seed);
  auto spread = [&](double most) { return (int64_t)std::exp(std::uniform_real_distribution<double>(0, std::log(most))(rng)); };
  *tight = 0.0;
  for (int i = 0; i < n; ++i) {
    const int heads = (int)spread(33), group = (int)spread(65), dim = 64 << (rng() % 3);
    const int64_t B = spread(600), q = spread(4000), len = spread(300000), window = rng() % 2 ? spread(100000) : 0;
    const AttnPlan p = attn_plan(B, heads * group, heads, dim, q, len, window);
    if (p.units > kAttnMaxUnits) continue;
    int64_t sizes[] = {B, heads * group, heads, dim, q, len, window};
    for (int k = 0; k < 7; ++k) at[k] = sizes[k];
    const int64_t have = attn_workspace_floats(B, heads * group, heads, dim, q, len);
    auto need = [](const AttnPlan& x) { return x.splits > 1 ? x.units * x.splits * x.part_floats : int64_t(0); };
    if (need(p) > have) return 1;
    if (have > 0 && (double)need(p) / have > *tight) *tight = (double)need(p) / have;
    const int64_t b1 = B - rng() % B, q1 = q - rng() % q, l1 = len - rng() % len;
    if (need(attn_plan(b1, heads * group, heads, dim, q1, l1, window)) > have) return 2;
    if (attn_workspace_floats(b1, heads * group, heads, dim, q1, l1) > have) return 3;
    if (!p.tiled && p.splits > 1 && p.units >= 1024) return 4;
    const int64_t span = window > 0 && window + q + 30 < len ? 0 : len;  // without a window, all keys
    if (window == 0 && (int64_t)p.splits * p.chunk < span) return 5;
  }
  return 0;
}
