// Plans of masked attention of random sizes, on the host: the splits of every
// row block's walk over sinks and window are among the plan's, and their
// partials fit the workspace.
#include "../nvfp4_quantized_dense_amd/csrc/kv_attention_plan.h"

#include <cmath>
#include <random>

using namespace nvfp4;

// 0, or what failed (1 the workspace, 2 more splits than planned, 3 arrivals
// without counters, 4 and 5 packed blocks) with the sizes in `at`: B, heads_q, heads, dim, max_q,
// max_len, window, sinks, tree, T. `used`: plans that split a walk with a gap.
extern "C" int scan(int seed, int n, int64_t* at, int64_t* used) {
  std::mt19937_64 rng(seed);
  auto spread = [&](double most) { return (int64_t)std::exp(std::uniform_real_distribution<double>(0, std::log(most))(rng)); };
  *used = 0;
  for (int k = 0; k < n; ++k) {
    const int heads = (int)spread(33), group = (int)spread(65), dim = 64 << (rng() % 3);
    const bool tree = rng() % 2;
    const int64_t B = spread(600), q = spread(4000), len = spread(300000), sinks = spread(3000);
    int64_t window = rng() % 4 ? spread(100000) : 0;
    if (tree && window > 0 && window < q) window = q;
    const int64_t T = rng() % 2 ? 1 + rng() % (B * q) : 0;  // of a ragged batch
    const AttnPlan p = attn_masked_plan(B, heads * group, heads, dim, q, len, window, sinks, tree, T);
    if (p.units > kAttnMaxUnits) continue;
    const int64_t sizes[] = {B, heads * group, heads, dim, q, len, window, sinks, tree, T};
    for (int i = 0; i < 10; ++i) at[i] = sizes[i];
    const int64_t have = attn_workspace_floats(B, heads * group, heads, dim, q, len);
    if (p.splits > 1 && p.units * p.splits * p.part_floats > have) return 1;
    if (!p.tiled && p.splits > 1 && p.units >= 1024) return 3;
    // Packed blocks: each sequence's begin behind the one before it, in all no more than planned.
    if (p.packed) {
      int64_t left = T, first = 0, end = 0;
      for (int64_t b = 0; b < B; ++b) {
        const int64_t mine = b + 1 < B ? (rng() % 3 ? rng() % (2 * left / (B - b) + 1) : 0) : left, n = mine < left ? mine : left;
        const int64_t at = attn_first_block(first, b, group, p.rows);
        if (at < end) return 4;
        end = at + ((n < q ? n : q) * group + p.rows - 1) / p.rows;
        first += n;
        left -= n;
      }
      if (end > p.row_blocks) return 5;
    }
    // A sequence of L keys and m queries: the walk of each of a few row blocks.
    for (int trial = 0; trial < 8; ++trial) {
      const int64_t L = trial ? len - rng() % len : len, m = trial % 3 ? 1 + rng() % q : q + (trial ? rng() % 50 : 0);
      const int64_t rows = (m < q ? m : q) * group, block = rng() % ((q * group + p.rows - 1) / p.rows);
      if (block * p.rows >= rows) continue;
      const int64_t last = block * p.rows + p.rows < rows ? block * p.rows + p.rows - 1 : rows - 1;
      auto hi_of = [&](int64_t i) { return L - m + i + 1 < 0 ? 0 : L - m + i + 1; };
      const int64_t hi = tree ? hi_of((m < q ? m : q) - 1) : hi_of(last / group), h0 = hi_of(tree ? 0 : block * p.rows / group);
      const int64_t lo = window > 0 && h0 > window ? h0 - window : 0, from = lo & ~int64_t(31);
      const int64_t head = sinks < from ? (sinks + 31) & ~int64_t(31) : from, end = hi - (from - head);
      const int64_t splits = end > 0 ? (end + p.chunk - 1) / p.chunk : 1;
      if (splits > p.splits) return 2;
      if (splits > 1 && from > head && head > 0) ++*used;
    }
  }
  return 0;
}
