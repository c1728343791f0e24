// kv_attention_plan.h -- how a call of the attention over the paged NVFP4 cache
// is cut into workgroups, and the workspace its parts need: by host-side sizes
// alone, without HIP.
#pragma once
#include <stdint.h>

#include <initializer_list>

namespace nvfp4 {

// The split of a call, by its host-side sizes alone; units alone if there are
// more than kAttnMaxUnits.
constexpr int64_t kAttnMaxUnits = int64_t(1) << 23;
struct AttnPlan {
  bool tiled;       // kv_attention_tile.hip, else kv_attention.hip
  int row_tiles;    // 16-row tiles per workgroup, tiled: per wave
  int64_t units;    // row_blocks * B * heads
  int rows;         // of a workgroup
  int row_blocks;   // per (sequence, head)
  int chunk;        // keys per split
  int splits;       // most splits of one unit
  int part_floats;  // per (unit, split)
};
constexpr int attn_tile_max(int dim) { return dim == 64 ? 4 : 2; }  // most row tiles of a wave

// Workgroups of many rows that run at once; of few rows, the number aimed at
// (at most); keys of a split (at least, tiled and not); splits of a unit (at most).
constexpr int64_t attn_tile_slots(int dim) { return dim == 256 ? 256 : 512; }
constexpr int64_t kAttnSlots = 1024, kAttnTileKeys = 256, kAttnKeys = 512, kAttnMaxSplits = 256;

inline AttnPlan attn_plan(int64_t B, int heads_q, int heads, int dim, int64_t max_q, int64_t max_len, int64_t window) {
  AttnPlan p{};
  const int64_t G = heads_q / heads, rows = max_q * G;
  int64_t per, slots;  // rows of a workgroup, workgroups that fill the chip
  p.tiled = rows > 64;
  if (p.tiled) {
    slots = attn_tile_slots(dim);
    const int64_t most = 64 * attn_tile_max(dim);
    int64_t blocks = (rows + most - 1) / most;
    // Few workgroups: smaller ones, unless their rows pay for the keys' second
    // making (8 heads, group 8: 16 x 16000 keys 28.2 us with 64 rows, 32.4 with
    // 128; 128 tokens x 8192 keys 66 and 58 us).
    const int64_t keys = window > 0 && window + 64 < max_len ? window + 64 : max_len;
    if (blocks * B * heads < slots && (keys <= 2048 || rows <= 512)) blocks = (rows + 63) / 64;
    p.row_tiles = (int)((rows + 64 * blocks - 1) / (64 * blocks));
    per = 64 * p.row_tiles;
  } else {
    p.row_tiles = rows <= 16 ? 1 : 2;
    per = 16 * p.row_tiles;
    // Three workgroups a CU fit at D 128; a few more even out sequences of
    // unlike length, of which there are more the more sequences (4 x 131072
    // keys: 768 / 1024 122 / 137 us; 16 of up to 32000: 88 / 71 us).
    slots = (rows + per - 1) / per * B * heads <= 64 ? 768 : kAttnSlots;
  }
  const int64_t blocks = (rows + per - 1) / per;
  p.units = blocks * B * heads;
  if (p.units > kAttnMaxUnits) return p;
  p.row_blocks = (int)blocks;
  p.rows = (int)per;
  p.part_floats = (int)per * (dim + 2);
  // Keys that a unit reads at most, from a multiple of 32 on: its rows are of
  // at most (per - 1) / G + 2 queries. (With a window the more splits for all
  // max_q queries' keys are mostly empty: 1000 tokens of 2 sequences, 20 heads
  // on 4, window 128 take 24 us so, 51 with those.)
  int64_t span = max_len;
  int64_t queries = (per - 1) / G + 2;
  if (queries > max_q) queries = max_q;
  if (window > 0 && window + queries + 30 < span) span = window + queries + 30;
  span = (span + 31) / 32 * 32;
  // At least 512 keys a split: one token of 4 sequences of 8000 keys 15.4 us
  // so, 21.1 with 256 (16 heads of 128 a kv head). Tiled 256, as a workgroup
  // has more to do a key (16 tokens of one sequence of 1000 keys 15.2 us, 20.0).
  const int64_t least = p.tiled ? kAttnTileKeys : kAttnKeys;
  int64_t most = (span + least - 1) / least;
  if (most > kAttnMaxSplits) most = kAttnMaxSplits;
  int64_t want = 1;
  if (p.units > 0 && !p.tiled) {
    want = (slots + p.units - 1) / p.units;
  } else if (p.units > 0) {
    // As many splits as run in 1, 2, .. rounds of workgroups, whichever count
    // takes least time by this measure, in units of a tile: the tiles of a
    // workgroup, fewer for earlier queries, and 5 to begin and end, times the
    // rounds (where two share a CU, a last one of half the workgroups takes
    // 0.6); 8 for the join and 10 for a round's partials. D 128, 4 kv heads:
    // 70 row blocks over 30000 keys 931 / 793 / 616 us with 1 / 2 / 3 splits,
    // 79 over 8192 keys 248 / 251 / 226; 75 of 64 rows over 600 keys 21 / 35
    // with 1 / 2.
    const double unseen = 0.5 * (double)max_q / (double)(max_len > max_q ? max_len : max_q);
    const double tiles = (double)((span + 63) / 64) * (window > 0 ? 1.0 : 1.0 - unseen);
    double least_cost = 0.0;
    for (int64_t rounds = (p.units + slots - 1) / slots, n = 0; n < 4; ++rounds, ++n) {
      int64_t w = rounds * slots / p.units;
      if (w > most) w = most;
      if (w < 1) w = 1;
      const int64_t full = p.units * w / slots, rest = p.units * w % slots;
      const double turns = (double)full + (rest == 0 ? 0.0 : dim != 256 && 2 * rest <= slots ? 0.6 : 1.0);
      const double cost = turns * (tiles / w + 5.0) + (w > 1 ? 8.0 + 10.0 * p.units * w / slots : 0.0);
      if (n == 0 || cost < least_cost) { least_cost = cost; want = w; }
    }
  }
  if (want > most) want = most;
  if (want < 1) want = 1;
  p.chunk = (int)(((span + want - 1) / want + 127) / 128 * 128);
  if (p.chunk < 128) p.chunk = 128;
  p.splits = span > 0 ? (int)((span + p.chunk - 1) / p.chunk) : 1;
  return p;
}

// Floats of the partials of any call of at most B sequences, max_q queries of
// each and max_len keys, with any window: at least units * splits * part_floats
// of all their plans that split, and itself never less for larger sizes.
//   Few rows: splits <= slots / units rounded up, slots <= kAttnSlots, so
//   units * splits < units + kAttnSlots, and units < kAttnSlots or splits = 1.
//   Tiled, S = attn_tile_slots: splits <= (r + 3) S / units, r = units / S
//   rounded up, so units * splits <= units + 4 S; two splits or more need
//   (r + 3) S >= 2 units > 2 (r - 1) S, thus r <= 4 and units * splits <= 7 S.
// No unit has more splits than its keys give.
inline int64_t attn_workspace_floats(int64_t B, int heads_q, int heads, int dim, int64_t max_q, int64_t max_len) {
  const int64_t rows = max_q * (heads_q / heads), groups = B * heads;
  auto least = [](int64_t a, int64_t b) { return a < b ? a : b; };
  auto splits = [&](int64_t keys) {
    const int64_t n = least(((max_len + 31) / 32 * 32 + keys - 1) / keys, kAttnMaxSplits);
    return n > 1 ? n : 0;
  };
  const int64_t units = groups * (rows > 32 ? 2 : 1);
  int64_t floats = least(units * splits(kAttnKeys), kAttnSlots + least(units, kAttnSlots)) * (rows > 16 ? 32 : 16);
  if (rows > 64) {
    // Row blocks of 64 rows and, separately, of as many as a workgroup takes.
    const int64_t slots = attn_tile_slots(dim);
    for (int64_t per : {64, 64 * attn_tile_max(dim)}) {
      const int64_t u = least(groups * ((rows + per - 1) / per), 8 * slots);
      const int64_t n = least(u * splits(kAttnTileKeys), least(u + 4 * slots, 7 * slots)) * per;
      if (n > floats) floats = n;
    }
  }
  return floats * (dim + 2);
}

}  // namespace nvfp4
