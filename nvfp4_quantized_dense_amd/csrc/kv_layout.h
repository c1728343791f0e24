// kv_layout.h -- the paged NVFP4 cache. A record holds 16 tokens of one head
// (18 * D bytes, D channels), in four parts:
//   K codes  [4 g][16 t][D/8]       token t, channels g D/4 + [0, D/4), two
//                                   per byte, low nibble first
//   V codes  [4 g][16 c][D/16 b][2] channel 16 b + c, tokens 4 g + {0, 1} and
//                                   4 g + {2, 3}, low nibble first
//   K scales [4 g][16 t][D/64]      blocks g D/64 + [0, D/64) of token t
//   V scales [4 g][D/16 b][4]       block b of tokens 4 g + [0, 4)
// These are the operands of the 16x16x32 matrix instruction as its lanes hold
// them: lane 16 g + t reads the K channels of its token, lane 16 g + c its
// channel's values of four tokens, D / 8 consecutive bytes each, so a wave
// takes a record's codes in full cache lines and moves nothing between lanes.
#pragma once
#include "device_common.h"

namespace nvfp4 {

template <int D>
struct KvRec {
  static constexpr int kLane = D / 8;              // code bytes per lane, K and V
  static constexpr int kV = 8 * D;                 // part offsets
  static constexpr int kKs = 16 * D;
  static constexpr int kVs = 17 * D;
  static constexpr int kBytes = 18 * D;
};

}  // namespace nvfp4
