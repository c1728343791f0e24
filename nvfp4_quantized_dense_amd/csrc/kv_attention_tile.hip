// kv_attention_tile.hip -- attention over the paged NVFP4 cache for many query
// rows per key: drafted tokens, prompt chunks. (The mathematics:
// kv_attention_common.h; few rows: kv_attention.hip.)
//
// A workgroup of four waves takes 64 RT query rows (query x head of one kv
// head's group), 16 RT a wave, and walks over its keys in tiles of 64. A
// tile's codes are made f16 once for all four waves, a quarter by each, and
// lie in LDS in the order in which the matrix instruction's lanes read them,
// so that neither side has a bank conflict.
//
// What bounds it is the waves' instruction issue: per 32 keys and 32 rows (D
// 128) 32 matrix instructions stand against 70 of the softmax and 50 of
// making f16 and fetching. So the three overlap: while the probabilities of
// 32 keys are computed, the scores of the next 32 are on the matrix core, and
// while values are added, the tile after the next is made. RT 2 at D 128 (4
// at 64): 16 rows a wave more would spill, fewer share the making less (8 x
// 1536 tokens x 64 heads over 8192 keys: RT 1 / 2 4215 / 2900 us, the latter
// 1030 TFLOP/s; without the making and fetching, for the time alone, 1355).
// Chunks of up to 2047 tokens of 3 sequences against up to 8192 keys: 418 to
// 490 us, 825 to 965 TFLOP/s, the rest being unequal workgroups at the end.
#include "kv_attention_common.h"

namespace nvfp4 {
namespace {

#if defined(__HIP_DEVICE_COMPILE__)
constexpr int kTile = 64;  // keys

#endif

// P: f16 parts of a probability. MASKED: sinks or a tree mask.
template <int D, int RT, int P, bool MASKED>
__global__ __launch_bounds__(256, D == 256 ? 1 : 2) void k_kv_attention_tile(AttnArgs a, AttnPlan p) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int kB = D / 16, kW = D / 32, kRows = 64 * RT;
  // Operands: [2 tiles][4 records][kW] K, [2 tiles][kB] V of the first pair,
  // [3 tiles][kB] V of the second, which is read while the barrier that
  // parts two tiles is already behind (one barrier a tile, not two).
  constexpr int kV = 8 * kW, kV2 = kV + 2 * kB, kOps = kV2 + 3 * kB;
  constexpr int kAhead = 4;
  __shared__ f16x8 lds[kOps * 64];
  __shared__ alignas(4) uint8_t page_ok[2][4];  // of a tile's records; CLEAN: 2 is added for what the next line holds
  __shared__ uint32_t no_number[3][2][kB];      // of a tile's pairs, by block: tokens whose values are NaN
  __shared__ uint32_t nan_rows[kRows];          // a bit for each block whose channels become NaN
  __shared__ uint32_t found_nan;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, quad = lane >> 4;
  const int G = a.heads_q / a.c.heads;
  // grid: (head, row block, sequence) fastest to slowest in x, split in y.
  // Later rows see more keys: they start first.
  const unsigned unit = blockIdx.x, heads = a.c.heads, blocks = p.row_blocks;
  const int h = (int)(unit % heads);
  unsigned rb = blocks - 1 - unit / heads % blocks, b = unit / heads / blocks;
  if (MASKED && p.packed) {
    const Block at = packed_block(a, p, unit, G, lane);
    b = at.b;
    rb = at.rb;
  }
  const int split = blockIdx.y;

  // MASKED: as in kv_attention.hip, page numbers are asked for before the lengths
  // where they do not depend on them, and the first two tiles before the query
  // rows (trees are short calls: one of 24 tokens over 4097 keys 25.8 -> 22.3
  // us). The plain kernel loses by it, 446 -> 458 us for chunks of up to 2047
  // tokens: its main loop comes out with other registers.
  Walk<D> walk;
  if constexpr (MASKED) walk = Walk<D>(a, b, h, a.window > 0 ? 0 : split * (p.chunk / 16), lane);
  const Seq seq = seq_of(a, b, G);
  if ((int64_t)rb * kRows >= seq.rows) return;
  const int row0 = (int)rb * kRows;
  const Stretch all = active_splits<MASKED>(a, p, seq, row0, kRows, G);
  const int hi_all = all.hi, lo_all = all.lo, active = all.splits;
  if (split >= active) return;
  const int s_first = all.start + split * p.chunk;
  const int s_last = all.end - s_first > p.chunk ? s_first + p.chunk : all.end;
  const int tiles = s_last > s_first ? (s_last - s_first + kTile - 1) / kTile : 0;

  Rows<D, RT> r;
  const int wrow0 = row0 + wave * 16 * RT;
  // MASKED: a hidden value that is NaN makes its channels NaN all the same, 0
  // times NaN. What comes out NaN is computed once more (CLEAN), with such
  // values left out and the rows noted that see them. So a call without any
  // pays for a look at its sums alone: chunks behind a window 87.2 -> 88.0 us;
  // with the notes in its one pass, whose loop came out with other registers,
  // 91.5.
  auto pass = [&](auto clean) {
    constexpr bool CLEAN = decltype(clean)::value;
    // Wave w brings K of the tile's record w and half w & 1 of V's channels of
    // the pair w >> 1.
    const int pair = wave >> 1, half = wave & 1;
    KFrag<D> fk, nk;  // of the tile at hand, of the one after the first
    VFrag<D, 2> fv[2], nv[2];
    bool ok[2] = {true, true}, nok[2] = {true, true};
    bool nans = false;
    int ahead = s_first + 32 * pair;  // the next of this wave's pairs fetched
    bool jump = ahead < all.head;
    auto fetch = [&](KFrag<D>& k, VFrag<D, 2> (&v)[2], bool (&okay)[2]) {
      if constexpr (MASKED) {
        if (jump && ahead >= all.head) {
          walk.start((ahead + all.gap) >> 4);
          jump = false;
        }
        ahead += kTile;
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const Rsrc rec = walk.record(okay[x], lane);
        load_v(v[x], rec, lane, half);
        if (x == half) load_k(k, rec, lane);
        walk.step(x == 0 ? 1 : 3);
      }
    };
    if constexpr (MASKED) {
      if (CLEAN) walk = Walk<D>(a, b, h, a.window > 0 ? 0 : split * (p.chunk / 16), lane);
      if (tiles > 0) {
        walk.start(all.key<MASKED>(ahead) >> 4);
        fetch(fk, fv, ok);
        fetch(nk, nv, nok);
      }
    }

    load_rows<D, RT, MASKED>(r, a, seq, wrow0, h, G, quad, col);
    // Keys that all of this wave's rows see, [lo_full, hi_full), need no mask.
    int hi_full = 0, lo_full = 0;
    if (wrow0 < seq.rows) {
      hi_full = sees_hi(seq, wrow0 / G);
      if (MASKED && a.tree != nullptr) {
        hi_full = tree_context(seq);
        lo_full = sees_lo(all.hi, a.window);
      } else lo_full = sees_lo(sees_hi(seq, (seq.rows < wrow0 + 16 * RT ? seq.rows - 1 : wrow0 + 16 * RT - 1) / G), a.window);
    }

    // Before what was fetched becomes operands: tokens no row sees may never
    // have been written. Their V scales become zero, so that no NaN code meets
    // a zero probability. `base`: the tile's first place.
    // CLEAN: `third` is the tile's buffer.
    auto clear_v = [&](int base, int third) {
      base = all.key<MASKED>(base + 32 * pair);
      if ((MASKED ? masked_edge(a, base, lo_all, hi_all) : base < lo_all || base + 32 > hi_all) || !ok[0] || !ok[1]) {
#pragma unroll
        for (int x = 0; x < 2; ++x) fv[x].s &= ok[x] ? (MASKED ? masked_bytes(a, base + 16 * x + 4 * quad, lo_all, hi_all) : byte_mask(base + 16 * x + 4 * quad, lo_all, hi_all)) : 0u;
      }
      if constexpr (CLEAN) {
        nans = any_nan(fv);
        if (nans) take_nans(fv, lane, no_number[third][pair] + half * (kB / 2));
      }
    };
    auto record_flags = [&] { return (uint8_t)(CLEAN ? (ok[half] ? 1 : 0) + (nans ? 2 : 0) : ok[half]); };
    // Operand n of the kB that this wave makes of what it fetched: K and V in
    // turn, for buffers `buf` and `third`.
    f16x4 ks, vs[2];
    auto scales = [&] {
      ks = e4m3x4_f16(fk.s);
      vs[0] = e4m3x4_f16(fv[0].s);
      vs[1] = e4m3x4_f16(fv[1].s);
    };
    auto put = [&](auto n, int buf, int third) {
      constexpr int kN = decltype(n)::value, kS = kN / 2;
      if constexpr (kN % 2 == 0) lds[((4 * buf + wave) * kW + kS) * 64 + lane] = deq8_f16(fk.c[kS], ks[kS >> 1]);
      else lds[((pair == 0 ? kV + buf * kB : kV2 + third * kB) + half * (kB / 2) + kS) * 64 + lane] = v_operand<kS>(fv, vs);
    };
    // One pair: its probabilities from the scores `now` while the matrix core
    // computes the next pair's scores `later`, K from operand k0 on; then its
    // values, V from operand v0 on, while make(0 .. kB - 1) fills in. Operands
    // are read kAhead products before they are used. The barriers keep this
    // order, and few registers alive.
    auto attend = [&](const f32x4 (&now)[RT][2], f32x4 (&later)[RT][2], float (&mx)[RT], int k0, int v0, auto&& make) {
      const f16x8 *kp = lds + k0 * 64 + lane, *vp = lds + v0 * 64 + lane;
      f16x8 op[kAhead], pf[P][RT];
      auto operand = [&](int n) { return n < 2 * kW ? kp[n * 64] : vp[(n - 2 * kW) * 64]; };
      float e[RT];
#pragma unroll
      for (int t = 0; t < RT; ++t) later[t][0] = later[t][1] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int n = 0; n < kAhead; ++n) op[n] = operand(n);
      static_for<2 * kW>([&](auto step) {
        constexpr int n = decltype(step)::value;
#pragma unroll
        for (int t = 0; t < RT; ++t) {
          later[t][n / kW] = mfma16x16x32(op[n % kAhead], r.q[t][n % kW], later[t][n / kW]);
#pragma unroll
          for (int i = 8 * n / (2 * kW); i < 8 * (n + 1) / (2 * kW); ++i) {
            const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(now[t][i >> 2][i & 3], r.f[t], r.a[t]));
            r.l[t] += p;
            if (i & 1) {
              put_probability(pf, t, i - 1, e[t]);
              put_probability(pf, t, i, p);
            }
            e[t] = p;
          }
        }
        op[n % kAhead] = operand(n + kAhead);
        __builtin_amdgcn_sched_barrier(0);
      });
      static_for<kB>([&](auto step) {
        constexpr int y = decltype(step)::value, n = 2 * kW + y;
#pragma unroll
        for (int x = 0; x < P; ++x)
#pragma unroll
          for (int t = 0; t < RT; ++t) r.o[t][y] = mfma16x16x32(op[n % kAhead], pf[x][t], r.o[t][y]);
        if constexpr (y + kAhead < kB) op[n % kAhead] = operand(n + kAhead);
        make(step);
        // The next pair's maximum, by lane.
#pragma unroll
        for (int i = 8 * y / kB; i < 8 * (y + 1) / kB; ++i) {
#pragma unroll
          for (int t = 0; t < RT; ++t)
            mx[t] = i == 0 ? later[t][0][0] : __builtin_fmaxf(mx[t], later[t][i >> 2][i & 3]);
        }
        __builtin_amdgcn_sched_barrier(0);
      });
#pragma unroll
      for (int t = 0; t < RT; ++t) asm volatile("" : "+v"(mx[t]), "+v"(r.l[t]));  // computed in here
    };
    auto renew = [&](f32x4 (&sc)[RT][2], float (&mx)[RT], int at, uint32_t oks, int third, int pair) {
      at = all.key<MASKED>(at);
      if ((MASKED ? masked_edge(a, at, lo_full, hi_full) : at + 32 > hi_full || at < lo_full) || oks != 0x101u) {
        asm volatile("");  // a branch: most pairs need no mask
        const bool okx[2] = {(oks & (CLEAN ? 1u : 255u)) != 0, (CLEAN ? oks >> 8 & 1u : oks >> 8) != 0};
        if constexpr (CLEAN) {
          hide_masked<D, RT>(r, a, seq, sc, at, quad, okx, [&](int t, uint32_t see) {
            if (oks & 0x202u)
              note_nans<D>(nan_rows + wave * 16 * RT + 16 * t, lane, see, no_number[third][pair], (oks & 2u) != 0, (oks & 512u) != 0);
          });
        } else if constexpr (MASKED) {
          hide_masked<D, RT>(r, a, seq, sc, at, quad, okx, [](int, uint32_t) {});
        } else {
          hide_scores<D, RT>(r, sc, at, quad, okx);
        }
        lane_maximum<RT>(sc, mx);
      }
      renew_maximum<D, RT>(r, mx);
    };
    auto make_tile = [&](int buf, int third) {
      scales();
      static_for<kB>([&](auto n) { put(n, buf, third); });
      if (lane == 0) page_ok[buf][wave] = record_flags();
    };
    if (tiles > 0) {
      if constexpr (!MASKED) {
        walk = Walk<D>(a, b, h, s_first >> 4, lane);
        walk.start(ahead >> 4);
        fetch(fk, fv, ok);
      }
      clear_v(s_first, 0);
      make_tile(0, 0);
      if constexpr (MASKED) {
        fk = nk;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          fv[x] = nv[x];
          ok[x] = nok[x];
        }
      } else {
        fetch(fk, fv, ok);
      }
      clear_v(s_first + kTile, 1);
      make_tile(1, 1);
      fetch(fk, fv, ok);
      __syncthreads();
      f32x4 sa[RT][2], sb[RT][2];
      float mx[RT];
#pragma unroll
      for (int t = 0; t < RT; ++t) sa[t][0] = sa[t][1] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int n = 0; n < 2 * kW; ++n) {
        const f16x8 op = lds[n * 64 + lane];
#pragma unroll
        for (int t = 0; t < RT; ++t) sa[t][n / kW] = mfma16x16x32(op, r.q[t][n % kW], sa[t][n / kW]);
      }
      lane_maximum<RT>(sa, mx);
      uint32_t oks = __builtin_amdgcn_readfirstlane(*reinterpret_cast<const uint32_t*>(page_ok[0]));
      // Tile j's first pair, then its second while tile j + 2 is made of what a
      // whole tile's time ago was asked for. After the barrier tile j + 1 is
      // there and K and the first pair's V of tile j have been read by all.
      for (int j = 0, third = 0; j < tiles; ++j) {
        const int base = s_first + kTile * j, buf = j & 1, third2 = third == 0 ? 2 : third - 1;
        renew(sa, mx, base, oks & 0xFFFFu, third, 0);
        attend(sa, sb, mx, (4 * buf + 2) * kW, kV + buf * kB, [](auto) {});
        renew(sb, mx, base + 32, oks >> 16, third, 1);
        clear_v(base + 2 * kTile, third2);
        __syncthreads();
        const uint32_t flags = *reinterpret_cast<const uint32_t*>(page_ok[buf ^ 1]);
        scales();
        attend(sb, sa, mx, 4 * (buf ^ 1) * kW, kV2 + third * kB, [&](auto n) { put(n, buf, third2); });
        if (lane == 0) page_ok[buf][wave] = record_flags();
        oks = __builtin_amdgcn_readfirstlane(flags);
        fetch(fk, fv, ok);
        third = third == 2 ? 0 : third + 1;
      }
    }
    finish_rows<D, RT>(r);
  };
  if (MASKED && threadIdx.x == 0) found_nan = 0;
  pass(std::false_type{});
  if constexpr (MASKED) {
    if (tiles > 0) {  // the same for all waves
      float sum = 0.0f;  // a block's channels are NaN together
#pragma unroll
      for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int y = 0; y < kB; ++y) sum += r.o[t][y][0];
      if (sum != sum) found_nan = 1;
      __syncthreads();
      if (__builtin_expect(__builtin_amdgcn_readfirstlane(found_nan) != 0, 0)) {
        if (lane < 16 * RT) nan_rows[wave * 16 * RT + lane] = 0;
        pass(std::true_type{});
#pragma unroll
        for (int t = 0; t < RT; ++t) {
          const uint32_t bad = nan_rows[wave * 16 * RT + 16 * t + col];
#pragma unroll
          for (int y = 0; y < kB; ++y) r.o[t][y] = nan_if(bad >> y & 1u, r.o[t][y]);
        }
      }
    }
  }

  const float vg = *a.v_g;
  // Partials of a split: [kRows] m, [kRows] l, [kRows][D] o.
  float* part = a.part + ((int64_t)unit * p.splits + split) * p.part_floats;
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    const int rr = wave * 16 * RT + 16 * t + col;
    if (row0 + rr >= seq.rows) continue;
    if (active == 1) {
      const float inv = inverse_sum(r.l[t], vg);
      const int64_t orow = out_row(a, seq, row0 + rr, h, G);
#pragma unroll
      for (int y = 0; y < kB; ++y) store4(a, orow * D + 16 * y + 4 * quad, r.o[t][y] * inv);
      if (quad == 0 && a.lse != nullptr) a.lse[orow] = lse_of(row_maximum<D, RT>(r, t), r.l[t]);
    } else {
#pragma unroll
      for (int y = 0; y < kB; ++y)
        *reinterpret_cast<f32x4*>(part + 2 * kRows + rr * D + 16 * y + 4 * quad) = r.o[t][y];
      if (quad == 0) {
        part[rr] = row_maximum<D, RT>(r, t);
        part[kRows + rr] = r.l[t];
      }
    }
  }
#endif  // __HIP_DEVICE_COMPILE__
}

template <int D, int RT>
void launch_rt(const AttnArgs& a, const AttnPlan& p, hipStream_t s) {
  if constexpr (RT <= attn_tile_max(D)) {
    if (p.row_tiles != RT) return launch_rt<D, RT + 1>(a, p, s);
    const dim3 grid((unsigned)p.units, (unsigned)p.splits);
    if (attn_masked(a)) {
      if (a.f32_out) k_kv_attention_tile<D, RT, 2, true><<<grid, dim3(256), 0, s>>>(a, p);
      else k_kv_attention_tile<D, RT, 1, true><<<grid, dim3(256), 0, s>>>(a, p);
    } else if (a.f32_out) {
      k_kv_attention_tile<D, RT, 2, false><<<grid, dim3(256), 0, s>>>(a, p);
    } else {
      k_kv_attention_tile<D, RT, 1, false><<<grid, dim3(256), 0, s>>>(a, p);
    }
  }
}

}  // namespace

hipError_t launch_kv_attention_tile(const AttnArgs& a, const AttnPlan& p, hipStream_t s) {
  if (a.c.dim == 64) launch_rt<64, 1>(a, p, s);
  else if (a.c.dim == 128) launch_rt<128, 1>(a, p, s);
  else launch_rt<256, 1>(a, p, s);
  return hipGetLastError();
}

}  // namespace nvfp4
