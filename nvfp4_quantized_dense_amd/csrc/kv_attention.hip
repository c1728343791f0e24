// kv_attention.hip -- attention over the paged NVFP4 cache for few query rows
// per key: one token per sequence, a few drafted tokens. (More rows:
// kv_attention_tile.hip; the mathematics: kv_attention_common.h.)
//
// A workgroup takes 16 or 32 query rows (query x head of one kv head's group)
// of a sequence and a stretch of its keys; its four waves take a quarter of
// the stretch each, with a running maximum and sum per row (one pass over the
// cache), and join in LDS. A long key axis is split over workgroups and
// joined by the one that arrives last.
#include "kv_attention_common.h"

namespace nvfp4 {
namespace {

#if defined(__HIP_DEVICE_COMPILE__)
template <int D, int RT, int Y>
__device__ __forceinline__ void pv(f32x4 (&o)[RT][D / 16], const VFrag<D> (&f)[2], const f16x4 (&vs)[2], const f16x8 (&pf)[RT]) {
  const f16x8 vf = v_operand<D, Y>(f, vs);
#pragma unroll
  for (int t = 0; t < RT; ++t) o[t][Y] = mfma16x16x32(vf, pf[t], o[t][Y]);
  if constexpr (Y + 1 < D / 16) pv<D, RT, Y + 1>(o, f, vs, pf);
}
#endif

// Workgroups per CU that the registers are held to.
template <int D, int RT>
constexpr int kAttnWgs = D == 256 ? 1 : RT == 2 ? 2 : D == 64 ? 4 : 3;

template <int D, int RT>
__global__ __launch_bounds__(256, (kAttnWgs<D, RT>)) void k_kv_attention(AttnArgs a, AttnPlan p) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int kB = D / 16, kW = D / 32, kRows = 16 * RT;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, quad = lane >> 4;
  const int G = a.heads_q / a.c.heads;
  // grid: (head, row block, sequence) fastest to slowest in x, split in y
  const unsigned unit = blockIdx.x, heads = a.c.heads, blocks = p.row_blocks;
  const int h = (int)(unit % heads);
  const unsigned rb = unit / heads % blocks, b = unit / heads / blocks;
  const int split = blockIdx.y;

  const Seq seq = seq_of(a, b, G);
  if ((int64_t)rb * kRows >= seq.rows) return;
  const int row0 = (int)rb * kRows;
  const int last_row = seq.rows - 1 < row0 + kRows - 1 ? seq.rows - 1 : row0 + kRows - 1;
  const int hi_all = sees_hi(seq, last_row / G), hi_full = sees_hi(seq, row0 / G);
  const int lo_all = sees_lo(hi_full, a.window), lo_full = sees_lo(hi_all, a.window);  // [lo_full, hi_full) need no mask
  const int start = lo_all & ~31;
  const int active = hi_all > lo_all ? (hi_all - start + p.chunk - 1) / p.chunk : 1;
  if (split >= active) return;

  Rows<D, RT> r;
  load_rows<D, RT>(r, a, seq, row0, h, G, quad, col);

  const int groups = a.c.page_size / 16;
  const int32_t* table = a.table + (int64_t)b * a.table_stride;
  // This wave's stretch, whole steps of 32 tokens.
  const int s_first = start + split * p.chunk;
  const int s_last = hi_all - s_first > p.chunk ? s_first + p.chunk : hi_all;
  const int steps = s_last > s_first ? (s_last - s_first + 31) / 32 : 0, per = (steps + 3) / 4;
  const int step0 = wave * per, step1 = step0 + per < steps ? step0 + per : steps;

  // Records are taken in order: group g is group `in` of page slot `ps`,
  // whose page number is in a lane of `tab` (64 slots from tab0 on). Groups
  // past the last key stand for the last key's and are masked.
  int g = (s_first >> 4) + 2 * step0, ps = g / groups, in = g - ps * groups, tab0 = ps;
  const int g_last = (hi_all - 1) >> 4, ps_last = g_last / groups;
  int tab = 0;
  struct Pair {
    KFrag<D> k[2];
    VFrag<D> v[2];
    bool ok[2];
  };
  auto load_tab = [&] {
    const int at = tab0 + lane;
    tab = table[at < ps_last ? at : ps_last];
  };
  auto fetch = [&](Pair& f) {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      if (ps - tab0 == 64) {
        tab0 = ps;
        load_tab();
      }
      const int page = __builtin_amdgcn_readlane(tab, ps - tab0);
      f.ok[x] = page >= 0 && page < a.c.pages;
      const uint8_t* rec = a.c.cache + rec_offset<D>(f.ok[x] ? page : 0, a.c.heads, h, groups, in);
      load_k<D>(f.k[x], rec, lane);
      load_v<D>(f.v[x], rec, lane);
      if (g < g_last) {
        ++g;
        if (++in == groups) { in = 0; ++ps; }
      }
    }
  };
  auto attend = [&](Pair& f, int base) {
    const bool edge = base + 32 > hi_full || base < lo_full || !f.ok[0] || !f.ok[1];
    f32x4 sc[RT][2];
#pragma unroll
    for (int t = 0; t < RT; ++t) sc[t][0] = sc[t][1] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const f16x4 ks = e4m3x4_f16(f.k[x].s);
#pragma unroll
      for (int s = 0; s < kW; ++s) {
        const f16x8 kf = deq8_f16(f.k[x].c[s], ks[s >> 1]);
#pragma unroll
        for (int t = 0; t < RT; ++t) sc[t][x] = mfma16x16x32(kf, r.q[t][s], sc[t][x]);
      }
    }
    if (edge) {
      asm volatile("");  // a branch: most steps need no mask
      hide_scores<D, RT>(r, sc, base, quad, f.ok);
      // Tokens no row sees may never have been written: their V scales
      // become zero, so that no NaN code meets a zero probability.
#pragma unroll
      for (int x = 0; x < 2; ++x) f.v[x].s &= f.ok[x] ? byte_mask(base + 16 * x + 4 * quad, lo_all, hi_all) : 0u;
    }
    f16x8 pf[RT];
    softmax_pair<D, RT>(r, sc, pf);
    const f16x4 vs[2] = {e4m3x4_f16(f.v[0].s), e4m3x4_f16(f.v[1].s)};
    pv<D, RT, 0>(r.o, f.v, vs, pf);
  };
  if (step0 < step1) {
    // The next step's records are on their way while one is computed.
    Pair fa, fb;
    load_tab();
    fetch(fa);
    for (int st = step0; st < step1; st += 2) {
      const int base = s_first + 32 * st;
      if (st + 1 < step1) fetch(fb);
      attend(fa, base);
      if (st + 1 >= step1) break;
      if (st + 2 < step1) fetch(fa);
      attend(fb, base + 32);
    }
  }
  finish_rows<D, RT>(r);

  // The four waves' results become one: weights exp2(m_w - m) per row.
  __shared__ float wm[4][kRows], wl[4][kRows];
  constexpr int kJoin = kStreamJoin;
  __shared__ f32x4 lds[4 * kB * 64 > kJoin / 2 ? 4 * kB * 64 : kJoin / 2];
  auto wo = [&](int w, int y) -> f32x4& { return lds[(w * kB + y) * 64 + lane]; };
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    if (quad == 0) {
      wm[wave][16 * t + col] = r.m[t];
      wl[wave][16 * t + col] = r.l[t];
    }
  }
  __syncthreads();
  const float vg = *a.v_g;
  float* part = a.part + ((int64_t)unit * p.splits + split) * p.part_floats;
  const Rsrc rp = make_rsrc(part, (uint32_t)(p.part_floats * 4));
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    const int rr = 16 * t + col;
    const float m = __builtin_fmaxf(__builtin_fmaxf(wm[0][rr], wm[1][rr]), __builtin_fmaxf(wm[2][rr], wm[3][rr]));
    const float alpha = __builtin_amdgcn_exp2f(r.m[t] - m);
    float l = 0.0f;
#pragma unroll
    for (int w = 0; w < 4; ++w) l += wl[w][rr] * __builtin_amdgcn_exp2f(wm[w][rr] - m);
    if (t > 0) __syncthreads();
#pragma unroll
    for (int y = 0; y < kB; ++y) wo(wave, y) = r.o[t][y] * alpha;
    __syncthreads();
    // Wave w finishes channel blocks w, w + 4, ...: lane (quad, col) holds
    // channels 16 y + 4 quad + [0, 4) of row 16 t + col.
    const bool live = row0 + rr < seq.rows;
    const int64_t orow = out_row(a, seq, row0 + rr, h, G);
    for (int y = wave; y < kB; y += 4) {
      const f32x4 v = wo(0, y) + wo(1, y) + wo(2, y) + wo(3, y);
      if (!live) continue;
      if (active == 1) store4(a, orow * D + 16 * y + 4 * quad, v * inverse_sum(l, vg));
      else bstore16_dev(rp, (uint32_t)(8 * kRows + (rr * D + 16 * y + 4 * quad) * 4), __builtin_bit_cast(u32x4, v));
    }
    if (wave == 0 && quad == 0) {
      if (active == 1) {
        if (a.lse != nullptr && live) a.lse[orow] = lse_of(m, l);
      } else {
        __hip_atomic_store(part + rr, m, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __hip_atomic_store(part + kRows + rr, l, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
    }
  }
  if (active == 1) return;
  __shared__ uint32_t arrived;
  if (!split_last(a.counters + unit, active, &arrived)) return;
  join_splits<D, kRows, kJoin>(a, p, seq, unit, active, row0, h, G, reinterpret_cast<float*>(lds));
#endif  // __HIP_DEVICE_COMPILE__
}

template <int D>
void launch_d(const AttnArgs& a, const AttnPlan& p, hipStream_t s) {
  const dim3 grid((unsigned)p.units, (unsigned)p.splits);
  if (p.row_tiles == 1) k_kv_attention<D, 1><<<grid, dim3(256), 0, s>>>(a, p);
  else k_kv_attention<D, 2><<<grid, dim3(256), 0, s>>>(a, p);
}

}  // namespace

AttnPlan attn_plan(int64_t B, int heads_q, int heads, int dim, int64_t max_q, int64_t max_len, int64_t window) {
  AttnPlan p{};
  const int64_t rows = max_q * (heads_q / heads);
  int64_t per, slots, join;  // rows of a workgroup, workgroups wanted, (split, row) pairs the join holds
  p.tiled = rows > 32;
  if (p.tiled) {
    const int64_t most = 64 * attn_tile_max(dim);
    const int64_t blocks = (rows + most - 1) / most;
    p.row_tiles = (int)((rows + 64 * blocks - 1) / (64 * blocks));
    per = 64 * p.row_tiles;
    slots = 512;
    join = kTileJoin;
  } else {
    p.row_tiles = rows <= 16 ? 1 : 2;
    per = 16 * p.row_tiles;
    slots = 1024;
    join = kStreamJoin;
  }
  const int64_t blocks = (rows + per - 1) / per;
  p.units = blocks * B * heads;
  if (p.units > kAttnMaxUnits) return p;
  p.row_blocks = (int)blocks;
  // Keys that a unit reads at most, from a multiple of 32 on.
  int64_t span = max_len;
  if (window > 0 && window + max_q + 31 < span) span = window + max_q + 31;
  span = (span + 31) / 32 * 32;
  int64_t want = p.units > 0 ? (slots + p.units - 1) / p.units : 1;
  int64_t bound = want;
  int64_t most = (span + 255) / 256;  // at least 256 keys each
  if (most > join / per) most = join / per;
  if (want > most) want = most;
  if (want < 1) want = 1;
  if (bound > (max_len + 255) / 256) bound = (max_len + 255) / 256;
  p.splits_bound = bound < 1 ? 1 : bound;
  p.chunk = (int)(((span + want - 1) / want + 127) / 128 * 128);
  if (p.chunk < 128) p.chunk = 128;
  p.splits = span > 0 ? (int)((span + p.chunk - 1) / p.chunk) : 1;
  p.part_floats = (int)per * (dim + 2);
  return p;
}

hipError_t launch_kv_attention(const AttnArgs& a, const AttnPlan& p, hipStream_t s) {
  if (p.tiled) return launch_kv_attention_tile(a, p, s);
  if (a.c.dim == 64) launch_d<64>(a, p, s);
  else if (a.c.dim == 128) launch_d<128>(a, p, s);
  else launch_d<256>(a, p, s);
  return hipGetLastError();
}

}  // namespace nvfp4
