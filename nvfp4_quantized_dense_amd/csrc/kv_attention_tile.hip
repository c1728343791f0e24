// kv_attention_tile.hip -- attention over the paged NVFP4 cache for many query
// rows per key: drafted tokens, prompt chunks. (The mathematics:
// kv_attention_common.h; few rows: kv_attention.hip.)
//
// A workgroup of four waves takes 64 RT query rows (query x head of one kv
// head's group), 16 RT a wave, and walks over its keys in tiles of 64. A
// tile's codes are made f16 once for all four waves, a quarter by each, and
// lie in LDS in the order in which the matrix instruction's lanes read them,
// so that neither side has a bank conflict. Two tiles are in LDS, a third is
// on its way in registers, one barrier per tile.
#include "kv_attention_common.h"

namespace nvfp4 {
namespace {

#if defined(__HIP_DEVICE_COMPILE__)
constexpr int kTile = 64;  // keys

// Writes V's operands of a pair, channel blocks Y on, `to` being the first's.
template <int D, int Y>
__device__ __forceinline__ void put_v(f16x8* to, const VFrag<D> (&f)[2], const f16x4 (&vs)[2]) {
  to[Y * 64] = v_operand<D, Y>(f, vs);
  if (Y & 1) __builtin_amdgcn_sched_barrier(0);  // few operands in flight: registers
  if constexpr (Y + 1 < D / 16) put_v<D, Y + 1>(to, f, vs);
}
#endif

template <int D, int RT>
__global__ __launch_bounds__(256, D == 256 ? 1 : 2) void k_kv_attention_tile(AttnArgs a, AttnPlan p) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int kB = D / 16, kW = D / 32, kRows = 64 * RT;
  constexpr int kOps = 4 * kW + 2 * kB;  // operands of a tile: [4 records][kW] K, [2 pairs][kB] V
  constexpr int kJoin = kTileJoin, kAhead = 4;
  __shared__ f16x8 lds[2 * kOps * 64 * 2 > kJoin ? 2 * kOps * 64 : kJoin / 2];
  __shared__ uint32_t page_ok[2][2];  // of a tile's pairs: bit x for record x
  __shared__ uint32_t arrived;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, quad = lane >> 4;
  const int G = a.heads_q / a.c.heads;
  // grid: (head, row block, sequence) fastest to slowest in x, split in y.
  // Later rows see more keys: they start first.
  const unsigned unit = blockIdx.x, heads = a.c.heads, blocks = p.row_blocks;
  const int h = (int)(unit % heads);
  const unsigned rb = blocks - 1 - unit / heads % blocks, b = unit / heads / blocks;
  const int split = blockIdx.y;

  const Seq seq = seq_of(a, b, G);
  if ((int64_t)rb * kRows >= seq.rows) return;
  const int row0 = (int)rb * kRows;
  const int last_row = seq.rows - 1 < row0 + kRows - 1 ? seq.rows - 1 : row0 + kRows - 1;
  const int hi_all = sees_hi(seq, last_row / G), lo_all = sees_lo(sees_hi(seq, row0 / G), a.window);
  const int start = lo_all & ~31;
  const int active = hi_all > lo_all ? (hi_all - start + p.chunk - 1) / p.chunk : 1;
  if (split >= active) return;
  const int s_first = start + split * p.chunk;
  const int s_last = hi_all - s_first > p.chunk ? s_first + p.chunk : hi_all;
  const int tiles = s_last > s_first ? (s_last - s_first + kTile - 1) / kTile : 0;

  Rows<D, RT> r;
  const int wrow0 = row0 + wave * 16 * RT;
  load_rows<D, RT>(r, a, seq, wrow0, h, G, quad, col);
  // Keys that all of this wave's rows see, [lo_full, hi_full), need no mask.
  int hi_full = 0, lo_full = 0;
  if (wrow0 < seq.rows) {
    hi_full = sees_hi(seq, wrow0 / G);
    lo_full = sees_lo(sees_hi(seq, (seq.rows < wrow0 + 16 * RT ? seq.rows - 1 : wrow0 + 16 * RT - 1) / G), a.window);
  }

  // Waves 0 and 1 bring K of the tile's first and second pair of records,
  // waves 2 and 3 V. The pair's first group is group `in` of page slot `ps`,
  // whose page number is in a lane of `tab` (64 slots from tab0 on); slots
  // past the last key's stand for that one and are masked.
  const int groups = a.c.page_size / 16, pair = wave & 1;
  const bool is_v = wave >= 2;
  const int32_t* table = a.table + (int64_t)b * a.table_stride;
  const int g0 = (s_first >> 4) + 2 * pair;
  int ps = g0 / groups, in = g0 - ps * groups, tab0 = ps, tab = 0;
  const int ps_last = hi_all > 0 ? ((hi_all - 1) >> 4) / groups : 0;
  auto load_tab = [&] {
    const int at = tab0 + lane;
    tab = table[at < ps_last ? at : ps_last];
  };
  KFrag<D> f[2];  // K's or V's codes and scales: one shape
  uint32_t ok = 0;
  auto step = [&](int by) {
    in += by;
    while (in >= groups) { in -= groups; ++ps; }
  };
  auto fetch = [&] {
    ok = 0;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      if (ps - tab0 >= 64) {
        tab0 = ps;
        load_tab();
      }
      const int page = __builtin_amdgcn_readlane(tab, ps - tab0);
      const bool good = page >= 0 && page < a.c.pages;
      ok |= good ? 1u << x : 0u;
      const uint8_t* rec = a.c.cache + rec_offset<D>(good ? page : 0, a.c.heads, h, groups, in);
      if (is_v) load_v<D>(reinterpret_cast<VFrag<D>&>(f[x]), rec, lane);
      else load_k<D>(f[x], rec, lane);
      step(x == 0 ? 1 : 3);
    }
  };
  // The fetched pair becomes operands of buffer `buf`; its first key is `base`.
  auto put = [&](int buf, int base) {
    f16x8* to = lds + buf * kOps * 64 + lane;
    if (is_v) {
      VFrag<D> v[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        v[x] = reinterpret_cast<VFrag<D>&>(f[x]);
        // Tokens no row sees may never have been written: their V scales
        // become zero, so that no NaN code meets a zero probability.
        if (base < lo_all || base + 32 > hi_all || ok != 3u)
          v[x].s &= (ok >> x) & 1 ? byte_mask(base + 16 * x + 4 * quad, lo_all, hi_all) : 0u;
      }
      const f16x4 vs[2] = {e4m3x4_f16(v[0].s), e4m3x4_f16(v[1].s)};
      put_v<D, 0>(to + (4 * kW + pair * kB) * 64, v, vs);
    } else {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const f16x4 ks = e4m3x4_f16(f[x].s);
#pragma unroll
        for (int s = 0; s < kW; ++s) {
          to[((2 * pair + x) * kW + s) * 64] = deq8_f16(f[x].c[s], ks[s >> 1]);
          if (s & 1) __builtin_amdgcn_sched_barrier(0);
        }
      }
      if (lane == 0) page_ok[buf][pair] = ok;
    }
  };
  auto attend = [&](int buf, int base) {
    const f16x8* from = lds + buf * kOps * 64 + lane;
#pragma unroll 1
    for (int pr = 0; pr < 2; ++pr) {
      const int at = base + 32 * pr;
      const uint32_t has = __builtin_amdgcn_readfirstlane(page_ok[buf][pr]);
      const bool edge = at + 32 > hi_full || at < lo_full || has != 3u;
      f32x4 sc[RT][2];
#pragma unroll
      for (int t = 0; t < RT; ++t) sc[t][0] = sc[t][1] = f32x4{0.f, 0.f, 0.f, 0.f};
      // Operands are read kAhead products before they are used.
      const f16x8* kp = from + 2 * pr * kW * 64;
      f16x8 op[kAhead];
#pragma unroll
      for (int n = 0; n < kAhead; ++n) op[n] = kp[n * 64];
#pragma unroll
      for (int n = 0; n < 2 * kW; ++n) {
#pragma unroll
        for (int t = 0; t < RT; ++t) sc[t][n / kW] = mfma16x16x32(op[n % kAhead], r.q[t][n % kW], sc[t][n / kW]);
        if (n + kAhead < 2 * kW) op[n % kAhead] = kp[(n + kAhead) * 64];
        __builtin_amdgcn_sched_barrier(0);
      }
      if (edge) {
        asm volatile("");  // a branch: most tiles need no mask
        const bool okx[2] = {(has & 1) != 0, (has & 2) != 0};
        hide_scores<D, RT>(r, sc, at, quad, okx);
      }
      f16x8 pf[RT];
      softmax_pair<D, RT>(r, sc, pf);
      const f16x8* vp = from + (4 * kW + pr * kB) * 64;
#pragma unroll
      for (int n = 0; n < kAhead; ++n) op[n] = vp[n * 64];
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int y = 0; y < kB; ++y) {
#pragma unroll
        for (int t = 0; t < RT; ++t) r.o[t][y] = mfma16x16x32(op[y % kAhead], pf[t], r.o[t][y]);
        if (y + kAhead < kB) op[y % kAhead] = vp[(y + kAhead) * 64];
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  };
  if (tiles > 0) {
    load_tab();
    fetch();
    put(0, s_first + 32 * pair);
    if (tiles > 1) fetch();
    __syncthreads();
    for (int j = 0; j < tiles; ++j) {
      const int base = s_first + kTile * j;
      if (j + 1 < tiles) {
        put((j + 1) & 1, base + kTile + 32 * pair);
        if (j + 2 < tiles) fetch();
      }
      attend(j & 1, base);
      __syncthreads();
    }
  }
  finish_rows<D, RT>(r);

  const float vg = *a.v_g;
  float* part = a.part + ((int64_t)unit * p.splits + split) * p.part_floats;
  const Rsrc rp = make_rsrc(part, (uint32_t)(p.part_floats * 4));
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    const int rr = wave * 16 * RT + 16 * t + col;
    const bool live = row0 + rr < seq.rows;
    if (active == 1) {
      if (!live) continue;
      const float inv = inverse_sum(r.l[t], vg);
      const int64_t orow = out_row(a, seq, row0 + rr, h, G);
#pragma unroll
      for (int y = 0; y < kB; ++y) store4(a, orow * D + 16 * y + 4 * quad, r.o[t][y] * inv);
      if (quad == 0 && a.lse != nullptr) a.lse[orow] = lse_of(r.m[t], r.l[t]);
    } else {
      if (live) {
#pragma unroll
        for (int y = 0; y < kB; ++y)
          bstore16_dev(rp, (uint32_t)(8 * kRows + (rr * D + 16 * y + 4 * quad) * 4), __builtin_bit_cast(u32x4, r.o[t][y]));
      }
      if (quad == 0) {
        __hip_atomic_store(part + rr, r.m[t], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __hip_atomic_store(part + kRows + rr, r.l[t], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
    }
  }
  if (active == 1) return;
  if (!split_last(a.counters + unit, active, &arrived)) return;
  join_splits<D, kRows, kJoin>(a, p, seq, unit, active, row0, h, G, reinterpret_cast<float*>(lds));
#endif  // __HIP_DEVICE_COMPILE__
}

template <int D, int RT>
void launch_rt(const AttnArgs& a, const AttnPlan& p, hipStream_t s) {
  if constexpr (RT <= attn_tile_max(D)) {
    if (p.row_tiles == RT) k_kv_attention_tile<D, RT><<<dim3((unsigned)p.units, (unsigned)p.splits), dim3(256), 0, s>>>(a, p);
    else launch_rt<D, RT + 1>(a, p, s);
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
