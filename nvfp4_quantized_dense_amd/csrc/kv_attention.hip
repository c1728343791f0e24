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
  const f16x8 vf = v_operand<Y>(f, vs);
#pragma unroll
  for (int t = 0; t < RT; ++t) o[t][Y] = mfma16x16x32(vf, pf[t], o[t][Y]);
  if constexpr (Y + 1 < D / 16) pv<D, RT, Y + 1>(o, f, vs, pf);
}
#endif

#if defined(__HIP_DEVICE_COMPILE__)
// Partials of a split: [kRows] m, [kRows] l, [kRows][D] o. Each wave's are at
// device scope before its workgroup counts as arrived; true for the last one
// of `active`, which resets the count for the next launch.
__device__ __forceinline__ bool split_last(uint32_t* counter, int active, uint32_t* arrived) {
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __builtin_amdgcn_s_waitcnt(0x3F70);  // vmcnt(0)
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __syncthreads();
  if (threadIdx.x == 0) *arrived = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __syncthreads();
  if (*arrived != (uint32_t)(active - 1)) return false;
  if (threadIdx.x == 0) __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  return true;
}

// Joins the splits of a unit in split order, so that the result does not
// depend on which workgroup arrived last. lds: 2 kStreamJoin floats. What
// this costs is trips to device scope: the first 16 partials of a thread's
// four channels are asked for together with the statistics.
template <int D, int kRows>
__device__ __forceinline__ void join_splits(const AttnArgs& a, const AttnPlan& p, const Seq& seq, unsigned unit, int active,
                                            int row0, int h, int G, float* lds) {
  constexpr int kBatch = 16;
  const float vg = *a.v_g;
  const float* parts = a.part + (int64_t)unit * p.splits * p.part_floats;
  const Rsrc ra = make_rsrc(parts, (uint32_t)(active * p.part_floats * 4));
  const int live = (seq.rows - row0 < kRows ? seq.rows - row0 : kRows) * (D / 4);
  f32x4 x[kBatch];
  auto load = [&](int n, int s) {  // past the last split or row: zeros, unread
    const uint32_t at = (uint32_t)(8 * kRows + n * 16);
#pragma unroll
    for (int e = 0; e < kBatch; ++e)
      x[e] = __builtin_bit_cast(f32x4, bload16_dev(ra, s + e < active && n < live ? at + (uint32_t)((s + e) * p.part_floats * 4)
                                                                                  : kOutOfRange));
  };
  load(threadIdx.x, 0);
  float* jm = lds;  // [active][kRows] m, then l
  float* jl = lds + kStreamJoin;
  for (int n = threadIdx.x; n < active * kRows; n += 256) {
    const uint32_t at = (uint32_t)((n / kRows * p.part_floats + n % kRows) * 4);
    jm[n] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(ra, (int)at, 0, 16));
    jl[n] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(ra, (int)at, 4 * kRows, 16));
  }
  __syncthreads();
  for (int n = threadIdx.x; n < live; n += 256) {
    const int rr = n / (D / 4), d = n % (D / 4) * 4;
    float m = kNoKey;
    for (int s = 0; s < active; ++s) m = __builtin_fmaxf(m, jm[s * kRows + rr]);
    float l = 0.0f;
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < active; s += kBatch) {
      if (s > 0 || n >= 256) load(n, s);
#pragma unroll
      for (int e = 0; e < kBatch; ++e) {
        if (s + e >= active) break;
        const float w = __builtin_amdgcn_exp2f(jm[(s + e) * kRows + rr] - m);
        l += w * jl[(s + e) * kRows + rr];
        v += x[e] * w;
      }
    }
    const int64_t orow = out_row(a, seq, row0 + rr, h, G);
    store4(a, orow * D + d, v * inverse_sum(l, vg));
    if (d == 0 && a.lse != nullptr) a.lse[orow] = lse_of(m, l);
  }
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
  const Stretch all = active_splits(a, p, seq, row0, kRows, G);
  const int hi_all = all.hi, lo_all = all.lo, active = all.splits;
  const int hi_full = sees_hi(seq, row0 / G), lo_full = sees_lo(hi_all, a.window);  // [lo_full, hi_full) need no mask
  if (split >= active) return;

  Rows<D, RT> r;
  load_rows<D, RT>(r, a, seq, row0, h, G, quad, col);

  // This wave's stretch, whole steps of 32 tokens.
  const int s_first = all.start + split * p.chunk;
  const int s_last = hi_all - s_first > p.chunk ? s_first + p.chunk : hi_all;
  const int steps = s_last > s_first ? (s_last - s_first + 31) / 32 : 0, per = (steps + 3) / 4;
  const int step0 = wave * per, step1 = step0 + per < steps ? step0 + per : steps;

  struct Pair {
    KFrag<D> k[2];
    VFrag<D> v[2];
    bool ok[2];
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
    float mx[RT];
    lane_maximum<RT>(sc, mx);
    renew_maximum<D, RT>(r, mx);
    probabilities<D, RT>(r, sc, pf);
    const f16x4 vs[2] = {e4m3x4_f16(f.v[0].s), e4m3x4_f16(f.v[1].s)};
    pv<D, RT, 0>(r.o, f.v, vs, pf);
  };
  if (step0 < step1) {
    // The next step's records are on their way while one is computed.
    Pair fa, fb;
    Walk<D> walk(a, b, h, (s_first >> 4) + 2 * step0, (hi_all - 1) >> 4, lane);
    auto fetch = [&](Pair& f) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const uint8_t* rec = walk.record(f.ok[x], lane);
        load_k(f.k[x], rec, lane);
        load_v(f.v[x], rec, lane, 0);
        walk.step(1);
      }
    };
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
  __shared__ f32x4 lds[4 * kB * 64 > kStreamJoin / 2 ? 4 * kB * 64 : kStreamJoin / 2];
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
  join_splits<D, kRows>(a, p, seq, unit, active, row0, h, G, reinterpret_cast<float*>(lds));
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
  int64_t per, slots, most_splits;  // rows of a workgroup, workgroups that fill the chip
  p.tiled = rows > 32;
  if (p.tiled) {
    slots = dim == 256 ? 256 : 512;
    most_splits = 256;
    const int64_t most = 64 * attn_tile_max(dim);
    int64_t blocks = (rows + most - 1) / most;
    if (blocks * B * heads < slots && max_len <= 2048) blocks = (rows + 63) / 64;
    p.row_tiles = (int)((rows + 64 * blocks - 1) / (64 * blocks));
    per = 64 * p.row_tiles;
  } else {
    p.row_tiles = rows <= 16 ? 1 : 2;
    per = 16 * p.row_tiles;
    slots = 1024;
    most_splits = kStreamJoin / per;
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
  if (most > most_splits) most = most_splits;
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
