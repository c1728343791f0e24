// kv_attention.hip -- attention over the paged NVFP4 cache for few query rows
// per key: one token per sequence, a few drafted tokens. (More rows:
// kv_attention_tile.hip; the mathematics: kv_attention_common.h.)
//
// A workgroup takes 16 or 32 query rows (query x head of one kv head's group)
// of a sequence and a stretch of its keys; its four waves take a quarter of
// the stretch each, with a running maximum and sum per row (one pass over the
// cache), and join in LDS. A long key axis is split over workgroups; up to 16
// splits are joined by the one that arrives last, more by a kernel of their own.
//
// Long axes are bound by memory: one token of 64 sequences of up to 8192 keys
// (8 heads of 128, 308 MB) 68 to 74 us, 4.2 to 4.5 TB/s; of 4 of 131072 keys
// (604 MB) 118 us, 5.1 TB/s. One sequence of 4097 keys takes 10.3 us, its chain of trips:
// lengths and page numbers, records, partials out, arrival, partials in. So
// page numbers are asked for before the lengths, records before the query
// rows, and a step's records while the step before is computed.
//
// Sinks and drafted trees are in kernels of their own (MASKED), which walk over
// the sinks and then the window, and take a mask of 32 bits a row from the
// tree's words in the few steps that need one. There this kernel also serves
// up to some hundred rows, where calls are too short for tiles: 16 trees of up
// to 61 tokens (8 heads of 64 a kv head, window 2000) 31 us, in tiles 47.
#include "kv_attention_common.h"

namespace nvfp4 {
namespace {

// More splits of a unit than this are joined by a kernel of their own: one
// workgroup takes 16 partials of its rows in one trip.
constexpr int kJoinHere = 16;

#if defined(__HIP_DEVICE_COMPILE__)
template <int D, int RT, int P, int Y>
__device__ __forceinline__ void pv(f32x4 (&o)[RT][D / 16], const VFrag<D> (&f)[2], const f16x4 (&vs)[2],
                                   const f16x8 (&pf)[P][RT]) {
  const f16x8 vf = v_operand<Y>(f, vs);
#pragma unroll
  for (int t = 0; t < RT; ++t)
#pragma unroll
    for (int x = 0; x < P; ++x) o[t][Y] = mfma16x16x32(vf, pf[x][t], o[t][Y]);
  if constexpr (Y + 1 < D / 16) pv<D, RT, P, Y + 1>(o, f, vs, pf);
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

// Joins the at most kJoinHere splits of a unit in split order, so that the
// result does not depend on which workgroup arrived last. What this costs is
// trips to device scope: partials are asked for together with the statistics.
// (Splits as a chain of branches: as a loop with a break one token of 64
// sequences of up to 8192 keys took 78 us, not 68; without branches 69.)
// PER items of a thread at a time, of at most kJoinHere / PER splits: 32 rows of
// 128 channels are 4 items a thread, whose trips one after the other were 5.6
// of the 20 us of a tree of 24 tokens over 4097 keys.
template <int D, int kRows, int PER>
__device__ __forceinline__ void join_splits(const AttnArgs& a, const AttnPlan& p, const Seq& seq, unsigned unit, int active,
                                            int row0, int h, int G, float* lds) {
  const float vg = *a.v_g;
  const float* parts = a.part + (int64_t)unit * p.splits * p.part_floats;
  const Rsrc ra = make_rsrc(parts, (uint32_t)(active * p.part_floats * 4));
  const int live = (seq.rows - row0 < kRows ? seq.rows - row0 : kRows) * (D / 4);
  constexpr int kSplits = kJoinHere / PER;
  f32x4 x[PER][kSplits];
  auto load = [&](int n0) {  // past the last split or row: zeros, unread
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int n = n0 + 256 * i;
      const uint32_t at = (uint32_t)(8 * kRows + n * 16);
#pragma unroll
      for (int s = 0; s < kSplits; ++s)
        x[i][s] = __builtin_bit_cast(f32x4, bload16_dev(ra, s < active && n < live ? at + (uint32_t)(s * p.part_floats * 4) : kOutOfRange));
    }
  };
  load(threadIdx.x);
  float* jm = lds;  // [active][kRows] m, then l
  float* jl = lds + kJoinHere * kRows;
  for (int n = threadIdx.x; n < active * kRows; n += 256) {
    const uint32_t at = (uint32_t)((n / kRows * p.part_floats + n % kRows) * 4);
    jm[n] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(ra, (int)at, 0, 16));
    jl[n] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(ra, (int)at, 4 * kRows, 16));
  }
  __syncthreads();
  for (int n0 = threadIdx.x; n0 < live; n0 += 256 * PER) {
    if (n0 >= 256) load(n0);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int n = n0 + 256 * i, rr = n / (D / 4), d = n % (D / 4) * 4;
      if (PER > 1 && n >= live) break;
      float m = kNoKey;
      for (int s = 0; s < active; ++s) m = __builtin_fmaxf(m, jm[s * kRows + rr]);
      float l = 0.0f;
      f32x4 v = {0.f, 0.f, 0.f, 0.f};
      static_for<kSplits>([&](auto step) {
        constexpr int s = decltype(step)::value;
        if (s < active) {
          const float w = __builtin_amdgcn_exp2f(jm[s * kRows + rr] - m);
          l += w * jl[s * kRows + rr];
          v += x[i][s] * w;
        }
      });
      const int64_t orow = out_row(a, seq, row0 + rr, h, G);
      store4(a, orow * D + d, v * inverse_sum(l, vg));
      if (d == 0 && a.lse != nullptr) a.lse[orow] = lse_of(m, l);
    }
  }
}
#endif

// Workgroups per CU that the registers are held to. 16 plain rows of 64
// channels: five, as 1280 units are one round of the chip so: 160 sequences of
// up to 2048 keys on 8 heads 31.5 us, 35.3 with four (bound 4 gave 98 registers,
// 2 too many); of 200 sequences of up to 3000 keys, f32, 64.8 and 62.7.
template <int D, int RT, bool MASKED>
constexpr int kAttnWgs = D == 256 ? 3 - RT : RT == 2 ? 2 : D == 64 ? (MASKED ? 4 : 5) : 3;

// P: f16 parts of a probability. MASKED: sinks or a tree mask.
template <int D, int RT, int P, bool MASKED>
__global__ __launch_bounds__(256, (kAttnWgs<D, RT, MASKED>)) void k_kv_attention(AttnArgs a, AttnPlan p) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int kB = D / 16, kW = D / 32, kRows = 16 * RT;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, quad = lane >> 4;
  const int G = a.heads_q / a.c.heads;
  // grid: (head, row block, sequence) fastest to slowest in x, split in y
  const unsigned unit = blockIdx.x, heads = a.c.heads, blocks = p.row_blocks;
  const int h = (int)(unit % heads);
  unsigned rb = unit / heads % blocks, b = unit / heads / blocks;
  if (MASKED && p.packed) {
    const Block at = packed_block(a, p, unit, G, lane);
    b = at.b;
    rb = at.rb;
  }
  const int split = blockIdx.y;

  // Without a window the page numbers of this split can be asked for before
  // the lengths are known.
  Walk<D> walk(a, b, h, a.window > 0 ? 0 : split * (p.chunk / 16), lane);
  const Seq seq = seq_of(a, b, G);
  if ((int64_t)rb * kRows >= seq.rows) return;
  const int row0 = (int)rb * kRows;
  const Stretch all = active_splits<MASKED>(a, p, seq, row0, kRows, G);
  const int active = all.splits;
  // [lo_full, hi_full) need no mask.
  const int hi_full = MASKED && a.tree != nullptr ? tree_context(seq) : sees_hi(seq, row0 / G);
  const int lo_full = sees_lo(all.hi, a.window);
  if (split >= active) return;

  // This wave's stretch, whole steps of 32 tokens. Its first records are asked
  // for before the query rows.
  const int s_first = all.start + split * p.chunk;
  const int s_last = all.end - s_first > p.chunk ? s_first + p.chunk : all.end;
  const int steps = s_last > s_first ? (s_last - s_first + 31) / 32 : 0, per = (steps + 3) / 4;
  const int step0 = wave * per, step1 = step0 + per < steps ? step0 + per : steps;

  struct Pair {
    KFrag<D> k[2];
    VFrag<D> v[2];
    bool ok[2];
  };
  int ahead = s_first + 32 * step0;  // the next step fetched
  auto fetch = [&](Pair& f) {
    if constexpr (MASKED) {
      if (ahead == all.head && all.gap > 0) walk.start((ahead + all.gap) >> 4);
      ahead += 32;
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const Rsrc rec = walk.record(f.ok[x], lane);
      load_k(f.k[x], rec, lane);
      load_v(f.v[x], rec, lane, 0);
      walk.step(1);
    }
  };
  // Trees at D 128: records two steps ahead (64 tokens over 4096 keys 26.2 ->
  // 24.9 us, 16 times over 8192 201 -> 195; with 16 rows 0 to 7% slower, at D 64
  // no difference, at D 256 no registers).
  constexpr bool kTwoAhead = MASKED && D == 128 && RT == 2;
  Pair fa, fb;
  if (step0 < step1) {
    walk.start(all.key<MASKED>(ahead) >> 4);
    fetch(fa);
    if (kTwoAhead && step0 + 1 < step1) fetch(fb);
  }
  __shared__ uint32_t no_number[4][kB], nan_rows[4][kRows];  // MASKED: by wave
  if (MASKED && lane < kRows) nan_rows[wave][lane] = 0;
  Rows<D, RT> r;
  load_rows<D, RT, MASKED>(r, a, seq, row0, h, G, quad, col);
  auto attend = [&](Pair& f, int base) {
    const bool edge = (MASKED ? masked_edge(a, base, lo_full, hi_full) : base + 32 > hi_full || base < lo_full) || !f.ok[0] || !f.ok[1];
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
      if constexpr (!MASKED) hide_scores<D, RT>(r, sc, base, quad, f.ok);
      // Tokens no row sees may never have been written: their V scales
      // become zero, so that no NaN code meets a zero probability.
#pragma unroll
      for (int x = 0; x < 2; ++x) f.v[x].s &= f.ok[x] ? (MASKED ? masked_bytes(a, base + 16 * x + 4 * quad, all.lo, all.hi) : byte_mask(base + 16 * x + 4 * quad, all.lo, all.hi)) : 0u;
      if constexpr (MASKED) {
        const bool nans = any_nan(f.v);
        if (nans) take_nans(f.v, lane, no_number[wave]);
        hide_masked<D, RT>(r, a, seq, sc, base, quad, f.ok, [&](int t, uint32_t see) {
          if (nans) note_nans<D>(nan_rows[wave] + 16 * t, lane, see, no_number[wave], true, true);
        });
      }
    }
    f16x8 pf[P][RT];
    float mx[RT];
    lane_maximum<RT>(sc, mx);
    renew_maximum<D, RT>(r, mx);
    probabilities<D, RT, P>(r, sc, pf);
    const f16x4 vs[2] = {e4m3x4_f16(f.v[0].s), e4m3x4_f16(f.v[1].s)};
    pv<D, RT, P, 0>(r.o, f.v, vs, pf);
  };
  // The next step's records are on their way while one is computed.
  if constexpr (kTwoAhead) {
    Pair fc;
    for (int st = step0; st < step1; st += 3) {
      const int base = s_first + 32 * st;
      if (st + 2 < step1) fetch(fc);
      attend(fa, all.key<MASKED>(base));
      if (st + 1 >= step1) break;
      if (st + 3 < step1) fetch(fa);
      attend(fb, all.key<MASKED>(base + 32));
      if (st + 2 >= step1) break;
      if (st + 4 < step1) fetch(fb);
      attend(fc, all.key<MASKED>(base + 64));
    }
  } else if (step0 < step1) {
    for (int st = step0; st < step1; st += 2) {
      const int base = s_first + 32 * st;
      if (st + 1 < step1) fetch(fb);
      attend(fa, all.key<MASKED>(base));
      if (st + 1 >= step1) break;
      if (st + 2 < step1) fetch(fa);
      attend(fb, all.key<MASKED>(base + 32));
    }
  }
  finish_rows<D, RT>(r);

  // The four waves' results become one: weights exp2(m_w - m) per row.
  __shared__ float wm[4][kRows], wl[4][kRows];
  __shared__ f32x4 lds[4 * kB * 64];
  auto wo = [&](int w, int y) -> f32x4& { return lds[(w * kB + y) * 64 + lane]; };
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    if (quad == 0) {
      wm[wave][16 * t + col] = row_maximum<D, RT>(r, t);
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
    const float alpha = __builtin_amdgcn_exp2f(wm[wave][rr] - m);
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
    const uint32_t bad = MASKED ? nan_rows[0][rr] | nan_rows[1][rr] | nan_rows[2][rr] | nan_rows[3][rr] : 0u;
    for (int y = wave; y < kB; y += 4) {
      const f32x4 v = nan_if(bad >> y & 1u, wo(0, y) + wo(1, y) + wo(2, y) + wo(3, y));
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
  if (active == 1 || p.splits > kJoinHere) return;
  __shared__ uint32_t arrived;
  if (!split_last(a.counters + unit, active, &arrived)) return;
  float* const stats = reinterpret_cast<float*>(lds);
  if (MASKED && active <= kJoinHere / 4) join_splits<D, kRows, 4>(a, p, seq, unit, active, row0, h, G, stats);
  else if (MASKED && active <= kJoinHere / 2) join_splits<D, kRows, 2>(a, p, seq, unit, active, row0, h, G, stats);
  else join_splits<D, kRows, 1>(a, p, seq, unit, active, row0, h, G, stats);
#endif  // __HIP_DEVICE_COMPILE__
}

// The join of split units by a kernel of its own: 1024 / D / SLICES rows a
// workgroup, a thread four channels of every SLICES-th run of kRun splits. In
// the order of the runs, whatever the timing. In one workgroup a unit (the
// last to arrive) it took 64 rows 5 us a split; so, spread over the chip and
// with 8 loads in flight a thread, about 5 us in all. One slice where a run
// holds all splits: with four, three of them idle, 512 units of 64 rows of 64
// channels took 19 us for two splits.
constexpr int kRun = 8;
template <int D, int SLICES, bool MASKED>
__global__ __launch_bounds__(256) void k_kv_join(AttnArgs a, AttnPlan p) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int kSlices = SLICES, kThreads = D / 4, kRowsHere = 256 / kThreads / kSlices;
  const int G = a.heads_q / a.c.heads, rows_wg = p.rows;
  const unsigned unit = blockIdx.x, heads = a.c.heads, blocks = p.row_blocks;
  const int h = (int)(unit % heads);
  unsigned rb = p.tiled ? blocks - 1 - unit / heads % blocks : unit / heads % blocks, b = unit / heads / blocks;
  if (MASKED && p.packed) {
    const Block at = packed_block(a, p, unit, G, threadIdx.x & 63);
    b = at.b;
    rb = at.rb;
  }
  const Seq seq = seq_of(a, b, G);
  const int slot = threadIdx.x / kThreads, slice = slot % kSlices, d = threadIdx.x % kThreads * 4;
  const int rr = blockIdx.y * kRowsHere + slot / kSlices;
  if ((int64_t)rb * rows_wg + blockIdx.y * kRowsHere >= seq.rows) return;
  const int row0 = (int)rb * rows_wg;
  const int active = active_splits<MASKED>(a, p, seq, row0, rows_wg, G).splits;
  if (active == 1) return;
  const float* part = a.part + (int64_t)unit * p.splits * p.part_floats;
  float m = kNoKey, l = 0.0f;
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
  if (row0 + rr < seq.rows) {
    for (int s0 = slice * kRun; s0 < active; s0 += kSlices * kRun) {
      float pm[kRun], pl[kRun];
      f32x4 px[kRun];
#pragma unroll
      for (int e = 0; e < kRun; ++e) {
        const int s = s0 + e < active ? s0 + e : active - 1;
        const float* ps = part + (int64_t)s * p.part_floats;
        pm[e] = ps[rr];
        pl[e] = ps[rows_wg + rr];
        px[e] = *reinterpret_cast<const f32x4*>(ps + 2 * rows_wg + rr * D + d);
      }
      float mn = m;
#pragma unroll
      for (int e = 0; e < kRun; ++e) mn = __builtin_fmaxf(mn, pm[e]);
      const float alpha = __builtin_amdgcn_exp2f(m - mn);
      m = mn;
      l *= alpha;
      v *= alpha;
#pragma unroll
      for (int e = 0; e < kRun; ++e) {
        const float w = s0 + e < active ? __builtin_amdgcn_exp2f(pm[e] - m) : 0.0f;
        l += w * pl[e];
        v += px[e] * w;
      }
    }
  }
  if constexpr (kSlices > 1) {
    __shared__ f32x4 jv[256];
    __shared__ float jm[256], jl[256];
    jm[threadIdx.x] = m;
    jl[threadIdx.x] = l;
    jv[threadIdx.x] = v;
    __syncthreads();
    if (slice != 0 || row0 + rr >= seq.rows) return;
#pragma unroll
    for (int z = 1; z < kSlices; ++z) m = __builtin_fmaxf(m, jm[threadIdx.x + z * kThreads]);
    l = 0.0f;
    v = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int z = 0; z < kSlices; ++z) {
      const int at = threadIdx.x + z * kThreads;
      const float w = __builtin_amdgcn_exp2f(jm[at] - m);
      l += w * jl[at];
      v += jv[at] * w;
    }
  } else if (row0 + rr >= seq.rows) {
    return;
  }
  const int64_t orow = out_row(a, seq, row0 + rr, h, G);
  store4(a, orow * D + d, v * inverse_sum(l, *a.v_g));
  if (d == 0 && a.lse != nullptr) a.lse[orow] = lse_of(m, l);
#endif
}

// The rows of a drafted tree's mask from its parents, a thread a row: it walks
// up its ancestors, whose numbers only fall, so that the words are finished
// from the last to the first. What bounds it is the chain of LDS reads: a read
// gives four ancestors. 16 trees of up to 61 tokens 3.1 us (4.1 with one), a
// chain of 4096 302.
constexpr int kTreeThreads = 256;
__global__ __launch_bounds__(kTreeThreads) void k_tree_mask(TreeArgs a) {
#if defined(__HIP_DEVICE_COMPILE__)
  __shared__ struct alignas(8) { int16_t up[4]; } above[kMaxTree];  // ancestors 1 to 4 steps up, or -1
  const int64_t b = blockIdx.x;
  int64_t q0 = b * a.max_q, n = a.max_q;
  if (a.q_offsets != nullptr) {
    q0 = a.q_offsets[b];
    n = a.q_offsets[b + 1] - q0;
    if (q0 < 0 || q0 > a.T) n = 0;
    if (n > a.T - q0) n = a.T - q0;
    if (n > a.max_q) n = a.max_q;
  }
  const int row0 = (int)blockIdx.y * kTreeThreads, i = row0 + (int)threadIdx.x;
  if (row0 >= n) return;
  const int first = a.positions != nullptr ? a.positions[q0] : 0;
  const int rows = row0 + kTreeThreads < n ? row0 + kTreeThreads : (int)n;
  for (int at = threadIdx.x; at < rows; at += kTreeThreads) {
    const int p = a.parents[q0 + at];
    above[at].up[0] = (int16_t)(p >= 0 && p < at ? p : -1);
  }
  __syncthreads();
  for (int at = threadIdx.x; at < rows; at += kTreeThreads) {
    const int p = above[at].up[0];
    above[at].up[1] = p < 0 ? (int16_t)-1 : above[p].up[0];
  }
  __syncthreads();
  for (int at = threadIdx.x; at < rows; at += kTreeThreads) {
    const int p = above[at].up[1];
    above[at].up[2] = p < 0 ? (int16_t)-1 : above[p].up[0];
    above[at].up[3] = p < 0 ? (int16_t)-1 : above[p].up[1];
  }
  __syncthreads();
  if (i >= n) return;
  uint64_t* out = a.tree + (q0 + i) * a.tree_words;
  int word = a.tree_words - 1, depth = -1;
  uint64_t bits = 0;
  auto take = [&](int at) {
    if (at < 0) return;
    for (; word > at >> 6; --word) {
      out[word] = bits;
      bits = 0;
    }
    bits |= uint64_t(1) << (at & 63);
    ++depth;
  };
  for (int at = i; at >= 0;) {
    const auto next = above[at];
    take(at);
#pragma unroll
    for (int x = 0; x < 3; ++x) take(next.up[x]);
    at = next.up[3];
  }
  for (; word >= 0; --word) {
    out[word] = bits;
    bits = 0;
  }
  // The first row's depth is 0: its position, which the others read, stays.
  if (a.positions != nullptr && i > 0) a.positions[q0 + i] = first + depth;
#endif
}

template <int D, int P, bool MASKED>
void launch_parts(const AttnArgs& a, const AttnPlan& p, hipStream_t s) {
  const dim3 grid((unsigned)p.units, (unsigned)p.splits);
  if (p.row_tiles == 1) k_kv_attention<D, 1, P, MASKED><<<grid, dim3(256), 0, s>>>(a, p);
  else k_kv_attention<D, 2, P, MASKED><<<grid, dim3(256), 0, s>>>(a, p);
}
template <int D>
void launch_stream(const AttnArgs& a, const AttnPlan& p, hipStream_t s) {
  if (attn_masked(a)) {
    if (a.f32_out) launch_parts<D, 2, true>(a, p, s);
    else launch_parts<D, 1, true>(a, p, s);
  } else if (a.f32_out) {
    launch_parts<D, 2, false>(a, p, s);
  } else {
    launch_parts<D, 1, false>(a, p, s);
  }
}
template <int D, int SLICES>
void launch_slices(const AttnArgs& a, const AttnPlan& p, hipStream_t s) {
  const dim3 grid((unsigned)p.units, (unsigned)(p.rows * D / (1024 / SLICES)));
  if (attn_masked(a)) k_kv_join<D, SLICES, true><<<grid, dim3(256), 0, s>>>(a, p);
  else k_kv_join<D, SLICES, false><<<grid, dim3(256), 0, s>>>(a, p);
}
template <int D>
void launch_join(const AttnArgs& a, const AttnPlan& p, hipStream_t s) {
  if (p.splits <= kRun) launch_slices<D, 1>(a, p, s);
  else launch_slices<D, 4>(a, p, s);
}

}  // namespace

hipError_t launch_tree_mask(const TreeArgs& a, int64_t B, hipStream_t s) {
  const dim3 grid((unsigned)B, (unsigned)((a.max_q + kTreeThreads - 1) / kTreeThreads));
  k_tree_mask<<<grid, dim3(kTreeThreads), 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_kv_attention(const AttnArgs& a, const AttnPlan& p, hipStream_t s) {
  if (p.tiled) {
    const hipError_t e = launch_kv_attention_tile(a, p, s);
    if (e != hipSuccess) return e;
  } else if (a.c.dim == 64) {
    launch_stream<64>(a, p, s);
  } else if (a.c.dim == 128) {
    launch_stream<128>(a, p, s);
  } else {
    launch_stream<256>(a, p, s);
  }
  if (p.splits > (p.tiled ? 1 : kJoinHere)) {
    if (a.c.dim == 64) launch_join<64>(a, p, s);
    else if (a.c.dim == 128) launch_join<128>(a, p, s);
    else launch_join<256>(a, p, s);
  }
  return hipGetLastError();
}

}  // namespace nvfp4
