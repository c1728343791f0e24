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
template <int D, int kRows>
__device__ __forceinline__ void join_splits(const AttnArgs& a, const AttnPlan& p, const Seq& seq, unsigned unit, int active,
                                            int row0, int h, int G, float* lds) {
  const float vg = *a.v_g;
  const float* parts = a.part + (int64_t)unit * p.splits * p.part_floats;
  const Rsrc ra = make_rsrc(parts, (uint32_t)(active * p.part_floats * 4));
  const int live = (seq.rows - row0 < kRows ? seq.rows - row0 : kRows) * (D / 4);
  f32x4 x[kJoinHere];
  auto load = [&](int n) {  // past the last split or row: zeros, unread
    const uint32_t at = (uint32_t)(8 * kRows + n * 16);
#pragma unroll
    for (int s = 0; s < kJoinHere; ++s)
      x[s] = __builtin_bit_cast(f32x4, bload16_dev(ra, s < active && n < live ? at + (uint32_t)(s * p.part_floats * 4) : kOutOfRange));
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
  for (int n = threadIdx.x; n < live; n += 256) {
    const int rr = n / (D / 4), d = n % (D / 4) * 4;
    float m = kNoKey;
    for (int s = 0; s < active; ++s) m = __builtin_fmaxf(m, jm[s * kRows + rr]);
    float l = 0.0f;
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
    if (n >= 256) load(n);
    static_for<kJoinHere>([&](auto step) {
      constexpr int s = decltype(step)::value;
      if (s < active) {
        const float w = __builtin_amdgcn_exp2f(jm[s * kRows + rr] - m);
        l += w * jl[s * kRows + rr];
        v += x[s] * w;
      }
    });
    const int64_t orow = out_row(a, seq, row0 + rr, h, G);
    store4(a, orow * D + d, v * inverse_sum(l, vg));
    if (d == 0 && a.lse != nullptr) a.lse[orow] = lse_of(m, l);
  }
}
#endif

// Workgroups per CU that the registers are held to.
template <int D, int RT>
constexpr int kAttnWgs = D == 256 ? 3 - RT : RT == 2 ? 2 : D == 64 ? 4 : 3;

// P: f16 parts of a probability.
template <int D, int RT, int P>
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

  // Without a window the page numbers of this split can be asked for before
  // the lengths are known.
  Walk<D> walk(a, b, h, a.window > 0 ? 0 : split * (p.chunk / 16), lane);
  const Seq seq = seq_of(a, b, G);
  if ((int64_t)rb * kRows >= seq.rows) return;
  const int row0 = (int)rb * kRows;
  const Stretch all = active_splits(a, p, seq, row0, kRows, G);
  const int hi_all = all.hi, lo_all = all.lo, active = all.splits;
  const int hi_full = sees_hi(seq, row0 / G), lo_full = sees_lo(hi_all, a.window);  // [lo_full, hi_full) need no mask
  if (split >= active) return;

  // This wave's stretch, whole steps of 32 tokens. Its first records are asked
  // for before the query rows.
  const int s_first = all.start + split * p.chunk;
  const int s_last = hi_all - s_first > p.chunk ? s_first + p.chunk : hi_all;
  const int steps = s_last > s_first ? (s_last - s_first + 31) / 32 : 0, per = (steps + 3) / 4;
  const int step0 = wave * per, step1 = step0 + per < steps ? step0 + per : steps;

  struct Pair {
    KFrag<D> k[2];
    VFrag<D> v[2];
    bool ok[2];
  };
  auto fetch = [&](Pair& f) {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const Rsrc rec = walk.record(f.ok[x], lane);
      load_k(f.k[x], rec, lane);
      load_v(f.v[x], rec, lane, 0);
      walk.step(1);
    }
  };
  Pair fa, fb;
  if (step0 < step1) {
    walk.start((s_first >> 4) + 2 * step0);
    fetch(fa);
  }
  Rows<D, RT> r;
  load_rows<D, RT>(r, a, seq, row0, h, G, quad, col);
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
    f16x8 pf[P][RT];
    float mx[RT];
    lane_maximum<RT>(sc, mx);
    renew_maximum<D, RT>(r, mx);
    probabilities<D, RT, P>(r, sc, pf);
    const f16x4 vs[2] = {e4m3x4_f16(f.v[0].s), e4m3x4_f16(f.v[1].s)};
    pv<D, RT, P, 0>(r.o, f.v, vs, pf);
  };
  // The next step's records are on their way while one is computed.
  if (step0 < step1) {
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
  if (active == 1 || p.splits > kJoinHere) return;
  __shared__ uint32_t arrived;
  if (!split_last(a.counters + unit, active, &arrived)) return;
  join_splits<D, kRows>(a, p, seq, unit, active, row0, h, G, reinterpret_cast<float*>(lds));
#endif  // __HIP_DEVICE_COMPILE__
}

// The join of split units by a kernel of its own: 1024 / D / kSlices rows a
// workgroup, a thread four channels of every kSlices-th run of kRun splits. In
// the order of the runs, whatever the timing. In one workgroup a unit (the
// last to arrive) it took 64 rows 5 us a split; so, spread over the chip and
// with 8 loads in flight a thread, about 5 us in all.
template <int D>
__global__ __launch_bounds__(256) void k_kv_join(AttnArgs a, AttnPlan p) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int kSlices = 4, kRun = 8, kThreads = D / 4, kRowsHere = 256 / kThreads / kSlices;
  const int G = a.heads_q / a.c.heads, rows_wg = p.rows;
  const unsigned unit = blockIdx.x, heads = a.c.heads, blocks = p.row_blocks;
  const int h = (int)(unit % heads);
  const unsigned rb = p.tiled ? blocks - 1 - unit / heads % blocks : unit / heads % blocks, b = unit / heads / blocks;
  const Seq seq = seq_of(a, b, G);
  const int slot = threadIdx.x / kThreads, slice = slot % kSlices, d = threadIdx.x % kThreads * 4;
  const int rr = blockIdx.y * kRowsHere + slot / kSlices;
  if ((int64_t)rb * rows_wg + blockIdx.y * kRowsHere >= seq.rows) return;
  const int row0 = (int)rb * rows_wg;
  const int active = active_splits(a, p, seq, row0, rows_wg, G).splits;
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
  const int64_t orow = out_row(a, seq, row0 + rr, h, G);
  store4(a, orow * D + d, v * inverse_sum(l, *a.v_g));
  if (d == 0 && a.lse != nullptr) a.lse[orow] = lse_of(m, l);
#endif
}

template <int D, int P>
void launch_parts(const AttnArgs& a, const AttnPlan& p, hipStream_t s) {
  const dim3 grid((unsigned)p.units, (unsigned)p.splits);
  if (p.row_tiles == 1) k_kv_attention<D, 1, P><<<grid, dim3(256), 0, s>>>(a, p);
  else k_kv_attention<D, 2, P><<<grid, dim3(256), 0, s>>>(a, p);
}
template <int D>
void launch_stream(const AttnArgs& a, const AttnPlan& p, hipStream_t s) {
  if (a.f32_out) launch_parts<D, 2>(a, p, s);
  else launch_parts<D, 1>(a, p, s);
}
template <int D>
void launch_join(const AttnArgs& a, const AttnPlan& p, hipStream_t s) {
  k_kv_join<D><<<dim3((unsigned)p.units, (unsigned)(p.rows * D / 256)), dim3(256), 0, s>>>(a, p);
}

}  // namespace

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
