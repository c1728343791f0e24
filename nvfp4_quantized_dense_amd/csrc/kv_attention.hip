// kv_attention.hip -- attention over the paged NVFP4 cache, for few query rows
// per key: one token per sequence, drafted tokens, short chunks.
//
//   o_i = sum_j softmax_j(scale q_i . k_j) v_j over the keys a query sees.
//
// A workgroup takes 16 or 32 query rows (query x head of one kv head's group)
// of a sequence and a stretch of its keys; its four waves take a quarter of
// the stretch each, with a running maximum and sum per row (one pass over the
// cache). Both products run on the f16 matrix core:
//   S^T = K Q^T  (rows: 16 tokens, columns: query rows)
//   O^T = V^T P  (rows: 16 channels, columns: query rows, 32 tokens deep)
// A code times its E4M3 scale has at most 6 significant bits and lies in
// [2^-10, 2688], exact in f16. A bf16 query row is scaled by a power of two
// to at most 1 before it becomes f16: exact but for elements 2^-14 below the
// row's largest, which are off by 2^-25 of it. Probabilities are rounded to
// f16 for the second product (half a step 2^-11, or 2^-25 absolute under
// 2^-14); their sum is kept in fp32. S^T leaves a lane with the tokens of
// one query row that the second product wants from that lane, because the
// record's V codes are stored in the same token order, so the probabilities
// never leave their registers, and the row statistics are one number a lane.
#include "attention.h"
#include "kv_layout.h"

namespace nvfp4 {
namespace {

typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));

constexpr float kNoKey = -3.0e38f;  // running maximum before the first key
constexpr float kLog2e = 1.44269504088896341f;
constexpr float kLn2 = 0.693147180559945309f;

__device__ __forceinline__ float sum_xor16(float v) {
  const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(p[0]) + __uint_as_float(p[1]);
}
__device__ __forceinline__ float sum_xor32(float v) {
  const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(p[0]) + __uint_as_float(p[1]);
}

// The 4 E4M3 bytes of a dword as f16 (exact).
__device__ __forceinline__ f16x4 e4m3x4_f16(uint32_t w) {
  const f16x2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, false);
  const f16x2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, true);
  return f16x4{a[0], a[1], b[0], b[1]};
}

// A lane's share of a record: the codes of its token (K) and channel (V), its
// token's K scales, and the V scales of block lane % (D / 16) of its quad (the
// other blocks' are with the quad's other lanes).
template <int D>
struct Frag {
  static constexpr int kW = D / 32;   // code dwords
  uint32_t k[kW], v[kW], ks, vs;
};

template <int N>
__device__ __forceinline__ void load_words(uint32_t (&w)[N], const uint8_t* p) {
  if constexpr (N == 2) {
    const u32x2 t = *reinterpret_cast<const u32x2*>(p);
    w[0] = t[0]; w[1] = t[1];
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const u32x4 t = *reinterpret_cast<const u32x4*>(p + 4 * i);
      w[i] = t[0]; w[i + 1] = t[1]; w[i + 2] = t[2]; w[i + 3] = t[3];
    }
  }
}

template <int D>
__device__ __forceinline__ void load_frag(Frag<D>& f, const uint8_t* rec, int lane) {
  using R = KvRec<D>;
  load_words(f.k, rec + lane * R::kLane);
  load_words(f.v, rec + R::kV + lane * R::kLane);
  const uint8_t* s = rec + R::kKs + lane * (D / 64);
  if constexpr (D == 64) f.ks = *s;
  else if constexpr (D == 128) f.ks = *reinterpret_cast<const uint16_t*>(s);
  else f.ks = *reinterpret_cast<const uint32_t*>(s);
  f.vs = *reinterpret_cast<const uint32_t*>(rec + R::kVs + (lane >> 4) * (D / 4) + (lane & (D / 16 - 1)) * 4);
}

// Lane N's value in each row of 16 lanes.
template <int N>
__device__ __forceinline__ uint32_t row_bcast(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x150 + N, 0xF, 0xF, true);
}

// V^T of channel block Y as an operand: 4 tokens of each of two records.
template <int D, int Y>
__device__ __forceinline__ f16x8 v_operand(const Frag<D> (&f)[2], const f16x4 (&vs)[2]) {
  f16x8 r;
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const uint32_t w = f[x].v[Y >> 1];
    const u32x2 s = __builtin_bit_cast(u32x2, vs[x]);
    const f16x2 lo = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 2 * (Y & 1)) * __builtin_bit_cast(f16x2, row_bcast<Y>(s[0]));
    const f16x2 hi = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 2 * (Y & 1) + 1) * __builtin_bit_cast(f16x2, row_bcast<Y>(s[1]));
    r[4 * x] = lo[0]; r[4 * x + 1] = lo[1]; r[4 * x + 2] = hi[0]; r[4 * x + 3] = hi[1];
  }
  return r;
}

template <int D, int RT, int Y>
__device__ __forceinline__ void pv(f32x4 (&o)[RT][D / 16], const Frag<D> (&f)[2], const f16x4 (&vs)[2], const f16x8 (&pf)[RT]) {
  const f16x8 vf = v_operand<D, Y>(f, vs);
#pragma unroll
  for (int t = 0; t < RT; ++t) o[t][Y] = mfma16x16x32(vf, pf[t], o[t][Y]);
  if constexpr (Y + 1 < D / 16) pv<D, RT, Y + 1>(o, f, vs, pf);
}

// Keeps the bytes of the quad's tokens first .. first + 3 that lie in [lo, hi).
__device__ __forceinline__ uint32_t byte_mask(int first, int lo, int hi) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (first + i >= lo && first + i < hi) m |= 255u << (8 * i);
  return m;
}

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
  int64_t unit = blockIdx.x;
  const int h = (int)(unit % a.c.heads);
  const int64_t rb = unit / a.c.heads % p.row_blocks, b = unit / a.c.heads / p.row_blocks;
  const int split = blockIdx.y;

  int64_t q0, nq;
  if (a.q_offsets != nullptr) {
    q0 = a.q_offsets[b];
    nq = a.q_offsets[b + 1] - q0;
    if (q0 < 0 || q0 > a.T) nq = 0;
    else if (nq > a.T - q0) nq = a.T - q0;
  } else {
    nq = a.T / a.B;
    q0 = b * nq;
  }
  const int64_t rows = (nq < a.max_q ? nq : a.max_q) * G, row0 = rb * kRows;
  if (row0 >= rows) return;
  // Keys: positions fit 31 bits (max_len and the table are bounded so).
  int len = a.seq_lens[b];
  len = len < 0 ? 0 : len;
  if (len > a.max_len) len = (int)a.max_len;
  const int64_t room = a.table_width * a.c.page_size;
  if (len > room) len = (int)room;
  const int i_first = (int)(row0 / G);
  const int64_t last_row = rows - 1 < row0 + kRows - 1 ? rows - 1 : row0 + kRows - 1;
  const int i_last = (int)(last_row / G);
  // Query i stands at position len - nq + i and sees [lo, hi) of it.
  auto hi_of = [&](int i) { const int64_t e = (int64_t)len - nq + i + 1; return (int)(e < 0 ? 0 : e); };
  auto lo_of = [&](int hi) { return a.window > 0 && hi > a.window ? (int)(hi - a.window) : 0; };
  const int hi_all = hi_of(i_last), lo_all = lo_of(hi_of(i_first));
  const int start = lo_all & ~31;
  const int active = hi_all > lo_all ? (int)((hi_all - start + p.chunk - 1) / p.chunk) : 1;
  if (split >= active) return;

  float row_m[RT], row_l[RT], row_f[RT], row_t[RT];
  int row_lo[RT], row_hi[RT];
  f16x8 qf[RT][kW];
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    const int64_t row = row0 + 16 * t + col;
    const bool live = row < rows;
    const int64_t i = live ? row / G : 0;
    const int head = h * G + (int)(row - i * G);
    row_hi[t] = live ? hi_of((int)i) : 0;
    row_lo[t] = live ? lo_of(row_hi[t]) : 0;
    row_m[t] = row_t[t] = kNoKey;
    row_l[t] = 0.0f;
    uint32_t w[kW * 4];
    uint32_t top = 0;
    if (live) {
      const uint16_t* q = a.q + (q0 + i) * a.q_stride + (int64_t)head * D + quad * (D / 4);
#pragma unroll
      for (int s = 0; s < kW; ++s) {
        const u32x4 x = reinterpret_cast<const u32x4*>(q)[s];
#pragma unroll
        for (int e = 0; e < 4; ++e) w[4 * s + e] = x[e];
      }
    } else {
#pragma unroll
      for (int s = 0; s < 4 * kW; ++s) w[s] = 0u;
    }
#pragma unroll
    for (int s = 0; s < 4 * kW; ++s) top = max(top, max((w[s] << 16) & 0x7FFFFFFFu, w[s] & 0x7FFF0000u));
    top = max(top, (uint32_t)__shfl_xor((int)top, 16));
    top = max(top, (uint32_t)__shfl_xor((int)top, 32));
    // 2^-e brings the row's largest element into [1, 2): e is its exponent
    // (bounded so that both factors are normal numbers).
    int e = (int)(top >> 23) - 127;
    e = e < -100 ? -100 : (e > 126 ? 126 : e);
    float down = __uint_as_float((uint32_t)(127 - e) << 23);
    // The factor's sign goes into q, so that the largest raw score is the
    // largest score.
    const float f = __uint_as_float((uint32_t)(127 + e) << 23) * (a.scale * *a.k_g) * kLog2e;
    row_f[t] = __builtin_fabsf(f);
    if (f < 0.0f) down = -down;
#pragma unroll
    for (int s = 0; s < kW; ++s)
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        qf[t][s][2 * x] = (_Float16)(__uint_as_float(w[4 * s + x] << 16) * down);
        qf[t][s][2 * x + 1] = (_Float16)(__uint_as_float(w[4 * s + x] & 0xFFFF0000u) * down);
      }
  }
  // Keys that every live row sees need no mask.
  const int hi_full = hi_of(i_first), lo_full = lo_of(hi_all);

  f32x4 o[RT][kB];
#pragma unroll
  for (int t = 0; t < RT; ++t)
#pragma unroll
    for (int x = 0; x < kB; ++x) o[t][x] = f32x4{0.f, 0.f, 0.f, 0.f};

  const int groups = a.c.page_size / 16;
  const int32_t* table = a.table + b * a.table_stride;
  // This wave's stretch, whole steps of 32 tokens.
  const int64_t s_first = start + (int64_t)split * p.chunk;
  const int64_t s_last = s_first + p.chunk < hi_all ? s_first + p.chunk : hi_all;
  const int steps = s_last > s_first ? (int)((s_last - s_first + 31) / 32) : 0, per = (steps + 3) / 4;
  const int step0 = wave * per, step1 = step0 + per < steps ? step0 + per : steps;

  // Records are taken in order: group g is group `in` of page slot `ps`,
  // whose page number is in a lane of `tab` (64 slots from tab0 on). Groups
  // past the last key stand for the last key's and are masked.
  int g = (int)(s_first >> 4) + 2 * step0, ps = g / groups, in = g - ps * groups, tab0 = ps;
  const int g_last = (hi_all - 1) >> 4, ps_last = g_last / groups;
  int tab = 0;
  auto load_tab = [&] {
    const int at = tab0 + lane;
    tab = table[at < ps_last ? at : ps_last];
  };
  auto fetch = [&](Frag<D> (&f)[2], bool (&ok)[2]) {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      if (ps - tab0 == 64) {
        tab0 = ps;
        load_tab();
      }
      const int page = __builtin_amdgcn_readlane(tab, ps - tab0);
      ok[x] = page >= 0 && page < a.c.pages;
      load_frag<D>(f[x], a.c.cache + rec_offset<D>(ok[x] ? page : 0, a.c.heads, h, groups, in), lane);
      if (g < g_last) {
        ++g;
        if (++in == groups) { in = 0; ++ps; }
      }
    }
  };
  auto attend = [&](Frag<D> (&f)[2], const bool (&ok)[2], int base) {
    const bool edge = base + 32 > hi_full || base < lo_full || !ok[0] || !ok[1];
    // S^T of two groups, all row tiles.
    f32x4 sc[RT][2];
#pragma unroll
    for (int t = 0; t < RT; ++t) sc[t][0] = sc[t][1] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const f16x4 ks = e4m3x4_f16(f[x].ks);
#pragma unroll
      for (int s = 0; s < kW; ++s) {
        const f16x8 kf = deq8_f16(f[x].k[s], ks[s >> 1]);
#pragma unroll
        for (int t = 0; t < RT; ++t) sc[t][x] = mfma16x16x32(kf, qf[t][s], sc[t][x]);
      }
    }
    uint32_t hide[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) hide[t] = 0;
    if (edge) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int first = base + 16 * x + 4 * quad;
        // Tokens no row sees may never have been written: their V scales
        // become zero, so that no NaN code meets a zero probability.
        f[x].vs &= ok[x] ? byte_mask(first, lo_all, hi_all) : 0u;
#pragma unroll
        for (int t = 0; t < RT; ++t)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (!ok[x] || first + r < row_lo[t] || first + r >= row_hi[t]) {
              hide[t] |= 1u << (4 * x + r);
              sc[t][x][r] = -__builtin_inff();
            }
      }
    }
    f16x8 pf[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      float mx = sc[t][0][0];
#pragma unroll
      for (int r = 1; r < 8; ++r) mx = __builtin_fmaxf(mx, sc[t][r >> 2][r & 3]);
      // The subtracted maximum follows the true one only when a score passes
      // it by more than 2^8 in probability: f16 holds probabilities up to
      // that as exactly as up to 1, and most steps then need neither the
      // exchange between lanes nor the rescaling.
      if (__any(mx > row_t[t])) {
        mx = max_xor32(max_xor16(mx));
        const float mn = __builtin_fmaxf(row_m[t], mx);
        const float alpha = __builtin_amdgcn_exp2f((row_m[t] - mn) * row_f[t]);
        row_m[t] = mn;
        row_t[t] = mn == kNoKey ? kNoKey : mn + 8.0f / row_f[t];
        row_l[t] *= alpha;
#pragma unroll
        for (int y = 0; y < kB; ++y) o[t][y] *= alpha;
      }
      const float mf = -row_m[t] * row_f[t];
      float e[8];
#pragma unroll
      for (int r = 0; r < 8; ++r) e[r] = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[t][r >> 2][r & 3], row_f[t], mf));
      if (edge) {
#pragma unroll
        for (int r = 0; r < 8; ++r) e[r] = (hide[t] >> r) & 1 ? 0.0f : e[r];
      }
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        row_l[t] += e[r];
        pf[t][r] = (_Float16)e[r];
      }
    }
    // O^T += V^T P, 16 channels at a time.
    const f16x4 vs[2] = {e4m3x4_f16(f[0].vs), e4m3x4_f16(f[1].vs)};
    pv<D, RT, 0>(o, f, vs, pf);
  };
  if (step0 < step1) {
    // The next step's records are on their way while one is computed.
    Frag<D> fa[2], fb[2];
    bool ka[2], kb[2];
    load_tab();
    fetch(fa, ka);
    for (int st = step0; st < step1; st += 2) {
      const int base = (int)s_first + 32 * st;
      if (st + 1 < step1) fetch(fb, kb);
      attend(fa, ka, base);
      if (st + 1 >= step1) break;
      if (st + 2 < step1) fetch(fa, ka);
      attend(fb, kb, base + 32);
    }
  }
  // From here on in units of log2.
#pragma unroll
  for (int t = 0; t < RT; ++t) row_l[t] = sum_xor32(sum_xor16(row_l[t]));
#pragma unroll
  for (int t = 0; t < RT; ++t) row_m[t] = row_m[t] == kNoKey ? kNoKey : row_m[t] * row_f[t];

  // The four waves' results become one: weights exp2(m_w - m) per row.
  __shared__ float wm[4][kRows], wl[4][kRows];
  constexpr int kJoin = 4096;  // (split, row) pairs that the join holds
  __shared__ f32x4 lds[4 * kB * 64 > kJoin / 2 ? 4 * kB * 64 : kJoin / 2];
  auto wo = [&](int w, int y) -> f32x4& { return lds[(w * kB + y) * 64 + lane]; };
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    if (quad == 0) {
      wm[wave][16 * t + col] = row_m[t];
      wl[wave][16 * t + col] = row_l[t];
    }
  }
  __syncthreads();
  const float vg = *a.v_g;
  const int64_t slot = unit * p.splits + split;
  float* part = a.part + slot * (int64_t)p.part_floats;  // [kRows] m, [kRows] l, [kRows][D] o
  const Rsrc rp = make_rsrc(part, (uint32_t)(p.part_floats * 4));
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    const int rr = 16 * t + col;
    const float m = __builtin_fmaxf(__builtin_fmaxf(wm[0][rr], wm[1][rr]), __builtin_fmaxf(wm[2][rr], wm[3][rr]));
    const float alpha = __builtin_amdgcn_exp2f(row_m[t] - m);
    float l = 0.0f;
#pragma unroll
    for (int w = 0; w < 4; ++w) l += wl[w][rr] * __builtin_amdgcn_exp2f(wm[w][rr] - m);
    if (t > 0) __syncthreads();
#pragma unroll
    for (int y = 0; y < kB; ++y) wo(wave, y) = o[t][y] * alpha;
    __syncthreads();
    // Wave w finishes channel blocks w, w + 4, ...: lane (quad, col) holds
    // channels 16 y + 4 quad + [0, 4) of row 16 t + col.
    const int64_t row = row0 + rr;
    const int64_t i = row / G;
    const int64_t orow = (q0 + i) * a.heads_q + h * G + (row - i * G);
    for (int y = wave; y < kB; y += 4) {
      const f32x4 v = wo(0, y) + wo(1, y) + wo(2, y) + wo(3, y);
      if (active == 1) {
        if (row < rows) {
          const float inv = l > 0.0f || l != l ? vg / l : 0.0f;
          const f32x4 r = v * inv;
          const int64_t at = orow * D + 16 * y + 4 * quad;
          if (a.f32_out) {
            *reinterpret_cast<f32x4*>(reinterpret_cast<float*>(a.out) + at) = r;
          } else {
            typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
            *reinterpret_cast<bf16x4*>(reinterpret_cast<__bf16*>(a.out) + at) =
                bf16x4{(__bf16)r[0], (__bf16)r[1], (__bf16)r[2], (__bf16)r[3]};
          }
        }
      } else {
if (row < rows) bstore16_dev(rp, (uint32_t)(8 * kRows + (rr * D + 16 * y + 4 * quad) * 4), __builtin_bit_cast(u32x4, v));
      }
    }
    if (wave == 0 && quad == 0) {
      if (active == 1) {
        if (a.lse != nullptr && row < rows)
          a.lse[orow] = l == 0.0f ? -__builtin_inff() : (m + __builtin_log2f(l)) * kLn2;
      } else {
        __hip_atomic_store(part + rr, m, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __hip_atomic_store(part + kRows + rr, l, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
    }
  }
  if (active == 1) return;

  // Splits of one unit: the workgroup that arrives last joins them in split
  // order, so the result does not depend on which one that is.
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __builtin_amdgcn_s_waitcnt(0x3F70);  // vmcnt(0): this wave's partials are at device scope
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __syncthreads();
  __shared__ uint32_t arrived;
  if (threadIdx.x == 0)
    arrived = __hip_atomic_fetch_add(a.counters + unit, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __syncthreads();
  if (arrived != (uint32_t)(active - 1)) return;
  if (threadIdx.x == 0) __hip_atomic_store(a.counters + unit, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  const float* parts = a.part + unit * p.splits * (int64_t)p.part_floats;
  const Rsrc ra = make_rsrc(parts, (uint32_t)(active * p.part_floats * 4));
  float* jm = reinterpret_cast<float*>(lds);  // [active][kRows] m, then l
  float* jl = jm + kJoin;
  for (int n = threadIdx.x; n < active * kRows; n += 256) {
    const uint32_t at = (uint32_t)((n / kRows * p.part_floats + n % kRows) * 4);
    jm[n] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(ra, (int)at, 0, 16));
    jl[n] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(ra, (int)at, 4 * kRows, 16));
  }
  __syncthreads();
  const int live = rows - row0 < kRows ? (int)(rows - row0) : kRows;
  for (int n = threadIdx.x; n < live * (D / 4); n += 256) {
    const int rr = n / (D / 4), d = n % (D / 4) * 4;
    const int64_t row = row0 + rr;
    float m = kNoKey;
    for (int s = 0; s < active; ++s) m = __builtin_fmaxf(m, jm[s * kRows + rr]);
    float l = 0.0f;
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
    const uint32_t at = (uint32_t)(8 * kRows + (rr * D + d) * 4);
    for (int s = 0; s < active; s += 8) {
      f32x4 x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e)  // past the last split: zeros, unread
        x[e] = __builtin_bit_cast(f32x4, bload16_dev(ra, s + e < active ? at + (uint32_t)((s + e) * p.part_floats * 4) : kOutOfRange));
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (s + e >= active) break;
        const float w = __builtin_amdgcn_exp2f(jm[(s + e) * kRows + rr] - m);
        l += w * jl[(s + e) * kRows + rr];
        v += x[e] * w;
      }
    }
    const float inv = l > 0.0f || l != l ? vg / l : 0.0f;
    const f32x4 r = v * inv;
    const int64_t i = row / G;
    const int64_t orow = (q0 + i) * a.heads_q + h * G + (row - i * G);
    if (a.f32_out) {
      *reinterpret_cast<f32x4*>(reinterpret_cast<float*>(a.out) + orow * D + d) = r;
    } else {
      typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
      *reinterpret_cast<bf16x4*>(reinterpret_cast<__bf16*>(a.out) + orow * D + d) =
          bf16x4{(__bf16)r[0], (__bf16)r[1], (__bf16)r[2], (__bf16)r[3]};
    }
    if (d == 0 && a.lse != nullptr) a.lse[orow] = l == 0.0f ? -__builtin_inff() : (m + __builtin_log2f(l)) * kLn2;
  }
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
  p.row_tiles = rows <= 16 ? 1 : 2;
  const int64_t per = 16 * p.row_tiles;
  p.row_blocks = (rows + per - 1) / per;
  p.units = p.row_blocks * B * heads;
  // Keys that a unit reads at most, from a multiple of 32 on.
  int64_t span = max_len;
  if (window > 0 && window + max_q + 31 < span) span = window + max_q + 31;
  span = (span + 31) / 32 * 32;
  // About 1024 workgroups (4 per CU), at least 256 keys each.
  int64_t want = p.units > 0 ? (1024 + p.units - 1) / p.units : 1;
  int64_t most = (span + 255) / 256;
  if (most > 4096 / per) most = 4096 / per;  // what the join holds
  if (want > most) want = most;
  if (want < 1) want = 1;
  int64_t bound = p.units > 0 ? (1024 + p.units - 1) / p.units : 1;
  if (bound > (max_len + 255) / 256) bound = (max_len + 255) / 256;
  p.splits_bound = bound < 1 ? 1 : bound;
  p.chunk = ((span + want - 1) / want + 127) / 128 * 128;
  if (p.chunk < 128) p.chunk = 128;
  p.splits = span > 0 ? (span + p.chunk - 1) / p.chunk : 1;
  p.part_floats = (size_t)per * (dim + 2);
  return p;
}

hipError_t launch_kv_attention(const AttnArgs& a, const AttnPlan& p, hipStream_t s) {
  if (a.c.dim == 64) launch_d<64>(a, p, s);
  else if (a.c.dim == 128) launch_d<128>(a, p, s);
  else launch_d<256>(a, p, s);
  return hipGetLastError();
}

}  // namespace nvfp4
