// kv_attention_common.h -- what the two attention kernels over the paged NVFP4
// cache share: operands from a record, the query rows, the running softmax,
// and the join of a split key axis.
//
//   o_i = sum_j softmax_j(scale q_i . k_j) v_j over the keys a query sees.
//
// Both products run on the f16 matrix core, keys in pairs of 16-token groups:
//   S^T = K Q^T  (rows: 16 tokens, columns: query rows)
//   O^T = V^T P  (rows: 16 channels, columns: query rows, 32 tokens deep)
// A code times its E4M3 scale has at most 6 significant bits and lies in
// [2^-10, 2688], exact in f16. A bf16 query row is scaled by a power of two
// to at most 1 before it becomes f16: exact but for elements 2^-14 below the
// row's largest, which are off by 2^-25 of it. Probabilities are rounded to
// f16 for the second product: half a step 2^-11, or under 2^-21 of the row's
// largest 2^-32 of that (kUp below); that is 1/8 of a bf16 output's own
// rounding, and f32 outputs take them in two parts, 2^-22. Their sum is kept
// in fp32. S^T leaves a lane with the tokens of one query row that the second
// product wants from that lane, because the record's V codes are stored in the
// same token order, so the probabilities never leave their registers, and the
// row statistics are one number a lane.
#pragma once
#include <type_traits>

#include "attention.h"
#include "kv_layout.h"

namespace nvfp4 {
namespace {

typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));

// The maximum of no key, in units of log2; and of raw scores, below all of
// them (D <= 256 products of at most 2 and 2688: under 2^21).
constexpr float kNoKey = -3.0e38f;
constexpr float kNoScore = -0x1p24f;
// Probabilities are computed 2^kUp times as large as they are and may pass the
// subtracted maximum by 2^kLazy: f16 holds up to 2^16, and has 11 bits down
// to 2^-14. With 10 and 5.9 (maxima renewed more often) the matrix-bound
// calls took 1 to 4% longer, with 13 and 2.9 3 to 8%; with 0 and 8 as long,
// but one key of value 0 that stood 16 above 4096 others (natural logarithm)
// left their sum 9% off.
constexpr float kUp = 7.0f, kLazy = 8.0f;
constexpr float kLog2e = 1.44269504088896341f;
constexpr float kLn2 = 0.693147180559945309f;

#if defined(__HIP_DEVICE_COMPILE__)

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

// f(0), .., f(N - 1) with the number as a constant.
template <int N, int I = 0, class F>
__device__ __forceinline__ void static_for(F&& f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    static_for<N, I + 1>(f);
  }
}

// ---- operands from a record ----------------------------------------------

// A lane's share of a record's K: the codes and scales of its token.
template <int D>
struct KFrag {
  uint32_t c[D / 32], s;
};
// Of V: the codes of its channel in all blocks or, PARTS = 2, in one half of
// them, and the scales of one of these blocks, lane % (D / 16 / PARTS), of its
// quad (the other blocks' are with the quad's other lanes).
template <int D, int PARTS = 1>
struct VFrag {
  uint32_t c[D / 32 / PARTS], s;
};

// A record as a buffer: a lane's offset into it is a constant of the kernel, and
// addresses cost no vector instructions.
template <int N>
__device__ __forceinline__ void load_words(uint32_t (&w)[N], Rsrc rec, uint32_t at) {
  if constexpr (N == 1) {
    w[0] = __builtin_amdgcn_raw_buffer_load_b32(rec, (int)at, 0, 0);
  } else if constexpr (N == 2) {
    const u32x2 t = __builtin_amdgcn_raw_buffer_load_b64(rec, (int)at, 0, 0);
    w[0] = t[0]; w[1] = t[1];
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const u32x4 t = bload16(rec, at + 4 * i);
      w[i] = t[0]; w[i + 1] = t[1]; w[i + 2] = t[2]; w[i + 3] = t[3];
    }
  }
}

template <int D>
__device__ __forceinline__ void load_k(KFrag<D>& f, Rsrc rec, unsigned lane) {
  load_words(f.c, rec, lane * KvRec<D>::kLane);
  const int s = KvRec<D>::kKs + lane * (D / 64);
  if constexpr (D == 64) f.s = __builtin_amdgcn_raw_buffer_load_b8(rec, s, 0, 0);
  else if constexpr (D == 128) f.s = __builtin_amdgcn_raw_buffer_load_b16(rec, s, 0, 0);
  else f.s = __builtin_amdgcn_raw_buffer_load_b32(rec, s, 0, 0);
}
template <int D, int PARTS>
__device__ __forceinline__ void load_v(VFrag<D, PARTS>& f, Rsrc rec, unsigned lane, unsigned part) {
  constexpr int kN = D / 16 / PARTS;
  load_words(f.c, rec, KvRec<D>::kV + lane * KvRec<D>::kLane + part * (2 * kN));
  f.s = __builtin_amdgcn_raw_buffer_load_b32(rec, KvRec<D>::kVs + (lane >> 4) * (D / 4) + (part * kN + (lane & (kN - 1))) * 4, 0, 0);
}

// Lane N's value in each row of 16 lanes.
template <int N>
__device__ __forceinline__ uint32_t row_bcast(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x150 + N, 0xF, 0xF, true);
}

// V^T of channel block Y (of f's) as an operand: 4 tokens of each of two
// records.
template <int Y, int D, int PARTS>
__device__ __forceinline__ f16x8 v_operand(const VFrag<D, PARTS> (&f)[2], const f16x4 (&vs)[2]) {
  f16x8 r;
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const uint32_t w = f[x].c[Y >> 1];
    const u32x2 s = __builtin_bit_cast(u32x2, vs[x]);
    const f16x2 lo = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 2 * (Y & 1)) * __builtin_bit_cast(f16x2, row_bcast<Y>(s[0]));
    const f16x2 hi = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 2 * (Y & 1) + 1) * __builtin_bit_cast(f16x2, row_bcast<Y>(s[1]));
    r[4 * x] = lo[0]; r[4 * x + 1] = lo[1]; r[4 * x + 2] = hi[0]; r[4 * x + 3] = hi[1];
  }
  return r;
}

// The records of head h in the pages of a block table row, one after the
// other: where record (page slot ps, group `in`) is. 64 page numbers, of the
// slots from tab0 on, are in the lanes of `tab`; slots past the table's last
// stand for that one. A page number outside the cache (as may stand past a
// sequence's length) makes `ok` false and the address that of page 0.
template <int D>
struct Walk {
  const int32_t* table;
  const uint8_t* base;
  uint64_t page_bytes;
  unsigned pages;
  int groups, last, ps, in, tab0, tab;
  __device__ __forceinline__ void load_tab(int lane) {
    const int at = tab0 + lane;
    if (last >= 0) tab = table[at < last ? at : last];
  }
  // The table from group g on.
  __device__ __forceinline__ Walk(const AttnArgs& a, unsigned b, int h, int g, int lane) {
    groups = a.c.page_size / 16;
    table = a.table + (int64_t)b * a.table_stride;
    base = a.c.cache + (uint64_t)h * groups * KvRec<D>::kBytes;
    page_bytes = (uint64_t)a.c.heads * groups * KvRec<D>::kBytes;
    pages = (unsigned)a.c.pages;
    last = (int)a.table_width - 1;
    ps = tab0 = g / groups;
    tab = -1;
    load_tab(lane);
  }
  // Records from group g on.
  __device__ __forceinline__ void start(int g) {
    ps = g / groups;
    in = g - ps * groups;
    asm volatile("" : "+v"(tab));  // waits here, not at each use for all loads in flight
  }
  __device__ __forceinline__ Rsrc record(bool& ok, int lane) {
    if (ps - tab0 >= 64) {
      tab0 = ps;
      load_tab(lane);
      asm volatile("" : "+v"(tab));
    }
    const unsigned page = (unsigned)__builtin_amdgcn_readlane(tab, ps - tab0);
    ok = page < pages;
    return make_rsrc(base + (ok ? page : 0u) * page_bytes + (unsigned)in * KvRec<D>::kBytes, KvRec<D>::kBytes);
  }
  __device__ __forceinline__ void step(int by) {
    in += by;
    while (in >= groups) { in -= groups; ++ps; }
  }
};

// Keeps the bytes of the quad's tokens first .. first + 3 that lie in [lo, hi).
__device__ __forceinline__ uint32_t byte_mask(int first, int lo, int hi) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (first + i >= lo && first + i < hi) m |= 255u << (8 * i);
  return m;
}

// ---- a workgroup's query rows ----------------------------------------------

// Sequence b: its first query, its queries, the rows (query x head of one kv
// head's group) computed, its keys. Positions and rows fit 31 bits (max_len
// and the number of workgroups are bounded so).
struct Seq {
  int64_t q0, nq;
  int rows, len;
};
__device__ __forceinline__ Seq seq_of(const AttnArgs& a, unsigned b, int G) {
  Seq s;
  if (a.q_offsets != nullptr) {
    s.q0 = a.q_offsets[b];
    s.nq = a.q_offsets[b + 1] - s.q0;
    if (s.q0 < 0 || s.q0 > a.T) s.nq = 0;
    else if (s.nq > a.T - s.q0) s.nq = a.T - s.q0;
  } else {
    s.nq = a.max_q;
    s.q0 = (int64_t)b * s.nq;
  }
  s.rows = s.nq < 0 ? 0 : (int)((s.nq < a.max_q ? s.nq : a.max_q) * G);
  int len = a.seq_lens[b];
  len = len < 0 ? 0 : len;
  if (len > a.max_len) len = (int)a.max_len;
  const int64_t room = a.table_width * a.c.page_size;
  s.len = len > room ? (int)room : len;
  return s;
}
// Query i stands at position len - nq + i and sees [lo, hi).
__device__ __forceinline__ int sees_hi(const Seq& s, int i) {
  const int64_t e = (int64_t)s.len - s.nq + i + 1;
  return (int)(e < 0 ? 0 : e);
}
__device__ __forceinline__ int sees_lo(int hi, int64_t window) {
  return window > 0 && hi > window ? (int)(hi - window) : 0;
}

// The keys [lo, hi) that any of a workgroup's rows sees (rows row0 on, row0
// one of them), walked over from `start` on in `splits` stretches.
struct Stretch {
  int lo, hi, start, splits;
};
__device__ __forceinline__ Stretch active_splits(const AttnArgs& a, const AttnPlan& p, const Seq& seq, int row0, int rows, int G) {
  const int last = seq.rows - 1 < row0 + rows - 1 ? seq.rows - 1 : row0 + rows - 1;
  Stretch s;
  s.hi = sees_hi(seq, last / G);
  s.lo = sees_lo(sees_hi(seq, row0 / G), a.window);
  s.start = s.lo & ~31;
  s.splits = s.hi > s.lo ? (s.hi - s.start + p.chunk - 1) / p.chunk : 1;
  return s;
}

// RT tiles of 16 rows: lane (quad, col) holds row col of a tile, of its output
// channels 16 y + 4 quad + [0, 4). A raw score s has the probability
// exp2(s f + a), 2^kUp times as large as it is under the subtracted maximum,
// which is kUp - a in units of log2. l: their sum so far, over this lane's
// tokens; t: the raw score above which the maximum is renewed, kNoScore before
// the first key. a is zero until then, so that a hidden score of -inf gives the
// probability 0 whatever the query holds.
template <int D, int RT>
struct Rows {
  f32x4 o[RT][D / 16];
  f16x8 q[RT][D / 32];
  float a[RT], l[RT], f[RT], t[RT];
  int lo[RT], n[RT];  // keys seen: lo .. lo + n - 1
};

template <int D, int RT>
__device__ __forceinline__ void load_rows(Rows<D, RT>& r, const AttnArgs& a, const Seq& seq, int row0, int h, int G,
                                          int quad, int col) {
  constexpr int kW = D / 32;
  const float unit = a.scale * *a.k_g * kLog2e;
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    const int row = row0 + 16 * t + col;
    const bool live = row < seq.rows;
    const int i = live ? (int)((unsigned)row / (unsigned)G) : 0;
    const int head = h * G + row - i * G, hi = live ? sees_hi(seq, i) : 0;
    r.lo[t] = sees_lo(hi, a.window);
    r.n[t] = hi - r.lo[t];
    r.t[t] = kNoScore;
    r.a[t] = r.l[t] = 0.0f;
    uint32_t w[kW * 4];
    uint32_t top = 0;
    if (live) {
      const uint16_t* q = a.q + (seq.q0 + i) * a.q_stride + (int64_t)head * D + quad * (D / 4);
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
    const float f = __uint_as_float((uint32_t)(127 + e) << 23) * unit;
    // Not zero, so that a hidden score of -inf gives the probability 0: this
    // small, all scores of a zero scale still give 1.
    r.f[t] = f == 0.0f ? 0x1p-126f : __builtin_fabsf(f);
    if (f < 0.0f) down = -down;
#pragma unroll
    for (int s = 0; s < kW; ++s) {
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        r.q[t][s][2 * x] = (_Float16)(__uint_as_float(w[4 * s + x] << 16) * down);
        r.q[t][s][2 * x + 1] = (_Float16)(__uint_as_float(w[4 * s + x] & 0xFFFF0000u) * down);
      }
      asm volatile("" : "+v"(r.q[t][s]));  // converted here, not at its first use: registers
    }
  }
#pragma unroll
  for (int t = 0; t < RT; ++t)
#pragma unroll
    for (int y = 0; y < D / 16; ++y) r.o[t][y] = f32x4{0.f, 0.f, 0.f, 0.f};
}

// Hidden scores of the pair of groups at `base` become -inf. ok: the groups'
// pages exist.
template <int D, int RT>
__device__ __forceinline__ void hide_scores(const Rows<D, RT>& r, f32x4 (&sc)[RT][2], int base, int quad, const bool (&ok)[2]) {
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    const int at = base + 4 * quad - r.lo[t];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int n = ok[x] ? r.n[t] : 0;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        sc[t][x][e] = (unsigned)(at + 16 * x + e) < (unsigned)n ? sc[t][x][e] : -__builtin_inff();
    }
  }
}

template <int RT>
__device__ __forceinline__ void lane_maximum(const f32x4 (&sc)[RT][2], float (&mx)[RT]) {
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    mx[t] = sc[t][0][0];
#pragma unroll
    for (int e = 1; e < 8; ++e) mx[t] = __builtin_fmaxf(mx[t], sc[t][e >> 2][e & 3]);
  }
}

// mx: the maximum of a pair's scores in this lane. The subtracted maximum
// follows the true one only when a score passes it by more than 2^kLazy in
// probability: f16 holds probabilities up to that as exactly as up to 1, and
// most steps then need neither the exchange between lanes nor the rescaling.
template <int D, int RT>
__device__ __forceinline__ void renew_maximum(Rows<D, RT>& r, const float (&mx)[RT]) {
  bool passed = false;
#pragma unroll
  for (int t = 0; t < RT; ++t) passed |= mx[t] > r.t[t];
  if (__any(passed)) {
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      const float mr = max_xor32(max_xor16(mx[t]));
      const float a = mr > r.t[t] ? __builtin_fmaf(-mr, r.f[t], kUp) : r.a[t];
      const float alpha = r.t[t] == kNoScore ? 0.0f : __builtin_amdgcn_exp2f(a - r.a[t]);
      r.t[t] = mr > r.t[t] ? mr + kLazy / r.f[t] : r.t[t];
      r.a[t] = a;
      r.l[t] *= alpha;
#pragma unroll
      for (int y = 0; y < D / 16; ++y) r.o[t][y] *= alpha;
    }
  }
}

// A probability as P f16 operands: of 11 bits, or of 22 in two parts for f32
// outputs. The second part costs half as many matrix instructions again and 3
// vector instructions a probability: 64 sequences of up to 8192 keys 68 / 75
// us, 4 of 131072 118 / 120, chunks of up to 2047 tokens 451 / 584.
template <int P, int RT>
__device__ __forceinline__ void put_probability(f16x8 (&pf)[P][RT], int t, int i, float p) {
  pf[0][t][i] = (_Float16)p;
  if constexpr (P == 2) pf[1][t][i] = (_Float16)(p - (float)pf[0][t][i]);
}

// Probabilities of a pair's scores, as operands.
template <int D, int RT, int P>
__device__ __forceinline__ void probabilities(Rows<D, RT>& r, const f32x4 (&sc)[RT][2], f16x8 (&pf)[P][RT]) {
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    float e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[t][i >> 2][i & 3], r.f[t], r.a[t]));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      r.l[t] += e[i];
      put_probability(pf, t, i, e[i]);
    }
  }
}

// After the last key: sums over all tokens.
template <int D, int RT>
__device__ __forceinline__ void finish_rows(Rows<D, RT>& r) {
#pragma unroll
  for (int t = 0; t < RT; ++t) r.l[t] = sum_xor32(sum_xor16(r.l[t]));
}
// The subtracted maximum of tile t's rows, in units of log2.
template <int D, int RT>
__device__ __forceinline__ float row_maximum(const Rows<D, RT>& r, int t) {
  return r.t[t] == kNoScore ? kNoKey : kUp - r.a[t];
}

// ---- results ----------------------------------------------------------------

__device__ __forceinline__ float inverse_sum(float l, float vg) { return l > 0.0f || l != l ? vg / l : 0.0f; }
// l is 2^kUp as large: taken off before the logarithm, whose bits are then those
// of the sum.
__device__ __forceinline__ float lse_of(float m, float l) {
  return l == 0.0f ? -__builtin_inff() : (m + __builtin_log2f(l * __builtin_exp2f(-kUp))) * kLn2;
}
__device__ __forceinline__ void store4(const AttnArgs& a, int64_t at, const f32x4& r) {
  if (a.f32_out) {
    *reinterpret_cast<f32x4*>(reinterpret_cast<float*>(a.out) + at) = r;
  } else {
    typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
    *reinterpret_cast<bf16x4*>(reinterpret_cast<__bf16*>(a.out) + at) =
        bf16x4{(__bf16)r[0], (__bf16)r[1], (__bf16)r[2], (__bf16)r[3]};
  }
}
// Row `row` of sequence seq and kv head h in out and lse.
__device__ __forceinline__ int64_t out_row(const AttnArgs& a, const Seq& seq, int row, int h, int G) {
  const int i = (int)((unsigned)row / (unsigned)G);
  return (seq.q0 + i) * a.heads_q + h * G + (row - i * G);
}

#endif  // __HIP_DEVICE_COMPILE__
}  // namespace
}  // namespace nvfp4
