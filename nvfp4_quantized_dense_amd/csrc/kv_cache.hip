// kv_cache.hip -- keys and values into the paged NVFP4 cache as they are
// written, turned by their positions where the caller wants that, and back to
// dense rows; and which pages and slots a step's tokens take.
#include <type_traits>

#include "attention.h"
#include "kv_layout.h"

namespace nvfp4 {
namespace {

// n / d for n < 2^31 by a product: m = ceil(2^(31 + l) / d), 2^l >= d.
struct Div {
  uint32_t m, d;
  int shift;  // 31 + l
};
Div div_by(uint32_t d) {
  int l = 0;
  while ((1u << l) < d) ++l;
  return {(uint32_t)(((uint64_t(1) << (31 + l)) + d - 1) / d), d, 31 + l};
}

// Where a slot is: record group `first` of the page (counted over all pages)
// + `group`, token t of it; not ok: nowhere, and the place of slot 0.
struct Slot {
  uint32_t first, group;
  int t;
  bool ok;
};
__device__ __forceinline__ Slot slot_at(int64_t slot, int64_t pages, const Div& groups) {
  Slot r;
  r.ok = slot >= 0 && slot < pages * groups.d * 16;
  const uint32_t n = r.ok ? (uint32_t)(slot >> 4) : 0u;  // the cache has fewer than 2^31 groups
  r.t = r.ok ? (int)slot & 15 : 0;
  r.group = n - (uint32_t)(((uint64_t)n * groups.m) >> groups.shift) * groups.d;
  r.first = n - r.group;
  return r;
}
// Its record of head h.
template <int D>
__device__ __forceinline__ int64_t record_at(const Slot& s, int heads, int h, const Div& groups) {
  return ((int64_t)s.first * heads + ((uint32_t)h * groups.d + s.group)) * KvRec<D>::kBytes;
}

template <bool F32>
__device__ __forceinline__ void load8_at(const void* base, int64_t elem, float (&v)[8]) {
  if constexpr (F32) {
    const f32x4* p = reinterpret_cast<const f32x4*>(reinterpret_cast<const float*>(base) + elem);
    const f32x4 a = p[0], b = p[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) { v[i] = a[i]; v[4 + i] = b[i]; }
  } else {
    const u32x4 a = *reinterpret_cast<const u32x4*>(reinterpret_cast<const uint16_t*>(base) + elem);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(a[i] << 16);
      v[2 * i + 1] = __uint_as_float(a[i] & 0xFFFF0000u);
    }
  }
}

// Rows on their way out are stored past the caches (nontemporal): 65536 tokens
// of 8 heads of 128 took 57 us so, 103 us with plain stores.
template <bool F32>
__device__ __forceinline__ void store8_at(void* base, int64_t elem, const float (&v)[8]) {
  if constexpr (F32) {
    f32x4* p = reinterpret_cast<f32x4*>(reinterpret_cast<float*>(base) + elem);
    __builtin_nontemporal_store(f32x4{v[0], v[1], v[2], v[3]}, p);
    __builtin_nontemporal_store(f32x4{v[4], v[5], v[6], v[7]}, p + 1);
  } else {
    bf16x8 b;
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = (__bf16)v[i];
    __builtin_nontemporal_store(__builtin_bit_cast(u32x4, b), reinterpret_cast<u32x4*>(reinterpret_cast<__bf16*>(base) + elem));
  }
}

// The same to the caches: rows that the next kernel reads.
template <bool F32>
__device__ __forceinline__ void put8_at(void* base, int64_t elem, const float (&v)[8]) {
  if constexpr (F32) {
    f32x4* p = reinterpret_cast<f32x4*>(reinterpret_cast<float*>(base) + elem);
    p[0] = f32x4{v[0], v[1], v[2], v[3]};
    p[1] = f32x4{v[4], v[5], v[6], v[7]};
  } else {
    bf16x8 b;
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = (__bf16)v[i];
    *reinterpret_cast<bf16x8*>(reinterpret_cast<__bf16*>(base) + elem) = b;
  }
}

// The value of lane ^ 1 and lane ^ 2, ^ 16 and ^ 32, without a trip to LDS. A
// swap of v with itself gives v and the partner's v in some order.
__device__ __forceinline__ uint32_t xor1(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, true);
}
__device__ __forceinline__ uint32_t xor2(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, true);
}
__device__ __forceinline__ uint32_t xor16(uint32_t v) {
  const auto p = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  return p[0] ^ p[1] ^ v;
}
__device__ __forceinline__ uint32_t xor32(uint32_t v) {
  const auto p = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return p[0] ^ p[1] ^ v;
}

// NVFP4 of 8 channels (the neighbouring lane holds the block's other 8), by
// k_quantize's rule.
__device__ __forceinline__ uint32_t quant8(const float (&v)[8], float g_inv, uint32_t& scale) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  m = max(m, xor1(m));
  const BlockScale bs = block_scale(__uint_as_float(m), g_inv);
  scale = bs.byte;
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = v[i] * bs.r;
  return e2m1_pack8(y);
}

// A wave takes four list entries, a row of 16 lanes each, and 16 units of the
// entry's heads x D / 8. Of K a unit is 8 channels. Of V it is channels
// 4 c4 + [0, 4) of blocks 2 m and 2 m + 1: what the record stores of them for
// a quad of tokens is then a dword per channel.
template <int D>
struct Unit {
  int h, j, m, c4;
  bool ok;
};
template <int D>
__device__ __forceinline__ Unit<D> unit_at(unsigned u, int heads) {
  Unit<D> r;
  r.h = (int)(u / (D / 8));
  r.j = (int)(u % (D / 8));
  r.m = r.j >> 2;
  r.c4 = r.j & 3;
  r.ok = r.h < heads;
  return r;
}
// Where unit u's V dwords of a quad begin, and its scale bytes.
template <int D>
__device__ __forceinline__ int v_at(const Unit<D>& u, int q) {
  return KvRec<D>::kV + (q * 16 + 4 * u.c4) * KvRec<D>::kLane + 4 * u.m;
}
template <int D>
__device__ __forceinline__ int vs_at(const Unit<D>& u, int q) {
  return KvRec<D>::kVs + (q * (D / 16) + 2 * u.m) * 4;
}

template <bool F32>
__device__ __forceinline__ void load4_at(const void* base, int64_t elem, float* v) {
  if constexpr (F32) {
    const f32x4 a = *reinterpret_cast<const f32x4*>(reinterpret_cast<const float*>(base) + elem);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = a[i];
  } else {
    const u32x2 a = *reinterpret_cast<const u32x2*>(reinterpret_cast<const uint16_t*>(base) + elem);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      v[2 * i] = __uint_as_float(a[i] << 16);
      v[2 * i + 1] = __uint_as_float(a[i] & 0xFFFF0000u);
    }
  }
}

// Two of V's blocks, 4 channels of each in this lane and the others in the
// neighbours': 8 codes (block 2 m in the low half). Even lanes compute the
// first block's scale, odd ones the second's: `scale` is that one's byte.
__device__ __forceinline__ uint32_t quant44(const float (&v)[8], float g_inv, bool odd, uint32_t& scale) {
  uint32_t m[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i) m[i >> 2] = max(m[i >> 2], __float_as_uint(v[i]) & 0x7FFFFFFFu);
  // Lane pairs hand each other the half that the other one needs.
  const uint32_t give = odd ? m[0] : m[1];
  uint32_t top = max(odd ? m[1] : m[0], xor1(give));
  top = max(top, xor2(top));
  const BlockScale bs = block_scale(__uint_as_float(top), g_inv);
  scale = bs.byte;
  const float other = __uint_as_float(xor1(__float_as_uint(bs.r)));
  const float r0 = odd ? other : bs.r, r1 = odd ? bs.r : other;
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = v[i] * (i < 4 ? r0 : r1);
  return e2m1_pack8(y);
}

// Row k of four holds the codes of token k of a quad, a nibble a channel;
// becomes the codes of channel k, a nibble a token (both halves alike).
__device__ __forceinline__ uint32_t quad_transpose(uint32_t w, int k) {
  const uint32_t p = xor16(w);
  w = k & 1 ? ((p >> 4) & 0x0F0F0F0Fu) | (w & 0xF0F0F0F0u) : (w & 0x0F0F0F0Fu) | ((p & 0x0F0F0F0Fu) << 4);
  const uint32_t r = xor32(w);
  return k & 2 ? ((r >> 8) & 0x00FF00FFu) | (w & 0xFF00FF00u) : (w & 0x00FF00FFu) | ((r & 0x00FF00FFu) << 8);
}

// ---- rotary positions ------------------------------------------------------

// Cosine and sine of an angle in 64 bits: reduced by multiples of pi/2 in two
// parts (the first difference is exact up to 2^31 quarter turns), then the
// series of both to the terms of 16th and 17th order: the first ones left out
// are below 2^-58 and 2^-63 at pi/4. So far positions keep their angle, and the
// 32-bit numbers are the nearest ones but for one case in 2^27.
__device__ __forceinline__ void cos_sin(double angle, double& c, double& s) {
  const double n = __builtin_rint(angle * 0.63661977236758134308);
  const double r = __builtin_fma(-n, 6.123233995736765886e-17, __builtin_fma(-n, 1.57079632679489661923, angle));
  const double x = r * r;
  double p = 1.0 / 355687428096000.0;  // 1 / 17!
  p = __builtin_fma(p, x, -1.0 / 1307674368000.0);
  p = __builtin_fma(p, x, 1.0 / 6227020800.0);
  p = __builtin_fma(p, x, -1.0 / 39916800.0);
  p = __builtin_fma(p, x, 1.0 / 362880.0);
  p = __builtin_fma(p, x, -1.0 / 5040.0);
  p = __builtin_fma(p, x, 1.0 / 120.0);
  p = __builtin_fma(p, x, -1.0 / 6.0);
  const double si = __builtin_fma(p * x, r, r);
  double q = 1.0 / 20922789888000.0;  // 1 / 16!
  q = __builtin_fma(q, x, -1.0 / 87178291200.0);
  q = __builtin_fma(q, x, 1.0 / 479001600.0);
  q = __builtin_fma(q, x, -1.0 / 3628800.0);
  q = __builtin_fma(q, x, 1.0 / 40320.0);
  q = __builtin_fma(q, x, -1.0 / 720.0);
  q = __builtin_fma(q, x, 1.0 / 24.0);
  q = __builtin_fma(q, x, -0.5);
  const double co = __builtin_fma(q, x, 1.0);
  const int quarter = (int)(n - 4.0 * __builtin_floor(n * 0.25));
  const double a = quarter & 1 ? si : co, b = quarter & 1 ? co : si;
  c = quarter == 1 || quarter == 2 ? -a : a;
  s = quarter >= 2 ? -b : b;
}

constexpr int kRopeTokens = 16;  // of a workgroup
// Workgroups aimed at: 8192 tokens of 40 heads of 128 in halves / half of the
// channels / neighbouring pairs 49 / 50 / 51 us, 49 / 53 / 55 with 1024 (each
// makes its tokens' table for itself).
constexpr int64_t kRopeGroups = 512;

// Cosine and sine of the workgroup's tokens, [kRopeTokens][rotary / 2] of LDS:
// once for all heads.
__device__ __forceinline__ void rope_table(const RopeArgs& r, int64_t first, int tokens, const Div& half, f32x2* table) {
  for (int n = threadIdx.x; n < tokens * (int)half.d; n += 256) {
    const int t = (int)(((uint64_t)(uint32_t)n * half.m) >> half.shift), i = n - t * (int)half.d;
    const int axis = r.axis != nullptr ? r.axis[i] : 0;
    const bool turns = (unsigned)axis < (unsigned)r.axes;
    const double angle = turns ? (double)r.positions[axis * r.axis_stride + first + t] * (double)r.inv_freq[i] : 0.0;
    double c, s;
    cos_sin(angle, c, s);
    const double factor = turns ? r.factor : 1.0;  // what is not turned stays as it is
    table[n] = f32x2{(float)(factor * c), (float)(factor * s)};
  }
}

// fl(fl(x c) - fl(y s)) and fl(fl(y c) + fl(x s)): no fused product, so that a
// key has the same bits whether it is turned here or with single operations.
__device__ __forceinline__ float turn_first(float x, float y, f32x2 cs) {
#pragma clang fp contract(off)
  return x * cs[0] - y * cs[1];
}
__device__ __forceinline__ float turn_second(float x, float y, f32x2 cs) {
#pragma clang fp contract(off)
  return y * cs[0] + x * cs[1];
}

// Units of a row: 8 channels and their partners half a rotation on, 8 channels
// of 4 neighbouring pairs, or 8 channels that only move. Each kind has a loop
// of its own, as a branch within a wave waits for both sides' loads: with half
// of the channels turned, 8192 tokens of 40 heads of 128 took 66 us in one.
struct RopeUnits {
  Div turned, rest, heads, half;  // units of a head
  bool copies;
};
RopeUnits rope_units(const RopeArgs& r) {
  const int rest = (r.dim - r.rotary) / 8;
  return {div_by((uint32_t)(r.neighbours ? r.rotary / 8 : r.rotary / 16)), div_by((uint32_t)(rest > 0 ? rest : 1)),
          div_by((uint32_t)(r.heads > 0 ? r.heads : 1)), div_by((uint32_t)r.rotary / 2), rest > 0 && r.x != r.out};
}
__device__ __forceinline__ uint32_t div_n(uint32_t n, const Div& d) { return (uint32_t)(((uint64_t)n * d.m) >> d.shift); }

// Part `part` of `parts` of the tokens' units.
template <bool IN32, bool OUT32>
__device__ __forceinline__ void rope_rows(const RopeArgs& r, const RopeUnits& units, int64_t first, int tokens, unsigned part,
                                          unsigned parts, const f32x2* table) {
  const uint32_t rows = (uint32_t)tokens * units.heads.d;
  const int half = r.rotary / 2;
  struct Place {
    int64_t from, to;
    int t, j;
  };
  auto place = [&](uint32_t n, const Div& per_head) {
    const uint32_t m = div_n(n, per_head), t = div_n(m, units.heads);
    const int h = (int)(m - t * units.heads.d);
    return Place{(first + t) * r.x_stride + (int64_t)h * r.dim, (first + t) * r.out_stride + (int64_t)h * r.dim, (int)t,
                 (int)(n - m * per_head.d)};
  };
  const uint32_t begin = part * 256 + threadIdx.x, step = parts * 256;
  if (!r.neighbours) {
    for (uint32_t n = begin; n < rows * units.turned.d; n += step) {
      const Place p = place(n, units.turned);
      float x[8], y[8], a[8], b[8];
      load8_at<IN32>(r.x, p.from + 8 * p.j, x);
      load8_at<IN32>(r.x, p.from + half + 8 * p.j, y);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const f32x2 cs = table[p.t * half + 8 * p.j + i];
        a[i] = turn_first(x[i], y[i], cs);
        b[i] = turn_second(x[i], y[i], cs);
      }
      put8_at<OUT32>(r.out, p.to + 8 * p.j, a);
      put8_at<OUT32>(r.out, p.to + half + 8 * p.j, b);
    }
  } else {
    for (uint32_t n = begin; n < rows * units.turned.d; n += 2 * step) {  // two units at a time, for as many loads in flight
      const uint32_t n2 = n + step;
      const bool two = n2 < rows * units.turned.d;
      const Place p[2] = {place(n, units.turned), place(two ? n2 : n, units.turned)};
      float x[2][8], a[8];
#pragma unroll
      for (int u = 0; u < 2; ++u) load8_at<IN32>(r.x, p[u].from + 8 * p[u].j, x[u]);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f32x2 cs = table[p[u].t * half + 4 * p[u].j + i];
          a[2 * i] = turn_first(x[u][2 * i], x[u][2 * i + 1], cs);
          a[2 * i + 1] = turn_second(x[u][2 * i], x[u][2 * i + 1], cs);
        }
        if (u == 0 || two) put8_at<OUT32>(r.out, p[u].to + 8 * p[u].j, a);
      }
    }
  }
  if (!units.copies) return;
  for (uint32_t n = begin; n < rows * units.rest.d; n += 2 * step) {
    const uint32_t n2 = n + step;
    const bool two = n2 < rows * units.rest.d;
    const Place p[2] = {place(n, units.rest), place(two ? n2 : n, units.rest)};
    float x[2][8];
#pragma unroll
    for (int u = 0; u < 2; ++u) load8_at<IN32>(r.x, p[u].from + r.rotary + 8 * p[u].j, x[u]);
#pragma unroll
    for (int u = 0; u < 2; ++u)
      if (u == 0 || two) put8_at<OUT32>(r.out, p[u].to + r.rotary + 8 * p[u].j, x[u]);
  }
}

// Rows alone. Bound by memory: 8192 tokens of 40 heads of 128, bf16 (168 MB) 38
// us, f32 (336 MB) 72, 4.4 and 4.6 TB/s; one token 2.4 us.
template <bool IN32, bool OUT32>
__global__ __launch_bounds__(256) void k_rope(RopeArgs r, RopeUnits units) {
  __shared__ f32x2 table[kRopeTokens * 256];
  const int64_t first = ((int64_t)blockIdx.z * gridDim.y + blockIdx.y) * kRopeTokens;
  if (first >= r.T) return;
  const int tokens = r.T - first < kRopeTokens ? (int)(r.T - first) : kRopeTokens;
  rope_table(r, first, tokens, units.half, table);
  __syncthreads();
  rope_rows<IN32, OUT32>(r, units, first, tokens, blockIdx.x, gridDim.x, table);
}

// Channels 8 j + [0, 8) of a key head at `from`, turned; `table`: its token's.
template <bool F32>
__device__ __forceinline__ void turn_key(const RopeArgs& r, const void* k, int64_t from, int j, const f32x2* table, float (&x)[8]) {
  const int half = r.rotary / 2, at = 8 * j;
  if (at >= r.rotary) return;
  float y[8];
  if (r.neighbours) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f32x2 cs = table[4 * j + i];
      y[2 * i] = turn_first(x[2 * i], x[2 * i + 1], cs);
      y[2 * i + 1] = turn_second(x[2 * i], x[2 * i + 1], cs);
    }
  } else {
    const bool second = at >= half;
    load8_at<F32>(k, second ? from - half : from + half, y);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const f32x2 cs = table[second ? at - half + i : at + i];
      y[i] = second ? turn_second(y[i], x[i], cs) : turn_first(x[i], y[i], cs);
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = y[i];
}

// 8192 tokens of 8 heads of 128 (43 MB) take 10 to 12 us, bound by instruction
// issue (two block scales with their exact divisions a lane) as much as by
// memory; 64 tokens 3.8 us, the dependent trips: slots, rows, stores. Entries
// of the list that fill an aligned quad of slots are written whole by the wave
// that holds the first of them; any other entry's V shares its dwords with
// tokens that another wave, or an earlier call, owns.
// ROPE: `table` holds the cosines and sines of the workgroup's tokens.
template <int D, bool F32, bool ROPE>
__device__ __forceinline__ void write_units(const CacheArgs& c, const void* k, const void* v, int64_t T, int64_t ks, int64_t vs,
                                            const int64_t* slots, const float* kg, const float* vg, const Div& groups,
                                            unsigned chunk, const RopeArgs& r, const f32x2* table) {
  using R = KvRec<D>;
  const int lane = threadIdx.x & 63, row = lane >> 4;
  const int64_t first = (((int64_t)blockIdx.z * gridDim.y + blockIdx.y) * 4 + (threadIdx.x >> 6)) * 4;
  if (first >= T) return;
  const Unit<D> u = unit_at<D>(chunk * 16 + (lane & 15), c.heads);
  const int64_t t = first + row;
  // K's row is asked for together with the slots.
  float x[8];
  if (t < T && u.ok) load8_at<F32>(k, t * ks + (int64_t)u.h * D + 8 * u.j, x);
  // Slots of the entries first - 3 on, one a lane.
  const int64_t near = first - 3 + (lane & 15);
  const int64_t s = near >= 0 && near < T && (lane & 15) < 10 ? slots[near] : -2;
  const int64_t after = __shfl_down(s, 1);
  const uint32_t runs = (uint32_t)__ballot(after == s + 1);
  const uint32_t leads = (uint32_t)__ballot(s >= 0 && (s & 3) == 0 && s < c.pages * c.page_size) & runs & (runs >> 1) & (runs >> 2) & 0x7Fu;
  const Slot at = slot_at(__shfl(s, 3 + row), c.pages, groups);
  if (t < T && at.ok && u.ok) {  // both lanes of a K block
    if constexpr (ROPE)
      turn_key<F32>(r, k, t * ks + (int64_t)u.h * D + 8 * u.j, u.j, table + ((threadIdx.x >> 6) * 4 + row) * (r.rotary / 2), x);
    uint32_t sc;
    const uint32_t kc = quant8(x, *kg, sc);
    uint8_t* rec = c.cache + record_at<D>(at, c.heads, u.h, groups);
    const int g = u.j / (D / 32), blk = u.j >> 1;
    *reinterpret_cast<uint32_t*>(rec + (g * 16 + at.t) * R::kLane + (u.j % (D / 32)) * 4) = kc;
    if ((u.j & 1) == 0) rec[R::kKs + (g * 16 + at.t) * (D / 64) + blk % (D / 64)] = (uint8_t)sc;
  }
  auto load_v = [&](int64_t entry) {
    const int64_t from = entry * vs + (int64_t)u.h * D + 32 * u.m + 4 * u.c4;
    load4_at<F32>(v, from, x);
    load4_at<F32>(v, from + 16, x + 4);
  };
  uint32_t sc;
  if ((leads >> 3) & 15u) {  // a quad's first entry is one of the wave's
    const int lead = __builtin_ctz(leads >> 3);
    // The quad's place is that of row `lead`.
    Slot q;
    q.first = (uint32_t)__builtin_amdgcn_readlane((int)at.first, 16 * lead);
    q.group = (uint32_t)__builtin_amdgcn_readlane((int)at.group, 16 * lead);
    q.t = __builtin_amdgcn_readlane(at.t, 16 * lead);
    if (u.ok) {
      load_v(first + lead + row);
      const uint32_t w = quad_transpose(quant44(x, *vg, u.c4 & 1, sc), row);
      uint8_t* rec = c.cache + record_at<D>(q, c.heads, u.h, groups);
      *reinterpret_cast<uint32_t*>(rec + v_at<D>(u, q.t >> 2) + row * R::kLane) = w;
      if (u.c4 < 2) rec[vs_at<D>(u, q.t >> 2) + 4 * u.c4 + row] = (uint8_t)sc;
    }
  }
  const bool alone = ((leads >> row) & 15u) == 0;  // none of the quads that could hold entry t is whole
  if (alone && t < T && at.ok && u.ok) {
    load_v(t);
    const uint32_t w = quant44(x, *vg, u.c4 & 1, sc);
    uint8_t* rec = c.cache + record_at<D>(at, c.heads, u.h, groups);
    // Another entry of this call may own the dword's other nibbles: change
    // this token's alone. Its old value is stable (no one else writes it), so
    // xor with old ^ new sets it whatever happens to the rest.
    const int sh = 4 * (at.t & 3);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t* p = reinterpret_cast<uint32_t*>(rec + v_at<D>(u, at.t >> 2) + i * R::kLane);
      const uint32_t old = __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      const uint32_t flip = (((old >> sh) ^ (w >> 4 * i)) & 0x000F000Fu) << sh;
      if (flip) __hip_atomic_fetch_xor(p, flip, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    if (u.c4 < 2) rec[vs_at<D>(u, at.t >> 2) + 4 * u.c4 + (at.t & 3)] = (uint8_t)sc;
  }
}

template <int D, bool F32>
__global__ __launch_bounds__(256) void k_kv_write(CacheArgs c, const void* k, const void* v, int64_t T, int64_t ks,
                                                  int64_t vs, const int64_t* slots, const float* kg, const float* vg,
                                                  Div groups) {
  write_units<D, F32, false>(c, k, v, T, ks, vs, slots, kg, vg, groups, blockIdx.x, RopeArgs{}, nullptr);
}

// The first kv_parts workgroups of a group of tokens write its keys and values,
// the others turn its queries. 8192 tokens of 40 query heads and 8 kv heads of
// 128 (212 MB) 47 to 51 us on inputs that no cache holds, 4.2 to 4.5 TB/s of the
// 4.7 of a copy; 40 on the same ones again, part of which the last-level cache
// keeps. (Nontemporal stores of the queries: 51 where these took 49.) One token
// 4.1 us. Apart, the rotation of the keys is another 34 MB.
template <int D, bool F32, bool OUT32>
__global__ __launch_bounds__(256) void k_rope_kv_write(RopeArgs r, RopeUnits units, CacheArgs c, const void* k, const void* v,
                                                       int64_t ks, int64_t vs, const int64_t* slots, const float* kg,
                                                       const float* vg, Div groups, unsigned kv_parts) {
  __shared__ f32x2 table[kRopeTokens * D / 2];
  const int64_t first = ((int64_t)blockIdx.z * gridDim.y + blockIdx.y) * kRopeTokens;
  if (first >= r.T) return;
  const int tokens = r.T - first < kRopeTokens ? (int)(r.T - first) : kRopeTokens;
  rope_table(r, first, tokens, units.half, table);
  __syncthreads();
  if (blockIdx.x >= kv_parts) {
    rope_rows<F32, OUT32>(r, units, first, tokens, blockIdx.x - kv_parts, gridDim.x - kv_parts, table);
    return;
  }
  for (unsigned chunk = blockIdx.x; chunk * 16 < (unsigned)c.heads * (D / 8); chunk += kv_parts)
    write_units<D, F32, true>(c, k, v, r.T, ks, vs, slots, kg, vg, groups, chunk, r, table);
}

// 8 numbers of a code dword: fl(fl(q s) g).
__device__ __forceinline__ void deq8(uint32_t w, const float (&s)[8], float g, float (&y)[8]) {
  const f32x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0), p1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1);
  const f32x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2), p3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3);
  const float q[8] = {p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = q[i] * s[i] * g;
}

template <bool F32>
__device__ __forceinline__ void store4_at(void* base, int64_t elem, const float* v) {
  if constexpr (F32) {
    __builtin_nontemporal_store(f32x4{v[0], v[1], v[2], v[3]}, reinterpret_cast<f32x4*>(reinterpret_cast<float*>(base) + elem));
  } else {
    typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
    const bf16x4 b = {(__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3]};
    __builtin_nontemporal_store(__builtin_bit_cast(u32x2, b), reinterpret_cast<u32x2*>(reinterpret_cast<__bf16*>(base) + elem));
  }
}

// Units as in k_kv_write: the four entries of a wave, neighbours in a record
// as a rule, read the same V dwords. Bound by memory: 65536 tokens of 8 heads
// of 128, 344 MB, in 53 to 65 us, 5.3 to 6.5 TB/s (most of it stores).
template <int D, bool F32>
__global__ __launch_bounds__(256) void k_kv_read(CacheArgs c, const int64_t* slots, int64_t T, const float* kg,
                                                 const float* vg, void* k, void* v, Div groups) {
  using R = KvRec<D>;
  const int lane = threadIdx.x & 63;
  const int64_t t = (((int64_t)blockIdx.z * gridDim.y + blockIdx.y) * 4 + (threadIdx.x >> 6)) * 4 + (lane >> 4);
  const Unit<D> u = unit_at<D>(blockIdx.x * 16 + (lane & 15), c.heads);
  if (t >= T || !u.ok) return;
  const Slot at = slot_at(slots[t], c.pages, groups);
  const int64_t to = t * c.heads * D + (int64_t)u.h * D;
  float y[8], z[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = z[i] = 0.0f;
  if (at.ok) {
    const uint8_t* rec = c.cache + record_at<D>(at, c.heads, u.h, groups);
    const int g = u.j / (D / 32), blk = u.j >> 1, sh = 4 * (at.t & 3);
    const uint32_t kc = *reinterpret_cast<const uint32_t*>(rec + (g * 16 + at.t) * R::kLane + (u.j % (D / 32)) * 4);
    const uint32_t ksc = rec[R::kKs + (g * 16 + at.t) * (D / 64) + blk % (D / 64)];
    const u32x2 vsc = *reinterpret_cast<const u32x2*>(rec + vs_at<D>(u, at.t >> 2));
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w |= ((*reinterpret_cast<const uint32_t*>(rec + v_at<D>(u, at.t >> 2) + i * R::kLane) >> sh) & 0x000F000Fu) << 4 * i;
    const float vs0 = e4m3_to_f32<0>(vsc[0] >> 2 * sh), vs1 = e4m3_to_f32<0>(vsc[1] >> 2 * sh);
    const float s[8] = {vs0, vs0, vs0, vs0, vs1, vs1, vs1, vs1};
    const float ks = e4m3_to_f32<0>(ksc);
    const float s2[8] = {ks, ks, ks, ks, ks, ks, ks, ks};
    deq8(kc, s2, *kg, y);
    deq8(w, s, *vg, z);
  }
  store8_at<F32>(k, to + 8 * u.j, y);
  store4_at<F32>(v, to + 32 * u.m + 4 * u.c4, z);
  store4_at<F32>(v, to + 32 * u.m + 16 + 4 * u.c4, z + 4);
}

// ---- pages and slots ---------------------------------------------------------

// All pages free, page 0 on top.
__global__ __launch_bounds__(256) void k_kv_pool_reset(int32_t* pool, int64_t pages) {
  for (int64_t i = blockIdx.x * 256 + threadIdx.x; i < pages + kPoolHead; i += (int64_t)gridDim.x * 256)
    pool[i] = i == 0 ? (int32_t)pages : i < kPoolHead ? 0 : (int32_t)(pages - 1 - (i - kPoolHead));
}

// Sums of a request's rows, pages taken and pages given back. They stop at
// 2^30: past T, the pool and a table's width nothing depends on their value.
struct Sums {
  uint32_t rows, taken, given;
};
__device__ __forceinline__ uint32_t sat_add(uint32_t a, uint32_t b) {
  const uint32_t s = a + b;
  return s < (1u << 30) ? s : 1u << 30;
}
__device__ __forceinline__ Sums operator+(const Sums& a, const Sums& b) {
  return {sat_add(a.rows, b.rows), sat_add(a.taken, b.taken), sat_add(a.given, b.given)};
}

// Requests in chunks of one a thread, with sums over those before. Every
// workgroup goes over the requests for itself (they are few numbers, and read
// only) and fills its rows; the last to arrive, when nobody reads them any
// more, writes lengths, the pages that are given back and the pool. So one
// launch does it all, a step of few rows in one workgroup. What bounds it is
// the chain of trips: requests, sums, search, page numbers, rows, arrival. 64
// requests of 5 rows 3.3 us, 61 prompts of 500000 rows 12.5 us (their 6 MB take
// 1.3); with a run of 512 rows a wave, to spare searches, 5.1 and 14, with
// eight rows of a thread at a time 4.0 and 12. ROWS: rows of a thread, N threads.
template <int N, int ROWS>
__global__ __launch_bounds__(N) void k_kv_advance(AdvanceArgs a, Div page) {
  constexpr int kAdvanceThreads = N, kAdvanceRows = ROWS * N;
  __shared__ Sums waves[kAdvanceThreads / 64];
  __shared__ uint32_t end[kAdvanceThreads], begin[kAdvanceThreads], before[kAdvanceThreads], given_end[kAdvanceThreads];
  __shared__ int old[kAdvanceThreads], held[kAdvanceThreads], first_gone[kAdvanceThreads];
  __shared__ uint32_t popped, status, arrived;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int32_t* stack = a.pool + kPoolHead;
  const int free = a.pool[0], top = free < 0 ? 0 : free > a.pages ? a.pages : free;
  const uint32_t T = (uint32_t)a.T, row0 = blockIdx.x * kAdvanceRows, row1 = T - row0 < kAdvanceRows ? T : row0 + kAdvanceRows;
  const int64_t room64 = (int64_t)a.table_width * a.page_size;
  const int room = room64 < (1 << 30) ? (int)room64 : 1 << 30;
  if (tid == 0) popped = status = 0;

  struct Request {
    int len;  // after the call
    bool ok;
  };
  int next_count, next_len;  // of the chunk to come, asked for a chunk ahead
  auto ask = [&](int64_t chunk) {
    const int64_t b = chunk * kAdvanceThreads + tid;
    next_count = b < a.B ? a.counts[b] : 0;
    next_len = b < a.B ? a.seq_lens[b] : 0;
  };
  // The chunk's requests: their numbers in LDS, and the sums up to its end.
  auto sweep = [&](int64_t chunk, Sums& sum) {
    const int c = next_count;
    int was = next_len;
    ask(chunk + 1);
    was = was < 0 ? 0 : was > 1 << 30 ? 1 << 30 : was;
    const int64_t next = (int64_t)was + c;
    const bool over = c > 0 && next > room;
    const int now = next < 0 ? 0 : over ? was : (int)next;
    int has = (int)div_n((uint32_t)was + page.d - 1, page), need = (int)div_n((uint32_t)now + page.d - 1, page);
    has = has < a.table_width ? has : a.table_width;
    need = need < a.table_width ? need : a.table_width;
    const Sums own{c > 0 ? ((uint32_t)c < (1u << 30) ? (uint32_t)c : 1u << 30) : 0u, need > has ? (uint32_t)(need - has) : 0u,
                   need < has ? (uint32_t)(has - need) : 0u};
    Sums up = own;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const Sums x{(uint32_t)__shfl_up((int)up.rows, d), (uint32_t)__shfl_up((int)up.taken, d), (uint32_t)__shfl_up((int)up.given, d)};
      if (lane >= d) up = up + x;
    }
    __syncthreads();  // what the chunk before left in LDS has been read
    if (lane == 63) waves[wave] = up;
    __syncthreads();
    Sums base = sum;
#pragma unroll
    for (int w = 0; w < kAdvanceThreads / 64; ++w) {
      if (w < wave) base = base + waves[w];
      sum = sum + waves[w];
    }
    up = base + up;
    const bool many = c > 0 && up.rows > T, lack = !many && own.taken > 0 && up.taken > (uint32_t)top;
    Request q;
    q.ok = !(over || many || lack);
    q.len = q.ok ? now : was;
    end[tid] = up.rows;
    begin[tid] = up.rows - own.rows;
    before[tid] = up.taken - own.taken;
    given_end[tid] = up.given;
    old[tid] = q.ok ? was : -1;
    held[tid] = has;
    first_gone[tid] = need;
    if (own.taken > 0 && q.ok) atomicMax(&popped, up.taken);
    const uint32_t bits = (lack ? 1u : 0u) | (over ? 2u : 0u) | (many ? 4u : 0u);
    if (bits) atomicOr(&status, bits);
    __syncthreads();
    return q;
  };
  // The first of the chunk's requests whose sum passes each n.
  auto find = [&](const uint32_t* sums, const auto& n, auto& i) {
    constexpr int kOf = sizeof(n) / sizeof(n[0]);
#pragma unroll
    for (int u = 0; u < kOf; ++u) i[u] = 0;
#pragma unroll
    for (int d = kAdvanceThreads / 2; d > 0; d /= 2)
#pragma unroll
      for (int u = 0; u < kOf; ++u) i[u] += sums[i[u] + d - 1] <= n[u] ? d : 0;
  };

  const int64_t chunks = (a.B + kAdvanceThreads - 1) / kAdvanceThreads;
  Sums sum{0, 0, 0};
  Request mine{0, false};
  int64_t swept = 0;
  ask(0);
  for (; swept < chunks; ++swept) {
    const int64_t chunk = swept;
    if (chunk > 0 && sum.rows >= row1) break;
    const uint32_t from = sum.rows;
    mine = sweep(chunk, sum);
    const uint32_t to = sum.rows < row1 ? sum.rows : row1;
    // A thread's rows without a branch, so that their searches and their page
    // numbers are on their way together.
    for (uint32_t t0 = (from > row0 ? from : row0) + tid; t0 < to; t0 += ROWS * kAdvanceThreads) {
      uint32_t t[ROWS];
      int i[ROWS], position[ROWS], p[ROWS], in[ROWS], shift[ROWS];
      int32_t* entry[ROWS];
      bool live[ROWS], comes[ROWS];
#pragma unroll
      for (int u = 0; u < ROWS; ++u) t[u] = t0 + u * kAdvanceThreads;
      find(end, t, i);
#pragma unroll
      for (int u = 0; u < ROWS; ++u) {
        const int was = old[i[u]];
        live[u] = t[u] < to && was >= 0;
        const int pos = live[u] ? was + (int)(t[u] - begin[i[u]]) : 0, col = (int)div_n((uint32_t)pos, page);
        const int64_t b = chunk * kAdvanceThreads + (live[u] ? i[u] : 0);
        in[u] = pos - col * (int)page.d;
        entry[u] = a.table + b * a.table_stride + col;
        comes[u] = live[u] && col >= held[i[u]];
        position[u] = pos;
        const int32_t* at = comes[u] ? stack + (top - 1 - (int)before[i[u]] - (col - held[i[u]])) : entry[u];
        p[u] = *(live[u] ? at : a.pool);
        shift[u] = a.offsets != nullptr ? a.offsets[b] : 0;
      }
#pragma unroll
      for (int u = 0; u < ROWS; ++u) {
        if (t[u] >= to) continue;
        if (comes[u] && in[u] == 0) *entry[u] = p[u];
        if (a.slots != nullptr) a.slots[t[u]] = live[u] ? (int64_t)p[u] * page.d + in[u] : -1;
        if (a.positions != nullptr) a.positions[t[u]] = live[u] ? position[u] + shift[u] : 0;
      }
    }
  }
  for (uint32_t t = (sum.rows > row0 ? sum.rows : row0) + tid; t < row1; t += kAdvanceThreads) {  // rows of no request
    if (a.slots != nullptr) a.slots[t] = -1;
    if (a.positions != nullptr) a.positions[t] = 0;
  }

  __syncthreads();
  if (tid == 0) arrived = gridDim.x == 1 ? 0u : __hip_atomic_fetch_add(a.pool + 2, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __syncthreads();
  if (arrived != gridDim.x - 1) return;
  for (; swept < chunks; ++swept) sweep(swept, sum);  // sums over all requests
  const int64_t left64 = (int64_t)top - popped + sum.given;
  const int left = left64 < a.pages ? (int)left64 : a.pages;
  sum = {0, 0, 0};
  // Pages of a chunk's requests from sum `from` on come back so that a growth
  // that is undone leaves the stack as it was; `of` of a thread at a time
  // (7800 pages one by one 22 us, by eight 12; few of them by eight 1 us more).
  auto back = [&](uint32_t from, int64_t chunk, auto of) {
    constexpr int kOf = decltype(of)::value;
    for (uint32_t j0 = from + tid; j0 < sum.given; j0 += kOf * kAdvanceThreads) {
      uint32_t j[kOf];
      int i[kOf], p[kOf];
      int32_t* entry[kOf];
#pragma unroll
      for (int u = 0; u < kOf; ++u) {
        const uint32_t n = j0 + u * kAdvanceThreads;
        j[u] = n < sum.given ? n : j0;
      }
      find(given_end, j, i);
#pragma unroll
      for (int u = 0; u < kOf; ++u) {
        const uint32_t i0 = i[u] > 0 ? given_end[i[u] - 1] : from;
        entry[u] = a.table + (chunk * kAdvanceThreads + i[u]) * a.table_stride + first_gone[i[u]] + (j[u] - i0);
        p[u] = *entry[u];
      }
#pragma unroll
      for (int u = 0; u < kOf; ++u) {
        if (u > 0 && j[u] == j0) break;
        const int at = left - 1 - (int)j[u];
        if (at >= 0) stack[at] = p[u];
        *entry[u] = -1;
      }
    }
  };
  ask(0);
  for (int64_t chunk = 0; chunk < chunks; ++chunk) {
    const uint32_t from = sum.given;
    if (chunks > 1) mine = sweep(chunk, sum);
    else sum.given = given_end[kAdvanceThreads - 1];
    const int64_t b = chunk * kAdvanceThreads + tid;
    if (b < a.B) {
      a.seq_lens[b] = mine.len;
      if (a.q_offsets != nullptr) a.q_offsets[b + 1] = (int32_t)(end[tid] < T ? end[tid] : T);
    }
    if (sum.given - from > 4 * kAdvanceThreads) back(from, chunk, std::integral_constant<int, 8>{});
    else back(from, chunk, std::integral_constant<int, 1>{});
  }
  if (tid == 0) {
    if (a.q_offsets != nullptr) a.q_offsets[0] = 0;
    a.pool[0] = left;
    if (status) a.pool[1] |= (int)status;
    a.pool[2] = 0;
  }
}

// x: 16 units of an entry; y, z: 16 entries.
dim3 unit_grid(int64_t T, int heads, int dim) {
  const int64_t n = (T + 15) / 16, gy = n < 32768 ? n : 32768;
  return dim3((unsigned)((heads * (dim / 8) + 15) / 16), (unsigned)gy, (unsigned)((n + gy - 1) / gy));
}

template <int D>
void write_d(const CacheArgs& c, const void* k, const void* v, bool f32, int64_t T, int64_t ks, int64_t vs,
             const int64_t* slots, const float* kg, const float* vg, hipStream_t s) {
  const dim3 grid = unit_grid(T, c.heads, D);
  const Div groups = div_by((uint32_t)c.page_size / 16);
  if (f32) k_kv_write<D, true><<<grid, dim3(256), 0, s>>>(c, k, v, T, ks, vs, slots, kg, vg, groups);
  else k_kv_write<D, false><<<grid, dim3(256), 0, s>>>(c, k, v, T, ks, vs, slots, kg, vg, groups);
}
// Workgroups of a group of tokens over `items` of them: as many as fill the
// chip, at most one an item.
unsigned rope_parts(int64_t T, int64_t items) {
  const int64_t groups = (T + kRopeTokens - 1) / kRopeTokens, want = (kRopeGroups + groups - 1) / groups;
  return (unsigned)(items < 1 ? 0 : items < want ? items : want);
}
int64_t rope_items(const RopeArgs& r, const RopeUnits& units) {
  const int64_t tokens = r.T < kRopeTokens ? r.T : kRopeTokens;
  return (tokens * r.heads * units.turned.d + 255) / 256;
}

template <int D, bool F32>
void rope_write_d(const RopeArgs& r, const CacheArgs& c, const void* k, const void* v, int64_t ks, int64_t vs, const int64_t* slots,
                  const float* kg, const float* vg, hipStream_t s) {
  const RopeUnits units = rope_units(r);
  dim3 grid = unit_grid(r.T, c.heads, D);
  const unsigned kv_parts = rope_parts(r.T, grid.x);
  grid.x = kv_parts + rope_parts(r.T, rope_items(r, units));
  const Div groups = div_by((uint32_t)c.page_size / 16);
  if (r.out_f32) k_rope_kv_write<D, F32, true><<<grid, dim3(256), 0, s>>>(r, units, c, k, v, ks, vs, slots, kg, vg, groups, kv_parts);
  else k_rope_kv_write<D, F32, false><<<grid, dim3(256), 0, s>>>(r, units, c, k, v, ks, vs, slots, kg, vg, groups, kv_parts);
}
template <int D>
void read_d(const CacheArgs& c, const int64_t* slots, int64_t T, const float* kg, const float* vg, void* k, void* v,
            bool f32, hipStream_t s) {
  const dim3 grid = unit_grid(T, c.heads, D);
  const Div groups = div_by((uint32_t)c.page_size / 16);
  if (f32) k_kv_read<D, true><<<grid, dim3(256), 0, s>>>(c, slots, T, kg, vg, k, v, groups);
  else k_kv_read<D, false><<<grid, dim3(256), 0, s>>>(c, slots, T, kg, vg, k, v, groups);
}

}  // namespace

hipError_t launch_kv_write(const CacheArgs& c, const void* k, const void* v, bool f32_in, int64_t T, int64_t k_stride,
                           int64_t v_stride, const int64_t* slots, const float* kg, const float* vg, hipStream_t s) {
  if (c.dim == 64) write_d<64>(c, k, v, f32_in, T, k_stride, v_stride, slots, kg, vg, s);
  else if (c.dim == 128) write_d<128>(c, k, v, f32_in, T, k_stride, v_stride, slots, kg, vg, s);
  else write_d<256>(c, k, v, f32_in, T, k_stride, v_stride, slots, kg, vg, s);
  return hipGetLastError();
}

hipError_t launch_rope_kv_write(const RopeArgs& r, const CacheArgs& c, const void* k, const void* v, int64_t ks, int64_t vs,
                                const int64_t* slots, const float* kg, const float* vg, hipStream_t s) {
  auto go = [&](auto f32) {
    constexpr bool F32 = decltype(f32)::value;
    if (c.dim == 64) rope_write_d<64, F32>(r, c, k, v, ks, vs, slots, kg, vg, s);
    else if (c.dim == 128) rope_write_d<128, F32>(r, c, k, v, ks, vs, slots, kg, vg, s);
    else rope_write_d<256, F32>(r, c, k, v, ks, vs, slots, kg, vg, s);
  };
  if (r.x_f32) go(std::true_type{});
  else go(std::false_type{});
  return hipGetLastError();
}

hipError_t launch_rope(const RopeArgs& r, hipStream_t s) {
  const RopeUnits units = rope_units(r);
  dim3 grid = unit_grid(r.T, 1, 64);
  grid.x = rope_parts(r.T, rope_items(r, units));
  if (r.x_f32 && r.out_f32) k_rope<true, true><<<grid, dim3(256), 0, s>>>(r, units);
  else if (r.x_f32) k_rope<true, false><<<grid, dim3(256), 0, s>>>(r, units);
  else if (r.out_f32) k_rope<false, true><<<grid, dim3(256), 0, s>>>(r, units);
  else k_rope<false, false><<<grid, dim3(256), 0, s>>>(r, units);
  return hipGetLastError();
}

hipError_t launch_kv_pool_reset(int32_t* pool, int64_t pages, hipStream_t s) {
  const int64_t n = (pages + kPoolHead + 255) / 256;
  k_kv_pool_reset<<<dim3((unsigned)(n < 1024 ? n : 1024)), dim3(256), 0, s>>>(pool, pages);
  return hipGetLastError();
}

hipError_t launch_kv_advance(const AdvanceArgs& a, hipStream_t s) {
  const Div page = div_by((uint32_t)a.page_size);
  auto groups = [&](int rows) { return dim3((unsigned)(a.T > rows ? (a.T + rows - 1) / rows : 1)); };
  // Many rows of a workgroup where there would be many workgroups, whose
  // arrivals queue: 512 threads of 4 / 256 of 2, 500000 rows and back 22.5 /
  // 29 us, 32000 11 / 10.3; and a chunk for as many requests as there are.
  if (a.B <= 256 && a.T <= 1 << 17) k_kv_advance<256, 2><<<groups(512), dim3(256), 0, s>>>(a, page);
  else if (a.B <= 512) k_kv_advance<512, 4><<<groups(2048), dim3(512), 0, s>>>(a, page);
  else k_kv_advance<1024, 2><<<groups(2048), dim3(1024), 0, s>>>(a, page);
  return hipGetLastError();
}

hipError_t launch_kv_read(const CacheArgs& c, const int64_t* slots, int64_t T, const float* kg, const float* vg, void* k,
                          void* v, bool f32_out, hipStream_t s) {
  if (c.dim == 64) read_d<64>(c, slots, T, kg, vg, k, v, f32_out, s);
  else if (c.dim == 128) read_d<128>(c, slots, T, kg, vg, k, v, f32_out, s);
  else read_d<256>(c, slots, T, kg, vg, k, v, f32_out, s);
  return hipGetLastError();
}

}  // namespace nvfp4
