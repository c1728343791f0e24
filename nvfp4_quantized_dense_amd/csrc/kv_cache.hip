// kv_cache.hip -- keys and values into the paged NVFP4 cache as they are
// written, and back to dense rows.
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

// 8192 tokens of 8 heads of 128 (43 MB) take 10 to 12 us, bound by instruction
// issue (two block scales with their exact divisions a lane) as much as by
// memory; 64 tokens 3.8 us, the dependent trips: slots, rows, stores. Entries
// of the list that fill an aligned quad of slots are written whole by the wave
// that holds the first of them; any other entry's V shares its dwords with
// tokens that another wave, or an earlier call, owns.
template <int D, bool F32>
__global__ __launch_bounds__(256) void k_kv_write(CacheArgs c, const void* k, const void* v, int64_t T, int64_t ks,
                                                  int64_t vs, const int64_t* slots, const float* kg, const float* vg,
                                                  Div groups) {
  using R = KvRec<D>;
  const int lane = threadIdx.x & 63, row = lane >> 4;
  const int64_t first = (((int64_t)blockIdx.z * gridDim.y + blockIdx.y) * 4 + (threadIdx.x >> 6)) * 4;
  if (first >= T) return;
  const Unit<D> u = unit_at<D>(blockIdx.x * 16 + (lane & 15), c.heads);
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

hipError_t launch_kv_read(const CacheArgs& c, const int64_t* slots, int64_t T, const float* kg, const float* vg, void* k,
                          void* v, bool f32_out, hipStream_t s) {
  if (c.dim == 64) read_d<64>(c, slots, T, kg, vg, k, v, f32_out, s);
  else if (c.dim == 128) read_d<128>(c, slots, T, kg, vg, k, v, f32_out, s);
  else read_d<256>(c, slots, T, kg, vg, k, v, f32_out, s);
  return hipGetLastError();
}

}  // namespace nvfp4
