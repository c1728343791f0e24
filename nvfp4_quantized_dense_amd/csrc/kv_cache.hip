// kv_cache.hip -- keys and values into the paged NVFP4 cache as they are
// written, and back to dense rows.
#include "attention.h"
#include "kv_layout.h"

namespace nvfp4 {
namespace {

// Where a slot is: its record group and token, or nothing.
struct Slot {
  int64_t page;
  int group, t;
  bool ok;
};
__device__ __forceinline__ Slot slot_at(int64_t slot, int64_t pages, int page_size) {
  Slot r{0, 0, 0, false};
  const int64_t page = slot / page_size;
  r.ok = slot >= 0 && page < pages;
  if (r.ok) {
    const int in = (int)(slot - page * page_size);
    r.page = page;
    r.group = in >> 4;
    r.t = in & 15;
  }
  return r;
}

// A V code byte holds two tokens and an aligned quad of tokens shares 16-bit
// units, so list entries t - a .. t - a + 3 that fill an aligned quad are
// handled together by the first of them. -1: entry t belongs to the quad of
// an earlier entry, 4: it leads a quad, 1: it stands alone.
__device__ __forceinline__ int quad_role(const int64_t* slots, int64_t T, int64_t t, int64_t slot) {
  const int a = (int)(slot & 3);
  const int64_t first = t - a;
  if (first < 0 || first + 3 >= T) return 1;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (slots[first + i] != slot - a + i) return 1;
  return a == 0 ? 4 : -1;
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

template <bool F32>
__device__ __forceinline__ void store8_at(void* base, int64_t elem, const float (&v)[8]) {
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

// NVFP4 of 8 channels (the neighbouring lane holds the block's other 8), by
// k_quantize's rule.
__device__ __forceinline__ uint32_t quant8(const float (&v)[8], float g_inv, uint32_t& scale) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  m = max(m, (uint32_t)__shfl_xor((int)m, 1));
  const BlockScale bs = block_scale(__uint_as_float(m), g_inv);
  scale = bs.byte;
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = v[i] * bs.r;
  return e2m1_pack8(y);
}

// One thread per (list entry, head, 8 channels).
template <int D, bool F32>
__global__ __launch_bounds__(256) void k_kv_write(CacheArgs c, const void* k, const void* v, int64_t T, int64_t ks,
                                                  int64_t vs, const int64_t* slots, const float* kg, const float* vg) {
  using R = KvRec<D>;
  constexpr int kTh = D / 8;
  const int64_t n = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 256 + threadIdx.x;
  const int j = (int)(n % kTh);
  const int64_t th = n / kTh, t = th / c.heads;
  if (t >= T) return;  // whole groups of kTh lanes
  const int h = (int)(th - t * c.heads);
  const int64_t slot = slots[t];
  const Slot s = slot_at(slot, c.pages, c.page_size);
  if (!s.ok) return;
  uint8_t* rec = c.cache + rec_offset<D>(s.page, c.heads, h, c.page_size / 16, s.group);
  const int64_t col = (int64_t)h * D + 8 * j;
  float x[8];
  uint32_t sc;
  // K: dword j % (D/32) of lane (j / (D/32), t).
  load8_at<F32>(k, t * ks + col, x);
  const uint32_t kc = quant8(x, *kg, sc);
  const int g = j / (D / 32), blk = j >> 1;
  *reinterpret_cast<uint32_t*>(rec + g * 16 * R::kLane + s.t * R::kLane + (j % (D / 32)) * 4) = kc;
  if ((j & 1) == 0) rec[R::kKs + (g * 16 + s.t) * (D / 64) + blk % (D / 64)] = (uint8_t)sc;
  // V: channel 16 blk + 8 (j & 1) + i, a 16-bit unit per channel and quad.
  const int role = quad_role(slots, T, t, slot);
  if (role < 0) return;
  const int q = s.t >> 2;
  uint8_t* vrec = rec + R::kV + (q * 16 + 8 * (j & 1)) * R::kLane + 2 * blk;
  uint8_t* srec = rec + R::kVs + (q * (D / 16) + blk) * 4;
  if (role == 4) {
    uint32_t w[4], s4 = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      load8_at<F32>(v, (t + i) * vs + col, x);
      w[i] = quant8(x, *vg, sc);
      s4 |= sc << (8 * i);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t u = ((w[0] >> 4 * i) & 15u) | (((w[1] >> 4 * i) & 15u) << 4) | (((w[2] >> 4 * i) & 15u) << 8) |
                         (((w[3] >> 4 * i) & 15u) << 12);
      *reinterpret_cast<uint16_t*>(vrec + i * R::kLane) = (uint16_t)u;
    }
    if ((j & 1) == 0) *reinterpret_cast<uint32_t*>(srec) = s4;
  } else {
    load8_at<F32>(v, t * vs + col, x);
    const uint32_t w = quant8(x, *vg, sc);
    // Another entry of this call may own the unit's other nibbles: change
    // this token's alone. Its old value is stable (no one else writes it), so
    // xor with old ^ new sets it whatever happens to the rest of the dword.
    const int sh = 16 * (blk & 1) + 4 * (s.t & 3);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t* p = reinterpret_cast<uint32_t*>(reinterpret_cast<uintptr_t>(vrec + i * R::kLane) & ~uintptr_t(3));
      const uint32_t old = __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      const uint32_t flip = (((old >> sh) ^ (w >> 4 * i)) & 15u) << sh;
      if (flip) __hip_atomic_fetch_xor(p, flip, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    if ((j & 1) == 0) srec[s.t & 3] = (uint8_t)sc;
  }
}

// 8 numbers of a code dword with one block scale: fl(fl(q s) g).
__device__ __forceinline__ void deq8(uint32_t w, float s, float g, float (&y)[8]) {
  const f32x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0), p1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1);
  const f32x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2), p3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3);
  y[0] = p0[0] * s * g; y[1] = p0[1] * s * g; y[2] = p1[0] * s * g; y[3] = p1[1] * s * g;
  y[4] = p2[0] * s * g; y[5] = p2[1] * s * g; y[6] = p3[0] * s * g; y[7] = p3[1] * s * g;
}

// One thread per (list entry, head, 8 channels).
template <int D, bool F32>
__global__ __launch_bounds__(256) void k_kv_read(CacheArgs c, const int64_t* slots, int64_t T, const float* kg,
                                                 const float* vg, void* k, void* v) {
  using R = KvRec<D>;
  constexpr int kTh = D / 8;
  const int64_t n = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 256 + threadIdx.x;
  const int j = (int)(n % kTh);
  const int64_t th = n / kTh, t = th / c.heads;
  if (t >= T) return;
  const int h = (int)(th - t * c.heads);
  const int64_t slot = slots[t];
  const Slot s = slot_at(slot, c.pages, c.page_size);
  const int64_t row = (int64_t)c.heads * D, col = (int64_t)h * D + 8 * j;
  float y[8];
  if (!s.ok) {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = 0.0f;
    store8_at<F32>(k, t * row + col, y);
    store8_at<F32>(v, t * row + col, y);
    return;
  }
  const uint8_t* rec = c.cache + rec_offset<D>(s.page, c.heads, h, c.page_size / 16, s.group);
  const int g = j / (D / 32), blk = j >> 1;
  const uint32_t kc = *reinterpret_cast<const uint32_t*>(rec + g * 16 * R::kLane + s.t * R::kLane + (j % (D / 32)) * 4);
  const uint32_t ksc = rec[R::kKs + (g * 16 + s.t) * (D / 64) + blk % (D / 64)];
  deq8(kc, e4m3_to_f32<0>(ksc), *kg, y);
  store8_at<F32>(k, t * row + col, y);
  const int role = quad_role(slots, T, t, slot);
  if (role < 0) return;
  const int q = s.t >> 2;
  const uint8_t* vrec = rec + R::kV + (q * 16 + 8 * (j & 1)) * R::kLane + 2 * blk;
  const uint32_t s4 = *reinterpret_cast<const uint32_t*>(rec + R::kVs + (q * (D / 16) + blk) * 4);
  uint32_t u[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) u[i] = *reinterpret_cast<const uint16_t*>(vrec + i * R::kLane);
  const int lo = role == 4 ? 0 : s.t & 3, hi = role == 4 ? 4 : lo + 1;
  for (int i = lo; i < hi; ++i) {
    uint32_t w = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) w |= ((u[e] >> 4 * i) & 15u) << 4 * e;
    deq8(w, e4m3_to_f32<0>((s4 >> 8 * i) & 255u), *vg, y);
    store8_at<F32>(v, (t + i - lo) * row + col, y);
  }
}

dim3 flat_grid(int64_t threads) {
  const int64_t wg = (threads + 255) / 256, gx = wg < (1 << 20) ? wg : (1 << 20);
  return dim3((unsigned)gx, (unsigned)((wg + gx - 1) / gx));
}

template <int D>
void write_d(const CacheArgs& c, const void* k, const void* v, bool f32, int64_t T, int64_t ks, int64_t vs,
             const int64_t* slots, const float* kg, const float* vg, hipStream_t s) {
  const dim3 grid = flat_grid(T * c.heads * (D / 8));
  if (f32) k_kv_write<D, true><<<grid, dim3(256), 0, s>>>(c, k, v, T, ks, vs, slots, kg, vg);
  else k_kv_write<D, false><<<grid, dim3(256), 0, s>>>(c, k, v, T, ks, vs, slots, kg, vg);
}
template <int D>
void read_d(const CacheArgs& c, const int64_t* slots, int64_t T, const float* kg, const float* vg, void* k, void* v,
            bool f32, hipStream_t s) {
  const dim3 grid = flat_grid(T * c.heads * (D / 8));
  if (f32) k_kv_read<D, true><<<grid, dim3(256), 0, s>>>(c, slots, T, kg, vg, k, v);
  else k_kv_read<D, false><<<grid, dim3(256), 0, s>>>(c, slots, T, kg, vg, k, v);
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
