// norm_quant.hip -- residual addition + root-mean-square norm + NVFP4
// quantization in one pass, and the way back from NVFP4 to numbers.
#include "attention.h"
#include "device_common.h"

namespace nvfp4 {
namespace {

__device__ __forceinline__ void unpack8(const u32x4& a, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(a[i] << 16);
    v[2 * i + 1] = __uint_as_float(a[i] & 0xFFFF0000u);
  }
}

// 8 consecutive elements, chunk c of a row or matrix.
template <bool F32>
__device__ __forceinline__ void load8(const void* p, int64_t c, float (&v)[8]) {
  if constexpr (F32) {
    const f32x4 a = reinterpret_cast<const f32x4*>(p)[2 * c], b = reinterpret_cast<const f32x4*>(p)[2 * c + 1];
#pragma unroll
    for (int i = 0; i < 4; ++i) { v[i] = a[i]; v[4 + i] = b[i]; }
  } else {
    unpack8(reinterpret_cast<const u32x4*>(p)[c], v);
  }
}

// Stored past the caches (nontemporal): the norm and dequantization of 8192 x
// 7168 take 92 us so, 113 us with plain stores (loads are better plain: 109).
template <bool F32>
__device__ __forceinline__ void store8(void* p, int64_t c, const float (&v)[8]) {
  if constexpr (F32) {
    f32x4* o = reinterpret_cast<f32x4*>(p) + 2 * c;
    __builtin_nontemporal_store(f32x4{v[0], v[1], v[2], v[3]}, o);
    __builtin_nontemporal_store(f32x4{v[4], v[5], v[6], v[7]}, o + 1);
  } else {
    bf16x8 b;
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = (__bf16)v[i];
    __builtin_nontemporal_store(__builtin_bit_cast(u32x4, b), reinterpret_cast<u32x4*>(p) + c);
  }
}

// One workgroup of NT threads per row:
//   z = round(x + residual),  ms = sum z^2 / K,  rstd = fl32(1 / sqrt(ms + eps)),
//   y = fl(fl(z rstd) w),  NVFP4(y) as k_quantize.
// The squares of 24-bit numbers are exact in 64 bits and their sum is off by
// 2^-53 per addition whatever the order, so rstd (and with it every code) is
// the same for any split of the row over threads. The first CH chunks of 8
// elements per thread stay in registers; a longer row (past 8192 elements) is
// read a second time. Bound by memory: 8192 x 7168 in bf16 with a bf16
// residual, 385 MB, in 59 to 68 us, 5.7 to 6.5 TB/s. One row is bound by its trips: load,
// sum, 64-bit root, store.
template <bool XF, bool RF, int NT, int CH>
__global__ __launch_bounds__(NT) void k_add_rmsnorm_quant(NormArgs a) {
  const int64_t row = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  if (row >= a.M) return;
  const int tid = threadIdx.x;
  const int64_t n8 = a.K / 8, base = row * n8;
  const bool has_res = a.residual != nullptr;
  auto load_z = [&](int64_t c, float (&z)[8]) {
    load8<XF>(a.x, base + c, z);
    if (has_res) {
      float r[8];
      load8<RF>(a.residual, base + c, r);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        z[i] += r[i];
        if constexpr (!RF) z[i] = (float)(__bf16)z[i];
      }
    }
  };
  auto store_z = [&](int64_t c, const float (&z)[8]) {
    if (a.residual_out == nullptr) return;
    if (has_res) store8<RF>(a.residual_out, base + c, z);
    else store8<XF>(a.residual_out, base + c, z);
  };
  float z[CH][8];
  double ss = 0.0;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int64_t c = tid + (int64_t)i * NT;
    if (c < n8) {
      load_z(c, z[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = __builtin_fma((double)z[i][j], (double)z[i][j], ss);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) z[i][j] = 0.0f;
    }
  }
  for (int64_t c = tid + (int64_t)CH * NT; c < n8; c += NT) {
    float t[8];
    load_z(c, t);
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = __builtin_fma((double)t[j], (double)t[j], ss);
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) ss += __shfl_xor(ss, o);
  constexpr int NW = NT / 64;
  __shared__ double wsum[NW];
  __shared__ uint32_t wmax[NW];
  if ((tid & 63) == 0) wsum[tid >> 6] = ss;
  __syncthreads();
  ss = 0.0;
#pragma unroll
  for (int w = 0; w < NW; ++w) ss += wsum[w];
  const float rstd = (float)(1.0 / __builtin_sqrt(ss / (double)a.K + a.eps));

  auto norm = [&](int64_t c, float (&t)[8]) {
    float w[8];
    if (a.w_f32) load8<true>(a.w, c, w);
    else load8<false>(a.w, c, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) t[j] = (t[j] * rstd) * w[j];
  };
  float g_inv;
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int64_t c = tid + (int64_t)i * NT;
    if (c < n8) {
      store_z(c, z[i]);
      norm(c, z[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(z[i][j]) & 0x7FFFFFFFu);
    }
  }
  if (a.g_inv == nullptr) {
    for (int64_t c = tid + (int64_t)CH * NT; c < n8; c += NT) {
      float t[8];
      load_z(c, t);
      norm(c, t);
#pragma unroll
      for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(t[j]) & 0x7FFFFFFFu);
    }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, o));
    if ((tid & 63) == 0) wmax[tid >> 6] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < NW; ++w) m = max(m, wmax[w]);
    const float g = __uint_as_float(m) / 2688.0f;
    g_inv = g != 0.0f ? 1.0f / g : 0.0f;
    if (tid == 0) a.row_g[row] = g;
  } else {
    g_inv = *a.g_inv;
  }
  // Lanes 2i and 2i + 1 hold a 16-element block (NT and n8 are even).
  auto quant = [&](int64_t c, const float (&t)[8]) {
    uint32_t bm = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) bm = max(bm, __float_as_uint(t[j]) & 0x7FFFFFFFu);
    bm = max(bm, (uint32_t)__shfl_xor((int)bm, 1));
    const BlockScale bs = block_scale(__uint_as_float(bm), g_inv);
    float y[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = t[j] * bs.r;
    reinterpret_cast<uint32_t*>(a.codes)[base + c] = e2m1_pack8(y);
    if ((c & 1) == 0) a.scales[(base + c) >> 1] = (uint8_t)bs.byte;
  };
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int64_t c = tid + (int64_t)i * NT;
    if (c < n8) quant(c, z[i]);
  }
  for (int64_t c = tid + (int64_t)CH * NT; c < n8; c += NT) {
    float t[8];
    load_z(c, t);
    store_z(c, t);  // the last read of this chunk: residual_out may be the residual
    norm(c, t);
    quant(c, t);
  }
}

// One thread per 8 elements: fl(fl(q s) g), rounded to the output's type.
// Bound by memory: 8192 x 7168 to bf16, 150 MB, in 22 us, 6.9 TB/s.
template <bool F32>
__global__ __launch_bounds__(256) void k_dequantize(const uint32_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                                                    int64_t n8, int64_t row8, const float* g, const float* row_g, void* out) {
  const int64_t t = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 256 + threadIdx.x;
  if (t >= n8) return;
  const uint32_t w = codes[t];
  const float s = e4m3_to_f32<0>(scales[t >> 1]);
  const float gg = row_g != nullptr ? row_g[t / row8] : *g;
  float y[8];
  const f32x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0), p1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1);
  const f32x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2), p3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3);
  y[0] = p0[0] * s * gg; y[1] = p0[1] * s * gg; y[2] = p1[0] * s * gg; y[3] = p1[1] * s * gg;
  y[4] = p2[0] * s * gg; y[5] = p2[1] * s * gg; y[6] = p3[0] * s * gg; y[7] = p3[1] * s * gg;
  store8<F32>(out, t, y);
}

// Threads by the row's length: enough that it stays in registers, no more than
// it has work for. 8000 rows (bf16, per token, with dequantization) of 512 /
// 4096 / 7168 elements take 11.0 / 73 / 132 us with 64 threads, 17.6 / 50.8 /
// 90.8 us with 256, 28.9 / 55.9 / 84.3 us with 512; one row of 7168 24 / 8.1 /
// 6.6 us.
template <bool XF, bool RF>
void norm_launch(const NormArgs& a, hipStream_t s) {
  const unsigned gx = (unsigned)(a.M < 65536 ? a.M : 65536);
  const dim3 grid(gx, (unsigned)((a.M + gx - 1) / gx));
  if (a.K <= 1024) k_add_rmsnorm_quant<XF, RF, 64, 2><<<grid, dim3(64), 0, s>>>(a);
  else if (a.K <= 4096) k_add_rmsnorm_quant<XF, RF, 256, 2><<<grid, dim3(256), 0, s>>>(a);
  else k_add_rmsnorm_quant<XF, RF, 512, 2><<<grid, dim3(512), 0, s>>>(a);
}

}  // namespace

hipError_t launch_add_rmsnorm_quant(const NormArgs& a, hipStream_t s) {
  // Without a residual z is x itself, kept in x's type.
  const bool rf = a.residual != nullptr ? a.res_f32 : a.x_f32;
  if (a.x_f32) rf ? norm_launch<true, true>(a, s) : norm_launch<true, false>(a, s);
  else rf ? norm_launch<false, true>(a, s) : norm_launch<false, false>(a, s);
  return hipGetLastError();
}

hipError_t launch_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t M, int64_t K, const float* g,
                             const float* row_g, void* out, bool f32_out, hipStream_t s) {
  const int64_t n8 = M * (K / 8);
  const int64_t wg = (n8 + 255) / 256, gx = wg < (1 << 20) ? wg : (1 << 20);
  const dim3 grid((unsigned)gx, (unsigned)((wg + gx - 1) / gx));
  const uint32_t* c = reinterpret_cast<const uint32_t*>(codes);
  if (f32_out) k_dequantize<true><<<grid, dim3(256), 0, s>>>(c, scales, n8, K / 8, g, row_g, out);
  else k_dequantize<false><<<grid, dim3(256), 0, s>>>(c, scales, n8, K / 8, g, row_g, out);
  return hipGetLastError();
}

}  // namespace nvfp4
