// ssm_delta.cuh -- device helpers of the gated delta rule: the gates, warp
// MMAs and their fragment loads, and the two-piece fp16 form of fp32 operands.
#pragma once

#include <cuda_fp16.h>

#include "ssm_chain.cuh"
#include "ssm_delta_internal.h"
#include "ssm_device.cuh"

namespace ssm {

// Delta of one token: softplus with the library's cut, in fp32 functions whose
// error is a few units in the last place (one call per token and head).
__device__ __forceinline__ float delta_step_size(float raw, int softplus) {
  return (softplus && raw <= kSoftplusCut) ? log1pf(expf(raw)) : raw;
}
__device__ __forceinline__ float delta_beta(float raw, int sigmoid) {
  return sigmoid ? 1.f / (1.f + expf(-raw)) : raw;
}

__device__ __forceinline__ float delta_beta_floor(float beta) {
  return fabsf(beta) < kBetaFloor ? copysignf(kBetaFloor, beta) : beta;
}

// ------------------------------------------------------ fragments and MMAs --
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void stsm4t(uint32_t addr, const uint32_t (&r)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
               : "memory");
}
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
  asm(  // not volatile: independent products may be interleaved
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Byte offset of 16-byte unit `c` of row `row` in a tile with RB-byte rows: the
// unit's low three bits are xored with the row's, so that the eight rows of an
// ldmatrix at one column lie in eight different bank groups.
template <int RB>
__device__ __forceinline__ uint32_t swz(int row, int c) {
  return (uint32_t)(row * RB + ((c ^ (row & 7)) << 4));
}

// Byte offset of 16-byte unit `u` of token `row` in a k or q tile: blocks of 64
// columns, 128-byte rows.
__device__ __forceinline__ uint32_t kq_at(int row, int u) {
  return (uint32_t)((u >> 3) * (kDeltaChunk * 128)) + swz<128>(row, u & 7);
}
// Byte offset inside a 16 x 16 block of a triangular tile (kDeltaTri).
__device__ __forceinline__ uint32_t tri_at(int row, int half) {
  return (uint32_t)(((row >> 3) * 2 + half) * 128 + (row & 7) * 16);
}
// Byte offset in a column tile (16 columns of v, 32-byte rows): the two halves
// of a row are swapped in rows 4 .. 7 of every eight.
__device__ __forceinline__ uint32_t col_at(int row, int half) {
  return (uint32_t)(row * 32 + ((half ^ ((row >> 2) & 1)) << 4));
}

// ------------------------------------- fp32 operands as two pieces of fp16 --
// x s = hi + lo with hi, lo fp16 and s a power of two that brings the largest
// magnitude of the row to [2^14, 2^15): the two pieces carry 22 bits of every
// element within 2^16 of the largest, and smaller ones to 2^-40 of the largest
// (what a row's scale must not hide goes token by token, ssm_delta_tc.cu), so
// products keep fp32's accuracy at two MMAs (three where both operands have two
// pieces; the dropped lo lo is 2^-24 of the product).
// bf16 operands (k, q) are one exact fp16 piece under a row scale of their own.
struct RowScale {
  float s, inv;
};
// s = 2^(14 - e) for a largest magnitude of biased exponent e
__device__ __forceinline__ RowScale row_scale(uint32_t e) {
  constexpr uint32_t top = 14;
  e = e < 1u + top ? 1u + top : (e > 253u ? 253u : e);
  RowScale r;
  r.s = __uint_as_float((254u + top - e) << 23);
  r.inv = __uint_as_float((e - top) << 23);
  return r;
}
__device__ __forceinline__ uint32_t exponent_of(float m) { return __float_as_uint(m) >> 23; }
// The larger one, or NaN where either is one.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ bool not_finite(float m) { return (__float_as_uint(m) & 0x7FFFFFFFu) >= 0x7F800000u; }
// Largest magnitude of fragment rows g (m0) and g + 8 (m1), over the quad; NaN where
// one of them is.
template <int T>
__device__ __forceinline__ void row_max(const float (&x)[T][4], float& m0, float& m1) {
  m0 = m1 = 0.f;
#pragma unroll
  for (int j = 0; j < T; ++j) {
    m0 = max_nan(m0, max_nan(fabsf(x[j][0]), fabsf(x[j][1])));
    m1 = max_nan(m1, max_nan(fabsf(x[j][2]), fabsf(x[j][3])));
  }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    m0 = max_nan(m0, __shfl_xor_sync(0xffffffffu, m0, o));
    m1 = max_nan(m1, __shfl_xor_sync(0xffffffffu, m1, o));
  }
}
// The transpose of the warp's 8 x 8 matrix of 16-bit values.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

__device__ __forceinline__ uint32_t h2_bits(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
// The pieces of two values that are in range already.
__device__ __forceinline__ void pieces2(float x, float y, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(x, y);
  const float2 f = __half22float2(h);
  const float2 d = fma2(f, make_float2(-1.f, -1.f), make_float2(x, y));
  hi = h2_bits(h);
  lo = h2_bits(__floats2half2_rn(d.x, d.y));
}
__device__ __forceinline__ void split2(float x, float y, float s, uint32_t& hi, uint32_t& lo) {
  const float2 v = mul2(make_float2(x, y), make_float2(s, s));
  pieces2(v.x, v.y, hi, lo);
}

}  // namespace ssm
