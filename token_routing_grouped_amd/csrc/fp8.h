// Device helpers of the 8-bit operators: e4m3 values with power-of-two scales.
//
// Scale of a block: the least 2^k with max|v| <= 448 * 2^k over the block's finite values,
// at least 2^-126. 448 = 1.75 * 2^8, so for max|v| = m * 2^e (1 <= m < 2) k is e - 8 where
// m <= 1.75 and e - 7 above: adding 0x1fffff to the fp32 bits carries into the exponent
// exactly when the mantissa exceeds 0.75. Multiplying by 2^-k is exact, so each value is
// rounded once, by the conversion to e4m3 (to nearest, ties to even), and never exceeds 448.
#pragma once
#include "common.h"

namespace moe {

constexpr int kQB = 128;  // values per block

// bits of |v| for a finite v, else 0 (their order is that of the values)
__device__ __forceinline__ uint32_t finite_abs_bits(float v) {
  const uint32_t b = __float_as_uint(v) & 0x7fffffffu;
  return b < 0x7f800000u ? b : 0u;
}
// biased exponent (1..247) of the scale of a block whose largest finite |v| has these bits
__device__ __forceinline__ uint32_t scale_exponent(uint32_t amax_bits) {
  const int e = (int)((amax_bits + 0x1fffffu) >> 23) - 8;
  return (uint32_t)(e > 1 ? e : 1);
}
__device__ __forceinline__ float exponent_value(uint32_t e) { return __uint_as_float(e << 23); }
// a scale as it was passed in, any of its type's values: byte 0 is 2^-127, 255 NaN
__device__ __forceinline__ float scale_value(const void *p, int e8m0, int64_t i) {
  if (!e8m0) return ((const float *)p)[i];
  const uint32_t b = ((const uint8_t *)p)[i];
  return __uint_as_float(b - 1 < 254 ? b << 23 : b ? 0x7fc00000u : 0x400000u);
}
__device__ __forceinline__ float exponent_inverse(uint32_t e) {
  return __uint_as_float((254u - e) << 23);
}
// v * inv for the conversion: what is not finite becomes NaN (e4m3 has no infinity)
__device__ __forceinline__ float to_q(float v, float inv) {
  const bool fin = (__float_as_uint(v) & 0x7fffffffu) < 0x7f800000u;
  return fin ? v * inv : __uint_as_float(0x7fc00000u);
}
// four values on e4m3, the first in bits 0-7
__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float d) {
  int v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true);
}

// biased exponent (15..254) of the largest finite |y| of a row's columns that share a scale:
// y is kept as fp16 of y 2^(141 - e), at most 2^15
__device__ __forceinline__ uint32_t y_exponent(uint32_t amax_bits) {
  const uint32_t e = amax_bits >> 23;
  return e < 15u ? 15u : e;
}
// maximum over each row of 16 lanes (DPP row_ror 8, 4, 2, 1); all lanes active
__device__ __forceinline__ uint32_t row16_max(uint32_t v) {
#define MOE_ROR(N)                                                                            \
  {                                                                                           \
    const uint32_t o_ =                                                                       \
        (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x120 + (N), 0xf, 0xf, false);       \
    v = v > o_ ? v : o_;                                                                      \
  }
  MOE_ROR(8) MOE_ROR(4) MOE_ROR(2) MOE_ROR(1)
#undef MOE_ROR
  return v;
}

// eight consecutive elements as fp32, and back
template <typename T>
struct Vec8;
template <>
struct Vec8<uint16_t> {  // bf16
  struct Raw { u32x4 v; };
  __device__ static Raw load(const uint16_t *p) { return {*(const u32x4 *)p}; }
  __device__ static Raw zero() { return {u32x4{0, 0, 0, 0}}; }
  __device__ static void get(const Raw &r, float *f) {
#pragma unroll
    for (int i = 0; i < 4; i++) {
      f[2 * i] = bf16_to_f32((uint16_t)(r.v[i] & 0xffffu));
      f[2 * i + 1] = bf16_to_f32((uint16_t)(r.v[i] >> 16));
    }
  }
  __device__ static Raw pack(const float *f) {
    return {u32x4{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                  pack_bf16x2(f[6], f[7])}};
  }
  __device__ static void store(uint16_t *p, const Raw &r) { *(u32x4 *)p = r.v; }
};
template <>
struct Vec8<float> {
  struct Raw { u32x4 a, b; };
  __device__ static Raw load(const float *p) {
    return {*(const u32x4 *)p, *(const u32x4 *)(p + 4)};
  }
  __device__ static Raw zero() { return {u32x4{0, 0, 0, 0}, u32x4{0, 0, 0, 0}}; }
  __device__ static void get(const Raw &r, float *f) {
#pragma unroll
    for (int i = 0; i < 4; i++) {
      f[i] = __uint_as_float(r.a[i]);
      f[4 + i] = __uint_as_float(r.b[i]);
    }
  }
  __device__ static Raw pack(const float *f) {
    Raw r;
#pragma unroll
    for (int i = 0; i < 4; i++) {
      r.a[i] = __float_as_uint(f[i]);
      r.b[i] = __float_as_uint(f[4 + i]);
    }
    return r;
  }
  __device__ static void store(float *p, const Raw &r) {
    *(u32x4 *)p = r.a;
    *(u32x4 *)(p + 4) = r.b;
  }
};

__device__ __forceinline__ void store_scale(void *scale, int e8m0, int64_t i, uint32_t e) {
  if (e8m0)
    ((uint8_t *)scale)[i] = (uint8_t)e;
  else
    ((float *)scale)[i] = exponent_value(e);
}

// The chunk of eight values of a lane whose row of 16 lanes holds one block (lanes past the
// end of the row hold zeros): the block's scale exponent and the lane's eight e4m3 bytes.
__device__ __forceinline__ uint32_t quantize8(const float *f, u32x2 *q) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const uint32_t b = finite_abs_bits(f[i]);
    m = m > b ? m : b;
  }
  const uint32_t e = scale_exponent(row16_max(m));
  const float inv = exponent_inverse(e);
  float g[8];
#pragma unroll
  for (int i = 0; i < 8; i++) g[i] = to_q(f[i], inv);
  *q = u32x2{pack_e4m3(g[0], g[1], g[2], g[3]), pack_e4m3(g[4], g[5], g[6], g[7])};
  return e;
}

}  // namespace moe
