// Codes of a row from its absolute maximum, shared by the row quantizer and
// the kernels that quantize a few tokens on the way, so that both produce the
// same codes and scales.
//
// Division: the codes need rne(fl32(x/s)) exactly.  Instead of a full IEEE
// division per element the kernel computes r = fl32(1/s) once per row and
//   q0 = fl32(x*r), e = fma(-q0, s, x), q = fma(e, r, q0)
// (one Markstein correction step).  Rows with s < 2^-100 first scale x and s
// by 2^100, which is exact and keeps 1/s finite.  An exhaustive host check
// over every finite bf16 (x, amax) pair with |x| <= amax shows the resulting
// codes equal those of the correctly rounded quotient.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace w8a8 {
namespace {

typedef unsigned short ushort2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, off, 64));
  return v;
}

__device__ __forceinline__ uint32_t absmax_bits(uint32_t acc, uint32_t w) {
  // packed max of the two 15-bit magnitudes held in one 32-bit word
  ushort2_t a = __builtin_bit_cast(ushort2_t, acc);
  ushort2_t b = __builtin_bit_cast(ushort2_t, w & 0x7fff7fffu);
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(a, b));
}

__device__ __forceinline__ int code(float x, float s, float r) {
  float q0 = x * r;
  float e = __builtin_fmaf(-q0, s, x);
  float q = __builtin_fmaf(e, r, q0);
  q = __builtin_rintf(q);
  q = __builtin_fminf(__builtin_fmaxf(q, -127.0f), 127.0f);
  return (int)q;
}

// fp8 variant: the quotient fl32(x/s) itself, for the e4m3 conversion; the
// clamp only guards the last fp32 rounding of |x/s| <= 448.  The correction
// step turns x = -0 into +0 (-0 + +0 = +0), and e4m3 keeps the sign of zero,
// so the sign is copied back from x (s > 0: x/s has the sign of x).
__device__ __forceinline__ float quot(float x, float s, float r) {
  const float q0 = x * r;
  const float e = __builtin_fmaf(-q0, s, x);
  const float q = __builtin_fminf(__builtin_fmaxf(__builtin_fmaf(e, r, q0), -448.0f), 448.0f);
  return __builtin_copysignf(q, x);
}

__device__ __forceinline__ uint32_t pack4(int a, int b, int c, int d) {
  return (uint32_t)(a & 0xff) | ((uint32_t)(b & 0xff) << 8) | ((uint32_t)(c & 0xff) << 16) |
         ((uint32_t)d << 24);
}

// 8 bf16 (one 16-byte chunk) -> 8 codes (8 bytes); xs scales x (1 or 2^100).
template <bool F8>
__device__ __forceinline__ u32x2 quant_chunk(u32x4 v, float xs, float s, float r) {
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
  if constexpr (F8) {
    float f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = quot(__uint_as_float(w[i] << 16) * xs, s, r);
      f[2 * i + 1] = quot(__uint_as_float(w[i] & 0xffff0000u) * xs, s, r);
    }
    int lo = __builtin_amdgcn_cvt_pk_fp8_f32(f[0], f[1], 0, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(f[2], f[3], lo, true);
    int hi = __builtin_amdgcn_cvt_pk_fp8_f32(f[4], f[5], 0, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(f[6], f[7], hi, true);
    return u32x2{(uint32_t)lo, (uint32_t)hi};
  }
  int c[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    c[2 * i] = code(__uint_as_float(w[i] << 16) * xs, s, r);
    c[2 * i + 1] = code(__uint_as_float(w[i] & 0xffff0000u) * xs, s, r);
  }
  return u32x2{pack4(c[0], c[1], c[2], c[3]), pack4(c[4], c[5], c[6], c[7])};
}

struct RowScale {
  float s;   // stored scale fl32(amax/127) (fp8: /448), 0 for a zero row
  float ss;  // scale used in the division (s, or s*2^100)
  float xs;  // factor applied to x (1 or 2^100)
  float r;   // fl32(1/ss)
};

template <bool F8>
__device__ __forceinline__ RowScale row_scale(uint32_t amax_bits) {
  RowScale rs;
  float amax = __uint_as_float(amax_bits << 16);
  rs.s = amax / (F8 ? 448.0f : 127.0f);  // correctly rounded (IEEE division)
  rs.xs = 1.0f;
  rs.ss = rs.s;
  if (rs.s < 0x1p-100f) {
    rs.xs = 0x1p100f;
    rs.ss = rs.s * 0x1p100f;
  }
  rs.r = 1.0f / rs.ss;   // correctly rounded
  return rs;
}

}  // namespace
}  // namespace w8a8
