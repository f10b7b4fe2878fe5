// q4_row8.h -- what the kernels that write a row in 8 bits with one scale
// share: rows spread over the lanes of 1..16 waves, and eight codes packed
// from eight fp32 values and the row's factor.
//
// Q4_INT8_ROW (include/q4.h): scale = a / 127, code = the integer nearest to
// the exact product x * f, ties to even, with a = max(amax, 1e-12) and
// f = fp32(127 / a).  |x| <= a, so |x f| <= 127 (1 + 2^-24): no clamp.
#pragma once

#include "q4_device.h"
#include "q4_wave.h"

namespace q4 {

constexpr int kRowInt8 = 0;   // output kinds of the row kernels
constexpr int kRowE4m3 = 1;

// Largest value that a code of the kind stands for.
template <int KIND>
constexpr float kRowTop = KIND == kRowInt8 ? 127.0f : 448.0f;

// Eight integer codes: x f + 1.5 * 2^23 in one fma rounds the exact product to
// the nearest integer (ties to even) and leaves its two's complement in the low
// byte; three byte permutes gather four of them.
__device__ __forceinline__ uint2 int8_pack8(const float (&x)[8], float f) {
  uint32_t u[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) u[j] = f2u(__builtin_fmaf(x[j], f, 12582912.0f));
  uint2 p;
  p.x = __builtin_amdgcn_perm(u[1], u[0], 0x0c0c0400u) | __builtin_amdgcn_perm(u[3], u[2], 0x04000c0cu);
  p.y = __builtin_amdgcn_perm(u[5], u[4], 0x0c0c0400u) | __builtin_amdgcn_perm(u[7], u[6], 0x04000c0cu);
  return p;
}

// Eight E4M3 codes of x f, |x f| <= 448 (1 + 2^-22), which rounds to 448 (the
// conversion rounds to nearest, ties to the even code, and keeps the sign).
__device__ __forceinline__ uint2 e4m3_pack8(const float (&x)[8], float f) {
  uint2 p;
  p.x = __builtin_amdgcn_cvt_pk_fp8_f32(x[0] * f, x[1] * f, 0, false);
  p.x = __builtin_amdgcn_cvt_pk_fp8_f32(x[2] * f, x[3] * f, p.x, true);
  p.y = __builtin_amdgcn_cvt_pk_fp8_f32(x[4] * f, x[5] * f, 0, false);
  p.y = __builtin_amdgcn_cvt_pk_fp8_f32(x[6] * f, x[7] * f, p.y, true);
  return p;
}

// 16 bytes read or written with (PAST) or without the hint that they are not used
// again: streams longer than the caches then do not turn over what they hold.
template <bool PAST>
__device__ __forceinline__ uint4 load16(const void* p) {
  typedef uint32_t quad_t __attribute__((ext_vector_type(4)));
  const quad_t* q = static_cast<const quad_t*>(p);
  return __builtin_bit_cast(uint4, PAST ? __builtin_nontemporal_load(q) : *q);
}
template <bool PAST>
__device__ __forceinline__ void store16(void* p, uint4 v) {
  typedef uint32_t quad_t __attribute__((ext_vector_type(4)));
  quad_t* q = static_cast<quad_t*>(p);
  if (PAST) __builtin_nontemporal_store(__builtin_bit_cast(quad_t, v), q);
  else *q = __builtin_bit_cast(quad_t, v);
}

__device__ __forceinline__ void unpack_bf16x8(const uint4& v, float (&x)[8]) {
  x[0] = bf16_lo(v.x); x[1] = bf16_hi(v.x);
  x[2] = bf16_lo(v.y); x[3] = bf16_hi(v.y);
  x[4] = bf16_lo(v.z); x[5] = bf16_hi(v.z);
  x[6] = bf16_lo(v.w); x[7] = bf16_hi(v.w);
}

// Magnitude bits of the largest of |x|: fp32 magnitudes order as integers, with
// infinity and then NaN above every number, so neither is passed over.
__device__ __forceinline__ uint32_t max_bits8(const float (&x)[8], uint32_t m) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t b = f2u(x[j]) & 0x7FFFFFFFu;
    m = b > m ? b : m;
  }
  return m;
}

}  // namespace q4
