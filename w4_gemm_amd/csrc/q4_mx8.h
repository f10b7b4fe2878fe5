// q4_mx8.h -- the 8-bit block formats of saved activations (Q4_MXINT8,
// Q4_MXFP8): blocks of 32 values along a row share one power-of-two scale
// 2^(b - 127), stored as the byte b.
//
//   b     the least with max|x| <= top * 2^(b - 127), at least 16 (2^-111);
//         top = 127 (integers) or 448 (E4M3)
//   code  x / 2^(b - 127) rounded to nearest, ties to even: a two's
//         complement byte, or an E4M3 byte
//
// The scale is the least that does not clip, so a block's largest value
// lands in (top/2, top] and is stored with an error of at most half a code.
// Scaling by a power of two is exact, an integer of up to 7 bits or an E4M3
// value (4 significant bits) times a power of two is exact in bf16, and from
// b = 16 on every value is a normal bf16 number: the products of the weight
// gradient therefore start from exactly what was stored.
//
// A block that holds an infinity or a NaN has b = 255 and reads back as NaN
// throughout (E4M3 codes 0x7F; integers 0 times 2^128 = inf), so that an
// overflow of the forward pass still shows in its gradients.  Where a code's
// value would reach 2^128 (|x| near the largest bf16) the next lower code is
// stored.
#pragma once

#include "q4_device.h"
#include "q4_mma.h"

namespace q4 {

constexpr int kMxFp8 = 5, kMxInt8 = 6;   // q4_format values
constexpr uint32_t kMxMinScale = 16;

// Largest |x| of eight bf16 (as bits; infinities and NaN compare above every
// finite value) joined with a.
__device__ __forceinline__ uint32_t mx8_absmax(const uint4& v, uint32_t a) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    a = max(a, w[i] & 0x7FFFu);
    a = max(a, (w[i] >> 16) & 0x7FFFu);
  }
  return a;
}

// Scale byte of a block whose largest |x| has the bf16 bits `amax`.  127 is
// 2^6 (1 + 126/128) and 448 is 2^8 (1 + 96/128), so the comparison with top
// is one of the seven mantissa bits.
template <int FMT>
__device__ __forceinline__ uint32_t mx8_scale(uint32_t amax) {
  if (amax >= 0x7F80u) return 255u;
  constexpr int top_exp = FMT == kMxInt8 ? 6 : 8, top_mant = FMT == kMxInt8 ? 126 : 96;
  const int b = (int)(amax >> 7) - top_exp + ((int)(amax & 0x7Fu) > top_mant ? 1 : 0);
  return (uint32_t)max(b, (int)kMxMinScale);
}

// Eight values -> eight code bytes in order.
template <int FMT>
__device__ __forceinline__ uint2 mx8_encode8(const uint4& v, uint32_t b) {
  if (b == 255u) return FMT == kMxInt8 ? make_uint2(0u, 0u) : make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
  const float r = u2f((254u - b) << 23);   // 2^(127 - b), exact
  const float x[8] = {bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y),
                      bf16_lo(v.z), bf16_hi(v.z), bf16_lo(v.w), bf16_hi(v.w)};
  uint32_t o[2];
  if constexpr (FMT == kMxInt8) {
    const float lim = b >= 249u ? 63.0f : 127.0f;   // 64 * 2^122 is 2^128
    uint32_t c[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float y = fminf(fmaxf(x[i] * r, -lim), lim);
      c[i] = f2u(y + 12582912.0f);         // 1.5 * 2^23: the low byte is rne(y)
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t p = __builtin_amdgcn_perm(c[4 * h + 1], c[4 * h], 0x0C0C0400u);
      const uint32_t q = __builtin_amdgcn_perm(c[4 * h + 3], c[4 * h + 2], 0x04000C0Cu);
      o[h] = p | q;
    }
  } else {
    const float lim = b >= 247u ? 240.0f : 448.0f;  // 256 * 2^120 is 2^128
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = fminf(fmaxf(x[4 * h + i] * r, -lim), lim);
      uint32_t w = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
      o[h] = __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], w, true);
    }
  }
  return make_uint2(o[0], o[1]);
}

// Eight code bytes -> the eight values they stand for.
template <int FMT>
__device__ __forceinline__ void mx8_decode8(uint2 c, uint32_t b, float (&x)[8]) {
  const float s = u2f(b << 23);            // b = 255: +inf, 0 * inf = NaN
  const uint32_t w[2] = {c.x, c.y};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if constexpr (FMT == kMxInt8) {
#pragma unroll
      for (int i = 0; i < 4; ++i) x[4 * h + i] = (float)(int)(int8_t)(w[h] >> (8 * i)) * s;
    } else {
      const f32x2_t lo = __builtin_amdgcn_cvt_pk_f32_fp8(w[h], false);
      const f32x2_t hi = __builtin_amdgcn_cvt_pk_f32_fp8(w[h], true);
      x[4 * h] = lo[0] * s;
      x[4 * h + 1] = lo[1] * s;
      x[4 * h + 2] = hi[0] * s;
      x[4 * h + 3] = hi[1] * s;
    }
  }
}

}  // namespace q4
