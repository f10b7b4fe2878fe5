// q4_piece.h -- 32 consecutive columns of one row of a matrix, whatever it is
// stored in, as 32 bf16: the operand whose rows the gradient products sum over
// (the quantized weight of dA = dC W', the saved activation of dW = dC^T A).
// Loading and converting are apart, so that a kernel can keep the loads of a
// later stage in flight.
//
// Every conversion is exact except INT4's (with or without a zero point): an
// integer of 4 bits times an fp16 scale has up to 15 significant bits and is
// rounded once to bf16, as the forward W4A16 products round it.  NVFP4's
// tensor scale is left out (code times E4M3 has at most 6 significant bits);
// the products apply it to their fp32 sums.
#pragma once

#include "q4_layout.h"
#include "q4_mma.h"
#include "q4_mx8.h"

namespace q4 {

constexpr int kBf16Piece = 7;   // beside the q4_format values 0..2, 4 (weights) and 5, 6 (saved activations)

struct PieceSrc {
  const uint8_t* data;     // codes, or the bf16 matrix
  const uint8_t* scales;
  int64_t cols;            // K
  int64_t ld;              // bf16: elements per row
};

template <int KIND>
struct Piece {
  static constexpr int kWords = KIND == kBf16Piece ? 4 : (KIND == kMxFp8 || KIND == kMxInt8) ? 2 : 1;
  u32x4_t q[kWords];
  uint32_t s;
};

// Row r, columns c .. c + 31 (c % 32 == 0, c < K; the K of a bf16 matrix may end
// inside the piece, at a multiple of 8: the columns past it repeat others).
template <int KIND, int LAYOUT>
__device__ __forceinline__ void piece_load(Piece<KIND>& p, const PieceSrc& src, int64_t r, int64_t c) {
  constexpr int W = Piece<KIND>::kWords;
  if constexpr (KIND == kBf16Piece) {
    const uint16_t* row = reinterpret_cast<const uint16_t*>(src.data) + r * src.ld + c;
#pragma unroll
    for (int i = 0; i < W; ++i)      // (always W loads: the kernels count them)
      p.q[i] = *reinterpret_cast<const u32x4_t*>(row + min((int64_t)8 * i, src.cols - 8 - c));
    p.s = 0u;
  } else if constexpr (KIND == kMxFp8 || KIND == kMxInt8) {
    const uint8_t* row = src.data + r * src.cols + c;
    p.q[0] = *reinterpret_cast<const u32x4_t*>(row);
    p.q[1] = *reinterpret_cast<const u32x4_t*>(row + 16);
    p.s = src.scales[(r * src.cols + c) >> 5];
  } else {
    p.q[0] = *reinterpret_cast<const u32x4_t*>(src.data + code_off8<LAYOUT>(r, c, src.cols));
    const int64_t so = scale_off<KIND, LAYOUT>(r, c, src.cols);
    if constexpr (KIND == 1) p.s = src.scales[so];
    else if constexpr (KIND == 4) p.s = reinterpret_cast<const uint32_t*>(src.scales)[so];
    else if constexpr (KIND == 0) p.s = reinterpret_cast<const uint16_t*>(src.scales)[so];
    else p.s = *reinterpret_cast<const uint16_t*>(src.scales + so);
  }
}

// A row without values: zeros, whatever was loaded in its place.
template <int KIND>
__device__ __forceinline__ void piece_clear(Piece<KIND>& p, bool clear) {
#pragma unroll
  for (int i = 0; i < Piece<KIND>::kWords; ++i) p.q[i] = clear ? u32x4_t{0u, 0u, 0u, 0u} : p.q[i];
  p.s = clear ? 0u : p.s;
}

// The piece as four times eight bf16 (out[i] holds columns 8i .. 8i + 7).
template <int KIND>
__device__ __forceinline__ void piece_convert(const Piece<KIND>& p, u32x4_t (&out)[4]) {
  if constexpr (KIND == kBf16Piece) {
#pragma unroll
    for (int i = 0; i < 4; ++i) out[i] = p.q[i];
  } else if constexpr (KIND == kMxFp8) {
    const float s = e8m0_value(p.s);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t w = p.q[i >> 1][2 * (i & 1) + h];
        out[i][2 * h] = as_u32(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, s, false));
        out[i][2 * h + 1] = as_u32(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, s, true));
      }
  } else if constexpr (KIND == kMxInt8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float x[8];
      mx8_decode8<KIND>(make_uint2(p.q[i >> 1][2 * (i & 1)], p.q[i >> 1][2 * (i & 1) + 1]), p.s, x);
#pragma unroll
      for (int j = 0; j < 4; ++j) out[i][j] = pk_bf16(x[2 * j], x[2 * j + 1]);
    }
  } else if constexpr (KIND == 1) {
    const float s = e8m0_value(p.s);
#pragma unroll
    for (int i = 0; i < 4; ++i) out[i] = __builtin_bit_cast(u32x4_t, dq8_e2m1(p.q[0][i], s));
  } else if constexpr (KIND == 2) {
    const float s0 = e4m3_value(p.s & 0xFFu), s1 = e4m3_value(p.s >> 8);
#pragma unroll
    for (int i = 0; i < 4; ++i) out[i] = __builtin_bit_cast(u32x4_t, dq8_e2m1_mul(p.q[0][i], i < 2 ? s0 : s1));
  } else if constexpr (KIND == 0) {
    const float s = fp16_value(p.s);
#pragma unroll
    for (int i = 0; i < 4; ++i) out[i] = __builtin_bit_cast(u32x4_t, dq8_int4(p.q[0][i], s));
  } else {
    float s, off;
    int4zp_scale(p.s, s, off);
#pragma unroll
    for (int i = 0; i < 4; ++i) out[i] = __builtin_bit_cast(u32x4_t, dq8_int4_off(p.q[0][i], s, off));
  }
}

}  // namespace q4
