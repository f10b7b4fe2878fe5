// q4_piece.h -- a thread's 32 values of a stage of a gradient product's second
// operand, whatever it is stored in, as 32 bf16: the operand whose rows the
// products sum over (the quantized weight of dA = dC W', the saved activation
// of dW = dC^T A).  Loading and converting are apart, so that a kernel can keep
// the loads of a later stage in flight.
//
// A wave holds 8 rows x 256 columns (activations) or 16 rows x 128 (weights).
// Which columns of its row a thread takes is chosen for the vector cache, which
// serves four neighbouring lanes at a time: 16 cycles for a 16-byte load whose
// lanes are consecutive, 32 where they are 64 bytes apart, 64 where each lane
// is on a row of its own (measured).  So:
//   4-bit weights  one load of 32 columns; lane l row l % 16, columns
//                  32 (l / 16): in the tiled layout one contiguous kilobyte.
//                  (Row-major it is the slow case, but there are few loads and
//                  they run under the products: dA 4096 x 8192 x 8192 MXFP4
//                  405 us, tiled 410; 16 rows 24.3 and 24.5.)
//   8-bit          two loads of 16 columns, 16 b + 128 h for lane b of 8
//   bf16           four loads of 8 columns, 8 b + 64 i for lane b of 8
//
// Every conversion is exact except INT4's (with or without a zero point): an
// integer of 4 bits times an fp16 scale has up to 15 significant bits and is
// rounded once to bf16, as the forward W4A16 and grouped products round it.  An
// output is then off by 2.4e-3 (2-norms) in place of the 1.7e-3 of its own
// rounding to bf16, against 1e-1 by which INT4 itself is off; the weight's
// second bf16 term would take every product twice.  NVFP4's tensor scale is
// left out (code times E4M3 has at most 6 significant bits); the products apply
// it to their fp32 sums.
#pragma once

#include "q4_layout.h"
#include "q4_mma.h"
#include "q4_mx8.h"

#include <type_traits>

namespace q4 {

constexpr int kBf16Piece = 7;   // beside the q4_format values 0..2, 4 (weights) and 5, 6 (saved activations)

constexpr bool piece_is_mx8(int kind) { return kind == kMxFp8 || kind == kMxInt8; }
constexpr bool piece_is_w4(int kind) { return kind != kBf16Piece && !piece_is_mx8(kind); }

template <int KIND>
struct Piece {
  static constexpr int kWords = KIND == kBf16Piece ? 4 : piece_is_mx8(KIND) ? 2 : 1;   // 16-byte loads
  static constexpr int kScales = KIND == kBf16Piece ? 0 : piece_is_mx8(KIND) ? 2 : 1;
  static constexpr int kLoads = kWords + kScales;                                      // load instructions
  u32x4_t q[kWords];
  // (bytes as loaded: widened any earlier, the widening waits for the load)
  std::conditional_t<KIND == 1 || piece_is_mx8(KIND), uint8_t, uint32_t> s[kScales ? kScales : 1];
};

// Where thread `tid` of a workgroup has its piece: row of the stage, and the
// 16-byte chunk of a 512-byte bf16 row for its i-th eight values.
template <int KIND>
__device__ __forceinline__ int piece_row(int tid) {
  return piece_is_w4(KIND) ? 16 * (tid >> 7) + (tid & 15) : tid >> 3;
}
template <int KIND>
__device__ __forceinline__ int piece_chunk(int tid, int i) {
  if constexpr (KIND == kBf16Piece) return (tid & 7) + 8 * i;
  else if constexpr (piece_is_mx8(KIND)) return 2 * (tid & 7) + 16 * (i >> 1) + (i & 1);
  else return 4 * (4 * ((tid >> 6) & 1) + ((tid & 63) >> 4)) + i;
}

// Bytes of a scale, and columns that share one.
template <int KIND>
struct PieceScale {
  static constexpr int kBytes = KIND == 4 ? 4 : KIND == 0 ? 2 : 1;
  static constexpr int kCols = (KIND == 0 || KIND == 4) ? 128 : KIND == 2 ? 16 : 32;
};

typedef decltype(__builtin_amdgcn_make_buffer_rsrc((void*)nullptr, 0, 0, 0)) rsrc_t;

// First columns of a thread's loads for the block of columns at k0, kept inside
// the K columns (a load past them repeats others, whose results are not used).
template <int KIND>
struct PieceCols {
  int c[Piece<KIND>::kWords];
};
template <int KIND>
__device__ __forceinline__ PieceCols<KIND> piece_cols(int tid, int k0, int K) {
  constexpr int W = Piece<KIND>::kWords, width = 32 / W;
  PieceCols<KIND> o;
#pragma unroll
  for (int i = 0; i < W; ++i) o.c[i] = min(k0 + 8 * piece_chunk<KIND>(tid, i * (4 / W)), K - width);
  return o;
}

// Byte offsets of a thread's loads in the buffers of a stage (which start a
// multiple of 16 rows into the matrix).  ld: elements per row of a bf16 matrix.
template <int KIND>
struct PieceAt {
  int q[Piece<KIND>::kWords], s[Piece<KIND>::kScales ? Piece<KIND>::kScales : 1];
};
template <int KIND, int LAYOUT>
__device__ __forceinline__ PieceAt<KIND> piece_at(int r, const PieceCols<KIND>& c, int K, int ld) {
  PieceAt<KIND> o{};
  if constexpr (piece_is_w4(KIND)) {
    o.q[0] = (int)code_off8<LAYOUT>(r, c.c[0], K);
    o.s[0] = (int)scale_off<KIND, LAYOUT>(r, c.c[0], K) * PieceScale<KIND>::kBytes;
  } else {
#pragma unroll
    for (int i = 0; i < Piece<KIND>::kWords; ++i) {
      if constexpr (KIND == kBf16Piece) {
        o.q[i] = (r * ld + c.c[i]) * 2;
      } else {
        o.q[i] = r * K + c.c[i];
        o.s[i] = o.q[i] >> 5;
      }
    }
  }
  return o;
}

template <int KIND>
__device__ __forceinline__ void piece_load(Piece<KIND>& p, rsrc_t data, rsrc_t scales, const PieceAt<KIND>& at) {
#pragma unroll
  for (int i = 0; i < Piece<KIND>::kWords; ++i) p.q[i] = __builtin_amdgcn_raw_buffer_load_b128(data, at.q[i], 0, 0);
#pragma unroll
  for (int i = 0; i < Piece<KIND>::kScales; ++i) {
    if constexpr (KIND == 4) p.s[i] = __builtin_amdgcn_raw_buffer_load_b32(scales, at.s[i], 0, 0);
    else if constexpr (KIND == 0 || KIND == 2) p.s[i] = __builtin_amdgcn_raw_buffer_load_b16(scales, at.s[i], 0, 0);
    else p.s[i] = __builtin_amdgcn_raw_buffer_load_b8(scales, at.s[i], 0, 0);
  }
}

// The same piece of an activation's row r (64-bit addresses: any row).
template <int KIND>
__device__ __forceinline__ void piece_load_row(Piece<KIND>& p, const uint8_t* data, const uint8_t* scales, int64_t r,
                                               const PieceCols<KIND>& c, int K, int64_t ld) {
  if constexpr (KIND == kBf16Piece) {
    const uint16_t* row = reinterpret_cast<const uint16_t*>(data) + r * ld;
#pragma unroll
    for (int i = 0; i < 4; ++i) p.q[i] = *reinterpret_cast<const u32x4_t*>(row + c.c[i]);
  } else {
    const uint8_t *row = data + r * K, *srow = scales + r * (K >> 5);
#pragma unroll
    for (int i = 0; i < 2; ++i) p.q[i] = *reinterpret_cast<const u32x4_t*>(row + c.c[i]);
#pragma unroll
    for (int i = 0; i < 2; ++i) p.s[i] = srow[c.c[i] >> 5];
  }
}

// A row without values: zeros, whatever was loaded in its place.
template <int KIND>
__device__ __forceinline__ void piece_clear(Piece<KIND>& p, bool clear) {
#pragma unroll
  for (int i = 0; i < Piece<KIND>::kWords; ++i) p.q[i] = clear ? u32x4_t{0u, 0u, 0u, 0u} : p.q[i];
#pragma unroll
  for (int i = 0; i < Piece<KIND>::kScales; ++i) p.s[i] = clear ? 0 : p.s[i];
}

// Eight of the piece's values as bf16: the i-th in the order of piece_chunk.
template <int KIND>
__device__ __forceinline__ u32x4_t piece_convert(const Piece<KIND>& p, int i) {
  if constexpr (KIND == kBf16Piece) {
    return p.q[i];
  } else if constexpr (KIND == kMxFp8) {
    const float s = e8m0_value(p.s[i >> 1]);
    const uint32_t w0 = p.q[i >> 1][2 * (i & 1)], w1 = p.q[i >> 1][2 * (i & 1) + 1];
    return u32x4_t{as_u32(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, s, false)),
                   as_u32(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, s, true)),
                   as_u32(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, s, false)),
                   as_u32(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, s, true))};
  } else if constexpr (KIND == kMxInt8) {
    float x[8];
    mx8_decode8<KIND>(make_uint2(p.q[i >> 1][2 * (i & 1)], p.q[i >> 1][2 * (i & 1) + 1]), p.s[i >> 1], x);
    return u32x4_t{pk_bf16(x[0], x[1]), pk_bf16(x[2], x[3]), pk_bf16(x[4], x[5]), pk_bf16(x[6], x[7])};
  } else if constexpr (KIND == 1) {
    return __builtin_bit_cast(u32x4_t, dq8_e2m1(p.q[0][i], e8m0_value(p.s[0])));
  } else if constexpr (KIND == 2) {
    const float s = e4m3_value(i < 2 ? p.s[0] & 0xFFu : p.s[0] >> 8);
    return __builtin_bit_cast(u32x4_t, dq8_e2m1_mul(p.q[0][i], s));
  } else if constexpr (KIND == 0) {
    return __builtin_bit_cast(u32x4_t, dq8_int4(p.q[0][i], fp16_value(p.s[0])));
  } else {
    float s, off;
    int4zp_scale(p.s[0], s, off);
    return __builtin_bit_cast(u32x4_t, dq8_int4_off(p.q[0][i], s, off));
  }
}

}  // namespace q4
