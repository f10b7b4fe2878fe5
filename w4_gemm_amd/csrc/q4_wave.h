// q4_wave.h -- reductions over the lanes of a wave in which every lane gets the
// result.  Steps within 16 lanes are DPP moves (exchanges in quads, then mirrors of
// 8 and 16 lanes: by then the lanes of a mirrored group hold the same value), those
// across are gfx950's lane swaps; none goes through LDS.  The order is the same in
// every lane and every run.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace q4 {

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_move(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
}

constexpr int kDppXor1 = 0xB1, kDppXor2 = 0x4E, kDppHalfMirror = 0x141, kDppMirror = 0x140;

struct AddOp {
  __device__ __forceinline__ uint32_t operator()(uint32_t a, uint32_t b) const {
    return __builtin_bit_cast(uint32_t, __builtin_bit_cast(float, a) + __builtin_bit_cast(float, b));
  }
};
struct MaxBitsOp {
  __device__ __forceinline__ uint32_t operator()(uint32_t a, uint32_t b) const { return a > b ? a : b; }
};

// Over aligned groups of LANES (16, 32 or 64) lanes.
template <int LANES, typename OP>
__device__ __forceinline__ uint32_t reduce_lanes(uint32_t v, OP op) {
  static_assert(LANES == 16 || LANES == 32 || LANES == 64, "groups of lanes");
  v = op(v, dpp_move<kDppXor1>(v));
  v = op(v, dpp_move<kDppXor2>(v));
  v = op(v, dpp_move<kDppHalfMirror>(v));
  v = op(v, dpp_move<kDppMirror>(v));
  if constexpr (LANES >= 32) {   // rows 0 and 1, 2 and 3 of 16 lanes
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = op(r[0], r[1]);
  }
  if constexpr (LANES == 64) {
    const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    v = op(r[0], r[1]);
  }
  return v;
}

template <int LANES = 64>
__device__ __forceinline__ float lanes_sum(float v) {
  return __builtin_bit_cast(float, reduce_lanes<LANES>(__builtin_bit_cast(uint32_t, v), AddOp()));
}
template <int LANES = 64>
__device__ __forceinline__ uint32_t lanes_max_bits(uint32_t v) {
  return reduce_lanes<LANES>(v, MaxBitsOp());
}

}  // namespace q4
