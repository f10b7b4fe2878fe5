// gemm_grad.hip -- the gradients of the W4 products.  Forward, for the rows p
// of expert e (a dense layer is one expert): c[p][n] = sum_k a[p][k] w'_e[n][k].
//
//   dgrad  dA[p][k]   = sum_n dC[p][n] w'_e[n][k]
//   wgrad  dW_e[n][k] = sum_{p in e} dC[p][n] a[gather[p]][k]
//
// Both are bf16 matrix products (v_mfma_f32_16x16x32_bf16, fp32 sums) whose
// second operand -- the 4-bit weight, the saved activation -- is stored with
// the summed index as its rows, so its fragments are read column-wise from
// bf16 rows in LDS (q4_piece.h converts it once per workgroup).
#include "q4_launch.h"
#include "q4_piece.h"

namespace q4 {
namespace {

constexpr int kT = 64;        // tile of C: 64 x 64, a wave 32 x 32 of it
constexpr int kR = 32;        // summed rows per stage
constexpr int kPad = 8;

// Segment of an expert, clamped to [0, P]; offsets NULL: all rows.
__device__ __forceinline__ void segment(const int32_t* offsets, int e, int64_t P, int64_t& lo, int64_t& hi) {
  lo = 0;
  hi = P;
  if (offsets) {
    lo = min(max((int64_t)offsets[e], (int64_t)0), P);
    hi = min(max((int64_t)offsets[e + 1], lo), P);
  }
}

// Row tile number `slot` over all experts: its expert and first row; false if
// there are fewer tiles.
__device__ __forceinline__ bool find_tile(const int32_t* offsets, int E, int64_t P, int64_t slot, int& e, int64_t& lo,
                                          int64_t& hi) {
  for (e = 0; e < E; ++e) {
    segment(offsets, e, P, lo, hi);
    const int64_t tiles = (hi - lo + kT - 1) / kT;
    if (slot < tiles) {
      lo += slot * kT;
      return true;
    }
    slot -= tiles;
  }
  return false;
}

template <bool WGRAD, int KIND, int LAYOUT>
__global__ void __launch_bounds__(256)
grad_simple_kernel(GradArgs g) {
  __shared__ uint16_t sa[kR][kT + kPad], sb[kR][kT + kPad];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const PieceSrc src{g.b, g.b_scales, g.K, g.ldb};
  const int64_t k0 = (int64_t)blockIdx.x * kT;
  int e;
  int64_t lo, hi, m0;     // the segment's rows; m0: first row (dgrad) / first n (wgrad) of the tile
  if constexpr (WGRAD) {
    e = blockIdx.z;
    segment(g.offsets, e, g.P, lo, hi);
    m0 = (int64_t)blockIdx.y * kT;
  } else {
    if (!find_tile(g.offsets, g.E, g.P, blockIdx.y, e, lo, hi)) return;
    m0 = lo;
  }
  const int64_t m_end = WGRAD ? g.N : hi, r_begin = WGRAD ? lo : 0, r_end = WGRAD ? hi : g.N;
  f32x4_t acc[2][2] = {};
  for (int64_t r0 = r_begin; r0 < r_end; r0 += kR) {
    __syncthreads();
    if constexpr (WGRAD) {
      const int r = tid >> 3, c = (tid & 7) * 8;
      u32x4_t v{0u, 0u, 0u, 0u};
      if (r0 + r < r_end && m0 + c < g.N) v = *reinterpret_cast<const u32x4_t*>(g.dc + (r0 + r) * g.lddc + m0 + c);
      *reinterpret_cast<u32x4_t*>(&sa[r][c]) = v;
    } else {
      const int m = tid >> 2, c = (tid & 3) * 8;
      u32x4_t v{0u, 0u, 0u, 0u};
      if (m0 + m < hi && r0 + c < g.N) v = *reinterpret_cast<const u32x4_t*>(g.dc + (m0 + m) * g.lddc + r0 + c);
#pragma unroll
      for (int i = 0; i < 8; ++i) sa[c + i][m] = (uint16_t)(v[i >> 1] >> (16 * (i & 1)));
    }
    if (tid < 64) {
      const int r = tid >> 1, c = (tid & 1) * 32;
      bool ok = r0 + r < r_end && k0 + c < g.K;
      int64_t row = WGRAD ? r0 + r : (int64_t)e * g.N + r0 + r;
      if constexpr (WGRAD) {
        if (ok && g.gather) row = g.gather[row];
        ok = ok && row >= 0 && row < g.T;
      }
      Piece<KIND> p;
      u32x4_t o[4];
      piece_load<KIND, LAYOUT>(p, src, row, k0 + c, ok);
      piece_convert<KIND>(p, o);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<u32x4_t*>(&sb[r][c + 8 * i]) = ok ? o[i] : u32x4_t{0u, 0u, 0u, 0u};
    }
    __syncthreads();
    bf16x8_t fa[2], fb[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      uint16_t xa[8], xb[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        xa[i] = sa[8 * (lane >> 4) + i][32 * (wave >> 1) + 16 * t + (lane & 15)];
        xb[i] = sb[8 * (lane >> 4) + i][32 * (wave & 1) + 16 * t + (lane & 15)];
      }
      fa[t] = __builtin_bit_cast(bf16x8_t, xa);
      fb[t] = __builtin_bit_cast(bf16x8_t, xb);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[i][j] = mma16x16x32(fb[j], fa[i], acc[i][j]);
  }
  // register q of lane l: column 4 (l / 16) + q, row l % 16 of a 16 x 16 tile
  const float gs = KIND == 2 ? *g.gs : 1.0f;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int64_t m = m0 + 32 * (wave >> 1) + 16 * i + (lane & 15);
      const int64_t k = k0 + 32 * (wave & 1) + 16 * j + 4 * (lane >> 4);
      if (m >= m_end || k >= g.K) continue;
      const f32x4_t v = acc[i][j] * gs;
      const int64_t row = WGRAD ? (int64_t)e * g.N + m : m;
      if (WGRAD && g.out_f32) {
        float* o = static_cast<float*>(g.out) + row * g.ldo + k;
#pragma unroll
        for (int q = 0; q < 4; ++q) o[q] = g.accumulate ? o[q] + v[q] : v[q];
      } else {
        store_bf16x4(static_cast<uint16_t*>(g.out) + row * g.ldo + k, v[0], v[1], v[2], v[3]);
      }
    }
}

template <bool WGRAD, int KIND, int LAYOUT>
hipError_t run(const GradArgs& g, hipStream_t stream) {
  const unsigned kt = (unsigned)((g.K + kT - 1) / kT);
  const dim3 grid = WGRAD ? dim3(kt, (unsigned)((g.N + kT - 1) / kT), (unsigned)g.E)
                          : dim3(kt, (unsigned)((g.P + kT - 1) / kT + g.E - 1), 1u);
  grad_simple_kernel<WGRAD, KIND, LAYOUT><<<grid, 256, 0, stream>>>(g);
  return hipGetLastError();
}

}  // namespace

size_t dgrad_workspace(int64_t, int32_t, int64_t, int64_t) { return 0; }
size_t wgrad_workspace(int64_t, int32_t, int64_t, int64_t) { return 0; }

bool dgrad_fits(int64_t P, int32_t E, int64_t, int64_t K) {
  return (P + kT - 1) / kT + E <= 65535 && (K + kT - 1) / kT < ((int64_t)1 << 24);
}
bool wgrad_fits(int64_t, int32_t, int64_t N, int64_t K) {
  return (N + kT - 1) / kT <= 65535 && (K + kT - 1) / kT < ((int64_t)1 << 24);
}

hipError_t launch_dgrad(int fmt, int layout, const GradArgs& g, hipStream_t stream) {
  const bool t = layout == kLayoutTiled;
  switch (fmt) {
    case 0: return t ? run<false, 0, kLayoutTiled>(g, stream) : run<false, 0, kLayoutRows>(g, stream);
    case 1: return t ? run<false, 1, kLayoutTiled>(g, stream) : run<false, 1, kLayoutRows>(g, stream);
    case 4: return t ? run<false, 4, kLayoutTiled>(g, stream) : run<false, 4, kLayoutRows>(g, stream);
    default: return t ? run<false, 2, kLayoutTiled>(g, stream) : run<false, 2, kLayoutRows>(g, stream);
  }
}

hipError_t launch_wgrad(int kind, const GradArgs& g, hipStream_t stream) {
  switch (kind) {
    case kMxFp8: return run<true, kMxFp8, kLayoutRows>(g, stream);
    case kMxInt8: return run<true, kMxInt8, kLayoutRows>(g, stream);
    default: return run<true, kBf16Piece, kLayoutRows>(g, stream);
  }
}

}  // namespace q4
