// mx8.hip -- activations saved in 8 bits for the backward pass: quantize and
// dequantize of the block formats (q4_mx8.h), the SwiGLU that saves its input
// on the way, and SwiGLU's gradient from what was saved.
//
// With sg = 1 / (1 + exp(-g)):  h = g sg u,
//   dg = dh u sg (1 + g (1 - sg)),   du = dh g sg.
// All math in fp32; exp and the reciprocal are the hardware's (v_exp_f32,
// v_rcp_f32: within an ulp or two of fp32), far below the one rounding to
// bf16 at the end.
//
// Bound by HBM, each value read and written once: quantize 8192 x 8192 (203 MB)
// 35 us, 5.8 TB/s, dequantize 31 us; SwiGLU of 32768 x 2 x 2048 (540 MB each way)
// 94 us to save and 80 back, each repeated by itself, 84 + 99 one after the
// other (of so few bytes the caches still hold a part for the next call).
// A block's maximum takes two lane exchanges, so nothing is staged in LDS.
#include "q4_device.h"
#include "q4_launch.h"
#include "q4_mma.h"
#include "q4_mx8.h"

namespace q4 {
namespace {

constexpr int kThreads = 256;
constexpr int64_t kMaxGrid = 1 << 20;

unsigned grid_of(int64_t pieces) {
  const int64_t b = (pieces + kThreads - 1) / kThreads;
  return (unsigned)(b < kMaxGrid ? b : kMaxGrid);
}

// Four neighbouring lanes hold a block of 32; every lane gets its maximum.
__device__ __forceinline__ uint32_t max_of_4(uint32_t a) {
  a = max(a, (uint32_t)__shfl_xor((int)a, 1));
  return max(a, (uint32_t)__shfl_xor((int)a, 2));
}

// 1 / (1 + e), e = exp(-g).  v_rcp_f32 returns 0 where the reciprocal is below
// the smallest normal number (g < -87.3), which times a large u is not small: it
// takes (1 + e) / 16, and the multiplication by 1/16 makes the denormal.  Powers
// of two: no other value changes.  (From e = 2^128 on, g < -88.7, it is 0, as in
// q4_swiglu.)
__device__ __forceinline__ float sigmoid(float g) {
  const float e = __builtin_amdgcn_exp2f(-1.4426950408889634f * g);
  return 0.0625f * __builtin_amdgcn_rcpf(__builtin_fmaf(e, 0.0625f, 0.0625f));
}

// Rows that the next kernel reads from far behind: written past the caches
// (gradient of 32768 x 2 x 2048, repeated: 95 -> 80 us).
__device__ __forceinline__ void store_past(uint16_t* p, u32x4_t v) {
  __builtin_nontemporal_store(v, reinterpret_cast<u32x4_t*>(p));
}

// 8 values per thread; rows of whole blocks, so four neighbouring lanes are
// in the loop together and hold one block.
template <int FMT>
__global__ void __launch_bounds__(kThreads)
mx8_quantize_kernel(const uint16_t* __restrict__ src, int64_t ld, int64_t rows, int64_t cols,
                    uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  const int64_t cpr = cols >> 3, total = rows * cpr;
  for (int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x; c < total; c += (int64_t)gridDim.x * kThreads) {
    const int64_t r = c / cpr, k = (c - r * cpr) * 8;
    const uint4 v = *reinterpret_cast<const uint4*>(src + r * ld + k);
    const uint32_t b = mx8_scale<FMT>(max_of_4(mx8_absmax(v, 0u)));
    *reinterpret_cast<uint2*>(codes + c * 8) = mx8_encode8<FMT>(v, b);
    if ((c & 3) == 0) scales[c >> 2] = (uint8_t)b;
  }
}

template <int FMT, bool F32>
__global__ void __launch_bounds__(kThreads)
mx8_dequant_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, int64_t rows, int64_t cols,
                   void* __restrict__ dst, int64_t ld) {
  const int64_t cpr = cols >> 3, total = rows * cpr;
  for (int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x; c < total; c += (int64_t)gridDim.x * kThreads) {
    const int64_t r = c / cpr, k = (c - r * cpr) * 8;
    float x[8];
    mx8_decode8<FMT>(*reinterpret_cast<const uint2*>(codes + c * 8), scales[c >> 2], x);
    if constexpr (F32) {
      float4* d = reinterpret_cast<float4*>(static_cast<float*>(dst) + r * ld + k);
      d[0] = make_float4(x[0], x[1], x[2], x[3]);
      d[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(dst) + r * ld + k) =
          make_uint4(pk_bf16(x[0], x[1]), pk_bf16(x[2], x[3]), pk_bf16(x[4], x[5]), pk_bf16(x[6], x[7]));
    }
  }
}

__device__ __forceinline__ void unpack(const uint4& v, float (&x)[8]) {
  x[0] = bf16_lo(v.x); x[1] = bf16_hi(v.x);
  x[2] = bf16_lo(v.y); x[3] = bf16_hi(v.y);
  x[4] = bf16_lo(v.z); x[5] = bf16_hi(v.z);
  x[6] = bf16_lo(v.w); x[7] = bf16_hi(v.w);
}

// I % 32 == 0, so the gate and the up half of a row have blocks of their own.
template <int FMT>
__global__ void __launch_bounds__(kThreads)
swiglu_save_kernel(const uint16_t* __restrict__ gu, int64_t ld_gu, int64_t P, int64_t I, uint16_t* __restrict__ h,
                   int64_t ldh, uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  const int64_t cpr = I >> 3, total = P * cpr;
  for (int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x; c < total; c += (int64_t)gridDim.x * kThreads) {
    const int64_t p = c / cpr, n = (c - p * cpr) * 8;
    const uint4 gv = *reinterpret_cast<const uint4*>(gu + p * ld_gu + n);
    const uint4 uv = *reinterpret_cast<const uint4*>(gu + p * ld_gu + I + n);
    const uint32_t gb = mx8_scale<FMT>(max_of_4(mx8_absmax(gv, 0u)));
    const uint32_t ub = mx8_scale<FMT>(max_of_4(mx8_absmax(uv, 0u)));
    float g[8], u[8];
    unpack(gv, g);
    unpack(uv, u);
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      o[j] = pk_bf16(g[2 * j] * sigmoid(g[2 * j]) * u[2 * j], g[2 * j + 1] * sigmoid(g[2 * j + 1]) * u[2 * j + 1]);
    store_past(h + p * ldh + n, u32x4_t{o[0], o[1], o[2], o[3]});
    uint8_t* row = codes + p * 2 * I;
    *reinterpret_cast<uint2*>(row + n) = mx8_encode8<FMT>(gv, gb);
    *reinterpret_cast<uint2*>(row + I + n) = mx8_encode8<FMT>(uv, ub);
    if ((c & 3) == 0) {
      uint8_t* s = scales + p * (I >> 4);
      s[n >> 5] = (uint8_t)gb;
      s[(I + n) >> 5] = (uint8_t)ub;
    }
  }
}

// FMT 0: gu itself in bf16 (codes is then the bf16 matrix, ld its stride).
template <int FMT, bool WITH_H>
__global__ void __launch_bounds__(kThreads)
swiglu_backward_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, int64_t ld, int64_t P,
                       int64_t I, const uint16_t* __restrict__ dh, int64_t lddh, uint16_t* __restrict__ dgu,
                       int64_t lddgu, uint16_t* __restrict__ h, int64_t ldh) {
  const int64_t cpr = I >> 3, total = P * cpr;
  for (int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x; c < total; c += (int64_t)gridDim.x * kThreads) {
    const int64_t p = c / cpr, n = (c - p * cpr) * 8;
    float g[8], u[8], d[8];
    if constexpr (FMT == 0) {
      const uint16_t* row = reinterpret_cast<const uint16_t*>(codes) + p * ld;
      unpack(*reinterpret_cast<const uint4*>(row + n), g);
      unpack(*reinterpret_cast<const uint4*>(row + I + n), u);
    } else {
      const uint8_t *row = codes + p * 2 * I, *s = scales + p * (I >> 4);
      mx8_decode8<FMT>(*reinterpret_cast<const uint2*>(row + n), s[n >> 5], g);
      mx8_decode8<FMT>(*reinterpret_cast<const uint2*>(row + I + n), s[(I + n) >> 5], u);
    }
    unpack(*reinterpret_cast<const uint4*>(dh + p * lddh + n), d);
    float dg[8], du[8], hv[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float sg = sigmoid(g[j]), act = g[j] * sg;
      dg[j] = d[j] * u[j] * (sg * (1.0f + g[j] * (1.0f - sg)));
      du[j] = d[j] * act;
      if constexpr (WITH_H) hv[j] = act * u[j];
    }
    uint16_t* row = dgu + p * lddgu;
    store_past(row + n, u32x4_t{pk_bf16(dg[0], dg[1]), pk_bf16(dg[2], dg[3]), pk_bf16(dg[4], dg[5]), pk_bf16(dg[6], dg[7])});
    store_past(row + I + n, u32x4_t{pk_bf16(du[0], du[1]), pk_bf16(du[2], du[3]), pk_bf16(du[4], du[5]), pk_bf16(du[6], du[7])});
    if constexpr (WITH_H)
      store_past(h + p * ldh + n, u32x4_t{pk_bf16(hv[0], hv[1]), pk_bf16(hv[2], hv[3]), pk_bf16(hv[4], hv[5]), pk_bf16(hv[6], hv[7])});
  }
}

}  // namespace

hipError_t launch_mx8_quantize(int fmt, const uint16_t* src, int64_t ld, int64_t rows, int64_t cols, uint8_t* codes,
                               uint8_t* scales, hipStream_t stream) {
  const int64_t pieces = rows * (cols >> 3);
  if (!pieces) return hipSuccess;
  if (fmt == kMxInt8)
    mx8_quantize_kernel<kMxInt8><<<grid_of(pieces), kThreads, 0, stream>>>(src, ld, rows, cols, codes, scales);
  else
    mx8_quantize_kernel<kMxFp8><<<grid_of(pieces), kThreads, 0, stream>>>(src, ld, rows, cols, codes, scales);
  return hipGetLastError();
}

hipError_t launch_mx8_dequant(int fmt, const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols,
                              void* dst, int dst_dtype, int64_t ld, hipStream_t stream) {
  const int64_t pieces = rows * (cols >> 3);
  if (!pieces) return hipSuccess;
  auto k = fmt == kMxInt8 ? (dst_dtype ? mx8_dequant_kernel<kMxInt8, true> : mx8_dequant_kernel<kMxInt8, false>)
                          : (dst_dtype ? mx8_dequant_kernel<kMxFp8, true> : mx8_dequant_kernel<kMxFp8, false>);
  k<<<grid_of(pieces), kThreads, 0, stream>>>(codes, scales, rows, cols, dst, ld);
  return hipGetLastError();
}

hipError_t launch_swiglu_save(int fmt, const uint16_t* gu, int64_t ld_gu, int64_t P, int64_t I, uint16_t* h,
                              int64_t ldh, uint8_t* codes, uint8_t* scales, hipStream_t stream) {
  const int64_t pieces = P * (I >> 3);
  if (!pieces) return hipSuccess;
  auto k = fmt == kMxInt8 ? swiglu_save_kernel<kMxInt8> : swiglu_save_kernel<kMxFp8>;
  k<<<grid_of(pieces), kThreads, 0, stream>>>(gu, ld_gu, P, I, h, ldh, codes, scales);
  return hipGetLastError();
}

hipError_t launch_swiglu_backward(int fmt, const void* gu, const uint8_t* scales, int64_t ld_gu, int64_t P, int64_t I,
                                  const uint16_t* dh, int64_t lddh, uint16_t* dgu, int64_t lddgu, uint16_t* h,
                                  int64_t ldh, hipStream_t stream) {
  const int64_t pieces = P * (I >> 3);
  if (!pieces) return hipSuccess;
  auto k = fmt == kMxInt8 ? (h ? swiglu_backward_kernel<kMxInt8, true> : swiglu_backward_kernel<kMxInt8, false>)
           : fmt == kMxFp8 ? (h ? swiglu_backward_kernel<kMxFp8, true> : swiglu_backward_kernel<kMxFp8, false>)
                           : (h ? swiglu_backward_kernel<0, true> : swiglu_backward_kernel<0, false>);
  k<<<grid_of(pieces), kThreads, 0, stream>>>(static_cast<const uint8_t*>(gu), scales, ld_gu, P, I, dh, lddh, dgu,
                                              lddgu, h, ldh);
  return hipGetLastError();
}

}  // namespace q4
