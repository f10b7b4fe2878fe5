// rmsnorm.hip -- root-mean-square norm with the residual's addition in front
// and the quantization of the 8-bit products behind it, and its gradient.
//
//   h = bf16(x + residual)                (the residual stream; h = x without)
//   y = (h * w) * r,   r = 1 / sqrt(mean(h^2) + eps)
//
// in fp32 from h as it is stored, so that the gradient, which has h alone, is
// that of what the forward pass computed.  y goes out in bf16, or in 8 bits with
// one scale per row (Q4_FP8_ROW, Q4_INT8_ROW) straight from the fp32 values, or
// both.  r is one factor of the whole row and fp32 multiplication is monotone,
// so the row's largest |y| is r times the largest |h w|: one reduction gives the
// sum of squares and the scale together, and a code is that of
// (h w) * (r * top / a), a the largest |y|.
//
// A row is held in registers by 1, 4 or 16 waves (lane i of them has the chunks
// of eight values i, i + 64 WAVES, ...) and read once.  Bound by HBM: 16385 x 8192 with
// a residual and 8-bit codes in 143 to 146 us, 6.4 to 6.6 TB/s, its gradient (16384 rows)
// in 172 to 186 us on several cards, 5.8 to 6.2 TB/s, and 7 us for the weight's sum; one
// row in 3.2 to 3.7 us, all latency.
#include "q4_launch.h"
#include "q4_layout.h"
#include "q4_mma.h"
#include "q4_row8.h"

#include <type_traits>

namespace q4 {
namespace {

// Eight weights: fp32, or bf16 widened.
template <bool WF32>
__device__ __forceinline__ void load_weight8(const void* w, int k0, float (&o)[8]) {
  if constexpr (WF32) {
    const float4 a = *reinterpret_cast<const float4*>(static_cast<const float*>(w) + k0);
    const float4 b = *reinterpret_cast<const float4*>(static_cast<const float*>(w) + k0 + 4);
    o[0] = a.x; o[1] = a.y; o[2] = a.z; o[3] = a.w;
    o[4] = b.x; o[5] = b.y; o[6] = b.z; o[7] = b.w;
  } else {
    unpack_bf16x8(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(w) + k0), o);
  }
}

__device__ __forceinline__ uint4 pack_bf16x8(const float (&v)[8]) {
  return make_uint4(pk_bf16(v[0], v[1]), pk_bf16(v[2], v[3]), pk_bf16(v[4], v[5]), pk_bf16(v[6], v[7]));
}

// mean(h^2) + eps, and 1 / sqrt of it; NaN where the sum of squares is no number below
// 2^128, so that a row whose squares overflow is not taken for zeros.
__device__ __forceinline__ float row_mean(float ss, int cols, float eps) {
  return ss <= 3.402823466e+38f ? ss / (float)cols + eps : u2f(0x7FC00000u);
}
__device__ __forceinline__ float row_rstd(float mean) { return 1.0f / __builtin_sqrtf(mean); }

// Rows so small that their squares vanish or lose bits in fp32 (with eps as small as
// they are): below kLeastMean the sums are made again from 2^80 h and 2^160 eps, and r
// then is 2^-80 of itself.  |h| is 2^-133 at least and sqrt(cols) 2^-30 < 2^-22 at most
// there, so that squares of 2^80 h are 2^-106 at least, their mean is 2^-121 at least
// and their sum, 32768 2^100 at most, far below 2^128.  Scales by powers of two commute
// with every step: a row that either way holds gets the same results bit for bit.  In a
// mean of 2^-60 and more, squares below fp32's normal range are less than 2^-66 of it.
constexpr float kLeastMean = 0x1p-60f, kRaise = 0x1p80f;
template <bool RAISED>
__device__ __forceinline__ float raised(float v) { return RAISED ? v * kRaise : v; }

// KIND: kRowInt8, kRowE4m3, or -1 for no output in 8 bits.  PAST: rows are read and h
// is written past the caches (kPastForward values and more: 16385 x 8192 in 144 us, 163
// without; 4096 x 8192, which they hold, 36.8 us and 42.6 with it).  The codes are not:
// the product reads them next, and 8 bytes at a time they gain nothing.
template <int WAVES, int CH, int KIND, bool WF32, bool PAST>
__global__ void __launch_bounds__(64 * (WAVES < 4 ? 4 : WAVES), WAVES == 16 ? 8 : 1)   // (two workgroups per CU)
rmsnorm_kernel(const NormArgs p) {
  constexpr int kRows = WAVES < 4 ? 4 / WAVES : 1;
  const int tid = threadIdx.x % (64 * WAVES), in = threadIdx.x / (64 * WAVES);
  const int64_t r = (int64_t)blockIdx.x * kRows + in;
  const int cols = p.cols;
  if (r >= p.rows) {  // (a wave of its own, or the whole workgroup: nobody waits for it)
    if (KIND == kRowE4m3 && p.tiled && r < p.srows)   // padding row of the last tile: zero codes
      for (int k0 = tid * 8; k0 < cols; k0 += 512 * WAVES) {
        *reinterpret_cast<uint32_t*>(p.codes + fp8_tiled_dword(r, k0, cols, 0)) = 0u;
        *reinterpret_cast<uint32_t*>(p.codes + fp8_tiled_dword(r, k0, cols, 1)) = 0u;
      }
    return;
  }
  const uint16_t* x = p.x + r * p.ldx;
  uint4 v[CH];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int k0 = (tid + 64 * WAVES * i) * 8;
    v[i] = load16<PAST>(x + (k0 < cols ? k0 : 0));
  }
  if (p.residual) {
    const uint16_t* res = p.residual + r * p.ldr;
    uint4 u[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int k0 = (tid + 64 * WAVES * i) * 8;
      u[i] = load16<PAST>(res + (k0 < cols ? k0 : 0));
    }
    uint16_t* h = p.h + r * p.ldh;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int k0 = (tid + 64 * WAVES * i) * 8;
      float a[8], b[8];
      unpack_bf16x8(v[i], a);
      unpack_bf16x8(u[i], b);
#pragma unroll
      for (int j = 0; j < 8; ++j) a[j] += b[j];
      v[i] = pack_bf16x8(a);
      if (k0 < cols) store16<PAST>(h + k0, v[i]);
    }
  }
  float hw[CH][8];
  float ss, mean;
  uint32_t most;
  __shared__ float sum[2][WAVES];
  __shared__ uint32_t top[2][WAVES];
  auto sums = [&](auto raise) {
    constexpr bool kRaised = decltype(raise)::value;
    ss = 0.0f;
    most = 0;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int k0 = (tid + 64 * WAVES * i) * 8;
      if (k0 < cols) {
        float a[8], w[8];
        unpack_bf16x8(kRaised ? load16<PAST>((p.residual ? p.h + r * p.ldh : x) + k0) : v[i], a);
        load_weight8<WF32>(p.w, k0, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          a[j] = raised<kRaised>(a[j]);
          ss = __builtin_fmaf(a[j], a[j], ss);
          hw[i][j] = a[j] * w[j];
        }
        if (KIND >= 0) most = max_bits8(hw[i], most);
      }
    }
    ss = lanes_sum(ss);
    if (KIND >= 0) most = lanes_max_bits(most);
    if constexpr (WAVES > 1) {
      if ((tid & 63) == 0) {
        sum[kRaised][tid >> 6] = ss;
        top[kRaised][tid >> 6] = most;
      }
      __syncthreads();
      ss = 0.0f;
#pragma unroll
      for (int w = 0; w < WAVES; ++w) {
        ss += sum[kRaised][w];
        most = top[kRaised][w] > most ? top[kRaised][w] : most;
      }
    }
    mean = row_mean(ss, cols, raised<kRaised>(raised<kRaised>(p.eps)));
  };
  sums(std::false_type());
  // (the same for all of a row; read again from where it stands, so that ordinary rows
  // need no registers for it)
  if (mean < kLeastMean) sums(std::true_type());
  const float rstd = row_rstd(mean);
  float f = 0.0f;
  if constexpr (KIND >= 0) {
    const float a = u2f(most) * rstd;              // the largest |y|
    const bool fine = a <= 3.402823466e+38f;
    const float least = fmaxf(a, 1e-12f);
    f = fine ? rstd * kRowTop<KIND> / least : 0.0f;
    if (tid == 0) p.scales[r] = fine ? least / kRowTop<KIND> : u2f(0x7FC00000u);
  }
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int k0 = (tid + 64 * WAVES * i) * 8;
    if (k0 >= cols) continue;
    if constexpr (KIND == kRowInt8) {
      *reinterpret_cast<uint2*>(p.codes + r * cols + k0) = int8_pack8(hw[i], f);
    } else if constexpr (KIND == kRowE4m3) {
      const uint2 q = e4m3_pack8(hw[i], f);
      // even elements in one word, odd ones in the next.  (4 bytes at a time, of a line that
      // eight rows share: 4096 x 8192 in 52 us, 36 in rows; 16384 rows 219 and 144.)
      if (p.tiled) {
        *reinterpret_cast<uint32_t*>(p.codes + fp8_tiled_dword(r, k0, cols, 0)) = __builtin_amdgcn_perm(q.y, q.x, 0x06040200u);
        *reinterpret_cast<uint32_t*>(p.codes + fp8_tiled_dword(r, k0, cols, 1)) = __builtin_amdgcn_perm(q.y, q.x, 0x07050301u);
      } else {
        *reinterpret_cast<uint2*>(p.codes + r * cols + k0) = q;
      }
    }
    if (KIND < 0 || p.y) {
#pragma unroll
      for (int j = 0; j < 8; ++j) hw[i][j] *= rstd;
      *reinterpret_cast<uint4*>(p.y + r * p.ldy + k0) = pack_bf16x8(hw[i]);
    }
  }
}

// ---- gradient ----------------------------------------------------------------
// With n = h r and g = dy w:
//   dx = dh + r (g - n mean(g n)),   dw = sum over rows of dy n
// mean(g n) = r sum(g h) / cols, so one reduction gives sum(h^2) and sum(g h)
// together and nothing but h need be kept from the forward pass.  Workgroups
// walk over rows with dw of their columns in registers; each writes its sum to
// the workspace, and a second kernel adds those in order.  PAST: rows are read past
// the caches (kPastBackward values and more; without the weight's gradient 16385 x 8192
// in 161 us, 192 without; 4096 x 8192 in 45 and 43, 512 x 8192 in 8.3 both ways); dx,
// which is read next, is not written so.  Above 8192 columns the 1024 threads have 128
// registers each and want more (129 to 161 spilled within the loop): 4096 x 16384 in
// 386 us with the weight's sum, five times what its bytes take.
template <int WAVES, int CH, bool WF32, bool PAST>
__global__ void __launch_bounds__(64 * (WAVES < 4 ? 4 : WAVES))
rmsnorm_backward_kernel(const NormGradArgs p) {
  constexpr int kRows = WAVES < 4 ? 4 / WAVES : 1;
  constexpr int kThreads = 64 * WAVES;
  const int tid = threadIdx.x % kThreads, in = threadIdx.x / kThreads;
  const int cols = p.cols;
  float w[CH][8], dw[CH][8];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int k0 = (tid + kThreads * i) * 8;
    if (k0 < cols) load_weight8<WF32>(p.w, k0, w[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = 0.0f;
  }
  __shared__ float part[3][2][WAVES];
  int turn = 0;
  for (int64_t r = (int64_t)blockIdx.x * kRows + in; r < p.rows; r += (int64_t)gridDim.x * kRows, turn ^= 1) {
    uint4 vd[CH], vh[CH], vr[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int k0 = (tid + kThreads * i) * 8, at = k0 < cols ? k0 : 0;
      vd[i] = load16<PAST>(p.dy + r * p.lddy + at);
      vh[i] = load16<PAST>(p.h + r * p.ldh + at);
      if (p.dh) vr[i] = load16<PAST>(p.dh + r * p.lddh + at);
    }
    // (a row whose mean is below kLeastMean comes round again, with `up` 2^80)
    float ss, c, mean, up = 1.0f, half = 1.0f;
    for (int set = turn;; set = 2) {
      ss = c = 0.0f;
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        if ((tid + kThreads * i) * 8 < cols) {
          float d[8], h[8];
          unpack_bf16x8(vd[i], d);
          unpack_bf16x8(vh[i], h);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            h[j] *= up;
            ss = __builtin_fmaf(h[j], h[j], ss);
            c = __builtin_fmaf(d[j] * w[i][j], h[j], c);
          }
        }
      }
      ss = lanes_sum(ss);
      c = lanes_sum(c);
      if constexpr (WAVES > 1) {
        // two sets in turn: a wave writes the next row's while others read this one's (the
        // third: between two rows that come round again there is a row's barrier)
        if ((tid & 63) == 0) {
          part[set][0][tid >> 6] = ss;
          part[set][1][tid >> 6] = c;
        }
        __syncthreads();
        ss = c = 0.0f;
#pragma unroll
        for (int v = 0; v < WAVES; ++v) {
          ss += part[set][0][v];
          c += part[set][1][v];
        }
      }
      mean = row_mean(ss, cols, p.eps * up * up);
      if (!(mean < kLeastMean) || set == 2) break;
      up = kRaise;
      half = 0x1p40f;
    }
    const float rstd = row_rstd(mean);
    const float t = c / (float)cols * rstd * rstd;
    // r is rstd times `up`, past fp32's range where h is least: half of the 80 on either side of a product
    const float by = rstd * half;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int k0 = (tid + kThreads * i) * 8;
      if (k0 < cols) {
        float d[8], h[8], o[8];
        unpack_bf16x8(vd[i], d);
        unpack_bf16x8(vh[i], h);
        if (p.dh) unpack_bf16x8(vr[i], o);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          h[j] *= up;
          const float e = by * __builtin_fmaf(-t, h[j], d[j] * w[i][j]) * half;
          o[j] = p.dh ? o[j] + e : e;
          dw[i][j] = __builtin_fmaf(d[j], h[j] * rstd, dw[i][j]);
        }
        *reinterpret_cast<uint4*>(p.dx + r * p.lddx + k0) = pack_bf16x8(o);
      }
    }
  }
  if (!p.partial) return;
  if constexpr (kRows > 1) {   // the rows side by side in a workgroup, added in order
    __shared__ float side[kRows][CH * 512 * WAVES];
#pragma unroll
    for (int i = 0; i < CH; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) side[in][(tid + kThreads * i) * 8 + j] = dw[i][j];
    __syncthreads();
    for (int k = threadIdx.x; k < cols; k += kThreads * kRows) {
      float s = 0.0f;
#pragma unroll
      for (int q = 0; q < kRows; ++q) s += side[q][k];
      p.partial[(int64_t)blockIdx.x * cols + k] = s;
    }
  } else {
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int k0 = (tid + kThreads * i) * 8;
      if (k0 < cols) {
        float4* o = reinterpret_cast<float4*>(p.partial + (int64_t)blockIdx.x * cols + k0);
        o[0] = make_float4(dw[i][0], dw[i][1], dw[i][2], dw[i][3]);
        o[1] = make_float4(dw[i][4], dw[i][5], dw[i][6], dw[i][7]);
      }
    }
  }
}

// dw[k] (+)= sum over the workgroups' sums: 32 columns by 32 slices per
// workgroup, the slices' sums added in order.  512 of them of 8192 columns, 17 MB, in
// 7 us: a slice's loads are each under a condition and so waited for one by one.
constexpr int kGradBlocks = 512;
__global__ void __launch_bounds__(1024)
rmsnorm_weight_sum_kernel(const float* __restrict__ partial, int blocks, int cols, float* __restrict__ dw,
                          int accumulate) {
  __shared__ float part[32][33];
  const int k = blockIdx.x * 32 + (threadIdx.x & 31), slice = threadIdx.x >> 5;
  float s = 0.0f;
  if (k < cols) {
#pragma unroll
    for (int i = 0; i < kGradBlocks / 32; ++i) {
      const int b = slice + 32 * i;
      if (b < blocks) s += partial[(int64_t)b * cols + k];
    }
  }
  part[slice][threadIdx.x & 31] = s;
  __syncthreads();
  if (slice == 0 && k < cols) {
#pragma unroll
    for (int q = 1; q < 32; ++q) s += part[q][threadIdx.x];
    dw[k] = accumulate ? dw[k] + s : s;
  }
}

constexpr int64_t kPastForward = (int64_t)48 << 20;    // values of a tensor
constexpr int64_t kPastBackward = (int64_t)16 << 20;

template <int WAVES, int CH, int KIND, bool WF32>
void norm_as(const NormArgs& a, hipStream_t stream) {
  constexpr int kRows = WAVES < 4 ? 4 / WAVES : 1;
  const unsigned grid = (unsigned)((a.srows + kRows - 1) / kRows), threads = 64 * WAVES * kRows;
  if (a.rows * a.cols >= kPastForward)
    rmsnorm_kernel<WAVES, CH, KIND, WF32, true><<<grid, threads, 0, stream>>>(a);
  else
    rmsnorm_kernel<WAVES, CH, KIND, WF32, false><<<grid, threads, 0, stream>>>(a);
}

template <int WAVES, int CH, bool WF32>
void norm_kind(const NormArgs& a, int kind, hipStream_t stream) {
  if (kind == kRowInt8) norm_as<WAVES, CH, kRowInt8, WF32>(a, stream);
  else if (kind == kRowE4m3) norm_as<WAVES, CH, kRowE4m3, WF32>(a, stream);
  else norm_as<WAVES, CH, -1, WF32>(a, stream);
}

template <int WAVES, int CH>
void norm(const NormArgs& a, int kind, hipStream_t stream) {
  if (a.w_f32) norm_kind<WAVES, CH, true>(a, kind, stream);
  else norm_kind<WAVES, CH, false>(a, kind, stream);
}

// Workgroups of the gradient, of one row (four of up to 2048 columns) at a time:
// enough for the loads, few enough that their sums are little beside the rows.  512
// where each has four turns and more (8192 x 8192: 92 us, 256 of them 103), else
// one for two turns, between 128 and 256 (512 x 8192: 16.9 us with 256 and 20.8
// with 512; 256 x 8192: 13.8 with 128 and 15.4 with 256).
int64_t grad_blocks(int64_t rows, int64_t cols) {
  const int64_t per = cols <= 2048 ? 4 : 1, turns = (rows + per - 1) / per;
  if (turns >= 4 * kGradBlocks) return kGradBlocks;
  if (turns <= 128) return turns;
  return turns >= 512 ? 256 : turns <= 256 ? 128 : turns / 2;
}

template <int WAVES, int CH>
void norm_backward(const NormGradArgs& a, hipStream_t stream) {
  constexpr int kRows = WAVES < 4 ? 4 / WAVES : 1;
  const bool past = a.rows * a.cols >= kPastBackward;
  auto kernel = a.w_f32 ? (past ? rmsnorm_backward_kernel<WAVES, CH, true, true> : rmsnorm_backward_kernel<WAVES, CH, true, false>)
                        : (past ? rmsnorm_backward_kernel<WAVES, CH, false, true> : rmsnorm_backward_kernel<WAVES, CH, false, false>);
  kernel<<<(unsigned)grad_blocks(a.rows, a.cols), 64 * WAVES * kRows, 0, stream>>>(a);
}

}  // namespace

hipError_t launch_rmsnorm(int fmt, const NormArgs& a, hipStream_t stream) {
  const int kind = fmt == 8 ? kRowInt8 : fmt == 3 ? kRowE4m3 : -1;
  if (a.cols <= 512)
    norm<1, 1>(a, kind, stream);
  else if (a.cols <= 2048)
    norm<1, 4>(a, kind, stream);
  else if (a.cols <= 8192)
    norm<4, 4>(a, kind, stream);
  else
    norm<16, 4>(a, kind, stream);
  return hipGetLastError();
}

size_t rmsnorm_backward_workspace(int64_t rows, int64_t cols) {
  return (size_t)grad_blocks(rows, cols) * (size_t)cols * 4;
}

hipError_t launch_rmsnorm_backward(const NormGradArgs& a, float* dweight, int accumulate, hipStream_t stream) {
  if (a.rows > 0) {
    if (a.cols <= 512)
      norm_backward<1, 1>(a, stream);
    else if (a.cols <= 2048)
      norm_backward<1, 4>(a, stream);
    else if (a.cols <= 8192)
      norm_backward<4, 4>(a, stream);
    else
      norm_backward<16, 4>(a, stream);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (dweight)
    rmsnorm_weight_sum_kernel<<<(unsigned)((a.cols + 31) / 32), 1024, 0, stream>>>(
        a.partial, a.rows > 0 ? (int)grad_blocks(a.rows, a.cols) : 0, a.cols, dweight, accumulate);
  return hipGetLastError();
}

}  // namespace q4
