// int8.hip -- rows in 8-bit integers with one scale each (Q4_INT8_ROW): the
// activations of a W8A8 product with a scale per token, and its weights with a
// scale per output channel ("Quantization in deployment", format cheat sheet,
// W8A8: one scale per token and per channel; "LLM quantization", the absmax
// method in 8 bits).
//
// scale = a / 127 and code = rne(x * fp32(127 / a)) with a = max(amax, 1e-12)
// (q4_row8.h).  A row with an infinity or a NaN gets the scale NaN, so that
// what is computed from it is NaN, and codes without meaning.  Bound by HBM: 4096 x
// 8192 in 16.7 us, 6.0 TB/s; one row in 2.7.
#include "q4_launch.h"
#include "q4_mma.h"
#include "q4_row8.h"

namespace q4 {
namespace {

__device__ __forceinline__ float row_scale(uint32_t amax_bits, float& f) {
  const float a = fmaxf(u2f(amax_bits), 1e-12f);
  const bool fine = amax_bits < 0x7F800000u;
  f = fine ? 127.0f / a : 0.0f;
  return fine ? a / 127.0f : u2f(0x7FC00000u);
}

// Rows of at most 512 * WAVES * CH values: WAVES waves hold a row in registers
// (lane i of them the chunks of eight values i, i + 64 WAVES, ...), every load
// issued before the first is used, so the row is read once.  Short rows go four
// to a workgroup.
template <int WAVES, int CH>
__global__ void __launch_bounds__(64 * (WAVES < 4 ? 4 : WAVES))
int8_rows_quantize_kernel(const uint16_t* __restrict__ src, int64_t ld, int64_t rows, int cols,
                          uint8_t* __restrict__ codes, float* __restrict__ scales) {
  constexpr int kRows = WAVES < 4 ? 4 / WAVES : 1;
  const int tid = threadIdx.x % (64 * WAVES), in = threadIdx.x / (64 * WAVES);
  const int64_t r = (int64_t)blockIdx.x * kRows + in;
  if (WAVES == 1 && r >= rows) return;
  // (with more waves per row every wave meets the barrier; a row past the end
  // reads the last one and stores nothing)
  const uint16_t* row = src + (r < rows ? r : rows - 1) * ld;
  uint4 v[CH];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int k0 = (tid + 64 * WAVES * i) * 8;
    // a chunk past the end reads the row's first one: the largest stays the same
    v[i] = *reinterpret_cast<const uint4*>(row + (k0 < cols ? k0 : 0));
  }
  __builtin_amdgcn_sched_barrier(0);
  uint32_t m = 0;
  float x[8];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    unpack_bf16x8(v[i], x);
    m = max_bits8(x, m);
  }
  m = lanes_max_bits(m);
  if constexpr (WAVES > 1) {
    __shared__ uint32_t part[kRows][WAVES];
    if ((tid & 63) == 0) part[in][tid >> 6] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < WAVES; ++w) m = part[in][w] > m ? part[in][w] : m;
    if (r >= rows) return;
  }
  float f;
  const float s = row_scale(m, f);
  if (tid == 0) scales[r] = s;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int k0 = (tid + 64 * WAVES * i) * 8;
    if (k0 < cols) {
      unpack_bf16x8(v[i], x);
      *reinterpret_cast<uint2*>(codes + r * cols + k0) = int8_pack8(x, f);
    }
  }
}

// Longer rows: a workgroup of 1024 threads reads a row twice.
__global__ void __launch_bounds__(1024)
int8_rows_quantize_long_kernel(const uint16_t* __restrict__ src, int64_t ld, int64_t cols,
                               uint8_t* __restrict__ codes, float* __restrict__ scales) {
  const int64_t r = blockIdx.x;
  const uint16_t* row = src + r * ld;
  __shared__ uint32_t part[16];
  float x[8];
  uint32_t m = 0;
  for (int64_t k0 = (int64_t)threadIdx.x * 8; k0 < cols; k0 += 8192) {
    unpack_bf16x8(*reinterpret_cast<const uint4*>(row + k0), x);
    m = max_bits8(x, m);
  }
  m = lanes_max_bits(m);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 16; ++w) m = part[w] > m ? part[w] : m;
  float f;
  const float s = row_scale(m, f);
  if (threadIdx.x == 0) scales[r] = s;
  for (int64_t k0 = (int64_t)threadIdx.x * 8; k0 < cols; k0 += 8192) {
    unpack_bf16x8(*reinterpret_cast<const uint4*>(row + k0), x);
    *reinterpret_cast<uint2*>(codes + r * cols + k0) = int8_pack8(x, f);
  }
}

constexpr int kThreads = 256;

// value = fp32(code * scale); 8 values per thread.
template <int OUT>
__global__ void __launch_bounds__(kThreads)
int8_rows_dequant_kernel(const uint8_t* __restrict__ codes, const float* __restrict__ scales, int64_t rows,
                         int64_t cols, void* __restrict__ dst, int64_t ld) {
  const int64_t cpr = cols >> 3, total = rows * cpr;
  for (int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x; c < total; c += (int64_t)gridDim.x * kThreads) {
    const int64_t r = c / cpr, k0 = (c - r * cpr) * 8;
    const uint2 v = *reinterpret_cast<const uint2*>(codes + r * cols + k0);
    const float s = scales[r];
    float x[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[j] = (float)(int8_t)(v.x >> (8 * j)) * s;
      x[4 + j] = (float)(int8_t)(v.y >> (8 * j)) * s;
    }
    if constexpr (OUT == 0) {
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(dst) + r * ld + k0) =
          make_uint4(pk_bf16(x[0], x[1]), pk_bf16(x[2], x[3]), pk_bf16(x[4], x[5]), pk_bf16(x[6], x[7]));
    } else {
      float4* o = reinterpret_cast<float4*>(static_cast<float*>(dst) + r * ld + k0);
      o[0] = make_float4(x[0], x[1], x[2], x[3]);
      o[1] = make_float4(x[4], x[5], x[6], x[7]);
    }
  }
}

template <int WAVES, int CH>
void quantize_rows(const uint16_t* src, int64_t ld, int64_t rows, int64_t cols, uint8_t* codes, float* scales,
                   hipStream_t stream) {
  constexpr int kRows = WAVES < 4 ? 4 / WAVES : 1;
  int8_rows_quantize_kernel<WAVES, CH><<<(unsigned)((rows + kRows - 1) / kRows), 64 * WAVES * kRows, 0, stream>>>(
      src, ld, rows, (int)cols, codes, scales);
}

}  // namespace

hipError_t launch_int8_rows_quantize(const uint16_t* src, int64_t ld, int64_t rows, int64_t cols, uint8_t* codes,
                                     float* scales, hipStream_t stream) {
  if (rows == 0 || cols == 0) return hipSuccess;
  if (cols <= 512)
    quantize_rows<1, 1>(src, ld, rows, cols, codes, scales, stream);
  else if (cols <= 2048)
    quantize_rows<1, 4>(src, ld, rows, cols, codes, scales, stream);
  else if (cols <= 8192)
    quantize_rows<4, 4>(src, ld, rows, cols, codes, scales, stream);
  else if (cols <= 32768)
    quantize_rows<16, 4>(src, ld, rows, cols, codes, scales, stream);
  else
    int8_rows_quantize_long_kernel<<<(unsigned)rows, 1024, 0, stream>>>(src, ld, cols, codes, scales);
  return hipGetLastError();
}

hipError_t launch_int8_rows_dequant(const uint8_t* codes, const float* scales, int64_t rows, int64_t cols, void* dst,
                                    int dst_dtype, int64_t ld, hipStream_t stream) {
  const int64_t chunks = rows * (cols >> 3);
  if (!chunks) return hipSuccess;
  int64_t b = (chunks + kThreads - 1) / kThreads;
  if (b > (1 << 20)) b = 1 << 20;
  if (dst_dtype == 0)
    int8_rows_dequant_kernel<0><<<(unsigned)b, kThreads, 0, stream>>>(codes, scales, rows, cols, dst, ld);
  else
    int8_rows_dequant_kernel<1><<<(unsigned)b, kThreads, 0, stream>>>(codes, scales, rows, cols, dst, ld);
  return hipGetLastError();
}

}  // namespace q4
