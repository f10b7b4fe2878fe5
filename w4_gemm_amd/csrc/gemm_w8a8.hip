// gemm_w8a8.hip -- the product of two operands in 8-bit integers, with a scale
// for each token and each output channel (Q4_INT8_ROW x Q4_INT8_ROW):
//
//   C[m][n] = bf16(s_a[m] * s_w[n] * sum_k a[m][k] w[n][k])
//
// The sum is exact in 32-bit integers (|code| <= 128, K < 2^17), so no split of
// K changes the result.
#include "q4_launch.h"
#include "q4_lds.h"
#include "q4_mma.h"

namespace q4 {
namespace {

typedef int i32x4_t __attribute__((ext_vector_type(4)));

constexpr int kB = 64;     // rows of A and of W per workgroup
constexpr int kK = 128;    // k per stage

// Four waves of 32 x 32 outputs; both operands' rows staged in LDS, the 16-byte
// chunk c of row r at place c ^ (r & 7) so that the eight rows that a fragment
// read meets at once lie in different banks.
__global__ void __launch_bounds__(256)
w8a8_kernel(const uint8_t* __restrict__ a, const float* __restrict__ sa, int64_t M, const uint8_t* __restrict__ w,
            const float* __restrict__ sw, int64_t N, int64_t K, uint16_t* __restrict__ C, int64_t ldc) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[2][kB * kK];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t m0 = (int64_t)blockIdx.y * kB, n0 = (int64_t)blockIdx.x * kB;
  i32x4_t acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[i][j] = i32x4_t{0, 0, 0, 0};
  for (int64_t k0 = 0; k0 < K; k0 += kK) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int c = threadIdx.x + 256 * i, r = c >> 3, p = c & 7;
      const int64_t ra = m0 + r < M ? m0 + r : M - 1, rw = n0 + r < N ? n0 + r : N - 1;
      *reinterpret_cast<uint4*>(&lds[0][r * kK + 16 * (p ^ (r & 7))]) =
          *reinterpret_cast<const uint4*>(a + ra * K + k0 + 16 * p);
      *reinterpret_cast<uint4*>(&lds[1][r * kK + 16 * (p ^ (r & 7))]) =
          *reinterpret_cast<const uint4*>(w + rw * K + k0 + 16 * p);
    }
    __syncthreads();
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      i32x4_t fa[2], fw[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int p = 16 * ((4 * s + (lane >> 4)) ^ (lane & 7));
        fa[i] = *reinterpret_cast<const i32x4_t*>(&lds[0][(32 * (wave >> 1) + 16 * i + (lane & 15)) * kK + p]);
        fw[i] = *reinterpret_cast<const i32x4_t*>(&lds[1][(32 * (wave & 1) + 16 * i + (lane & 15)) * kK + p]);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[j], fa[i], acc[i][j], 0, 0, 0);
    }
  }
  // lane l, register r of tile (i, j): row 16i + l % 16, column 16j + 4 (l / 16) + r
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t m = m0 + 32 * (wave >> 1) + 16 * i + (lane & 15);
    if (m >= M) continue;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int64_t n = n0 + 32 * (wave & 1) + 16 * j + 4 * (lane >> 4) + r;
        if (n < N) C[m * ldc + n] = (uint16_t)pk_bf16((float)acc[i][j][r] * (sa[m] * sw[n]), 0.0f);
      }
  }
}

}  // namespace

hipError_t launch_gemm_w8a8(const uint8_t* a, const float* sa, int64_t M, const uint8_t* w, const float* sw, int64_t N,
                            int64_t K, uint16_t* C, int64_t ldc, hipStream_t stream) {
  const dim3 grid((unsigned)((N + kB - 1) / kB), (unsigned)((M + kB - 1) / kB));
  w8a8_kernel<<<grid, 256, 0, stream>>>(a, sa, M, w, sw, N, K, C, ldc);
  return hipGetLastError();
}

}  // namespace q4
