// gemm_w8a8.hip -- the product of two operands in 8-bit integers, with a scale
// for each token and each output channel (Q4_INT8_ROW x Q4_INT8_ROW):
//
//   C[m][n] = bf16(s_a[m] * s_w[n] * sum_k a[m][k] w[n][k])
//
// The sum is exact in 32-bit integers (|code| <= 128, K < 2^17), so no split of
// K changes the result.
//
// Both operands are row-major.  Their rows are copied to LDS by direct
// global->LDS loads (1 KB per wave instruction, whole 128-byte lines of a row),
// the 16-byte chunk c of row r to place c ^ key(r): a copy permutes chunks within
// a line, and a fragment read meets eight rows of different keys at once.  So neither
// side has bank conflicts where a row is one line of 128 bytes (BK = 128, and the large
// blocks); longer rows begin at multiples of 256 bytes, a key of three bits keeps a
// read in one half of the banks, and each has 4 conflicts (1.4e6 in the 28672 x 8192
// product of one token, 0.7e6 in 33 x 8192 x 8192).
//
// v_mfma_i32_16x16x64_i8: lane l supplies row l % 16, k = 16 (l / 16) .. +15 of
// both operands.  The weight is the instruction's row operand, so a lane ends
// with 4 columns of one row of C; two tiles take the weight's rows
// 32 q + 8 (i / 4) + i % 4 and the same + 4 (i = l % 16), which leaves 8
// consecutive columns, 16 bytes of bf16, in a lane and 64 in four lanes.
#include "q4_launch.h"
#include "q4_lds.h"
#include "q4_mma.h"

#include <type_traits>

namespace q4 {
namespace {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x16_t __attribute__((ext_vector_type(16)));

struct Args {
  const uint8_t* a;
  const float* sa;
  const uint8_t* w;
  const float* sw;
  uint16_t* c;
  int64_t M, N, K, ldc;
  int whole;        // rows of C at multiples of 16 bytes
  uint32_t tm, tn;  // blocks of C
};

// Keys of a row of A (fragments take 16 rows in order) and of W (the order above).
__device__ __forceinline__ int key_a(int r) { return r & 7; }
__device__ __forceinline__ int key_w(int r) { return (r & 3) | ((r >> 1) & 4); }

__device__ __forceinline__ i32x4_t mma(i32x4_t w, i32x4_t a, i32x4_t c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(w, a, c, 0, 0, 0);
}

__device__ __forceinline__ i32x4_t read16(const uint8_t* p) { return *reinterpret_cast<const i32x4_t*>(p); }

// Eight columns n .. n + 7 of row m from two tiles' sums.
__device__ __forceinline__ void store8(const Args& p, int64_t m, int64_t n, i32x4_t lo, i32x4_t hi, float sa,
                                       const float* sw) {
  if (m >= p.M) return;
  const float4 u = *reinterpret_cast<const float4*>(sw), v = *reinterpret_cast<const float4*>(sw + 4);
  const uint32_t o[4] = {pk_bf16((float)lo[0] * (sa * u.x), (float)lo[1] * (sa * u.y)),
                         pk_bf16((float)lo[2] * (sa * u.z), (float)lo[3] * (sa * u.w)),
                         pk_bf16((float)hi[0] * (sa * v.x), (float)hi[1] * (sa * v.y)),
                         pk_bf16((float)hi[2] * (sa * v.z), (float)hi[3] * (sa * v.w))};
  uint16_t* c = p.c + m * p.ldc + n;
  if (p.whole && n + 8 <= p.N) {
    *reinterpret_cast<uint4*>(c) = make_uint4(o[0], o[1], o[2], o[3]);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (n + j < p.N) c[j] = (uint16_t)(o[j >> 1] >> (16 * (j & 1)));
  }
}

// The block of C of a workgroup: an XCD's workgroups (every eighth) take
// consecutive blocks of groups of `rows` block rows, so that those running at
// once share panels of both operands in its L2.
__device__ __forceinline__ void block_of(const Args& p, int rows, int64_t& bm, int64_t& bn) {
  const uint32_t tn = p.tn, tm = p.tm, t = tm * tn, b = blockIdx.x;
  const uint32_t lin = t % 8 == 0 ? (b % 8) * (t / 8) + b / 8 : b;
  const uint32_t group = rows * tn, first = lin / group * rows, in = lin % group;
  const uint32_t g = tm - first < (uint32_t)rows ? tm - first : (uint32_t)rows;
  bm = first + in % g;
  bn = in / g;
}

// ---- many rows ----------------------------------------------------------------
// 256 x 256 of C by four waves of 128 x 128 (4 x 4 tiles of v_mfma_i32_32x32x32_i8,
// 256 sums per lane, one wave per SIMD).  A stage is 128 k: 32 KB of A and 32 KB of
// W, which take turns in a ring of five places, all of the LDS.  A stage has two
// halves of 64 k; while the products of one run, one behind each of them a wave
// issues the reads of the next half's fragments into the other register set and
// its copies of stage u + 2: A's in the first half, into the place that W of stage
// u - 1 left, W's in the second, into that of A of stage u, which every wave has
// read by then.  One barrier per stage, in its middle.
// 4096 x 8192 x 8192: 207 to 221 us, 2.5 to 2.7 POPS, the instruction alone on random
// registers 3.3 to 3.6; passes without a pause 241 to 252 us.  The matrix
// pipe is busy in 78% of a CU's cycles, and the XCDs run those at 1.30 to 1.45 GHz:
// bound by the clock that the load leaves.  A block's stores are 8 of its 120 us.
// No faster: eight waves of 64 x 128 (two per SIMD), stages of 64 k in four places
// (lines of 64 bytes: 7% slower), lines asked for three to five stages ahead,
// groups of 2, 8 or 16 block rows per XCD (1, 0 and 9% slower).  16 x 16 x 64
// products do not fit: the compiler moves accumulators about.
// Fragments of 32 rows: lane l supplies row l % 32, k = 16 (l / 32) .. +15.  The
// weight's row for index i of a tile is 16 (i / 16) + 8 (i / 4 % 2) +
// 4 (i / 8 % 2) + i % 4, which leaves twice 8 consecutive columns in a lane.
constexpr int kBig = 256;
constexpr int kPlace = kBig * 128;
constexpr int kBigLds = 5 * kPlace;

// Keys of rows for these fragments: of the 16 rows that a read meets in two lines
// of 128 bytes, the even ones have different keys, and so have the odd ones.
__device__ __forceinline__ int key32_a(int r) { return (r >> 1) & 7; }
__device__ __forceinline__ int key32_w(int r) { return ((r >> 1) & 1) | ((r >> 2) & 2) | (r & 4); }

// A buffer descriptor of `rows` rows of K bytes (raw bytes, bounds checked).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_of(const uint8_t* p, int rows, int K) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p), 0, rows * K, 0x00020000);
}

__global__ void __launch_bounds__(256, 1)
w8a8_big_kernel(const Args p) {
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  int64_t bm, bn;
  block_of(p, 4, bm, bn);
  const int64_t m0 = bm * kBig, n0 = bn * kBig;
  const int K = (int)p.K, U = K >> 7;
  const int left_m = (int)(p.M - m0 < kBig ? p.M - m0 : kBig), left_n = (int)(p.N - n0 < kBig ? p.N - n0 : kBig);

  // copies: wave w takes rows 64 w .. of A and of W, eight rows at a time
  const uint8_t* src_a = uniform_ptr(p.a + m0 * K);
  const uint8_t* src_w = uniform_ptr(p.w + n0 * K);
  uint32_t at_a[8], at_w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = 64 * wave + 8 * i + (lane >> 3);
    at_a[i] = (uint32_t)(r < left_m ? r : left_m - 1) * (uint32_t)K + 16 * ((lane & 7) ^ key32_a(r));
    at_w[i] = (uint32_t)(r < left_n ? r : left_n - 1) * (uint32_t)K + 16 * ((lane & 7) ^ key32_w(r));
  }
  // (buffer loads: a descriptor of the rows, one offset per lane and copy, the stage's
  // offset in a scalar; nothing is computed per copy)
  const __amdgpu_buffer_rsrc_t rows_a = rows_of(src_a, left_m, K), rows_w = rows_of(src_w, left_n, K);
  auto copy_a = [&](int place, int u, int i) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rows_a, (lptr_t)(smem + place + (64 * wave + 8 * i) * 128), 16, at_a[i], u * 128, 0, 0);
  };
  auto copy_w = [&](int place, int u, int i) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rows_w, (lptr_t)(smem + place + (64 * wave + 8 * i) * 128), 16, at_w[i], u * 128, 0, 0);
  };

  const int i32 = lane & 31, half = lane >> 5;
  const int row_a = 128 * wm + i32;
  const int row_w = 128 * wn + 16 * (i32 >> 4) + 8 * ((i32 >> 2) & 1) + 4 * ((i32 >> 3) & 1) + (i32 & 3);
  const int pa = row_a * 128 + 16 * (half ^ key32_a(row_a)), pw = row_w * 128 + 16 * (half ^ key32_w(row_w));
  i32x4_t fa[2][8], fw[2][8];
  i32x16_t acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0;
  // fragment i of sixteen (A and W in turn, tile i / 4, k 32 (i / 2 % 2) ..) of half s
  auto read = [&](int place_a, int place_w, int s, int i) {
    const int f = i >> 1, x = 64 * s + 32 * (f & 1), t = (i >> 2) * 4096;
    if (i & 1) fw[s][f] = read16(smem + place_w + (pw ^ x) + t); else fa[s][f] = read16(smem + place_a + (pa ^ x) + t);
  };
  auto product = [&](int s, int i) {   // i of 32: k half i / 16, tile (i / 4 % 4, i % 4)
    const int h = i >> 4, r = (i >> 2) & 3, c = i & 3;
    acc[r][c] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fw[s][2 * c + h], fa[s][2 * r + h], acc[r][c], 0, 0, 0);
  };

  const int second = U > 1 ? 1 : 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) copy_a(0, 0, i);
#pragma unroll
  for (int i = 0; i < 8; ++i) copy_w(kPlace, 0, i);
#pragma unroll
  for (int i = 0; i < 8; ++i) copy_a(2 * kPlace, second, i);
#pragma unroll
  for (int i = 0; i < 8; ++i) copy_w(3 * kPlace, second, i);
  wait_vmcnt_lgkm0<16>();
  stage_barrier();
#pragma unroll
  for (int i = 0; i < 16; ++i) read(0, kPlace, 0, i);
  // places of A and W of this stage and the next, and the free one
  int a0 = 0, w0 = kPlace, a1 = 2 * kPlace, w1 = 3 * kPlace, spare = 4 * kPlace;
  for (int u = 0; u < U; ++u) {
    const int from = u + 2 < U ? u + 2 : U - 1;   // (past the end: the last stage again, never read)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      copy_a(spare, from, i);
      product(0, 4 * i);
      read(a0, w0, 1, 2 * i);
      product(0, 4 * i + 1);
      read(a0, w0, 1, 2 * i + 1);
      product(0, 4 * i + 2);
      product(0, 4 * i + 3);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x010, 1, 0);   // a copy
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);   // a product
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);   // a read
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x008, 2, 0);
    }
    // this wave's part of stage u + 1 is there (of the later copies only A's eight
    // may be on their way), and it has read all of stage u
    wait_vmcnt_lgkm0<8>();
    stage_barrier();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      copy_w(a0, from, i);
      product(1, 4 * i);
      read(a1, w1, 0, 2 * i);
      product(1, 4 * i + 1);
      read(a1, w1, 0, 2 * i + 1);
      product(1, 4 * i + 2);
      product(1, 4 * i + 3);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x010, 1, 0);   // a copy
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);   // a product
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);   // a read
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x008, 2, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
    const int a2 = spare, w2 = a0;
    spare = w0;
    a0 = a1;
    w0 = w1;
    a1 = a2;
    w1 = w2;
  }

  // the scales, where the stages were
  wait_vmcnt<0>();
  __syncthreads();
  float* scale_a = reinterpret_cast<float*>(smem);
  float* scale_w = scale_a + kBig;
  {
    const int t = threadIdx.x;
    scale_a[t] = p.sa[m0 + (t < left_m ? t : left_m - 1)];
    scale_w[t] = p.sw[n0 + (t < left_n ? t : left_n - 1)];
  }
  __syncthreads();
  // lane l, register 4 q + e of tile (i, j): row 32 i + l % 32, column 32 j + 16 (q / 2) + 8 (l / 32) + 4 (q % 2) + e
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 128 * wm + 32 * i + i32;
    const float s = scale_a[r];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int n = 128 * wn + 32 * j + 16 * q + 8 * half;
        const i32x16_t v = acc[i][j];
        store8(p, m0 + r, n0 + n, i32x4_t{v[8 * q], v[8 * q + 1], v[8 * q + 2], v[8 * q + 3]},
               i32x4_t{v[8 * q + 4], v[8 * q + 5], v[8 * q + 6], v[8 * q + 7]}, s, scale_w + n);
      }
  }
}

// ---- fewer rows ----------------------------------------------------------------
// WM x WN x WK waves of 16 TM x 32 TN outputs; the WK waves of a place share its k
// and add their sums through LDS at the end.  Stages of BK k in S buffers, S - 1
// of them on their way.
template <int WM, int WN, int WK, int TM, int TN, int BK, int S>
struct Tile {
  static constexpr int kWaves = WM * WN * WK, kThreads = 64 * kWaves;
  static constexpr int kM = 16 * TM * WM, kN = 32 * TN * WN, kRows = kM + kN;
  static constexpr int kStage = kRows * BK;
  static constexpr int kCopiesA = kM * BK / 1024 / kWaves, kCopiesW = kN * BK / 1024 / kWaves;   // of a wave per stage
  static constexpr size_t kLds = (size_t)S * kStage + (size_t)kRows * 4;
  static_assert(kM * BK % (1024 * kWaves) == 0 && kN * BK % (1024 * kWaves) == 0, "whole copies for every wave");
  static_assert(BK % (64 * WK) == 0 && (WK - 1) * WM * WN * TM * TN * 2048 <= S * kStage, "sums fit into the stages");
};

template <int WM, int WN, int WK, int TM, int TN, int BK, int S>
__global__ void __launch_bounds__((Tile<WM, WN, WK, TM, TN, BK, S>::kThreads))
w8a8_tile_kernel(const Args p) {
  using T = Tile<WM, WN, WK, TM, TN, BK, S>;
  constexpr int kChunks = BK / 16, kCopyRows = 1024 / BK, kSteps = BK / 64 / WK;
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  float* scale_a = reinterpret_cast<float*>(smem + (size_t)S * T::kStage);
  float* scale_w = scale_a + T::kM;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wk = wave % WK, wn = wave / WK % WN, wm = wave / (WK * WN);
  int64_t bm, bn;
  block_of(p, 4, bm, bn);
  const int64_t m0 = bm * T::kM, n0 = bn * T::kN;
  const int K = (int)p.K, U = (K + BK - 1) / BK;
  const int left_m = (int)(p.M - m0 < T::kM ? p.M - m0 : T::kM), left_n = (int)(p.N - n0 < T::kN ? p.N - n0 : T::kN);

  // Copy i of a wave: W's first, then A's, each kCopyRows rows; those behind the last
  // row take it again.  (Without the copies of A that are only such rows, a third of
  // all for one row of 28672 x 8192: 38.9 us for 39.0.)
  constexpr int kCopies = T::kCopiesW + T::kCopiesA;
  const uint8_t* src_w = uniform_ptr(p.w + n0 * K);
  const uint8_t* src_a = uniform_ptr(p.a + m0 * K);
  uint32_t row_at[kCopies], chunk_at[kCopies];
#pragma unroll
  for (int i = 0; i < kCopies; ++i) {
    const bool is_w = i < T::kCopiesW;
    const int r = ((is_w ? i : i - T::kCopiesW) * T::kWaves + wave) * kCopyRows + lane / kChunks;
    const int left = is_w ? left_n : left_m;
    row_at[i] = (uint32_t)(r < left ? r : left - 1) * (uint32_t)K;
    chunk_at[i] = 16 * ((lane % kChunks) ^ (is_w ? key_w(r) : key_a(r)));
  }
  auto copy = [&](int u) {
    uint8_t* d = smem + (u % S) * T::kStage + wave * 1024;
    const int64_t k0 = (int64_t)u * BK;
    const uint32_t left = (uint32_t)(K - k0);
#pragma unroll
    for (int i = 0; i < kCopies; ++i) {
      const bool is_w = i < T::kCopiesW;
      // (in the last stage of a K that is no multiple, chunks behind it read its first one, and are not used)
      const uint32_t c = BK == 128 || chunk_at[i] < left ? chunk_at[i] : 0u;
      copy16_to_lds((is_w ? src_w : src_a) + k0 + (row_at[i] + c),
                    d + (is_w ? T::kM * BK + i * T::kWaves * 1024 : (i - T::kCopiesW) * T::kWaves * 1024));
    }
  };
  // loads on their way when stage u is needed: those of the later stages that were begun
  auto wait = [&](int u) {
    const int later = U - 1 - u < S - 2 ? U - 1 - u : S - 2;
    if (later <= 0) wait_vmcnt_lgkm0<0>();
    else if (later == 1) wait_vmcnt_lgkm0<kCopies>();
    else wait_vmcnt_lgkm0<2 * kCopies>();
  };
  static_assert(S >= 2 && S <= 4, "the counts above");

  for (int t = threadIdx.x; t < T::kRows; t += T::kThreads)
    scale_a[t] = t < T::kM ? p.sa[m0 + (t < left_m ? t : left_m - 1)]
                           : p.sw[n0 + (t - T::kM < left_n ? t - T::kM : left_n - 1)];
#pragma unroll
  for (int u = 0; u < S - 1; ++u)
    if (u < U) copy(u);

  const int i16 = lane & 15, g = lane >> 4;
  const int row_a = 16 * TM * wm + i16, row_w = 32 * TN * wn + 8 * (i16 >> 2) + (i16 & 3);
  const int pa = row_a * BK, pw = (T::kM + row_w) * BK, ka = key_a(row_a), kw = key_w(row_w);
  i32x4_t acc[TM][2 * TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < 2 * TN; ++j) acc[i][j] = i32x4_t{0, 0, 0, 0};
  for (int u = 0; u < U; ++u) {
    wait(u);
    stage_barrier();
    if (u + S - 1 < U) copy(u + S - 1);
    const uint8_t* b = smem + (u % S) * T::kStage;
    const int left = K - u * BK;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int step = wk * kSteps + s;
      if (BK > 128 && step * 64 >= left) break;
      i32x4_t fa[TM], fw[2 * TN];
#pragma unroll
      for (int j = 0; j < 2 * TN; ++j)
        fw[j] = read16(b + pw + 16 * ((4 * step + g) ^ kw) + (32 * (j >> 1) + 4 * (j & 1)) * BK);
#pragma unroll
      for (int i = 0; i < TM; ++i) fa[i] = read16(b + pa + 16 * ((4 * step + g) ^ ka) + 16 * i * BK);
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < 2 * TN; ++j) acc[i][j] = mma(fw[j], fa[i], acc[i][j]);
    }
  }
  if constexpr (WK > 1) {
    __syncthreads();     // every stage has been read
    i32x4_t* side = reinterpret_cast<i32x4_t*>(smem);
    const int place = (wm * WN + wn) * (WK - 1);
    if (wk > 0) {
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < 2 * TN; ++j) side[((place + wk - 1) * TM * 2 * TN + i * 2 * TN + j) * 64 + lane] = acc[i][j];
    }
    __syncthreads();
    if (wk > 0) return;
#pragma unroll
    for (int v = 0; v < WK - 1; ++v)
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < 2 * TN; ++j) acc[i][j] += side[((place + v) * TM * 2 * TN + i * 2 * TN + j) * 64 + lane];
  }
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int r = 16 * (TM * wm + i) + i16;
    const float s = scale_a[r];
#pragma unroll
    for (int q = 0; q < TN; ++q) {
      const int n = 32 * (TN * wn + q) + 8 * g;
      store8(p, m0 + r, n0 + n, acc[i][2 * q], acc[i][2 * q + 1], s, scale_w + n);
    }
  }
}

template <int WM, int WN, int WK, int TM, int TN, int BK, int S>
hipError_t run_tile(const Args& p, hipStream_t stream) {
  using T = Tile<WM, WN, WK, TM, TN, BK, S>;
  const hipError_t attr = set_max_lds<&w8a8_tile_kernel<WM, WN, WK, TM, TN, BK, S>>(T::kLds);
  if (attr != hipSuccess) return attr;
  w8a8_tile_kernel<WM, WN, WK, TM, TN, BK, S><<<p.tm * p.tn, T::kThreads, T::kLds, stream>>>(p);
  return hipGetLastError();
}

hipError_t run_big(const Args& p, hipStream_t stream) {
  const hipError_t attr = set_max_lds<&w8a8_big_kernel>(kBigLds);
  if (attr != hipSuccess) return attr;
  w8a8_big_kernel<<<p.tm * p.tn, 256, kBigLds, stream>>>(p);
  return hipGetLastError();
}

// ---- which block ---------------------------------------------------------------
// The block whose estimated time is least.  256 CUs take a round of up to 256
// workgroups in `one`, of up to 512 in `two` (two on a CU; twice `one` where the LDS
// holds one), in units of 0.01 us per 128 k, plus `fixed` for the first copies and
// the stores, all measured on 8192 x 8192, 2048 x 7168 and 7168 x 2048 weights.  So
// 33 rows of 8192 x 8192 take 256 workgroups of 48 x 32 (15.3 us; 256 of 32 x 64:
// 16.1, 768 of 16 x 32: 21), 256 rows 256 of 128 x 64 (30 us; 512 of 64 x 64: 37,
// 128 of 128 x 128: 44), 1024 rows 512 of 128 x 128 (70 us; 128 of 256 x 256: 82),
// 2048 rows 256 of 256 x 256 (108 us; 1024 of 128 x 128: 137).  Up to 256
// workgroups, which have a CU each, have longer or more stages on the way: one row
// of 2048 x 7168 6.0 us and 6.9 without, 64 rows of 8192 x 8192 17.5 and 18.6, 100
// rows 20.4 and 21.8, 256 rows 30.0 and 32.4, 512 rows 46 and 56.
struct Choice {
  int rows, cols, one, two, fixed;
  hipError_t (*few)(const Args&, hipStream_t);    // up to 256 workgroups
  hipError_t (*run)(const Args&, hipStream_t);
};

const Choice kChoices[] = {
    {16, 32, 12, 20, 150, run_tile<1, 1, 8, 1, 1, 1024, 3>, run_tile<1, 1, 8, 1, 1, 512, 3>},
    {32, 32, 13, 26, 150, run_tile<1, 1, 8, 2, 1, 512, 3>, run_tile<1, 1, 8, 2, 1, 512, 3>},
    {48, 32, 21, 42, 200, run_tile<1, 1, 8, 3, 1, 512, 3>, run_tile<1, 1, 8, 3, 1, 512, 3>},
    {32, 64, 22, 40, 200, run_tile<1, 2, 4, 2, 1, 512, 3>, run_tile<1, 2, 4, 2, 1, 256, 3>},
    {64, 64, 31, 53, 200, run_tile<2, 2, 2, 2, 1, 256, 4>, run_tile<2, 2, 2, 2, 1, 128, 4>},
    {128, 64, 41, 78, 400, run_tile<2, 2, 2, 4, 1, 256, 3>, run_tile<2, 2, 1, 4, 1, 128, 3>},
    {128, 128, 70, 106, 500, run_tile<2, 2, 1, 4, 2, 128, 3>, run_tile<2, 2, 1, 4, 2, 128, 2>},
    {256, 256, 166, 332, 800, run_big, run_big},
};

const Choice& choose(int64_t M, int64_t N, int64_t K, int64_t& tm, int64_t& tn) {
  const Choice* best = nullptr;
  int64_t least = 0;
  for (const Choice& c : kChoices) {
    const int64_t blocks = ((M + c.rows - 1) / c.rows) * ((N + c.cols - 1) / c.cols);
    const int64_t rest = blocks % 512, rounds = blocks / 512 * c.two + (rest > 256 ? c.two : rest > 0 ? c.one : 0);
    const int64_t t = rounds * (K / 128) + c.fixed;
    if (!best || t < least) {
      best = &c;
      least = t;
    }
  }
  tm = (M + best->rows - 1) / best->rows;
  tn = (N + best->cols - 1) / best->cols;
  return *best;
}

}  // namespace

void w8a8_plan(int64_t M, int64_t N, int64_t K, int32_t& rows, int32_t& cols, int64_t& workgroups) {
  int64_t tm = 0, tn = 0;
  const Choice& c = choose(M, N, K, tm, tn);
  rows = c.rows;
  cols = c.cols;
  workgroups = tm * tn;
}

hipError_t launch_gemm_w8a8(const uint8_t* a, const float* sa, int64_t M, const uint8_t* w, const float* sw, int64_t N,
                            int64_t K, uint16_t* C, int64_t ldc, hipStream_t stream) {
  Args p{a, sa, w, sw, C, M, N, K, ldc, (reinterpret_cast<uintptr_t>(C) & 15) == 0 && (ldc % 8 == 0 || M == 1), 0, 0};
  int64_t tm = 0, tn = 0;
  const Choice& c = choose(M, N, K, tm, tn);
  if (tm * tn >= (int64_t)1 << 23) return hipErrorInvalidConfiguration;   // 2^32 threads: no C that large exists
  p.tm = (uint32_t)tm;
  p.tn = (uint32_t)tn;
  return (tm * tn <= 256 ? c.few : c.run)(p, stream);
}

}  // namespace q4
