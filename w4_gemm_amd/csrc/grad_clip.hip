// grad_clip.hip -- the norm over all gradients of a step and the gradients
// scaled down to a largest norm.
//
//   norm = sqrt(sum over all tensors of g^2)
//   out  = g * min(1, max_norm / (norm + 1e-6))
//
// Squares are added in 64 bits: fp32 gradients neither overflow (1e38^2) nor
// vanish (1e-30^2) in them, and the sums of the workgroups are added in an order
// that sizes and alignment alone decide.  A launch takes up to kTensors tensors; their
// pointers and sizes travel in the kernel's arguments, so that a captured graph
// keeps them.
#include "q4_launch.h"
#include "q4_mma.h"
#include "q4_row8.h"

namespace q4 {
namespace {

constexpr int kThreads = 256;
constexpr int kTensors = 128;           // 29 bytes each of a kernel's 4096 bytes of arguments
constexpr int64_t kChunk = 1 << 15;     // bytes of a tensor that a workgroup takes at a time
constexpr int kBlocks = 1024;           // workgroups of a launch at most (512: 14% slower, 2048: 5%)
constexpr int64_t kCached = (int64_t)256 << 20;   // bytes of the memory-side cache

struct Table {
  const uint8_t* in[kTensors];
  uint8_t* out[kTensors];
  int64_t count[kTensors];      // values
  int32_t chunk[kTensors + 1];  // first chunk of each tensor; the last entry: all chunks
  uint8_t f32[kTensors];
  int32_t n;
};

// The tensor that a chunk belongs to (empty tensors have none).
__device__ __forceinline__ int tensor_of(const Table& t, int chunk) {
  int lo = 0, hi = t.n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (t.chunk[mid] <= chunk) lo = mid; else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ double block_sum(double s) {
  __shared__ double part[kThreads / 64];
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) s += __shfl_xor(s, off);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = s;
  __syncthreads();
  s = 0.0;
#pragma unroll
  for (int w = 0; w < kThreads / 64; ++w) s += part[w];
  return s;
}

__device__ __forceinline__ void add_square(double& s, float v) { s = __builtin_fma((double)v, (double)v, s); }

// Values [at, end) of tensor i that a chunk covers.  Chunks are cut at multiples
// of 16 bytes of address, so the first one may be short.
template <int SIZE>
__device__ __forceinline__ void chunk_range(const Table& t, int i, int chunk, int64_t& at, int64_t& end) {
  const int64_t head = (int64_t)((reinterpret_cast<uintptr_t>(t.in[i]) & 15) / SIZE);   // values missing in front
  const int64_t c = chunk - t.chunk[i];
  at = c * (kChunk / SIZE) - head;
  end = at + kChunk / SIZE;
  if (at < 0) at = 0;
  if (end > t.count[i]) end = t.count[i];
}

template <int SIZE, bool PAST>
__device__ __forceinline__ double squares(const uint8_t* p, int64_t at, int64_t end) {
  constexpr int kPer = 16 / SIZE;
  double s = 0.0;
  auto one = [&](int64_t k) {
    if constexpr (SIZE == 4)
      add_square(s, reinterpret_cast<const float*>(p)[k]);
    else
      add_square(s, bf16_lo(reinterpret_cast<const uint16_t*>(p)[k]));
  };
  // values up to a 16-byte boundary, whole pieces, values behind the last one
  const int64_t off = (int64_t)((16 - (reinterpret_cast<uintptr_t>(p + at * SIZE) & 15)) & 15) / SIZE;
  const int64_t body = at + off < end ? at + off : end, pieces = (end - body) / kPer, tail = body + pieces * kPer;
  if (threadIdx.x < body - at) one(at + threadIdx.x);
  if (threadIdx.x < end - tail) one(tail + threadIdx.x);
  const uint4* v = reinterpret_cast<const uint4*>(p + body * SIZE);
#pragma unroll 4
  for (int64_t q = threadIdx.x; q < pieces; q += kThreads) {
    const uint4 u = load16<PAST>(v + q);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (SIZE == 4) {
        add_square(s, u2f(w[j]));
      } else {
        add_square(s, bf16_lo(w[j]));
        add_square(s, bf16_hi(w[j]));
      }
    }
  }
  return s;
}

// PAST: read past the caches, where the gradients are more than they hold (3.88 GB in
// 545 to 590 us, 6.6 to 7.1 TB/s, 662 without where it took 586 with); fewer are read
// again from there by the clipping.
template <bool PAST>
__global__ void __launch_bounds__(kThreads)
grad_square_kernel(const Table t, double* __restrict__ sums) {
  double s = 0.0;
  for (int chunk = blockIdx.x; chunk < t.chunk[t.n]; chunk += gridDim.x) {
    const int i = tensor_of(t, chunk);
    int64_t at, end;
    if (t.f32[i]) {
      chunk_range<4>(t, i, chunk, at, end);
      s += squares<4, PAST>(t.in[i], at, end);
    } else {
      chunk_range<2>(t, i, chunk, at, end);
      s += squares<2, PAST>(t.in[i], at, end);
    }
  }
  s = block_sum(s);
  if (threadIdx.x == 0) sums[blockIdx.x] = s;
}

// Sums of squares up to which every workgroup of the clipping adds them for itself:
// those of one full launch.  More are added once, by a launch of one workgroup, and the
// clipping reads its norm, since all workgroups of all launches would read the sums of
// all launches, a time with the square of the tensors' number.  Tensors of 256 KB, in
// a graph: 20 take 10.3 us and would take 11.5 with that launch, 129 29.6 (29.2 without
// it), 300 59.3 (61.7), 20000 3.8 ms (14.7).
constexpr int kOwnSums = kBlocks;

// The norm from the workgroups' sums, added by every caller in the same order.
__device__ __forceinline__ double norm_of(const double* sums, int count) {
  double s = 0.0;
  for (int i = threadIdx.x; i < count; i += kThreads) s += sums[i];
  return sqrt(block_sum(s));
}

// norm, whole: either may be NULL.
__global__ void __launch_bounds__(kThreads)
grad_norm_kernel(const double* __restrict__ sums, int count, float* __restrict__ norm, double* __restrict__ whole) {
  const double n = norm_of(sums, count);
  if (threadIdx.x != 0) return;
  if (norm) *norm = (float)n;
  if (whole) *whole = n;
}

// The factor stays in 64 bits: where the norm passes fp32's range it is itself
// below fp32's least normal number.
__device__ __forceinline__ float times(float v, double by) { return (float)((double)v * by); }

template <int SIZE>
__device__ __forceinline__ void scale(const uint8_t* p, uint8_t* o, int64_t at, int64_t end, double by) {
  constexpr int kPer = 16 / SIZE;
  auto one = [&](int64_t k) {
    if constexpr (SIZE == 4) {
      reinterpret_cast<float*>(o)[k] = times(reinterpret_cast<const float*>(p)[k], by);
    } else {
      const float v = times(bf16_lo(reinterpret_cast<const uint16_t*>(p)[k]), by);
      reinterpret_cast<uint16_t*>(o)[k] = (uint16_t)pk_bf16(v, 0.0f);
    }
  };
  if (((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(o)) & 15) != 0) {   // no common 16-byte pieces
    for (int64_t k = at + threadIdx.x; k < end; k += kThreads) one(k);
    return;
  }
  const int64_t off = (int64_t)((16 - (reinterpret_cast<uintptr_t>(p + at * SIZE) & 15)) & 15) / SIZE;
  const int64_t body = at + off < end ? at + off : end, pieces = (end - body) / kPer, tail = body + pieces * kPer;
  if (threadIdx.x < body - at) one(at + threadIdx.x);
  if (threadIdx.x < end - tail) one(tail + threadIdx.x);
  const uint4* v = reinterpret_cast<const uint4*>(p + body * SIZE);
  uint4* w = reinterpret_cast<uint4*>(o + body * SIZE);
#pragma unroll 4
  for (int64_t q = threadIdx.x; q < pieces; q += kThreads) {
    const uint4 u = load16<true>(v + q);
    uint32_t x[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (SIZE == 4)
        x[j] = f2u(times(u2f(x[j]), by));
      else
        x[j] = pk_bf16(times(bf16_lo(x[j]), by), times(bf16_hi(x[j]), by));
    }
    store16<true>(w + q, make_uint4(x[0], x[1], x[2], x[3]));
  }
}

// Read and written past the caches (3.88 GB each way in 1376 us, 5.6 TB/s, 1436
// without in turn on one card; 1395 to 1452 behind the squares; from the last chunk to the first, to find what the squares read last in
// the memory-side cache: no faster).
// FROM: the norm is the caller's, was made from the sums (and lies at `sums`), or
// every workgroup makes it from them (in the same order, so the same one) and the
// first writes it down.
enum { kFromCaller, kFromWhole, kFromSums };
template <int FROM>
__global__ void __launch_bounds__(kThreads)
grad_clip_kernel(const Table t, const double* __restrict__ sums, int count, const float* __restrict__ given,
                 float max_norm, float* __restrict__ norm, int in_place) {
  const double n = FROM == kFromCaller ? (double)*given : FROM == kFromWhole ? *sums : norm_of(sums, count);
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)n;
  double by = (double)max_norm / (n + 1e-6);
  if (by > 1.0) by = 1.0;               // (NaN stays NaN)
  if (in_place && by == 1.0) return;    // nothing changes
  for (int chunk = blockIdx.x; chunk < t.chunk[t.n]; chunk += gridDim.x) {
    const int i = tensor_of(t, chunk);
    int64_t at, end;
    if (t.f32[i]) {
      chunk_range<4>(t, i, chunk, at, end);
      scale<4>(t.in[i], t.out[i], at, end, by);
    } else {
      chunk_range<2>(t, i, chunk, at, end);
      scale<2>(t.in[i], t.out[i], at, end, by);
    }
  }
}

int64_t chunks_of(const void* p, int64_t count, int f32) {
  if (!count) return 0;
  const int64_t head = (int64_t)(reinterpret_cast<uintptr_t>(p) & 15);
  return (head + count * (f32 ? 4 : 2) + kChunk - 1) / kChunk;
}

// The table of tensors [from, from + kTensors), and its chunks.
int64_t fill(Table& t, const GradList& g, int64_t from, void* const* out) {
  t.n = (int32_t)(g.n - from < kTensors ? g.n - from : kTensors);
  int64_t chunks = 0;
  for (int i = 0; i < t.n; ++i) {
    t.in[i] = static_cast<const uint8_t*>(g.data[from + i]);
    t.out[i] = static_cast<uint8_t*>(out ? out[from + i] : const_cast<void*>(g.data[from + i]));
    t.count[i] = g.count[from + i];
    t.f32[i] = g.dtype[from + i] != 0;
    t.chunk[i] = (int32_t)chunks;
    chunks += chunks_of(g.data[from + i], g.count[from + i], g.dtype[from + i]);
  }
  t.chunk[t.n] = (int32_t)chunks;
  return chunks;
}

unsigned blocks_of(int64_t chunks) { return (unsigned)(chunks < kBlocks ? chunks : kBlocks); }

// Sums of squares of all tensors, kBlocks places for each launch; how many.
hipError_t squares_of_all(const GradList& g, double* sums, int* count, hipStream_t stream) {
  *count = 0;
  int64_t bytes = 0;
  for (int64_t i = 0; i < g.n; ++i) bytes += g.count[i] * (g.dtype[i] ? 4 : 2);
  auto kernel = bytes > kCached ? grad_square_kernel<true> : grad_square_kernel<false>;
  for (int64_t from = 0; from < g.n; from += kTensors) {
    Table t;
    const int64_t chunks = fill(t, g, from, nullptr);
    if (!chunks) continue;
    kernel<<<blocks_of(chunks), kThreads, 0, stream>>>(t, sums + *count);
    *count += (int)blocks_of(chunks);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

// The sums of every launch and, behind them, the norm in 64 bits.
size_t grad_workspace(int64_t n) { return n ? (size_t)((n + kTensors - 1) / kTensors) * kBlocks * 8 + 8 : 0; }

// Chunks are counted in 32 bits.
bool grad_fits(const GradList& g) {
  for (int64_t from = 0; from < g.n; from += kTensors) {
    int64_t chunks = 0;
    for (int64_t i = from; i < g.n && i < from + kTensors; ++i) {
      chunks += chunks_of(g.data[i], g.count[i], g.dtype[i]);
      if (chunks >= ((int64_t)1 << 31) - kBlocks) return false;
    }
  }
  return true;
}

hipError_t launch_grad_norm(const GradList& g, float* norm, double* sums, hipStream_t stream) {
  int count = 0;
  const hipError_t e = squares_of_all(g, sums, &count, stream);
  if (e != hipSuccess) return e;
  grad_norm_kernel<<<1, kThreads, 0, stream>>>(sums, count, norm, nullptr);
  return hipGetLastError();
}

hipError_t launch_grad_clip(const GradList& g, void* const* out, const float* given, float max_norm, float* norm,
                            double* sums, hipStream_t stream) {
  int count = 0;
  auto kernel = grad_clip_kernel<kFromCaller>;
  if (!given) {
    hipError_t e = squares_of_all(g, sums, &count, stream);
    if (e != hipSuccess) return e;
    kernel = grad_clip_kernel<kFromSums>;
    if (count > kOwnSums || count == 0) {   // (no launch of the clipping writes the norm of no values)
      double* whole = count ? sums + count : nullptr;
      if (norm || count) grad_norm_kernel<<<1, kThreads, 0, stream>>>(sums, count, norm, whole);
      e = hipGetLastError();
      if (e != hipSuccess) return e;
      kernel = grad_clip_kernel<kFromWhole>;
      sums = whole;
      norm = nullptr;
    }
  }
  for (int64_t from = 0; from < g.n; from += kTensors) {
    Table t;
    const int64_t chunks = fill(t, g, from, out);
    if (!chunks) continue;
    kernel<<<blocks_of(chunks), kThreads, 0, stream>>>(t, sums, count, given, max_norm, norm, out == nullptr);
    norm = nullptr;   // (written by the first)
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace q4
