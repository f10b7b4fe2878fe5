// moe_grad.hip -- tokens sorted by expert and back, and the gradients of that
// path: a stable sort of any number of choices, the tokens' rows copied into
// expert order and summed back, the gradients of the gated combine and of the
// softmax gates.
//
//   sort      inv[t][j] = offsets[e] + #{(t', j') before (t, j) with the same e},
//             gather[inv[t][j]] = t; a choice outside 0 .. E-1 is dropped: inv -1
//   permute   xs[inv[t][j]] = x[t];      backward  dx[t] = sum_j dxs[inv[t][j]]
//   combine   out[t] = sum_j w[t][j] y[inv[t][j]];
//             backward  dy[inv[t][j]] = w[t][j] dout[t],
//                       dw[t][j] = sum_n dout[t][n] y[inv[t][j]][n]
//   gates     w[t][j] = p[ids[t][j]], p = softmax(logits[t]);
//             backward  dl[e] = p[e] (d[e] - sum_e' p[e'] d[e']),
//                       d[e] = sum of dw[t][j] over the j with ids[t][j] = e
//
// A dropped choice takes no part: its row is neither read nor written and its
// dw is 0.  Rows that no choice owns are left as they were.  Sums are in fp32
// in a fixed order, so results do not vary from run to run.
#include "q4_device.h"
#include "q4_launch.h"
#include "q4_mma.h"

namespace q4 {
namespace {

// The k rows of every token are more than the caches hold where it matters:
// written past them.  16385 tokens, 7 of 8 choices kept, 7168 columns: 339 ->
// 306 us, 1.88 GB at 6.1 TB/s.
__device__ __forceinline__ void store_past(uint16_t* p, uint4 v) {
  __builtin_nontemporal_store(__builtin_bit_cast(u32x4_t, v), reinterpret_cast<u32x4_t*>(p));
}

// ---- sort ------------------------------------------------------------------
// Workgroups take consecutive chunks of the flattened choices, their 16 waves
// consecutive parts of a chunk.  With more than one chunk a first kernel
// writes each chunk's counts per expert to the workspace and every workgroup
// of the second sums them over the chunks before its own (and over all, for
// the offsets): at most 256 chunks, so that this reads at most 256 E words per
// workgroup from L2.  Bound by latency: 8 choices 4.0 us, 131080 choices of 64
// experts 4.8 + 7.9 us.
constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / 64;
constexpr int64_t kSortMaxChunks = 256;
constexpr int64_t kSortOneChunk = 4096;    // choices one workgroup sorts by itself

int64_t sort_chunk(int64_t P) {
  if (P <= kSortOneChunk) return kSortOneChunk;
  const int64_t c = (P + kSortMaxChunks - 1) / kSortMaxChunks;
  return ((c + kSortThreads - 1) / kSortThreads) * kSortThreads;
}

__global__ void __launch_bounds__(kSortThreads)
moe_sort_count_kernel(const int32_t* __restrict__ ids, int64_t P, int E, int64_t chunk, uint32_t* __restrict__ counts) {
  extern __shared__ uint32_t lds[];
  for (int e = threadIdx.x; e < E; e += kSortThreads) lds[e] = 0u;
  __syncthreads();
  const int64_t begin = blockIdx.x * chunk, end = min(begin + chunk, P);
  for (int64_t i = begin + threadIdx.x; i < end; i += kSortThreads) {
    const int e = ids[i];
    if ((unsigned)e < (unsigned)E) atomicAdd(&lds[e], 1u);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kSortThreads) counts[(int64_t)blockIdx.x * E + e] = lds[e];
}

__global__ void __launch_bounds__(kSortThreads)
moe_sort_place_kernel(const int32_t* __restrict__ ids, int64_t P, int k, int E, int64_t chunk, int chunks,
                      const uint32_t* __restrict__ counts, int32_t* __restrict__ offsets,
                      int32_t* __restrict__ gather, int32_t* __restrict__ inv) {
  extern __shared__ uint32_t lds[];
  uint32_t* next = lds;                       // [16][E] the wave's next row per expert
  uint32_t* before = lds + kSortWaves * E;    // [E] choices of earlier chunks
  uint32_t* total = before + E;               // [E] choices of all chunks, then their offsets
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (int i = tid; i < (kSortWaves + 2) * E; i += kSortThreads) lds[i] = 0u;
  __syncthreads();

  const int64_t part = chunk / kSortWaves;    // a multiple of 64
  const int64_t begin = blockIdx.x * chunk + wave * part, end = min(begin + part, P);
  for (int64_t i = begin + lane; i < end; i += 64) {
    const int e = ids[i];
    if ((unsigned)e < (unsigned)E) atomicAdd(&next[wave * E + e], 1u);
  }
  if (chunks > 1) {
    // threads in groups of E share the chunks (E > 1024 does not occur)
    const int groups = max(kSortThreads / E, 1), g = tid / E;
    if (g < groups) {
      const int e = tid - g * E;
      uint32_t pre = 0, all = 0;
      for (int c = g; c < chunks; c += groups) {
        const uint32_t n = counts[(int64_t)c * E + e];
        all += n;
        if (c < (int)blockIdx.x) pre += n;
      }
      atomicAdd(&before[e], pre);
      atomicAdd(&total[e], all);
    }
  }
  __syncthreads();
  if (chunks == 1) {
    for (int e = tid; e < E; e += kSortThreads) {
      uint32_t n = 0;
      for (int w = 0; w < kSortWaves; ++w) n += next[w * E + e];
      total[e] = n;
    }
    __syncthreads();
  }
  // exclusive sums of the totals: lane l of wave 0 takes experts 16l .. 16l+15
  if (wave == 0) {
    const int e0 = lane * 16;
    uint32_t c[16], sum = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      c[i] = e0 + i < E ? total[e0 + i] : 0u;
      sum += c[i];
    }
    uint32_t x = sum;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const uint32_t y = __shfl_up(x, off);
      if (lane >= off) x += y;
    }
    uint32_t run = x - sum;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if (e0 + i < E) {
        total[e0 + i] = run;
        if (blockIdx.x == 0) offsets[e0 + i] = (int32_t)run;
      }
      run += c[i];
    }
    if (lane == 63 && blockIdx.x == 0) offsets[E] = (int32_t)x;
  }
  __syncthreads();
  for (int e = tid; e < E; e += kSortThreads) {
    uint32_t run = total[e] + before[e];
    for (int w = 0; w < kSortWaves; ++w) {
      const uint32_t n = next[w * E + e];
      next[w * E + e] = run;
      run += n;
    }
  }
  __syncthreads();

  // 64 choices at a time in order: a choice's rank among the wave's lanes with
  // the same expert, found by comparing the id bit by bit; the last of them
  // moves the expert's next row on
  uint32_t* mine = next + wave * E;
  int bits = 0;
  while ((1 << bits) < E) ++bits;
  const int64_t first = blockIdx.x * chunk + wave * part;
  for (int64_t i0 = first; i0 < end; i0 += 64) {
    const int64_t i = i0 + lane;
    const int e = i < end ? ids[i] : -1;
    const bool has = (unsigned)e < (unsigned)E;
    uint64_t same = __ballot(has);
    for (int b = 0; b < bits; ++b) {
      const bool bit = (e >> b) & 1;
      const uint64_t on = __ballot(has && bit);
      same &= bit ? on : ~on;
    }
    const uint64_t below = same & ((1ull << lane) - 1ull);
    const uint32_t base = has ? mine[e] : 0u;
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    if (has) {
      const int32_t pos = (int32_t)(base + (uint32_t)__popcll(below));
      if ((same >> lane) == 1ull) mine[e] = (uint32_t)pos + 1u;   // no lane above has this expert
      gather[pos] = (int32_t)(i / k);
      inv[i] = pos;
    } else if (i < end) {
      inv[i] = -1;
    }
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  }
}

// ---- permute and its gradient ------------------------------------------------
// 8 columns per thread, a workgroup per (token, 1024 columns): each token's row
// is read once and written to its k rows (reading through gather would read it
// k times).  Bound by HBM (store_past above; the gradient, 8192 tokens of 8
// rows, 203 us, 1.06 GB at 5.2 TB/s).
constexpr int kRowThreads = 128;
constexpr int kRowCols = kRowThreads * 8;

__global__ void __launch_bounds__(kRowThreads)
moe_permute_kernel(const uint16_t* __restrict__ x, int64_t ldx, const int32_t* __restrict__ inv, int k, int64_t K,
                   int64_t P, uint16_t* __restrict__ xs, int64_t ldxs, uint32_t slices) {
  const int64_t t = blockIdx.x / slices;
  const int64_t n = (int64_t)(blockIdx.x % slices) * kRowCols + threadIdx.x * 8;
  if (n >= K) return;
  const uint4 v = *reinterpret_cast<const uint4*>(x + t * ldx + n);
  for (int j = 0; j < k; ++j) {
    const int64_t p = inv[t * k + j];
    if (p >= 0 && p < P) store_past(xs + p * ldxs + n, v);
  }
}

__device__ __forceinline__ void add8(float (&a)[8], const uint4& v) {
  a[0] += bf16_lo(v.x); a[1] += bf16_hi(v.x);
  a[2] += bf16_lo(v.y); a[3] += bf16_hi(v.y);
  a[4] += bf16_lo(v.z); a[5] += bf16_hi(v.z);
  a[6] += bf16_lo(v.w); a[7] += bf16_hi(v.w);
}

// Eight rows' loads in flight at a time, added in choice order.
__global__ void __launch_bounds__(kRowThreads)
moe_permute_backward_kernel(const uint16_t* __restrict__ dxs, int64_t lds_, const int32_t* __restrict__ inv, int k,
                            int64_t K, int64_t P, uint16_t* __restrict__ dx, int64_t ldx, uint32_t slices) {
  const int64_t t = blockIdx.x / slices;
  const int64_t n = (int64_t)(blockIdx.x % slices) * kRowCols + threadIdx.x * 8;
  if (n >= K) return;
  float a[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
  for (int j0 = 0; j0 < k; j0 += 8) {
    uint4 v[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int64_t p = j0 + q < k ? inv[t * k + j0 + q] : -1;
      v[q] = p >= 0 && p < P ? *reinterpret_cast<const uint4*>(dxs + p * lds_ + n) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) add8(a, v[q]);
  }
  *reinterpret_cast<uint4*>(dx + t * ldx + n) =
      make_uint4(pk_bf16(a[0], a[1]), pk_bf16(a[2], a[3]), pk_bf16(a[4], a[5]), pk_bf16(a[6], a[7]));
}

// ---- the combine's gradient --------------------------------------------------
// A workgroup per token, a wave per choice (waves take every blockDim/64-th):
// the wave walks the row, so dw's sum stays inside it, and dout[t] is read from
// the cache by the other waves.  Bound by HBM: 8192 tokens of 8 choices, 7168
// columns, 394 us, 2.0 GB at 5.1 TB/s (a plain copy reaches 4.8).
template <bool GATES>
__global__ void __launch_bounds__(512)
moe_combine_backward_kernel(const uint16_t* __restrict__ dout, int64_t ldo, const uint16_t* __restrict__ y, int64_t ldy,
                            const int32_t* __restrict__ inv, const float* __restrict__ w, int k, int64_t N, int64_t P,
                            uint16_t* __restrict__ dy, int64_t lddy, float* __restrict__ dw) {
  const int64_t t = blockIdx.x;
  const int lane = threadIdx.x & 63;
  const uint16_t* d = dout + t * ldo;
  for (int j = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); j < k; j += blockDim.x >> 6) {
    const int64_t p = inv[t * k + j];
    float s = 0.0f;
    if (p >= 0 && p < P) {
      const float g = w[t * k + j];
      const uint16_t* yr = y + p * ldy;
      uint16_t* o = dy + p * lddy;
      for (int64_t n = lane * 8; n < N; n += 512) {
        const uint4 dv = *reinterpret_cast<const uint4*>(d + n);
        const uint32_t dwd[4] = {dv.x, dv.y, dv.z, dv.w};
        uint32_t r[4];
        uint4 yv = make_uint4(0u, 0u, 0u, 0u);
        if constexpr (GATES) yv = *reinterpret_cast<const uint4*>(yr + n);
        const uint32_t yw[4] = {yv.x, yv.y, yv.z, yv.w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float a = bf16_lo(dwd[q]), b = bf16_hi(dwd[q]);
          r[q] = pk_bf16(g * a, g * b);
          if constexpr (GATES) {
            s = __builtin_fmaf(a, bf16_lo(yw[q]), s);
            s = __builtin_fmaf(b, bf16_hi(yw[q]), s);
          }
        }
        store_past(o + n, make_uint4(r[0], r[1], r[2], r[3]));
      }
    }
    if constexpr (GATES) {
#pragma unroll
      for (int off = 32; off > 0; off >>= 1) s += __shfl_xor(s, off);
      if (lane == 0) dw[t * k + j] = s;
    }
  }
}

// ---- the gates' gradient -----------------------------------------------------
// One wave per token, the E <= 64 * PER logits in registers (PER 1, 4 or 16).
// A token whose logits are all -inf has no softmax; its gradient is written as
// 0.  A NaN among them is carried by the sum of the exponentials into the whole
// row (the maximum alone, which passes over NaN, cannot tell a row of NaN and
// -inf from one of -inf).  8192 tokens of 64 experts: 7 us.
constexpr int kTopkWaves = 4;

template <int PER>
__global__ void __launch_bounds__(64 * kTopkWaves)
moe_topk_backward_kernel(const float* __restrict__ logits, int64_t ld, int64_t T, int E, int k,
                         const int32_t* __restrict__ ids, const float* __restrict__ dw, float* __restrict__ dl,
                         int64_t lddl) {
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * kTopkWaves + (threadIdx.x >> 6);
  if (t >= T) return;
  float v[PER], d[PER];
  float m = -INFINITY;
  bool nan = false;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = lane + 64 * i;
    v[i] = e < E ? logits[t * ld + e] : -INFINITY;
    d[i] = 0.0f;
    m = fmaxf(m, v[i]);
    nan |= v[i] != v[i];
  }
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor(m, off));
  const bool none = m == -INFINITY && __ballot(nan) == 0;
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    v[i] = lane + 64 * i < E ? expf(v[i] - m) : 0.0f;
    s += v[i];
  }
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) s += __shfl_xor(s, off);
  // (k <= 32: lane j holds choice j)
  const int id = lane < k ? ids[t * k + lane] : -1;
  const float dwj = lane < k ? dw[t * k + lane] : 0.0f;
  for (int j = 0; j < k; ++j) {
    const int e = __shfl(id, j);
    const float g = __shfl(dwj, j);
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (e == lane + 64 * i && e < E) d[i] += g;
  }
  float c = 0.0f;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    v[i] = v[i] / s;
    if (lane + 64 * i < E) c = __builtin_fmaf(v[i], d[i], c);
  }
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) c += __shfl_xor(c, off);
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = lane + 64 * i;
    if (e < E) dl[t * lddl + e] = none ? 0.0f : v[i] * (d[i] - c);
  }
}

}  // namespace

size_t moe_sort_workspace(int64_t P, int32_t E) {
  const int64_t chunk = sort_chunk(P), chunks = (P + chunk - 1) / chunk;
  return chunks > 1 ? (size_t)chunks * (size_t)E * 4 : 0;
}

hipError_t launch_moe_sort(const int32_t* ids, int64_t T, int32_t k, int32_t E, int32_t* offsets, int32_t* gather,
                           int32_t* inv, uint32_t* workspace, hipStream_t stream) {
  const int64_t P = T * k, chunk = sort_chunk(P);
  const int chunks = (int)((P + chunk - 1) / chunk);
  if (chunks > 1) moe_sort_count_kernel<<<chunks, kSortThreads, (size_t)E * 4, stream>>>(ids, P, E, chunk, workspace);
  const size_t lds = (size_t)(kSortWaves + 2) * E * 4;
  const hipError_t attr = set_max_lds<&moe_sort_place_kernel>((size_t)(kSortWaves + 2) * 1024 * 4);
  if (attr != hipSuccess) return attr;
  moe_sort_place_kernel<<<chunks > 1 ? chunks : 1, kSortThreads, lds, stream>>>(
      ids, P, k, E, chunk, chunks > 1 ? chunks : 1, workspace, offsets, gather, inv);
  return hipGetLastError();
}

hipError_t launch_moe_permute(const uint16_t* x, int64_t ldx, const int32_t* inv, int64_t T, int32_t k, int64_t K,
                              int64_t P, uint16_t* xs, int64_t ldxs, hipStream_t stream) {
  const int64_t slices = (K + kRowCols - 1) / kRowCols;
  moe_permute_kernel<<<(unsigned)(T * slices), kRowThreads, 0, stream>>>(x, ldx, inv, k, K, P, xs, ldxs,
                                                                         (uint32_t)slices);
  return hipGetLastError();
}

hipError_t launch_moe_permute_backward(const uint16_t* dxs, int64_t lddxs, const int32_t* inv, int64_t T, int32_t k,
                                       int64_t K, int64_t P, uint16_t* dx, int64_t lddx, hipStream_t stream) {
  const int64_t slices = (K + kRowCols - 1) / kRowCols;
  moe_permute_backward_kernel<<<(unsigned)(T * slices), kRowThreads, 0, stream>>>(dxs, lddxs, inv, k, K, P, dx, lddx,
                                                                                  (uint32_t)slices);
  return hipGetLastError();
}

hipError_t launch_moe_combine_backward(const uint16_t* dout, int64_t ldo, const uint16_t* y, int64_t ldy,
                                       const int32_t* inv, const float* w, int64_t T, int32_t k, int64_t N, int64_t P,
                                       uint16_t* dy, int64_t lddy, float* dw, hipStream_t stream) {
  const unsigned threads = 64 * (unsigned)(k < 8 ? k : 8);
  if (dw)
    moe_combine_backward_kernel<true><<<(unsigned)T, threads, 0, stream>>>(dout, ldo, y, ldy, inv, w, k, N, P, dy,
                                                                          lddy, dw);
  else
    moe_combine_backward_kernel<false><<<(unsigned)T, threads, 0, stream>>>(dout, ldo, y, ldy, inv, w, k, N, P, dy,
                                                                           lddy, dw);
  return hipGetLastError();
}

hipError_t launch_moe_topk_backward(const float* logits, int64_t ld, int64_t T, int32_t E, int32_t k,
                                    const int32_t* ids, const float* dw, float* dl, int64_t lddl,
                                    hipStream_t stream) {
  const unsigned grid = (unsigned)((T + kTopkWaves - 1) / kTopkWaves);
  auto kernel = E <= 64 ? moe_topk_backward_kernel<1> : E <= 256 ? moe_topk_backward_kernel<4> : moe_topk_backward_kernel<16>;
  kernel<<<grid, 64 * kTopkWaves, 0, stream>>>(logits, ld, T, E, k, ids, dw, dl, lddl);
  return hipGetLastError();
}

}  // namespace q4
