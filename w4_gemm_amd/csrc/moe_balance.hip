// moe_balance.hip -- a router's balance loss, the choices that each expert
// received, and the gradient for the router's logits.
//
// With p = softmax of a token's logits, n the tokens that count (all, or those
// that the mask keeps), c[e] the choices of expert e among theirs and P[e] the
// sum of p[e] over them:
//
//   slope[e] = coef E c[e] / (k n^2)        loss = sum_e slope[e] P[e]
//   dlogits[t][e] = dloss p[e] (slope[e] - sum_e' p[e'] slope[e'])
//
// (the counts are whole numbers and have no gradient).  Workgroups walk over the
// tokens and write their sums of p, their counts and their tokens to the
// workspace; a second kernel adds those in order, in 64 bits, so the results do
// not vary.
#include "q4_launch.h"
#include "q4_row8.h"

namespace q4 {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kBlocks = 256;         // workgroups of the first kernel at most

// LPT lanes hold a token's E <= LPT * PER logits, lane i of them the experts
// i, i + LPT, ...
template <int LPT>
__device__ __forceinline__ float part_max(float v) {
#pragma unroll
  for (int off = LPT / 2; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor(v, off));
  return v;
}
template <int LPT>
__device__ __forceinline__ float part_sum(float v) {
#pragma unroll
  for (int off = LPT / 2; off > 0; off >>= 1) v += __shfl_xor(v, off);
  return v;
}

// Softmax of the token's logits v; all zeros where every logit is -inf, NaN
// where one is NaN (the sum carries it: a maximum passes over NaN).
template <int LPT, int PER>
__device__ __forceinline__ void softmax(float (&v)[PER], int sub, int E) {
  float m = v[0];
#pragma unroll
  for (int i = 1; i < PER; ++i) m = fmaxf(m, v[i]);
  m = part_max<LPT>(m);
  const float from = m == -INFINITY ? 0.0f : m;
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    v[i] = sub + LPT * i < E ? expf(v[i] - from) : 0.0f;
    s += v[i];
  }
  s = part_sum<LPT>(s);
  const float by = s == 0.0f ? 0.0f : 1.0f / s;
#pragma unroll
  for (int i = 0; i < PER; ++i) v[i] *= by;
}

template <int LPT, int PER>
__global__ void __launch_bounds__(kThreads)
moe_balance_kernel(const BalanceArgs a) {
  constexpr int kTokens = 64 / LPT;   // of a wave at once
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, sub = lane % LPT;
  const int E = a.E;
  extern __shared__ uint32_t lds[];
  uint32_t* count = lds;                                    // [E]
  uint32_t* tokens = lds + E;                               // [1]
  float* side = reinterpret_cast<float*>(lds + E + 1);      // [kWaves][E]
  for (int e = threadIdx.x; e < E + 1; e += kThreads) lds[e] = 0u;
  __syncthreads();
  float sum[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) sum[i] = 0.0f;
  uint32_t mine = 0;
  const int64_t step = (int64_t)gridDim.x * kWaves * kTokens;
  for (int64_t t0 = ((int64_t)blockIdx.x * kWaves + wave) * kTokens; t0 < a.T; t0 += step) {
    const int64_t t = t0 + lane / LPT;
    const bool here = t < a.T && (!a.mask || a.mask[t] != 0);
    float v[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = sub + LPT * i;
      v[i] = here && e < E ? a.logits[t * a.ld + e] : -INFINITY;
    }
    if (here) {
      for (int j = sub; j < a.k; j += LPT) {
        const uint32_t id = (uint32_t)a.ids[t * a.k + j];
        if (id < (uint32_t)E) atomicAdd(&count[id], 1u);
      }
      if (sub == 0) ++mine;
    }
    softmax<LPT, PER>(v, sub, E);
#pragma unroll
    for (int i = 0; i < PER; ++i) sum[i] += v[i];
  }
  if (mine) atomicAdd(tokens, mine);
#pragma unroll
  for (int i = 0; i < PER; ++i) {
#pragma unroll
    for (int off = LPT; off < 64; off <<= 1) sum[i] += __shfl_xor(sum[i], off);
    const int e = sub + LPT * i;
    if (lane < LPT && e < E) side[wave * E + e] = sum[i];
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kThreads) {
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) s += side[w * E + e];
    a.sums[(int64_t)blockIdx.x * E + e] = s;
    a.part_counts[(int64_t)blockIdx.x * E + e] = (int32_t)count[e];
  }
  if (threadIdx.x == 0) a.part_tokens[blockIdx.x] = (int32_t)*tokens;
}

// The workgroups' sums, added in order: a thread per expert and slice of them.
constexpr int kFinish = 1024;
__global__ void __launch_bounds__(kFinish)
moe_balance_finish_kernel(const BalanceArgs a, int blocks) {
  __shared__ double psum[kFinish];
  __shared__ int64_t csum[kFinish];
  __shared__ double loss[kFinish / 64];
  const int E = a.E, tid = threadIdx.x;
  int lanes = 64;                       // experts side by side
  while (lanes < E) lanes <<= 1;        // (E <= 1024 = kFinish)
  const int slices = kFinish / lanes, e = tid % lanes, slice = tid / lanes;
  int64_t n = 0;
  for (int b = 0; b < blocks; ++b) n += a.part_tokens[b];
  double p = 0.0;
  int64_t c = 0;
  if (e < E)
    for (int b = slice; b < blocks; b += slices) {
      p += (double)a.sums[(int64_t)b * E + e];
      c += a.part_counts[(int64_t)b * E + e];
    }
  psum[tid] = p;
  csum[tid] = c;
  __syncthreads();
  double l = 0.0;
  if (slice == 0 && e < E) {
    for (int s = 1; s < slices; ++s) {
      p += psum[s * lanes + e];
      c += csum[s * lanes + e];
    }
    const double slope = n ? (double)a.coef * E * (double)c / ((double)a.k * (double)n * (double)n) : 0.0;
    l = slope * p;
    a.counts[e] = (int32_t)c;
    a.slopes[e] = (float)slope;
  }
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) l += __shfl_xor(l, off);
  if ((tid & 63) == 0) loss[tid >> 6] = l;
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < kFinish / 64; ++w) l += loss[w];
    *a.loss = (float)l;
  }
}

template <int LPT, int PER>
__global__ void __launch_bounds__(kThreads)
moe_balance_backward_kernel(const BalanceGradArgs a) {
  constexpr int kTokens = 64 / LPT;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, sub = lane % LPT;
  const int E = a.E;
  const float dloss = a.dloss ? *a.dloss : 1.0f;
  float slope[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) slope[i] = sub + LPT * i < E ? a.slopes[sub + LPT * i] : 0.0f;
  const int64_t step = (int64_t)gridDim.x * kWaves * kTokens;
  for (int64_t t0 = ((int64_t)blockIdx.x * kWaves + wave) * kTokens; t0 < a.T; t0 += step) {
    const int64_t t = t0 + lane / LPT;
    const bool here = t < a.T && (!a.mask || a.mask[t] != 0);
    float v[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = sub + LPT * i;
      v[i] = here && e < E ? a.logits[t * a.ld + e] : -INFINITY;
    }
    softmax<LPT, PER>(v, sub, E);
    float c = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i) c = __builtin_fmaf(v[i], slope[i], c);
    c = part_sum<LPT>(c);
    if (t >= a.T || (a.accumulate && !here)) continue;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = sub + LPT * i;
      if (e < E) {
        float* o = a.dlogits + t * a.lddl + e;
        const float g = dloss * (v[i] * (slope[i] - c));
        *o = here ? (a.accumulate ? *o + g : g) : 0.0f;
      }
    }
  }
}

// Tokens per workgroup at once for E experts.
int tokens_at_once(int E) { return kWaves * (E <= 64 ? 4 : E <= 128 ? 2 : 1); }

unsigned balance_blocks(int64_t T, int E) {
  const int64_t per = tokens_at_once(E), b = (T + per - 1) / per;
  return (unsigned)(b < kBlocks ? b : kBlocks);
}

}  // namespace

size_t moe_balance_workspace(int64_t T, int32_t E) { return (size_t)balance_blocks(T, E) * ((size_t)E * 8 + 4); }

hipError_t launch_moe_balance(BalanceArgs a, void* workspace, hipStream_t stream) {
  const unsigned blocks = a.T ? balance_blocks(a.T, a.E) : 0;
  a.sums = static_cast<float*>(workspace);
  a.part_counts = reinterpret_cast<int32_t*>(a.sums + (size_t)blocks * a.E);
  a.part_tokens = a.part_counts + (size_t)blocks * a.E;
  if (blocks) {
    auto kernel = a.E <= 64    ? moe_balance_kernel<16, 4>
                  : a.E <= 128 ? moe_balance_kernel<32, 4>
                  : a.E <= 256 ? moe_balance_kernel<64, 4>
                               : moe_balance_kernel<64, 16>;
    kernel<<<blocks, kThreads, ((size_t)a.E * (1 + kWaves) + 1) * 4, stream>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  moe_balance_finish_kernel<<<1, kFinish, 0, stream>>>(a, (int)blocks);
  return hipGetLastError();
}

hipError_t launch_moe_balance_backward(const BalanceGradArgs& a, hipStream_t stream) {
  const int64_t per = tokens_at_once(a.E), b = (a.T + per - 1) / per;
  auto kernel = a.E <= 64    ? moe_balance_backward_kernel<16, 4>
                : a.E <= 128 ? moe_balance_backward_kernel<32, 4>
                : a.E <= 256 ? moe_balance_backward_kernel<64, 4>
                             : moe_balance_backward_kernel<64, 16>;
  kernel<<<(unsigned)(b < 4096 ? b : 4096), kThreads, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace q4
