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
// (the counts are whole numbers and have no gradient).  p is fp32; every sum of it
// over tokens is in 64 bits from the first addition on: in fp32 those of a lane, some
// thousands in a row of nearly equal values, would lose 2^-16 at 2^24 tokens.
// Workgroups walk over the tokens and write their sums of p, their counts and their
// tokens to the workspace; a second kernel adds those in order, so the results do
// not vary.  Where there is little to read, one workgroup does it all in one launch.
#include "q4_launch.h"
#include "q4_wave.h"

namespace q4 {
namespace {

constexpr int kThreads = 1024;        // of the forward kernels
constexpr int kWaves = kThreads / 64;
constexpr int kBlocks = 256;          // workgroups of the first kernel at most
constexpr int kBackThreads = 256;
constexpr int kBackWaves = kBackThreads / 64;

// Entries of a workgroup's row in the workspace: whole pieces of 16 bytes.
__host__ __device__ __forceinline__ int padded(int E) { return (E + 3) & ~3; }

// LPT lanes hold a token's E <= LPT * PER logits, in groups of four: value 4 q + j
// of lane i is expert 4 LPT q + 4 i + j.
template <int LPT>
__device__ __forceinline__ int expert_of(int sub, int i) { return 4 * LPT * (i >> 2) + 4 * sub + (i & 3); }

// What lane `lane` reads of a token: offsets from the first token of its wave (the
// same for every turn, so that a load's address is a scalar and one of these), at a
// valid place also where the lane has nothing to read.
template <int LPT, int PER, bool WIDE>
struct Lane {
  uint32_t at[WIDE ? PER / 4 : PER];
  bool has[WIDE ? PER / 4 : PER];
  __device__ __forceinline__ Lane(int lane, int E, int64_t ld) {
#pragma unroll
    for (int i = 0; i < (WIDE ? PER / 4 : PER); ++i) {
      const int e = expert_of<LPT>(lane % LPT, WIDE ? 4 * i : i);
      has[i] = e < E;
      at[i] = (uint32_t)(lane / LPT) * (uint32_t)ld + (uint32_t)(has[i] ? e : 0);
    }
  }
  // (row: of the wave's first token)
  __device__ __forceinline__ void load(const float* row, float (&v)[PER]) const {
    if constexpr (WIDE) {
#pragma unroll
      for (int q = 0; q < PER / 4; ++q) {
        const float4 f = *reinterpret_cast<const float4*>(row + at[q]);
        v[4 * q] = f.x;
        v[4 * q + 1] = f.y;
        v[4 * q + 2] = f.z;
        v[4 * q + 3] = f.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < PER; ++i) v[i] = row[at[i]];
    }
  }
  // -inf for what is no expert of a token that counts
  __device__ __forceinline__ void keep(float (&v)[PER], bool here) const {
#pragma unroll
    for (int i = 0; i < PER; ++i) v[i] = here && has[WIDE ? i / 4 : i] ? v[i] : -INFINITY;
  }
};

// The greater of two, in one instruction (fmaxf first makes a quiet NaN of each
// loaded value); what it makes of a NaN does not matter here.
__device__ __forceinline__ float greater(float a, float b) { return __builtin_amdgcn_fmed3f(a, b, INFINITY); }
struct GreaterOp {
  __device__ __forceinline__ uint32_t operator()(uint32_t a, uint32_t b) const {
    return __builtin_bit_cast(uint32_t, greater(__builtin_bit_cast(float, a), __builtin_bit_cast(float, b)));
  }
};

// Exponentials of a token's logits, v[e] = exp(l[e] - max), and the reciprocal of
// their sum: p[e] = v[e] * by.  by is 0 where every logit is -inf; NaN where one is
// NaN: its exponential and so the sum are.  exp(d) as 2^(d log2 e) in one
// instruction, within a few 2^-24 of it times 1 + |d|.
template <int LPT, int PER>
__device__ __forceinline__ float exponentials(float (&v)[PER]) {
  float m = v[0];
#pragma unroll
  for (int i = 1; i < PER; ++i) m = greater(m, v[i]);
  m = __builtin_bit_cast(float, reduce_lanes<LPT>(__builtin_bit_cast(uint32_t, m), GreaterOp()));
  const float from = m == -INFINITY ? 0.0f : m;
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    v[i] = __builtin_amdgcn_exp2f((v[i] - from) * 1.44269504f);
    s += v[i];
  }
  s = lanes_sum<LPT>(s);
  return s == 0.0f ? 0.0f : __builtin_amdgcn_rcpf(s);   // (within 1 ulp; 1 <= s <= 1024, or NaN)
}

// slope and loss's part of an expert with c choices and probabilities p among n
// tokens.
__device__ __forceinline__ double finish_expert(const BalanceArgs& a, int e, double p, int64_t c, int64_t n) {
  const double slope = n ? (double)a.coef * a.E * (double)c / ((double)a.k * (double)n * (double)n) : 0.0;
  a.counts[e] = (int32_t)c;
  a.slopes[e] = (float)slope;
  return slope * p;
}

// Sum of the threads' parts of the loss, in order (in the first thread).
__device__ __forceinline__ double block_loss(double l, double (&part)[kWaves]) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) l += __shfl_xor(l, off);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = l;
  __syncthreads();
  if (threadIdx.x == 0)
#pragma unroll
    for (int w = 1; w < kWaves; ++w) l += part[w];
  return l;
}

// ONE: a single workgroup, which finishes by itself.  Bound by its VALU instructions,
// 83 a token in 61% of its cycles (8 of them for sums in 64 bits: 16.3 us without, and
// 18 with eight turns together), and by the loads of its first turns: 65537 tokens of
// 256 experts in 17.4 us, 4.0 TB/s.
template <int LPT, int PER, bool WIDE, bool ONE>
__global__ void __launch_bounds__(kThreads)
moe_balance_kernel(const BalanceArgs a) {
  constexpr int kTokens = 64 / LPT;          // of a wave side by side
  constexpr int kTurns = PER == 4 ? 4 : 1;   // and one behind the other with their loads on the way together
  constexpr int kIds = LPT == 16 ? 2 : 1;    // choices of a lane (k <= 32)
  const int lane = threadIdx.x & 63, sub = lane % LPT;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int E = a.E, k = a.k;
  __shared__ uint32_t count[1024];
  __shared__ uint32_t tokens;
  __shared__ double part[kWaves];
  extern __shared__ double side[];           // [kWaves][E]
  for (int e = threadIdx.x; e < E; e += kThreads) count[e] = 0u;
  if (threadIdx.x == 0) tokens = 0u;
  __syncthreads();
  const Lane<LPT, PER, WIDE> mine(lane, E, a.ld);
  uint32_t id_at[kIds];
#pragma unroll
  for (int j = 0; j < kIds; ++j)
    id_at[j] = (uint32_t)(lane / LPT * k + (sub + LPT * j < k ? sub + LPT * j : 0));
  double sum[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) sum[i] = 0.0;
  uint32_t seen = 0;
  auto use = [&](float (&v)[PER], const uint32_t (&id)[kIds], bool here) {
#pragma unroll
    for (int j = 0; j < kIds; ++j)
      if (here && sub + LPT * j < k && id[j] < (uint32_t)E) atomicAdd(&count[id[j]], 1u);
    seen += here;
    mine.keep(v, here);
    const float by = exponentials<LPT, PER>(v);
#pragma unroll
    for (int i = 0; i < PER; ++i) sum[i] += (double)(v[i] * by);
  };
  const int T = (int)a.T;                    // (below 2^26)
  const int step = (int)gridDim.x * kWaves * kTokens;
  int t0 = ((int)blockIdx.x * kWaves + wave) * kTokens;
  for (; t0 + (kTurns - 1) * step + kTokens <= T; t0 += kTurns * step) {
    float v[kTurns][PER];
    uint32_t id[kTurns][kIds];
    uint8_t mask[kTurns];
#pragma unroll
    for (int u = 0; u < kTurns; ++u) {
      const int64_t t = t0 + u * step;
      mine.load(a.logits + t * a.ld, v[u]);
      mask[u] = a.mask ? a.mask[t + lane / LPT] : 1;
#pragma unroll
      for (int j = 0; j < kIds; ++j) id[u][j] = (uint32_t)a.ids[t * k + id_at[j]];
    }
#pragma unroll
    for (int u = 0; u < kTurns; ++u) use(v[u], id[u], mask[u] != 0);
  }
  for (; t0 < T; t0 += step) {               // the last turns, one at a time
    const int64_t t = t0;
    const bool there = t0 + lane / LPT < T;
    float v[PER];
    uint32_t id[kIds];
    uint8_t mask = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) v[i] = 0.0f;
#pragma unroll
    for (int j = 0; j < kIds; ++j) id[j] = ~0u;
    if (there) {
      mine.load(a.logits + t * a.ld, v);
      mask = a.mask ? a.mask[t + lane / LPT] : 1;
#pragma unroll
      for (int j = 0; j < kIds; ++j) id[j] = (uint32_t)a.ids[t * k + id_at[j]];
    }
    use(v, id, mask != 0);
  }
  if (seen && sub == 0) atomicAdd(&tokens, seen);
#pragma unroll
  for (int i = 0; i < PER; ++i) {
#pragma unroll
    for (int off = LPT; off < 64; off <<= 1) sum[i] += __shfl_xor(sum[i], off);
    const int e = expert_of<LPT>(sub, i);
    if (lane < LPT && e < E) side[wave * E + e] = sum[i];
  }
  __syncthreads();
  double l = 0.0;
  if (threadIdx.x < E) {   // (E <= 1024 = kThreads)
    const int e = threadIdx.x;
    if constexpr (ONE) {
      double p = 0.0;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) p += side[w * E + e];
      l = finish_expert(a, e, p, count[e], tokens);
    } else {
      double s = 0.0;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) s += side[w * E + e];
      a.sums[(int64_t)blockIdx.x * padded(E) + e] = s;
      a.part_counts[(int64_t)blockIdx.x * padded(E) + e] = (int32_t)count[e];
    }
  }
  if constexpr (ONE) {
    l = block_loss(l, part);
    if (threadIdx.x == 0) *a.loss = (float)l;
  } else if (threadIdx.x == 0) {
    a.part_tokens[blockIdx.x] = (int32_t)tokens;
    if (blockIdx.x == 0) *a.ticket = 0u;
  }
}

// The workgroups' sums, added in order: a workgroup per 64 experts, in it a thread
// per four of them and 64th of the sums, then 16 threads per expert.  The last
// workgroup to end (the ticket was cleared by the first kernel) adds their parts
// of the loss, in their order.  256 workgroups' sums of 256 experts: 8.5 us, latency: a
// thread's turns are waited for one by one, since each may be the last (10 us in a single
// workgroup; with sums of fp32 both kernels 22.9 us, 23.7 with 32 experts per workgroup
// and 23.5 with 16, of 1024 experts 27.2, 29.2 and 32.4).
constexpr int kFinishExperts = 64;
constexpr int kFinishMost = 1024 / kFinishExperts;   // workgroups
__global__ void __launch_bounds__(kThreads)
moe_balance_finish_kernel(const BalanceArgs a, int blocks) {
  constexpr int kSlices = kThreads / (kFinishExperts / 4);
  __shared__ double psum[kSlices][kFinishExperts];
  __shared__ int32_t csum[kSlices][kFinishExperts];
  __shared__ double part[kWaves];
  __shared__ uint32_t tokens;
  const int row = padded(a.E), tid = threadIdx.x, quad = tid % 16, slice = tid / 16;
  const int e0 = blockIdx.x * kFinishExperts;
  if (tid == 0) tokens = 0u;
  const uint32_t here = tid < blocks ? (uint32_t)a.part_tokens[tid] : 0u;
  double p[4] = {0.0, 0.0, 0.0, 0.0};
  int32_t c[4] = {0, 0, 0, 0};
  if (e0 + 4 * quad < row) {
#pragma unroll
    for (int i = 0; i < (kBlocks + kSlices - 1) / kSlices; ++i) {
      const int b = slice + i * kSlices;
      if (b >= blocks) break;
      const double2 s = *reinterpret_cast<const double2*>(a.sums + (int64_t)b * row + e0 + 4 * quad);
      const double2 s2 = *reinterpret_cast<const double2*>(a.sums + (int64_t)b * row + e0 + 4 * quad + 2);
      const int4 n = *reinterpret_cast<const int4*>(a.part_counts + (int64_t)b * row + e0 + 4 * quad);
      p[0] += s.x;
      p[1] += s.y;
      p[2] += s2.x;
      p[3] += s2.y;
      c[0] += n.x;
      c[1] += n.y;
      c[2] += n.z;
      c[3] += n.w;
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    psum[slice][4 * quad + j] = p[j];
    csum[slice][4 * quad + j] = c[j];
  }
  __syncthreads();
  if (here) atomicAdd(&tokens, here);
  const int e = tid / 16;              // (64 experts of 16 threads)
  double ps = 0.0;
  int32_t cs = 0;
#pragma unroll
  for (int i = 0; i < kSlices / 16; ++i) {
    ps += psum[tid % 16 + 16 * i][e];
    cs += csum[tid % 16 + 16 * i][e];
  }
#pragma unroll
  for (int off = 8; off > 0; off >>= 1) {
    ps += __shfl_xor(ps, off);
    cs += __shfl_xor(cs, off);
  }
  __syncthreads();
  double l = 0.0;
  if (tid % 16 == 0 && e0 + e < a.E) l = finish_expert(a, e0 + e, ps, cs, tokens);
  l = block_loss(l, part);
  if (tid != 0) return;
  if (gridDim.x == 1) {
    *a.loss = (float)l;
    return;
  }
  // (the parts and the ticket pass between XCDs: agent scope)
  uint64_t* parts = reinterpret_cast<uint64_t*>(a.parts);
  __hip_atomic_store(parts + blockIdx.x, __builtin_bit_cast(uint64_t, l), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  if (__hip_atomic_fetch_add(a.ticket, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) != gridDim.x - 1) return;
  l = 0.0;
  for (unsigned b = 0; b < gridDim.x; ++b)
    l += __builtin_bit_cast(double, __hip_atomic_load(parts + b, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
  *a.loss = (float)l;
}

// The gradient: the same softmax again, from the logits alone.  65537 tokens of 256
// experts in 20 to 22 us, 6.1 to 6.9 TB/s: bound by HBM.
template <int LPT, int PER, bool WIDE>
__global__ void __launch_bounds__(kBackThreads)
moe_balance_backward_kernel(const BalanceGradArgs a) {
  constexpr int kTokens = 64 / LPT;
  const int lane = threadIdx.x & 63, sub = lane % LPT;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int E = a.E;
  const float dloss = a.dloss ? *a.dloss : 1.0f;
  const Lane<LPT, PER, WIDE> mine(lane, E, a.ld), out(lane, E, a.lddl);
  float slope[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = expert_of<LPT>(sub, i);
    slope[i] = e < E ? a.slopes[e] : 0.0f;
  }
  const int T = (int)a.T, step = (int)gridDim.x * kBackWaves * kTokens;
  for (int t0 = ((int)blockIdx.x * kBackWaves + wave) * kTokens; t0 < T; t0 += step) {
    const int64_t t = t0;
    const bool there = t0 + lane / LPT < T;
    float v[PER];
    uint8_t mask = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) v[i] = 0.0f;
    if (there) {
      mine.load(a.logits + t * a.ld, v);
      mask = a.mask ? a.mask[t + lane / LPT] : 1;
    }
    const bool here = mask != 0;
    mine.keep(v, here);
    const float by = exponentials<LPT, PER>(v);
    float c = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      v[i] *= by;
      c = __builtin_fmaf(v[i], slope[i], c);
    }
    c = lanes_sum<LPT>(c);
    if (!there || (a.accumulate && !here)) continue;
    // (not here: v and c are 0)
#pragma unroll
    for (int i = 0; i < PER; ++i) v[i] = dloss * (v[i] * (slope[i] - c));
    if (!here) {   // (not NaN or inf times 0)
#pragma unroll
      for (int i = 0; i < PER; ++i) v[i] = 0.0f;
    }
    float* row = a.dlogits + t * a.lddl;
    if constexpr (WIDE) {
#pragma unroll
      for (int q = 0; q < PER / 4; ++q) {
        if (!out.has[q]) continue;
        float4* o = reinterpret_cast<float4*>(row + out.at[q]);
        float4 f = make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
        if (a.accumulate) {
          const float4 b = *o;
          f = make_float4(b.x + f.x, b.y + f.y, b.z + f.z, b.w + f.w);
        }
        *o = f;
      }
    } else {
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (out.has[i]) row[out.at[i]] = a.accumulate ? row[out.at[i]] + v[i] : v[i];
    }
  }
}

// Tokens of a wave side by side.
int tokens_at_once(int E) { return E <= 64 ? 4 : E <= 128 ? 2 : 1; }

// One workgroup up to 8 turns of all its waves (512 tokens of 64 experts): 1024
// tokens take it 13 us, and 5.5 us and a second launch of 5.5 us over the card; each
// launch costs the caller 3.3 us besides.
unsigned balance_blocks(int64_t T, int E) {
  const int64_t per = kWaves * tokens_at_once(E), turns = (T + per - 1) / per;
  if (turns <= 8) return 1;
  return (unsigned)(turns < kBlocks ? turns : kBlocks);
}

bool wide(const void* p, int64_t ld, int E) {
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && ld % 4 == 0 && E % 4 == 0;
}

template <int LPT, int PER, bool WIDE, bool ONE>
hipError_t balance_as(const BalanceArgs& a, unsigned blocks, hipStream_t stream) {
  const size_t side = (size_t)a.E * kWaves * 8;
  if (side > 32768) {   // (with the kernel's own LDS past 64 KB from 481 experts on)
    const hipError_t attr = set_max_lds<&moe_balance_kernel<LPT, PER, WIDE, ONE>>(131072);
    if (attr != hipSuccess) return attr;
  }
  moe_balance_kernel<LPT, PER, WIDE, ONE><<<blocks, kThreads, side, stream>>>(a);
  return hipGetLastError();
}

template <int LPT, int PER, bool ONE>
hipError_t balance(const BalanceArgs& a, unsigned blocks, hipStream_t stream) {
  return wide(a.logits, a.ld, a.E) ? balance_as<LPT, PER, true, ONE>(a, blocks, stream)
                                   : balance_as<LPT, PER, false, ONE>(a, blocks, stream);
}

template <int LPT, int PER>
void balance_backward(const BalanceGradArgs& a, hipStream_t stream) {
  const int64_t per = kBackWaves * tokens_at_once(a.E), b = (a.T + per - 1) / per;
  auto kernel = wide(a.logits, a.ld, a.E) && wide(a.dlogits, a.lddl, a.E) ? moe_balance_backward_kernel<LPT, PER, true>
                                                                         : moe_balance_backward_kernel<LPT, PER, false>;
  kernel<<<(unsigned)(b < 4096 ? b : 4096), kBackThreads, 0, stream>>>(a);
}

template <bool ONE>
hipError_t balance_of(const BalanceArgs& a, unsigned blocks, hipStream_t stream) {
  if (a.E <= 64) return balance<16, 4, ONE>(a, blocks, stream);
  if (a.E <= 128) return balance<32, 4, ONE>(a, blocks, stream);
  if (a.E <= 256) return balance<64, 4, ONE>(a, blocks, stream);
  return balance<64, 16, ONE>(a, blocks, stream);
}

}  // namespace

size_t moe_balance_workspace(int64_t T, int32_t E) {
  const unsigned b = balance_blocks(T, E);
  return b > 1 ? kFinishMost * 8 + (size_t)b * ((size_t)padded(E) * 12 + 4) + 4 : 0;
}

hipError_t launch_moe_balance(BalanceArgs a, void* workspace, hipStream_t stream) {
  const unsigned blocks = balance_blocks(a.T, a.E);
  if (blocks == 1) return balance_of<true>(a, 1, stream);
  a.parts = static_cast<double*>(workspace);
  a.sums = a.parts + kFinishMost;
  a.part_counts = reinterpret_cast<int32_t*>(a.sums + (size_t)blocks * padded(a.E));
  a.part_tokens = a.part_counts + (size_t)blocks * padded(a.E);
  a.ticket = reinterpret_cast<uint32_t*>(a.part_tokens + blocks);
  const hipError_t e = balance_of<false>(a, blocks, stream);
  if (e != hipSuccess) return e;
  moe_balance_finish_kernel<<<(a.E + kFinishExperts - 1) / kFinishExperts, kThreads, 0, stream>>>(a, (int)blocks);
  return hipGetLastError();
}

hipError_t launch_moe_balance_backward(const BalanceGradArgs& a, hipStream_t stream) {
  if (a.E <= 64) balance_backward<16, 4>(a, stream);
  else if (a.E <= 128) balance_backward<32, 4>(a, stream);
  else if (a.E <= 256) balance_backward<64, 4>(a, stream);
  else balance_backward<64, 16>(a, stream);
  return hipGetLastError();
}

}  // namespace q4
