// gemm_grad.hip -- the gradients of the W4 products.  Forward, for the rows p
// of expert e (a dense layer is one expert): c[p][n] = sum_k a[p][k] w'_e[n][k].
//
//   dgrad  dA[p][k]   = sum_n dC[p][n] w'_e[n][k]
//   wgrad  dW_e[n][k] = sum_{p in e} dC[p][n] a[gather[p]][k]
//
// Both are bf16 matrix products (v_mfma_f32_16x16x32_bf16, fp32 sums) whose
// second operand B -- the 4-bit weight, the saved activation -- is stored with
// the summed index as its rows; in wgrad so is the first operand A = dC.
//
//   * B is converted once per workgroup: a thread loads 32 columns of one row
//     (q4_piece.h), converts them to bf16 and writes them to LDS as rows; the
//     fragments are read column-wise from there by ds_read_b64_tr_b16, which
//     hands lane i of 16 the column i of four rows.  A transposes the same way
//     in wgrad; in dgrad its rows hold the summed index already.
//   * A goes to LDS by direct copies (buffer loads to LDS: unlike global_load_lds
//     they leave the compiler's load counts exact, so that B's loads are not
//     waited for as a whole).  Rows and columns past the sum's end are filled
//     with zeros by the buffer's range check, so that whatever B holds there
//     (clamped to existing rows) adds nothing.
//   * Rows and 16-byte chunks are placed in LDS so that the lanes that it serves
//     at once never meet on a bank (column_place, swizzle_rows).
//   * A workgroup of kWM x kWK waves makes a block of C of 16 kMT kWM rows by
//     256 columns and takes R = 8 kWM kWK summed rows per stage (one piece of B
//     per thread).  A is copied two stages ahead (three buffers), B is loaded
//     into registers up to two stages ahead and converted one ahead (two
//     buffers).
//   * The outputs go out as whole cache lines (see the epilogue).
//
// What bounds it.  Dense: the matrix pipe is busy 60% of the time (back to back:
// dgrad 4096 x 8192 x 8192, INT4, 450 us = 1220 TF/s, wgrad 8192^3 930 us = 1180,
// after some 50 passes; the first ten after an idle moment take a fifth longer,
// 540 and 1080); a loop of nothing but the stage's matrix, LDS and conversion
// instructions reaches about 1430 under the card's power limit.  Grouped dgrad
// (64 x 2048 x 7168, 32768 ragged rows, MXFP4): 950 us, 1010 at first.  Grouped
// wgrad (the same, 1.30 - 1.35 ms): 3.8 GB of fp32 gradients, whose stores take
// 0.68 ms alone; the products take 0.95 ms alone, and the two add up by more
// than half, since a CU's loads queue behind its stores.  (Not mended by
// delaying every other workgroup, by a persistent workgroup that loads the next
// block's first stages before it stores -- wgrad 4% faster, dgrad 5% slower for
// its registers --, nor by two 128-row workgroups per CU.)  Few rows: the time
// of a stage, 0.4 - 0.8 us of load latency over two stages in flight.
#include "q4_launch.h"
#include "q4_lds.h"
#include "q4_piece.h"

#include <algorithm>
#include <cstdint>
#include <type_traits>

namespace q4 {
namespace {

typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4_t* trptr_t;
typedef const __attribute__((address_space(3))) u32x4_t* u32x4_lds_t;

constexpr int kBK = 256;              // columns of a block of C
constexpr int kABufs = 3, kBBufs = 2;

// A is copied through buffers, where an offset past the end loads zeros.  wgrad's
// end with the matrix; dgrad's offsets lie in the matrix or are kPast.
constexpr int kPast = 0x7FFFFFF0;
constexpr int kRsrcFlags = 0x00020000;   // a raw buffer of 32-bit words

// A buffer at p (wave-uniform) of the first `rows` of R rows of `bytes` bytes,
// the last of them `tail` bytes short; empty for rows <= 0.
__device__ __forceinline__ rsrc_t rows_buffer(const uint8_t* p, int rows, int R, int bytes, int tail = 0) {
  const int n = rows >= R ? R * bytes - tail : rows > 0 ? rows * bytes - tail : 0;
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p), 0, __builtin_amdgcn_readfirstlane(n), kRsrcFlags);
}

// Segment of an expert, clamped to [0, P]; offsets NULL: all rows.
__device__ __forceinline__ void segment(const int32_t* offsets, int e, int P, int& lo, int& hi) {
  lo = 0;
  hi = P;
  if (offsets) {
    lo = min(max(offsets[e], 0), P);
    hi = min(max(offsets[e + 1], lo), P);
  }
}

// Row tile number `slot` over all experts: its expert, first row and the
// expert's end; false if there are fewer tiles.  Each wave looks at 64 experts
// at a time.
template <int BM>
__device__ __forceinline__ bool find_tile(const int32_t* offsets, int E, int P, int slot, int& e, int& lo, int& hi) {
  if (!offsets) {
    e = 0;
    lo = slot * BM;
    hi = P;
    return lo < P;
  }
  const int lane = threadIdx.x & 63;
  for (int e0 = 0; e0 < E; e0 += 64) {
    int l = 0, h = 0;
    if (e0 + lane < E) segment(offsets, e0 + lane, P, l, h);
    const int tiles = (h - l + BM - 1) / BM;
    int x = tiles;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int y = __shfl_up(x, off);
      if (lane >= off) x += y;
    }
    const uint64_t at = __ballot(slot < x);
    if (at) {
      const int first = __builtin_ctzll(at);
      e = e0 + first;
      lo = __shfl(l + (slot - (x - tiles)) * BM, first);
      hi = __shfl(h, first);
      return true;
    }
    slot -= __shfl(x, 63);
  }
  return false;
}

// Place of element (row r, 16-byte chunk c) of an operand that is read
// column-wise: blocks of 32 columns (4 chunks, 64 bytes per row), in a block
// every 32 rows of a matrix step in the order in which they are read.  A read
// takes, for 16 lanes, 32 bytes of four rows 8 g + 4 h + 0..3 (g the lane group,
// h the half of the fragment); LDS serves two groups at once, so the rows of a
// pair of groups lie together (8 rows, 512 bytes) and one of their fours has
// the halves of its 64 bytes swapped: 8 x 32 bytes on 256 bytes of banks; which
// of them alternates with h, so that a wave that writes one chunk of rows 0..15
// does not meet itself either.  Steps and pairs of tiles are constant offsets;
// an odd tile and the second half are address ^ 32.
//
// of_b: B's tiles are not 16 consecutive columns.  So that the epilogue's stores
// need few exchanges, tile j of a wave's 64 columns takes two chunks 32 columns
// apart, j / 2 + 2 (j % 2) of either block, and the chunks of an odd block trade
// places with their neighbours: again 256 bytes of banks.  The rows of block b
// are XORed with b % 4, so that threads that write neighbouring blocks of one
// row meet no bank twice.
__device__ __forceinline__ int row_place(int r) {        // r in 0..31 -> 0..31, its own inverse
  return (r & 16) | ((r & 4) << 1) | ((r & 8) >> 1) | (r & 3);
}
__device__ __forceinline__ int place_swap(int p) { return ((p >> 1) ^ (p >> 2)) & 2; }   // on the chunk's number
__device__ __forceinline__ int column_place(int r, int c, int block_bytes, bool of_b) {
  const int block = c >> 2, p = row_place(r & 31) ^ (of_b ? block & 3 : 0);
  return block * block_bytes + ((r & ~31) + p) * 64 + (((c & 3) ^ place_swap(p) ^ (of_b ? block & 1 : 0)) << 4);
}

// Chunk permutation of dgrad's A, whose rows of R summed values are read by
// ds_read_b128, lane l row l % 16 and chunk l / 16.  LDS serves lanes 0-3, 12-15
// and 20-27 at once, and 4-11, 16-19 and 28-31 (measured): rows four apart take
// the chunks 0, 3, 2, 1 (R = 32), pairs of rows consecutive ones (R = 64).
template <int R>
__device__ __forceinline__ int swizzle_rows(int m) {
  return R == 32 ? -(m >> 2) & 3 : (m >> 1) & 7;
}

// Eight values along the summed index for lane l's column of a 16-column tile:
// rows 8 (l / 16) + 0..7 of 32, from the lane's address for the first half (p0)
// and that of the other tile of the pair (p1).
// (restrict: the reads do not alias a copy in flight, which the kernel waits
// for by count; without it every read would wait for all copies.)
__device__ __forceinline__ bf16x8_t read_columns(const trptr_t __restrict__ p0, const trptr_t __restrict__ p1) {
  const s16x4_t a = __builtin_amdgcn_ds_read_tr16_b64_v4i16(p0);
  const s16x4_t b = __builtin_amdgcn_ds_read_tr16_b64_v4i16(p1 + 512 / sizeof(s16x4_t));
  typedef short s16x8_t __attribute__((ext_vector_type(8)));
  const s16x8_t v = __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
  return __builtin_bit_cast(bf16x8_t, v);
}

// Exchanges between lanes and registers: a lane bit trades places with the bit
// that tells a from b.  Bit 0 or 1 of the lane (within its quad), `set` in this
// lane; bit 4 (v_permlane16_swap exchanges the odd groups of 16 lanes of one
// register with the even ones of the other).
template <int BIT>
__device__ __forceinline__ void swap_quad(bool set, uint32_t& a, uint32_t& b) {
  constexpr int kPerm = BIT == 0 ? 0xB1 : 0x4E;        // quad_perm: lane ^ 1, lane ^ 2
  const uint32_t from_b = __builtin_amdgcn_update_dpp(0, b, kPerm, 0xF, 0xF, true);
  const uint32_t from_a = __builtin_amdgcn_update_dpp(0, a, kPerm, 0xF, 0xF, true);
  a = set ? from_b : a;
  b = set ? b : from_a;
}
__device__ __forceinline__ void swap16(uint32_t& a, uint32_t& b) {
  const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
  a = r[0];
  b = r[1];
}

// fp32 weight gradients are far larger than the caches and read by a later
// kernel: written past them (64 x 2048 x 7168, 32768 ragged rows: 1500 us through
// them, 1300 past them).
__device__ __forceinline__ void store_f32(float* p, f32x4_t v, int accumulate) {
  f32x4_t* const o = reinterpret_cast<f32x4_t*>(p);
  if (accumulate) v += *o;
  __builtin_nontemporal_store(v, o);
}

template <bool WGRAD, int KIND, int LAYOUT, bool GATHER, int kWM, int kWK, int kMT>
struct Kern {
  static constexpr int kWaves = kWM * kWK, kThreads = 64 * kWaves, R = 8 * kWaves;
  static constexpr int kKT = kBK / 16 / kWK;              // 16-column tiles per wave
  static constexpr int BM = 16 * kMT * kWM;
  static constexpr int kSteps = R / 32;                   // matrix steps per stage
  static constexpr int kBlock = R * 64;                   // 32 columns of a stage
  static constexpr int kABytes = R * BM * 2, kBBytes = R * kBK * 2;
  static constexpr int kSmem = kABufs * kABytes + kBBufs * kBBytes;
  static constexpr int kCopies = kABytes / 1024;          // copy instructions per stage
  static constexpr int kCPW = kCopies / kWaves;           // per wave: what its waits count
  static_assert(kCopies % kWaves == 0, "every wave makes as many copies");
};

// One block of C: of expert e's rows lo .. hi - 1, from row (dgrad) or n (wgrad)
// m0 and column k0 on; part `split` of the sum.
template <bool WGRAD, int KIND, int LAYOUT, bool GATHER, int kWM, int kWK, int kMT>
__device__ __forceinline__ void make_block(const GradArgs& g, uint8_t* const smem, int e, int lo, int hi, int m0,
                                           int k0, int split, int splits) {
  using C = Kern<WGRAD, KIND, LAYOUT, GATHER, kWM, kWK, kMT>;
  constexpr int R = C::R;
  uint8_t* const bbase = smem;                        // (first: its offsets fit the instructions)
  uint8_t* const abase = smem + kBBufs * C::kBBytes;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / kWK, wk = wave % kWK;
  const int P = (int)g.P, N = (int)g.N, K = (int)g.K;
  // this workgroup's part of the sum: whole stages
  int r_begin = WGRAD ? lo : 0, r_end = WGRAD ? hi : N;
  if (kWM == 1 && splits > 1) {
    const int part = ((r_end - r_begin + R - 1) / R + splits - 1) / splits * R;
    r_begin = min(r_begin + split * part, r_end);
    r_end = min(r_begin + part, r_end);
  }
  const int stages = (r_end - r_begin + R - 1) / R;
  const int m_end = WGRAD ? N : hi;

  // ---- A: this lane's part of each copy, as a byte offset from the stage's
  // first row or column.  wgrad: 16 rows of a block of 32 columns, in the order
  // of column_place; a wave's copies are 64 columns apart, and what they hold
  // of columns from N on is not used (the buffer ends with column N of the last
  // row).  dgrad: a lane with nothing to copy takes an offset past the buffer's
  // end and gets zeros.
  constexpr int AC = R / 8, RPC = 64 / AC;
  int aoff[WGRAD ? 1 : C::kCPW];
  if constexpr (WGRAD) {
    const int at = wave * 16 + (lane >> 2), p = at % R, c = at / R * 4 + ((lane & 3) ^ place_swap(p));
    aoff[0] = (((p & ~31) + row_place(p & 31)) * (int)g.lddc + 8 * c) * 2;
  } else {
#pragma unroll
    for (int q = 0; q < C::kCPW; ++q) {
      const int m = (wave + C::kWaves * q) * RPC + lane / AC, c = (lane % AC) ^ swizzle_rows<R>(m);
      aoff[q] = (min(m, hi - 1 - m0) * (int)g.lddc + 8 * c) * 2;
    }
  }
  // the copies run through the stages in order: position and summed rows left
  // (0 or less past the last stage: the buffer is empty)
  const uint8_t* apos = reinterpret_cast<const uint8_t*>(
      g.dc + (WGRAD ? (int64_t)r_begin * g.lddc + m0 : (int64_t)m0 * g.lddc + r_begin));
  const int64_t astep = WGRAD ? (int64_t)R * g.lddc * 2 : R * 2;
  int aleft = r_end - r_begin;
  auto copy_a = [&](int buf) {
    const rsrc_t rsrc = WGRAD ? rows_buffer(apos, aleft, R, (int)g.lddc * 2, ((int)g.lddc - (N - m0)) * 2)
                              : rows_buffer(apos, aleft > 0 ? R : 0, R, kPast / R);
    uint8_t* dst = abase + buf * C::kABytes;
#pragma unroll
    for (int q = 0; q < C::kCPW; ++q) {
      const int ci = wave + C::kWaves * q;
      int off;
      if constexpr (WGRAD) {
        off = aoff[0];
        asm volatile("" : "+v"(off));                   // (one register, not one per copy)
        off += 128 * q;
      } else {
        const int m = ci * RPC + lane / AC, c = (lane % AC) ^ swizzle_rows<R>(m);
        off = 8 * c >= aleft ? kPast : aoff[q];
      }
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lptr_t)(dst + ci * 1024), 16, off, 0, 0, 0);
    }
    apos += astep;
    aleft -= R;
  };

  // ---- B: a thread's 32 values of a stage (q4_piece.h).  The buffers start at
  // the stage's first row and end with the expert's last, so that rows past the
  // sum's end are zeros.
  const int br = piece_row<KIND>(tid);
  const PieceCols<KIND> bcols_at = piece_cols<KIND>(tid, k0, K);
  const PieceAt<KIND> at = piece_at<KIND, LAYOUT>(br, bcols_at, K, (int)g.ldb);
  const int drow = KIND == kBf16Piece ? 2 * (int)g.ldb : WGRAD ? K : K / 2;     // bytes of a row
  const int srow = KIND == kBf16Piece ? 0 : K / PieceScale<KIND>::kCols * PieceScale<KIND>::kBytes;
  const int64_t row0 = WGRAD ? r_begin : (int64_t)e * N + r_begin;
  const uint8_t *bpos = g.b + row0 * drow, *spos = g.b_scales + row0 * srow;
  int bleft = WGRAD ? r_end - r_begin : (LAYOUT == kLayoutTiled ? (N + 15) / 16 * 16 : N) - r_begin;
  int bdst[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) bdst[i] = column_place(br, piece_chunk<KIND>(tid, i), C::kBlock, true);
  auto row_index = [&](int u) -> int {                 // gather's entry for stage u
    return GATHER ? g.gather[min(r_begin + u * R + br, r_end - 1)] : 0;
  };
  auto load_b = [&](Piece<KIND>& p, int idx, bool& ok) {   // stage after stage, like copy_a
    if constexpr (GATHER) {
      ok = br < bleft && idx >= 0 && idx < (int)g.T;
      piece_load_row<KIND>(p, g.b, g.b_scales, ok ? idx : 0, bcols_at, K, g.ldb);
    } else {
      // (a bf16 matrix ends with its last row's K columns)
      const int tail = KIND == kBf16Piece ? drow - 2 * K : 0;
      piece_load<KIND>(p, rows_buffer(bpos, bleft, R, drow, tail), rows_buffer(spos, bleft, R, srow), at);
      ok = true;
      bpos += (int64_t)R * drow;
      spos += (int64_t)R * srow;
    }
    bleft -= R;
  };
  // eight values (of four times eight) of a piece, converted and written
  auto store_b = [&](Piece<KIND>& p, bool ok, int buf, int i) {
    if constexpr (GATHER)
      if (i == 0) piece_clear(p, !ok);
    *reinterpret_cast<u32x4_t*>(bbase + buf * C::kBBytes + bdst[i]) = piece_convert<KIND>(p, i);
  };

  // ---- fragment addresses in LDS (of the first half in the first step): of
  // B's tiles, of an even and an odd tile of wgrad's A, of the two steps of
  // dgrad's A
  const int i16 = lane & 15, gq = lane >> 4;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(lptr_t)smem;
  const uint32_t col0 = lds0 + column_place(8 * gq + (i16 >> 2), (i16 & 3) >> 1, 0, false) + (i16 & 1) * 8;
  uint32_t acols[2], bcols[C::kKT];
  static_assert(C::kKT == 4, "a wave's columns are two blocks");
#pragma unroll
  for (int j = 0; j < C::kKT; ++j)
    bcols[j] = lds0 + (i16 & 1) * 8 +
               column_place(8 * gq + (i16 >> 2), 4 * (2 * wk + ((i16 & 3) >> 1)) + (j >> 1) + 2 * (j & 1), C::kBlock, true);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if constexpr (WGRAD) {
      acols[h] = (col0 ^ (h << 5)) + kBBufs * C::kBBytes + wm * (kMT / 2) * C::kBlock;
    } else {
      const int m = 16 * kMT * wm + i16;
      acols[h] = lds0 + kBBufs * C::kBBytes + m * (R * 2) + (((4 * h + gq) ^ swizzle_rows<R>(m)) & (R / 8 - 1)) * 16;
    }
  }

  f32x4_t acc[kMT][C::kKT];
#pragma unroll
  for (int t = 0; t < kMT; ++t)
#pragma unroll
    for (int j = 0; j < C::kKT; ++j) acc[t][j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};

  // ---- a stage is kGroups groups of kGT row tiles by all of the wave's
  // column tiles; the fragments of a group are read under the group before
  constexpr int kGT = C::kSteps == 1 && kMT > 4 ? 2 : 1, kG = kMT / kGT, kGroups = C::kSteps * kG;
  static_assert(kGroups >= 4, "the loads, copies and conversions of a stage come before its last group");
  bf16x8_t fa[2][kGT], fb[C::kKT];
  // (step s is 32 rows on, the second half of a fragment 8 places)
  // this lane's addresses in A's buffer of the stage being read (opaque, so
  // that the constants below stay in the instructions' offsets)
  uint32_t acur[2];
  auto set_a = [&](int buf) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      acur[h] = acols[h] + buf * C::kABytes;
      asm("" : "+v"(acur[h]));
    }
  };
  auto read_a = [&](int gi) {
    const int s = gi / kG;
#pragma unroll
    for (int q = 0; q < kGT; ++q) {
      const int t = kGT * (gi % kG) + q;
      if constexpr (WGRAD)
        fa[gi & 1][q] = read_columns((trptr_t)(acur[t & 1] + (t >> 1) * C::kBlock + s * 2048),
                                     (trptr_t)(acur[1 - (t & 1)] + (t >> 1) * C::kBlock + s * 2048));
      else
        fa[gi & 1][q] = as_bf16x8(*(u32x4_lds_t)(acur[s] + t * 32 * R));
    }
  };
  auto read_b = [&](int buf, int s, int j) {
    fb[j] = read_columns((trptr_t)(bcols[j] + buf * C::kBBytes + s * 2048),
                         (trptr_t)(bcols[j ^ 1] + buf * C::kBBytes + s * 2048));
  };

  if (stages > 0) {
    // pieces of B in registers: of two stages, or (R = 64, whose registers are
    // full) of one that is loaded again as soon as it is converted
    constexpr int kSets = C::kSteps == 1 ? 2 : 1;
    Piece<KIND> raw[kSets];
    bool ok[kSets];
    int idx[4] = {0, 0, 0, 0};
    if constexpr (GATHER) {
#pragma unroll
      for (int i = 0; i < 4; ++i) idx[i] = row_index(i);
      asm volatile("" : "+v"(idx[2]), "+v"(idx[3]));   // loaded here, ahead of the copies that the loop counts
    }
    // Loads run two stages ahead, past the last stage without reading anything.
    // Within a stage B's go first: loads complete in order, and B's are waited
    // for a stage earlier than A's copies.
    load_b(raw[0], idx[0], ok[0]);
    copy_a(0);
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (kSets == 2) load_b(raw[kSets - 1], idx[1], ok[kSets - 1]);
    else
#pragma unroll
      for (int i = 0; i < 4; ++i) store_b(raw[0], ok[0], 0, i);
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (kSets == 1) load_b(raw[0], idx[1], ok[0]);
    __builtin_amdgcn_sched_barrier(0);
    copy_a(1);
    __builtin_amdgcn_sched_barrier(0);
    idx[0] = idx[2];
    idx[1] = idx[3];
    if constexpr (kSets == 2)
#pragma unroll
      for (int i = 0; i < 4; ++i) store_b(raw[0], ok[0], 0, i);
    wait_vmcnt_lgkm0<C::kCPW + Piece<KIND>::kLoads>();
    stage_barrier();
#pragma unroll
    for (int j = 0; j < C::kKT; ++j) read_b(0, 0, j);
    set_a(0);
    read_a(0);
    int abuf = 0;
    auto stage = [&](int u, auto par) {
      constexpr int J = decltype(par)::value;          // u % 2
      const int nbuf = abuf == 0 ? 2 : abuf - 1;       // (u + 2) % 3
      const int abuf1 = abuf == 2 ? 0 : abuf + 1;      // (u + 1) % 3
#pragma unroll
      for (int gi = 0; gi < kGroups; ++gi) {
        if (gi == kGroups - 1) {
          // copy_a(u + 1) is done once at most the loads and copies of stage
          // u + 2 are outstanding; this wave has read all of stage u and
          // written its part of stage u + 1.  Behind the barrier the buffers of
          // stage u are free and those of stage u + 1 whole.
          wait_vmcnt_lgkm0<C::kCPW + Piece<KIND>::kLoads>();
          stage_barrier();
          set_a(abuf1);
          read_a(0);
        } else {
          read_a(gi + 1);
        }
        __builtin_amdgcn_sched_barrier(0);
        // pieces of stages u + 1 and u + 2; groups that load, copy and convert
        constexpr int kNext = kSets == 2 ? 1 - J : 0, kLoad = kSets == 2 ? J : 0;
        constexpr int kPer = 2, kConv = kSets == 2 ? 1 : 0;
        constexpr int kLoadAt = kSets == 2 ? 0 : 4 / kPer, kCopyAt = kLoadAt + 1;
        static_assert(kCopyAt < kGroups - 1 && kConv + 4 / kPer <= kGroups - 1, "before the last group's wait");
        if (gi == kLoadAt) {
          load_b(raw[kLoad], idx[J], ok[kLoad]);
          if constexpr (GATHER) idx[J] = row_index(u + 4);
        }
        if (gi == kCopyAt) copy_a(nbuf);
        // The group's products.  A product occupies the matrix pipe for 16
        // cycles, in which three or four other instructions issue: the loads'
        // addresses, the conversion of a part of stage u + 1's B, and in a
        // step's last group B's next fragments, each as soon as the products
        // of the one before it are issued.
        constexpr int kLast = kG - 1;
        const bool conv = gi >= kConv && gi < kConv + 4 / kPer, last = gi % kG == kLast;
#pragma unroll
        for (int j = 0; j < C::kKT; ++j) {
#pragma unroll
          for (int q = 0; q < kGT; ++q)
            acc[kGT * (gi % kG) + q][j] = mma16x16x32(fb[j], fa[gi & 1][q], acc[kGT * (gi % kG) + q][j]);
          if (last) read_b(gi == kGroups - 1 ? 1 - J : J, gi == kGroups - 1 ? 0 : gi / kG + 1, j);
        }
        if (conv) {
#pragma unroll
          for (int i = 0; i < kPer; ++i) store_b(raw[kNext], ok[kNext], 1 - J, kPer * (gi - kConv) + i);
        }
        if (last) {
#pragma unroll
          for (int j = 0; j < C::kKT; ++j) {
            __builtin_amdgcn_sched_group_barrier(0x008, kGT, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
          }
        } else {
#pragma unroll
          for (int q = 0; q < kGT * C::kKT; ++q) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x006, 6, 0);
            if (!conv) __builtin_amdgcn_sched_group_barrier(0x020, 2, 0);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      abuf = abuf1;
    };
    int u = 0;
    for (; u + 1 < stages; u += 2) {
      stage(u, std::integral_constant<int, 0>());
      stage(u + 1, std::integral_constant<int, 1>());
    }
    if (u < stages) stage(u, std::integral_constant<int, 0>());
    wait_vmcnt_lgkm0<0>();  // no copy into LDS may still be running at exit
  }

  // Register q of tile j in lane 16 g + 4 a + b holds row 4 a + b and, of the
  // wave's 64 columns, 32 (g / 2) + 16 (j % 2) + 8 (j / 2) + 4 (g % 2) + q.
  // Stores go out at four lanes (one quad) per cycle if these lie in one 64-byte
  // piece, else at a quarter of that (a CU: 151 against 35 GB/s), so lanes trade
  // registers until quads do: fp32, 4 rows of 256 bytes per instruction, column
  // 16 g + 4 b + q; bf16, 8 rows of 128 bytes.
  const float gs = KIND == 2 ? *g.gs : 1.0f;
  const bool odd = lane & 1, upper = lane & 2;
  const int kw = k0 + 64 * wk;
  const bool f32 = (kWM == 1 && splits > 1) || (WGRAD && g.out_f32);
#pragma unroll
  for (int t = 0; t < kMT; ++t) {
    const int mt0 = m0 + 16 * (wm * kMT + t) + (lane & 12);
    if constexpr (KIND == 2)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[t][j] *= gs;
    if (f32) {
      u32x4_t v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = __builtin_bit_cast(u32x4_t, acc[t][j]);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint32_t x[4] = {v[0][q], v[1][q], v[2][q], v[3][q]};
        swap16(x[0], x[1]);
        swap16(x[2], x[3]);
        swap_quad<0>(odd, x[0], x[1]);
        swap_quad<0>(odd, x[2], x[3]);
        swap_quad<1>(upper, x[0], x[2]);
        swap_quad<1>(upper, x[1], x[3]);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j][q] = x[j];
      }
      const int k = kw + 16 * gq + 4 * (lane & 3);
#pragma unroll
      for (int j = 0; j < 4; ++j) {                            // rows 4 a + j
        const f32x4_t o4 = __builtin_bit_cast(f32x4_t, v[j]);
        const int64_t row = WGRAD ? (int64_t)e * N + mt0 + j : mt0 + j;
        if (k >= K || mt0 + j >= m_end) continue;
        if (kWM == 1 && splits > 1)                            // a part of the sum, for join_kernel
          *reinterpret_cast<f32x4_t*>(g.workspace + ((int64_t)split * (WGRAD ? (int64_t)g.E * N : P) + row) * K + k) = o4;
        else
          store_f32(static_cast<float*>(g.out) + row * g.ldo + k, o4, g.accumulate);
      }
    } else {
      u32x4_t v[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t x[4];                                         // words h of the four tiles
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          x[2 * j] = pk_bf16(acc[t][2 * j][2 * h], acc[t][2 * j][2 * h + 1]);
          x[2 * j + 1] = pk_bf16(acc[t][2 * j + 1][2 * h], acc[t][2 * j + 1][2 * h + 1]);
          swap16(x[2 * j], x[2 * j + 1]);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          swap_quad<0>(odd, x[j], x[j + 2]);
          swap16(x[j], x[j + 2]);
          swap_quad<1>(upper, x[j], x[j + 2]);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          v[0][2 * j + h] = x[j];
          v[1][2 * j + h] = x[j + 2];
        }
      }
      const int k = kw + 32 * (gq >> 1) + 8 * (lane & 3);
#pragma unroll
      for (int j = 0; j < 2; ++j) {                            // rows 4 a + 2 j + g % 2
        const int m = mt0 + 2 * j + (gq & 1);
        if (k < K && m < m_end)
          *reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(g.out) + (WGRAD ? (int64_t)e * N + m : m) * g.ldo + k) = v[j];
      }
    }
  }
}

template <bool WGRAD, int KIND, int LAYOUT, bool GATHER, int kWM, int kWK, int kMT>
__global__ void __launch_bounds__(64 * kWM * kWK, kMT > 4 ? 2 : 3)
grad_kernel(GradArgs g, int mtiles, int ktiles, int tiles, int splits, int turn) {
  constexpr int BM = 16 * kMT * kWM;
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  // block of C: the XCDs take turns of `turn` blocks, in groups of 4 row tiles
  const int xcd = blockIdx.x & 7, i = blockIdx.x >> 3;
  const int all = (i / turn * 8 + xcd) * turn + i % turn;
  if (all >= tiles * splits) return;
  const int split = all / tiles, lin = all - split * tiles;
  const int P = (int)g.P;
  const int per_e = WGRAD ? mtiles * ktiles : tiles;
  int e = WGRAD ? lin / per_e : 0;
  const int in_e = lin - e * per_e;
  const int gsz = 4 * ktiles, first_m = (in_e / gsz) * 4, gm = min(mtiles - first_m, 4);
  const int mt = first_m + (in_e % gsz) % gm, k0 = ((in_e % gsz) / gm) * kBK;
  int lo, hi, m0;     // the expert's rows; first row (dgrad) / first n (wgrad) of the block
  if constexpr (WGRAD) {
    segment(g.offsets, e, P, lo, hi);
    m0 = mt * BM;
  } else {
    if (!find_tile<BM>(g.offsets, g.E, P, mt, e, lo, hi)) return;
    e = __builtin_amdgcn_readfirstlane(e);
    lo = __builtin_amdgcn_readfirstlane(lo);
    hi = __builtin_amdgcn_readfirstlane(hi);
    m0 = lo;
    // an expert's last rows: half a block does (64 x 2048 x 7168, 32768 ragged
    // rows 951 -> 931 us, 16384 rows 572 -> 540; of 64-row blocks it does not:
    // 512 rows 141 -> 171)
    if constexpr (kWM == 1 && kMT > 4)
      if (hi - m0 <= BM / 2)
        return make_block<WGRAD, KIND, LAYOUT, GATHER, kWM, kWK, kMT / 2>(g, smem, e, lo, hi, m0, k0, split, splits);
  }
  make_block<WGRAD, KIND, LAYOUT, GATHER, kWM, kWK, kMT>(g, smem, e, lo, hi, m0, k0, split, splits);
}

// out[row][k] (+)= the sum of the splits' parts, in order; four columns per
// thread.  dgrad: only the rows inside the experts' ranges.
__global__ void __launch_bounds__(256)
join_kernel(GradArgs g, int64_t rows, int splits, int wgrad) {
  const int64_t cpr = g.K / 4, c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (c >= rows * cpr) return;
  const int64_t row = c / cpr, k = (c - row * cpr) * 4;
  if (!wgrad && g.offsets && (row < g.offsets[0] || row >= g.offsets[g.E])) return;
  const float* p = g.workspace + row * g.K + k;
  f32x4_t v{0.0f, 0.0f, 0.0f, 0.0f};
  for (int s = 0; s < splits; ++s) v += *reinterpret_cast<const f32x4_t*>(p + (int64_t)s * rows * g.K);
  if (wgrad && g.out_f32) {
    f32x4_t* o = reinterpret_cast<f32x4_t*>(static_cast<float*>(g.out) + row * g.ldo + k);
    *o = g.accumulate ? *o + v : v;
  } else {
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(g.out) + row * g.ldo + k) =
        make_uint2(pk_bf16(v[0], v[1]), pk_bf16(v[2], v[3]));
  }
}

// ---- which block and how many parts ------------------------------------------
// By the sizes alone (the experts' own row counts are on the device; P / E is
// their mean).  Measured on 2048 x 7168 experts and dense layers:
//   256 rows  (8 waves, one workgroup per CU) moves a third less from L2 per
//             product and converts B half as often as 128 rows (4 waves, two
//             per CU), but overlaps less and rounds the experts' rows up
//             further: dgrad 4 x 2048 rows 215 vs 246 us, 8 x 1024 rows 257 vs
//             249, 16 x 512 300 vs 250; wgrad (8-bit, ragged) 8 x 1024 rows 293
//             vs 305, 64 x 256 1017 vs 1055; dense 8192 x 8192 with 1024 rows
//             168 vs 177, 512 116 vs 110, 256 88 vs 77.  It needs a block for
//             each of the 256 CUs.
//   64 rows   wins where rows are few: dgrad 64 x 32 rows 205 vs 251 us, 64 x 8
//             154 vs 222, 64 x 256 655 vs 609; wgrad 64 x 8 rows 652 vs 735.
// Where the blocks would leave CUs idle, 64 rows also put more CUs to work (wgrad
// 512 x 2048 x 2048, 8 bits: 15 vs 19 us), and the sum may be split over
// workgroups that write fp32 parts, joined by a second kernel: the block and as
// many parts as cost least by the measured time of a stage of 32 summed rows in
// a workgroup that has its CU to itself (dgrad 0.45 us, wgrad 0.6 in 64 rows and
// 0.8 in 128), of the second launch (8 us with its host time) and of the parts
// (3.5 TB/s).  dgrad 16 x 8192 x 8192: 106 us in one part, 24 in 16; 256 x 8192
// x 8192: 111 in one, 59 in 4; wgrad 8192 x 2048 x 2048 (8-bit): 182 in one,
// 84 in 4 of 128 rows, 108 in 2 of 64; 1000 x 640 x 512: 29 in one, 14 in 4.
constexpr int64_t kFill = 512;      // workgroups that fill the GPU: two per CU
constexpr int64_t kDgradStageNs = 450, kWgradStage64Ns = 600, kWgradStage128Ns = 800;
constexpr int64_t kJoinNs = 8000, kJoinBytesPerNs = 3500;
enum { kBlock64, kBlock128, kBlock256 };
struct Plan {
  int block, splits;
};

Plan plan(bool wgrad, int64_t P, int64_t E, int64_t N, int64_t K) {
  const int64_t per = P / E, kt = (K + kBK - 1) / kBK;
  auto tiles = [&](int64_t bm) { return wgrad ? E * ((N + bm - 1) / bm) * kt : ((P + bm - 1) / bm + E - 1) * kt; };
  if (tiles(256) >= 256 && per >= (!wgrad ? 2048 : E > 1 ? 256 : 1024)) return {kBlock256, 1};
  const int64_t stages = ((wgrad ? per : N) + 31) / 32;
  const int64_t part = (wgrad ? E * N : P) * K * 8 / kJoinBytesPerNs;   // writing and reading a part, ns
  Plan best{};
  int64_t least = INT64_MAX;
  auto consider = [&](int block, int64_t bm, int64_t stage_ns) {
    const int64_t most = std::min(kFill / tiles(bm), stages);
    for (int s = 1; s == 1 || s <= most; ++s) {
      const int64_t ns = (stages + s - 1) / s * stage_ns + (s > 1 ? kJoinNs + s * part : 0);
      if (ns < least) {
        least = ns;
        best = {block, s};
      }
    }
  };
  const bool few = per <= (wgrad ? 32 : 128), idle = tiles(128) < 256;
  if (few || idle) consider(kBlock64, 64, wgrad ? kWgradStage64Ns : kDgradStageNs);
  if (!few && (wgrad || !idle)) consider(kBlock128, 128, wgrad ? kWgradStage128Ns : kDgradStageNs);
  return best;
}

// Blocks that an XCD takes in a row, neighbours that meet in its L2: 4 row tiles
// by up to 8 columns, so that every XCD has a part of each expert (their rows
// differ, and unused row tiles come last); with few blocks, its whole share.
// Against whole shares always, ragged experts of 2048 x 7168: wgrad (8-bit) 16 x
// 512 rows 462 -> 374 us, 64 x 256 1116 -> 1011, dgrad 64 x 32 205 -> 173; dense
// the same.
int64_t turn_of(int64_t total, int64_t kt) {
  const int64_t share = (total + 7) / 8, part = 4 * ((kt + (kt + 7) / 8 - 1) / ((kt + 7) / 8));
  return total >= 64 * part ? part : std::max<int64_t>(share, 1);
}

template <bool WGRAD, int KIND, int LAYOUT, bool GATHER, int kWM, int kWK, int kMT>
hipError_t run(const GradArgs& g, int splits, hipStream_t stream) {
  using C = Kern<WGRAD, KIND, LAYOUT, GATHER, kWM, kWK, kMT>;
  const int64_t kt = (g.K + kBK - 1) / kBK;
  const int64_t mt = WGRAD ? (g.N + C::BM - 1) / C::BM : (g.P + C::BM - 1) / C::BM + g.E - 1;
  const int64_t tiles = mt * kt * (WGRAD ? g.E : 1);
  const hipError_t attr = set_max_lds<&grad_kernel<WGRAD, KIND, LAYOUT, GATHER, kWM, kWK, kMT>>(C::kSmem);
  if (attr != hipSuccess) return attr;
  const int64_t total = tiles * splits, turn = turn_of(total, kt);
  grad_kernel<WGRAD, KIND, LAYOUT, GATHER, kWM, kWK, kMT>
      <<<(unsigned)((total + 8 * turn - 1) / (8 * turn) * (8 * turn)), C::kThreads, C::kSmem, stream>>>(
          g, (int)mt, (int)kt, (int)tiles, splits, (int)turn);
  if (splits > 1) {
    const int64_t rows = WGRAD ? g.E * g.N : g.P;
    join_kernel<<<(unsigned)((rows * (g.K / 4) + 255) / 256), 256, 0, stream>>>(g, rows, splits, WGRAD);
  }
  return hipGetLastError();
}

template <bool WGRAD, int KIND, int LAYOUT, bool GATHER>
hipError_t run_plan(const GradArgs& g, hipStream_t stream) {
  const GradPlan p = grad_plan(WGRAD, KIND == kBf16Piece, g.P, g.E, g.N, g.K);
  if (p.rows == 64) return run<WGRAD, KIND, LAYOUT, GATHER, 1, 4, 4>(g, p.parts, stream);
  if (p.rows == 128 || KIND == kBf16Piece) return run<WGRAD, KIND, LAYOUT, GATHER, 1, 4, 8>(g, p.parts, stream);
  if constexpr (KIND != kBf16Piece) return run<WGRAD, KIND, LAYOUT, GATHER, 2, 4, 8>(g, 1, stream);
}

template <int KIND, int LAYOUT>
hipError_t run_dgrad(const GradArgs& g, hipStream_t stream) {
  return run_plan<false, KIND, LAYOUT, false>(g, stream);
}

template <int KIND>
hipError_t run_wgrad(const GradArgs& g, hipStream_t stream) {
  return g.gather ? run_plan<true, KIND, kLayoutRows, true>(g, stream)
                  : run_plan<true, KIND, kLayoutRows, false>(g, stream);
}

size_t parts_bytes(bool wgrad, int64_t P, int64_t E, int64_t N, int64_t K) {
  const int splits = plan(wgrad, P, E, N, K).splits;
  return splits > 1 ? (size_t)splits * (size_t)(wgrad ? E * N : P) * (size_t)K * 4 : 0;
}

constexpr int64_t kMaxTiles = (int64_t)1 << 22;   // of at most 512 threads each
constexpr int64_t kMaxSum = (int64_t)1 << 30;

}  // namespace

GradPlan grad_plan(bool wgrad, bool a_bf16, int64_t P, int32_t E, int64_t N, int64_t K) {
  const Plan p = plan(wgrad, P, E, N, K);
  // (bf16 activations fill the registers of the 256-row block)
  return {p.block == kBlock64 ? 64 : p.block == kBlock128 || a_bf16 ? 128 : 256, p.splits};
}
size_t dgrad_workspace(int64_t P, int32_t E, int64_t N, int64_t K) { return parts_bytes(false, P, E, N, K); }
size_t wgrad_workspace(int64_t P, int32_t E, int64_t N, int64_t K) { return parts_bytes(true, P, E, N, K); }

// (64-row tiles, the smallest; a summed row plus a stage stays an int)
bool dgrad_fits(int64_t P, int32_t E, int64_t N, int64_t K) {
  return ((P + 63) / 64 + E) * ((K + kBK - 1) / kBK) <= kMaxTiles;
}
bool wgrad_fits(int64_t P, int32_t E, int64_t N, int64_t K) {
  return P <= kMaxSum && E * ((N + 63) / 64) * ((K + kBK - 1) / kBK) <= kMaxTiles;
}

hipError_t launch_dgrad(int fmt, int layout, const GradArgs& g, hipStream_t stream) {
  const bool t = layout == kLayoutTiled;
  switch (fmt) {
    case 0: return t ? run_dgrad<0, kLayoutTiled>(g, stream) : run_dgrad<0, kLayoutRows>(g, stream);
    case 1: return t ? run_dgrad<1, kLayoutTiled>(g, stream) : run_dgrad<1, kLayoutRows>(g, stream);
    case 4: return t ? run_dgrad<4, kLayoutTiled>(g, stream) : run_dgrad<4, kLayoutRows>(g, stream);
    default: return t ? run_dgrad<2, kLayoutTiled>(g, stream) : run_dgrad<2, kLayoutRows>(g, stream);
  }
}

hipError_t launch_wgrad(int kind, const GradArgs& g, hipStream_t stream) {
  switch (kind) {
    case kMxFp8: return run_wgrad<kMxFp8>(g, stream);
    case kMxInt8: return run_wgrad<kMxInt8>(g, stream);
    default: return run_wgrad<kBf16Piece>(g, stream);
  }
}

}  // namespace q4
