/*
 * q4.h -- C ABI of libq4.so: 4-bit absmax block quantization of bf16
 * weights (INT4 g128, MXFP4, NVFP4) and the W4 matmuls that consume them,
 * as hand-written HIP kernels for AMD gfx950 (MI355X).
 *
 * Formats (one row of K values is split into blocks of g along K):
 *   Q4_INT4_G128  codes -8..7 (4-bit two's complement), one fp16 scale per
 *                 128 values, scale = fp16(amax/7), code = clamp(rne(w/s)).
 *                 ("Quantization in deployment", format cheat sheet, W4A16
 *                 row; "Low-bit inference for very large MoE", fake_int4;
 *                 "Quantization chains", bits per weight: 4.125.)
 *   Q4_MXFP4      E2M1 codes (grid +-{0,0.5,1,1.5,2,3,4,6}), one E8M0
 *                 power-of-two scale per 32 values,
 *                 scale = 2^(floor(log2(max(amax,1e-12))) - 2).
 *                 ("Quantization in deployment", formats.py mxfp4(); 4.25 bits.)
 *   Q4_NVFP4      E2M1 codes, one E4M3 scale per 16 values plus one fp32
 *                 tensor scale gs = max(amax_tensor,1e-12)/2688;
 *                 block scale = E4M3(min(amax_b/6/gs, 448)), element
 *                 divided by E4M3(scale)*gs.  ("Quantization in deployment",
 *                 formats.py nvfp4(); "Quantization chains", NVFP4 vs MXFP4.)
 *   Q4_INT4_ZP_G128  INT4 with a zero point: codes -8..7 (4-bit two's
 *                 complement), per group of 128 one fp16 scale and one zero
 *                 point z (an integer code), value = (q - z) * scale; min-max
 *                 rounding over the group widened to include 0: lo =
 *                 min(min,0), hi = max(max,0), scale = fp16((hi-lo)/15),
 *                 z = clamp(-8 - rne(lo/scale), -8, 7), q = clamp(rne(w/
 *                 scale) + z, -8, 7).  ("Quantization in deployment",
 *                 format cheat sheet, W4A16 INT4 GPTQ/AWQ row: one scale
 *                 per 128 numbers plus a zero point.)  Scales are 32-bit
 *                 words: fp16 bits | (z & 0xFF) << 16.
 *   Q4_FP8_ROW    the activation operand of W4A8, not a weight format:
 *                 one E4M3 byte per value and one fp32 scale per row
 *                 (token), scale = max(amax_row,1e-12)/448, code =
 *                 E4M3(clamp(x/scale, +-448)).  ("Quantization in
 *                 deployment", formats.py fp8() per row; "Quantization
 *                 chains", "One outlier sets the scale".)
 *   Q4_INT8_ROW   both operands of W8A8: one two's complement byte per value
 *                 and one fp32 scale per row (a token of the activations, an
 *                 output channel of a weight), with a = max(amax_row, 1e-12):
 *                 scale = a/127, code = rne(x * fp32(127/a)) of the exact
 *                 product, so -127..127.  A row with an infinity or a NaN gets
 *                 the scale NaN, and every product with it is NaN.
 *                 ("Quantization in deployment", format cheat sheet, W8A8;
 *                 "LLM quantization", the absmax method.)
 *   Q4_MXINT8, Q4_MXFP8  activations saved for the backward pass, not an
 *                 operand of a W4 product: one byte per value and one
 *                 power-of-two scale per 32 values, stored as the byte b of
 *                 2^(b-127).  scale = the least 2^e >= 2^-111 with
 *                 max|x| <= top * 2^e; code = rne(x / scale) as a two's
 *                 complement byte (MXINT8, top = 127) or an E4M3 byte (MXFP8,
 *                 top = 448).  Integers err by at most scale / 2 everywhere:
 *                 1/254 to 1/127 of the block's largest value, more where
 *                 that is below 2^-104 (2^-111 is the least scale).  E4M3 errs
 *                 by at most max(2^-4 |x|, 2^-10 scale) of each value x:
 *                 integers suit ordinary blocks, E4M3 blocks in which one
 *                 outlier would leave the rest few codes.  A block with
 *                 an infinity or a NaN has b = 255 and reads back as NaN
 *                 throughout; a code whose value would reach 2^128 is stored
 *                 one lower (so the largest bf16 number errs by 3/4 scale in
 *                 integers).  8.25 bits per value.
 *                 Not the interchange formats of these names: MXINT8's
 *                 codes are whole scales, not 64ths of one, and both
 *                 formats' rule for the scale (the least that does not clip)
 *                 is this library's own.
 * Every rounding is to nearest, ties to the even code; E2M1 and E4M3 keep
 * the sign bit of the input; a block whose stored scale is 0 has magnitude
 * codes 0.
 *
 * Layouts of a quantized tensor (q4_tensor); all device memory is owned by
 * the caller.  Within a byte, element k sits in bits 3:0 when k is even and
 * in bits 7:4 when k is odd.  INT4 codes are 4-bit two's complement; an
 * E2M1 code is sign*8 + index into {0,0.5,1,1.5,2,3,4,6}.
 *
 * Q4_LAYOUT_ROWS (row-major, dense):
 *   codes   uint8 [rows][cols/2], 16-byte aligned.
 *   scales  INT4: fp16 bits [rows][cols/128]; MXFP4: biased E8M0 exponent
 *           [rows][cols/32]; NVFP4: E4M3 bits [rows][cols/16]; INT4 with a
 *           zero point: 32-bit words [rows][cols/128].  4-byte aligned.
 *
 * Q4_LAYOUT_TILED (the weights pre-shuffled so that one 64-lane load is one
 * contiguous kilobyte holding a whole matrix-core operand; cols % 512 == 0).
 * Rows are grouped in tiles of 16 (RT = ceil(rows/16) tiles, the last one
 * padded), K in super-chunks of 128 (S = cols/128) and super-chunks in
 * groups of four (Q = S/4).  Lane index l = 16*g + n, n = row in the tile
 * (0..15), g = 32-wide k group in the super-chunk (0..3).
 *   codes   RT*S tiles of 1024 bytes; tile (t, s) starts at byte
 *           (t*S + s)*1024 and its bytes [16l, 16l+16) hold the 32 codes
 *           k = 128s + 32g + j (j = 0..31) of row 16t + n.
 *   scales  MXFP4: byte ((t*Q + q)*64 + l)*4 + i is the E8M0 of row 16t+n,
 *                  32-block 4(4q+i) + g                 (RT*Q*256 bytes);
 *           NVFP4: byte ((t*Q + q)*64 + l)*8 + 2i + h is the E4M3 of row
 *                  16t+n, 16-block 8(4q+i) + 2g + h    (RT*Q*512 bytes);
 *           INT4:  fp16 element ((t*Q + q)*16 + n)*4 + i is the scale of
 *                  row 16t+n, 128-group 4q + i          (RT*Q*128 bytes);
 *           INT4 with a zero point: the 32-bit word at the same element
 *                  index                                (RT*Q*256 bytes).
 *   Padding rows (16t+n >= rows) hold the quantization of zeros.
 *
 * Q4_FP8_ROW in the two layouts (cols % 16 == 0 row-major, % 512 tiled):
 *   row-major  codes uint8 [rows][cols] (E4M3 bytes, sign in bit 7).
 *   tiled      RT*S tiles of 2048 bytes, tile (t, s) at (t*S + s)*2048.
 *              Lane l = 16g + n owns 32 operand bytes of row 16t+n:
 *              operand byte 4d + i (dword d = 2w + h, w = 0..3, h = 0..1,
 *              i = 0..3) holds k = 128s + 32g + 8w + 2i + h.  Operand
 *              bytes 0..15 of lane l sit at tile byte 16l, operand bytes
 *              16..31 at 1024 + 16l.  Padding rows hold code 0.
 *   scales     fp32 [rows] in both layouts; global_scale is NULL.
 *
 * Q4_INT8_ROW (row-major only, cols % 16 == 0): codes int8 [rows][cols],
 *   scales fp32 [rows]; global_scale is NULL.
 *
 * Q4_MXINT8 and Q4_MXFP8 (row-major only, cols % 32 == 0): codes uint8
 *   [rows][cols], scales uint8 [rows][cols/32]; global_scale is NULL.
 *
 *   global_scale  NVFP4 only: device fp32[1], the multiplier gs; else NULL.
 *
 * Conventions for every call:
 *   - Pointers named *_bf16 are device bf16 arrays; leading dimensions (ld*)
 *     are in elements, >= the row length, multiples of 8, and the base
 *     pointers 16-byte aligned.
 *   - `stream` is a hipStream_t (NULL = the default stream).  All device work
 *     is enqueued on it; the call returns after the launch, not after the
 *     work.  The library never allocates, frees or synchronizes.
 *   - Arguments are validated on the host before any HIP call; a bad
 *     argument returns its error code and launches nothing.  A failed launch
 *     returns Q4_ERR_HIP; q4_last_hip_error() gives the hipError_t of the
 *     calling thread's last failure.
 *   - Inputs must be finite, but where a format or call says what it makes
 *     of infinities and NaN.  Calls on distinct outputs may run
 *     concurrently; outputs must not alias inputs.
 *   - The first launch of a kernel that uses more than 64 KB of LDS on a
 *     device raises that kernel's LDS limit there (hipFuncSetAttribute, once
 *     per kernel and device); no other state is kept.
 */
#ifndef Q4_H
#define Q4_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum q4_format {
    Q4_INT4_G128 = 0,
    Q4_MXFP4 = 1,
    Q4_NVFP4 = 2,
    Q4_FP8_ROW = 3,
    Q4_INT4_ZP_G128 = 4,
    Q4_MXFP8 = 5,
    Q4_MXINT8 = 6,
    Q4_INT8_ROW = 8 /* (7 is no format) */
} q4_format;

typedef enum q4_layout {
    Q4_LAYOUT_ROWS = 0,
    Q4_LAYOUT_TILED = 1
} q4_layout;

typedef enum q4_status {
    Q4_OK = 0,
    Q4_ERR_NULL = -1,   /* a required pointer is NULL                      */
    Q4_ERR_SHAPE = -2,  /* a size is negative, too large or not a multiple */
    Q4_ERR_ALIGN = -3,  /* a pointer or leading dimension is misaligned    */
    Q4_ERR_FORMAT = -4, /* unknown format, or a format the call rejects    */
    Q4_ERR_HIP = -6     /* the HIP launch failed; see q4_last_hip_error()  */
} q4_status;

typedef struct q4_tensor {
    int32_t fmt;          /* q4_format                                     */
    int32_t layout;       /* q4_layout                                     */
    int64_t rows;         /* N for weights, M for activations              */
    int64_t cols;         /* K, a multiple of the format's block size      */
    void* codes;          /* packed codes, see the layouts above           */
    void* scales;         /* block scales, see the layouts above           */
    float* global_scale;  /* NVFP4: fp32[1]; other formats: NULL           */
} q4_tensor;

/* Library version (major*100 + minor). */
int q4_version(void);

/* Static text for a q4_status value. */
const char* q4_status_string(int status);

/* hipError_t of the calling thread's last Q4_ERR_HIP (0 if none). */
int q4_last_hip_error(void);

/*
 * Bytes of codes and scales for a rows x cols tensor of format fmt in
 * layout `layout` ("Quantization chains", bits per weight: codes are 4 bits,
 * scales 16/128, 8/32 and 8/16 bits per value; the tiled layout adds the
 * padding of the last row tile).  Either output pointer may be NULL.
 * Q4_ERR_SHAPE if rows < 0, cols < 0 or cols is not a multiple of the block
 * (of 512 for the tiled layout); Q4_ERR_FORMAT for an unknown fmt/layout.
 */
q4_status q4_sizes(int fmt, int layout, int64_t rows, int64_t cols, size_t* codes_bytes,
                   size_t* scales_bytes);

/*
 * Moves a quantized tensor from one layout to the other (row-major <->
 * tiled, the layouts above), bit for bit: the same codes and scales at the
 * other layout's positions, the NVFP4 global scale copied.  Tiled padding
 * rows receive the quantization of zeros (as q4_quantize writes them).  The
 * GEMM kernels are built for the tiled layout (its fragments are contiguous
 * kilobytes; "Low-bit inference for very large MoE", "A few details":
 * pre-shuffled weights), so weights quantized or packed row-major are worth
 * converting once, when they are loaded.
 *   src, dst  the same weight format (else Q4_ERR_FORMAT), rows and cols
 *             (else Q4_ERR_SHAPE); each validated like any q4_tensor (the
 *             tiled one needs cols % 512 == 0).  Equal layouts: a copy.
 *   dst must not overlap src.  Empty tensors: only the NVFP4 global scale
 *   is copied.
 */
q4_status q4_relayout(const q4_tensor* src, const q4_tensor* dst, void* stream);

/*
 * Quantize a bf16 matrix src [dst->rows][ld] (first dst->cols columns) into
 * dst, by round-to-nearest absmax block quantization along each row
 * ("LLM quantization", the absmax method: the group's largest magnitude
 * sets the scale, every value is divided by it and rounded).
 * NVFP4: if nv_global_in (device fp32[1]) is not NULL its value is used as
 * gs; otherwise gs is computed from the whole matrix (one extra read pass)
 * and written to dst->global_scale.  nv_global_in must be NULL for the other
 * formats.  rows == 0 or cols == 0 is a no-op (for NVFP4 without
 * nv_global_in, gs is still written: max(0,1e-12)/2688).  Q4_FP8_ROW
 * quantizes each row with its own scale (the W4A8 activations), Q4_INT8_ROW
 * likewise (W8A8's activations and weights; rows < 2^22, else Q4_ERR_SHAPE).
 */
q4_status q4_quantize(const void* src_bf16, int64_t ld, const q4_tensor* dst,
                      const float* nv_global_in, void* stream);

/*
 * Dequantize src into dst [src->rows][ld]: value = fp32(code * scale) with
 * the scale as stored (NVFP4: scale = fp32(E4M3 * gs)).  dst_dtype 0 writes
 * bf16 (the fp32 value rounded to nearest even), 1 writes fp32 (ld a
 * multiple of 4 for fp32).  This is the step that multiplies the rounded
 * values back by their scale in the worked example of "LLM quantization".
 * Either layout is read; the output is always row-major.
 */
q4_status q4_dequant(const q4_tensor* src, void* dst, int dst_dtype, int64_t ld, void* stream);

/*
 * W4A16 GEMV for decode: y[b][n] = sum_k x[b][k] * w'[n][k] for b < B,
 * n < W->rows, w' the dequantized weight; fp32 accumulation, bf16 output
 * ("Low-bit inference for very large MoE", table "Kernels on different
 * hardware", row W4A16: weights dequantized in registers, 16-bit compute).
 * x_bf16 [B][ldx], y_bf16 [B][ldy].  1 <= B <= 16; K = W->cols must be a
 * multiple of 128.  B == 0 or W->rows == 0 is a no-op.
 */
q4_status q4_gemv(const q4_tensor* W, const void* x_bf16, int64_t B, int64_t ldx,
                  void* y_bf16, int64_t ldy, void* stream);

/*
 * GEMM C[m][n] = sum_k a'[m][k] * w'[n][k], fp32 accumulation, bf16 output
 * C_bf16 [M][ldc].  Exactly one of A_bf16 / A_q is given:
 *   A_bf16 [M][lda]  -> W4A16: W of any format dequantized to bf16 feeding
 *                       bf16 matrix cores (same table, row W4A16);
 *   A_q (MXFP4, rows M, cols K) with W MXFP4 -> W4A4: both operands enter
 *                       the block-scaled FP4 matrix cores directly (same
 *                       table, row W4A4);
 *   A_q (NVFP4, rows M, cols K) with W NVFP4 -> W4A4 NVFP4: each code times
 *                       its E4M3 block scale is exact in fp16, so both
 *                       operands are dequantized to fp16 in registers and
 *                       multiplied on fp16 matrix cores; the two tensor
 *                       scales are applied to the fp32 sum:
 *                       C = (sum_k (qa sa)(qw sw)) * gs_a * gs_w.  A_q's
 *                       global_scale is its own (q4_quantize of A computes
 *                       it from A's amax, or takes the caller's).  gfx950's
 *                       FP4 matrix cores take E8M0 scales per 32, which
 *                       cannot carry E4M3 per 16 ("Quantization in
 *                       deployment", cheat sheet, NVFP4 and MXFP4 rows);
 *   A_q (Q4_FP8_ROW, rows M, cols K) with W INT4 -> W4A8: the INT4 codes
 *                       become exact E4M3 values, the products run on FP8
 *                       matrix cores, and each 128-wide group's partial sum
 *                       is multiplied by its fp16 weight scale in fp32 (same
 *                       table, row W4A8; "Quantization in deployment", the
 *                       per-block promotion of block-scaled FP8 GEMMs);
 *                       C = s_a[m] * sum_g s_w[n][g] * sum_(k in g) a8*q.
 *   A_q (Q4_INT8_ROW, rows M, cols K) with W Q4_INT8_ROW -> W8A8: sums of
 *                       products of bytes, exact in 32-bit integers (K < 2^17
 *                       and N < 2^27, else Q4_ERR_SHAPE), one scale of the token and one of
 *                       the channel on the sum:
 *                       C = (s_a[m] * s_w[n]) * sum_k a8*w8.
 * Other format pairs, and a Q4_FP8_ROW W: Q4_ERR_FORMAT.
 * K = W->cols must be a multiple of 128.  M == 0 or N == 0 is a no-op.
 */
q4_status q4_gemm(int64_t M, const void* A_bf16, int64_t lda, const q4_tensor* A_q,
                  const q4_tensor* W, void* C_bf16, int64_t ldc, void* stream);

/*
 * The GEMM of q4_gemm with its output written quantized by the kernel's
 * epilogue: C_q receives exactly the codes and scales that q4_quantize(C_q)
 * writes for the bf16 C that q4_gemm writes (each fp32 sum rounded to bf16,
 * then block-quantized), and C is never written in bf16 nor read back.  This
 * is the activation quantization of the next W4A4 layer done at the end of
 * the kernel that produces the activations, which saves a pass that reads
 * and writes them ("Quantization in deployment", Exercises, "The cost of
 * block FP8": activation scales computed at the end of the previous kernel).
 *   C_q  MXFP4, or NVFP4 with the tensor scale taken from nv_global_in
 *        (device fp32[1]; required for NVFP4 and NULL otherwise; its value
 *        is also written to C_q->global_scale: an epilogue cannot wait for
 *        the amax of the whole output, so the scale is the caller's, e.g.
 *        a calibrated one).  C_q->rows == M, C_q->cols == N == W->rows,
 *        N % 32 == 0; either layout (tiled: N % 512 == 0, padding rows
 *        written as the quantization of zeros).
 *   Operands: A_bf16 [M][lda] with W of any weight format in the tiled
 *        layout (W4A16), or A_q MXFP4 tiled with W MXFP4 tiled (W4A4).
 *        Other combinations: Q4_ERR_FORMAT.
 * M == 0 or N == 0 is a no-op.  C_q must not alias the operands.
 */
q4_status q4_gemm_quantized(int64_t M, const void* A_bf16, int64_t lda, const q4_tensor* A_q,
                            const q4_tensor* W, const q4_tensor* C_q, const float* nv_global_in,
                            void* stream);

/*
 * Root-mean-square norm in front of the products, with the residual's addition
 * and the quantization of their activations in the same pass ("Quantization in
 * deployment", Exercises, "The cost of block FP8": activation scales computed
 * at the end of the previous kernel):
 *     h = bf16(x + residual)           (without a residual h = x, not written)
 *     y = h * weight / sqrt(mean_k(h^2) + eps)        (fp32, from h as stored)
 * y_bf16 receives y rounded to bf16, y_q (Q4_FP8_ROW in either layout, or
 * Q4_INT8_ROW) its 8-bit codes and row scales, from the fp32 values and not by
 * way of bf16: scale = max(amax_row(|y|), 1e-12) / top (448, 127), code = the
 * nearest to y / scale, ties to even, y and the quotient within a few fp32
 * roundings.  One or both of y_bf16 and y_q are given.
 *   x_bf16 [rows][ldx], residual_bf16 [rows][ldr] or NULL, weight [cols] bf16
 *   (w_dtype 0) or fp32 (1), 16-byte aligned, eps finite and >= 0, h_bf16
 *   [rows][ldh] with a residual (else NULL; Q4_ERR_FORMAT for one without the
 *   other), y_bf16 [rows][ldy].  cols % 8 == 0 (y_q: % 16, tiled % 512),
 *   cols <= 32768, rows < 2^22.  h may be x or the residual itself (same
 *   pointer and leading dimension).  Other overlaps are not allowed.
 * A row with an infinity or a NaN, or whose sum of squares reaches 2^128, gives
 * NaN throughout (in 8 bits: the scale NaN, codes without meaning), and so does a
 * row of zeros with eps = 0.  Other rows are not touched by it.  Small rows are what
 * the formula says down to bf16's least number, also where their squares are below
 * fp32's range (eps = 0, or as small).  Weights are meant to be below 2^64: h * weight
 * is a product in fp32, for such rows of 2^80 h.
 */
q4_status q4_rmsnorm(const void* x_bf16, int64_t ldx, const void* residual_bf16, int64_t ldr, const void* weight,
                     int w_dtype, float eps, int64_t rows, int64_t cols, void* h_bf16, int64_t ldh, void* y_bf16,
                     int64_t ldy, const q4_tensor* y_q, void* stream);

/*
 * Its gradient, from h as the forward call wrote it (or x without a residual);
 * an 8-bit output's is that of y (straight through).  With
 * r = 1 / sqrt(mean_k(h^2) + eps), n = h * r, g = dy * weight:
 *     dx         = bf16(dh + r * (g - n * mean_k(g * n)))
 *     dweight[k] (+)= sum over rows of dy * n                          (fp32)
 * dx is the gradient of x and of the residual alike; dh_bf16 [rows][lddh] is
 * the one that reaches h on its own path (NULL: none).  dweight fp32 [cols],
 * written whole, added to with accumulate != 0; NULL: not wanted.  dx may be dh
 * or dy itself (same pointer and leading dimension).  Limits as above.  Results
 * do not vary from run to run.  workspace: as for the gradient products below,
 * of the size the query gives (not read without dweight).
 */
q4_status q4_rmsnorm_backward_workspace(int64_t rows, int64_t cols, size_t* bytes);
q4_status q4_rmsnorm_backward(const void* dy_bf16, int64_t lddy, const void* h_bf16, int64_t ldh, const void* weight,
                              int w_dtype, float eps, const void* dh_bf16, int64_t lddh, int64_t rows, int64_t cols,
                              void* dx_bf16, int64_t lddx, float* dweight, int accumulate, void* workspace,
                              size_t workspace_bytes, void* stream);

/*
 * Grouped per-expert GEMM for MoE ("Low-bit inference for very large MoE",
 * "A few details": one low-bit weight matrix per expert, rows grouped by
 * routing).  W holds E experts stacked expert-major: W->rows == E*N, expert
 * e owns rows [e*N, (e+1)*N).  For every expert e and every routed row p in
 * [expert_offsets[e], expert_offsets[e+1]):
 *     C[p][n] = sum_k A[gather[p]][k] * w'[e*N + n][k]
 * A_bf16 [T][lda] (T tokens), gather int32 [P] (device; NULL means the
 * identity, row p reads A[p], and needs T >= P), expert_offsets
 * int32 [E+1] (device, non-decreasing, offsets[0] = 0, offsets[E] = P),
 * C_bf16 [P][ldc].  The kernels read the offsets on the device (no host
 * sync) and clamp every range to [0, P]; a row whose gather index is outside
 * [0, T) is written as zeros.  K = W->cols must be a multiple of 128.
 */
q4_status q4_grouped_gemm(const void* A_bf16, int64_t lda, int64_t T, const int32_t* gather,
                          const int32_t* expert_offsets, int32_t E, int64_t P,
                          const q4_tensor* W, int64_t N, void* C_bf16, int64_t ldc,
                          void* stream);

/*
 * The steps of an MoE layer around q4_grouped_gemm ("Low-bit inference for
 * very large MoE", "A few details": one low-bit matrix per expert, tokens
 * grouped by routing).  A layer is
 *   q4_moe_route -> q4_grouped_gemm (gate/up: W rows [e*2I, (e+1)*2I) =
 *   [W_gate_e; W_up_e]) -> q4_swiglu -> q4_grouped_gemm (down: gather =
 *   0..P-1, W rows [e*K, (e+1)*K)) -> q4_moe_combine.
 */

/*
 * The gate/up expert GEMM with the SwiGLU activation fused into its
 * epilogue: for expert e and routed row p,
 *     H[p][n] = bf16(silu(sum_k a[k] w_gate_e[n][k]) * sum_k a[k] w_up_e[n][k])
 * with a = A[gather[p]] as in q4_grouped_gemm (NULL gather = identity).
 * W (tiled layout only, else Q4_ERR_FORMAT) holds 2I rows per expert that
 * alternate 16-row tiles of W_gate and W_up: rows e*2I + 32j + r are gate
 * row 16j + r and rows e*2I + 32j + 16 + r are up row 16j + r (r < 16);
 * I % 16 == 0.  H_bf16 [P][ldh].  Replaces q4_grouped_gemm + q4_swiglu
 * without writing the gate/up products.
 */
q4_status q4_grouped_gemm_swiglu(const void* A_bf16, int64_t lda, int64_t T, const int32_t* gather,
                                 const int32_t* expert_offsets, int32_t E, int64_t P,
                                 const q4_tensor* W, int64_t I, void* H_bf16, int64_t ldh,
                                 void* stream);

/*
 * Routing of T tokens over E experts from fp32 router logits [T][ld].
 * Token t's experts are its k largest logits, largest first, ties to the
 * lower expert id: topk_ids [T][k]; its gate for each is that expert's
 * softmax probability over all E logits (fp32, not renormalized):
 * topk_weights [T][k].  Routed rows are ordered expert-major and, within an
 * expert, by token: expert_offsets [E+1], gather [T*k] (token of each row)
 * and inv [T][k] (row of each choice).  All int32/fp32 device arrays, 4-byte
 * aligned.  1 <= E <= 1024, 1 <= k <= min(E, 32), and the dispatch runs in
 * one workgroup whose LDS holds a token bitmap per expert:
 * 8*E*(ceil(T/32) + 1) bytes <= 160 KB (E = 64: T <= 10208), else
 * Q4_ERR_SHAPE.  T == 0 writes expert_offsets = 0.  Logits compare as
 * values (-0 equal to +0); a NaN logit, outside the finite-input contract,
 * ranks above +inf (sign bit clear) or below -inf (set), so every token
 * still gets k distinct experts and every output index stays in range.
 */
q4_status q4_moe_route(const float* logits, int64_t ld, int64_t T, int32_t E, int32_t k,
                       int32_t* topk_ids, float* topk_weights, int32_t* expert_offsets,
                       int32_t* gather, int32_t* inv, void* stream);

/*
 * SwiGLU between the expert GEMMs: h[p][n] = bf16(silu(g) * u), g =
 * gu[p][n], u = gu[p][I + n], silu(z) = z / (1 + exp(-z)), fp32 math.
 * gu_bf16 [P][ld_gu] (ld_gu >= 2I), h_bf16 [P][ldh]; I % 8 == 0.
 */
q4_status q4_swiglu(const void* gu_bf16, int64_t ld_gu, int64_t P, int64_t I, void* h_bf16,
                    int64_t ldh, void* stream);

/*
 * Gated combine: out[t][n] = bf16(sum_j weights[t][j] * y[inv[t][j]][n]),
 * fp32 accumulation in choice order.  y_bf16 [P][ldy] (expert outputs in
 * routed-row order), inv/weights [T][k] as q4_moe_route or q4_moe_sort write
 * them (a choice with inv < 0 was dropped and adds nothing), out_bf16
 * [T][ldo]; N % 8 == 0.
 */
q4_status q4_moe_combine(const void* y_bf16, int64_t ldy, const int32_t* inv, const float* weights,
                         int64_t T, int32_t k, int64_t N, void* out_bf16, int64_t ldo, void* stream);

/*
 * The backward pass of the products and of the MoE layer on 4-bit weights:
 * gradients for activations through frozen weights, gradients for the
 * full-precision weights that a quantization-aware run trains ("Low-bit
 * inference for very large MoE", "Why quantization-aware training": the
 * straight-through gradient of a fake-quantized weight is that of the weight),
 * activations saved in 8 bits in between, and tokens sorted by expert and back.
 * A training step of one layer is
 *   q4_moe_topk -> q4_moe_sort -> q4_grouped_gemm (gate/up) ->
 *   q4_swiglu_save -> q4_grouped_gemm (down) -> q4_moe_combine
 * and backwards
 *   q4_moe_combine_backward -> q4_grouped_gemm_dgrad (down) ->
 *   q4_swiglu_backward -> q4_grouped_gemm_dgrad (gate/up) ->
 *   q4_moe_permute_backward, with q4_grouped_gemm_wgrad for the weights and
 *   q4_moe_topk_backward for the router.
 *
 * Results do not vary from run to run: sums are in fp32 in an order that the
 * sizes alone decide, with no floating-point atomics.  Workspaces are the
 * caller's, 16-byte aligned, of at least the size the matching *_workspace
 * call gives (host arithmetic only; 0 for many sizes, then NULL may be passed),
 * without contents to keep; two calls that may run at once (two streams, two
 * captured graphs) need one each.  The per-token calls need T < 2^23 and
 * T * ceil(columns/1024) < 2^25; the products N, K and the leading dimensions
 * of dC and A up to 2^21, summed rows up to 2^30, and at most 2^22 blocks of
 * 64 x 256 outputs (else Q4_ERR_SHAPE).
 */

/*
 * The first half of q4_moe_route, for any number of tokens: the k largest
 * logits' ids and softmax gates.  T <= 2^26 - 4, here and in its gradient.
 */
q4_status q4_moe_topk(const float* logits, int64_t ld, int64_t T, int32_t E, int32_t k,
                      int32_t* topk_ids, float* topk_weights, void* stream);

/*
 * Gradient of the softmax gates for the router logits: with p = softmax of
 * token t's logits and d[e] the sum of dweights[t][j] over the choices j with
 * topk_ids[t][j] == e (ids outside 0 .. E-1 take no part),
 *     dlogits[t][e] = p[e] * (d[e] - sum_e' p[e'] d[e']).
 * A token whose logits are all -inf gets 0, one with a NaN among them NaN
 * throughout.  logits [T][ld], dlogits
 * [T][lddl] fp32; topk_ids, dweights [T][k].  E <= 1024, 1 <= k <= 32.
 */
q4_status q4_moe_topk_backward(const float* logits, int64_t ld, int64_t T, int32_t E, int32_t k,
                               const int32_t* topk_ids, const float* dweights, float* dlogits,
                               int64_t lddl, void* stream);

/*
 * Balance of a router: the loss that grows where experts that receive many
 * choices also have large probabilities, and the choices per expert.  Over the n
 * tokens that count (mask[t] != 0, all with mask NULL), c[e] of whose choices are
 * e and whose softmax probabilities of e add up to P[e]:
 *     counts[e] = c[e]                                             (int32)
 *     slopes[e] = coef * E * c[e] / (k * n^2)                      (fp32)
 *     loss      = sum_e slopes[e] * P[e]                           (fp32 [1])
 * so loss = coef for choices and probabilities spread evenly, and 0 (slopes too)
 * with n = 0.  Choices with ids outside 0 .. E-1 are in no c[e].  Probabilities
 * are fp32 (0 below 2^-126 of the token's largest), their sums over tokens in 64
 * bits, in an order that the sizes alone decide.
 * Backward (the counts have no gradient), with p the softmax of token t:
 *     dlogits[t][e] (+)= dloss * p[e] * (slopes[e] - sum_e' p[e'] slopes[e'])
 * 0 for tokens that do not count; dloss fp32 [1] on the device, NULL: 1;
 * accumulate != 0 adds, e.g. to what q4_moe_topk_backward wrote.
 * A token whose logits are all -inf has no probabilities: it adds nothing to P
 * and its gradient is 0; one with a NaN or +inf makes the loss NaN and its own
 * gradient alone NaN.
 * logits [T][ld], dlogits [T][lddl] fp32, ids [T][k] int32, mask uint8 [T].
 * 1 <= E <= 1024, 1 <= k <= 32, T <= 2^26 - 4, leading dimensions <= 2^27.
 */
q4_status q4_moe_balance_workspace(int64_t T, int32_t E, size_t* bytes);
q4_status q4_moe_balance(const float* logits, int64_t ld, int64_t T, int32_t E, int32_t k, const int32_t* topk_ids,
                         const uint8_t* mask, float coef, float* loss, int32_t* counts, float* slopes,
                         void* workspace, size_t workspace_bytes, void* stream);
q4_status q4_moe_balance_backward(const float* logits, int64_t ld, int64_t T, int32_t E, const uint8_t* mask,
                                  const float* slopes, const float* dloss, float* dlogits, int64_t lddl,
                                  int accumulate, void* stream);

/*
 * Tokens sorted by expert, for choices from any router and any number of
 * tokens: a stable sort of topk_ids [T][k] (read as T*k choices in order) by
 * expert.  Writes expert_offsets [E+1], gather (the token of each row) and inv
 * [T][k] (the row of each choice), as q4_moe_route does for its own ids.  A
 * choice with an id outside 0 .. E-1 is dropped (an expert of another rank, one
 * over capacity): its inv is -1, it has no row, and gather's entries from
 * expert_offsets[E] on are left as they were.  The same expert twice in a token
 * gives two rows.  gather holds T*k entries.  1 <= E <= 1024, 1 <= k <= 32,
 * T*k < 2^31.
 */
q4_status q4_moe_sort_workspace(int64_t T, int32_t k, int32_t E, size_t* bytes);
q4_status q4_moe_sort(const int32_t* topk_ids, int64_t T, int32_t k, int32_t E,
                      int32_t* expert_offsets, int32_t* gather, int32_t* inv, void* workspace,
                      size_t workspace_bytes, void* stream);

/*
 * The tokens' rows in expert order: xs[inv[t][j]] = x[t] for every choice with
 * 0 <= inv[t][j] < P; other rows of xs are left as they were.  x_bf16 [T][ldx],
 * xs_bf16 [P][ldxs], K % 8 == 0; no row may be named by two choices.  (The
 * grouped products read tokens through gather by themselves; the copy is for
 * sending rows to other ranks and for operators that want them in order.)
 * Backward: dx[t] = bf16(sum_j dxs[inv[t][j]]), fp32 in choice order, 0 for a
 * token without rows.
 */
q4_status q4_moe_permute(const void* x_bf16, int64_t ldx, const int32_t* inv, int64_t T, int32_t k,
                         int64_t K, int64_t P, void* xs_bf16, int64_t ldxs, void* stream);
q4_status q4_moe_permute_backward(const void* dxs_bf16, int64_t lddxs, const int32_t* inv, int64_t T,
                                  int32_t k, int64_t K, int64_t P, void* dx_bf16, int64_t lddx,
                                  void* stream);

/*
 * Gradients of q4_moe_combine: for every choice with 0 <= inv[t][j] < P
 *     dy[inv[t][j]] = bf16(weights[t][j] * dout[t])
 *     dweights[t][j] = sum_n dout[t][n] * y[inv[t][j]][n]      (fp32)
 * and dweights[t][j] = 0 for the others; rows of dy that no choice names are
 * left as they were.  dout_bf16 [T][ldo], y_bf16 [P][ldy], dy_bf16 [P][lddy],
 * N % 8 == 0.  dweights may be NULL (gates without gradient); y is then not
 * read and may be NULL too.
 */
q4_status q4_moe_combine_backward(const void* dout_bf16, int64_t ldo, const void* y_bf16, int64_t ldy,
                                  const int32_t* inv, const float* weights, int64_t T, int32_t k,
                                  int64_t N, int64_t P, void* dy_bf16, int64_t lddy, float* dweights,
                                  void* stream);

/*
 * q4_swiglu that also saves its input in 8 bits for the backward pass, in the
 * same pass over it: h as in q4_swiglu (exp and reciprocal in hardware
 * precision: h may differ from q4_swiglu's in the last bf16 place) and gu_q
 * (Q4_MXINT8 or Q4_MXFP8, [P][2I]) exactly what q4_quantize writes for gu.
 * I % 32 == 0.
 * Backward, with g, u the values gu_q stands for (or gu itself in bf16; exactly
 * one of gu_bf16 / gu_q is given) and s = 1 / (1 + exp(-g)):
 *     dgu[p][n]     = bf16(dh * u * s * (1 + g * (1 - s)))
 *     dgu[p][I + n] = bf16(dh * g * s)
 * and, if h_bf16 is not NULL, h = bf16(g * s * u) again (the down projection's
 * input, so that it need not be kept).  I % 32 == 0 (8 with gu_bf16).
 */
q4_status q4_swiglu_save(const void* gu_bf16, int64_t ld_gu, int64_t P, int64_t I, void* h_bf16,
                         int64_t ldh, const q4_tensor* gu_q, void* stream);
q4_status q4_swiglu_backward(const void* gu_bf16, int64_t ld_gu, const q4_tensor* gu_q,
                             const void* dh_bf16, int64_t lddh, int64_t P, int64_t I, void* dgu_bf16,
                             int64_t lddgu, void* h_bf16, int64_t ldh, void* stream);

/*
 * Gradient of the W4 products for their activations:
 *     dA[p][k] = sum_n dC[p][n] * w'[e*N + n][k]
 * over the rows p of expert e (q4_gemm_dgrad: one dense weight, all rows).
 * bf16 matrix cores, fp32 sums, bf16 output.  W: any weight format, either
 * layout, as the forward call takes it; INT4 weights (with or without a zero
 * point) are rounded to bf16 as in q4_gemm from bf16 and q4_grouped_gemm, MXFP4
 * and NVFP4 enter exactly.  dC_bf16 [P][lddc], dA_bf16 [P][ldda]; N % 8 == 0 (16 for the
 * grouped call in the tiled layout), K % 128 == 0.  expert_offsets as in
 * q4_grouped_gemm; rows of dA outside every expert's range are left as they
 * were.  N == 0 writes zeros.
 */
q4_status q4_dgrad_workspace(int64_t P, int32_t E, int64_t N, int64_t K, size_t* bytes);
q4_status q4_gemm_dgrad(int64_t M, const void* dC_bf16, int64_t lddc, const q4_tensor* W,
                        void* dA_bf16, int64_t ldda, void* workspace, size_t workspace_bytes,
                        void* stream);
q4_status q4_grouped_gemm_dgrad(const void* dC_bf16, int64_t lddc, const int32_t* expert_offsets,
                                int32_t E, int64_t P, const q4_tensor* W, int64_t N, void* dA_bf16,
                                int64_t ldda, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Gradient of the products for the weight, from activations kept in bf16
 * (A_bf16) or in 8 bits (A_q, Q4_MXINT8 or Q4_MXFP8; exactly one is given):
 *     dW[e*N + n][k] (+)= sum over expert e's rows p of dC[p][n] * a[gather[p]][k]
 * (q4_gemm_wgrad: one dense weight, all M rows, row p reads a[p]).  The 8-bit
 * values enter the bf16 matrix cores exactly; fp32 sums.  dC_bf16 [P][lddc],
 * A [T][lda] (gather NULL: row p reads a[p], T >= P; an index outside [0, T)
 * reads zeros), dW [E*N][lddw] bf16 (dw_dtype 0) or fp32 (1), written whole:
 * an expert without rows gets zeros.  accumulate != 0 (fp32 only, else
 * Q4_ERR_FORMAT) adds to what dW holds.  N % 8 == 0, K % 8 == 0 (32 with A_q);
 * dW 16-byte aligned, lddw a multiple of 8 (4 for fp32).
 */
q4_status q4_wgrad_workspace(int64_t P, int32_t E, int64_t N, int64_t K, size_t* bytes);
q4_status q4_gemm_wgrad(int64_t M, const void* dC_bf16, int64_t lddc, const void* A_bf16, int64_t lda,
                        const q4_tensor* A_q, int64_t N, int64_t K, void* dW, int dw_dtype,
                        int64_t lddw, int accumulate, void* workspace, size_t workspace_bytes,
                        void* stream);
q4_status q4_grouped_gemm_wgrad(const void* dC_bf16, int64_t lddc, const void* A_bf16, int64_t lda,
                                const q4_tensor* A_q, int64_t T, const int32_t* gather,
                                const int32_t* expert_offsets, int32_t E, int64_t P, int64_t N,
                                int64_t K, void* dW, int dw_dtype, int64_t lddw, int accumulate,
                                void* workspace, size_t workspace_bytes, void* stream);

/*
 * The norm over all gradients of a step, and the gradients scaled down to a
 * largest norm:
 *     norm = sqrt(sum over all tensors of g^2)
 *     out  = g * min(1, max_norm / (norm + 1e-6))
 * grads, counts and dtypes are host arrays of n entries, read during the call:
 * device pointers to counts[i] contiguous values, bf16 (dtypes[i] 0) or fp32 (1),
 * aligned to their own size; empty tensors are allowed (and may be NULL), n <=
 * 2^20.  norm: device fp32 [1].  The squares are added in 64 bits, in an order
 * that sizes and alignment alone decide; a norm past fp32's range is inf in norm
 * and as it is for the factor.  A NaN or an infinity among the gradients makes
 * norm NaN or inf, as arithmetic has it: every output is then NaN, or 0 where g
 * is finite and the norm inf.  The factor and the product are made in 64 bits,
 * and the product rounded to fp32 and, for bf16, from there.
 * q4_grad_clip takes the norm from norm_in (e.g. one combined over ranks), or
 * with norm_in NULL makes it in the same call and writes it to norm_out (which
 * may be NULL; not written with norm_in).  out: host array of n pointers of the
 * same counts and types, or NULL: in place (nothing is written where the factor
 * is 1).  An out[i] may be grads[i] itself; otherwise outputs must overlap
 * neither each other nor any gradient (Q4_ERR_ALIGN: also a tensor that is
 * listed twice), and no output a norm, which workgroups read while others write
 * (nor norm_out a gradient).  max_norm >= 0, inf for no limit.
 * workspace: 16-byte aligned, of the size the query gives (not read with
 * norm_in); the contents need not be kept.
 */
q4_status q4_grad_workspace(int64_t n, size_t* bytes);
q4_status q4_grad_norm(int64_t n, const void* const* grads, const int64_t* counts, const int32_t* dtypes,
                       float* norm, void* workspace, size_t workspace_bytes, void* stream);
q4_status q4_grad_clip(int64_t n, const void* const* grads, const int64_t* counts, const int32_t* dtypes,
                       void* const* out, const float* norm_in, float max_norm, float* norm_out, void* workspace,
                       size_t workspace_bytes, void* stream);

/*
 * Which kernel the products take for these sizes (host arithmetic only; the
 * sizes as in the matching *_workspace call): the rows of a block of outputs
 * that a workgroup makes, 64, 128 or 256 by 256 columns, and the parts that
 * its sum is split into; 0 and 0 where nothing is launched.  For tests and
 * measurements that have to reach a certain block.  a_is_bf16: dW from A_bf16.
 */
q4_status q4_dgrad_plan(int64_t P, int32_t E, int64_t N, int64_t K, int32_t* block_rows, int32_t* parts);
q4_status q4_wgrad_plan(int64_t P, int32_t E, int64_t N, int64_t K, int a_is_bf16, int32_t* block_rows,
                        int32_t* parts);

/*
 * The same of the W8A8 product: the block of C that a workgroup makes and how many
 * workgroups there are (0, 0 and 0 where nothing is launched).  Up to 256 of them
 * take a variant of their kind with more on the way.
 */
q4_status q4_w8a8_plan(int64_t M, int64_t N, int64_t K, int32_t* block_rows, int32_t* block_cols,
                       int64_t* workgroups);

/*
 * Measurement helper, not a step of the method: reads `bytes` of device
 * memory at src with a plain streaming kernel (16-byte non-temporal loads,
 * each wave 8 KB in flight) and discards the data.  Decode GEMVs are bound
 * by their weight reads ("Low-bit inference for very large MoE", table
 * "Kernels on different hardware", row W4A16), so timing this read on a
 * buffer of the weight's size gives the rate the GEMV can approach on this
 * part.  src 16-byte aligned, bytes a multiple of 1024 (else Q4_ERR_ALIGN /
 * Q4_ERR_SHAPE); sink: device uint32[1], written only if the folded data
 * equals one fixed 32-bit constant (which keeps the loads alive).
 * bytes == 0 is a no-op.
 */
q4_status q4_read_probe(const void* src, int64_t bytes, uint32_t* sink, void* stream);

/*
 * Measurement helper, not a step of the method: the rate at which this part
 * sustains one kind of matrix instruction, back to back, with operands in
 * registers -- the ceiling a GEMM built on that instruction can approach.
 * The operands are pseudo-random bits drawn from `seed` (as quantized data
 * is): with random operands the part lowers its clock to stay within its
 * power limit, so this rate lies below the published dense peak.
 *   kind   Q4_PROBE_FP4  scaled 16x16x128 with E2M1 operands (the W4A4
 *                        MXFP4 GEMM's instruction)
 *          Q4_PROBE_BF16 16x16x32 bf16 (GEMV, W4A16 GEMM, grouped GEMM)
 *          Q4_PROBE_F16  16x16x32 fp16 (the NVFP4 W4A4 GEMM)
 *          Q4_PROBE_FP8  scaled 16x16x128 with E4M3 operands (W4A8)
 *          Q4_PROBE_FP4_COPY  the FP4 instruction with one direct
 *                        global->LDS copy (1 KB per wave) issued per 8
 *                        instructions: the copy rate per SIMD of the tiled
 *                        W4A4 kernel
 *          Q4_PROBE_FP4_MIX   the same plus three 16-byte-per-lane LDS
 *                        fragment reads per 8 instructions: that kernel's
 *                        whole memory-instruction mix, so the rate its loop
 *                        can approach on this part
 *          Q4_PROBE_BF16_MIX  the bf16 instruction with the tiled W4A16
 *                        GEMM's mix on NVFP4 weights: per 16 instructions
 *                        one weight fragment dequantized (their row
 *                        operand), one copy and eight fragment reads
 *          other values: Q4_ERR_FORMAT
 *   iters  iterations of 8 instructions per wave, 0 .. 2^24 (else
 *          Q4_ERR_SHAPE); the launch runs two waves per SIMD on every
 *          compute unit; iters == 0 is a no-op (*flops = 0)
 *   sink   device uint32[1] (the three mix kinds: 16384 uint32, 16-byte
 *          aligned, else Q4_ERR_ALIGN -- the 64 KB the copies read; their
 *          contents do not matter), written only if the folded sums equal
 *          one fixed constant (which keeps the products alive)
 *   flops  host double: receives the floating-point operations the launch
 *          performs (2*16*16*K per instruction); NULL: Q4_ERR_NULL
 */
typedef enum q4_probe_kind {
    Q4_PROBE_FP4 = 0,
    Q4_PROBE_BF16 = 1,
    Q4_PROBE_F16 = 2,
    Q4_PROBE_FP8 = 3,
    Q4_PROBE_FP4_COPY = 4,
    Q4_PROBE_FP4_MIX = 5,
    Q4_PROBE_BF16_MIX = 6
} q4_probe_kind;

q4_status q4_mfma_probe(int32_t kind, int64_t iters, uint32_t seed, uint32_t* sink, double* flops,
                        void* stream);

#ifdef __cplusplus
}
#endif

#endif /* Q4_H */
