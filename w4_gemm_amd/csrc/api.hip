// api.hip -- the C ABI of libq4.so (declared in include/q4.h): argument
// validation on the host, then one launcher per call.  No call allocates,
// frees or synchronizes; every error is returned before any HIP call.
#include "../../include/q4.h"

#include <hip/hip_runtime.h>

#include "q4_launch.h"

namespace {

thread_local int g_last_hip_error = 0;

constexpr int64_t kMaxDim = (int64_t)1 << 31;  // kernels index rows/cols in int
constexpr int64_t kMaxGradLd = (int64_t)1 << 21;      // the gradient products address 256 rows in 2^30 bytes
constexpr int64_t kMaxTopkTokens = ((int64_t)1 << 26) - 4;  // a wave per token, four a workgroup: below 2^32 threads

int block_of(int fmt) {
  switch (fmt) {
    case Q4_INT4_G128: return 128;
    case Q4_MXFP4: return 32;
    case Q4_NVFP4: return 16;
    case Q4_FP8_ROW: return 16;  // row-major rows are stored in 16-byte pieces
    case Q4_INT4_ZP_G128: return 128;
    case Q4_MXFP8:
    case Q4_MXINT8: return 32;
    default: return 0;
  }
}

// The saved-activation formats: row-major only, no operand of a W4 product.
bool is_mx8(int fmt) { return fmt == Q4_MXFP8 || fmt == Q4_MXINT8; }
bool is_weight(int fmt) { return fmt != Q4_FP8_ROW && !is_mx8(fmt); }

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

q4_status hip_status(hipError_t e) {
  if (e == hipSuccess) return Q4_OK;
  g_last_hip_error = (int)e;
  return Q4_ERR_HIP;
}

// Validates a quantized tensor descriptor: known format and layout, sizes
// in range and multiples of the block (of 512 in the tiled layout), buffers
// present and aligned when the tensor is not empty.
q4_status check_tensor(const q4_tensor* t) {
  if (!t) return Q4_ERR_NULL;
  const int g = block_of(t->fmt);
  if (!g || (t->layout != Q4_LAYOUT_ROWS && t->layout != Q4_LAYOUT_TILED)) return Q4_ERR_FORMAT;
  if (is_mx8(t->fmt) && t->layout != Q4_LAYOUT_ROWS) return Q4_ERR_FORMAT;
  if (t->rows < 0 || t->cols < 0 || t->rows >= kMaxDim || t->cols >= kMaxDim) return Q4_ERR_SHAPE;
  if (t->cols % (t->layout == Q4_LAYOUT_TILED ? 512 : g)) return Q4_ERR_SHAPE;
  if (t->fmt == Q4_NVFP4) {
    if (!t->global_scale) return Q4_ERR_NULL;
    if (!aligned(t->global_scale, 4)) return Q4_ERR_ALIGN;
  } else if (t->global_scale) {
    return Q4_ERR_FORMAT;
  }
  if (t->rows > 0 && t->cols > 0) {
    if (!t->codes || !t->scales) return Q4_ERR_NULL;
    if (!aligned(t->codes, 16) || !aligned(t->scales, 4)) return Q4_ERR_ALIGN;
  }
  return Q4_OK;
}

// A bf16 matrix argument: rows x cols with leading dimension ld.
q4_status check_bf16(const void* p, int64_t rows, int64_t cols, int64_t ld) {
  if (rows < 0 || cols < 0) return Q4_ERR_SHAPE;
  if (rows == 0 || cols == 0) return Q4_OK;
  if (!p) return Q4_ERR_NULL;
  if (ld < cols) return Q4_ERR_SHAPE;
  if (!aligned(p, 16) || ld % 8) return Q4_ERR_ALIGN;
  return Q4_OK;
}

// An output bf16 matrix written element by element (2-byte alignment).
q4_status check_out_bf16(const void* p, int64_t rows, int64_t cols, int64_t ld) {
  if (rows < 0 || cols < 0) return Q4_ERR_SHAPE;
  if (rows == 0 || cols == 0) return Q4_OK;
  if (!p) return Q4_ERR_NULL;
  if (ld < cols) return Q4_ERR_SHAPE;
  if (!aligned(p, 2)) return Q4_ERR_ALIGN;
  return Q4_OK;
}

// Token counts of the per-token kernels: a workgroup of up to 512 threads per
// token, or one of 128 per token and 1024 columns, within 2^32 threads.
q4_status check_tokens(int64_t T, int32_t k, int64_t cols) {
  if (T < 0 || cols < 0 || T >= ((int64_t)1 << 23) || cols >= kMaxDim || k < 1 || k > 32) return Q4_ERR_SHAPE;
  if (T * ((cols + 1023) / 1024) >= ((int64_t)1 << 25)) return Q4_ERR_SHAPE;
  return cols % 8 ? Q4_ERR_SHAPE : Q4_OK;
}

// The arguments q4_gemm_dgrad and q4_grouped_gemm_dgrad share.
q4_status dgrad(const void* dC, int64_t lddc, const int32_t* offsets, int32_t E, int64_t P, const q4_tensor* W,
                int64_t N, void* dA, int64_t ldda, void* workspace, size_t workspace_bytes, void* stream);
q4_status wgrad(const void* dC, int64_t lddc, const void* A_bf16, int64_t lda, const q4_tensor* A_q, int64_t T,
                const int32_t* gather, const int32_t* offsets, int32_t E, int64_t P, int64_t N, int64_t K, void* dW,
                int dw_dtype, int64_t lddw, int accumulate, void* workspace, size_t workspace_bytes, void* stream);

hipStream_t as_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }

}  // namespace

extern "C" {

int q4_version(void) { return 104; }

const char* q4_status_string(int status) {
  switch (status) {
    case Q4_OK: return "ok";
    case Q4_ERR_NULL: return "a required pointer is NULL";
    case Q4_ERR_SHAPE: return "invalid size (negative, too large or not a multiple of the block)";
    case Q4_ERR_ALIGN: return "misaligned pointer or leading dimension";
    case Q4_ERR_FORMAT: return "unknown or unsupported format for this call";
    case Q4_ERR_HIP: return "HIP launch failed (see q4_last_hip_error)";
    default: return "unknown status";
  }
}

int q4_last_hip_error(void) { return g_last_hip_error; }

q4_status q4_sizes(int fmt, int layout, int64_t rows, int64_t cols, size_t* codes_bytes,
                   size_t* scales_bytes) {
  const int g = block_of(fmt);
  if (!g || (layout != Q4_LAYOUT_ROWS && layout != Q4_LAYOUT_TILED)) return Q4_ERR_FORMAT;
  if (is_mx8(fmt) && layout != Q4_LAYOUT_ROWS) return Q4_ERR_FORMAT;
  if (rows < 0 || cols < 0 || rows >= kMaxDim || cols >= kMaxDim) return Q4_ERR_SHAPE;
  if (cols % (layout == Q4_LAYOUT_TILED ? 512 : g)) return Q4_ERR_SHAPE;
  // the tiled layout stores whole 16-row tiles; per stored row both layouts
  // hold cols/2 code bytes and cols/g scales (fp16 for INT4)
  const size_t srows = layout == Q4_LAYOUT_TILED ? (size_t)((rows + 15) / 16) * 16 : (size_t)rows;
  if (fmt == Q4_FP8_ROW) {  // one byte per value, one fp32 scale per row
    if (codes_bytes) *codes_bytes = srows * (size_t)cols;
    if (scales_bytes) *scales_bytes = (size_t)rows * 4;
    return Q4_OK;
  }
  if (is_mx8(fmt)) {  // one byte per value, one scale byte per 32
    if (codes_bytes) *codes_bytes = srows * (size_t)cols;
    if (scales_bytes) *scales_bytes = srows * (size_t)(cols / g);
    return Q4_OK;
  }
  if (codes_bytes) *codes_bytes = srows * (size_t)cols / 2;
  if (scales_bytes)
    *scales_bytes = srows * (size_t)(cols / g) * (fmt == Q4_INT4_G128 ? 2 : fmt == Q4_INT4_ZP_G128 ? 4 : 1);
  return Q4_OK;
}

q4_status q4_quantize(const void* src_bf16, int64_t ld, const q4_tensor* dst,
                      const float* nv_global_in, void* stream) {
  q4_status st = check_tensor(dst);
  if (st != Q4_OK) return st;
  if (nv_global_in && dst->fmt != Q4_NVFP4) return Q4_ERR_FORMAT;
  if (nv_global_in && !aligned(nv_global_in, 4)) return Q4_ERR_ALIGN;
  st = check_bf16(src_bf16, dst->rows, dst->cols, ld);
  if (st != Q4_OK) return st;
  if (dst->fmt != Q4_NVFP4 && (dst->rows == 0 || dst->cols == 0)) return Q4_OK;
  if (dst->fmt == Q4_FP8_ROW)
    return hip_status(q4::launch_fp8_rows_quantize(dst->layout, static_cast<const uint16_t*>(src_bf16), ld,
                                                   dst->rows, dst->cols, static_cast<uint8_t*>(dst->codes),
                                                   static_cast<float*>(dst->scales), as_stream(stream)));
  if (is_mx8(dst->fmt))
    return hip_status(q4::launch_mx8_quantize(dst->fmt, static_cast<const uint16_t*>(src_bf16), ld, dst->rows,
                                              dst->cols, static_cast<uint8_t*>(dst->codes),
                                              static_cast<uint8_t*>(dst->scales), as_stream(stream)));
  return hip_status(q4::launch_quantize(
      dst->fmt, dst->layout, static_cast<const uint16_t*>(src_bf16), ld, dst->rows, dst->cols,
      static_cast<uint8_t*>(dst->codes), dst->scales, dst->global_scale, nv_global_in,
      as_stream(stream)));
}

q4_status q4_dequant(const q4_tensor* src, void* dst, int dst_dtype, int64_t ld, void* stream) {
  q4_status st = check_tensor(src);
  if (st != Q4_OK) return st;
  if (dst_dtype != 0 && dst_dtype != 1) return Q4_ERR_FORMAT;
  if (src->rows == 0 || src->cols == 0) return Q4_OK;
  if (!dst) return Q4_ERR_NULL;
  if (ld < src->cols) return Q4_ERR_SHAPE;
  if (!aligned(dst, 16) || ld % (dst_dtype == 0 ? 8 : 4)) return Q4_ERR_ALIGN;
  if (src->fmt == Q4_FP8_ROW)
    return hip_status(q4::launch_fp8_rows_dequant(src->layout, static_cast<const uint8_t*>(src->codes),
                                                  static_cast<const float*>(src->scales), src->rows,
                                                  src->cols, dst, dst_dtype, ld, as_stream(stream)));
  if (is_mx8(src->fmt))
    return hip_status(q4::launch_mx8_dequant(src->fmt, static_cast<const uint8_t*>(src->codes),
                                             static_cast<const uint8_t*>(src->scales), src->rows, src->cols, dst,
                                             dst_dtype, ld, as_stream(stream)));
  return hip_status(q4::launch_dequant(src->fmt, src->layout, static_cast<const uint8_t*>(src->codes),
                                       src->scales, src->global_scale, src->rows, src->cols, dst,
                                       dst_dtype, ld, as_stream(stream)));
}

q4_status q4_relayout(const q4_tensor* src, const q4_tensor* dst, void* stream) {
  q4_status st = check_tensor(src);
  if (st != Q4_OK) return st;
  st = check_tensor(dst);
  if (st != Q4_OK) return st;
  if (src->fmt != dst->fmt || !is_weight(src->fmt)) return Q4_ERR_FORMAT;
  if (src->rows != dst->rows || src->cols != dst->cols) return Q4_ERR_SHAPE;
  hipStream_t s = as_stream(stream);
  if (src->fmt == Q4_NVFP4 && (src->rows == 0 || src->cols == 0 || src->layout == dst->layout)) {
    const hipError_t e = hipMemcpyAsync(dst->global_scale, src->global_scale, 4, hipMemcpyDeviceToDevice, s);
    if (e != hipSuccess) return hip_status(e);
  }
  if (src->rows == 0 || src->cols == 0) return Q4_OK;
  if (src->layout == dst->layout) {  // same layout: a copy
    size_t cb = 0, sb = 0;
    st = q4_sizes(src->fmt, src->layout, src->rows, src->cols, &cb, &sb);
    if (st != Q4_OK) return st;
    hipError_t e = hipMemcpyAsync(dst->codes, src->codes, cb, hipMemcpyDeviceToDevice, s);
    if (e == hipSuccess) e = hipMemcpyAsync(dst->scales, src->scales, sb, hipMemcpyDeviceToDevice, s);
    return hip_status(e);
  }
  return hip_status(q4::launch_relayout(src->fmt, dst->layout, static_cast<const uint8_t*>(src->codes), src->scales,
                                        src->global_scale, static_cast<uint8_t*>(dst->codes), dst->scales,
                                        dst->global_scale, src->rows, src->cols, s));
}

q4_status q4_gemv(const q4_tensor* W, const void* x_bf16, int64_t B, int64_t ldx, void* y_bf16,
                  int64_t ldy, void* stream) {
  q4_status st = check_tensor(W);
  if (st != Q4_OK) return st;
  if (!is_weight(W->fmt)) return Q4_ERR_FORMAT;
  if (B < 0 || B > 16) return Q4_ERR_SHAPE;
  if (W->cols % 128) return Q4_ERR_SHAPE;
  if (B == 0 || W->rows == 0) return Q4_OK;
  if (W->cols == 0) return Q4_ERR_SHAPE;
  st = check_bf16(x_bf16, B, W->cols, ldx);
  if (st != Q4_OK) return st;
  st = check_out_bf16(y_bf16, B, W->rows, ldy);
  if (st != Q4_OK) return st;
  return hip_status(q4::launch_gemv(W->fmt, W->layout, static_cast<const uint8_t*>(W->codes), W->scales,
                                    W->global_scale, W->rows, W->cols,
                                    static_cast<const uint16_t*>(x_bf16), ldx, B,
                                    static_cast<uint16_t*>(y_bf16), ldy, as_stream(stream)));
}

q4_status q4_gemm(int64_t M, const void* A_bf16, int64_t lda, const q4_tensor* A_q,
                  const q4_tensor* W, void* C_bf16, int64_t ldc, void* stream) {
  q4_status st = check_tensor(W);
  if (st != Q4_OK) return st;
  if (!is_weight(W->fmt)) return Q4_ERR_FORMAT;
  if (M < 0 || M >= kMaxDim || M > (int64_t)65535 * 64) return Q4_ERR_SHAPE;
  if ((A_bf16 == nullptr) == (A_q == nullptr)) return A_bf16 ? Q4_ERR_FORMAT : Q4_ERR_NULL;
  const int64_t N = W->rows, K = W->cols;
  if (K % 128) return Q4_ERR_SHAPE;
  if (A_q) {
    st = check_tensor(A_q);
    if (st != Q4_OK) return st;
    const bool w4a4 = A_q->fmt == W->fmt && (W->fmt == Q4_MXFP4 || W->fmt == Q4_NVFP4);
    const bool w4a8 = A_q->fmt == Q4_FP8_ROW && W->fmt == Q4_INT4_G128;
    if (!w4a4 && !w4a8) return Q4_ERR_FORMAT;
    if (A_q->rows != M || A_q->cols != K) return Q4_ERR_SHAPE;
  }
  if (M == 0 || N == 0) return Q4_OK;
  if (K == 0) return Q4_ERR_SHAPE;
  if (!A_q) {
    st = check_bf16(A_bf16, M, K, lda);
    if (st != Q4_OK) return st;
  }
  st = check_out_bf16(C_bf16, M, N, ldc);
  if (st != Q4_OK) return st;
  if (A_q && A_q->fmt == Q4_FP8_ROW)
    return hip_status(q4::launch_gemm_w4a8(
        A_q->layout, W->layout, static_cast<const uint8_t*>(A_q->codes), static_cast<const float*>(A_q->scales),
        M, static_cast<const uint8_t*>(W->codes), static_cast<const uint16_t*>(W->scales), N, K,
        static_cast<uint16_t*>(C_bf16), ldc, as_stream(stream)));
  if (A_q && A_q->fmt == Q4_NVFP4)
    return hip_status(q4::launch_gemm_w4a4_nvfp4(
        A_q->layout, W->layout, static_cast<const uint8_t*>(A_q->codes), static_cast<const uint8_t*>(A_q->scales),
        A_q->global_scale, M, static_cast<const uint8_t*>(W->codes), static_cast<const uint8_t*>(W->scales),
        W->global_scale, N, K, static_cast<uint16_t*>(C_bf16), ldc, as_stream(stream)));
  if (A_q)
    return hip_status(q4::launch_gemm_w4a4(
        A_q->layout, W->layout, static_cast<const uint8_t*>(A_q->codes), static_cast<const uint8_t*>(A_q->scales), M,
        static_cast<const uint8_t*>(W->codes), static_cast<const uint8_t*>(W->scales), N, K,
        static_cast<uint16_t*>(C_bf16), ldc, as_stream(stream)));
  return hip_status(q4::launch_gemm_w4a16(W->fmt, W->layout, static_cast<const uint8_t*>(W->codes),
                                          W->scales, W->global_scale, N, K,
                                          static_cast<const uint16_t*>(A_bf16), lda, M,
                                          static_cast<uint16_t*>(C_bf16), ldc,
                                          as_stream(stream)));
}

q4_status q4_gemm_quantized(int64_t M, const void* A_bf16, int64_t lda, const q4_tensor* A_q,
                            const q4_tensor* W, const q4_tensor* C_q, const float* nv_global_in,
                            void* stream) {
  q4_status st = check_tensor(W);
  if (st != Q4_OK) return st;
  st = check_tensor(C_q);
  if (st != Q4_OK) return st;
  if (!is_weight(W->fmt) || W->layout != Q4_LAYOUT_TILED) return Q4_ERR_FORMAT;
  if (C_q->fmt != Q4_MXFP4 && C_q->fmt != Q4_NVFP4) return Q4_ERR_FORMAT;
  if (C_q->fmt == Q4_NVFP4) {
    if (!nv_global_in) return Q4_ERR_NULL;
    if (!aligned(nv_global_in, 4)) return Q4_ERR_ALIGN;
  } else if (nv_global_in) {
    return Q4_ERR_FORMAT;
  }
  if (M < 0 || M >= kMaxDim || M > (int64_t)65535 * 64) return Q4_ERR_SHAPE;
  if ((A_bf16 == nullptr) == (A_q == nullptr)) return A_bf16 ? Q4_ERR_FORMAT : Q4_ERR_NULL;
  const int64_t N = W->rows, K = W->cols;
  if (C_q->rows != M || C_q->cols != N || N % 32) return Q4_ERR_SHAPE;
  if (A_q) {
    st = check_tensor(A_q);
    if (st != Q4_OK) return st;
    if (A_q->fmt != Q4_MXFP4 || W->fmt != Q4_MXFP4 || A_q->layout != Q4_LAYOUT_TILED) return Q4_ERR_FORMAT;
    if (A_q->rows != M || A_q->cols != K) return Q4_ERR_SHAPE;
  }
  if (M == 0 || N == 0) return Q4_OK;
  if (K == 0) return Q4_ERR_SHAPE;
  if (!A_q) {
    st = check_bf16(A_bf16, M, K, lda);
    if (st != Q4_OK) return st;
  }
  const q4::QOut qo{static_cast<uint8_t*>(C_q->codes), static_cast<uint8_t*>(C_q->scales), nv_global_in,
                    C_q->global_scale, C_q->layout == Q4_LAYOUT_TILED ? 1 : 0};
  const int out = C_q->fmt == Q4_MXFP4 ? q4::kOutMxfp4 : q4::kOutNvfp4;
  if (A_q)
    return hip_status(q4::launch_gemm_w4a4_tiled_qout(
        out, static_cast<const uint8_t*>(A_q->codes), static_cast<const uint8_t*>(A_q->scales), M,
        static_cast<const uint8_t*>(W->codes), static_cast<const uint8_t*>(W->scales), N, K, qo,
        as_stream(stream)));
  return hip_status(q4::launch_gemm_w4a16_tiled_qout(W->fmt, out, static_cast<const uint8_t*>(W->codes),
                                                     W->scales, W->global_scale, N, K,
                                                     static_cast<const uint16_t*>(A_bf16), lda, M, qo,
                                                     as_stream(stream)));
}

q4_status q4_grouped_gemm(const void* A_bf16, int64_t lda, int64_t T, const int32_t* gather,
                          const int32_t* expert_offsets, int32_t E, int64_t P,
                          const q4_tensor* W, int64_t N, void* C_bf16, int64_t ldc,
                          void* stream) {
  q4_status st = check_tensor(W);
  if (st != Q4_OK) return st;
  if (!is_weight(W->fmt)) return Q4_ERR_FORMAT;
  if (E < 0 || E > 65535 || N < 0 || T < 0 || P < 0 || P >= kMaxDim || T >= kMaxDim)
    return Q4_ERR_SHAPE;
  if (W->rows != (int64_t)E * N) return Q4_ERR_SHAPE;
  if (W->layout == Q4_LAYOUT_TILED && N % 16) return Q4_ERR_SHAPE;  // experts own whole tiles
  const int64_t K = W->cols;
  if (K % 128) return Q4_ERR_SHAPE;
  if (E == 0 || N == 0 || P == 0) return Q4_OK;
  if (K == 0) return Q4_ERR_SHAPE;
  if (!expert_offsets) return Q4_ERR_NULL;
  if (!gather && T < P) return Q4_ERR_SHAPE;  // identity gather reads rows 0..P-1 of A
  if ((gather && !aligned(gather, 4)) || !aligned(expert_offsets, 4)) return Q4_ERR_ALIGN;
  st = check_bf16(A_bf16, T, K, lda);
  if (st != Q4_OK) return st;
  st = check_out_bf16(C_bf16, P, N, ldc);
  if (st != Q4_OK) return st;
  return hip_status(q4::launch_grouped(W->fmt, W->layout, static_cast<const uint16_t*>(A_bf16), lda, T,
                                       gather, expert_offsets, E, P,
                                       static_cast<const uint8_t*>(W->codes), W->scales,
                                       W->global_scale, N, K, static_cast<uint16_t*>(C_bf16),
                                       ldc, as_stream(stream)));
}

q4_status q4_grouped_gemm_swiglu(const void* A_bf16, int64_t lda, int64_t T, const int32_t* gather,
                                 const int32_t* expert_offsets, int32_t E, int64_t P, const q4_tensor* W,
                                 int64_t I, void* H_bf16, int64_t ldh, void* stream) {
  q4_status st = check_tensor(W);
  if (st != Q4_OK) return st;
  if (!is_weight(W->fmt) || W->layout != Q4_LAYOUT_TILED) return Q4_ERR_FORMAT;
  if (E < 0 || E > 65535 || I < 0 || T < 0 || P < 0 || P >= kMaxDim || T >= kMaxDim) return Q4_ERR_SHAPE;
  if (I % 16 || W->rows != (int64_t)E * 2 * I) return Q4_ERR_SHAPE;
  const int64_t K = W->cols;
  if (E == 0 || I == 0 || P == 0) return Q4_OK;
  if (K == 0 || T == 0) return Q4_ERR_SHAPE;
  if (!expert_offsets) return Q4_ERR_NULL;
  if (!gather && T < P) return Q4_ERR_SHAPE;
  if ((gather && !aligned(gather, 4)) || !aligned(expert_offsets, 4)) return Q4_ERR_ALIGN;
  st = check_bf16(A_bf16, T, K, lda);
  if (st != Q4_OK) return st;
  st = check_bf16(H_bf16, P, I, ldh);
  if (st != Q4_OK) return st;
  return hip_status(q4::launch_grouped_tiled_swiglu(
      W->fmt, static_cast<const uint16_t*>(A_bf16), lda, T, gather, expert_offsets, E, P,
      static_cast<const uint8_t*>(W->codes), W->scales, W->global_scale, 2 * I, K, static_cast<uint16_t*>(H_bf16),
      ldh, as_stream(stream)));
}

q4_status q4_moe_route(const float* logits, int64_t ld, int64_t T, int32_t E, int32_t k, int32_t* topk_ids,
                       float* topk_weights, int32_t* expert_offsets, int32_t* gather, int32_t* inv,
                       void* stream) {
  if (T < 0 || T >= kMaxDim || E < 1 || E > 1024 || k < 1 || k > 32 || k > E) return Q4_ERR_SHAPE;
  if (q4::moe_dispatch_lds_bytes(T, E) > q4::kMoeDispatchMaxLds) return Q4_ERR_SHAPE;
  if (!expert_offsets) return Q4_ERR_NULL;
  if (!aligned(expert_offsets, 4)) return Q4_ERR_ALIGN;
  if (T > 0) {
    if (!logits || !topk_ids || !topk_weights || !gather || !inv) return Q4_ERR_NULL;
    if (ld < E) return Q4_ERR_SHAPE;
    if (!aligned(logits, 4) || !aligned(topk_ids, 4) || !aligned(topk_weights, 4) || !aligned(gather, 4) ||
        !aligned(inv, 4))
      return Q4_ERR_ALIGN;
  }
  return hip_status(q4::launch_moe_route(logits, ld, T, E, k, topk_ids, topk_weights, expert_offsets, gather,
                                         inv, as_stream(stream)));
}

q4_status q4_swiglu(const void* gu_bf16, int64_t ld_gu, int64_t P, int64_t I, void* h_bf16, int64_t ldh,
                    void* stream) {
  if (P < 0 || I < 0 || P >= kMaxDim || I >= kMaxDim) return Q4_ERR_SHAPE;
  if (I % 8) return Q4_ERR_SHAPE;
  if (P == 0 || I == 0) return Q4_OK;
  q4_status st = check_bf16(gu_bf16, P, 2 * I, ld_gu);
  if (st != Q4_OK) return st;
  st = check_bf16(h_bf16, P, I, ldh);
  if (st != Q4_OK) return st;
  return hip_status(q4::launch_swiglu(static_cast<const uint16_t*>(gu_bf16), ld_gu, P, I,
                                      static_cast<uint16_t*>(h_bf16), ldh, as_stream(stream)));
}

q4_status q4_moe_combine(const void* y_bf16, int64_t ldy, const int32_t* inv, const float* weights, int64_t T,
                         int32_t k, int64_t N, void* out_bf16, int64_t ldo, void* stream) {
  if (T < 0 || N < 0 || T >= kMaxDim || N >= kMaxDim || k < 1 || k > 32) return Q4_ERR_SHAPE;
  if (N % 8) return Q4_ERR_SHAPE;
  if (T == 0 || N == 0) return Q4_OK;
  if (!inv || !weights) return Q4_ERR_NULL;
  if (!aligned(inv, 4) || !aligned(weights, 4)) return Q4_ERR_ALIGN;
  q4_status st = check_bf16(y_bf16, 1, N, ldy);
  if (st != Q4_OK) return st;
  st = check_bf16(out_bf16, T, N, ldo);
  if (st != Q4_OK) return st;
  return hip_status(q4::launch_moe_combine(static_cast<const uint16_t*>(y_bf16), ldy, inv, weights, T, k, N,
                                           static_cast<uint16_t*>(out_bf16), ldo, as_stream(stream)));
}

q4_status q4_mfma_probe(int32_t kind, int64_t iters, uint32_t seed, uint32_t* sink, double* flops,
                        void* stream) {
  if (kind < Q4_PROBE_FP4 || kind > Q4_PROBE_BF16_MIX) return Q4_ERR_FORMAT;
  if (iters < 0 || iters > ((int64_t)1 << 24)) return Q4_ERR_SHAPE;
  if (!flops) return Q4_ERR_NULL;
  *flops = 0.0;
  if (iters == 0) return Q4_OK;
  if (!sink) return Q4_ERR_NULL;
  // the instruction-mix kinds copy 16 bytes per lane from the sink window
  if (!aligned(sink, kind >= Q4_PROBE_FP4_COPY ? 16 : 4)) return Q4_ERR_ALIGN;
  const int grid = q4::mfma_probe_grid();
  if (grid <= 0) return hip_status(hipErrorInvalidDevice);
  const double per = (kind == Q4_PROBE_BF16 || kind == Q4_PROBE_F16 || kind == Q4_PROBE_BF16_MIX)
                         ? 2.0 * 16 * 16 * 32 : 2.0 * 16 * 16 * 128;
  const q4_status st = hip_status(q4::launch_mfma_probe(kind, iters, seed, sink, grid, as_stream(stream)));
  if (st == Q4_OK) *flops = (double)grid * 4 * 8 * (double)iters * per;
  return st;
}

q4_status q4_read_probe(const void* src, int64_t bytes, uint32_t* sink, void* stream) {
  if (bytes < 0 || bytes % 1024) return Q4_ERR_SHAPE;
  if (bytes == 0) return Q4_OK;
  if (!src || !sink) return Q4_ERR_NULL;
  if (!aligned(src, 16) || !aligned(sink, 4)) return Q4_ERR_ALIGN;
  return hip_status(q4::launch_read_probe(static_cast<const uint8_t*>(src), bytes, sink, as_stream(stream)));
}

q4_status q4_moe_topk(const float* logits, int64_t ld, int64_t T, int32_t E, int32_t k, int32_t* topk_ids,
                      float* topk_weights, void* stream) {
  if (T < 0 || T > kMaxTopkTokens || E < 1 || E > 1024 || k < 1 || k > 32 || k > E) return Q4_ERR_SHAPE;
  if (T == 0) return Q4_OK;
  if (!logits || !topk_ids || !topk_weights) return Q4_ERR_NULL;
  if (ld < E) return Q4_ERR_SHAPE;
  if (!aligned(logits, 4) || !aligned(topk_ids, 4) || !aligned(topk_weights, 4)) return Q4_ERR_ALIGN;
  return hip_status(q4::launch_moe_topk(logits, ld, T, E, k, topk_ids, topk_weights, as_stream(stream)));
}

q4_status q4_moe_topk_backward(const float* logits, int64_t ld, int64_t T, int32_t E, int32_t k,
                               const int32_t* topk_ids, const float* dweights, float* dlogits, int64_t lddl,
                               void* stream) {
  if (T < 0 || T > kMaxTopkTokens || E < 1 || E > 1024 || k < 1 || k > 32) return Q4_ERR_SHAPE;
  if (T == 0) return Q4_OK;
  if (!logits || !topk_ids || !dweights || !dlogits) return Q4_ERR_NULL;
  if (ld < E || lddl < E) return Q4_ERR_SHAPE;
  if (!aligned(logits, 4) || !aligned(topk_ids, 4) || !aligned(dweights, 4) || !aligned(dlogits, 4))
    return Q4_ERR_ALIGN;
  return hip_status(q4::launch_moe_topk_backward(logits, ld, T, E, k, topk_ids, dweights, dlogits, lddl,
                                                 as_stream(stream)));
}

q4_status q4_moe_sort_workspace(int64_t T, int32_t k, int32_t E, size_t* bytes) {
  if (!bytes) return Q4_ERR_NULL;
  if (T < 0 || T >= kMaxDim || E < 1 || E > 1024 || k < 1 || k > 32 || T * k >= kMaxDim) return Q4_ERR_SHAPE;
  *bytes = q4::moe_sort_workspace(T * k, E);
  return Q4_OK;
}

q4_status q4_moe_sort(const int32_t* topk_ids, int64_t T, int32_t k, int32_t E, int32_t* expert_offsets,
                      int32_t* gather, int32_t* inv, void* workspace, size_t workspace_bytes, void* stream) {
  size_t need = 0;
  const q4_status st = q4_moe_sort_workspace(T, k, E, &need);
  if (st != Q4_OK) return st;
  if (!expert_offsets || (T > 0 && (!topk_ids || !gather || !inv)) || (need && !workspace)) return Q4_ERR_NULL;
  if (workspace_bytes < need) return Q4_ERR_SHAPE;
  if (!aligned(expert_offsets, 4) || !aligned(topk_ids, 4) || !aligned(gather, 4) || !aligned(inv, 4) ||
      (need && !aligned(workspace, 4)))
    return Q4_ERR_ALIGN;
  return hip_status(q4::launch_moe_sort(topk_ids, T, k, E, expert_offsets, gather, inv,
                                        static_cast<uint32_t*>(workspace), as_stream(stream)));
}

q4_status q4_moe_permute(const void* x_bf16, int64_t ldx, const int32_t* inv, int64_t T, int32_t k, int64_t K,
                         int64_t P, void* xs_bf16, int64_t ldxs, void* stream) {
  q4_status st = check_tokens(T, k, K);
  if (st != Q4_OK) return st;
  if (P < 0 || P >= kMaxDim) return Q4_ERR_SHAPE;
  if (T == 0 || K == 0 || P == 0) return Q4_OK;
  if (!inv) return Q4_ERR_NULL;
  if (!aligned(inv, 4)) return Q4_ERR_ALIGN;
  st = check_bf16(x_bf16, T, K, ldx);
  if (st != Q4_OK) return st;
  st = check_bf16(xs_bf16, P, K, ldxs);
  if (st != Q4_OK) return st;
  return hip_status(q4::launch_moe_permute(static_cast<const uint16_t*>(x_bf16), ldx, inv, T, k, K, P,
                                           static_cast<uint16_t*>(xs_bf16), ldxs, as_stream(stream)));
}

q4_status q4_moe_permute_backward(const void* dxs_bf16, int64_t lddxs, const int32_t* inv, int64_t T, int32_t k,
                                  int64_t K, int64_t P, void* dx_bf16, int64_t lddx, void* stream) {
  q4_status st = check_tokens(T, k, K);
  if (st != Q4_OK) return st;
  if (P < 0 || P >= kMaxDim) return Q4_ERR_SHAPE;
  if (T == 0 || K == 0) return Q4_OK;
  if (!inv) return Q4_ERR_NULL;
  if (!aligned(inv, 4)) return Q4_ERR_ALIGN;
  st = check_bf16(dxs_bf16, P, K, lddxs);
  if (st != Q4_OK) return st;
  st = check_bf16(dx_bf16, T, K, lddx);
  if (st != Q4_OK) return st;
  return hip_status(q4::launch_moe_permute_backward(static_cast<const uint16_t*>(dxs_bf16), lddxs, inv, T, k, K, P,
                                                    static_cast<uint16_t*>(dx_bf16), lddx, as_stream(stream)));
}

q4_status q4_moe_combine_backward(const void* dout_bf16, int64_t ldo, const void* y_bf16, int64_t ldy,
                                  const int32_t* inv, const float* weights, int64_t T, int32_t k, int64_t N,
                                  int64_t P, void* dy_bf16, int64_t lddy, float* dweights, void* stream) {
  q4_status st = check_tokens(T, k, N);
  if (st != Q4_OK) return st;
  if (P < 0 || P >= kMaxDim) return Q4_ERR_SHAPE;
  if (T == 0) return Q4_OK;
  if (!inv || !weights) return Q4_ERR_NULL;
  if (!aligned(inv, 4) || !aligned(weights, 4) || !aligned(dweights, 4)) return Q4_ERR_ALIGN;
  st = check_bf16(dout_bf16, T, N, ldo);
  if (st != Q4_OK) return st;
  st = check_bf16(dy_bf16, P, N, lddy);
  if (st != Q4_OK) return st;
  if (dweights) {
    st = check_bf16(y_bf16, P, N, ldy);
    if (st != Q4_OK) return st;
  }
  return hip_status(q4::launch_moe_combine_backward(static_cast<const uint16_t*>(dout_bf16), ldo,
                                                    static_cast<const uint16_t*>(y_bf16), ldy, inv, weights, T, k, N,
                                                    P, static_cast<uint16_t*>(dy_bf16), lddy, dweights,
                                                    as_stream(stream)));
}

q4_status q4_swiglu_save(const void* gu_bf16, int64_t ld_gu, int64_t P, int64_t I, void* h_bf16, int64_t ldh,
                         const q4_tensor* gu_q, void* stream) {
  q4_status st = check_tensor(gu_q);
  if (st != Q4_OK) return st;
  if (!is_mx8(gu_q->fmt)) return Q4_ERR_FORMAT;
  if (P < 0 || I < 0 || P >= kMaxDim || I >= kMaxDim / 2 || I % 32) return Q4_ERR_SHAPE;
  if (gu_q->rows != P || gu_q->cols != 2 * I) return Q4_ERR_SHAPE;
  if (P == 0 || I == 0) return Q4_OK;
  st = check_bf16(gu_bf16, P, 2 * I, ld_gu);
  if (st != Q4_OK) return st;
  st = check_bf16(h_bf16, P, I, ldh);
  if (st != Q4_OK) return st;
  return hip_status(q4::launch_swiglu_save(gu_q->fmt, static_cast<const uint16_t*>(gu_bf16), ld_gu, P, I,
                                           static_cast<uint16_t*>(h_bf16), ldh, static_cast<uint8_t*>(gu_q->codes),
                                           static_cast<uint8_t*>(gu_q->scales), as_stream(stream)));
}

q4_status q4_swiglu_backward(const void* gu_bf16, int64_t ld_gu, const q4_tensor* gu_q, const void* dh_bf16,
                             int64_t lddh, int64_t P, int64_t I, void* dgu_bf16, int64_t lddgu, void* h_bf16,
                             int64_t ldh, void* stream) {
  q4_status st;
  if ((gu_bf16 == nullptr) == (gu_q == nullptr)) return gu_bf16 ? Q4_ERR_FORMAT : Q4_ERR_NULL;
  if (P < 0 || I < 0 || P >= kMaxDim || I >= kMaxDim / 2 || I % (gu_q ? 32 : 8)) return Q4_ERR_SHAPE;
  if (gu_q) {
    st = check_tensor(gu_q);
    if (st != Q4_OK) return st;
    if (!is_mx8(gu_q->fmt)) return Q4_ERR_FORMAT;
    if (gu_q->rows != P || gu_q->cols != 2 * I) return Q4_ERR_SHAPE;
  }
  if (P == 0 || I == 0) return Q4_OK;
  if (!gu_q) {
    st = check_bf16(gu_bf16, P, 2 * I, ld_gu);
    if (st != Q4_OK) return st;
  }
  st = check_bf16(dh_bf16, P, I, lddh);
  if (st != Q4_OK) return st;
  st = check_bf16(dgu_bf16, P, 2 * I, lddgu);
  if (st != Q4_OK) return st;
  if (h_bf16) {
    st = check_bf16(h_bf16, P, I, ldh);
    if (st != Q4_OK) return st;
  }
  return hip_status(q4::launch_swiglu_backward(
      gu_q ? gu_q->fmt : 0, gu_q ? gu_q->codes : gu_bf16, gu_q ? static_cast<const uint8_t*>(gu_q->scales) : nullptr,
      ld_gu, P, I, static_cast<const uint16_t*>(dh_bf16), lddh, static_cast<uint16_t*>(dgu_bf16), lddgu,
      static_cast<uint16_t*>(h_bf16), ldh, as_stream(stream)));
}

q4_status q4_dgrad_workspace(int64_t P, int32_t E, int64_t N, int64_t K, size_t* bytes) {
  if (!bytes) return Q4_ERR_NULL;
  if (P < 0 || E < 0 || E > 65535 || N < 0 || K < 0 || P >= kMaxDim || N > kMaxGradLd || K > kMaxGradLd)
    return Q4_ERR_SHAPE;
  *bytes = P && E && K ? q4::dgrad_workspace(P, E, N, K) : 0;
  return Q4_OK;
}

q4_status q4_wgrad_workspace(int64_t P, int32_t E, int64_t N, int64_t K, size_t* bytes) {
  if (!bytes) return Q4_ERR_NULL;
  if (P < 0 || E < 0 || E > 65535 || N < 0 || K < 0 || P >= kMaxDim || N > kMaxGradLd || K > kMaxGradLd)
    return Q4_ERR_SHAPE;
  *bytes = E && N && K ? q4::wgrad_workspace(P, E, N, K) : 0;
  return Q4_OK;
}

q4_status q4_dgrad_plan(int64_t P, int32_t E, int64_t N, int64_t K, int32_t* block_rows, int32_t* parts) {
  if (!block_rows || !parts) return Q4_ERR_NULL;
  size_t bytes = 0;
  const q4_status st = q4_dgrad_workspace(P, E, N, K, &bytes);
  if (st != Q4_OK) return st;
  const q4::GradPlan p = P && E && K ? q4::grad_plan(false, false, P, E, N, K) : q4::GradPlan{0, 0};
  *block_rows = p.rows;
  *parts = p.parts;
  return Q4_OK;
}

q4_status q4_wgrad_plan(int64_t P, int32_t E, int64_t N, int64_t K, int a_is_bf16, int32_t* block_rows,
                        int32_t* parts) {
  if (!block_rows || !parts) return Q4_ERR_NULL;
  size_t bytes = 0;
  const q4_status st = q4_wgrad_workspace(P, E, N, K, &bytes);
  if (st != Q4_OK) return st;
  const q4::GradPlan p = E && N && K ? q4::grad_plan(true, a_is_bf16 != 0, P, E, N, K) : q4::GradPlan{0, 0};
  *block_rows = p.rows;
  *parts = p.parts;
  return Q4_OK;
}

q4_status q4_gemm_dgrad(int64_t M, const void* dC_bf16, int64_t lddc, const q4_tensor* W, void* dA_bf16, int64_t ldda,
                        void* workspace, size_t workspace_bytes, void* stream) {
  if (!W) return Q4_ERR_NULL;
  return dgrad(dC_bf16, lddc, nullptr, 1, M, W, W->rows, dA_bf16, ldda, workspace, workspace_bytes, stream);
}

q4_status q4_grouped_gemm_dgrad(const void* dC_bf16, int64_t lddc, const int32_t* expert_offsets, int32_t E, int64_t P,
                                const q4_tensor* W, int64_t N, void* dA_bf16, int64_t ldda, void* workspace,
                                size_t workspace_bytes, void* stream) {
  if (E > 0 && P > 0 && !expert_offsets) return Q4_ERR_NULL;
  return dgrad(dC_bf16, lddc, expert_offsets, E, P, W, N, dA_bf16, ldda, workspace, workspace_bytes, stream);
}

q4_status q4_gemm_wgrad(int64_t M, const void* dC_bf16, int64_t lddc, const void* A_bf16, int64_t lda,
                        const q4_tensor* A_q, int64_t N, int64_t K, void* dW, int dw_dtype, int64_t lddw,
                        int accumulate, void* workspace, size_t workspace_bytes, void* stream) {
  return wgrad(dC_bf16, lddc, A_bf16, lda, A_q, M, nullptr, nullptr, 1, M, N, K, dW, dw_dtype, lddw, accumulate,
               workspace, workspace_bytes, stream);
}

q4_status q4_grouped_gemm_wgrad(const void* dC_bf16, int64_t lddc, const void* A_bf16, int64_t lda,
                                const q4_tensor* A_q, int64_t T, const int32_t* gather, const int32_t* expert_offsets,
                                int32_t E, int64_t P, int64_t N, int64_t K, void* dW, int dw_dtype, int64_t lddw,
                                int accumulate, void* workspace, size_t workspace_bytes, void* stream) {
  if (E > 0 && !expert_offsets) return Q4_ERR_NULL;
  return wgrad(dC_bf16, lddc, A_bf16, lda, A_q, T, gather, expert_offsets, E, P, N, K, dW, dw_dtype, lddw, accumulate,
               workspace, workspace_bytes, stream);
}

}  // extern "C"

namespace {

q4_status dgrad(const void* dC, int64_t lddc, const int32_t* offsets, int32_t E, int64_t P, const q4_tensor* W,
                int64_t N, void* dA, int64_t ldda, void* workspace, size_t workspace_bytes, void* stream) {
  q4_status st = check_tensor(W);
  if (st != Q4_OK) return st;
  if (!is_weight(W->fmt)) return Q4_ERR_FORMAT;
  size_t need = 0;
  const int64_t K = W->cols;
  st = q4_dgrad_workspace(P, E, N, K, &need);
  if (st != Q4_OK) return st;
  if (W->rows != (int64_t)E * N || N % 8 || K % 128) return Q4_ERR_SHAPE;
  if (offsets && W->layout == Q4_LAYOUT_TILED && N % 16) return Q4_ERR_SHAPE;  // experts own whole tiles
  if (E == 0 || P == 0 || K == 0) return Q4_OK;
  if (!q4::dgrad_fits(P, E, N, K)) return Q4_ERR_SHAPE;
  if (!aligned(offsets, 4)) return Q4_ERR_ALIGN;
  st = check_bf16(dC, P, N, lddc);
  if (st != Q4_OK) return st;
  if (P > 1 && lddc > kMaxGradLd) return Q4_ERR_SHAPE;
  st = check_bf16(dA, P, K, ldda);
  if (st != Q4_OK) return st;
  if (need && !workspace) return Q4_ERR_NULL;
  if (workspace_bytes < need) return Q4_ERR_SHAPE;
  if (need && !aligned(workspace, 16)) return Q4_ERR_ALIGN;
  q4::GradArgs g{};
  g.dc = static_cast<const uint16_t*>(dC);
  g.lddc = P > 1 ? lddc : N;  // (a single row's stride is never used)
  g.offsets = offsets;
  g.E = E;
  g.P = P;
  g.N = N;
  g.K = K;
  g.b = static_cast<const uint8_t*>(W->codes);
  g.b_scales = static_cast<const uint8_t*>(W->scales);
  g.gs = W->global_scale;
  g.out = dA;
  g.ldo = ldda;
  g.workspace = static_cast<float*>(workspace);
  return hip_status(q4::launch_dgrad(W->fmt, W->layout, g, as_stream(stream)));
}

q4_status wgrad(const void* dC, int64_t lddc, const void* A_bf16, int64_t lda, const q4_tensor* A_q, int64_t T,
                const int32_t* gather, const int32_t* offsets, int32_t E, int64_t P, int64_t N, int64_t K, void* dW,
                int dw_dtype, int64_t lddw, int accumulate, void* workspace, size_t workspace_bytes, void* stream) {
  size_t need = 0;
  q4_status st = q4_wgrad_workspace(P, E, N, K, &need);
  if (st != Q4_OK) return st;
  if (dw_dtype != 0 && dw_dtype != 1) return Q4_ERR_FORMAT;
  if (accumulate && dw_dtype != 1) return Q4_ERR_FORMAT;
  if ((A_bf16 == nullptr) == (A_q == nullptr)) return A_bf16 ? Q4_ERR_FORMAT : Q4_ERR_NULL;
  if (T < 0 || T >= kMaxDim || N % 8 || K % (A_q ? 32 : 8)) return Q4_ERR_SHAPE;
  if (A_q) {
    st = check_tensor(A_q);
    if (st != Q4_OK) return st;
    if (!is_mx8(A_q->fmt)) return Q4_ERR_FORMAT;
    if (A_q->rows != T || A_q->cols != K) return Q4_ERR_SHAPE;
  }
  if (E == 0 || N == 0 || K == 0) return Q4_OK;
  if (!q4::wgrad_fits(P, E, N, K)) return Q4_ERR_SHAPE;
  if (!gather && T < P) return Q4_ERR_SHAPE;  // row p of dC goes with row p of A
  if (!aligned(gather, 4) || !aligned(offsets, 4)) return Q4_ERR_ALIGN;
  st = check_bf16(dC, P, N, lddc);
  if (st != Q4_OK) return st;
  if (P > 1 && lddc > kMaxGradLd) return Q4_ERR_SHAPE;
  if (!A_q) {
    st = check_bf16(A_bf16, T, K, lda);
    if (st != Q4_OK) return st;
    if (T > 1 && lda > kMaxGradLd) return Q4_ERR_SHAPE;
  }
  if (!dW) return Q4_ERR_NULL;
  if (lddw < K) return Q4_ERR_SHAPE;
  if (!aligned(dW, 16) || lddw % (dw_dtype ? 4 : 8)) return Q4_ERR_ALIGN;
  if (need && !workspace) return Q4_ERR_NULL;
  if (workspace_bytes < need) return Q4_ERR_SHAPE;
  if (need && !aligned(workspace, 16)) return Q4_ERR_ALIGN;
  q4::GradArgs g{};
  g.dc = static_cast<const uint16_t*>(dC);
  g.lddc = P > 1 ? lddc : N;  // (a single row's stride is never used)
  g.offsets = offsets;
  g.gather = gather;
  g.E = E;
  g.P = T ? P : 0;  // no activations: every row reads zeros
  g.N = N;
  g.K = K;
  g.T = T;
  g.b = static_cast<const uint8_t*>(A_q ? A_q->codes : A_bf16);
  g.b_scales = A_q ? static_cast<const uint8_t*>(A_q->scales) : nullptr;
  g.ldb = T > 1 ? lda : K;
  g.out = dW;
  g.ldo = lddw;
  g.out_f32 = dw_dtype;
  g.accumulate = accumulate;
  g.workspace = static_cast<float*>(workspace);
  return hip_status(q4::launch_wgrad(A_q ? A_q->fmt : 7, g, as_stream(stream)));
}

}  // namespace
