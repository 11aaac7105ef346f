/*
 * libqlora -- RMS norm and the 8-bit integer linear, on one B200 (sm_100a).
 *
 * The operators next to the NF4 linear of qlora.h in a model: the RMS norm with
 * the residual's addition that feeds every linear, and the linear on an 8-bit
 * base (the merged weight of qlora_nf4_merge on its way to serving, or a frozen
 * 8-bit base under adapters), whose activations the norm can hand over in 8
 * bits. The conventions of qlora.h hold: row-major contiguous matrices, bf16 as
 * 16-bit patterns, device pointers 16-byte aligned (per-row and per-channel
 * fp32 vectors included) and in the current device's memory, nothing allocated
 * or synchronised, argument errors returned before anything is launched. A call's
 * kernels may set themselves up while earlier work on the stream still runs; they
 * read and write nothing before it has finished.
 *
 * An int8 matrix is codes int8 [rows, cols] and scale fp32 [rows], value
 * codes * scale: one scale a token for activations, one an output channel for
 * a weight [N, K].
 */
#ifndef QLORA_I8_H
#define QLORA_I8_H

#include "qlora.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of the arguments that come in two. */
typedef enum { QLORA_TYPE_BF16 = 0, QLORA_TYPE_F32 = 1 } qlora_type_t;

/* Quantise the rows of X (device, [M, K] of x_type) to int8, one scale a row:
 *   v = x, or fp32_rn(x * col_scale[k]) when col_scale [K] is given;
 *   c = max_k |v|;  scale = fp32_rn(c * fp32_rn(1 / 127));
 *   code = rint(fp32_rn(v / scale)) (half to even) clamped to +-127; 0 when scale is 0.
 * A row that holds a NaN or an infinity (after the column scale) gets the
 * scale NaN and codes 0, so that what is computed from it is NaN.
 * codes int8 [M, K], scale fp32 [M]. M >= 1, 1 <= K <= 65536, M * K < 2^47.
 * Errors: INVALID_ARG, UNSUPPORTED_SHAPE, MISALIGNED, CUDA. */
qlora_status_t qlora_i8_quantize(const void *X, int32_t x_type, int64_t M, int64_t K, const float *col_scale,
                                 int8_t *codes, float *scale, qlora_stream_t stream);

/* out [M, K] bf16 = bf16_rn(fp32_rn(code * scale[row])). Shapes and errors as
 * qlora_i8_quantize. */
qlora_status_t qlora_i8_dequantize(const int8_t *codes, const float *scale, int64_t M, int64_t K, uint16_t *out,
                                   qlora_stream_t stream);

/* RMS norm of the residual stream, with the residual's addition:
 *   h = x + r rounded to h_type (h = x, or h = r, when only one is given);
 *   y = h / sqrt(mean_k h^2 + eps) * w   in fp32, from the h that is stored.
 * X [M, K] bf16 (a block's output) and R [M, K] of h_type (the stream): one of
 *   the two may be NULL; with R NULL h_type is QLORA_TYPE_BF16.
 * weight [K] of w_type. eps >= 0, finite.
 * Outputs, each optional, at least one of Y and codes: H [M, K] of h_type (may
 *   be R, or X where h_type is bf16: every element is read before it is
 *   written); Y [M, K] = bf16_rn(y) (may be X where H is not: H and Y in one
 *   buffer are refused); codes [M, K] and scale [M] (both or neither) = the int8
 *   rows of y as qlora_i8_quantize would give them for the fp32 y (y is not
 *   rounded to bf16 first).
 * M >= 1, 1 <= K <= 32768. Errors: INVALID_ARG, UNSUPPORTED_SHAPE, MISALIGNED, CUDA. */
qlora_status_t qlora_rmsnorm_fwd(const uint16_t *X, const void *R, int32_t h_type, const void *weight,
                                 int32_t w_type, float eps, int64_t M, int64_t K, void *H, uint16_t *Y,
                                 int8_t *codes, float *scale, qlora_stream_t stream);

/* Workspace bytes of qlora_rmsnorm_bwd when dW is asked for, on the current
 * device (it scales with the SM count); 0 for a few short rows, which need
 * none (ws may then be NULL). It needs no initialisation. The
 * workspace may be reused by consecutive calls on one stream; calls that run
 * concurrently need separate ones. Errors: INVALID_ARG, UNSUPPORTED_SHAPE. */
qlora_status_t qlora_rmsnorm_workspace(int64_t M, int64_t K, size_t *bytes);

/* Backward of qlora_rmsnorm_fwd, with rstd = 1 / sqrt(mean h^2 + eps) formed
 * again from H (the forward keeps nothing for it):
 *   dh[m, k] = rstd (w dy - h rstd^2 mean_k(w dy h)) + dR
 *   dW[k]    = sum_m dy h rstd                       (fp32, overwritten)
 * dY [M, K] bf16; H [M, K] of h_type, the forward's h; dR [M, K] of h_type or
 * NULL: the gradient that reaches h along the residual stream.
 * dH [M, K] of h_type (may be dR, or dY where h_type is bf16): the gradient of
 * both x and r. dX [M, K] bf16 or NULL: dh rounded to bf16, for the block
 * output's backward where the stream is fp32 (may be dY). dH or dX may be NULL,
 * not both. dW [K] or NULL (a frozen norm); with dW, ws of at least
 * qlora_rmsnorm_workspace() bytes, 16-byte aligned, else ws is not read. The
 * result does not depend on timing.
 * M >= 1, 1 <= K <= 32768. Errors: INVALID_ARG, UNSUPPORTED_SHAPE, MISALIGNED,
 * WORKSPACE, CUDA. */
qlora_status_t qlora_rmsnorm_bwd(const uint16_t *dY, const void *H, int32_t h_type, const void *weight,
                                 int32_t w_type, float eps, const void *dR, int64_t M, int64_t K, void *dH,
                                 uint16_t *dX, float *dW, void *ws, size_t ws_bytes, qlora_stream_t stream);

/* The 8-bit linear with the adapter's term:
 *   Y[m, n] = bf16_rn(fp32(sum_k Xq[m, k] Wq[n, k]) sx[m] sw[n] + sum_j sU[m, j] B[n, j])
 * The sum over k is exact (int32); the rest is fp32, rounded once.
 * Xq int8 [M, K] with sx fp32 [M]; Wq int8 [N, K] with sw fp32 [N] (any codes,
 * -128 among them). sU [M, r] and B [N, r] bf16 as in qlora_fused_fwd, r as
 * there (r % 8 == 0, 8 <= r <= 64), or r = 0 and both ignored. Y [M, N] bf16.
 * M >= 1, N % 16 == 0, K % 16 == 0, 16 <= K <= 131056 (the int32 sum then
 * cannot overflow).
 * dev_status: as in qlora_linear_fwd (TIMEOUT).
 * Errors: INVALID_ARG, UNSUPPORTED_SHAPE, MISALIGNED, CUDA. */
qlora_status_t qlora_i8_linear_fwd(const int8_t *Xq, const float *sx, int64_t M, const int8_t *Wq, const float *sw,
                                   int64_t N, int64_t K, const uint16_t *sU, const uint16_t *B, int32_t r,
                                   uint16_t *Y, int32_t *dev_status, qlora_stream_t stream);

/* Workspace bytes of qlora_i8_linear_dx (the gradient's codes and scales); it
 * needs no initialisation and is shared as qlora_rmsnorm_workspace's.
 * Errors: INVALID_ARG, UNSUPPORTED_SHAPE. */
qlora_status_t qlora_i8_linear_workspace(int64_t M, int64_t N, int64_t K, size_t *bytes);

/* The gradient of the 8-bit linear's input, W frozen, through int8 products:
 *   (gq, sg) = qlora_i8_quantize of dY with col_scale = sw (rows of N)
 *   dX[m, k] = bf16_rn(fp32(sum_n gq[m, n] Wq[n, k]) sg[m] + sum_j sT[m, j] A[j, k])
 * An element of dY sw is off by up to half its row's step, max_n |dY sw| / 254: a
 * row with one loud element loses what is far smaller.
 * dY [M, N] bf16; sT [M, r] and A [r, K] bf16 as in qlora_fused_dx, or r = 0.
 * dX [M, K] bf16. The adapter's gradients are qlora_lora_grads as for the NF4
 * linear. M >= 1, N % 16 == 0, K % 16 == 0, N <= 65536; K, which is not summed
 * over, may pass the forward's limit.
 * Errors: as qlora_i8_linear_fwd, and WORKSPACE. */
qlora_status_t qlora_i8_linear_dx(const uint16_t *dY, int64_t M, const int8_t *Wq, const float *sw, int64_t N,
                                  int64_t K, const uint16_t *sT, const uint16_t *A, int32_t r, uint16_t *dX,
                                  void *ws, size_t ws_bytes, int32_t *dev_status, qlora_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* QLORA_I8_H */
