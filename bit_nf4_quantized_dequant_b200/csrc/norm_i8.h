// Launchers of the RMS norm and int8 kernels (not part of the ABI). Each
// returns the cudaError_t of its launches.
#pragma once

#include "qlora_internal.h"
#include "qlora_i8.h"

namespace qlora {

cudaError_t launch_i8_quantize(const void *X, bool f32, int64_t M, int64_t K, const float *col_scale, int8_t *codes,
                               float *scale, cudaStream_t st);
cudaError_t launch_i8_dequantize(const int8_t *codes, const float *scale, int64_t M, int64_t K, uint16_t *out,
                                 cudaStream_t st);

// hf, wf: the stream / the weight is fp32 (else bf16).
cudaError_t launch_rmsnorm_fwd(const uint16_t *X, const void *R, bool hf, const void *w, bool wf, float eps, int64_t M,
                               int64_t K, void *H, uint16_t *Y, int8_t *codes, float *scale, cudaStream_t st);
size_t rmsnorm_bwd_ws_bytes(int64_t M, int64_t K);
cudaError_t launch_rmsnorm_bwd(const uint16_t *dY, const void *H, bool hf, const void *w, bool wf, float eps,
                               const void *dR, int64_t M, int64_t K, void *dH, uint16_t *dX, float *dW, void *ws,
                               cudaStream_t st);

}  // namespace qlora
