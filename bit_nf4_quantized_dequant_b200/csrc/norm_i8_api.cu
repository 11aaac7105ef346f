// The C ABI of include/qlora_i8.h: argument checks and launches. Nothing here
// allocates device memory or synchronises.
#include <cmath>

#include "i8_gemm.cuh"
#include "norm_i8.h"

using namespace qlora;

namespace {

constexpr int64_t kMaxQuantCols = 65536, kMaxNormCols = 32768, kMaxContraction = 131056;
constexpr int64_t kMaxRows = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxLinear = (int64_t(1) << 31) - 1024;   // tile coordinates stay in 31 bits

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
template <class... P>
bool all_aligned16(const P *...p) {
  return (aligned16(p) && ...);
}
bool type_ok(int32_t t) { return t == QLORA_TYPE_BF16 || t == QLORA_TYPE_F32; }
size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
qlora_status_t cuda_status(cudaError_t e) { return e == cudaSuccess ? QLORA_OK : QLORA_ERR_CUDA; }
cudaStream_t cu(qlora_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

qlora_status_t check_rows(int64_t M, int64_t K, int64_t most) {
  if (M < 1 || K < 1) return QLORA_ERR_INVALID_ARG;
  if (K > most || M > kMaxRows) return QLORA_ERR_UNSUPPORTED_SHAPE;
  return QLORA_OK;
}

// The shapes and adapter of both products. Only the dimension that is summed over
// has a limit of its own: K in the forward, N in the gradient (whose rows of N the
// codec also quantises, the lower limit of the two).
qlora_status_t check_i8_shape(bool dx, int64_t M, int64_t N, int64_t K, int32_t r) {
  if (M < 1 || N < 1 || K < 1) return QLORA_ERR_INVALID_ARG;
  if (N % 16 || K % 16 || M > kMaxLinear) return QLORA_ERR_UNSUPPORTED_SHAPE;
  if (N > (dx ? kMaxQuantCols : kMaxLinear) || K > (dx ? kMaxLinear : kMaxContraction)) return QLORA_ERR_UNSUPPORTED_SHAPE;
  if (r != 0 && (r < 8 || r > 64 || r % 8)) return QLORA_ERR_UNSUPPORTED_SHAPE;
  return QLORA_OK;
}

}  // namespace

extern "C" {

qlora_status_t qlora_i8_quantize(const void *X, int32_t x_type, int64_t M, int64_t K, const float *col_scale,
                                 int8_t *codes, float *scale, qlora_stream_t stream) {
  if (!X || !codes || !scale || !type_ok(x_type)) return QLORA_ERR_INVALID_ARG;
  const qlora_status_t st = check_rows(M, K, kMaxQuantCols);
  if (st != QLORA_OK) return st;
  if (!all_aligned16(X, col_scale, codes, scale)) return QLORA_ERR_MISALIGNED;
  return cuda_status(launch_i8_quantize(X, x_type == QLORA_TYPE_F32, M, K, col_scale, codes, scale, cu(stream)));
}

qlora_status_t qlora_i8_dequantize(const int8_t *codes, const float *scale, int64_t M, int64_t K, uint16_t *out,
                                   qlora_stream_t stream) {
  if (!codes || !scale || !out) return QLORA_ERR_INVALID_ARG;
  const qlora_status_t st = check_rows(M, K, kMaxQuantCols);
  if (st != QLORA_OK) return st;
  if (!all_aligned16(codes, scale, out)) return QLORA_ERR_MISALIGNED;
  return cuda_status(launch_i8_dequantize(codes, scale, M, K, out, cu(stream)));
}

qlora_status_t qlora_rmsnorm_fwd(const uint16_t *X, const void *R, int32_t h_type, const void *weight, int32_t w_type,
                                 float eps, int64_t M, int64_t K, void *H, uint16_t *Y, int8_t *codes, float *scale,
                                 qlora_stream_t stream) {
  if ((!X && !R) || !weight || !type_ok(h_type) || !type_ok(w_type)) return QLORA_ERR_INVALID_ARG;
  if (!R && h_type != QLORA_TYPE_BF16) return QLORA_ERR_INVALID_ARG;
  if ((!Y && !codes) || !codes != !scale) return QLORA_ERR_INVALID_ARG;
  if (Y && H == Y) return QLORA_ERR_INVALID_ARG;   // both outputs in one buffer
  if (!std::isfinite(eps) || eps < 0.f) return QLORA_ERR_INVALID_ARG;
  const qlora_status_t st = check_rows(M, K, kMaxNormCols);
  if (st != QLORA_OK) return st;
  if (!all_aligned16(X, R, weight, H, Y, codes, scale)) return QLORA_ERR_MISALIGNED;
  return cuda_status(launch_rmsnorm_fwd(X, R, h_type == QLORA_TYPE_F32, weight, w_type == QLORA_TYPE_F32, eps, M, K, H,
                                        Y, codes, scale, cu(stream)));
}

qlora_status_t qlora_rmsnorm_workspace(int64_t M, int64_t K, size_t *bytes) {
  if (!bytes) return QLORA_ERR_INVALID_ARG;
  const qlora_status_t st = check_rows(M, K, kMaxNormCols);
  if (st != QLORA_OK) return st;
  *bytes = rmsnorm_bwd_ws_bytes(M, K);
  return QLORA_OK;
}

qlora_status_t qlora_rmsnorm_bwd(const uint16_t *dY, const void *H, int32_t h_type, const void *weight, int32_t w_type,
                                 float eps, const void *dR, int64_t M, int64_t K, void *dH, uint16_t *dX, float *dW,
                                 void *ws, size_t ws_bytes, qlora_stream_t stream) {
  if (!dY || !H || !weight || !type_ok(h_type) || !type_ok(w_type) || (!dH && !dX)) return QLORA_ERR_INVALID_ARG;
  if (!std::isfinite(eps) || eps < 0.f) return QLORA_ERR_INVALID_ARG;
  const qlora_status_t st = check_rows(M, K, kMaxNormCols);
  if (st != QLORA_OK) return st;
  if (!all_aligned16(dY, H, weight, dR, dH, dX, dW)) return QLORA_ERR_MISALIGNED;
  const size_t need = dW ? rmsnorm_bwd_ws_bytes(M, K) : 0;
  if (need && (!ws || ws_bytes < need)) return QLORA_ERR_WORKSPACE;
  if (need && !aligned16(ws)) return QLORA_ERR_MISALIGNED;
  return cuda_status(launch_rmsnorm_bwd(dY, H, h_type == QLORA_TYPE_F32, weight, w_type == QLORA_TYPE_F32, eps, dR, M,
                                        K, dH, dX, dW, ws, cu(stream)));
}

qlora_status_t qlora_i8_linear_fwd(const int8_t *Xq, const float *sx, int64_t M, const int8_t *Wq, const float *sw,
                                   int64_t N, int64_t K, const uint16_t *sU, const uint16_t *B, int32_t r, uint16_t *Y,
                                   int32_t *dev_status, qlora_stream_t stream) {
  if (!Xq || !sx || !Wq || !sw || !Y) return QLORA_ERR_INVALID_ARG;
  const qlora_status_t st = check_i8_shape(false, M, N, K, r);
  if (st != QLORA_OK) return st;
  if (r && (!sU || !B)) return QLORA_ERR_INVALID_ARG;
  if (!all_aligned16(Xq, sx, Wq, sw, Y) || (r && !all_aligned16(sU, B))) return QLORA_ERR_MISALIGNED;
  if (reinterpret_cast<uintptr_t>(dev_status) & 3u) return QLORA_ERR_MISALIGNED;
  I8GemmArgs a{};
  a.act = Xq;
  a.act_scale = sx;
  a.w = Wq;
  a.w_scale = sw;
  a.M = M;
  a.F = N;
  a.C = K;
  a.r = r;
  a.lora_act = sU;
  a.lora_w = B;
  a.out = Y;
  a.status = dev_status;
  return cuda_status(launch_i8_gemm(a, cu(stream)));
}

qlora_status_t qlora_i8_linear_workspace(int64_t M, int64_t N, int64_t K, size_t *bytes) {
  if (!bytes) return QLORA_ERR_INVALID_ARG;
  const qlora_status_t st = check_i8_shape(true, M, N, K, 0);
  if (st != QLORA_OK) return st;
  *bytes = round_up(static_cast<size_t>(M) * N, 256) + static_cast<size_t>(M) * 4;
  return QLORA_OK;
}

qlora_status_t qlora_i8_linear_dx(const uint16_t *dY, int64_t M, const int8_t *Wq, const float *sw, int64_t N,
                                  int64_t K, const uint16_t *sT, const uint16_t *A, int32_t r, uint16_t *dX, void *ws,
                                  size_t ws_bytes, int32_t *dev_status, qlora_stream_t stream) {
  if (!dY || !Wq || !sw || !dX) return QLORA_ERR_INVALID_ARG;
  qlora_status_t st = check_i8_shape(true, M, N, K, r);
  if (st != QLORA_OK) return st;
  if (r && (!sT || !A)) return QLORA_ERR_INVALID_ARG;
  if (!all_aligned16(dY, Wq, sw, dX) || (r && !all_aligned16(sT, A))) return QLORA_ERR_MISALIGNED;
  if (reinterpret_cast<uintptr_t>(dev_status) & 3u) return QLORA_ERR_MISALIGNED;
  size_t need = 0;
  st = qlora_i8_linear_workspace(M, N, K, &need);
  if (st != QLORA_OK) return st;
  if (!ws || ws_bytes < need) return QLORA_ERR_WORKSPACE;
  if (!aligned16(ws)) return QLORA_ERR_MISALIGNED;
  int8_t *gq = static_cast<int8_t *>(ws);
  float *sg = reinterpret_cast<float *>(gq + round_up(static_cast<size_t>(M) * N, 256));
  const cudaError_t e = launch_i8_quantize(dY, false, M, N, sw, gq, sg, cu(stream));
  if (e != cudaSuccess) return QLORA_ERR_CUDA;
  I8GemmArgs a{};
  a.dx = true;
  a.act = gq;
  a.act_scale = sg;
  a.w = Wq;
  a.M = M;
  a.F = K;
  a.C = N;
  a.r = r;
  a.lora_act = sT;
  a.lora_w = A;
  a.out = dX;
  a.status = dev_status;
  return cuda_status(launch_i8_gemm(a, cu(stream)));
}

}  // extern "C"
