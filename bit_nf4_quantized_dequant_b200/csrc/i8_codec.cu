// Int8 rows with one fp32 scale a row: quantise and dequantise.
//
//   v = x (or fp32_rn(x * col_scale)),  s = fp32_rn(max |v| * fp32_rn(1 / 127)),
//   code = rint(fp32_rn(v / s)) clamped to +-127.
//
// Both are bound by memory (2 to 4 bytes read and 1 written an element), so a
// row is read once and kept in registers between its maximum and its codes.
#include "norm_i8.h"
#include "row_device.cuh"

namespace qlora {
namespace {

// A row per warp (WARP) or per block; a thread holds NV vectors of VEC
// elements: element (i * T + t) * VEC of thread t.
template <int VEC, int NV, bool WARP, bool F32>
__global__ void __launch_bounds__(WARP ? 256 : 1024)
    i8_quantize_kernel(const void *__restrict__ X, const float *__restrict__ col_scale, int64_t M, int64_t K,
                       int8_t *__restrict__ codes, float *__restrict__ scale) {
  __shared__ uint32_t slot[32];
  const int T = WARP ? 32 : blockDim.x;
  const int t = WARP ? (threadIdx.x & 31) : threadIdx.x;
  const int64_t m = WARP ? static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
  if (WARP && m >= M) return;
  const void *row = F32 ? static_cast<const void *>(static_cast<const float *>(X) + m * K)
                        : static_cast<const void *>(static_cast<const uint16_t *>(X) + m * K);
  float f[NV][VEC];
  uint32_t mx = 0;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t k = static_cast<int64_t>(i * T + t) * VEC;
    if (k < K) {
      load_row<VEC, F32>(f[i], row, k);
    } else {
#pragma unroll
      for (int j = 0; j < VEC; ++j) f[i][j] = 0.f;
    }
  }
  if (col_scale) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t k = static_cast<int64_t>(i * T + t) * VEC;
      if (k < K) {
        float c[VEC];
        load_row<VEC, true>(c, col_scale, k);
#pragma unroll
        for (int j = 0; j < VEC; ++j) f[i][j] = __fmul_rn(f[i][j], c[j]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) mx = max(mx, mag_bits(f[i][j]));
  const RowScale rs = row_scale(row_max<WARP>(mx, slot));
  if (t == 0) scale[m] = rs.s;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t k = static_cast<int64_t>(i * T + t) * VEC;
    if (k < K) store_codes<VEC>(f[i], rs, codes + m * K, k);
  }
}

// Rows too long for registers: read twice (the second time mostly from L2).
template <int VEC, bool F32>
__global__ void __launch_bounds__(1024)
    i8_quantize_long_kernel(const void *__restrict__ X, const float *__restrict__ col_scale, int64_t M, int64_t K,
                            int8_t *__restrict__ codes, float *__restrict__ scale) {
  __shared__ uint32_t slot[32];
  const int64_t m = blockIdx.x;
  const void *row = F32 ? static_cast<const void *>(static_cast<const float *>(X) + m * K)
                        : static_cast<const void *>(static_cast<const uint16_t *>(X) + m * K);
  auto load = [&](float (&f)[VEC], int64_t k) {
    load_row<VEC, F32>(f, row, k);
    if (col_scale) {
      float c[VEC];
      load_row<VEC, true>(c, col_scale, k);
#pragma unroll
      for (int j = 0; j < VEC; ++j) f[j] = __fmul_rn(f[j], c[j]);
    }
  };
  uint32_t mx = 0;
  for (int64_t k = static_cast<int64_t>(threadIdx.x) * VEC; k < K; k += static_cast<int64_t>(blockDim.x) * VEC) {
    float f[VEC];
    load(f, k);
#pragma unroll
    for (int j = 0; j < VEC; ++j) mx = max(mx, mag_bits(f[j]));
  }
  const RowScale rs = row_scale(row_max<false>(mx, slot));
  if (threadIdx.x == 0) scale[m] = rs.s;
  for (int64_t k = static_cast<int64_t>(threadIdx.x) * VEC; k < K; k += static_cast<int64_t>(blockDim.x) * VEC) {
    float f[VEC];
    load(f, k);
    store_codes<VEC>(f, rs, codes + m * K, k);
  }
}

template <int VEC>
__global__ void __launch_bounds__(256)
    i8_dequantize_kernel(const int8_t *__restrict__ codes, const float *__restrict__ scale, int64_t M, int64_t K,
                         uint16_t *__restrict__ out) {
  const int64_t per_row = (K + VEC - 1) / VEC, total = M * per_row;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t m = i / per_row, k = (i - m * per_row) * VEC;
    const float s = scale[m];
    float f[VEC];
    if constexpr (VEC == 8) {
      const uint2 u = *reinterpret_cast<const uint2 *>(codes + m * K + k);
      const uint32_t w[2] = {u.x, u.y};
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = __fmul_rn(static_cast<float>(static_cast<int8_t>(w[j >> 2] >> (8 * (j & 3)))), s);
    } else {
      f[0] = __fmul_rn(static_cast<float>(codes[m * K + k]), s);
    }
    store_row<VEC, false>(f, out + m * K, k);
  }
}

template <int VEC, int NV, bool WARP>
cudaError_t quantize_nv(const void *X, bool f32, const float *cs, int64_t M, int64_t K, int8_t *codes, float *scale,
                        int threads, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>(WARP ? (M + threads / 32 - 1) / (threads / 32) : M));
  if (f32) i8_quantize_kernel<VEC, NV, WARP, true><<<grid, threads, 0, st>>>(X, cs, M, K, codes, scale);
  else i8_quantize_kernel<VEC, NV, WARP, false><<<grid, threads, 0, st>>>(X, cs, M, K, codes, scale);
  return cudaGetLastError();
}

template <int VEC>
cudaError_t quantize_long(const void *X, bool f32, const float *cs, int64_t M, int64_t K, int8_t *codes, float *scale,
                          cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>(M));
  if (f32) i8_quantize_long_kernel<VEC, true><<<grid, 1024, 0, st>>>(X, cs, M, K, codes, scale);
  else i8_quantize_long_kernel<VEC, false><<<grid, 1024, 0, st>>>(X, cs, M, K, codes, scale);
  return cudaGetLastError();
}

int round32(int64_t t) { return static_cast<int>((t + 31) / 32 * 32); }

}  // namespace

cudaError_t launch_i8_quantize(const void *X, bool f32, int64_t M, int64_t K, const float *cs, int8_t *codes,
                               float *scale, cudaStream_t st) {
  if (K % 8 == 0) {
    const int64_t v = K / 8;
    if (v <= 32) return quantize_nv<8, 1, true>(X, f32, cs, M, K, codes, scale, 128, st);
    if (v <= 128) return quantize_nv<8, 4, true>(X, f32, cs, M, K, codes, scale, 128, st);
    if (v <= 1024 && M <= 2 * device_sm_count())
      return quantize_nv<8, 1, false>(X, f32, cs, M, K, codes, scale, round32(v), st);
    if (v <= 2048) return quantize_nv<8, 2, false>(X, f32, cs, M, K, codes, scale, round32((v + 1) / 2), st);
    if (v <= 4096) return quantize_nv<8, 4, false>(X, f32, cs, M, K, codes, scale, round32((v + 3) / 4), st);
    return quantize_long<8>(X, f32, cs, M, K, codes, scale, st);
  }
  if (K <= 128) return quantize_nv<1, 4, true>(X, f32, cs, M, K, codes, scale, 128, st);
  if (K <= 8192) return quantize_nv<1, 8, false>(X, f32, cs, M, K, codes, scale, round32((K + 7) / 8), st);
  if (K <= 32768) return quantize_nv<1, 32, false>(X, f32, cs, M, K, codes, scale, round32((K + 31) / 32), st);
  return quantize_long<1>(X, f32, cs, M, K, codes, scale, st);
}

cudaError_t launch_i8_dequantize(const int8_t *codes, const float *scale, int64_t M, int64_t K, uint16_t *out,
                                 cudaStream_t st) {
  const int vec = K % 8 ? 1 : 8;
  const int64_t blocks = (M * ((K + vec - 1) / vec) + 255) / 256, most = static_cast<int64_t>(device_sm_count()) * 8;
  const unsigned grid = static_cast<unsigned>(blocks < most ? blocks : most);
  if (vec == 8) i8_dequantize_kernel<8><<<grid, 256, 0, st>>>(codes, scale, M, K, out);
  else i8_dequantize_kernel<1><<<grid, 256, 0, st>>>(codes, scale, M, K, out);
  return cudaGetLastError();
}

}  // namespace qlora
