// RMS norm with the residual's addition, forward and backward.
//
//   h = x + r (rounded to the stream's type);  rstd = 1 / sqrt(mean h^2 + eps)
//   y = h rstd w, as bf16 and / or as int8 codes with one scale a row
//   dh = rstd (w dy - h rstd^2 mean(w dy h)) + dr;   dw[k] = sum_m dy h rstd
//
// Both are bound by memory: a row is read once and stays in registers between
// its sums and its outputs. All sums are fp32: a thread adds its own elements,
// then the warp and the block add in a fixed order.
#include "norm_i8.h"
#include "row_device.cuh"

namespace qlora {
namespace {

struct NormArgs {
  const uint16_t *x;
  const void *r;
  const void *w;
  float eps;
  int64_t M, K;
  void *h;
  uint16_t *y;
  int8_t *codes;
  float *scale;
};

template <bool F32>
__device__ __forceinline__ const void *at(const void *p, int64_t i) {
  return F32 ? static_cast<const void *>(static_cast<const float *>(p) + i)
             : static_cast<const void *>(static_cast<const uint16_t *>(p) + i);
}
template <bool F32>
__device__ __forceinline__ void *at(void *p, int64_t i) {
  return F32 ? static_cast<void *>(static_cast<float *>(p) + i) : static_cast<void *>(static_cast<uint16_t *>(p) + i);
}

__device__ __forceinline__ float inv_rms(float sum, int64_t K, float eps) {
  return __frcp_rn(__fsqrt_rn(__fadd_rn(__fdiv_rn(sum, static_cast<float>(K)), eps)));
}

// A row per warp (WARP) or per block; a thread holds NV vectors of VEC
// elements: element (i * T + t) * VEC of thread t.
template <int VEC, int NV, bool WARP, bool HF32, bool WF32>
__global__ void __launch_bounds__(WARP ? 128 : 1024) rmsnorm_fwd_kernel(const NormArgs a) {
  __shared__ float slot_sum[32];
  __shared__ uint32_t slot_max[32];
  const int T = WARP ? 32 : blockDim.x;
  const int t = WARP ? (threadIdx.x & 31) : threadIdx.x;
  const int64_t m = WARP ? static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
  if (WARP && m >= a.M) return;
  const int64_t K = a.K;
  float f[NV][VEC];
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t k = static_cast<int64_t>(i * T + t) * VEC;
#pragma unroll
    for (int j = 0; j < VEC; ++j) f[i][j] = 0.f;
    if (k < K) {
      if (a.r) load_row<VEC, HF32>(f[i], at<HF32>(a.r, m * K), k);
      if (a.x) {
        float x[VEC];
        load_row<VEC, false>(x, a.x + m * K, k);
        if (a.r) {
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            const float h = __fadd_rn(f[i][j], x[j]);
            f[i][j] = HF32 ? h : bf16_round(h);
          }
        } else {
#pragma unroll
          for (int j = 0; j < VEC; ++j) f[i][j] = x[j];
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t k = static_cast<int64_t>(i * T + t) * VEC;
    if (a.h && k < K) store_row<VEC, HF32>(f[i], at<HF32>(a.h, m * K), k);
#pragma unroll
    for (int j = 0; j < VEC; ++j) sum = fmaf(f[i][j], f[i][j], sum);
  }
  const float rstd = inv_rms(row_sum<WARP>(sum, slot_sum), K, a.eps);
  uint32_t mx = 0;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t k = static_cast<int64_t>(i * T + t) * VEC;
    if (k < K) {
      float w[VEC];
      load_row<VEC, WF32>(w, a.w, k);
#pragma unroll
      for (int j = 0; j < VEC; ++j) f[i][j] = __fmul_rn(__fmul_rn(f[i][j], rstd), w[j]);
      if (a.y) store_row<VEC, false>(f[i], a.y + m * K, k);
#pragma unroll
      for (int j = 0; j < VEC; ++j) mx = max(mx, mag_bits(f[i][j]));
    }
  }
  if (!a.codes) return;
  const RowScale rs = row_scale(row_max<WARP>(mx, slot_max));
  if (t == 0) a.scale[m] = rs.s;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t k = static_cast<int64_t>(i * T + t) * VEC;
    if (k < K) store_codes<VEC>(f[i], rs, a.codes + m * K, k);
  }
}

struct NormGradArgs {
  const uint16_t *dy;
  const void *h;
  const void *w;
  float eps;
  const void *dr;
  int64_t M, K;
  void *dh;
  uint16_t *dx;
  float *part;   // [gridDim.x, K] partial dw, or null
};

// The row's two sums, over the threads of a block.
struct Sums {
  float hh, wdyh;
};
__device__ __forceinline__ Sums block_sums(float hh, float wdyh, float2 *slot) {
  hh = warp_sum(hh);
  wdyh = warp_sum(wdyh);
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  if (lane == 0) slot[threadIdx.x >> 5] = make_float2(hh, wdyh);
  __syncthreads();
  const float2 v = lane < warps ? slot[lane] : make_float2(0.f, 0.f);
  return {warp_sum(v.x), warp_sum(v.y)};
}

// Persistent blocks over the rows; a thread keeps its columns' weight and dw
// sums in registers. Two slots for the sums: a block barrier lies between a
// slot's reads and its next write.
template <int VEC, int NV, bool HF32, bool WF32>
__global__ void __launch_bounds__(NV * VEC <= 8 ? 1024 : 512) rmsnorm_bwd_kernel(const NormGradArgs a) {
  __shared__ float2 slot[2][32];
  const int T = blockDim.x, t = threadIdx.x;
  const int64_t K = a.K;
  float w[NV][VEC], dw[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t k = static_cast<int64_t>(i * T + t) * VEC;
#pragma unroll
    for (int j = 0; j < VEC; ++j) w[i][j] = dw[i][j] = 0.f;
    if (k < K) load_row<VEC, WF32>(w[i], a.w, k);
  }
  int flip = 0;
  for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x, flip ^= 1) {
    float h[NV][VEC], g[NV][VEC];
    float hh = 0.f, gh = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t k = static_cast<int64_t>(i * T + t) * VEC;
#pragma unroll
      for (int j = 0; j < VEC; ++j) h[i][j] = g[i][j] = 0.f;
      if (k < K) {
        load_row<VEC, HF32>(h[i], at<HF32>(a.h, m * K), k);
        load_row<VEC, false>(g[i], a.dy + m * K, k);
      }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        hh = fmaf(h[i][j], h[i][j], hh);
        gh = fmaf(w[i][j] * g[i][j], h[i][j], gh);
      }
    const Sums s = block_sums(hh, gh, slot[flip]);
    const float rstd = inv_rms(s.hh, K, a.eps);
    const float c = s.wdyh / static_cast<float>(K) * rstd * rstd;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t k = static_cast<int64_t>(i * T + t) * VEC;
      if (k < K) {
        float d[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          dw[i][j] = fmaf(g[i][j], h[i][j] * rstd, dw[i][j]);
          d[j] = rstd * (w[i][j] * g[i][j] - h[i][j] * c);
        }
        if (a.dr) {
          float r[VEC];
          load_row<VEC, HF32>(r, at<HF32>(a.dr, m * K), k);
#pragma unroll
          for (int j = 0; j < VEC; ++j) d[j] += r[j];
        }
        if (a.dh) store_row<VEC, HF32>(d, at<HF32>(a.dh, m * K), k);
        if (a.dx) store_row<VEC, false>(d, a.dx + m * K, k);
      }
    }
  }
  if (a.part) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t k = static_cast<int64_t>(i * T + t) * VEC;
      if (k < K) store_row<VEC, true>(dw[i], a.part + static_cast<int64_t>(blockIdx.x) * K, k);
    }
  }
}

// Rows too long for registers: dw sums in shared memory (each word has one
// thread), a row's data read twice, the second time mostly from L1 and L2.
template <int VEC, bool HF32, bool WF32>
__global__ void __launch_bounds__(1024) rmsnorm_bwd_long_kernel(const NormGradArgs a) {
  __shared__ float2 slot[2][32];
  extern __shared__ float dw_sum[];
  const int64_t K = a.K, step = static_cast<int64_t>(blockDim.x) * VEC, k0 = static_cast<int64_t>(threadIdx.x) * VEC;
  if (a.part)
    for (int64_t k = k0; k < K; k += step)
#pragma unroll
      for (int j = 0; j < VEC; ++j) dw_sum[k + j] = 0.f;
  int flip = 0;
  for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x, flip ^= 1) {
    const void *h_row = at<HF32>(a.h, m * K);
    float hh = 0.f, gh = 0.f;
    for (int64_t k = k0; k < K; k += step) {
      float h[VEC], g[VEC], w[VEC];
      load_row<VEC, HF32>(h, h_row, k);
      load_row<VEC, false>(g, a.dy + m * K, k);
      load_row<VEC, WF32>(w, a.w, k);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        hh = fmaf(h[j], h[j], hh);
        gh = fmaf(w[j] * g[j], h[j], gh);
      }
    }
    const Sums s = block_sums(hh, gh, slot[flip]);
    const float rstd = inv_rms(s.hh, K, a.eps);
    const float c = s.wdyh / static_cast<float>(K) * rstd * rstd;
    for (int64_t k = k0; k < K; k += step) {
      float h[VEC], g[VEC], w[VEC], d[VEC];
      load_row<VEC, HF32>(h, h_row, k);
      load_row<VEC, false>(g, a.dy + m * K, k);
      load_row<VEC, WF32>(w, a.w, k);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        if (a.part) dw_sum[k + j] = fmaf(g[j], h[j] * rstd, dw_sum[k + j]);
        d[j] = rstd * (w[j] * g[j] - h[j] * c);
      }
      if (a.dr) {
        float r[VEC];
        load_row<VEC, HF32>(r, at<HF32>(a.dr, m * K), k);
#pragma unroll
        for (int j = 0; j < VEC; ++j) d[j] += r[j];
      }
      if (a.dh) store_row<VEC, HF32>(d, at<HF32>(a.dh, m * K), k);
      if (a.dx) store_row<VEC, false>(d, a.dx + m * K, k);
    }
  }
  if (a.part)
    for (int64_t k = k0; k < K; k += step)
#pragma unroll
      for (int j = 0; j < VEC; ++j) a.part[static_cast<int64_t>(blockIdx.x) * K + k + j] = dw_sum[k + j];
}

// dw[k] = the sum of the blocks' partials: 32 columns a block, 32 threads a
// column, each adding every 32nd partial, then a fixed tree.
__global__ void __launch_bounds__(1024)
    rmsnorm_dw_kernel(const float *__restrict__ part, int rows, int64_t K, float *__restrict__ dw) {
  __shared__ float s[32][33];
  const int c = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int64_t k = static_cast<int64_t>(blockIdx.x) * 32 + c;
  float v = 0.f;
  if (k < K)
    for (int i = g; i < rows; i += 32) v += part[static_cast<int64_t>(i) * K + k];
  s[g][c] = v;
  __syncthreads();
  v = warp_sum(s[c][g]);
  const int64_t ko = static_cast<int64_t>(blockIdx.x) * 32 + g;
  if (c == 0 && ko < K) dw[ko] = v;
}

int round32(int64_t t) { return static_cast<int>((t + 31) / 32 * 32); }

template <int VEC, int NV, bool WARP>
cudaError_t fwd_nv(const NormArgs &a, bool hf, bool wf, int threads, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>(WARP ? (a.M + threads / 32 - 1) / (threads / 32) : a.M));
  if (hf && wf) rmsnorm_fwd_kernel<VEC, NV, WARP, true, true><<<grid, threads, 0, st>>>(a);
  else if (hf) rmsnorm_fwd_kernel<VEC, NV, WARP, true, false><<<grid, threads, 0, st>>>(a);
  else if (wf) rmsnorm_fwd_kernel<VEC, NV, WARP, false, true><<<grid, threads, 0, st>>>(a);
  else rmsnorm_fwd_kernel<VEC, NV, WARP, false, false><<<grid, threads, 0, st>>>(a);
  return cudaGetLastError();
}

template <int VEC, int NV>
cudaError_t bwd_nv(const NormGradArgs &a, bool hf, bool wf, unsigned grid, int threads, cudaStream_t st) {
  if (hf && wf) rmsnorm_bwd_kernel<VEC, NV, true, true><<<grid, threads, 0, st>>>(a);
  else if (hf) rmsnorm_bwd_kernel<VEC, NV, true, false><<<grid, threads, 0, st>>>(a);
  else if (wf) rmsnorm_bwd_kernel<VEC, NV, false, true><<<grid, threads, 0, st>>>(a);
  else rmsnorm_bwd_kernel<VEC, NV, false, false><<<grid, threads, 0, st>>>(a);
  return cudaGetLastError();
}

template <int VEC, bool HF32, bool WF32>
cudaError_t bwd_long_one(const NormGradArgs &a, unsigned grid, cudaStream_t st) {
  const int smem = a.part ? static_cast<int>(a.K * 4) : 0;
  const cudaError_t e = cudaFuncSetAttribute(rmsnorm_bwd_long_kernel<VEC, HF32, WF32>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  rmsnorm_bwd_long_kernel<VEC, HF32, WF32><<<grid, 1024, smem, st>>>(a);
  return cudaGetLastError();
}
template <int VEC>
cudaError_t bwd_long(const NormGradArgs &a, bool hf, bool wf, unsigned grid, cudaStream_t st) {
  if (hf) return wf ? bwd_long_one<VEC, true, true>(a, grid, st) : bwd_long_one<VEC, true, false>(a, grid, st);
  return wf ? bwd_long_one<VEC, false, true>(a, grid, st) : bwd_long_one<VEC, false, false>(a, grid, st);
}

// Blocks of the backward: at most two a SM, and no more than there are rows.
unsigned bwd_blocks(int64_t M) {
  const int64_t most = 2 * static_cast<int64_t>(device_sm_count());
  return static_cast<unsigned>(M < most ? M : most);
}

}  // namespace

cudaError_t launch_rmsnorm_fwd(const uint16_t *X, const void *R, bool hf, const void *w, bool wf, float eps, int64_t M,
                               int64_t K, void *H, uint16_t *Y, int8_t *codes, float *scale, cudaStream_t st) {
  const NormArgs a{X, R, w, eps, M, K, H, Y, codes, scale};
  if (K % 8 == 0) {
    const int64_t v = K / 8;
    if (v <= 32) return fwd_nv<8, 1, true>(a, hf, wf, 128, st);
    if (v <= 1024 && M <= 2 * device_sm_count()) return fwd_nv<8, 1, false>(a, hf, wf, round32(v), st);
    if (v <= 64) return fwd_nv<8, 2, true>(a, hf, wf, 128, st);
    if (v <= 2048) return fwd_nv<8, 2, false>(a, hf, wf, round32((v + 1) / 2), st);
    return fwd_nv<8, 4, false>(a, hf, wf, round32((v + 3) / 4), st);
  }
  if (K <= 128) return fwd_nv<1, 4, true>(a, hf, wf, 128, st);
  if (K <= 8192) return fwd_nv<1, 8, false>(a, hf, wf, round32((K + 7) / 8), st);
  return fwd_nv<1, 32, false>(a, hf, wf, round32((K + 31) / 32), st);
}

size_t rmsnorm_bwd_ws_bytes(int64_t M, int64_t K) { return static_cast<size_t>(bwd_blocks(M)) * K * 4; }

cudaError_t launch_rmsnorm_bwd(const uint16_t *dY, const void *H, bool hf, const void *w, bool wf, float eps,
                               const void *dR, int64_t M, int64_t K, void *dH, uint16_t *dX, float *dW, void *ws,
                               cudaStream_t st) {
  const unsigned grid = bwd_blocks(M);
  const NormGradArgs a{dY, H, w, eps, dR, M, K, dH, dX, dW ? static_cast<float *>(ws) : nullptr};
  cudaError_t e;
  if (K % 8 == 0) {
    const int64_t v = K / 8;
    if (v <= 1024) e = bwd_nv<8, 1>(a, hf, wf, grid, round32(v), st);
    else e = bwd_long<8>(a, hf, wf, grid, st);
  } else if (K <= 8192) {
    e = bwd_nv<1, 8>(a, hf, wf, grid, round32((K + 7) / 8), st);
  } else {
    e = bwd_long<1>(a, hf, wf, grid, st);
  }
  if (e != cudaSuccess || !dW) return e;
  rmsnorm_dw_kernel<<<static_cast<unsigned>((K + 31) / 32), 1024, 0, st>>>(a.part, static_cast<int>(grid), K, dW);
  return cudaGetLastError();
}

}  // namespace qlora
