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

__device__ __forceinline__ float inv_rms(float sum, int64_t K, float eps) {
  return __frcp_rn(__fsqrt_rn(__fadd_rn(__fdiv_rn(sum, static_cast<float>(K)), eps)));
}

// A row per warp (WARP) or per block; vector i * T + t belongs to thread t.
template <int NV, bool WARP, bool ALIGNED, bool HF32, bool WF32>
__global__ void __launch_bounds__(row_threads(NV, WARP), WARP ? 8 : (NV == 2 ? 2 : 1)) rmsnorm_fwd_kernel(const NormArgs a) {
  __shared__ float slot_sum[32];
  __shared__ uint32_t slot_max[32];
  const int T = WARP ? 32 : blockDim.x;
  const int t = WARP ? (threadIdx.x & 31) : threadIdx.x;
  const int64_t m = WARP ? static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
  if (WARP && m >= a.M) return;
  const int K = static_cast<int>(a.K);
  const int64_t base = m * K;
  const int e0 = t * 8 - (ALIGNED ? 0 : static_cast<int>(base & 7));
  float f[NV][8];
  {
    Vec8<false> x[NV];
    Vec8<HF32> r[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (a.x) x[i].template load<ALIGNED>(a.x + base, e0 + i * T * 8, K);
      if (a.r) r[i].template load<ALIGNED>(row_at<HF32>(a.r, base), e0 + i * T * 8, K);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (a.x && a.r) {
        float xv[8];
        x[i].get(xv);
        r[i].get(f[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float h = __fadd_rn(f[i][j], xv[j]);
          f[i][j] = HF32 ? h : bf16_round(h);
        }
      } else if (a.x) {
        x[i].get(f[i]);
      } else {
        r[i].get(f[i]);
      }
    }
  }
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (a.h) store_vec<ALIGNED, HF32>(f[i], row_at<HF32>(a.h, base), e0 + i * T * 8, K);
#pragma unroll
    for (int j = 0; j < 8; ++j) sum = fmaf(f[i][j], f[i][j], sum);
  }
  const float rstd = inv_rms(row_sum<WARP>(sum, slot_sum), K, a.eps);
  float mx = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = e0 + i * T * 8;
    float w[8];
    load_cols<ALIGNED, WF32>(w, a.w, e, K);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[i][j] = __fmul_rn(__fmul_rn(f[i][j], rstd), w[j]);
    if (!ALIGNED) {   // 0 * rstd is NaN where rstd is not finite: elements outside the row stay out of its maximum
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (e + j < 0 || e + j >= K) f[i][j] = 0.f;
    } else if (e >= K) {
#pragma unroll
      for (int j = 0; j < 8; ++j) f[i][j] = 0.f;
    }
    if (a.y) store_vec<ALIGNED, false>(f[i], a.y + base, e, K);
#pragma unroll
    for (int j = 0; j < 8; ++j) mx = max_mag(mx, f[i][j]);
  }
  if (!a.codes) return;
  const RowScale rs = row_scale(row_max<WARP>(__float_as_uint(mx), slot_max));
  if (t == 0) a.scale[m] = rs.s;
#pragma unroll
  for (int i = 0; i < NV; ++i) store_codes<ALIGNED>(f[i], rs, a.codes + base, e0 + i * T * 8, K);
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
  float *part;   // persistent kernel: [gridDim.x, K] partial dw
  float *rstd;   // row kernels: [M], or null
};

// The row's two sums, over the threads that share it.
struct Sums {
  float hh, wdyh;
};
template <bool WARP>
__device__ __forceinline__ Sums row_sums(float hh, float wdyh, float2 *slot) {
  hh = warp_sum(hh);
  wdyh = warp_sum(wdyh);
  if constexpr (WARP) return {hh, wdyh};
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  if (lane == 0) slot[threadIdx.x >> 5] = make_float2(hh, wdyh);
  __syncthreads();
  const float2 v = lane < warps ? slot[lane] : make_float2(0.f, 0.f);
  return {warp_sum(v.x), warp_sum(v.y)};
}

// dh of a vector and its stores; c = rstd^2 mean(w dy h).
template <bool ALIGNED, bool HF32>
__device__ __forceinline__ void store_dh(const NormGradArgs &a, int64_t base, int e, int K, const float (&h)[8],
                                         const float (&g)[8], const float (&w)[8], const float (&r)[8], float rstd,
                                         float c) {
  float d[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) d[j] = fmaf(rstd, w[j] * g[j] - h[j] * c, r[j]);
  if (a.dh) store_vec<ALIGNED, HF32>(d, row_at<HF32>(a.dh, base), e, K);
  if (a.dx) store_vec<ALIGNED, false>(d, a.dx + base, e, K);
}

// Rows of up to 8192 elements: persistent blocks. A
// thread keeps its columns' weight and dw sums in registers, and the next row's
// loads are issued before the current row's sums, so that a block always has a
// row in flight (4096 x 4096 bf16: PREFETCH). Two slots for the sums: a block
// barrier lies between a slot's reads and its next write.
template <int NV, bool HF32, bool WF32>
__global__ void __launch_bounds__(512, NV == 1 && !HF32 ? 2 : 1) rmsnorm_bwd_kernel(const NormGradArgs a) {
  __shared__ float2 slot[2][32];
  const int T = blockDim.x, t = threadIdx.x;
  const int K = static_cast<int>(a.K);
  float w[NV][8], dw[NV][8];
  Vec8<HF32> h[NV], r[NV];
  Vec8<false> g[NV];
  auto fetch = [&](int64_t m) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int k = (i * T + t) * 8;
      if (m < a.M) {
        h[i].template load<true>(row_at<HF32>(a.h, m * K), k, K);
        g[i].template load<true>(a.dy + m * K, k, K);
        if (a.dr) r[i].template load<true>(row_at<HF32>(a.dr, m * K), k, K);
      }
    }
  };
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int k = (i * T + t) * 8;
    h[i].zero();
    g[i].zero();
    r[i].zero();
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = 0.f;
    load_cols<true, WF32>(w[i], a.w, k, K);
  }
  int64_t m = blockIdx.x;
  fetch(m);
  int flip = 0;
  for (; m < a.M; m += gridDim.x, flip ^= 1) {
    Vec8<HF32> hc[NV], rc[NV];
    Vec8<false> gc[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      hc[i] = h[i];
      gc[i] = g[i];
      rc[i] = r[i];
    }
    fetch(m + gridDim.x);
    float hh = 0.f, gh = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float hv[8], gv[8];
      hc[i].get(hv);
      gc[i].get(gv);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        hh = fmaf(hv[j], hv[j], hh);
        gh = fmaf(w[i][j] * gv[j], hv[j], gh);
      }
    }
    const Sums s = row_sums<false>(hh, gh, slot[flip]);
    const float rstd = inv_rms(s.hh, K, a.eps);
    const float c = s.wdyh / static_cast<float>(K) * rstd * rstd;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int k = (i * T + t) * 8;
      float hv[8], gv[8], rv[8];
      hc[i].get(hv);
      gc[i].get(gv);
      rc[i].get(rv);
#pragma unroll
      for (int j = 0; j < 8; ++j) dw[i][j] = fmaf(gv[j], hv[j] * rstd, dw[i][j]);
      store_dh<true, HF32>(a, m * K, k, K, hv, gv, w[i], rv, rstd, c);
    }
  }
  if (!a.part) return;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int k = (i * T + t) * 8;
    store_vec<true, true>(dw[i], a.part + static_cast<int64_t>(blockIdx.x) * K, k, K);
  }
}

// A row per warp or block, as the forward; the weight's gradient, if any, is
// left to rmsnorm_dw_rows_kernel, for which the row's rstd is kept.
template <int NV, bool WARP, bool ALIGNED, bool HF32, bool WF32>
__global__ void __launch_bounds__(row_threads(NV, WARP)) rmsnorm_bwd_rows_kernel(const NormGradArgs a) {
  __shared__ float2 slot[32];
  const int T = WARP ? 32 : blockDim.x;
  const int t = WARP ? (threadIdx.x & 31) : threadIdx.x;
  const int64_t m = WARP ? static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
  if (WARP && m >= a.M) return;
  const int K = static_cast<int>(a.K);
  const int64_t base = m * K;
  const int e0 = t * 8 - (ALIGNED ? 0 : static_cast<int>(base & 7));
  Vec8<HF32> h[NV];
  Vec8<false> g[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    h[i].template load<ALIGNED>(row_at<HF32>(a.h, base), e0 + i * T * 8, K);
    g[i].template load<ALIGNED>(a.dy + base, e0 + i * T * 8, K);
  }
  float hh = 0.f, gh = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float hv[8], gv[8], w[8];
    load_cols<ALIGNED, WF32>(w, a.w, e0 + i * T * 8, K);
    h[i].get(hv);
    g[i].get(gv);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      hh = fmaf(hv[j], hv[j], hh);
      gh = fmaf(w[j] * gv[j], hv[j], gh);
    }
  }
  const Sums s = row_sums<WARP>(hh, gh, slot);
  const float rstd = inv_rms(s.hh, K, a.eps);
  const float c = s.wdyh / static_cast<float>(K) * rstd * rstd;
  if (a.rstd && t == 0) a.rstd[m] = rstd;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = e0 + i * T * 8;
    float hv[8], gv[8], w[8], r[8] = {};
    load_cols<ALIGNED, WF32>(w, a.w, e, K);
    if (a.dr) {
      Vec8<HF32> v;
      v.template load<ALIGNED>(row_at<HF32>(a.dr, base), e, K);
      v.get(r);
    }
    h[i].get(hv);
    g[i].get(gv);
    store_dh<ALIGNED, HF32>(a, base, e, K, hv, gv, w, r, rstd, c);
  }
}

// Rows too long for registers: read twice, the second time mostly from L2.
template <bool ALIGNED, bool HF32, bool WF32>
__global__ void __launch_bounds__(1024) rmsnorm_bwd_long_kernel(const NormGradArgs a) {
  __shared__ float2 slot[32];
  const int K = static_cast<int>(a.K);
  const int64_t base = static_cast<int64_t>(blockIdx.x) * K;
  const int e0 = static_cast<int>(threadIdx.x) * 8 - (ALIGNED ? 0 : static_cast<int>(base & 7));
  float h[8], g[8], w[8], hh = 0.f, gh = 0.f;
  auto load = [&](int e) {
    Vec8<HF32> hv;
    Vec8<false> gv;
    hv.template load<ALIGNED>(row_at<HF32>(a.h, base), e, K);
    gv.template load<ALIGNED>(a.dy + base, e, K);
    load_cols<ALIGNED, WF32>(w, a.w, e, K);
    hv.get(h);
    gv.get(g);
  };
  for (int e = e0; e < K; e += 8192) {
    load(e);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      hh = fmaf(h[j], h[j], hh);
      gh = fmaf(w[j] * g[j], h[j], gh);
    }
  }
  const Sums s = row_sums<false>(hh, gh, slot);
  const float rstd = inv_rms(s.hh, K, a.eps);
  const float c = s.wdyh / static_cast<float>(K) * rstd * rstd;
  if (a.rstd && threadIdx.x == 0) a.rstd[blockIdx.x] = rstd;
  for (int e = e0; e < K; e += 8192) {
    float r[8] = {};
    load(e);
    if (a.dr) {
      Vec8<HF32> v;
      v.template load<ALIGNED>(row_at<HF32>(a.dr, base), e, K);
      v.get(r);
    }
    store_dh<ALIGNED, HF32>(a, base, e, K, h, g, w, r, rstd, c);
  }
}

// dw from the rows themselves, after a row kernel: a block takes 32 vectors of
// columns and a share of the rows (blockIdx.y of gridDim.y), its eight warps
// every eighth row of them; out is dw, or this share's row of partials.
template <int VEC, bool HF32>   // VEC: 8, or 1 where K is no multiple of 8 (a column's phase changes with the row)
__global__ void __launch_bounds__(256)
    rmsnorm_dw_rows_kernel(const uint16_t *dy, const void *h, const float *rstd, int64_t M, int64_t K, float *out) {
  __shared__ float s[8][32 * VEC];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int k = (static_cast<int>(blockIdx.x) * 32 + lane) * VEC;
  const int64_t m0 = M * blockIdx.y / gridDim.y, m1 = M * (blockIdx.y + 1) / gridDim.y;
  float dw[VEC];
#pragma unroll
  for (int j = 0; j < VEC; ++j) dw[j] = 0.f;
  if (k < K) {
#pragma unroll 4
    for (int64_t m = m0 + warp; m < m1; m += 8) {
      float g[VEC], hv[VEC];
      if constexpr (VEC == 8) {
        load_cols<true, false>(g, dy + m * K, k, static_cast<int>(K));
        load_cols<true, HF32>(hv, row_at<HF32>(h, m * K), k, static_cast<int>(K));
      } else {
        g[0] = bf16_to_f32(dy[m * K + k]);
        hv[0] = HF32 ? static_cast<const float *>(h)[m * K + k] : bf16_to_f32(static_cast<const uint16_t *>(h)[m * K + k]);
      }
      const float rs = rstd[m];
#pragma unroll
      for (int j = 0; j < VEC; ++j) dw[j] = fmaf(g[j], hv[j] * rs, dw[j]);
    }
  }
#pragma unroll
  for (int j = 0; j < VEC; ++j) s[warp][lane * VEC + j] = dw[j];
  __syncthreads();
  const int k0 = static_cast<int>(blockIdx.x) * 32 * VEC;
  for (int c = threadIdx.x; c < 32 * VEC && k0 + c < K; c += 256) {
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) v += s[i][c];
    out[static_cast<int64_t>(blockIdx.y) * K + k0 + c] = v;
  }
}

// dw[k] = the sum of the partials: 32 columns a block, 32 threads a column,
// each adding every 32nd partial, then a fixed tree.
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

// Calls go(hf, wf) with the types as types.
template <class F>
cudaError_t with_types(bool hf, bool wf, F go) {
  if (hf) return wf ? go(Num<1>{}, Num<1>{}) : go(Num<1>{}, Num<0>{});
  return wf ? go(Num<0>{}, Num<1>{}) : go(Num<0>{}, Num<0>{});
}

// The backward's shape: persistent blocks (their count), or a row kernel and,
// for the weight's gradient, shares of the rows after it.
struct GradPlan {
  bool persistent;
  int parts;
};
GradPlan grad_plan(int64_t M, int64_t K) {
  const int64_t sms = device_sm_count();
  if (K % 8 == 0 && K <= 8192) {
    const int64_t threads = (K / 8 + 31) / 32 * 32;
    int64_t per_sm = 1024 / threads;   // blocks a SM
    per_sm = per_sm < 2 ? 2 : (per_sm > 8 ? 8 : per_sm);
    return {true, static_cast<int>(M < per_sm * sms ? M : per_sm * sms)};
  }
  const int64_t cols = K % 8 ? (K + 31) / 32 : (K + 255) / 256;
  int64_t parts = (4 * sms + cols - 1) / cols, most = (M + 31) / 32;   // 32 rows a block or more
  if (parts > most) parts = most;
  return {false, static_cast<int>(parts < 1 ? 1 : parts)};
}
size_t round16(size_t b) { return (b + 15) / 16 * 16; }

cudaError_t dw_from_rows(const NormGradArgs &a, bool hf, const GradPlan &gp, float *dW, void *ws, cudaStream_t st) {
  const int64_t M = a.M, K = a.K;
  float *part = gp.parts == 1 ? dW : reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + round16(static_cast<size_t>(M) * 4));
  const unsigned vec = K % 8 ? 1 : 8;
  const dim3 grid(static_cast<unsigned>((K + 32 * vec - 1) / (32 * vec)), static_cast<unsigned>(gp.parts));
  if (vec == 8 && hf) rmsnorm_dw_rows_kernel<8, true><<<grid, 256, 0, st>>>(a.dy, a.h, a.rstd, M, K, part);
  else if (vec == 8) rmsnorm_dw_rows_kernel<8, false><<<grid, 256, 0, st>>>(a.dy, a.h, a.rstd, M, K, part);
  else if (hf) rmsnorm_dw_rows_kernel<1, true><<<grid, 256, 0, st>>>(a.dy, a.h, a.rstd, M, K, part);
  else rmsnorm_dw_rows_kernel<1, false><<<grid, 256, 0, st>>>(a.dy, a.h, a.rstd, M, K, part);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || gp.parts == 1) return e;
  rmsnorm_dw_kernel<<<static_cast<unsigned>((K + 31) / 32), 1024, 0, st>>>(part, gp.parts, K, dW);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rmsnorm_fwd(const uint16_t *X, const void *R, bool hf, const void *w, bool wf, float eps, int64_t M,
                               int64_t K, void *H, uint16_t *Y, int8_t *codes, float *scale, cudaStream_t st) {
  const NormArgs a{X, R, w, eps, M, K, H, Y, codes, scale};
  const RowPlan p = row_plan(M, K, device_sm_count(), 2);
  return dispatch_row(p, [&](auto nv, auto warp, auto aligned) {
    return with_types(hf, wf, [&](auto h32, auto w32) {
      rmsnorm_fwd_kernel<nv.value, warp.value, aligned.value, h32.value, w32.value>
          <<<row_grid(p, M), p.threads, 0, st>>>(a);
      return cudaGetLastError();
    });
  });
}

size_t rmsnorm_bwd_ws_bytes(int64_t M, int64_t K) {
  const GradPlan g = grad_plan(M, K);
  const size_t part = static_cast<size_t>(g.parts) * K * 4;
  return g.persistent ? part : round16(static_cast<size_t>(M) * 4) + part;
}

cudaError_t launch_rmsnorm_bwd(const uint16_t *dY, const void *H, bool hf, const void *w, bool wf, float eps,
                               const void *dR, int64_t M, int64_t K, void *dH, uint16_t *dX, float *dW, void *ws,
                               cudaStream_t st) {
  NormGradArgs a{dY, H, w, eps, dR, M, K, dH, dX, nullptr, nullptr};
  const GradPlan gp = grad_plan(M, K);
  cudaError_t e;
  if (gp.persistent) {
    a.part = dW ? static_cast<float *>(ws) : nullptr;
    const int64_t v = K / 8;
    const int nv = v <= 512 ? 1 : 2, threads = static_cast<int>((v + 32 * nv - 1) / (32 * nv) * 32);
    e = with_types(hf, wf, [&](auto h32, auto w32) {
      if (nv == 1) rmsnorm_bwd_kernel<1, h32.value, w32.value><<<gp.parts, threads, 0, st>>>(a);
      else rmsnorm_bwd_kernel<2, h32.value, w32.value><<<gp.parts, threads, 0, st>>>(a);
      return cudaGetLastError();
    });
  } else {
    if (dW) a.rstd = static_cast<float *>(ws);
    const RowPlan p = row_plan(M, K, device_sm_count(), 2);
    auto rows = [&](const NormGradArgs &a) {
      return with_types(hf, wf, [&](auto h32, auto w32) {
        if (p.nv == 8) {   // a row's h and dy together do not fit in registers
          const unsigned grid = static_cast<unsigned>(M);
          if (p.aligned) rmsnorm_bwd_long_kernel<true, h32.value, w32.value><<<grid, 1024, 0, st>>>(a);
          else rmsnorm_bwd_long_kernel<false, h32.value, w32.value><<<grid, 1024, 0, st>>>(a);
          return cudaGetLastError();
        }
        return dispatch_row(p, [&](auto nv, auto warp, auto aligned) {
          if constexpr (nv.value < 8)
            rmsnorm_bwd_rows_kernel<nv.value, warp.value, aligned.value, h32.value, w32.value>
                <<<row_grid(p, M), p.threads, 0, st>>>(a);
          return cudaGetLastError();
        });
      });
    };
    // dw is formed from dy after rstd: where dh or dx overwrites dy, they wait for it
    const bool over = dW && (static_cast<const void *>(dY) == dH || dY == dX);
    NormGradArgs first = a;
    if (over) first.dh = first.dx = nullptr;
    e = rows(first);
    if (e == cudaSuccess && dW) e = dw_from_rows(a, hf, gp, dW, ws, st);
    if (e == cudaSuccess && over) {
      a.rstd = nullptr;
      e = rows(a);
    }
    return e;
  }
  if (e != cudaSuccess || !dW) return e;
  rmsnorm_dw_kernel<<<static_cast<unsigned>((K + 31) / 32), 1024, 0, st>>>(a.part, gp.parts, K, dW);
  return cudaGetLastError();
}

}  // namespace qlora
