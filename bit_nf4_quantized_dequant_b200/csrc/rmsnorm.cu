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
  float eps, inv_k;   // inv_k: 1 / K
  int64_t M, K;
  void *h;
  uint16_t *y;
  int8_t *codes;
  float *scale;
};

__device__ __forceinline__ float inv_rms(float sum, float inv_k, float eps) { return rsqrtf(fmaf(sum, inv_k, eps)); }

// A row per warp (WARP) or per block; vector i * T + t belongs to thread t. What
// bounds it is memory: 4096 x 4096 bf16 takes 21.5 us, 134 MB at 6.2 TB/s (95% of
// a copy's rate), with an fp32 stream 31.2 us (99%). The int8 rows of a bf16
// stream, 4096 x 4096 25.8 us for 18.0, are held by instructions (61% of the issue
// slots); with an fp32 stream 30.2 us for 28.2. Off phase the weights come element
// by element, which makes the L1 the busiest unit (46%; issue 33%) and the waits
// for it long; three blocks a SM hide some: 1001 x 5127 bf16 11.6 us, with two
// 13.2; with an fp32 stream and bf16 output 15.3 us, int8 output 16.3.
template <int NV, bool WARP, bool ALIGNED, bool HF32, bool WF32>
__global__ void __launch_bounds__(row_threads(NV, WARP), WARP ? 8 : (NV == 2 ? (ALIGNED ? 2 : 3) : 1))
    rmsnorm_fwd_kernel(const NormArgs a) {
  grid_dep_wait();
  grid_dep_launch();
  __shared__ float slot_sum[32];
  __shared__ uint32_t slot_max[32];
  const int T = WARP ? 32 : blockDim.x;
  const int t = WARP ? (threadIdx.x & 31) : threadIdx.x;
  const int64_t m = WARP ? static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
  if (WARP && m >= a.M) return;
  const int K = static_cast<int>(a.K);
  const int64_t base = m * K;
  const int e0 = t * 8 - (ALIGNED ? 0 : static_cast<int>(base & 7));
  f2 f[NV][4], w[NV][4];
  {
    Vec8<false> x[NV];
    Vec8<HF32> r[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (a.x) x[i].template load<ALIGNED>(a.x + base, e0 + i * T * 8, K);
      if (a.r) r[i].template load<ALIGNED>(row_at<HF32>(a.r, base), e0 + i * T * 8, K);
    }
    if constexpr (NV <= 2 && ALIGNED) {   // the weights too are on their way before the row's sum
#pragma unroll
      for (int i = 0; i < NV; ++i) load_cols<ALIGNED, WF32>(w[i], a.w, e0 + i * T * 8, K);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (a.x && a.r) {
        f2 xv[4];
        x[i].get(xv);
        r[i].get(f[i]);
#pragma unroll
        for (int j = 0; j < 4; ++j) f[i][j] = add2(f[i][j], xv[j]);
        if constexpr (!HF32) {   // as it is stored
          Vec8<false> h;
#pragma unroll
          for (int j = 0; j < 4; ++j) h.w[j] = pack_bf16x2(lo2(f[i][j]), hi2(f[i][j]));
          h.get(f[i]);
        }
      } else if (a.x) {
        x[i].get(f[i]);
      } else {
        r[i].get(f[i]);
      }
    }
  }
  f2 sum2 = both(0.f);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (a.h) store_vec<ALIGNED, HF32>(f[i], row_at<HF32>(a.h, base), e0 + i * T * 8, K);
#pragma unroll
    for (int j = 0; j < 4; ++j) sum2 = fma2(f[i][j], f[i][j], sum2);
  }
  const float rstd = inv_rms(row_sum<WARP>(lo2(sum2) + hi2(sum2), slot_sum), a.inv_k, a.eps);
  Magnitude mag;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = e0 + i * T * 8;
    if constexpr (NV > 2 || !ALIGNED) load_cols<ALIGNED, WF32>(w[i], a.w, e, K);
#pragma unroll
    for (int j = 0; j < 4; ++j) f[i][j] = mul2(mul2(f[i][j], both(rstd)), w[i][j]);
    if (a.y) store_vec<ALIGNED, false>(f[i], a.y + base, e, K);
    if (a.codes) {
      if (ALIGNED ? e >= K : (e < 0 || e + 8 > K)) {   // 0 * rstd may be NaN: elements outside the row stay out of its maximum
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          auto in = [&](int k) { return k >= 0 && k < K; };
          f[i][j] = pair2(in(e + 2 * j) ? lo2(f[i][j]) : 0.f, in(e + 2 * j + 1) ? hi2(f[i][j]) : 0.f);
        }
      }
      mag.add(f[i]);
    }
  }
  if (!a.codes) return;
  const RowScale rs = row_scale(row_max<WARP>(mag.bits(), slot_max));
  if (t == 0) a.scale[m] = rs.s;
#pragma unroll
  for (int i = 0; i < NV; ++i) store_codes<ALIGNED>(f[i], rs, a.codes + base, e0 + i * T * 8, K);
}

struct NormGradArgs {
  const uint16_t *dy;
  const void *h;
  const void *w;
  float eps, inv_k;
  const void *dr;
  int64_t M, K;
  void *dh;
  uint16_t *dx;
  float *part;   // persistent kernel: [gridDim.x, K] partial dw
  float *rstd;   // long rows: [M], or null
};

// The row's two sums, over the threads that share it.
struct Sums {
  float hh, wdyh;
};
__device__ __forceinline__ Sums row_sums(f2 hh, f2 wdyh, float2 *slot) {
  float v = warp_sum2(lo2(hh) + hi2(hh), lo2(wdyh) + hi2(wdyh));
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  float *s = reinterpret_cast<float *>(slot);   // 32 sums hh, then 32 sums w dy h
  if ((lane & 15) == 0) s[(threadIdx.x >> 5) + 2 * (lane & 16)] = v;
  __syncthreads();
  v = warp_sum2(lane < warps ? s[lane] : 0.f, lane < warps ? s[32 + lane] : 0.f);
  return {__shfl_sync(0xffffffffu, v, 0), __shfl_sync(0xffffffffu, v, 16)};
}
// One row's share of the sums; and what both kernels make of them: rstd, and
// rstd^2 mean(w dy h).
__device__ __forceinline__ void add_sums(const f2 (&h)[4], const f2 (&g)[4], const f2 (&w)[4], f2 &hh, f2 &gh) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    hh = fma2(h[j], h[j], hh);
    gh = fma2(mul2(w[j], g[j]), h[j], gh);
  }
}

// dh of a vector and its stores; c = rstd^2 mean(w dy h).
template <bool ALIGNED, bool HF32>
__device__ __forceinline__ void store_dh(const NormGradArgs &a, int64_t base, int e, int K, const f2 (&h)[4],
                                         const f2 (&g)[4], const f2 (&w)[4], const f2 (&r)[4], float rstd, float c) {
  f2 d[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) d[j] = fma2(both(rstd), fma2(h[j], both(-c), mul2(w[j], g[j])), r[j]);
  if (a.dh) store_vec<ALIGNED, HF32>(d, row_at<HF32>(a.dh, base), e, K);
  if (a.dx) store_vec<ALIGNED, false>(d, a.dx + base, e, K);
}

// Persistent blocks, a row at a time: a thread keeps its columns' weight and dw
// sums in registers and copies its own elements of the next kDepth - 1 rows to
// shared memory ahead of time (nobody else reads them, so there is no barrier
// but the two of the row's sums). What bounds it is the bytes in flight: one
// row ahead in registers instead made 4096 x 4096 bf16 33.4 us, two in shared
// memory 31.0 (26.8 with the arithmetic in pairs; 134 MB, 5.0 TB/s).
// Two slots for the sums: a block barrier lies between a slot's reads and its
// next write. Where K is no multiple of 8 the blocks' count is (or each has one
// row), so that all rows of a block have the same phase; a row's first vector
// may then begin in the row before (read, and dropped), its last one is cut.
// Shared memory of a thread's vector of one row: h, dr and dy.
constexpr int vec_bytes(bool hf32) { return hf32 ? 80 : 48; }

template <int kDepth, int NV, bool ALIGNED, bool HF32, bool WF32>
__global__ void __launch_bounds__(NV == 1 ? 512 : 1024, NV == 1 ? 2 : 1) rmsnorm_bwd_kernel(const NormGradArgs a) {
  grid_dep_wait();
  grid_dep_launch();
  __shared__ float2 slot[2][32];
  extern __shared__ __align__(16) uint8_t ring[];   // [depth][NV][16-byte part][thread]
  constexpr int kH = HF32 ? 2 : 1, kParts = 2 * kH + 1;   // parts: h, dr, dy
  const int T = blockDim.x, t = threadIdx.x;
  const int K = static_cast<int>(a.K);
  const int e0 = t * 8 - (ALIGNED ? 0 : static_cast<int>((static_cast<int64_t>(blockIdx.x) * K) & 7));
  f2 w[NV][4], dw[NV][4];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    load_cols<ALIGNED, WF32>(w[i], a.w, e0 + i * T * 8, K);
#pragma unroll
    for (int j = 0; j < 4; ++j) dw[i][j] = both(0.f);
  }
  auto part = [&](int d, int i, int q) -> uint8_t * { return ring + (((d * NV + i) * kParts + q) * T + t) * 16; };
  auto fetch = [&](int64_t m, int d) {
    if (m < a.M) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int e = e0 + i * T * 8;
        if (e < K) {
          const uint8_t *h = static_cast<const uint8_t *>(row_at<HF32>(a.h, m * K + e));
          const uint8_t *r = static_cast<const uint8_t *>(row_at<HF32>(a.dr, m * K + e));
          // bytes of part q of a vector of `size`-byte elements that lie before the row's end
          auto bytes = [&](int size, int q) { return ALIGNED ? 16 : min(max((K - e) * size - 16 * q, 0), 16); };
#pragma unroll
          for (int q = 0; q < kH; ++q) {
            const int n = bytes(HF32 ? 4 : 2, q);
            copy16<HF32, !ALIGNED>(smem_u32(part(d, i, q)), h + 16 * q, n);
            if (a.dr) copy16<HF32, !ALIGNED>(smem_u32(part(d, i, kH + q)), r + 16 * q, n);
          }
          copy16<false, !ALIGNED>(smem_u32(part(d, i, 2 * kH)), a.dy + m * K + e, bytes(2, 0));
        }
      }
    }
    copy_commit();   // a group a row, empty past the last
  };
  auto read = [&](int d, int i, int q, auto &v) {
    constexpr int n = sizeof(v.w) / 16;
#pragma unroll
    for (int j = 0; j < n; ++j) {
      const uint4 u = *reinterpret_cast<const uint4 *>(part(d, i, q + j));
      v.w[4 * j] = u.x; v.w[4 * j + 1] = u.y; v.w[4 * j + 2] = u.z; v.w[4 * j + 3] = u.w;
    }
  };
  // h and dy of a vector; what its first one holds of the row before becomes zero
  auto rows_of = [&](int d, int i, f2 (&hv)[4], f2 (&gv)[4]) {
    Vec8<HF32> h;
    Vec8<false> g;
    read(d, i, 0, h);
    read(d, i, 2 * kH, g);
    h.get(hv);
    g.get(gv);
    if (!ALIGNED && i == 0 && e0 < 0) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        hv[j] = pair2(e0 + 2 * j < 0 ? 0.f : lo2(hv[j]), e0 + 2 * j + 1 < 0 ? 0.f : hi2(hv[j]));
        gv[j] = pair2(e0 + 2 * j < 0 ? 0.f : lo2(gv[j]), e0 + 2 * j + 1 < 0 ? 0.f : hi2(gv[j]));
      }
    }
  };
  int64_t m = blockIdx.x;
#pragma unroll
  for (int d = 0; d < kDepth - 1; ++d) fetch(m + static_cast<int64_t>(d) * gridDim.x, d);
  int flip = 0, d = 0;
  for (; m < a.M; m += gridDim.x, flip ^= 1, d = d + 1 == kDepth ? 0 : d + 1) {
    fetch(m + static_cast<int64_t>(kDepth - 1) * gridDim.x, d == 0 ? kDepth - 1 : d - 1);
    copy_wait<kDepth - 1>();
    f2 hh = both(0.f), gh = both(0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (e0 + i * T * 8 < K) {
        f2 hv[4], gv[4];
        rows_of(d, i, hv, gv);
        add_sums(hv, gv, w[i], hh, gh);
      }
    }
    const Sums s = row_sums(hh, gh, slot[flip]);
    const float rstd = inv_rms(s.hh, a.inv_k, a.eps);
    const float c = s.wdyh * a.inv_k * rstd * rstd;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = e0 + i * T * 8;
      if (e < K) {
        Vec8<HF32> r;
        f2 hv[4], gv[4], rv[4] = {};
        rows_of(d, i, hv, gv);
        if (a.dr) {
          read(d, i, kH, r);
          r.get(rv);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) dw[i][j] = fma2(gv[j], mul2(hv[j], both(rstd)), dw[i][j]);
        store_dh<ALIGNED, HF32>(a, m * K, e, K, hv, gv, w[i], rv, rstd, c);
      }
    }
  }
  copy_wait<0>();
  if (!a.part) return;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = e0 + i * T * 8;
    float *row = a.part + static_cast<int64_t>(blockIdx.x) * K;
    if constexpr (ALIGNED) {
      store_vec<true, true>(dw[i], row, e, K);
    } else {   // the partials' rows have phases of their own
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (e + j >= 0 && e + j < K) row[e + j] = j & 1 ? hi2(dw[i][j >> 1]) : lo2(dw[i][j >> 1]);
    }
  }
}

// Rows too long for that: a block each, read twice, the second time mostly from
// L2. The weight's gradient, if any, is left to rmsnorm_dw_rows_kernel, for which
// the row's rstd is kept (1000 x 20000 bf16: 72 us in all, 2.2 TB/s).
template <bool ALIGNED, bool HF32, bool WF32>
__global__ void __launch_bounds__(1024) rmsnorm_bwd_long_kernel(const NormGradArgs a) {
  grid_dep_wait();
  grid_dep_launch();
  __shared__ float2 slot[32];
  const int K = static_cast<int>(a.K);
  const int64_t base = static_cast<int64_t>(blockIdx.x) * K;
  const int e0 = static_cast<int>(threadIdx.x) * 8 - (ALIGNED ? 0 : static_cast<int>(base & 7));
  f2 h[4], g[4], w[4], hh = both(0.f), gh = both(0.f);
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
    add_sums(h, g, w, hh, gh);
  }
  const Sums s = row_sums(hh, gh, slot);
  const float rstd = inv_rms(s.hh, a.inv_k, a.eps);
  const float c = s.wdyh * a.inv_k * rstd * rstd;
  if (a.rstd && threadIdx.x == 0) a.rstd[blockIdx.x] = rstd;
  for (int e = e0; e < K; e += 8192) {
    f2 r[4] = {};
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
// columns (one of `strips`) and a share of the rows, its eight warps
// every eighth row of them; out is dw, or this share's row of partials.
template <int VEC, bool HF32>   // VEC: 8, or 1 where K is no multiple of 8 (a column's phase changes with the row)
__global__ void __launch_bounds__(256)
    rmsnorm_dw_rows_kernel(const uint16_t *dy, const void *h, const float *rstd, int64_t M, int64_t K, int strips,
                           float *out) {
  grid_dep_wait();
  grid_dep_launch();
  __shared__ float s[8][32 * VEC];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int strip = static_cast<int>(blockIdx.x) % strips, share = static_cast<int>(blockIdx.x) / strips;
  const int shares = static_cast<int>(gridDim.x) / strips;
  const int k = (strip * 32 + lane) * VEC;
  const int64_t m0 = M * share / shares, m1 = M * (share + 1) / shares;
  f2 dw[4] = {};
  if (k < K) {
#pragma unroll 8
    for (int64_t m = m0 + warp; m < m1; m += 8) {
      const float rs = rstd[m];
      if constexpr (VEC == 8) {
        f2 g[4], hv[4];
        load_cols<true, false>(g, dy + m * K, k, static_cast<int>(K));
        load_cols<true, HF32>(hv, row_at<HF32>(h, m * K), k, static_cast<int>(K));
#pragma unroll
        for (int j = 0; j < 4; ++j) dw[j] = fma2(g[j], mul2(hv[j], both(rs)), dw[j]);
      } else {
        const float hv = HF32 ? static_cast<const float *>(h)[m * K + k] : bf16_to_f32(static_cast<const uint16_t *>(h)[m * K + k]);
        dw[0] = pair2(fmaf(bf16_to_f32(dy[m * K + k]), hv * rs, lo2(dw[0])), 0.f);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < VEC; ++j) s[warp][lane * VEC + j] = j & 1 ? hi2(dw[j >> 1]) : lo2(dw[j >> 1]);
  __syncthreads();
  const int k0 = strip * 32 * VEC;
  for (int c = threadIdx.x; c < 32 * VEC && k0 + c < K; c += 256) {
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) v += s[i][c];
    out[static_cast<int64_t>(share) * K + k0 + c] = v;
  }
}

// dw[k] = the sum of the partials: COLS columns a block, 1024 / COLS threads a
// column, each adding every so many-th partial, then a fixed tree. 32 columns,
// or 8 where that would leave most SMs without a block (8192 x 1024, 1184
// partials: 19.5 us with 32, 18.4 with 8; 4096 x 4096, 296 partials: 26.8 and 29.0).
template <int COLS>
__global__ void __launch_bounds__(1024)
    rmsnorm_dw_kernel(const float *part, int rows, int64_t K, float *__restrict__ dw) {
  grid_dep_wait();
  grid_dep_launch();
  constexpr int G = 1024 / COLS;
  __shared__ float s[G][COLS + 1];
  const int c = threadIdx.x % COLS, g = threadIdx.x / COLS;
  const int64_t k = static_cast<int64_t>(blockIdx.x) * COLS + c;
  float v = 0.f;
  if (k < K)
#pragma unroll 5
    for (int i = g; i < rows; i += G) v += part[static_cast<int64_t>(i) * K + k];
  s[g][c] = v;
  __syncthreads();
  const int col = threadIdx.x >> 5, lane = threadIdx.x & 31;   // a warp a column
  if (col < COLS) {
    v = 0.f;
#pragma unroll
    for (int i = 0; i < G / 32; ++i) v += s[32 * i + lane][col];
    v = warp_sum(v);
    const int64_t ko = static_cast<int64_t>(blockIdx.x) * COLS + col;
    if (lane == 0 && ko < K) dw[ko] = v;
  }
}
cudaError_t launch_dw(const float *part, int rows, int64_t K, float *dw, cudaStream_t st) {
  if (K > 8 * device_sm_count() || rows < 128)
    return launch_dependent(rmsnorm_dw_kernel<32>, static_cast<unsigned>((K + 31) / 32), 1024, 0, st, 1, part, rows, K, dw);
  return launch_dependent(rmsnorm_dw_kernel<8>, static_cast<unsigned>((K + 7) / 8), 1024, 0, st, 1, part, rows, K, dw);
}

// A few short rows with the weight's gradient, in one launch: a block takes 128
// columns of all rows. Every block forms all rows' sums for itself (from L2),
// 32 / M warps a row, so no block waits for another and no partial sums are
// kept. Where dh or dx overwrites dy, which other blocks would still read, one
// block does it all. What it saves is the host's share: a call among others takes
// 8.6 us (two launches and a workspace 13.7), on the device alone 5.3 us for 8 x
// 4096 (3.8), 4.3 for 16 x 1024 (3.0), 4.9 for 4 x 8192 (5.2). A call waited for
// takes 19.9 us for 8 x 4096 (21.8), but 22.6 for 16 x 4096 (21.6) and 25.2 for
// 16 x 8192 (23.4): hence 32768 elements. A row's sums come in the persistent
// kernel's order (vectors warp by warp of its T threads, NV each, then the warps),
// so that a row's gradient is the same bits whatever stands beside it.
constexpr int kFewRows = 16, kFewCols = 128;
constexpr int64_t kFewElements = 32768, kFewWidth = 8192;
template <bool ALIGNED, bool HF32, bool WF32>
__global__ void __launch_bounds__(1024) rmsnorm_bwd_few_kernel(const NormGradArgs a, int T, int nv, float *dw) {
  grid_dep_wait();
  grid_dep_launch();
  __shared__ float sums[kFewRows][64];   // 32 warps' sums hh, then w dy h
  __shared__ float2 row_c[kFewRows];     // rstd, rstd^2 mean(w dy h)
  __shared__ float part[8][kFewCols];
  const int K = static_cast<int>(a.K), M = static_cast<int>(a.M);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int share = 32 / M, row = warp / share;   // a row's warps; what is left over of 32 idles
  if (row < M) {
    const int64_t base = static_cast<int64_t>(row) * K;
    const int phase = ALIGNED ? 0 : static_cast<int>(base & 7);
#pragma unroll 4
    for (int j = warp - row * share; j < T / 32; j += share) {
      f2 hh = both(0.f), gh = both(0.f);
      for (int i = 0; i < nv; ++i) {
        const int e = (i * T + j * 32 + lane) * 8 - phase;
        if (e < K) {
          Vec8<HF32> h;
          Vec8<false> g;
          f2 hv[4], gv[4], w[4];
          h.template load<ALIGNED>(row_at<HF32>(a.h, base), e, K);
          g.template load<ALIGNED>(a.dy + base, e, K);
          load_cols<ALIGNED, WF32>(w, a.w, e, K);
          h.get(hv);
          g.get(gv);
          add_sums(hv, gv, w, hh, gh);
        }
      }
      const float v = warp_sum2(lo2(hh) + hi2(hh), lo2(gh) + hi2(gh));
      if ((lane & 15) == 0) sums[row][j + 2 * (lane & 16)] = v;
    }
  }
  __syncthreads();
  if (warp < M) {
    const bool in = lane < T / 32;
    const float v = warp_sum2(in ? sums[warp][lane] : 0.f, in ? sums[warp][32 + lane] : 0.f);
    const float hh = __shfl_sync(0xffffffffu, v, 0), wdyh = __shfl_sync(0xffffffffu, v, 16);
    const float rstd = inv_rms(hh, a.inv_k, a.eps);
    if (lane == 0) row_c[warp] = make_float2(rstd, wdyh * a.inv_k * rstd * rstd);
  }
  __syncthreads();
  const int c = threadIdx.x % kFewCols;
  for (int k0 = static_cast<int>(blockIdx.x) * kFewCols; k0 < K; k0 += static_cast<int>(gridDim.x) * kFewCols) {
    const int k = k0 + c;
    float sum = 0.f;
    if (k < K) {
      const float w = WF32 ? static_cast<const float *>(a.w)[k] : bf16_to_f32(static_cast<const uint16_t *>(a.w)[k]);
      auto at = [&](const void *p, int64_t i) {
        return HF32 ? static_cast<const float *>(p)[i] : bf16_to_f32(static_cast<const uint16_t *>(p)[i]);
      };
      for (int m = threadIdx.x / kFewCols; m < M; m += 1024 / kFewCols) {
        const int64_t i = static_cast<int64_t>(m) * K + k;
        const float g = bf16_to_f32(a.dy[i]), h = at(a.h, i), rstd = row_c[m].x;
        sum = fmaf(g, h * rstd, sum);
        const float d = fmaf(rstd, fmaf(h, -row_c[m].y, w * g), a.dr ? at(a.dr, i) : 0.f);
        if (a.dh) {
          if constexpr (HF32) static_cast<float *>(a.dh)[i] = d;
          else static_cast<uint16_t *>(a.dh)[i] = static_cast<uint16_t>(pack_bf16x2(d, 0.f));
        }
        if (a.dx) a.dx[i] = static_cast<uint16_t>(pack_bf16x2(d, 0.f));
      }
    }
    part[threadIdx.x / kFewCols][c] = sum;
    __syncthreads();
    if (threadIdx.x < kFewCols && k < K) {
#pragma unroll
      for (int i = 1; i < 8; ++i) sum += part[i][c];
      dw[k] = sum;
    }
    __syncthreads();
  }
}
bool few_rows(int64_t M, int64_t K) { return M <= kFewRows && K <= kFewWidth && M * K <= kFewElements; }

// Calls go(hf, wf) with the types as types.
template <class F>
cudaError_t with_types(bool hf, bool wf, F go) {
  if (hf) return wf ? go(Num<1>{}, Num<1>{}) : go(Num<1>{}, Num<0>{});
  return wf ? go(Num<0>{}, Num<1>{}) : go(Num<0>{}, Num<0>{});
}

// The backward's shape. Persistent blocks (`parts` of them), where `depth` rows
// fit in shared memory: one vector a thread up to
// 512 threads, then two; as many blocks a SM as leave it about 1024 threads;
// three rows deep where that leaves room for two blocks (or all of them). Or
// a block a row and, for the weight's gradient, `parts` shares of the rows after it.
struct GradPlan {
  bool persistent;
  int parts, nv, threads, depth;
  size_t smem;
};
GradPlan grad_plan(int64_t M, int64_t K, bool hf) {
  const int64_t sms = device_sm_count(), v = K % 8 ? (K + 7) / 8 + 1 : K / 8;
  GradPlan g{};
  g.nv = v <= 512 ? 1 : 2;
  g.threads = static_cast<int>((v + 32 * g.nv - 1) / (32 * g.nv) * 32);
  const size_t row = static_cast<size_t>(g.nv) * g.threads * vec_bytes(hf);
  if (g.threads <= 1024 && 2 * row <= 220 * 1024) {
    auto fit = [&](int depth) { return static_cast<int64_t>(222 * 1024 / (depth * row + 1024)); };
    int64_t per_sm = 1024 / g.threads;
    per_sm = per_sm > 8 ? 8 : per_sm;
    g.depth = fit(3) >= (per_sm < 2 ? per_sm : 2) ? 3 : 2;
    if (per_sm > fit(g.depth)) per_sm = fit(g.depth);
    g.smem = g.depth * row;
    g.persistent = true;
    const int64_t most = K % 8 ? per_sm * sms / 8 * 8 : per_sm * sms;
    g.parts = static_cast<int>(M < most ? M : most);
    return g;
  }
  const int64_t cols = K % 8 ? (K + 31) / 32 : (K + 255) / 256;
  int64_t parts = (8 * sms + cols - 1) / cols, most = (M + 15) / 16;   // 16 rows a block or more
  if (parts > most) parts = most;
  g.parts = static_cast<int>(parts < 1 ? 1 : parts);
  return g;
}
size_t round16(size_t b) { return (b + 15) / 16 * 16; }

cudaError_t dw_from_rows(const NormGradArgs &a, bool hf, const GradPlan &gp, float *dW, void *ws, cudaStream_t st) {
  const int64_t M = a.M, K = a.K;
  float *part = gp.parts == 1 ? dW : reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + round16(static_cast<size_t>(M) * 4));
  const unsigned vec = K % 8 ? 1 : 8;
  const int strips = static_cast<int>((K + 32 * vec - 1) / (32 * vec));
  auto kernel = vec == 8 ? (hf ? rmsnorm_dw_rows_kernel<8, true> : rmsnorm_dw_rows_kernel<8, false>)
                         : (hf ? rmsnorm_dw_rows_kernel<1, true> : rmsnorm_dw_rows_kernel<1, false>);
  const cudaError_t e = launch_dependent(kernel, static_cast<unsigned>(strips * gp.parts), 256, 0, st, 1, a.dy, a.h,
                                         a.rstd, M, K, strips, part);
  if (e != cudaSuccess || gp.parts == 1) return e;
  return launch_dw(part, gp.parts, K, dW, st);
}

}  // namespace

cudaError_t launch_rmsnorm_fwd(const uint16_t *X, const void *R, bool hf, const void *w, bool wf, float eps, int64_t M,
                               int64_t K, void *H, uint16_t *Y, int8_t *codes, float *scale, cudaStream_t st) {
  const NormArgs a{X, R, w, eps, 1.f / static_cast<float>(K), M, K, H, Y, codes, scale};
  const RowPlan p = row_plan(M, K, device_sm_count(), 2);
  return dispatch_row(p, [&](auto nv, auto warp, auto aligned) {
    return with_types(hf, wf, [&](auto h32, auto w32) {
      return launch_dependent(rmsnorm_fwd_kernel<nv.value, warp.value, aligned.value, h32.value, w32.value>,
                              row_grid(p, M), p.threads, 0, st, 1, a);
    });
  });
}

// The caller does not say the stream's type: the larger of the two.
size_t rmsnorm_bwd_ws_bytes(int64_t M, int64_t K) {
  if (few_rows(M, K)) return 0;
  size_t most = 0;
  for (const bool hf : {false, true}) {
    const GradPlan g = grad_plan(M, K, hf);
    const size_t b = static_cast<size_t>(g.parts) * K * 4 + (g.persistent ? 0 : round16(static_cast<size_t>(M) * 4));
    most = b > most ? b : most;
  }
  return most;
}

cudaError_t launch_rmsnorm_bwd(const uint16_t *dY, const void *H, bool hf, const void *w, bool wf, float eps,
                               const void *dR, int64_t M, int64_t K, void *dH, uint16_t *dX, float *dW, void *ws,
                               cudaStream_t st) {
  NormGradArgs a{dY, H, w, eps, 1.f / static_cast<float>(K), dR, M, K, dH, dX, nullptr, nullptr};
  // dy is read by other threads than those that write dh and dx
  const bool over = dW && (static_cast<const void *>(dY) == dH || dY == dX);
  const GradPlan gp = grad_plan(M, K, hf);
  if (dW && few_rows(M, K)) {
    const unsigned blocks = over ? 1u : static_cast<unsigned>((K + kFewCols - 1) / kFewCols);
    return with_types(hf, wf, [&](auto h32, auto w32) {
      auto *kernel = K % 8 ? rmsnorm_bwd_few_kernel<false, h32.value, w32.value>
                           : rmsnorm_bwd_few_kernel<true, h32.value, w32.value>;
      return launch_dependent(kernel, blocks, 1024, 0, st, 1, a, gp.threads, gp.nv, dW);
    });
  }
  cudaError_t e;
  if (gp.persistent) {
    a.part = dW ? static_cast<float *>(ws) : nullptr;
    auto go = [&](auto kernel) {
      const cudaError_t e = allow_smem(kernel);
      if (e != cudaSuccess) return e;
      return launch_dependent(kernel, static_cast<unsigned>(gp.parts), gp.threads, gp.smem, st, 1, a);
    };
    e = with_types(hf, wf, [&](auto h32, auto w32) {
      auto with = [&](auto aligned) {
        constexpr bool al = aligned.value;
        if (gp.depth == 3)
          return gp.nv == 1 ? go(rmsnorm_bwd_kernel<3, 1, al, h32.value, w32.value>)
                            : go(rmsnorm_bwd_kernel<3, 2, al, h32.value, w32.value>);
        return gp.nv == 1 ? go(rmsnorm_bwd_kernel<2, 1, al, h32.value, w32.value>)
                          : go(rmsnorm_bwd_kernel<2, 2, al, h32.value, w32.value>);
      };
      return K % 8 ? with(Num<0>{}) : with(Num<1>{});
    });
  } else {
    if (dW) a.rstd = static_cast<float *>(ws);
    auto rows = [&](const NormGradArgs &a) {
      return with_types(hf, wf, [&](auto h32, auto w32) {
        auto *kernel = K % 8 ? rmsnorm_bwd_long_kernel<false, h32.value, w32.value>
                             : rmsnorm_bwd_long_kernel<true, h32.value, w32.value>;
        return launch_dependent(kernel, static_cast<unsigned>(M), 1024, 0, st, 1, a);
      });
    };
    // dw is formed from dy after rstd: where dh or dx overwrites dy (`over`), they wait for it
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
  return launch_dw(a.part, gp.parts, K, dW, st);
}

}  // namespace qlora
