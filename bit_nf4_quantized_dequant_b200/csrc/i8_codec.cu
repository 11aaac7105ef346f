// Int8 rows with one fp32 scale a row: quantise and dequantise.
//
//   v = x (or fp32_rn(x * col_scale)),  s = fp32_rn(max |v| * fp32_rn(1 / 127)),
//   code = rint(fp32_rn(v / s)) clamped to +-127.
//
// Both are bound by memory (2 to 4 bytes read and 1 written an element), so a
// row is read once and kept in registers, as it was loaded, between its maximum
// and its codes. Measured: quantise 4096 x 14336 fp32 46 us (6.4 TB/s), 4096 x
// 11008 bf16 26 us (5.2 TB/s), with column scales 33 us: there the scales' loads
// from L1 and the instructions (67% of the issue slots) set the pace.
// Dequantise 4096 x 4096 9 us (5.6 TB/s).
#include "norm_i8.h"
#include "row_device.cuh"

namespace qlora {
namespace {

template <bool F32, bool COLS>
__device__ __forceinline__ void scaled(f2 (&f)[4], const Vec8<F32> &v, const f2 (&c)[4]) {
  v.get(f);
  if constexpr (COLS) {
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = mul2(f[j], c[j]);
  }
}

// A row per warp (WARP) or per block; vector i * T + t belongs to thread t. The
// row stays in registers as it was loaded (a bf16 row in half of what its fp32
// values take, so that three blocks fit a SM where two would) and is unpacked,
// and scaled by its columns (COLS), twice.
template <int NV, bool WARP, bool ALIGNED, bool F32, bool COLS>
__global__ void __launch_bounds__(row_threads(NV, WARP), WARP ? 8 : (NV == 1 || NV == 8 ? 1 : (F32 ? 2 : 3)))
    i8_quantize_kernel(const void *X, const float *col_scale, int64_t M, int K,
                       int8_t *__restrict__ codes, float *__restrict__ scale) {
  grid_dep_wait();
  grid_dep_launch();
  __shared__ uint32_t slot[32];
  const int T = WARP ? 32 : blockDim.x;
  const int t = WARP ? (threadIdx.x & 31) : threadIdx.x;
  const int64_t m = WARP ? static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
  if (WARP && m >= M) return;
  const void *row = row_at<F32>(X, m * K);
  const int e0 = t * 8 - (ALIGNED ? 0 : static_cast<int>((m * K) & 7));
  Vec8<F32> v[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) v[i].template load<ALIGNED>(row, e0 + i * T * 8, K);
  Magnitude mag;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    f2 f[4], c[4];
    if constexpr (COLS) load_cols<ALIGNED, true>(c, col_scale, e0 + i * T * 8, K);
    scaled<F32, COLS>(f, v[i], c);
    mag.add(f);
    v[i].forget();
  }
  const RowScale rs = row_scale(row_max<WARP>(mag.bits(), slot));
  if (t == 0) scale[m] = rs.s;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    f2 f[4], c[4];
    if constexpr (COLS) load_cols<ALIGNED, true>(c, col_scale, e0 + i * T * 8, K);
    scaled<F32, COLS>(f, v[i], c);
    store_codes<ALIGNED>(f, rs, codes + m * K, e0 + i * T * 8, K);
  }
}

// Rows too long for registers: read twice (the second time mostly from L2).
template <bool ALIGNED, bool F32, bool COLS>
__global__ void __launch_bounds__(1024)
    i8_quantize_long_kernel(const void *X, const float *col_scale, int64_t M, int K,
                            int8_t *__restrict__ codes, float *__restrict__ scale) {
  grid_dep_wait();
  grid_dep_launch();
  __shared__ uint32_t slot[32];
  const int64_t m = blockIdx.x;
  const void *row = row_at<F32>(X, m * K);
  const int e0 = static_cast<int>(threadIdx.x) * 8 - (ALIGNED ? 0 : static_cast<int>((m * K) & 7));
  Magnitude mag;
  for (int e = e0; e < K; e += 8192) {
    Vec8<F32> v;
    f2 f[4], c[4];
    v.template load<ALIGNED>(row, e, K);
    if constexpr (COLS) load_cols<ALIGNED, true>(c, col_scale, e, K);
    scaled<F32, COLS>(f, v, c);
    mag.add(f);
  }
  const RowScale rs = row_scale(row_max<false>(mag.bits(), slot));
  if (threadIdx.x == 0) scale[m] = rs.s;
  for (int e = e0; e < K; e += 8192) {
    Vec8<F32> v;
    f2 f[4], c[4];
    v.template load<ALIGNED>(row, e, K);
    if constexpr (COLS) load_cols<ALIGNED, true>(c, col_scale, e, K);
    scaled<F32, COLS>(f, v, c);
    store_codes<ALIGNED>(f, rs, codes + m * K, e, K);
  }
}

// A block takes 1024 vectors of 8 codes of one row.
template <bool ALIGNED>
__global__ void __launch_bounds__(256)
    i8_dequantize_rows_kernel(const int8_t *codes, const float *scale, int K, int blocks_a_row,
                              uint16_t *__restrict__ out) {
  grid_dep_wait();
  grid_dep_launch();
  const uint32_t m = blockIdx.x / static_cast<uint32_t>(blocks_a_row), b = blockIdx.x - m * static_cast<uint32_t>(blocks_a_row);
  const float s = scale[m];
  const int64_t base = static_cast<int64_t>(m) * K;
  const int e0 = static_cast<int>(b) * 8192 + static_cast<int>(threadIdx.x) * 8 - (ALIGNED ? 0 : static_cast<int>(base & 7));
  uint2 u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e = e0 + i * 2048;
    if (ALIGNED ? e < K : (e >= 0 && e + 8 <= K)) {
      u[i] = *reinterpret_cast<const uint2 *>(codes + base + e);
    } else if constexpr (!ALIGNED) {
      u[i] = make_uint2(0u, 0u);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (e + j >= 0 && e + j < K)
          (j < 4 ? u[i].x : u[i].y) |= static_cast<uint32_t>(static_cast<uint8_t>(codes[base + e + j])) << (8 * (j & 3));
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (e0 + i * 2048 < K) {
      f2 f[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        auto code = [&](int b) { return static_cast<float>(static_cast<int8_t>((b < 4 ? u[i].x : u[i].y) >> (8 * (b & 3)))); };
        f[j] = mul2(pair2(code(2 * j), code(2 * j + 1)), both(s));
      }
      store_vec<ALIGNED, false>(f, out + base, e0 + i * 2048, K);
    }
  }
}

// Short rows: vectors of 8 codes over the whole matrix as one array; a vector
// may cross into the next rows.
__global__ void __launch_bounds__(256)
    i8_dequantize_kernel(const int8_t *codes, const float *scale, int64_t M, int K,
                         uint16_t *__restrict__ out) {
  grid_dep_wait();
  grid_dep_launch();
  const int64_t total = M * K, i = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 8;
  if (i >= total) return;
  // the block's first row by one division, this vector's from there
  const int64_t m0 = static_cast<int64_t>(blockIdx.x) * 2048 / K;
  const uint32_t in = static_cast<uint32_t>(i - m0 * K);   // below K + 2048
  int64_t m = m0 + in / static_cast<uint32_t>(K), next = (m + 1) * K;   // next: the next row's first element
  float s = scale[m], f[8];
  const int n = static_cast<int>(total - i < 8 ? total - i : 8);
  uint32_t w[2] = {};
  if (n == 8) {
    const uint2 u = *reinterpret_cast<const uint2 *>(codes + i);
    w[0] = u.x;
    w[1] = u.y;
  } else {
    for (int j = 0; j < n; ++j) w[j >> 2] |= static_cast<uint32_t>(static_cast<uint8_t>(codes[i + j])) << (8 * (j & 3));
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (i + j == next && j < n) {
      s = scale[++m];
      next += K;
    }
    f[j] = __fmul_rn(static_cast<float>(static_cast<int8_t>(w[j >> 2] >> (8 * (j & 3)))), s);
  }
  const f2 v[4] = {pair2(f[0], f[1]), pair2(f[2], f[3]), pair2(f[4], f[5]), pair2(f[6], f[7])};
  store_vec<false, false>(v, out + i, 0, n);
}

}  // namespace

cudaError_t launch_i8_quantize(const void *X, bool f32, int64_t M, int64_t K, const float *cs, int8_t *codes,
                               float *scale, cudaStream_t st) {
  const RowPlan p = row_plan(M, K, device_sm_count(), 4);
  const int k = static_cast<int>(K);
  if (p.nv == 0) {
    auto run = [&](auto aligned, auto f32, auto cols) {
      return launch_dependent(i8_quantize_long_kernel<aligned.value, f32.value, cols.value>, static_cast<unsigned>(M),
                              1024, 0, st, 1, X, cs, M, k, codes, scale);
    };
    auto with = [&](auto aligned) {
      if (f32) return cs ? run(aligned, Num<1>{}, Num<1>{}) : run(aligned, Num<1>{}, Num<0>{});
      return cs ? run(aligned, Num<0>{}, Num<1>{}) : run(aligned, Num<0>{}, Num<0>{});
    };
    return p.aligned ? with(Num<1>{}) : with(Num<0>{});
  }
  return dispatch_row(p, [&](auto nv, auto warp, auto aligned) {
    if constexpr (nv.value == 2 && !warp.value) return cudaErrorInvalidValue;   // not a plan of this launch
    else {
      auto run = [&](auto f32, auto cols) {
        return launch_dependent(i8_quantize_kernel<nv.value, warp.value, aligned.value, f32.value, cols.value>,
                                row_grid(p, M), p.threads, 0, st, 1, X, cs, M, k, codes, scale);
      };
      if (f32) return cs ? run(Num<1>{}, Num<1>{}) : run(Num<1>{}, Num<0>{});
      return cs ? run(Num<0>{}, Num<1>{}) : run(Num<0>{}, Num<0>{});
    }
  });
}

cudaError_t launch_i8_dequantize(const int8_t *codes, const float *scale, int64_t M, int64_t K, uint16_t *out,
                                 cudaStream_t st) {
  const int64_t a_row = (K + (K % 8 ? 7 : 0) + 8191) / 8192;   // a row off phase may touch one vector more
  if (K >= 1024 && M * a_row < (int64_t(1) << 31)) {
    auto *kernel = K % 8 ? i8_dequantize_rows_kernel<false> : i8_dequantize_rows_kernel<true>;
    return launch_dependent(kernel, static_cast<unsigned>(M * a_row), 256, 0, st, 1, codes, scale, static_cast<int>(K),
                            static_cast<int>(a_row), out);
  }
  return launch_dependent(i8_dequantize_kernel, static_cast<unsigned>((M * K + 2047) / 2048), 256, 0, st, 1, codes, scale,
                          M, static_cast<int>(K), out);
}

}  // namespace qlora
