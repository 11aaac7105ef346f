// Device helpers of the row kernels (RMS norm, int8 row codec): vector loads
// and stores of a row's elements as fp32, reductions over the threads of a
// row, and the int8 code of a value.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

#include "qlora_device.cuh"

namespace qlora {

// VEC consecutive elements (1 or 8) of a bf16 or fp32 row, as fp32. The
// 8-element forms need the address aligned to 16 bytes.
template <int VEC, bool F32>
__device__ __forceinline__ void load_row(float (&f)[VEC], const void *row, int64_t i) {
  if constexpr (F32) {
    const float *p = static_cast<const float *>(row) + i;
    if constexpr (VEC == 8) {
      const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
      f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
      f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    } else {
      f[0] = *p;
    }
  } else {
    const uint16_t *p = static_cast<const uint16_t *>(row) + i;
    if constexpr (VEC == 8) {
      const uint4 u = *reinterpret_cast<const uint4 *>(p);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        f[2 * j] = __uint_as_float(w[j] << 16);
        f[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
      }
    } else {
      f[0] = __uint_as_float(static_cast<uint32_t>(*p) << 16);
    }
  }
}

template <int VEC, bool F32>
__device__ __forceinline__ void store_row(const float (&f)[VEC], void *row, int64_t i) {
  if constexpr (F32) {
    float *p = static_cast<float *>(row) + i;
    if constexpr (VEC == 8) {
      *reinterpret_cast<float4 *>(p) = make_float4(f[0], f[1], f[2], f[3]);
      *reinterpret_cast<float4 *>(p + 4) = make_float4(f[4], f[5], f[6], f[7]);
    } else {
      *p = f[0];
    }
  } else {
    uint16_t *p = static_cast<uint16_t *>(row) + i;
    if constexpr (VEC == 8) {
      *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                                 pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
    } else {
      *p = static_cast<uint16_t>(pack_bf16x2(f[0], 0.f));
    }
  }
}

__device__ __forceinline__ float bf16_round(float x) { return __uint_as_float(pack_bf16x2(x, 0.f) << 16); }

// ---- reductions over the threads that share a row ---------------------------
// One warp, or a whole block of up to 32 warps. `slot`: 32 words of shared
// memory, not written again before every thread has passed a block barrier
// (each reduction of a row has its own slot). Every thread gets the result,
// summed in the same order.
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
template <bool WARP>
__device__ __forceinline__ float row_sum(float v, float *slot) {
  v = warp_sum(v);
  if constexpr (WARP) return v;
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  if (lane == 0) slot[threadIdx.x >> 5] = v;
  __syncthreads();
  return warp_sum(lane < warps ? slot[lane] : 0.f);
}
template <bool WARP>
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t *slot) {
  v = __reduce_max_sync(0xffffffffu, v);
  if constexpr (WARP) return v;
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  if (lane == 0) slot[threadIdx.x >> 5] = v;
  __syncthreads();
  return __reduce_max_sync(0xffffffffu, lane < warps ? slot[lane] : 0u);
}

// |v| as an ordered integer: infinities and NaN sort above every finite value,
// so one integer maximum finds the row's largest magnitude and whether the row
// holds anything that is not finite.
__device__ __forceinline__ uint32_t mag_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// The int8 code of a value, rint(fp32_rn(v / s)): v * (1 / s) is within
// 3 * 127.5 * 2^-24 < 3e-5 of the quotient, so its rounding can differ only
// next to a tie; there (about one value in five thousand) the division is
// done. Adding 1.5 * 2^23 rounds to an integer, half to even, and leaves the
// code in the low byte. |v| <= 127 s (1 + 2^-22) keeps the code within +-127
// unless s is subnormal (rounded coarsely) or its reciprocal overflows: such
// rows always divide, and clamp.
struct RowScale {
  float s, inv;
  bool zero, divide;
};
constexpr float kRoundMagic = 12582912.f;

__device__ __forceinline__ RowScale row_scale(uint32_t max_bits) {
  RowScale r;
  const bool finite = max_bits < 0x7f800000u;
  r.s = finite ? __fmul_rn(__uint_as_float(max_bits), 1.f / 127.f) : __uint_as_float(0x7fc00000u);
  r.zero = !(r.s > 0.f);   // an empty row, or one that is not finite
  r.divide = r.s < 1e-30f;
  r.inv = r.zero || r.divide ? 0.f : __frcp_rn(r.s);
  return r;
}
__device__ __forceinline__ uint32_t code_bits(float v, const RowScale &r) {
  if (r.zero) return 0u;
  if (r.divide) {
    const float q = fminf(fmaxf(rintf(__fdiv_rn(v, r.s)), -127.f), 127.f);
    return static_cast<uint32_t>(static_cast<int>(q));
  }
  float m = __fmaf_rn(v, r.inv, kRoundMagic);
  const float d = __fmaf_rn(v, r.inv, -(m - kRoundMagic));
  if (fabsf(fabsf(d) - 0.5f) < 1e-4f) m = __fadd_rn(__fdiv_rn(v, r.s), kRoundMagic);
  return __float_as_uint(m);   // the code is the low byte
}

template <int VEC>
__device__ __forceinline__ void store_codes(const float (&f)[VEC], const RowScale &r, int8_t *row, int64_t i) {
  if constexpr (VEC == 8) {
    uint32_t c[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) c[j] = code_bits(f[j], r);
    uint32_t w[2];
#pragma unroll
    for (int j = 0; j < 2; ++j)
      w[j] = prmt(prmt(c[4 * j], c[4 * j + 1], 0x0040u), prmt(c[4 * j + 2], c[4 * j + 3], 0x0040u), 0x5410u);
    *reinterpret_cast<uint2 *>(row + i) = make_uint2(w[0], w[1]);
  } else {
    row[i] = static_cast<int8_t>(code_bits(f[0], r) & 0xffu);
  }
}

}  // namespace qlora
