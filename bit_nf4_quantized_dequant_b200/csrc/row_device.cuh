// Device helpers of the row kernels (RMS norm, int8 row codec): a row's elements
// in vectors of eight, reductions over the threads of a row, the int8 code of a
// value, and how threads share a row.
//
// All matrices of a call have the same shape [M, K], so their rows start at the
// same phase (m K mod 8) of eight-element groups, and such a group is aligned
// for a 16-byte access in each of them whatever K is (32 bytes of fp32, 16 of
// bf16, 8 of codes). A row's vectors are those groups: vector i of a row of
// phase p covers its elements 8 i - p .. 8 i - p + 7; where K is a multiple of 8
// the phase is always 0, else a row's first and last vector may be partial and
// are read and written element by element. Only the per-column vectors (weight,
// column scales) are then out of phase, and come element by element from L1.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

#include "qlora_device.cuh"

namespace qlora {

__device__ __forceinline__ float bf16_to_f32(uint16_t b) { return __uint_as_float(static_cast<uint32_t>(b) << 16); }

// Two fp32 values in one 64-bit register: sm_100 multiplies and adds such pairs
// in one instruction, each half rounded as the scalar operation would. These
// kernels are as much bound by instructions as by memory (the norm's gradient
// with scalar operations: 50 instructions an element, 77% of the issue slots).
using f2 = unsigned long long;
__device__ __forceinline__ f2 pair2(float lo, float hi) {
  f2 d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ f2 both(float v) { return pair2(v, v); }
__device__ __forceinline__ float lo2(f2 v) { return __uint_as_float(static_cast<uint32_t>(v)); }
__device__ __forceinline__ float hi2(f2 v) { return __uint_as_float(static_cast<uint32_t>(v >> 32)); }
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// Eight elements kept as they were loaded: four words of bf16, eight of fp32.
template <bool F32>
struct Vec8 {
  static constexpr int kWords = F32 ? 8 : 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int j = 0; j < kWords; ++j) w[j] = 0u;
  }
  // What was unpacked of it is not kept: a later get() unpacks again.
  __device__ __forceinline__ void forget() {
#pragma unroll
    for (int j = 0; j < kWords; ++j) asm volatile("" : "+r"(w[j]));
  }
  __device__ __forceinline__ void get(f2 (&f)[4]) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (F32) f[j] = pair2(__uint_as_float(w[2 * j]), __uint_as_float(w[2 * j + 1]));
      else f[j] = pair2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xffff0000u));
    }
  }
  // Elements e .. e + 7 of a row of K; those outside it are zero.
  template <bool ALIGNED>
  __device__ __forceinline__ void load(const void *row, int e, int K) {
    if (ALIGNED ? e < K : (e >= 0 && e + 8 <= K)) {
      const uint4 *p = F32 ? reinterpret_cast<const uint4 *>(static_cast<const float *>(row) + e)
                           : reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(row) + e);
#pragma unroll
      for (int j = 0; j < kWords / 4; ++j) {
        const uint4 u = p[j];
        w[4 * j] = u.x; w[4 * j + 1] = u.y; w[4 * j + 2] = u.z; w[4 * j + 3] = u.w;
      }
    } else {
      zero();
      if constexpr (!ALIGNED) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (e + j >= 0 && e + j < K) {
            if constexpr (F32) w[j] = static_cast<const uint32_t *>(row)[e + j];
            else w[j >> 1] |= static_cast<uint32_t>(static_cast<const uint16_t *>(row)[e + j]) << (16 * (j & 1));
          }
        }
      }
    }
  }
};

// Elements e .. e + 7 of a per-column vector (anything outside 0 .. K - 1 where K is no multiple of 8).
template <bool ALIGNED, bool F32>
__device__ __forceinline__ void load_cols(f2 (&f)[4], const void *p, int e, int K) {
  if constexpr (ALIGNED) {
    if constexpr (F32) {
      // 32 bytes a lane in one access where the address allows: two of 16 need twice the L1 wavefronts
      if (e < K && (reinterpret_cast<uintptr_t>(p) & 31u) == 0) {
        // volatile, with memory: else nothing keeps it behind grid_dep_wait, which the values may depend on
        asm volatile("ld.global.v4.b64 {%0, %1, %2, %3}, [%4];"
                     : "=l"(f[0]), "=l"(f[1]), "=l"(f[2]), "=l"(f[3])
                     : "l"(static_cast<const float *>(p) + e)
                     : "memory");
        return;
      }
    }
    Vec8<F32> v;
    v.template load<true>(p, e, K);
    v.get(f);
  } else {
    // whatever lies outside is multiplied by the zeros of a row's elements there
    auto at = [&](int k) -> float {
      k = min(max(k, 0), K - 1);
      if constexpr (F32) return static_cast<const float *>(p)[k];
      else return bf16_to_f32(static_cast<const uint16_t *>(p)[k]);
    };
    if (e >= 0 && e + 8 <= K) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (F32) f[j] = pair2(static_cast<const float *>(p)[e + 2 * j], static_cast<const float *>(p)[e + 2 * j + 1]);
        else f[j] = pair2(bf16_to_f32(static_cast<const uint16_t *>(p)[e + 2 * j]), bf16_to_f32(static_cast<const uint16_t *>(p)[e + 2 * j + 1]));
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) f[j] = pair2(at(e + 2 * j), at(e + 2 * j + 1));
    }
  }
}

template <bool ALIGNED, bool F32>
__device__ __forceinline__ void store_vec(const f2 (&v)[4], void *row, int e, int K) {
  float f[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f[2 * j] = lo2(v[j]);
    f[2 * j + 1] = hi2(v[j]);
  }
  if (ALIGNED ? e < K : (e >= 0 && e + 8 <= K)) {
    if constexpr (F32) {
      float4 *p = reinterpret_cast<float4 *>(static_cast<float *>(row) + e);
      p[0] = make_float4(f[0], f[1], f[2], f[3]);
      p[1] = make_float4(f[4], f[5], f[6], f[7]);
    } else {
      *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(row) + e) =
          make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
    }
  } else if constexpr (!ALIGNED) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (e + j >= 0 && e + j < K) {
        if constexpr (F32) static_cast<float *>(row)[e + j] = f[j];
        else static_cast<uint16_t *>(row)[e + j] = static_cast<uint16_t>(pack_bf16x2(f[j], 0.f));
      }
    }
  }
}

// A row's first element, by type.
template <bool F32>
__device__ __forceinline__ const void *row_at(const void *p, int64_t i) {
  return F32 ? static_cast<const void *>(static_cast<const float *>(p) + i)
             : static_cast<const void *>(static_cast<const uint16_t *>(p) + i);
}
template <bool F32>
__device__ __forceinline__ void *row_at(void *p, int64_t i) {
  return F32 ? static_cast<void *>(static_cast<float *>(p) + i) : static_cast<void *>(static_cast<uint16_t *>(p) + i);
}

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
// The sums of two values: of `a` in lanes 0 to 15, of `b` in the others, with
// one exchange a step for both.
__device__ __forceinline__ float warp_sum2(float a, float b) {
  const bool high = (threadIdx.x & 16) != 0;
  float v = (high ? b : a) + __shfl_xor_sync(0xffffffffu, high ? a : b, 16);
#pragma unroll
  for (int o = 8; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
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

// The largest magnitude of a row's values, and whether all are finite: 0 * v is
// NaN for the others. As bits, NaN sorts above every finite magnitude.
struct Magnitude {
  float most = 0.f;
  f2 zero = 0;
  __device__ __forceinline__ void add(const f2 (&f)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      most = fmaxf(most, fmaxf(fabsf(lo2(f[j])), fabsf(hi2(f[j]))));
      zero = fma2(f[j], both(0.f), zero);
    }
  }
  __device__ __forceinline__ uint32_t bits() const {
    const float z = lo2(zero) + hi2(zero);
    return z == z ? __float_as_uint(most) : 0x7fc00000u;
  }
};

// 16 bytes from global to shared memory, asynchronously; a thread waits for its
// own copies by groups. Through L1 (kHalves) where 32-byte sectors come as two
// halves: fp32 vectors, 4096 x 4096 in fp32 65 us past L1, 46 us through it.
// kCut: of the 16 bytes the first `bytes` are read, the rest become zero.
template <bool kHalves, bool kCut>
__device__ __forceinline__ void copy16(uint32_t smem, const void *g, int bytes) {
  if constexpr (kHalves && kCut) asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(smem), "l"(g), "r"(bytes) : "memory");
  else if constexpr (kHalves) asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(smem), "l"(g) : "memory");
  else if constexpr (kCut) asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem), "l"(g), "r"(bytes) : "memory");
  else asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem), "l"(g) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// ---- int8 codes -------------------------------------------------------------
// The code of a value, rint(fp32_rn(v / s)): v * (1 / s) is within
// 3 * 127.5 * 2^-24 < 3e-5 of the quotient, so its rounding can differ only
// next to a tie; vectors with such a value (about one in six hundred) divide.
// Adding 1.5 * 2^23 rounds to an integer, half to even, and leaves the code in
// the low byte. |v| <= 127 s (1 + 2^-22) keeps the code within +-127 unless s is
// subnormal (rounded coarsely) or its reciprocal overflows: such rows always
// divide, and clamp.
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

// Codes of elements e .. e + 7 of a row of K.
template <bool ALIGNED>
__device__ __forceinline__ void store_codes(const f2 (&f)[4], const RowScale &r, int8_t *row, int e, int K) {
  uint32_t c[8];
  if (r.zero) {   // the same for the whole row, as is r.divide
#pragma unroll
    for (int j = 0; j < 8; ++j) c[j] = 0u;
  } else {
    float off = 0.f;   // the farthest of the values from its code
    const f2 inv = both(r.inv), magic = both(kRoundMagic), back = both(-kRoundMagic);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const f2 m = fma2(f[j], inv, magic);
      // code - v / s; the subtraction of the magic number is exact
      const f2 d = fma2(f[j], both(-r.inv), add2(m, back));
      off = fmaxf(off, fmaxf(fabsf(lo2(d)), fabsf(hi2(d))));
      c[2 * j] = static_cast<uint32_t>(m);
      c[2 * j + 1] = static_cast<uint32_t>(m >> 32);
    }
    if (r.divide || off > 0.4999f) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float v = j & 1 ? hi2(f[j >> 1]) : lo2(f[j >> 1]);
        c[j] = static_cast<uint32_t>(static_cast<int>(fminf(fmaxf(rintf(__fdiv_rn(v, r.s)), -127.f), 127.f)));
      }
    }
  }
  if (ALIGNED ? e < K : (e >= 0 && e + 8 <= K)) {
    uint32_t w[2];
#pragma unroll
    for (int j = 0; j < 2; ++j)
      w[j] = prmt(prmt(c[4 * j], c[4 * j + 1], 0x0040u), prmt(c[4 * j + 2], c[4 * j + 3], 0x0040u), 0x5410u);
    *reinterpret_cast<uint2 *>(row + e) = make_uint2(w[0], w[1]);
  } else if constexpr (!ALIGNED) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (e + j >= 0 && e + j < K) row[e + j] = static_cast<int8_t>(c[j] & 0xffu);
  }
}

// ---- how threads share a row -------------------------------------------------
// A warp or a block a row, `nv` vectors a thread (nv 0: as many passes as it
// takes, for rows too long for registers). Few rows: one vector a thread, for
// the latency. Many: `many` vectors, so that each SM holds several blocks, none
// of which waits long at its barriers, with enough loads in flight.
struct RowPlan {
  int nv, threads;
  bool warp, aligned;
};
inline RowPlan row_plan(int64_t M, int64_t K, int sms, int many) {
  const int64_t v = K % 8 ? (K + 7) / 8 + 1 : K / 8;   // a row off phase may touch one vector more
  auto per = [&](int nv) { return static_cast<int>((v + 32 * nv - 1) / (32 * nv) * 32); };
  const bool aligned = K % 8 == 0;
  if (v <= 32) return {1, 128, true, aligned};
  if (v <= 64) return {2, 128, true, aligned};
  if (v <= 1024 && M <= 2 * sms) return {1, per(1), false, aligned};
  if (v <= 128) return {4, 128, true, aligned};
  if (many == 2 && v <= 1024) return {2, per(2), false, aligned};
  if (v <= 2048) return {4, per(4), false, aligned};
  if (v <= 4097) return {8, per(8), false, aligned};
  return {0, 1024, false, aligned};
}

// Numbers as types, and a call of go(nv, warp, aligned) with the plan's.
template <int V>
struct Num {
  static constexpr int value = V;
};
template <class F>
auto dispatch_row(const RowPlan &p, F go) {
  auto with = [&](auto aligned) {
    if (p.warp) return p.nv == 1 ? go(Num<1>{}, Num<1>{}, aligned) : p.nv == 2 ? go(Num<2>{}, Num<1>{}, aligned) : go(Num<4>{}, Num<1>{}, aligned);
    return p.nv == 1   ? go(Num<1>{}, Num<0>{}, aligned)
           : p.nv == 2 ? go(Num<2>{}, Num<0>{}, aligned)
           : p.nv == 4 ? go(Num<4>{}, Num<0>{}, aligned)
                       : go(Num<8>{}, Num<0>{}, aligned);
  };
  return p.aligned ? with(Num<1>{}) : with(Num<0>{});
}
inline unsigned row_grid(const RowPlan &p, int64_t M) {
  return static_cast<unsigned>(p.warp ? (M + p.threads / 32 - 1) / (p.threads / 32) : M);
}
// The most threads a plan gives a block of nv vectors a thread.
constexpr int row_threads(int nv, bool warp) { return warp ? 128 : (nv == 1 ? 1024 : (nv == 8 ? 544 : 512)); }

}  // namespace qlora
