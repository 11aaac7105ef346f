// What the int8 GEMM kernels share: their arguments and the tcgen05 kind::i8
// wrappers.
//
// Both products contract int8 codes exactly into int32 and scale afterwards:
//   FWD: D[m, n] = sum_k Xq[m, k] Wq[n, k]   -> Y[m, n]  = D sx[m] sw[n] + sum_j sU[m, j] B[n, j]
//   DX:  D[m, k] = sum_n gq[m, n] Wq[n, k]   -> dX[m, k] = D sg[m]       + sum_j sT[m, j] A[j, k]
// In both, "features" are the output's columns (n, or k for DX) and the
// contraction is cut into steps of 128 codes: 128 bytes, one swizzled row. The
// weight tile of a step is the same box of 128 x 128 codes; FWD reads it
// K-major (rows are features), DX MN-major (rows are contraction steps).
#pragma once

#include "qlora_device.cuh"

namespace qlora {

constexpr int kI8Step = 128;   // contraction codes per step

struct I8GemmArgs {
  bool dx;
  const int8_t *act;        // Xq [M, K] or gq [M, N]
  const float *act_scale;   // [M]
  const int8_t *w;          // Wq [N, K]
  const float *w_scale;     // [N] (FWD), not read by DX
  int64_t M, F, C;          // tokens, features, contraction length
  int r;                    // 0: no adapter
  const uint16_t *lora_act; // sU or sT [M, r]
  const uint16_t *lora_w;   // B [F, r] (FWD) or A [r, F] (DX)
  uint16_t *out;            // [M, F]
  int32_t *status;
};

// Instruction descriptor: kind::i8 with signed A and B, int32 D, no saturation.
__host__ __device__ constexpr uint32_t idesc_i8(uint32_t M, uint32_t N, bool a_mn_major, bool b_mn_major) {
  return (2u << 4)                        // D format: s32
         | (1u << 7)                      // A format: s8
         | (1u << 10)                     // B format: s8
         | ((a_mn_major ? 1u : 0u) << 15) // A major
         | ((b_mn_major ? 1u : 0u) << 16) // B major
         | ((N >> 3) << 17)               // N / 8
         | ((M >> 4) << 24);              // M / 16
}

// D[tmem] (+)= A[smem desc] * B[smem desc]^T over 32 int8 codes.
__device__ __forceinline__ void umma_i8(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void umma_i8_pair(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// One load of a ring slot: waits (bounded) until a slot's copies have landed,
// so that none outlives the CTA's shared memory after an abort.
__device__ __forceinline__ void drain_slot(uint64_t *full, uint32_t parity) {
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(full, parity) && global_timer_ns() - t0 < kWaitLimitNs) {
  }
}

cudaError_t launch_i8_split(const I8GemmArgs &a, cudaStream_t st);   // i8_gemm_split.cu
cudaError_t launch_i8_pair(const I8GemmArgs &a, cudaStream_t st);    // i8_gemm_pair.cu
cudaError_t launch_i8_gemm(const I8GemmArgs &a, cudaStream_t st);    // the one of the two that fits the sizes

}  // namespace qlora
