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

// 64 (or 32) columns of 16 TMEM lanes as eight (four) m16n8 accumulator fragments: of the n8
// block j, thread T has columns 2 (T % 4), + 1 of lane T / 4 in r[4 j], r[4 j + 1]
// and of lane T / 4 + 8 in r[4 j + 2], r[4 j + 3].
__device__ __forceinline__ void tmem_ld_frag64(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}

__device__ __forceinline__ void tmem_ld_frag32(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// Two neighbouring ranks (k, k + 1) of the adapter's activations sU / sT at a
// token, and of its weight at a feature: a register of an m16n8k16 fragment.
// Ranks past r, tokens past M and features past F are zero.
__device__ __forceinline__ uint32_t lora_act_pair(Waited after, const uint16_t *u, int64_t M, int r, int64_t m, int k) {
  return load_after(after, reinterpret_cast<const uint32_t *>(u + m * r + k), m < M && k < r);
}
template <bool kDx>
__device__ __forceinline__ uint32_t lora_w_pair(Waited after, const uint16_t *w, int64_t F, int r, int64_t f, int k) {
  if constexpr (kDx) {   // A [r, F]
    const uint16_t *a = w + static_cast<int64_t>(k) * F + f;
    return load_after(after, a, a + F, f < F && k < r);
  } else {               // B [F, r]
    return load_after(after, reinterpret_cast<const uint32_t *>(w + f * r + k), f < F && k < r);
  }
}

// Whether a phase is complete, without ever suspending the thread (try_wait may).
__device__ __forceinline__ bool mbar_test_wait(uint64_t *bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// One load of a ring slot: waits (bounded) until a slot's copies have landed,
// so that none outlives the CTA's shared memory after an abort.
__device__ __forceinline__ void drain_slot(uint64_t *full, uint32_t parity) {
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(full, parity) && global_timer_ns() - t0 < kWaitLimitNs) {
  }
}

int i8_split_ways(int64_t M, int64_t F, int64_t C);                  // how many CTAs the split kernel gives a tile
cudaError_t launch_i8_split(const I8GemmArgs &a, cudaStream_t st);   // i8_gemm_split.cu
cudaError_t launch_i8_pair(const I8GemmArgs &a, cudaStream_t st);    // i8_gemm_pair.cu
cudaError_t launch_i8_gemm(const I8GemmArgs &a, cudaStream_t st);    // the one of the two that fits the sizes

}  // namespace qlora
