// Int8 GEMM with the contraction split over a cluster: the kernel for token
// counts that leave most SMs without an output tile of their own.
//
// One CTA holds a tile of 128 features (UMMA M) by up to 256 tokens (UMMA N),
// so a weight code is read once per 256 tokens; the CTAs of a cluster (1, 2, 4
// or 8) take consecutive parts of the tile's contraction and their int32
// partial sums are added over distributed shared memory. Integer sums are
// exact, so the result does not depend on the split. Few tokens are bound by
// the weight's bytes: the split brings enough CTAs to keep every SM loading,
// and a ring of 128 x 128-code boxes up to 200 KB deep keeps them in flight.
//
// Warps: 0 TMA producer, 1 MMA issuer and TMEM owner; 0-3 move the accumulator
// from TMEM to shared memory (one lane per feature), all eight finish.
#include "i8_gemm.cuh"

namespace qlora {

bool encode_2d(CUtensorMap *map, CUtensorMapDataType dtype, const void *base, uint64_t inner, uint64_t outer,
               uint64_t row_bytes, uint32_t box_inner, uint32_t box_outer, CUtensorMapSwizzle swizzle);

namespace {

constexpr int kThreads = 256;
constexpr int kFeat = 128;                                // features per tile
constexpr uint32_t kWBytes = kFeat * kI8Step;             // weight box of a step
constexpr int kMaxStages = 12;

struct SplitParams {
  const float *act_scale, *w_scale;
  const uint16_t *lora_act, *lora_w;
  uint16_t *out;
  int32_t *status;
  int64_t M, F;
  int r, tn, stages, nk, feat_tiles;
  uint32_t tmem_cols;
};

__host__ __device__ inline uint32_t ring_bytes(int tn, int stages) {
  const uint32_t ring = static_cast<uint32_t>(stages) * (kWBytes + static_cast<uint32_t>(tn) * kI8Step);
  const uint32_t part = static_cast<uint32_t>(tn) * kFeat * 4;
  return ring > part ? ring : part;
}

__device__ __forceinline__ int2 ld_dsmem_int2(uint32_t addr) {
  int2 v;
  asm volatile("ld.shared::cluster.v2.s32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  return v;
}

template <bool kDx>
__global__ void __launch_bounds__(kThreads, 1)
    i8_split_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_act,
                    const SplitParams p, const int split) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint16_t *lora = reinterpret_cast<uint16_t *>(ring + ring_bytes(p.tn, p.stages));   // [r][128]
  uint64_t *full = reinterpret_cast<uint64_t *>(lora + static_cast<size_t>(p.r) * kFeat);
  uint64_t *empty = full + kMaxStages;
  uint64_t *done = empty + kMaxStages;
  uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(done + 1);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = split > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int tile = static_cast<int>(blockIdx.x) / split;
  const int ft = tile % p.feat_tiles, tt = tile / p.feat_tiles;
  const int64_t f0 = static_cast<int64_t>(ft) * kFeat, t0 = static_cast<int64_t>(tt) * p.tn;
  const int s0 = p.nk * rank / split, s1 = p.nk * (rank + 1) / split;
  const uint32_t act_bytes = static_cast<uint32_t>(p.tn) * kI8Step, slot_bytes = kWBytes + act_bytes;

  if (threadIdx.x == 0) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_mbarrier_init();
    tma_prefetch_desc(&tm_w);
    tma_prefetch_desc(&tm_act);
  }
  if (warp == 1) {
    tmem_alloc(tmem_holder, p.tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;

  if (warp == 0) {
    if (elect_one()) {
      int slot = 0;
      uint32_t ph = 0, landed = 0, par = 0;
      bool ok = true;
      for (int s = s0; s < s1; ++s) {
        if (!mbar_wait(&empty[slot], ph ^ 1u, abort_flag, p.status)) {
          ok = false;
          break;
        }
        mbar_arrive_expect_tx(&full[slot], slot_bytes);
        uint8_t *w = ring + static_cast<uint32_t>(slot) * slot_bytes;
        if (!kDx) tma_load_2d(w, &tm_w, &full[slot], s * kI8Step, static_cast<int32_t>(f0));
        else      tma_load_2d(w, &tm_w, &full[slot], static_cast<int32_t>(f0), s * kI8Step);
        tma_load_2d(w + kWBytes, &tm_act, &full[slot], s * kI8Step, static_cast<int32_t>(t0));
        landed |= 1u << slot;
        par = (par & ~(1u << slot)) | (ph << slot);
        if (++slot == p.stages) {
          slot = 0;
          ph ^= 1u;
        }
      }
      if (!ok)
        for (int i = 0; i < p.stages; ++i)
          if (landed & (1u << i)) drain_slot(&full[i], (par >> i) & 1u);
    }
  } else if (warp == 1) {
    if (elect_one()) {
      const uint32_t idesc = idesc_i8(kFeat, static_cast<uint32_t>(p.tn), kDx, false);
      // a step of 32 codes: +32 bytes along a K-major row, or 32 rows of 128 bytes (MN-major)
      const uint64_t a0 = smem_desc(smem_u32(ring), kDx ? kWBytes : 16u, 1024u, kLayoutSW128);
      const uint64_t b0 = smem_desc(smem_u32(ring) + kWBytes, 16u, 1024u, kLayoutSW128);
      constexpr uint32_t a_step = (kDx ? 32u * 128u : 32u) >> 4;
      int slot = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int s = s0; s < s1; ++s) {
        if (!mbar_wait(&full[slot], ph, abort_flag, p.status)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint64_t off = (static_cast<uint32_t>(slot) * slot_bytes) >> 4;
#pragma unroll
        for (uint32_t j = 0; j < kI8Step / 32; ++j)
          umma_i8(tmem, a0 + off + j * a_step, b0 + off + j * 2u, idesc, s > s0 || j);
        umma_commit(&empty[slot]);
        if (++slot == p.stages) {
          slot = 0;
          ph ^= 1u;
        }
      }
      // also after an abort: the MMAs issued so far must be over before the CTA leaves
      umma_commit(done);
      if (!ok) drain_slot(done, 0);
    }
  } else if (warp >= 4 && p.r) {
    // the adapter's tile as [j][feature], while the main loop runs
    for (int i = threadIdx.x - 128; i < p.r * kFeat; i += kThreads - 128) {
      const int j = kDx ? i / kFeat : i % p.r, n = kDx ? i % kFeat : i / p.r;
      uint16_t v = 0;
      if (f0 + n < p.F) v = kDx ? p.lora_w[static_cast<int64_t>(j) * p.F + f0 + n] : p.lora_w[(f0 + n) * p.r + j];
      lora[j * kFeat + n] = v;
    }
  }
  __syncwarp();

  // ---- accumulator -> shared memory [token][feature], over the finished ring ----
  int *part = reinterpret_cast<int *>(ring);
  if (warp < 4) {
    // the TMEM loads are warp-wide: every lane takes the same way
    if (__all_sync(0xffffffffu, mbar_wait(done, 0, abort_flag, p.status))) {
      tc_fence_after();
      const int n = warp * 32 + lane;
      for (int c = 0; c < p.tn; c += 16) {
        uint32_t v[16];
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
            "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
            : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
              "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
            : "r"(tmem + (static_cast<uint32_t>(warp * 32) << 16) + static_cast<uint32_t>(c))
            : "memory");
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 16; ++j) part[(c + j) * kFeat + n] = static_cast<int>(v[j]);
      }
      tc_fence_before();
    }
  }
  __syncwarp();
  if (split > 1) cluster_sync_all();
  else __syncthreads();

  // ---- sum over the cluster, scales, adapter: this CTA's share of the tokens ----
  if (!*abort_flag) {
    const int per = (p.tn + split - 1) / split;
    const int tb = rank * per, te = min(min(tb + per, p.tn), static_cast<int>(p.M - t0 < p.tn ? p.M - t0 : p.tn));
    const int n = 2 * (threadIdx.x & 63);
    if (f0 + n < p.F) {
      const float w0 = kDx ? 1.f : p.w_scale[f0 + n], w1 = kDx ? 1.f : p.w_scale[f0 + n + 1];
      uint32_t peer[8];
      const uint32_t mine = smem_u32(part);
#pragma unroll
      for (int q = 0; q < 8; ++q) peer[q] = q < split ? (split > 1 ? mapa_shared(mine, q) : mine) : 0u;
      for (int t = tb + (threadIdx.x >> 6); t < te; t += kThreads / 64) {
        int a0 = 0, a1 = 0;
        const uint32_t off = static_cast<uint32_t>(t * kFeat + n) * 4u;
#pragma unroll
        for (int q = 0; q < 8; ++q)
          if (q < split) {
            const int2 v = ld_dsmem_int2(peer[q] + off);
            a0 += v.x;
            a1 += v.y;
          }
        const int64_t m = t0 + t;
        const float sx = p.act_scale[m];
        float y0 = static_cast<float>(a0) * sx * w0, y1 = static_cast<float>(a1) * sx * w1;
        const uint16_t *u = p.lora_act + m * p.r;
        for (int j = 0; j < p.r; ++j) {
          const float uj = __uint_as_float(static_cast<uint32_t>(u[j]) << 16);
          const uint32_t b = *reinterpret_cast<const uint32_t *>(lora + j * kFeat + n);
          y0 = fmaf(uj, __uint_as_float(b << 16), y0);
          y1 = fmaf(uj, __uint_as_float(b & 0xffff0000u), y1);
        }
        *reinterpret_cast<uint32_t *>(p.out + m * p.F + f0 + n) = pack_bf16x2(y0, y1);
      }
    }
  }
  // no CTA leaves while a peer may still read its partial sums
  if (split > 1) cluster_sync_all();
  else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, p.tmem_cols);
  }
}

}  // namespace

cudaError_t launch_i8_split(const I8GemmArgs &a, cudaStream_t st) {
  SplitParams p{};
  p.act_scale = a.act_scale;
  p.w_scale = a.w_scale;
  p.lora_act = a.lora_act;
  p.lora_w = a.lora_w;
  p.out = a.out;
  p.status = a.status;
  p.M = a.M;
  p.F = a.F;
  p.r = a.r;
  p.tn = a.M >= 256 ? 256 : static_cast<int>((a.M + 15) / 16 * 16);
  p.tmem_cols = 32;
  while (p.tmem_cols < static_cast<uint32_t>(p.tn)) p.tmem_cols *= 2;
  p.nk = static_cast<int>((a.C + kI8Step - 1) / kI8Step);
  p.feat_tiles = static_cast<int>((a.F + kFeat - 1) / kFeat);
  const int64_t tiles = static_cast<int64_t>(p.feat_tiles) * ((a.M + p.tn - 1) / p.tn);
  int split = 1;
  while (split < 8 && tiles * split * 2 <= device_sm_count() && p.nk >= split * 2) split *= 2;
  const int per_cta = (p.nk + split - 1) / split;
  const uint32_t slot = kWBytes + static_cast<uint32_t>(p.tn) * kI8Step;
  p.stages = static_cast<int>((200u * 1024u - static_cast<uint32_t>(p.r) * kFeat * 2u) / slot);
  if (p.stages > kMaxStages) p.stages = kMaxStages;
  if (p.stages > per_cta) p.stages = per_cta;
  const size_t smem = 1024 + ring_bytes(p.tn, p.stages) + static_cast<size_t>(p.r) * kFeat * 2 + (2 * kMaxStages + 1) * 8 + 16;

  CUtensorMap tm_w, tm_act;
  const uint64_t wrow = static_cast<uint64_t>(a.dx ? a.F : a.C), wrows = static_cast<uint64_t>(a.dx ? a.C : a.F);
  bool ok = encode_2d(&tm_w, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.w, wrow, wrows, wrow, 128, 128, CU_TENSOR_MAP_SWIZZLE_128B);
  ok &= encode_2d(&tm_act, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.act, a.C, a.M, a.C, kI8Step, p.tn,
                  CU_TENSOR_MAP_SWIZZLE_128B);
  if (!ok) return cudaErrorInvalidValue;
  const void *fn = a.dx ? reinterpret_cast<const void *>(i8_split_kernel<true>)
                        : reinterpret_cast<const void *>(i8_split_kernel<false>);
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * split));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(split);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  void *args[] = {&tm_w, &tm_act, &p, &split};
  return cudaLaunchKernelExC(&cfg, fn, args);
}

}  // namespace qlora
