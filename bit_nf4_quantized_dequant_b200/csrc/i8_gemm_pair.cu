// Int8 GEMM on CTA pairs: the kernel for token counts whose output tiles fill
// the SMs.
//
// A pair (cta_group::2, a cluster of two) computes a tile of 256 tokens (UMMA
// M, 128 a CTA) by 256 features (UMMA N, each CTA loads 128 of them), so a step
// of 128 codes needs 32 KB of shared memory a CTA for 512 tensor cycles. The
// int32 accumulator takes 256 TMEM columns and is double-buffered: the epilogue
// of one tile runs under the main loop of the next.
//
// The epilogue reads TMEM in the fragment layout of the warp-level MMA
// (16x256b: a thread holds two neighbouring features of rows T / 4 and
// T / 4 + 8), scales to fp32 and adds the adapter's term by mma.m16n8k16 into
// the same registers: the rank-r product needs neither a second accumulator nor
// more than r / 8 warp MMAs per 16 x 8 outputs. bf16 results leave through
// swizzled shared memory and TMA stores, which clip the ragged edges.
//
// Warps (384 threads): 0 TMA producer, 1 MMA issuer and TMEM owner, 4-11
// epilogue (TMEM lane quadrant warp % 4, half of the columns each).
#include "i8_gemm.cuh"

namespace qlora {

bool encode_2d(CUtensorMap *map, CUtensorMapDataType dtype, const void *base, uint64_t inner, uint64_t outer,
               uint64_t row_bytes, uint32_t box_inner, uint32_t box_outer, CUtensorMapSwizzle swizzle);

namespace {

constexpr int kThreads = 384;
constexpr int kTile = 256;                                 // tokens and features per pair tile
constexpr uint32_t kBoxBytes = 128 * kI8Step;              // 16 KiB: 128 tokens, or 128 features, of a step
constexpr uint32_t kSlotBytes = 2 * kBoxBytes;
constexpr int kStages = 6;
constexpr uint32_t kOutBytes = 32 * 128;                   // 32 tokens x 64 features bf16, per epilogue warp
constexpr int kEpiWarps = 8;

struct PairParams {
  const float *act_scale, *w_scale;
  const uint16_t *lora_act, *lora_w;
  int32_t *status;
  int64_t M, F;
  int r, nk, feat_tiles, tok_tiles;
};

struct PairSmem {
  uint8_t ring[kStages][kSlotBytes];
  uint8_t out[kEpiWarps][kOutBytes];
  uint64_t full[kStages], empty[kStages], accf[2], acce[2], drain;
  uint32_t tmem_holder;
  int abort_flag;
};

__device__ __forceinline__ void stmatrix_x4(uint32_t saddr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(saddr), "r"(a), "r"(b), "r"(c),
               "r"(d)
               : "memory");
}

// kSteps: mma steps of 16 ranks (0: no adapter).
template <bool kDx, int kSteps>
__global__ void __launch_bounds__(kThreads, 1)
    i8_pair_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_act,
                   const __grid_constant__ CUtensorMap tm_out, const PairParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  PairSmem &sm = *reinterpret_cast<PairSmem *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  volatile int *abort_flag = &sm.abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int ntiles = p.feat_tiles * p.tok_tiles;
  const int first = static_cast<int>(blockIdx.x >> 1), stride = static_cast<int>(gridDim.x >> 1);
  // tile -> (tokens, features): tokens fastest, so that the pairs at work share few weight tiles
  auto tok0 = [&](int tile) { return (tile % p.tok_tiles) * kTile; };
  auto feat0 = [&](int tile) { return (tile / p.tok_tiles) * kTile; };

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&sm.full[i], 1);
      mbar_init(&sm.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.accf[i], 1);
      mbar_init(&sm.acce[i], 2 * kEpiWarps);
    }
    mbar_init(&sm.drain, 1);
    sm.abort_flag = 0;
    fence_mbarrier_init();
    tma_prefetch_desc(&tm_w);
    tma_prefetch_desc(&tm_act);
    tma_prefetch_desc(&tm_out);
  }
  if (warp == 1) {
    tmem_alloc_pair(&sm.tmem_holder, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();   // the peer's barriers exist before anyone signals them
  tc_fence_after();
  const uint32_t tmem = sm.tmem_holder;

  if (warp == 0) {
    // ---------------- producer: this CTA's tokens and features ----------------
    if (elect_one()) {
      int slot = 0;
      uint32_t ph = 0, landed = 0, par = 0;
      bool ok = true;
      for (int tile = first; tile < ntiles && ok; tile += stride) {
        const int t0 = tok0(tile) + static_cast<int>(rank) * 128, f0 = feat0(tile) + static_cast<int>(rank) * 128;
        for (int s = 0; s < p.nk; ++s) {
          if (!mbar_wait(&sm.empty[slot], ph ^ 1u, abort_flag, p.status)) {
            ok = false;
            break;
          }
          if (leader) mbar_arrive_expect_tx(&sm.full[slot], 2 * kSlotBytes);
          const uint32_t bar = mapa_shared(smem_u32(&sm.full[slot]), 0u);
          tma_load_2d_pair(sm.ring[slot], &tm_act, bar, s * kI8Step, t0);
          if (!kDx) tma_load_2d_pair(sm.ring[slot] + kBoxBytes, &tm_w, bar, s * kI8Step, f0);
          else      tma_load_2d_pair(sm.ring[slot] + kBoxBytes, &tm_w, bar, f0, s * kI8Step);
          landed |= 1u << slot;
          par = (par & ~(1u << slot)) | (ph << slot);
          if (++slot == kStages) {
            slot = 0;
            ph ^= 1u;
          }
        }
      }
      if (!ok && leader)
        for (int i = 0; i < kStages; ++i)
          if (landed & (1u << i)) drain_slot(&sm.full[i], (par >> i) & 1u);
    }
  } else if (warp == 1) {
    // ---------------- MMA issuer (even CTA) ----------------
    if (leader && elect_one()) {
      constexpr uint32_t idesc = idesc_i8(256, kTile, false, kDx);
      const uint64_t a0 = smem_desc(smem_u32(sm.ring[0]), 16u, 1024u, kLayoutSW128);
      const uint64_t b0 = smem_desc(smem_u32(sm.ring[0]) + kBoxBytes, kDx ? kBoxBytes : 16u, 1024u, kLayoutSW128);
      // a step of 32 codes: +32 bytes along a K-major row, or 32 rows of 128 bytes (MN-major)
      constexpr uint32_t b_step = (kDx ? 32u * 128u : 32u) >> 4;
      int slot = 0, n = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int tile = first; tile < ntiles && ok; tile += stride, ++n) {
        const int buf = n & 1;
        if (!mbar_wait(&sm.acce[buf], ((n >> 1) & 1u) ^ 1u, abort_flag, p.status)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem + static_cast<uint32_t>(buf) * kTile;
        for (int s = 0; s < p.nk; ++s) {
          if (!mbar_wait(&sm.full[slot], ph, abort_flag, p.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t off = (static_cast<uint32_t>(slot) * kSlotBytes) >> 4;
#pragma unroll
          for (uint32_t j = 0; j < kI8Step / 32; ++j)
            umma_i8_pair(d, a0 + off + j * 2u, b0 + off + j * b_step, idesc, s || j);
          umma_commit_pair(&sm.empty[slot]);
          if (++slot == kStages) {
            slot = 0;
            ph ^= 1u;
          }
        }
        if (ok) umma_commit_pair(&sm.accf[buf]);
      }
      if (!ok) {   // the MMAs issued so far must be over before the CTA leaves
        umma_commit_pair(&sm.drain);
        drain_slot(&sm.drain, 0);
      }
    }
  } else if (warp >= 4) {
    // ---------------- epilogue ----------------
    const int quad = warp & 3, half = (warp - 4) >> 2;   // 32 tokens, 128 features of the CTA's 128 x 256
    uint8_t *stage = sm.out[warp - 4];
    const uint32_t stage_a = smem_u32(stage);
    const int g = lane >> 2, q2 = (lane & 3) * 2;        // fragment row and column pair
    int n = 0;
    bool ok = true;
    for (int tile = first; tile < ntiles && ok; tile += stride, ++n) {
      const int buf = n & 1;
      const int64_t m0 = static_cast<int64_t>(tok0(tile)) + rank * 128 + quad * 32;
      const int64_t f0 = static_cast<int64_t>(feat0(tile)) + half * 128;
      // this thread's four tokens: scales and adapter fragments, ahead of the accumulator
      float sx[4];
      uint32_t u[2][kSteps ? kSteps : 1][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t m = m0 + g + 8 * i;
        sx[i] = m < p.M ? __ldg(p.act_scale + m) : 0.f;
        if constexpr (kSteps > 0) {
#pragma unroll
          for (int ks = 0; ks < kSteps; ++ks)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const int k = ks * 16 + c * 8 + q2;
              u[i >> 1][ks][(i & 1) + 2 * c] = lora_act_pair(p.lora_act, p.M, p.r, m, k);
            }
        }
      }
      if (!__all_sync(0xffffffffu, mbar_wait(&sm.accf[buf], (n >> 1) & 1u, abort_flag, p.status))) {
        ok = false;
        break;
      }
      tc_fence_after();
#pragma unroll 1
      for (int ch = 0; ch < 2; ++ch) {
        const int64_t fc = f0 + ch * 64;
        uint32_t acc[2][32];
        const uint32_t ta = tmem + (static_cast<uint32_t>(quad * 32) << 16) + buf * kTile + half * 128 + ch * 64;
        tmem_ld_frag64(ta, acc[0]);
        tmem_ld_frag64(ta + (16u << 16), acc[1]);
        float y[2][8][4];
        // feature scales of this thread's columns, under the TMEM loads
        float2 sw[8];
        if constexpr (!kDx) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int64_t f = fc + j * 8 + q2;
            sw[j] = f < p.F ? __ldg(reinterpret_cast<const float2 *>(p.w_scale + f)) : make_float2(0.f, 0.f);
          }
        }
        uint32_t b[kSteps ? 8 : 1][2];
        auto load_b = [&](int ks) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int c = 0; c < 2; ++c)
              b[j][c] = lora_w_pair<kDx>(p.lora_w, p.F, p.r, fc + j * 8 + g, ks * 16 + c * 8 + q2);
        };
        if constexpr (kSteps > 0) load_b(0);
        tmem_ld_wait();
        if (ch == 1) {   // the accumulator is in registers: the next tile but one may have it
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&sm.acce[buf]), 0u));
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float v = static_cast<float>(static_cast<int>(acc[h][4 * j + e])) * sx[2 * h + (e >> 1)];
              if constexpr (!kDx) v *= (e & 1) ? sw[j].y : sw[j].x;
              y[h][j][e] = v;
            }
        if constexpr (kSteps > 0) {
#pragma unroll
          for (int ks = 0; ks < kSteps; ++ks) {
            if (ks) load_b(ks);
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int j = 0; j < 8; ++j) mma_16816(y[h][j], u[h][ks], b[j][0], b[j][1]);
          }
        }
        // the staging tile is free again once the previous store has read it
        if (lane == 0) bulk_wait_group_read<0>();
        __syncwarp();
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < 8; j += 2) {
            const uint32_t row = static_cast<uint32_t>(h * 16 + ((lane >> 3) & 1) * 8 + (lane & 7));
            const uint32_t chunk = static_cast<uint32_t>(j + (lane >> 4));
            stmatrix_x4(stage_a + row * 128u + ((chunk ^ (row & 7u)) << 4), pack_bf16x2(y[h][j][0], y[h][j][1]),
                        pack_bf16x2(y[h][j][2], y[h][j][3]), pack_bf16x2(y[h][j + 1][0], y[h][j + 1][1]),
                        pack_bf16x2(y[h][j + 1][2], y[h][j + 1][3]));
          }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && m0 < p.M && fc < p.F) {
          tma_store_2d(&tm_out, stage, static_cast<int32_t>(fc), static_cast<int32_t>(m0));
          bulk_commit_group();
        }
      }
    }
    if (lane == 0) bulk_wait_group<0>();
  }
  __syncthreads();
  cluster_sync_all();   // the pair is done with each other's shared memory and TMEM
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

template <bool kDx>
const void *pair_fn(int steps) {
  switch (steps) {
    case 0: return reinterpret_cast<const void *>(i8_pair_kernel<kDx, 0>);
    case 1: return reinterpret_cast<const void *>(i8_pair_kernel<kDx, 1>);
    case 2: return reinterpret_cast<const void *>(i8_pair_kernel<kDx, 2>);
    case 3: return reinterpret_cast<const void *>(i8_pair_kernel<kDx, 3>);
    default: return reinterpret_cast<const void *>(i8_pair_kernel<kDx, 4>);
  }
}

}  // namespace

cudaError_t launch_i8_pair(const I8GemmArgs &a, cudaStream_t st) {
  PairParams p{};
  p.act_scale = a.act_scale;
  p.w_scale = a.w_scale;
  p.lora_act = a.lora_act;
  p.lora_w = a.lora_w;
  p.status = a.status;
  p.M = a.M;
  p.F = a.F;
  p.r = a.r;
  p.nk = static_cast<int>((a.C + kI8Step - 1) / kI8Step);
  p.feat_tiles = static_cast<int>((a.F + kTile - 1) / kTile);
  p.tok_tiles = static_cast<int>((a.M + kTile - 1) / kTile);

  CUtensorMap tm_w, tm_act, tm_out;
  const uint64_t wrow = static_cast<uint64_t>(a.dx ? a.F : a.C), wrows = static_cast<uint64_t>(a.dx ? a.C : a.F);
  bool ok = encode_2d(&tm_w, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.w, wrow, wrows, wrow, 128, 128, CU_TENSOR_MAP_SWIZZLE_128B);
  ok &= encode_2d(&tm_act, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.act, a.C, a.M, a.C, kI8Step, 128, CU_TENSOR_MAP_SWIZZLE_128B);
  ok &= encode_2d(&tm_out, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.out, a.F, a.M, a.F * 2, 64, 32, CU_TENSOR_MAP_SWIZZLE_128B);
  if (!ok) return cudaErrorInvalidValue;
  const int steps = (a.r + 15) / 16;
  const void *fn = a.dx ? pair_fn<true>(steps) : pair_fn<false>(steps);
  const size_t smem = sizeof(PairSmem) + 1024;
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  const int64_t tiles = static_cast<int64_t>(p.feat_tiles) * p.tok_tiles, pairs = device_sm_count() / 2;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * (tiles < pairs ? tiles : pairs)));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  void *args[] = {&tm_w, &tm_act, &tm_out, &p};
  return cudaLaunchKernelExC(&cfg, fn, args);
}

// Single tiles of 128 x 128 as long as one wave of CTAs holds them; past that
// the pairs' 256 x 256 tiles, which need half the operand bytes per output. A
// little more than one wave of pairs goes back to single tiles, two to a SM.
// Measured (rank 16): 512 tokens 4096 x 4096 (128 tiles, 32 pair tiles) 12.9 us
// split, 16.3 pair; 768 tokens (192, 48) 20.2 and 17.4; 200 tokens 11008 x 4096
// (172, 43) 21.1 and 18.5; 384 tokens (258, 86) 23.0 and 29.5.
cudaError_t launch_i8_gemm(const I8GemmArgs &a, cudaStream_t st) {
  auto tiles = [&](int64_t t) { return ((a.F + t - 1) / t) * ((a.M + t - 1) / t); };
  const int64_t sms = device_sm_count(), single = tiles(128);
  const bool split = single <= sms || (single <= 2 * sms && tiles(kTile) > sms / 2);
  return split ? launch_i8_split(a, st) : launch_i8_pair(a, st);
}

}  // namespace qlora
