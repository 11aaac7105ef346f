// Int8 GEMM on CTA pairs: the kernel for token counts whose output tiles fill
// the SMs.
//
// A pair (cta_group::2, a cluster of two) computes a tile of 256 tokens (UMMA
// M, 128 a CTA) by up to 256 features (UMMA N, each CTA loads half of them), so
// a step of 128 codes needs 32 KB of shared memory a CTA for 512 tensor cycles.
// The int32 accumulator takes 256 TMEM columns and is double-buffered: the
// epilogue of one tile runs under the main loop of the next.
//
// The epilogue reads TMEM in the fragment layout of the warp-level MMA
// (16x256b: a thread holds two neighbouring features of rows T / 4 and
// T / 4 + 8), scales to fp32, packs bf16 and stores through swizzled shared
// memory by TMA, which clips the ragged edges.
//
// With an adapter the scaled fp32 sums go back to the TMEM columns they came
// from; one bf16 MMA per 16 ranks then adds sU B^T (or sT A) in place, and a
// second read takes the finished values. The issuer slips that MMA in between
// the next tile's steps, so only the epilogue waits for it. Adding the term by
// warp-level MMAs in the epilogue instead stalls the tcgen05 stream, which
// shares the tensor cores: 4096 tokens 14336 x 4096 took 152 us without an
// adapter, 176 at rank 16 and 273 at rank 64.
//
// Bound by the tensor rate and, in long runs, by the board's power: 4096 tokens
// 14336 x 4096 at rank 16 takes 152 to 154 us in bursts of five calls after a pause
// (3.1 Pop/s, 95% of twice the measured bf16 rate), 175 to 181 in a long run under
// the cap; 4096 x 4096 49 us (256 tiles, 3.5 turns of 74 pairs). Below about 2048
// codes of contraction the epilogue sets the pace: 4096 x 1024 19 us without an
// adapter, 26 with one, and a third more on a board that is at its cap.
//
// Warps (384 threads): 0 TMA producer, 1 MMA issuer and TMEM owner, 2 adapter
// producer, 4-11 epilogue (TMEM lane quadrant warp % 4, half of the columns
// each).
#include <climits>

#include "i8_gemm.cuh"
#include "norm_i8.h"

namespace qlora {

bool encode_2d(CUtensorMap *map, CUtensorMapDataType dtype, const void *base, uint64_t inner, uint64_t outer,
               uint64_t row_bytes, uint32_t box_inner, uint32_t box_outer, CUtensorMapSwizzle swizzle);

namespace {

constexpr int kThreads = 384;
constexpr int kTile = 256;                                 // tokens per pair tile, and the most features
constexpr uint32_t kBoxBytes = 128 * kI8Step;              // 16 KiB: 128 tokens, or 128 features, of a step
constexpr int kMaxStages = 9;
constexpr uint32_t kOutBytes = 32 * 64;                    // 32 tokens x 32 features bf16, per epilogue warp
constexpr int kEpiWarps = 8;
constexpr int kMaxSmem = 227 * 1024;

struct PairParams {
  const float *act_scale, *w_scale;
  int32_t *status;
  int64_t M, F;
  int r_pad, stages;   // adapter ranks in shared memory (0, 16, 32 or 64), ring depth
  int feat;            // features per pair tile, a multiple of 32
  int nk, feat_tiles, tok_tiles;
};

// Shared memory: ring, epilogue staging, the adapter's two tiles (128 tokens
// and 128 features of r_pad ranks, bf16), barriers.
struct PairBars {
  uint64_t full[kMaxStages], empty[kMaxStages], accf[2], acce[2], loraf, lorae, scaled, added, drain;
  uint32_t tmem_holder;
  int abort_flag;
};
__host__ __device__ inline uint32_t lora_bytes(int r_pad) { return 128u * static_cast<uint32_t>(r_pad) * 2u; }
// A CTA's 128 tokens and its half of the features (DX: 128, of which it uses
// the first feat / 2) of a step.
__host__ __device__ inline uint32_t slot_bytes(bool dx, int feat) {
  return kBoxBytes + (dx ? kBoxBytes : static_cast<uint32_t>(feat / 2) * kI8Step);
}
__host__ __device__ inline uint32_t bars_offset(uint32_t slot, int stages, int r_pad) {
  return static_cast<uint32_t>(stages) * slot + kEpiWarps * kOutBytes + 2u * lora_bytes(r_pad);
}

// The reverse of tmem_ld_frag32.
__device__ __forceinline__ void tmem_st_frag32(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x4.b32 [%16], "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void stmatrix_x4(uint32_t saddr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(saddr), "r"(a), "r"(b), "r"(c),
               "r"(d)
               : "memory");
}

template <bool kDx, bool kLora>
__global__ void __launch_bounds__(kThreads, 1)
    i8_pair_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_act,
                   const __grid_constant__ CUtensorMap tm_out, const __grid_constant__ CUtensorMap tm_lora_w,
                   const __grid_constant__ CUtensorMap tm_lora_act, const PairParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t slot_sz = slot_bytes(kDx, p.feat), half_feat = static_cast<uint32_t>(p.feat) / 2u;
  uint8_t *out_stage = ring + static_cast<uint32_t>(p.stages) * slot_sz;
  uint8_t *lora_a = out_stage + kEpiWarps * kOutBytes, *lora_b = lora_a + lora_bytes(p.r_pad);
  PairBars &sm = *reinterpret_cast<PairBars *>(ring + bars_offset(slot_sz, p.stages, p.r_pad));
  volatile int *abort_flag = &sm.abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int ntiles = p.feat_tiles * p.tok_tiles;
  const int first = static_cast<int>(blockIdx.x >> 1), stride = static_cast<int>(gridDim.x >> 1);
  // tile -> (tokens, features): tokens fastest, so that the pairs at work share few weight tiles
  auto tok0 = [&](int tile) { return (tile % p.tok_tiles) * kTile; };
  auto feat0 = [&](int tile) { return (tile / p.tok_tiles) * p.feat; };

  if (threadIdx.x == 0) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&sm.full[i], 1);
      mbar_init(&sm.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.accf[i], 1);
      mbar_init(&sm.acce[i], 2 * kEpiWarps);
    }
    mbar_init(&sm.loraf, 1);
    mbar_init(&sm.lorae, 1);
    mbar_init(&sm.scaled, 2 * kEpiWarps);
    mbar_init(&sm.added, 1);
    mbar_init(&sm.drain, 1);
    sm.abort_flag = 0;
    fence_mbarrier_init();
    tma_prefetch_desc(&tm_w);
    tma_prefetch_desc(&tm_act);
    tma_prefetch_desc(&tm_out);
    if (kLora) {
      tma_prefetch_desc(&tm_lora_w);
      tma_prefetch_desc(&tm_lora_act);
    }
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
  grid_dep_launch();   // behind the allocation: a following kernel's CTAs do not take TMEM that this one still needs
  const Waited after = grid_dep_wait();

  if (warp == 0) {
    // ---------------- producer: this CTA's tokens and features ----------------
    if (elect_one()) {
      int slot = 0;
      uint32_t ph = 0, landed = 0, par = 0;
      bool ok = true;
      for (int tile = first; tile < ntiles && ok; tile += stride) {
        const int t0 = tok0(tile) + static_cast<int>(rank) * 128, f0 = feat0(tile) + static_cast<int>(rank * half_feat);
        for (int s = 0; s < p.nk; ++s) {
          if (!mbar_wait(&sm.empty[slot], ph ^ 1u, abort_flag, p.status)) {
            ok = false;
            break;
          }
          if (leader) mbar_arrive_expect_tx(&sm.full[slot], 2 * slot_sz);
          const uint32_t bar = mapa_shared(smem_u32(&sm.full[slot]), 0u);
          uint8_t *x = ring + static_cast<uint32_t>(slot) * slot_sz;
          tma_load_2d_pair(x, &tm_act, bar, s * kI8Step, t0);
          if (!kDx) tma_load_2d_pair(x + kBoxBytes, &tm_w, bar, s * kI8Step, f0);
          else      tma_load_2d_pair(x + kBoxBytes, &tm_w, bar, f0, s * kI8Step);
          landed |= 1u << slot;
          par = (par & ~(1u << slot)) | (ph << slot);
          if (++slot == p.stages) {
            slot = 0;
            ph ^= 1u;
          }
        }
      }
      if (!ok && leader)
        for (int i = 0; i < p.stages; ++i)
          if (landed & (1u << i)) drain_slot(&sm.full[i], (par >> i) & 1u);
    }
  } else if (warp == 2) {
    // ---------------- adapter producer: this CTA's tokens and features, once a tile ----------------
    if (kLora && elect_one()) {
      bool issued = false, ok = true;
      uint32_t ph = 0;
      const uint32_t bar = mapa_shared(smem_u32(&sm.loraf), 0u), span = 2u * static_cast<uint32_t>(p.r_pad);
      for (int tile = first; tile < ntiles; tile += stride, ph ^= 1u) {
        if (!mbar_wait(&sm.lorae, ph ^ 1u, abort_flag, p.status)) {
          ok = false;
          break;
        }
        const int t0 = tok0(tile) + static_cast<int>(rank) * 128, f0 = feat0(tile) + static_cast<int>(rank * half_feat);
        if (leader) mbar_arrive_expect_tx(&sm.loraf, 2 * (lora_bytes(p.r_pad) + (kDx ? 128u : half_feat) * span));
        tma_load_2d_pair(lora_a, &tm_lora_act, bar, 0, t0);
        if (!kDx) {
          tma_load_2d_pair(lora_b, &tm_lora_w, bar, 0, f0);
        } else {
          tma_load_2d_pair(lora_b, &tm_lora_w, bar, f0, 0);
          tma_load_2d_pair(lora_b + 128u * p.r_pad, &tm_lora_w, bar, f0 + 64, 0);
        }
        issued = true;
      }
      if (!ok && issued && leader) drain_slot(&sm.loraf, ph ^ 1u);
    }
  } else if (warp == 1) {
    // ---------------- MMA issuer (even CTA) ----------------
    if (leader && elect_one()) {
      const uint32_t idesc = idesc_i8(256, static_cast<uint32_t>(p.feat), false, kDx);
      const uint64_t a0 = smem_desc(smem_u32(ring), 16u, 1024u, kLayoutSW128);
      const uint64_t b0 = smem_desc(smem_u32(ring) + kBoxBytes, kDx ? kBoxBytes : 16u, 1024u, kLayoutSW128);
      // a step of 32 codes: +32 bytes along a K-major row, or 32 rows of 128 bytes (MN-major)
      constexpr uint32_t b_step = (kDx ? 32u * 128u : 32u) >> 4;
      // The adapter's MMAs into the scaled accumulator of the pair's tile i.
      const uint32_t span = 2u * static_cast<uint32_t>(p.r_pad);   // bytes of a K-major row of ranks
      const uint32_t lsw = span == 32u ? kLayoutSW32 : (span == 64u ? kLayoutSW64 : kLayoutSW128);
      auto add_lora = [&](int i) -> bool {
        if (!mbar_wait(&sm.loraf, static_cast<uint32_t>(i) & 1u, abort_flag, p.status)) return false;
        tc_fence_after();
        const uint32_t lidesc = idesc_bf16(256, static_cast<uint32_t>(p.feat), false, kDx);
        for (uint32_t j = 0; j < static_cast<uint32_t>(p.r_pad) / 16u; ++j) {
          const uint64_t ad = smem_desc(smem_u32(lora_a) + 32u * j, 16u, 8u * span, lsw);
          const uint64_t bd = kDx ? smem_desc(smem_u32(lora_b) + 2048u * j, 64u * span, 1024u, kLayoutSW128)
                                  : smem_desc(smem_u32(lora_b) + 32u * j, 16u, 8u * span, lsw);
          umma_bf16_pair(tmem + static_cast<uint32_t>(i & 1) * kTile, ad, bd, lidesc, 1u);
        }
        umma_commit_pair(&sm.lorae);
        umma_commit_pair(&sm.added);
        return true;
      };
      int slot = 0, n = 0, added = 0;   // added: tiles whose adapter term is issued
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
          if (kLora && added < n && mbar_test_wait(&sm.scaled, static_cast<uint32_t>(added) & 1u)) {
            if (!add_lora(added++)) {
              ok = false;
              break;
            }
          }
          if (!mbar_wait(&sm.full[slot], ph, abort_flag, p.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t off = (static_cast<uint32_t>(slot) * slot_sz) >> 4;
#pragma unroll
          for (uint32_t j = 0; j < kI8Step / 32; ++j)
            umma_i8_pair(d, a0 + off + j * 2u, b0 + off + j * b_step, idesc, s || j);
          umma_commit_pair(&sm.empty[slot]);
          if (++slot == p.stages) {
            slot = 0;
            ph ^= 1u;
          }
        }
        if (!ok) break;
        umma_commit_pair(&sm.accf[buf]);
        // the previous tile's term is due before its accumulator can be had again; after the last tile, its own too
        if (kLora)
          for (const int due = tile + stride < ntiles ? n : n + 1; added < due && ok;)
            ok = mbar_wait(&sm.scaled, static_cast<uint32_t>(added) & 1u, abort_flag, p.status) && add_lora(added++);
      }
      if (!ok) {   // the MMAs issued so far must be over before the CTA leaves
        umma_commit_pair(&sm.drain);
        drain_slot(&sm.drain, 0);
      }
    }
  } else if (warp >= 4) {
    // ---------------- epilogue ----------------
    const int quad = warp & 3, half = (warp - 4) >> 2;   // 32 tokens; every other chunk of 32 features
    uint8_t *stage = out_stage + static_cast<uint32_t>(warp - 4) * kOutBytes;
    const int g = lane >> 2, q2 = (lane & 3) * 2;        // fragment row and column pair
    const int chunks = p.feat / 32;
    const uint32_t t_warp = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    // this lane's stmatrix address for tokens h * 16 .. + 15: row of 64 bytes, swizzled 16-byte chunks
    auto st_addr = [&](int h, int j) -> uint32_t {
      const uint32_t row = static_cast<uint32_t>(h * 16 + (lane & 15)), chunk = static_cast<uint32_t>(j + (lane >> 4));
      return smem_u32(stage) + swizzle_off(row * 64u + chunk * 16u, 64u);
    };
    int n = 0;
    bool ok = true;
    for (int tile = first; tile < ntiles && ok; tile += stride, ++n) {
      const int buf = n & 1;
      const int64_t m0 = static_cast<int64_t>(tok0(tile)) + rank * 128 + quad * 32;
      const int64_t f0 = static_cast<int64_t>(feat0(tile));
      const uint32_t t_acc = t_warp + buf * kTile;
      float sx[4];   // tokens g, g + 8, g + 16, g + 24
#pragma unroll
      for (int i = 0; i < 4; ++i) sx[i] = m0 + g + 8 * i < p.M ? load_after(after, p.act_scale + m0 + g + 8 * i) : 0.f;
      float2 sw[4][4];   // the features of this warp's chunks
      if constexpr (!kDx) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int64_t f = f0 + (half + 2 * i) * 32 + j * 8 + q2;
            sw[i][j] = f < p.F ? load_after(after, reinterpret_cast<const float2 *>(p.w_scale + f)) : make_float2(0.f, 0.f);
          }
      }
      if (!__all_sync(0xffffffffu, mbar_wait(&sm.accf[buf], (n >> 1) & 1u, abort_flag, p.status))) {
        ok = false;
        break;
      }
      tc_fence_after();
      // sums to scaled fp32: the thread's 2 x 8 values of 32 features by 16 tokens (h: which 16)
      auto scale = [&](uint32_t (&v)[16], const float2 (&sw)[4], int h) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float y = static_cast<float>(static_cast<int>(v[4 * j + e])) * (h ? sx[2 + (e >> 1)] : sx[e >> 1]);
            if constexpr (!kDx) y *= (e & 1) ? sw[j].y : sw[j].x;
            v[4 * j + e] = __float_as_uint(y);
          }
      };
      if constexpr (kLora) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c = half + 2 * i;
          if (c >= chunks) break;
          uint32_t v[2][16];
          tmem_ld_frag32(t_acc + c * 32, v[0]);
          tmem_ld_frag32(t_acc + c * 32 + (16u << 16), v[1]);
          tmem_ld_wait();
          scale(v[0], sw[i], 0);
          tmem_st_frag32(t_acc + c * 32, v[0]);
          scale(v[1], sw[i], 1);
          tmem_st_frag32(t_acc + c * 32 + (16u << 16), v[1]);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&sm.scaled), 0u));
        if (!__all_sync(0xffffffffu, mbar_wait(&sm.added, static_cast<uint32_t>(n) & 1u, abort_flag, p.status))) {
          ok = false;
          break;
        }
        tc_fence_after();
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = half + 2 * i;
        if (c >= chunks) break;
        const int64_t fc = f0 + c * 32;
        uint32_t v[2][16];
        tmem_ld_frag32(t_acc + c * 32, v[0]);
        tmem_ld_frag32(t_acc + c * 32 + (16u << 16), v[1]);
        tmem_ld_wait();
        if (c + 2 >= chunks) {   // this warp's part is in registers: the next tile but one may have the accumulator
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&sm.acce[buf]), 0u));
        }
        // the staging tile is free again once the previous store has read it
        if (lane == 0) bulk_wait_group_read<0>();
        __syncwarp();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if constexpr (!kLora) scale(v[h], sw[i], h);
          auto pack = [&](int i) { return pack_bf16x2(__uint_as_float(v[h][i]), __uint_as_float(v[h][i + 1])); };
#pragma unroll
          for (int j = 0; j < 4; j += 2)
            stmatrix_x4(st_addr(h, j), pack(4 * j), pack(4 * j + 2), pack(4 * j + 4), pack(4 * j + 6));
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

using PairKernel = void(const CUtensorMap, const CUtensorMap, const CUtensorMap, const CUtensorMap, const CUtensorMap,
                        const PairParams);
template <bool kDx>
PairKernel *pair_fn(bool lora) {
  return lora ? i8_pair_kernel<kDx, true> : i8_pair_kernel<kDx, false>;
}

}  // namespace

cudaError_t launch_i8_pair(const I8GemmArgs &a, cudaStream_t st) {
  PairParams p{};
  p.act_scale = a.act_scale;
  p.w_scale = a.w_scale;
  p.status = a.status;
  p.M = a.M;
  p.F = a.F;
  p.r_pad = a.r == 0 ? 0 : (a.r <= 16 ? 16 : (a.r <= 32 ? 32 : 64));
  p.nk = static_cast<int>((a.C + kI8Step - 1) / kI8Step);
  p.tok_tiles = static_cast<int>((a.M + kTile - 1) / kTile);
  // Features per tile (FWD): the least waves times the bytes of a step, so that
  // a launch of less than one wave spreads over the SMs. DX loads 128 features a
  // CTA in any case (a swizzled row of the weight box): 256.
  const int64_t pairs = device_sm_count() / 2;
  p.feat = kTile;
  if (!a.dx) {
    int64_t best = LLONG_MAX;
    for (int feat = kTile; feat >= 96; feat -= 32) {
      const int64_t tiles = (a.F + feat - 1) / feat * p.tok_tiles, cost = (tiles + pairs - 1) / pairs * (kTile + feat);
      if (cost < best) {
        best = cost;
        p.feat = feat;
      }
    }
  }
  p.feat_tiles = static_cast<int>((a.F + p.feat - 1) / p.feat);
  const uint32_t slot = slot_bytes(a.dx, p.feat);
  // what 227 KB hold beside the staging, the adapter's tiles, the barriers and the alignment
  p.stages = static_cast<int>((static_cast<uint32_t>(kMaxSmem) - 1024u - 512u - bars_offset(slot, 0, p.r_pad)) / slot);
  if (p.stages > kMaxStages) p.stages = kMaxStages;

  CUtensorMap tm_w, tm_act, tm_out, tm_lora_w, tm_lora_act;
  const uint64_t wrow = static_cast<uint64_t>(a.dx ? a.F : a.C), wrows = static_cast<uint64_t>(a.dx ? a.C : a.F);
  bool ok = encode_2d(&tm_w, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.w, wrow, wrows, wrow, 128,
                      a.dx ? 128 : p.feat / 2, CU_TENSOR_MAP_SWIZZLE_128B);
  ok &= encode_2d(&tm_act, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.act, a.C, a.M, a.C, kI8Step, 128, CU_TENSOR_MAP_SWIZZLE_128B);
  ok &= encode_2d(&tm_out, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.out, a.F, a.M, a.F * 2, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B);
  tm_lora_w = tm_lora_act = tm_out;
  if (a.r) {
    const CUtensorMapSwizzle sw = p.r_pad == 16   ? CU_TENSOR_MAP_SWIZZLE_32B
                                  : p.r_pad == 32 ? CU_TENSOR_MAP_SWIZZLE_64B
                                                  : CU_TENSOR_MAP_SWIZZLE_128B;
    ok &= encode_2d(&tm_lora_act, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.lora_act, a.r, a.M, a.r * 2, p.r_pad, 128, sw);
    ok &= a.dx ? encode_2d(&tm_lora_w, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.lora_w, a.F, a.r, a.F * 2, 64, p.r_pad,
                           CU_TENSOR_MAP_SWIZZLE_128B)
               : encode_2d(&tm_lora_w, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.lora_w, a.r, a.F, a.r * 2, p.r_pad,
                           p.feat / 2, sw);
  }
  if (!ok) return cudaErrorInvalidValue;
  auto *fn = a.dx ? pair_fn<true>(a.r != 0) : pair_fn<false>(a.r != 0);
  static_assert(sizeof(PairBars) <= 512, "room kept for the barriers");
  const size_t smem = 1024 + bars_offset(slot, p.stages, p.r_pad) + sizeof(PairBars);
  const cudaError_t e = allow_smem(fn, kMaxSmem);
  if (e != cudaSuccess) return e;
  const int64_t tiles = static_cast<int64_t>(p.feat_tiles) * p.tok_tiles;
  return launch_dependent(fn, static_cast<unsigned>(2 * (tiles < pairs ? tiles : pairs)), kThreads, smem, st, 2, tm_w,
                          tm_act, tm_out, tm_lora_w, tm_lora_act, p);
}

// Single tiles of 128 x 128 as long as one wave of CTAs holds them; past that
// the pairs' 256 x 256 tiles, which need half the operand bytes per output. A
// little more than one wave of pairs goes back to single tiles, two to a SM.
// Measured (rank 16): 512 tokens 4096 x 4096 (128 tiles, 32 pair tiles) 11.0 us
// split, 11.8 pair; 768 tokens (192, 48) 18.2 and 14.8; 200 tokens 11008 x 4096
// (172, 43) 19.5 and 15.5; 384 tokens (258, 86) 20.5 and 21.5.
//
// Past rank 16 the single tiles' warp MMAs and fragment loads for the adapter cost
// more than the pairs' tcgen05 term: about 0.25 us (gradient: 0.38) for each
// further 16 ranks and block of 16 x 16 that a warp finishes, 8 / ways of them. The
// pairs start about 0.9 us later and do a tile's whole contraction in one place,
// at 0.13 us (0.32) a step where few tiles are at work, the CTAs of a cluster their
// part at 0.25 us. Measured at ranks 24, 32 and 64, split / pair (ways, steps):
//   tokens x features x contraction     forward                    gradient
//   4096 x 432 x 192 (1, 2)       7.6/7.1 8.2/6.8 14.6/6.9    9.7/10.2 9.9/10.1 14.6/10.0
//   300 x 4096 x 1024 (1, 8)      7.5/7.9 7.7/7.6 10.8/7.7    11.2/12.4 11.7/12.2 16.6/12.4
//   512 x 4096 x 4096 (1, 32)     12.7/12.4 12.8/12.0 16.0/12.2  20.0/21.8 20.4/21.3 25.5/21.8
//   700 x 1040 x 2064 (2, 17)     9.9/9.8 10.3/9.7 13.2/9.7   15.7/16.9 15.9/16.8 18.9/17.0
//   1024 x 1024 x 4096 (2, 32)    9.9/10.6 10.2/10.2 13.2/10.1  16.4/21.7 16.8/21.6 20.3/21.7
//   300 x 1040 x 2064 (4, 17)     7.9/9.6 7.9/9.5 8.8/9.5     11.8/16.3 11.9/16.2 13.1/16.4
//   256 x 1024 x 14336 (8, 112)   10.7/20.0 10.8/19.8 11.2/19.9  17.0/43.5 17.0/43.3 18.8/43.8
// Up to 128 tokens half of a pair's tile is empty: 100 x 1040 x 2064 7.3/9.0,
// 7.3/8.9, 7.9/8.9 and 9.3/14.0, 9.4/14.0, 10.7/14.2; one way and past rank 32 the
// pairs would be the faster ones there too (120 x 14336 x 4096 20.4/19.1, 25.3/22.2).
bool adapter_fits_split(const I8GemmArgs &a) {
  if (a.r <= 16 || a.M <= 128) return true;
  const int64_t nk = (a.C + kI8Step - 1) / kI8Step, ways = i8_split_ways(a.M, a.F, a.C);
  const int64_t adapter = (a.dx ? 38 : 25) * ((8 + ways - 1) / ways) * ((a.r + 15) / 16 - 1);   // in 10 ns
  return adapter <= 90 + (a.dx ? 32 : 13) * nk - 25 * ((nk + ways - 1) / ways);
}

cudaError_t launch_i8_gemm(const I8GemmArgs &a, cudaStream_t st) {
  auto tiles = [&](int64_t t) { return ((a.F + t - 1) / t) * ((a.M + t - 1) / t); };
  const int64_t sms = device_sm_count(), single = tiles(128);
  const bool split = (single <= sms || (single <= 2 * sms && tiles(kTile) > sms / 2)) && adapter_fits_split(a);
  return split ? launch_i8_split(a, st) : launch_i8_pair(a, st);
}

}  // namespace qlora
