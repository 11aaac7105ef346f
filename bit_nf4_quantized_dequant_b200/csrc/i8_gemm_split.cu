// Int8 GEMM with the contraction split over a cluster: the kernel for token
// counts that leave most SM pairs without an output tile of their own.
//
// One CTA holds a tile of 128 tokens (UMMA M) by 128 features (UMMA N); the
// CTAs of a cluster (1 to 8) take consecutive parts of the tile's contraction
// and their int32 partial sums are added over distributed shared memory.
// Integer sums are exact, so the result does not depend on the split. Few
// tokens are bound by the weight's bytes: the split brings enough CTAs to keep
// every SM loading. A token box has only the rows that exist (rounded up to
// 8): the MMA then reads past it into the weight box behind, which gives
// integers in accumulator rows that nobody reads.
//
// The accumulator is read in the fragment layout of the warp-level MMA (see
// i8_gemm_pair.cu) and cut into blocks of 16 tokens x 16 features; the CTAs of
// a cluster share the blocks that hold tokens, and each finishes its own:
// sum, scales, adapter (mma.m16n8k16), bf16, 32-byte row segments stored.
//
// Measured: one token of 14336 x 4096 12.0 us, 59 MB at 4.9 TB/s (0.30 us, 6.1
// TB/s, for each further step of the contraction; the rest is the launch, the
// filling of a pipeline and the epilogue); of 4096 x 4096 5.3 us, most of it those;
// 512 tokens of 4096 x 4096 11 us at rank 16. 301 tokens of 1040 x 2064, gradient,
// rank 8 (51 tiles of 9 steps): 11.4 us in all, of which quantising is 3.1; one
// step instead of nine takes 5.9.
//
// Warps: 0 TMA producer, 1 MMA issuer and TMEM owner; all eight finish.
#include <atomic>

#include "i8_gemm.cuh"
#include "norm_i8.h"

namespace qlora {

bool encode_2d(CUtensorMap *map, CUtensorMapDataType dtype, const void *base, uint64_t inner, uint64_t outer,
               uint64_t row_bytes, uint32_t box_inner, uint32_t box_outer, CUtensorMapSwizzle swizzle);

namespace {

constexpr int kThreads = 256;
constexpr int kTile = 128;                                // tokens and features per tile
constexpr uint32_t kWBytes = kTile * kI8Step;             // weight box of a step
constexpr int kMaxStages = 10;
constexpr int kMaxSplit = 8;

struct SplitParams {
  const float *act_scale, *w_scale;
  const uint16_t *lora_act, *lora_w;
  uint16_t *out;
  int32_t *status;
  int64_t M, F;
  int r, rows, stages, nk, feat_tiles, split;   // rows: tokens of an activation box
};

__host__ __device__ inline uint32_t slot_bytes(int rows) { return kWBytes + static_cast<uint32_t>(rows) * kI8Step; }
// the ring, later the partial sums: 16 x 16 blocks of 1 KiB, eight a row of blocks
__host__ __device__ inline uint32_t ring_bytes(int rows, int stages, int split) {
  const uint32_t ring = static_cast<uint32_t>(stages) * slot_bytes(rows);
  const uint32_t part = split > 1 ? static_cast<uint32_t>((rows + 15) / 16) * 8u * 1024u : 0u;
  return ring > part ? ring : part;
}

__device__ __forceinline__ int4 ld_dsmem_int4(uint32_t addr) {
  int4 v;
  asm volatile("ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// What a thread needs besides the sums to finish a block: of its two tokens the
// scales and the adapter's fragments, and the same of its four features.
template <int kSteps>
struct RowOperands {
  float sx[2];
  uint32_t u[kSteps ? kSteps : 1][4];

  __device__ __forceinline__ void load(Waited after, const SplitParams &p, int64_t m0, int lane) {
    const int g = lane >> 2, q2 = (lane & 3) * 2;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t m = m0 + g + 8 * i;
      sx[i] = m < p.M ? load_after(after, p.act_scale + m) : 0.f;
#pragma unroll
      for (int ks = 0; ks < kSteps; ++ks)
#pragma unroll
        for (int c = 0; c < 2; ++c) u[ks][i + 2 * c] = lora_act_pair(after, p.lora_act, p.M, p.r, m, ks * 16 + c * 8 + q2);
    }
  }
};
template <bool kDx, int kSteps>
struct ColOperands {
  float2 sw[2];
  uint32_t b[kSteps ? kSteps : 1][2][2];

  __device__ __forceinline__ void load(Waited after, const SplitParams &p, int64_t f0, int lane) {
    const int g = lane >> 2, q2 = (lane & 3) * 2;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t f = f0 + 8 * i + q2;
      sw[i] = make_float2(1.f, 1.f);
      if (!kDx && f < p.F) sw[i] = load_after(after, reinterpret_cast<const float2 *>(p.w_scale + f));
#pragma unroll
      for (int ks = 0; ks < kSteps; ++ks)
#pragma unroll
        for (int c = 0; c < 2; ++c)
          b[ks][i][c] = lora_w_pair<kDx>(after, p.lora_w, p.F, p.r, f0 + 8 * i + g, ks * 16 + c * 8 + q2);
    }
  }
};
// s: the block's sums, fragment by fragment
template <bool kDx, int kSteps>
__device__ __forceinline__ void finish_block(const SplitParams &p, int64_t m0, int64_t f0, int lane, const int (&s)[8],
                                             const RowOperands<kSteps> &row, const ColOperands<kDx, kSteps> &col) {
  const int g = lane >> 2, q2 = (lane & 3) * 2;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    float y[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      y[e] = static_cast<float>(s[4 * j + e]) * row.sx[e >> 1];
      if constexpr (!kDx) y[e] *= (e & 1) ? col.sw[j].y : col.sw[j].x;
    }
#pragma unroll
    for (int ks = 0; ks < kSteps; ++ks) mma_16816(y, row.u[ks], col.b[ks][j][0], col.b[ks][j][1]);
    const int64_t f = f0 + 8 * j + q2;
    if (f < p.F) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int64_t m = m0 + g + 8 * i;
        if (m < p.M) *reinterpret_cast<uint32_t *>(p.out + m * p.F + f) = pack_bf16x2(y[2 * i], y[2 * i + 1]);
      }
    }
  }
}

template <bool kDx, int kSteps>
__global__ void __launch_bounds__(kThreads, 2)
    i8_split_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_act,
                    const SplitParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t *full = reinterpret_cast<uint64_t *>(ring + ring_bytes(p.rows, p.stages, p.split));
  uint64_t *empty = full + kMaxStages;
  uint64_t *done = empty + kMaxStages;
  uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(done + 1);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = p.split;
  const int rank = split > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int tile = static_cast<int>(blockIdx.x) / split;
  const int ft = tile % p.feat_tiles, tt = tile / p.feat_tiles;
  const int64_t f0 = static_cast<int64_t>(ft) * kTile, t0 = static_cast<int64_t>(tt) * kTile;
  const int s0 = p.nk * rank / split, s1 = p.nk * (rank + 1) / split;
  const uint32_t act_bytes = static_cast<uint32_t>(p.rows) * kI8Step, slot_sz = slot_bytes(p.rows);

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
    tmem_alloc(tmem_holder, kTile);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  grid_dep_launch();   // behind the allocation: a following kernel's CTAs do not take TMEM that this one still needs
  const Waited after = grid_dep_wait();

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
        mbar_arrive_expect_tx(&full[slot], slot_sz);
        uint8_t *x = ring + static_cast<uint32_t>(slot) * slot_sz;
        tma_load_2d(x, &tm_act, &full[slot], s * kI8Step, static_cast<int32_t>(t0));
        if (!kDx) tma_load_2d(x + act_bytes, &tm_w, &full[slot], s * kI8Step, static_cast<int32_t>(f0));
        else      tma_load_2d(x + act_bytes, &tm_w, &full[slot], static_cast<int32_t>(f0), s * kI8Step);
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
      constexpr uint32_t idesc = idesc_i8(kTile, kTile, false, kDx);
      // a step of 32 codes: +32 bytes along a K-major row, or 32 rows of 128 bytes (MN-major)
      const uint64_t a0 = smem_desc(smem_u32(ring), 16u, 1024u, kLayoutSW128);
      const uint64_t b0 = smem_desc(smem_u32(ring) + act_bytes, kDx ? kWBytes : 16u, 1024u, kLayoutSW128);
      constexpr uint32_t b_step = (kDx ? 32u * 128u : 32u) >> 4;
      int slot = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int s = s0; s < s1; ++s) {
        if (!mbar_wait(&full[slot], ph, abort_flag, p.status)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint64_t off = (static_cast<uint32_t>(slot) * slot_sz) >> 4;
#pragma unroll
        for (uint32_t j = 0; j < kI8Step / 32; ++j)
          umma_i8(tmem, a0 + off + j * 2u, b0 + off + j * b_step, idesc, s > s0 || j);
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
  }
  __syncwarp();

  // ---- this warp's part of the accumulator: tokens 32 quad .. + 31, features 64 half .. + 63 ----
  const int quad = warp & 3, half = warp >> 2;
  const int tokens = static_cast<int>(p.M - t0 < kTile ? p.M - t0 : kTile);
  RowOperands<kSteps> row;
  if (split > 1) {
    // blocks (row of blocks rb, column of blocks cb) that hold tokens, dealt out to the cluster's warps
    const int blocks = (tokens + 15) / 16 * 8, step = split * (kThreads / 32);
    int b = warp * split + rank;
    ColOperands<kDx, kSteps> col;
    auto load = [&](int b) {
      row.load(after, p, t0 + (b >> 3) * 16, lane);
      col.load(after, p, f0 + (b & 7) * 16, lane);
    };
    if (b < blocks) load(b);   // under the main loop
    int4 *part = reinterpret_cast<int4 *>(ring);   // [block][2][lane]
    // the TMEM loads are warp-wide: every lane takes the same way
    if (__all_sync(0xffffffffu, mbar_wait(done, 0, abort_flag, p.status))) {
      tc_fence_after();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (quad * 32 + h * 16 < tokens) {
          uint32_t v[32];
          tmem_ld_frag64(tmem + (static_cast<uint32_t>(quad * 32 + h * 16) << 16) + half * 64, v);
          tmem_ld_wait();
          int4 *d = part + ((quad * 2 + h) * 8 + half * 4) * 64 + lane;
#pragma unroll
          for (int j = 0; j < 8; ++j)
            d[j * 32] = make_int4(static_cast<int>(v[4 * j]), static_cast<int>(v[4 * j + 1]),
                                  static_cast<int>(v[4 * j + 2]), static_cast<int>(v[4 * j + 3]));
        }
      }
      tc_fence_before();
    }
    __syncwarp();
    cluster_sync_all();
    if (!*abort_flag) {
      const uint32_t mine = smem_u32(part) + static_cast<uint32_t>(lane) * 16u;
      for (; b < blocks; b += step) {
        int s[8] = {};
#pragma unroll
        for (int q = 0; q < kMaxSplit; ++q)
          if (q < split) {
            const uint32_t at = mapa_shared(mine + static_cast<uint32_t>(b) * 1024u, static_cast<uint32_t>(q));
            const int4 lo = ld_dsmem_int4(at), hi = ld_dsmem_int4(at + 512u);
            s[0] += lo.x; s[1] += lo.y; s[2] += lo.z; s[3] += lo.w;
            s[4] += hi.x; s[5] += hi.y; s[6] += hi.z; s[7] += hi.w;
          }
        finish_block(p, t0 + (b >> 3) * 16, f0 + (b & 7) * 16, lane, s, row, col);
        if (b + step < blocks) load(b + step);
      }
    }
    // no CTA leaves while a peer may still read its partial sums
    cluster_sync_all();
  } else {
    // all four blocks' features under the main loop, where they fit the registers: an
    // ordinary load does not pass the stores of the block before
    constexpr int kHeld = kSteps <= 1 ? 4 : 1;
    ColOperands<kDx, kSteps> col[kHeld];
    if (quad * 32 < tokens) {
      row.load(after, p, t0 + quad * 32, lane);
#pragma unroll
      for (int c = 0; c < kHeld; ++c) col[c].load(after, p, f0 + half * 64 + c * 16, lane);
    }
    if (__all_sync(0xffffffffu, mbar_wait(done, 0, abort_flag, p.status))) {
      tc_fence_after();
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        const int64_t m0 = t0 + quad * 32 + h * 16;
        if (quad * 32 + h * 16 >= tokens) break;
        uint32_t v[32];
        if (h) row.load(after, p, m0, lane);
        tmem_ld_frag64(tmem + (static_cast<uint32_t>(quad * 32 + h * 16) << 16) + half * 64, v);
        tmem_ld_wait();
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          int s[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) s[e] = static_cast<int>(v[8 * c + e]);
          if (kHeld == 1 && (h || c)) col[0].load(after, p, f0 + half * 64 + c * 16, lane);
          finish_block(p, m0, f0 + half * 64 + c * 16, lane, s, row, col[kHeld == 1 ? 0 : c]);
        }
      }
      tc_fence_before();
    }
    __syncthreads();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTile);
  }
}

using SplitKernel = void(const CUtensorMap, const CUtensorMap, const SplitParams);
template <bool kDx>
SplitKernel *split_fn(int steps) {
  switch (steps) {
    case 0: return i8_split_kernel<kDx, 0>;
    case 1: return i8_split_kernel<kDx, 1>;
    case 2: return i8_split_kernel<kDx, 2>;
    case 3: return i8_split_kernel<kDx, 3>;
    default: return i8_split_kernel<kDx, 4>;
  }
}

}  // namespace

// Clusters of `split` CTAs that the current device holds at a time, one CTA a
// SM: what the driver says, asked once a device and size.
static int resident_clusters(int split) {
  static std::atomic<int> known[64][kMaxSplit + 1];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  int n = known[dev][split].load(std::memory_order_relaxed);
  if (n == 0) {
    auto *fn = i8_split_kernel<false, 0>;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(split * device_sm_count()));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = 200 * 1024;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(split);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (allow_smem(fn) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, fn, &cfg) != cudaSuccess || n < 1) {
      cudaGetLastError();   // no answer is no reason to fail: no split
      n = 1;
    }
    known[dev][split].store(n, std::memory_order_relaxed);
  }
  return n;
}

// As many CTAs as there are SMs, each with about four steps or more. Measured
// with one token of 4096 x 4096 (32 tiles of 32 steps): 4 ways 5.2 us, 3 ways
// 5.5, 2 ways 5.7, one 7.0, 8 ways (two CTAs a SM) 5.8; 1024 x 4096: 8 ways 4.0, 4
// ways 4.6; 14336 x 4096 (112 tiles): one 11.9, 2 ways 14.2, 4 ways 17.4. The
// gradient of 301 tokens 1040 x 2064 takes 11.4 us with its 2 ways, 10.7 with one
// and 12.4 with 4.
// A cluster stays inside one GPC, which leaves some SMs out: see resident_clusters.
int i8_split_ways(int64_t M, int64_t F, int64_t C) {
  const int64_t tiles = ((F + kTile - 1) / kTile) * ((M + kTile - 1) / kTile), nk = (C + kI8Step - 1) / kI8Step;
  int split = static_cast<int>((nk + 3) / 4 < kMaxSplit ? (nk + 3) / 4 : kMaxSplit);
  while (split > 1 && tiles > resident_clusters(split)) --split;
  return split;
}

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
  p.rows = a.M >= kTile ? kTile : static_cast<int>((a.M + 7) / 8 * 8);
  p.nk = static_cast<int>((a.C + kI8Step - 1) / kI8Step);
  p.feat_tiles = static_cast<int>((a.F + kTile - 1) / kTile);
  const int64_t tiles = static_cast<int64_t>(p.feat_tiles) * ((a.M + kTile - 1) / kTile);
  p.split = i8_split_ways(a.M, a.F, a.C);
  const int per_cta = (p.nk + p.split - 1) / p.split;
  // two CTAs a SM where there are more than SMs, else one with a deeper ring
  const uint32_t room = (tiles * p.split > device_sm_count() ? 108u : 200u) * 1024u;
  p.stages = static_cast<int>(room / slot_bytes(p.rows));
  if (p.stages > kMaxStages) p.stages = kMaxStages;
  if (p.stages > per_cta) p.stages = per_cta;
  const size_t smem = 1024 + ring_bytes(p.rows, p.stages, p.split) + (2 * kMaxStages + 1) * 8 + 16;

  CUtensorMap tm_w, tm_act;
  const uint64_t wrow = static_cast<uint64_t>(a.dx ? a.F : a.C), wrows = static_cast<uint64_t>(a.dx ? a.C : a.F);
  bool ok = encode_2d(&tm_w, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.w, wrow, wrows, wrow, 128, 128, CU_TENSOR_MAP_SWIZZLE_128B);
  ok &= encode_2d(&tm_act, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.act, a.C, a.M, a.C, kI8Step, p.rows,
                  CU_TENSOR_MAP_SWIZZLE_128B);
  if (!ok) return cudaErrorInvalidValue;
  const int steps = (a.r + 15) / 16;
  auto *fn = a.dx ? split_fn<true>(steps) : split_fn<false>(steps);
  const cudaError_t e = allow_smem(fn);
  if (e != cudaSuccess) return e;
  return launch_dependent(fn, static_cast<unsigned>(tiles * p.split), kThreads, smem, st, p.split, tm_w, tm_act, p);
}

}  // namespace qlora
