// train_kernel.cuh -- persistent, warp-specialised tcgen05 products of the
// training-side operators: the head's logits with a softmax cross-entropy
// epilogue, and the gradient products, whose operands lie transposed in memory.
//
//   D[m][n] = sum_k a(m,k) * b(n,k),  BF16 operands, FP32 accumulation in tensor memory
//
// Each operand is either K-major (row m holds consecutive k: rows of X, W, dD)
// or MN-major (row k holds consecutive m or n: the same matrices read for
// their gradients).  A stage holds 64 k of a tile.  K-major tiles are rows of
// 128 bytes (64 k), 128-byte swizzle; MN-major tiles are chunks of 64 m (or n)
// by 64 k, each k a 128-byte row under the same swizzle, so that both kinds
// take the same shared memory and TMA writes both directly: nothing is ever
// transposed in memory.  The MMA descriptors carry the difference.
//
// Roles (one CTA per SM; CG CTAs per cluster share one MMA when CG == 2), the
// bounded waits and the abort protocol are those of gemm_kernel.cuh:
//   warp 0 TMA producer, warp 1 MMA issuer, warp 2 tensor-memory allocation and
//   the cluster-launch-control tile scheduler, warps 4-11 epilogue.
// Two 256-column accumulators: a tile's epilogue overlaps the next tile's MMAs.
//
// Epilogues (EPI):
//   LOSS     a thread owns 128 consecutive logits of one row: their maximum and
//            sum of exponentials in base 2 (one FFMA and one ex2 per logit) and,
//            where the row's label falls among them, its logit.  8 bytes per 128
//            logits go to memory, never the logits.
//   DLOGITS  g = (exp(z - lse) - [v = label]) * alpha * dloss, rounded to BF16 (the
//            tensor cores' operand type; each g carries a relative error of at
//            most 2^-9, independent between elements), by TMA into a piece.
//   BF16     alpha * D rounded to nearest even.
//   F32      alpha * D stored, or added by the TMA unit to what is there (one add
//            per element and launch, so the order of additions is fixed).
#pragma once
#include "gemm_kernel.cuh"

namespace tkg {

enum : int { EPI_LOSS = 0, EPI_DLOGITS = 1, EPI_BF16 = 2, EPI_F32 = 3 };
// GRP_ROWS: groups of consecutive output rows, each with its own B; GRP_K: groups
// of consecutive k, each with its own output matrix.  Row counts in device memory.
enum : int { GRP_NONE = 0, GRP_ROWS = 1, GRP_K = 2 };

struct TrainParams {
  int m, n, k;                 // output rows and columns, contraction length (GRP_K: row capacity)
  int kstages;                 // ceil(k / 64)
  int splits, split_stages;    // k split: part z covers stages [z * split_stages, ...)
  int tiles_m, tiles_n, num_tiles;
  int raster_group;
  uint32_t tx_bytes;           // bytes landing on the (leader's) full barrier per stage
  float alpha;
  unsigned int* status;
  unsigned long long timeout_ns;
  int inject_stall;
  // cross entropy
  float c2;                    // alpha * log2(e)
  int vocab0, vocab;           // first vocabulary entry of this piece, and all there are
  const long long* labels;
  const float* lse;
  const float* dloss;
  float2* part;                // LOSS: (maximum, sum) per 128 columns and row
  float* zlabel;               // LOSS: the label's logit per row
  // F32
  int accumulate;
  // groups
  const int* sizes;            // device
  int groups;
  void* d;                     // GRP_ROWS: D for the row-masked stores at group ends
  const uint8_t* maps;         // GRP_K: tensor maps of A and B per group (256 bytes each)
};

namespace ptx {
__device__ __forceinline__ void tma_store_3d(const void* tmap, uint32_t src, int32_t x, int32_t y, int32_t z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(tmap),
               "r"(x), "r"(y), "r"(z), "r"(src)
               : "memory");
}
__device__ __forceinline__ void tma_add_3d(const void* tmap, uint32_t src, int32_t x, int32_t y, int32_t z) {
  asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                   tmap),
               "r"(x), "r"(y), "r"(z), "r"(src)
               : "memory");
}
// Before a tensor map written by an earlier kernel is used.
__device__ __forceinline__ void tmap_acquire(const void* tmap) {
  asm volatile("fence.proxy.tensormap::generic.acquire.gpu [%0], 128;" ::"l"(tmap) : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
}  // namespace ptx

// MN-major operand: 64-element chunks kTrainChunk bytes apart, 8-k groups 1024 bytes apart, 128-byte swizzle.
constexpr int kTrainChunk = 64 * 128;
__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t addr) {
  return uint64_t((addr >> 4) & 0x3FFF) | (uint64_t(kTrainChunk >> 4) << 16) | (uint64_t(1024 >> 4) << 32) |
         (1ull << 46) | (2ull << 61);
}

template <bool A_MN, bool B_MN, int EPI, int CG, int GRP>
struct TrainConfig {
  static constexpr int kThreads = 384;
  static constexpr int kEpiWarps = 8;
  static constexpr int kBN = 256;
  static constexpr int kMmaM = 128 * CG;
  static constexpr int kBRows = kBN / CG;           // n of B held by each CTA
  static constexpr int kStages = CG == 2 ? 6 : 4;
  static constexpr int kAcc = 2;
  static constexpr int kABytes = 128 * 128;
  static constexpr int kBBytes = kBRows * 128;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kEpiBufBytes = 32 * 64;      // 32 rows x 32 BF16 (or 16 FP32)
  static constexpr int kEpiBytes = EPI == EPI_LOSS ? 0 : kEpiWarps * 2 * kEpiBufBytes;
  static constexpr int kBarOffset = kStages * kStageBytes + kEpiBytes;
  static constexpr int kNumBars = 2 * kStages + 2 * kAcc + 2 + 4;
  static constexpr int kSmemBytes = kBarOffset + kNumBars * 8 + 2 * 16 + 16 + 1024;
  static constexpr bool kClc = GRP != GRP_ROWS;     // GRP_ROWS: the tile count is known on the device only
  static constexpr int kClcConsumers = CG * (1 + kEpiWarps) + 2;
  // GRP_ROWS: first tile, first row and rows per group, tile count; GRP_K: group and rows by rank
  static constexpr int kTabInts = GRP == GRP_ROWS ? 3 * kMaxGroups + 1 : (GRP == GRP_K ? 2 * kMaxGroups : 1);
  static constexpr uint32_t kIdesc =
      idesc_f16(kMmaM, kBN) | (A_MN ? 1u << 15 : 0u) | (B_MN ? 1u << 16 : 0u);
  static_assert(kSmemBytes + kTabInts * 4 + 64 <= 232448, "shared memory overflow");
};

struct TrainTile {
  int mb, nb;
  int a0, b0;        // this CTA's first m of A and first n of B
  int row_limit;     // output rows at or past this one are not stored
  int z;             // k part (GRP_NONE) or group
  int ks0, nks;      // first k stage and number of stages
  int k_end;         // contraction stops here
};

template <bool A_MN, bool B_MN, int EPI, int CG, int GRP>
__global__ void __launch_bounds__(384, 1)
    train_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                 const __grid_constant__ CUtensorMap tmD, const TrainParams p) {
  using C = TrainConfig<A_MN, B_MN, EPI, CG, GRP>;
  constexpr int STAGES = C::kStages;
  constexpr int ACC = C::kAcc;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint32_t s_tmem_base;
  __shared__ int s_abort;
  __shared__ int s_tab[C::kTabInts];

  ptx::pdl_launch_dependents();
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = (CG == 2) ? ptx::cluster_ctarank() : 0u;
  const bool leader = rank == 0;

  const uint32_t raw = ptx::smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  auto stage_a = [&](uint32_t s) { return base + s * uint32_t(C::kStageBytes); };
  auto stage_b = [&](uint32_t s) { return base + s * uint32_t(C::kStageBytes) + uint32_t(C::kABytes); };
  const uint32_t epi_base = base + uint32_t(STAGES * C::kStageBytes);
  const uint32_t bars = base + uint32_t(C::kBarOffset);
  auto full_bar = [&](uint32_t s) { return bars + 8u * s; };
  auto empty_bar = [&](uint32_t s) { return bars + 8u * (uint32_t(STAGES) + s); };
  auto accf_bar = [&](uint32_t a) { return bars + 8u * (uint32_t(2 * STAGES) + a); };
  auto acce_bar = [&](uint32_t a) { return bars + 8u * (uint32_t(2 * STAGES + ACC) + a); };
  const uint32_t drain_bar = bars + uint32_t(8 * (2 * STAGES + 2 * ACC));
  const uint32_t never_bar = drain_bar + 8;
  auto clc_full = [&](uint32_t i) { return never_bar + 8u + 8u * i; };
  auto clc_empty = [&](uint32_t i) { return never_bar + 24u + 8u * i; };
  auto clc_resp = [&](uint32_t i) { return ((never_bar + 40u + 15u) & ~15u) + 16u * i; };

  auto coords = [&](int t) {
    TrainTile tc;
    if constexpr (GRP == GRP_ROWS) {
      // last group whose first tile is <= t (empty groups are skipped)
      int lo = 0, hi = p.groups;
#pragma unroll 1
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_tab[mid] <= t) lo = mid; else hi = mid;
      }
      const int rows = s_tab[2 * kMaxGroups + lo];
      tile_coords(t - s_tab[lo], (rows + C::kMmaM - 1) / C::kMmaM, p.tiles_n, p.raster_group, tc.mb, tc.nb);
      tc.a0 = s_tab[kMaxGroups + lo] + tc.mb * C::kMmaM + int(rank) * 128;
      tc.row_limit = min(s_tab[kMaxGroups + lo] + rows, p.m);
      tc.z = lo;
      tc.ks0 = 0;
      tc.nks = p.kstages;
      tc.k_end = p.k;
    } else {
      const int per = p.tiles_m * p.tiles_n;
      const int z = t / per;
      tile_coords(t - z * per, p.tiles_m, p.tiles_n, p.raster_group, tc.mb, tc.nb);
      tc.a0 = tc.mb * C::kMmaM + int(rank) * 128;
      tc.row_limit = p.m;
      if constexpr (GRP == GRP_K) {   // the groups with most rows first
        tc.z = s_tab[z];
        tc.k_end = s_tab[kMaxGroups + z];
        tc.ks0 = 0;
        tc.nks = (tc.k_end + 63) >> 6;
      } else {
        tc.z = z;
        tc.ks0 = z * p.split_stages;
        tc.nks = min(p.split_stages, p.kstages - tc.ks0);
        tc.k_end = p.k;
      }
    }
    tc.b0 = tc.nb * C::kBN + int(rank) * C::kBRows;
    return tc;
  };

  if (threadIdx.x == 0) {
    s_abort = 0;
    for (uint32_t s = 0; s < uint32_t(STAGES); ++s) {
      ptx::mbar_init(full_bar(s), 1);
      ptx::mbar_init(empty_bar(s), 1);
    }
    for (uint32_t a = 0; a < uint32_t(ACC); ++a) {
      ptx::mbar_init(accf_bar(a), 1);
      ptx::mbar_init(acce_bar(a), CG * C::kEpiWarps);
    }
    ptx::mbar_init(drain_bar, 1);
    ptx::mbar_init(never_bar, 1);
    for (uint32_t i = 0; i < 2; ++i) {
      ptx::mbar_init(clc_full(i), 1);
      ptx::mbar_init(clc_empty(i), C::kClcConsumers);
    }
    ptx::fence_mbar_init();
    if (GRP != GRP_K) {
      ptx::prefetch_tmap(&tmA);
      ptx::prefetch_tmap(&tmB);
    }
    if (EPI != EPI_LOSS) ptx::prefetch_tmap(&tmD);
  }
  if (warp == 2) {
    ptx::tmem_alloc<CG>(ptx::smem_u32(&s_tmem_base), 512u);
    ptx::tmem_relinquish<CG>();
  }
  ptx::tc_fence_before();
  __syncthreads();
  // see gemm_kernel.cuh: the barriers' initialisation is published by its fence
  if (CG == 2) ptx::cluster_sync_relaxed();
  ptx::tc_fence_after();
  const uint32_t tmem = s_tmem_base;

  // Dependency wait: the roles that read global memory or hand out work wait for
  // the previous grid, as in gemm_kernel.cuh; with group sizes the whole CTA.
  int num_tiles = p.num_tiles;
  if constexpr (GRP != GRP_NONE) {
    ptx::pdl_wait();
    // sizes may have been cached by this SM before the previous grid wrote them: read through L2
    const int g = threadIdx.x;
    if constexpr (GRP == GRP_ROWS) {
      if (warp == 3) {
        int carry_t = 0, carry_r = 0;
#pragma unroll 1
        for (int g0 = 0; g0 < p.groups; g0 += 32) {
          const int gg = g0 + lane;
          // sums stop at the capacity: rows past it are cut off, and nothing leaves 32 bits
          const uint32_t cap = uint32_t(p.m);
          uint32_t sr = gg < p.groups ? min(uint32_t(max(__ldcg(p.sizes + gg), 0)), cap) : 0u;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const uint32_t x = __shfl_up_sync(0xffffffffu, sr, o);
            if (lane >= o) sr = min(sr + x, cap);
          }
          const int end = int(min(uint32_t(carry_r) + sr, cap));
          int before = __shfl_up_sync(0xffffffffu, end, 1);
          if (lane == 0) before = carry_r;
          const int rows = end - before;
          int tl = ((rows + C::kMmaM - 1) / C::kMmaM) * p.tiles_n;
          const int mine = tl;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, tl, o);
            if (lane >= o) tl += x;
          }
          if (gg < p.groups) {
            s_tab[gg] = carry_t + tl - mine;
            s_tab[kMaxGroups + gg] = before;
            s_tab[2 * kMaxGroups + gg] = rows;
          }
          carry_t += __shfl_sync(0xffffffffu, tl, 31);
          carry_r = __shfl_sync(0xffffffffu, end, 31);
        }
        if (lane == 0) s_tab[3 * kMaxGroups] = carry_t;
      }
    } else {
      // (group, rows) by rank, written next to the groups' tensor maps
      const int* tab = reinterpret_cast<const int*>(p.maps + size_t(p.groups) * 256);
      if (g < p.groups) {
        s_tab[g] = __ldcg(tab + g);
        s_tab[kMaxGroups + g] = __ldcg(tab + kMaxGroups + g);
      }
    }
    __syncthreads();
    if constexpr (GRP == GRP_ROWS) num_tiles = s_tab[3 * kMaxGroups];
  }

  Ctl ctl;
  ctl.abort_flag = &s_abort;
  ctl.abort_smem = ptx::smem_u32(&s_abort);
  ctl.rank = rank;
  ctl.ncta = CG;
  ctl.status = p.status;
  ctl.timeout_ns = p.timeout_ns;

  const int cluster_id = blockIdx.x / CG;
  const int num_clusters = gridDim.x / CG;
  const int first_tile = cluster_id < num_tiles ? cluster_id : -1;

  // Next tile: a fixed stride (GRP_ROWS), or the tile of a cluster not yet
  // started (cluster launch control, one cluster per tile).  -1: none left,
  // -2: aborting.  WARP: called by a whole converged warp.
  auto next_tile = [&](auto whole_warp, int t, uint32_t& cslot, uint32_t& cphase) -> int {
    [[maybe_unused]] constexpr bool WARP = decltype(whole_warp)::value;
    if constexpr (!C::kClc) {
      return t + num_clusters < num_tiles ? t + num_clusters : -1;
    } else {
      if (!(WARP ? wait_bar_warp<false>(clc_full(cslot), cphase, ctl) : wait_bar<false>(clc_full(cslot), cphase, ctl)))
        return -2;
      uint32_t x = 0;
      const bool got = ptx::clc_read(clc_resp(cslot), x);
      if constexpr (WARP) __syncwarp();
      if (!WARP || lane == 0) {
        if (leader)
          ptx::mbar_arrive(clc_empty(cslot));
        else
          ptx::mbar_arrive_relaxed_cluster(ptx::map_to_rank(clc_empty(cslot), 0));
      }
      if (++cslot == 2) {
        cslot = 0;
        cphase ^= 1u;
      }
      return got ? int(x) / CG : -1;
    }
  };
  using Lane = std::false_type;
  using Warp = std::true_type;

  // ------------------------------------------------------------------ producer
  if (warp == 0) {
    if (ptx::elect_one()) {
      const uint64_t pol_a = ptx::policy_evict_normal();
      const uint64_t pol_b = ptx::policy_evict_normal();
      const uint32_t lead_full0 = (CG == 2) ? ptx::map_to_rank(full_bar(0), 0) : full_bar(0);
      uint32_t stage = 0, phase = 0;
      uint32_t armed = 0, armed_par = 0;   // stages whose last arming is not yet known complete, and its parity
      bool ok = true;
      uint32_t cslot = 0, cphase = 0;
      if (GRP == GRP_NONE) ptx::pdl_wait();
#pragma unroll 1
      for (int t = first_tile; t >= 0 && ok;) {
        const TrainTile tc = coords(t);
        const void* mA = &tmA;
        const void* mB = &tmB;
        if constexpr (GRP == GRP_K) {
          mA = p.maps + size_t(tc.z) * 256;
          mB = p.maps + size_t(tc.z) * 256 + 128;
          if (tc.nks > 0) {
            ptx::tmap_acquire(mA);
            ptx::tmap_acquire(mB);
          }
        }
#pragma unroll 1
        for (int it = 0; it < tc.nks; ++it) {
          const int k0 = (tc.ks0 + it) * 64;
          if (!wait_bar<false>(empty_bar(stage), phase ^ 1u, ctl)) {
            ok = false;
            break;
          }
          armed &= ~(1u << stage);
          const uint32_t fb = lead_full0 + 8u * stage;
          if (leader) {
            ptx::mbar_arrive_expect_tx(full_bar(stage), p.tx_bytes);
            armed |= 1u << stage;
            armed_par = (armed_par & ~(1u << stage)) | (phase << stage);
          }
          if (invariant(t < num_tiles && stage < uint32_t(STAGES) && tc.z >= 0 && (tc.a0 % 8 == 0 || !A_MN) &&
                            tc.b0 % 8 == 0,
                        p.status)) {
            if constexpr (A_MN) {
#pragma unroll
              for (int c = 0; c < 2; ++c)
                ptx::tma_load_2d<CG>(stage_a(stage) + uint32_t(c * kTrainChunk), mA, tc.a0 + c * 64, k0, fb, pol_a);
            } else {
              ptx::tma_load_2d<CG>(stage_a(stage), mA, k0, tc.a0, fb, pol_a);
            }
            if constexpr (B_MN) {
#pragma unroll
              for (int c = 0; c < C::kBRows / 64; ++c) {
                const uint32_t dst = stage_b(stage) + uint32_t(c * kTrainChunk);
                if constexpr (GRP == GRP_ROWS)
                  ptx::tma_load_3d<CG>(dst, mB, tc.b0 + c * 64, k0, tc.z, fb, pol_b);
                else
                  ptx::tma_load_2d<CG>(dst, mB, tc.b0 + c * 64, k0, fb, pol_b);
              }
            } else {
              ptx::tma_load_2d<CG>(stage_b(stage), mB, k0, tc.b0, fb, pol_b);
            }
          }
          if (++stage == uint32_t(STAGES)) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        t = next_tile(Lane{}, t, cslot, cphase);
        if (t == -2) ok = false;
      }
      if (!ok && leader) {
        // drain: every armed stage completes once its bytes land
        Ctl quiet = ctl;
        int dummy = 0;
        quiet.abort_flag = &dummy;
#pragma unroll 1
        for (uint32_t s = 0; s < uint32_t(STAGES); ++s)
          if (armed & (1u << s)) wait_bar<false>(full_bar(s), (armed_par >> s) & 1u, quiet);
      }
    }
    __syncwarp();
  }
  // ------------------------------------------------------------------ MMA issuer
  else if (warp == 1) {
    if (leader && ptx::elect_one()) {
      uint32_t stage = 0, phase = 0, acc = 0, accph = 0;
      bool ok = true;
      if (p.inject_stall) ok = wait_bar<false>(never_bar, 0u, ctl);
      const uint16_t mask = (CG == 2) ? uint16_t(0x3) : uint16_t(0x1);
      uint32_t cslot = 0, cphase = 0;
      uint32_t committed = 0;
#pragma unroll 1
      for (int t = first_tile; t >= 0 && ok;) {
        if (!wait_bar<CG == 2>(acce_bar(acc), accph ^ 1u, ctl)) {
          ok = false;
          break;
        }
        ptx::tc_fence_after();
        const uint32_t d_tmem = tmem + acc * uint32_t(C::kBN);
        const TrainTile tc = coords(t);
#pragma unroll 1
        for (int it = 0; it < tc.nks; ++it) {
          if (!wait_bar<false>(full_bar(stage), phase, ctl)) {
            ok = false;
            break;
          }
          const uint64_t adesc = A_MN ? sdesc_mn_sw128(stage_a(stage)) : sdesc_sw128(stage_a(stage));
          const uint64_t bdesc = B_MN ? sdesc_mn_sw128(stage_b(stage)) : sdesc_sw128(stage_b(stage));
          const int left = tc.k_end - (tc.ks0 + it) * 64;   // k past it are zero, or not there
          const bool stage_ok = invariant(stage < uint32_t(STAGES) && acc < uint32_t(ACC), p.status);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (j * 16 >= left || !stage_ok) break;
            // 16 k: 32 bytes along K-major rows, two 8-k groups of 1024 bytes in MN-major chunks
            const uint64_t aoff = A_MN ? uint64_t((j * 2048) >> 4) : uint64_t((j * 32) >> 4);
            const uint64_t boff = B_MN ? uint64_t((j * 2048) >> 4) : uint64_t((j * 32) >> 4);
            ptx::mma_f16<CG>(d_tmem, adesc + aoff, bdesc + boff, C::kIdesc, (it > 0 || j > 0) ? 1u : 0u);
          }
          ptx::tc_commit<CG>(empty_bar(stage), mask);
          if (++stage == uint32_t(STAGES)) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        ptx::tc_commit<CG>(accf_bar(acc), mask);
        ++committed;
        if (++acc == uint32_t(ACC)) {
          acc = 0;
          accph ^= 1u;
        }
        t = next_tile(Lane{}, t, cslot, cphase);
        if (t == -2) ok = false;
      }
      // every MMA issued here has finished before tensor memory goes away, and every hand-back has landed
      ptx::tc_commit<CG>(drain_bar, uint16_t(1u << rank));
      Ctl quiet = ctl;
      int dummy = 0;
      quiet.abort_flag = &dummy;
      wait_bar<false>(drain_bar, 0u, quiet);
      if (ok) {
#pragma unroll 1
        for (uint32_t a = 0; a < uint32_t(ACC); ++a) {
          const uint32_t uses = committed / uint32_t(ACC) + (a < committed % uint32_t(ACC) ? 1u : 0u);
          if (uses) wait_bar<CG == 2>(acce_bar(a), (uses & 1u) ^ 1u, quiet);
        }
      }
    }
    __syncwarp();
  }
  // ------------------------------------------------------------------ tile scheduler
  else if (warp == 2) {
    if constexpr (C::kClc) {
      if (GRP == GRP_NONE) ptx::pdl_wait();
      if (leader && ptx::elect_one()) {
        uint32_t slot = 0, ph = 0;
#pragma unroll 1
        while (true) {
          if (!wait_bar<CG == 2>(clc_empty(slot), ph ^ 1u, ctl)) break;
          ptx::mbar_arrive_expect_tx(clc_full(slot), 16u);
          if (CG == 2) ptx::mbar_expect_tx_relaxed_cluster(ptx::map_to_rank(clc_full(slot), 1), 16u);
          ptx::clc_try_cancel<CG == 2>(clc_resp(slot), clc_full(slot));
          if (!wait_bar<false>(clc_full(slot), ph, ctl)) break;
          uint32_t x = 0;
          const bool got = ptx::clc_read(clc_resp(slot), x);
          ptx::mbar_arrive(clc_empty(slot));
          if (++slot == 2) {
            slot = 0;
            ph ^= 1u;
          }
          if (!got) break;
        }
      }
    }
    __syncwarp();
  }
  // ------------------------------------------------------------------ epilogue
  else if (warp >= 4) {
    const int e = warp - 4;
    const int q = warp & 3;              // accumulator lane quadrant this warp may read
    const int h = e >> 2;                // columns [0, 128) or [128, 256) of the tile
    const uint32_t my_buf0 = epi_base + uint32_t(e * 2 * C::kEpiBufBytes);
    const uint32_t acce_lead0 = (CG == 2) ? ptx::map_to_rank(acce_bar(0), 0) : acce_bar(0);
    if (GRP == GRP_NONE) ptx::pdl_wait();
    uint32_t acc = 0, accph = 0;
    uint32_t cslot = 0, cphase = 0;
    uint32_t nbuf = 0;                   // staging buffers used so far
    // one 32-row x 64-byte box from four 16-byte pieces per lane, in the 64-byte swizzle
    auto stage_box = [&](const uint32_t (&w)[16], auto&& send) {
      const uint32_t buf = my_buf0 + (nbuf & 1u) * uint32_t(C::kEpiBufBytes);
      ++nbuf;
      if (lane == 0) ptx::bulk_wait_group_read<1>();
      __syncwarp();
      const uint32_t row_addr = buf + uint32_t(lane * 64);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t chunk = uint32_t(j) ^ ((uint32_t(lane) >> 1) & 3u);
        ptx::st_shared_v4(row_addr + chunk * 16u, w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
      }
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        send(buf);
        ptx::bulk_commit_group();
      }
    };
#pragma unroll 1
    for (int t = first_tile; t >= 0;) {
      const TrainTile tc = coords(t);
      const int row0 = tc.a0 + q * 32;
      const int row = row0 + lane;
      const int col0 = tc.nb * C::kBN + h * 128;
      // the row's label as an offset from this warp's first column (-1: not among its 128)
      int hit = -1;
      float l2 = 0.f, coef = 0.f;
      uint32_t keep = 0;
      if constexpr (EPI == EPI_LOSS || EPI == EPI_DLOGITS) {
        if (row < p.m) {
          const long long y = __ldcg(p.labels + row);
          const long long off = y - (long long)(p.vocab0) - col0;
          if (off >= 0 && off < 128 && col0 + int(off) < p.n) hit = int(off);
          if constexpr (EPI == EPI_DLOGITS) {
            // rows of ignored labels are cleared by mask, whatever lse, dloss and the row hold
            l2 = __ldcg(p.lse + row) * 1.4426950408889634f;
            coef = __ldcg(p.dloss + row) * p.alpha;
            keep = (y >= 0 && y < p.vocab) ? 0xffffffffu : 0u;
          }
        }
      }
      if (!wait_bar_warp<false>(accf_bar(acc), accph, ctl)) break;
      ptx::tc_fence_after();
      const bool idle = !invariant(acc < uint32_t(ACC) && t < num_tiles, p.status);
      const uint32_t tbase = tmem + (uint32_t(q * 32) << 16) + acc * uint32_t(C::kBN) + uint32_t(h * 128);
      uint32_t v[4][32];
      if (!idle) {
#pragma unroll
        for (int c = 0; c < 4; ++c) ptx::tmem_ld_32x32b_x32(tbase + uint32_t(c * 32), v[c]);
      }
      ptx::tmem_ld_wait();
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (CG == 1 || leader)
          ptx::mbar_arrive(acce_bar(acc));
        else
          ptx::mbar_arrive_relaxed_cluster(acce_lead0 + 8u * acc);
      }
      if (++acc == uint32_t(ACC)) {
        acc = 0;
        accph ^= 1u;
      }
      if (GRP == GRP_K && tc.nks == 0) {   // no rows: the sum is empty, the accumulator undefined
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int j = 0; j < 32; ++j) v[c][j] = 0u;
      }
      if (!idle) {
        if constexpr (EPI == EPI_LOSS) {
          const int ncol = p.n - col0;
          float sum = 0.f, top = -INFINITY;
          if (ncol > 0) {
            if (ncol < 128) {   // columns that are not there: the least logit there is
              const uint32_t low = p.c2 >= 0.f ? 0xff800000u : 0x7f800000u;
#pragma unroll
              for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int j = 0; j < 32; ++j)
                  if (c * 32 + j >= ncol) v[c][j] = low;
            }
            // the largest z * c2: by the largest or, for a negative scale, the least z
            float ext = __uint_as_float(v[0][0]);
            if (p.c2 >= 0.f) {
#pragma unroll
              for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int j = 0; j < 32; ++j) ext = fmaxf(ext, __uint_as_float(v[c][j]));
            } else {
#pragma unroll
              for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int j = 0; j < 32; ++j) ext = fminf(ext, __uint_as_float(v[c][j]));
            }
            top = p.c2 == 0.f ? 0.f : ext * p.c2;
            const float sub = fabsf(top) == INFINITY ? 0.f : top;   // no inf - inf
            float s4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
              for (int j = 0; j < 32; ++j) s4[j & 3] += ptx::ex2(fmaf(__uint_as_float(v[c][j]), p.c2, -sub));
            sum = (s4[0] + s4[1]) + (s4[2] + s4[3]);
            if (p.c2 == 0.f && ncol < 128) sum = float(ncol);   // scale 0: every logit there is counts 1
            if (__any_sync(0xffffffffu, hit >= 0)) {
              float z = 0.f;
#pragma unroll
              for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int j = 0; j < 32; ++j)
                  if (hit == c * 32 + j) z = __uint_as_float(v[c][j]);
              if (hit >= 0) p.zlabel[row] = z * p.alpha;
            }
          }
          if (row < p.m) p.part[size_t(tc.nb * 2 + h) * size_t(p.m) + row] = make_float2(top, sum);
        } else if constexpr (EPI == EPI_DLOGITS) {
          const bool any_hit = __any_sync(0xffffffffu, hit >= 0);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            float g[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) g[j] = ptx::ex2(fmaf(__uint_as_float(v[c][j]), p.c2, -l2));
            if (any_hit) {
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (hit == c * 32 + j) g[j] -= 1.f;
            }
            uint32_t w[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) w[j] = ptx::pack_bf16x2(g[2 * j] * coef, g[2 * j + 1] * coef) & keep;
            if (col0 + c * 32 < p.n && row0 < p.m)
              stage_box(w, [&](uint32_t buf) { ptx::tma_store_3d(&tmD, buf, col0 + c * 32, row0, 0); });
          }
        } else if constexpr (EPI == EPI_BF16) {
          const int z = GRP == GRP_K ? tc.z : 0;
          const bool masked = GRP == GRP_ROWS && row0 + 32 > tc.row_limit;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t w[16];
#pragma unroll
            for (int j = 0; j < 16; ++j)
              w[j] = ptx::pack_bf16x2(__uint_as_float(v[c][2 * j]) * p.alpha, __uint_as_float(v[c][2 * j + 1]) * p.alpha);
            const int col = col0 + c * 32;
            if (masked) {   // a box that crosses the end of its group: row by row
              if (row < tc.row_limit) {
                uint16_t* dst = static_cast<uint16_t*>(p.d) + size_t(row) * size_t(p.n) + col;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                  if (col + j * 8 < p.n)
                    *reinterpret_cast<uint4*>(dst + j * 8) = make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
              }
            } else if (col < p.n && row0 < p.m) {
              stage_box(w, [&](uint32_t buf) { ptx::tma_store_3d(&tmD, buf, col, row0, z); });
            }
          }
        } else {
          if (!(GRP == GRP_K && p.accumulate && tc.nks == 0)) {   // adding nothing
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              uint32_t w[16];
#pragma unroll
              for (int j = 0; j < 16; ++j)
                w[j] = __float_as_uint(__uint_as_float(v[c >> 1][(c & 1) * 16 + j]) * p.alpha);
              const int col = col0 + c * 16;
              if (col < p.n && row0 < p.m)
                stage_box(w, [&](uint32_t buf) {
                  if (p.accumulate)
                    ptx::tma_add_3d(&tmD, buf, col, row0, tc.z);
                  else
                    ptx::tma_store_3d(&tmD, buf, col, row0, tc.z);
                });
            }
          }
        }
      }
      t = __shfl_sync(0xffffffffu, next_tile(Warp{}, t, cslot, cphase), 0);
    }
    if (EPI != EPI_LOSS && lane == 0) ptx::bulk_wait_group_read<0>();
    __syncwarp();
  }

  // ------------------------------------------------------------------ teardown
  __syncthreads();
  if (s_abort && threadIdx.x == 0) {
    // let any copy still in flight land before this CTA's shared memory is released
    const uint64_t t0 = ptx::globaltimer();
    while (ptx::globaltimer() - t0 < 50000ull) {
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (CG == 2) ptx::cluster_sync_relaxed();
  if (warp == 2) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc<CG>(tmem, 512u);
  }
}

}  // namespace tkg
