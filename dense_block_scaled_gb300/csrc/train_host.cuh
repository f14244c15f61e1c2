// train_host.cuh -- host side of train_kernel.cuh: tensor maps of the two operand
// orders and of the outputs, and the launch.
#pragma once
#include "host_common.cuh"
#include "train_kernel.cuh"

namespace tkg {

// tkg_api.cu: as encode_3d, with a swizzle
tkg_status encode_3d_swizzled(CUtensorMap* map, CUtensorMapDataType dtype, const void* base, uint64_t dim0,
                              uint64_t dim1, uint64_t dim2, uint64_t stride1_bytes, uint64_t stride2_bytes,
                              uint32_t box0, uint32_t box1, uint32_t box2, CUtensorMapSwizzle swz);

inline bool aligned_to(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Largest size of the training-side operators: indexes run past a size by less than 2^16 where tiles and grids are
// rounded up, and are 32 bits.
constexpr int kMaxSize = 0x7fff0000;

constexpr int kSMs = 152;   // of a GB300

// k rows of an MN-major box: 64, or all there are rounded up to the MMA's 16 (rows past the end arrive as
// zeros; a box that runs mostly past the end slows the load stream)
inline uint32_t mn_box_rows(int k) { return k >= 64 ? 64u : uint32_t((k + 15) / 16 * 16); }

// K-major operand: `rows` rows of k BF16; boxes of 64 k by up to `box` rows.
inline tkg_status map_k_major(CUtensorMap* map, const void* base, int rows, int k, size_t row_bytes, int box) {
  return encode_2d(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base, uint64_t(k), uint64_t(rows), row_bytes, 64,
                   uint32_t(rows < box ? rows : box), CU_TENSOR_MAP_SWIZZLE_128B);
}
// MN-major operand: k rows of `mn` BF16; boxes of 64 mn by up to 64 k.
inline tkg_status map_mn_major(CUtensorMap* map, const void* base, int mn, int k, size_t row_bytes, int box_rows = 0) {
  return encode_2d(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base, uint64_t(mn), uint64_t(k), row_bytes, 64,
                   box_rows ? uint32_t(box_rows) : mn_box_rows(k), CU_TENSOR_MAP_SWIZZLE_128B);
}
// Output: `parts` matrices of m x n.  Store boxes of 16 rows by 128 bytes, or (half: BF16 in 32 columns, a chunk of
// DLOGITS or, turned, a warp's 32 rows of D) by 64 bytes.
inline tkg_status map_out(CUtensorMap* map, const void* base, int m, int n, int parts, size_t row_bytes,
                          size_t part_bytes, bool f32, bool half = false) {
  return encode_3d_swizzled(map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base,
                            uint64_t(n), uint64_t(m), uint64_t(parts), row_bytes, part_bytes, f32 || half ? 32 : 64, 16,
                            1, half ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B);
}
// The same matrices in the boxes that fetch what is added to into L2.
inline tkg_status map_prefetch(CUtensorMap* map, const void* base, int m, int n, int parts, size_t row_bytes,
                               size_t part_bytes) {
  return encode_3d(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, base, uint64_t(n), uint64_t(m), uint64_t(parts), row_bytes,
                   part_bytes, 256, 32, 1);
}
// Multiple that an output's tiles are wide: a store box's columns (of tokens: the MMA's 16).
constexpr int kTileBF16 = 64, kTileF32 = 32, kTileTokens = 16;

// Fills the fields common to every launch and launches.  The caller sets p.m, n,
// k, n_tile, alpha, splits and split_stages (GRP_NONE) and the epilogue's own fields.
template <bool A_MN, bool B_MN, int EPI, int GRP, int SHAPE = SHAPE_WIDE>
tkg_status launch_train(const CUtensorMap& tmA, const CUtensorMap& tmB, const CUtensorMap& tmD, TrainParams p,
                        cudaStream_t stream,
                        const ExtraMaps<EPI, GRP>& extra = {}) {
  using C = TrainConfig<A_MN, B_MN, EPI, GRP, SHAPE>;
  auto kern = train_kernel<A_MN, B_MN, EPI, GRP, SHAPE>;
  // a block that takes all of tensor memory takes more than half of shared memory too, so that no two share an SM
  static_assert(C::kNarrow || C::kSmemBytes > 118784, "one CTA per SM");
  if (C::kDual) p.n_tile = 2 * kTrainBN;
  if (p.n_tile > C::kSubs * C::kBN) return TKG_ERR_UNSUPPORTED;   // (no caller asks for it)
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return TKG_ERR_CUDA;
  static std::atomic<bool> attr_set[64] = {};   // per instantiation and device (set twice alike if two threads race)
  if (!attr_set[dev]) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes) != cudaSuccess) {
      cudaGetLastError();
      return TKG_ERR_CUDA;
    }
    attr_set[dev] = true;
  }
  tkg_status st;
  if ((st = device_status_word(&p.status)) != TKG_OK) return st;
  const int tmo = option(TKG_OPT_TIMEOUT_MS);
  p.timeout_ns = 1000000ull * (unsigned long long)(tmo > 0 ? tmo : 1000);
  p.inject_stall = option(TKG_OPT_INJECT_STALL);
  p.kstages = ceil_div(p.k, 64);
  p.tiles_m = ceil_div(p.m, 256);
  p.tiles_n = ceil_div(p.n, p.n_tile);
  // what a stage of one CTA takes and brings: A's 128 rows (fewer when there are fewer) or two chunks, and
  // its half of B's n_tile
  const int kb = GRP == GRP_K ? 64 : int(mn_box_rows(p.k));   // k rows of an MN-major box
  const int half = p.n_tile / 2 / C::kSubs;
  const int a_bytes = A_MN ? 2 * kb * 128 : (p.m < 128 ? p.m : 128) * 128;
  const int b_slot = B_MN ? (GRP == GRP_K ? 2 : ceil_div(half, 64)) * kTrainChunk : (GRP == GRP_ROWS ? (half + 31) / 32 * 32 : half) * 128;
  p.tx_a = uint32_t(2 * a_bytes);
  p.tx_box = uint32_t(2 * (B_MN ? kb : (GRP == GRP_ROWS ? 32 : (p.n < half ? p.n : half))) * 128);
  p.stage_bytes = uint32_t(C::kABytes + C::kSubs * b_slot);
  p.stages = C::kRingBytes / int(p.stage_bytes);
  if (p.stages > kTrainMaxStages) p.stages = kTrainMaxStages;
  p.raster_group = raster_group(256, GRP == GRP_K ? ceil_div(p.k, p.groups) : p.k, FMT_BF16, p.tiles_m);
  long long tiles = (long long)p.tiles_m * p.tiles_n;
  if (GRP == GRP_NONE) tiles *= p.splits;
  if (GRP == GRP_K) tiles *= p.groups;
  if (GRP == GRP_ROWS) tiles = (long long)p.tiles_m * (ceil_div(p.n, kTrainBN) + p.groups);   // at most
  if (tiles * 2 > 0x7fffffffLL) return TKG_ERR_UNSUPPORTED;
  p.num_tiles = int(tiles);

  long long clusters = tiles;   // cluster launch control: one cluster per tile
  if (!C::kClc) {
    int resident = 0;
    if ((st = device_max_clusters(2, &resident)) != TKG_OK) return st;
    if (clusters > resident) clusters = resident;
  }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  cfg.gridDim = dim3(unsigned(clusters * 2), 1, 1);
  cfg.blockDim = dim3(C::kThreads, 1, 1);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, kern, tmA, tmB, tmD, p, extra) != cudaSuccess) {
    cudaGetLastError();
    return TKG_ERR_CUDA;
  }
  return TKG_OK;
}

// Rounds of `tiles` on the GB300's 76 CTA pairs: whole ones while they are few; with more the clusters have
// drifted apart and the last one overlaps.  (Whole ones always: dW of 2502 tokens x 45493 x 2920 1117 us in place of
// 1045, dX of 5063 x 130171 x 264 1045 of 924; but 7 experts of 1276 rows, 3640 x 1808, 91 of 111.)
constexpr int kPairs = 76;
inline double train_rounds(double tiles) {
  const double r = tiles / kPairs;
  return r < 4.0 ? double((long long)(r + 0.999999)) : r + 0.5;
}
// Time of a round of tiles in units of a 64-k stage of a 256-wide tile: a 512-wide tile's stage takes 4% less
// than two, its start and read-out as long as two.  Under the power cap, back to back, 8 groups of 256, 512, 1024
// and 2048 rows of 4096 x 7168 took 123.7, 200.9, 339 and 610 us in 256-wide tiles and 122.8, 192.0, 327 and 593
// in 512-wide ones, 8192 rows of 32768 x 4096 1366 and 1308.  Sums of one to three stages have their read-outs
// exposed on the wide tiles (8 groups of 64 rows: 81 against 92 us).
inline double train_tile_time(int stages, bool dual) { return dual ? 1.92 * stages + 16 : stages + 8.0; }

// Whether `count` products of m x n with `stages` stages per tile run on 256 x 512 tiles.  TKG_OPT_BF16_TILE_N
// (256 or 512) decides it instead.
inline bool train_dual(int m, int n, long long count, int stages) {
  const int forced = option(TKG_OPT_BF16_TILE_N);
  if (forced == 512) return true;
  if (forced == 256) return false;
  if (stages < 4) return false;
  const double rows = double(ceil_div(m, 256)) * double(count);
  return train_rounds(rows * ceil_div(n, 512)) * train_tile_time(stages, true) <
         train_rounds(rows * ceil_div(n, 256)) * train_tile_time(stages, false);
}

// Whether the loss's logits of n tokens run in the kernel's narrow form, given their tiles.  It needs more
// of them than there are pairs of SMs: 16 tokens take 32.5 us narrow and 46.9 wide at 20000 x 4096, 162.8 and
// 175.2 at 131072 x 4096, 8.7 and 10.7 at 50000 x 256, but 13.1 and 12.7 at 8000 x 2048.  Past 64 tokens its four
// epilogue warps tell (a block has a quarter of the wide form's), and it pays while it spares a thin second round:
// 128 tokens 13.4 and 15.4 us at 23000 x 1024, 44.4 and 49.2 at 27000 x 4096, but 30.5 and 29.1 at 32768 x 2048
// and 76.0 and 72.2 at 40000 x 4096.
constexpr int kNarrowTokens = 128;
inline bool train_narrow(int n, int tiles) {
  return n <= kNarrowTokens && tiles > kPairs && (n <= kNarrowTokens / 2 || 2 * tiles <= 3 * kPairs);
}
// The same of the gradient's logits, whose epilogue does more per logit and writes them: the narrow form pays only where it
// spares a thin second round, and where the sums are long for the tokens.  dX and dW, narrow and wide: 40 tokens x
// 21648 x 1024 43.4 and 44.8 us, 64 x 25000 x 2048 69.7 and 70.7, 128 x 20000 x 4096 110.0 and 115.8, 1 x 19713 x 768
// 37.0 and 37.9; but (more tiles) 128 x 29000 x 4096 154.3 and 147.0, 40 x 32768 x 2048 95.0 and 93.6, (shorter sums)
// 128 x 20000 x 2048 69.1 and 67.8, 128 x 27000 x 1024 53.4 and 48.3, 16 x 21648 x 512 31.1 and 30.6, 1 x 20000 x 256
// 25.7 and 24.9.
inline bool train_narrow_gradient(int n, int hidden, int tiles) {
  return n <= kNarrowTokens && tiles > kPairs && 3 * tiles <= 4 * kPairs && hidden >= 768 && hidden >= 24 * n;
}
// Stages (64 k each) that one accumulator sums where the result is FP32 (logits, FP32 weight gradients).  Tensor memory
// adds towards zero, so a sum's error grows with its length: terms of one sign lose 3e-6 of it over 2048 terms,
// 6.7e-5 over 16384 and 1.5e-4 over 30000; of lse, 6.3e-7 at 2048 products and 1.3e-6 at 4096 in one sum.
// Sums of at most 2048 are added in the epilogue's registers.  The gradient's logits are the loss's, bit for bit: where
// lse is the label's own logit, g is exactly 0.  BF16 results, dX from its FP32 parts among them, take one sum each:
// what it loses is 1/30 of their own rounding's 2^-9 at 16384 terms of one sign, and less where signs differ.
constexpr int kSumStages = 32;

// Launch of a small kernel that waits for the previous grid itself (griddepcontrol.wait), in clusters of `cluster` blocks.
template <typename... P, typename... Args>
tkg_status launch_small_cluster(void (*kern)(P...), dim3 grid, dim3 block, unsigned cluster, cudaStream_t stream,
                                unsigned smem, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  if (cudaLaunchKernelEx(&cfg, kern, P(args)...) != cudaSuccess) {
    cudaGetLastError();
    return TKG_ERR_CUDA;
  }
  return TKG_OK;
}
template <typename... P, typename... Args>
tkg_status launch_small(void (*kern)(P...), dim3 grid, dim3 block, cudaStream_t stream, unsigned smem, Args... args) {
  return launch_small_cluster(kern, grid, block, 1u, stream, smem, args...);
}

}  // namespace tkg
