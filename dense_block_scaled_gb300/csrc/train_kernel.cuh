// train_kernel.cuh -- persistent, warp-specialised tcgen05 products of the
// training-side operators: the head's logits with a softmax cross-entropy
// epilogue, and the gradient products, whose operands lie transposed in memory.
//
//   D[m][n] = sum_k a(m,k) * b(n,k),  BF16 operands, FP32 accumulation in tensor memory
//
// M is the side of the weights (vocabulary, hidden, an expert's columns): long,
// and the same for every call.  N is, in all but the weight gradients, the side
// of the tokens: short, ragged, different per group.  An MMA takes any N that is
// a multiple of 16, so a batch of T tokens is cut into ceil(T / 256) tiles of
// equal width, T / tiles rounded up to 16, and next to nothing is computed for
// tokens that do not exist; with the tokens on M (tiles of 256) 777 tokens cost
// 1024 and 64 uneven experts of 250 rows on average 1.4 times their rows (loss of
// 777 x 50001 x 2048: 129 us against 112; rows' gradient of 64 experts x 2048 x
// 2048, 16000 rows: 144 against 126).
//
// Each operand is either K-major (row m holds consecutive k: rows of X, W, dD)
// or MN-major (row k holds consecutive m or n: the same matrices read for
// their gradients).  A stage holds 64 k of a tile.  K-major tiles are rows of
// 128 bytes (64 k), 128-byte swizzle; MN-major tiles are chunks of 64 m (or n)
// by 64 k, each k a 128-byte row under the same swizzle.  TMA writes both
// directly and the MMA descriptors carry the difference: nothing is ever
// transposed in memory.
//
// Roles (one CTA per SM; the two CTAs of a cluster share one MMA of 256 x N),
// the bounded waits and the abort protocol are those of gemm_kernel.cuh:
//   warp 0 TMA producer, warp 1 MMA issuer, warp 2 tensor-memory allocation and
//   the cluster-launch-control tile scheduler, warp 3 the group table and
//   the producer of the stages in which a group of k ends (with DLOGITS: the weighted
//   rows of X), warps 4-19 epilogue: 16 (DUAL 8, NARROW 4),
//   as the cross-entropy epilogues are bound by latency (with 8 warps they took
//   8000 cycles for a 256 x 256 tile, twice its MMAs at hidden = 512, at 40% of
//   the issue slots).
// Two 256-column accumulators: a tile's epilogue overlaps the next tile's MMAs.
// The ring takes as many stages as fit: 6 for 256-wide tiles, up to 12 where few
// tokens leave most of a stage to the weights (bytes in flight are what a
// bandwidth-bound call needs).
//
// DUAL (weight gradients and dX with long sums): 256 x 512 tiles, A's stage shared by
// two MMAs.  The SMs read a quarter fewer bytes from L2 for the same products;
// these kernels run under the power cap, where that shows as clock.
//
// SUMS (logits and FP32 weight gradients of more than 2048 products): tensor memory adds
// towards zero, so a sum's error grows with its length.  An accumulator takes at most 2048
// products; the epilogue gathers such sums in registers (64 a thread) and hands the
// accumulator back before it turns to the rest.  lse of 4096 x 131072 x 4096: 6e-7 off
// (relative) against 1.2e-6 in one sum, 2497 against 2480 us.
//
// NARROW (logits of at most 128 tokens with more tiles than pairs of SMs, where reading the
// weights bounds the time): two blocks per SM, each with half the shared memory and 4
// epilogue warps.  Twice the tiles run at once, so that few tiles do not leave a thin last
// round, and one block's set-up and epilogue run under the other's loads.
// Two sums at most, in the two accumulators.
//
// Epilogues (EPI):
//   LOSS     per token (column) and 128 vocabulary rows: the largest logit, the
//            sum of exponentials relative to it, and, where the token's label falls among
//            them, its logit.  A thread holds 8 columns by 4 rows of each 32 x 32
//            block (the 16x256b load); columns are joined over 8 lanes by exchanging
//            halves (7 shuffles down for the maximum, 7 back, 7 for the sum, against
//            a 5-step butterfly per column), then over the four warps in shared
//            memory.  8 bytes per 128 logits go to memory, never the logits.
//   DLOGITS  g = exp(z - lse) - [v = label], rounded to BF16 (the tensor cores'
//            operand type; u = 2^-8, independent between elements) into a piece
//            [vocabulary][token].  The tokens' weights are left out, so that the
//            rounding does not hit them all the same way: they multiply dX's rows in
//            FP32 and, relative to the largest, X's rows for dW.
//   BF16     alpha * D rounded to nearest even.
//   BF16_T   the same, transposed: D's columns are rows of the output.  Neighbouring
//            lanes swap halves (one shuffle per two values) and store 32-bit words.
//   F32      alpha * D stored, or added by the TMA unit to what is there (one add
//            per element and launch, so the order of additions is fixed).
#pragma once
#include "gemm_kernel.cuh"

namespace tkg {

enum : int { EPI_LOSS = 0, EPI_DLOGITS = 1, EPI_BF16 = 2, EPI_F32 = 3, EPI_BF16_T = 4 };
// GRP_ROWS: groups of consecutive n, each with its own A; GRP_K: groups of
// consecutive k, each with its own output matrix.  Row counts in device memory.
enum : int { GRP_NONE = 0, GRP_ROWS = 1, GRP_K = 2 };
// Tile shapes: 256 x up to 256; NARROW 256 x up to 128, two blocks per SM; DUAL 256 x 512.
// SUMS: WIDE with sums longer than one accumulator takes.
enum : int { SHAPE_WIDE = 0, SHAPE_NARROW = 1, SHAPE_DUAL = 2, SHAPE_SUMS = 3 };

struct TrainParams {
  int m, n, k;                 // output rows and columns, contraction length (GRP_ROWS: n, GRP_K: k is the row capacity)
  int kstages;                 // ceil(k / 64)
  int splits, split_stages;    // k split: part z covers stages [z * split_stages, ...)
  int sum_stages;              // NARROW, SUMS: stages summed in one accumulator; the epilogue adds the next to it
  int tiles_m, tiles_n, num_tiles;
  int n_tile;                  // tile width, a multiple of 16 (GRP_ROWS: per group, by its rows; DUAL: 512)
  int raster_group;
  int stages;                  // ring slots, and the bytes of one in each CTA
  uint32_t stage_bytes;
  uint32_t tx_a, tx_box;       // bytes landing on the leader's full barrier per stage: of A, and of one box of B in each CTA
  float alpha;
  const float* scale;          // device, may be null: multiplies alpha
  unsigned int* status;
  unsigned long long timeout_ns;
  int inject_stall;
  // cross entropy
  float c2;                    // alpha * log2(e)
  int vocab0, vocab;           // first vocabulary entry of this piece, and all there are
  const long long* labels;
  const float* lse;
  float2* part;                // LOSS: (maximum, sum) per 128 vocabulary rows and token
  float* zlabel;               // LOSS: the label's logit per token
  // DLOGITS: the rows of X with the tokens' weights (see ce_weighted_row), written on the side; null: not wanted
  const uint16_t* x;
  size_t ldx;
  const float* dloss;
  uint16_t* rows;
  float* rows_scale;
  // outputs written from registers: their first element and row pitch in elements
  void* d;
  size_t ldd;
  int accumulate;              // F32
  // groups
  const int* sizes;            // device
  int groups;
};

// GRP_K: A and B in boxes of 16, 8, 4, 2 and 1 k rows, for the stage in which a group ends.
constexpr int kTailMaps = 5;
struct TailMaps {
  CUtensorMap a[kTailMaps], b[kTailMaps];
};
// F32: D in boxes of 256 columns by 32 rows, to fetch into L2 what is about to be added to.
struct PrefetchMap {
  CUtensorMap d;
};
struct NoTail {};
struct NoPrefetch {
  int unused;
};
template <int EPI, int GRP>
struct ExtraMaps : std::conditional_t<GRP == GRP_K, TailMaps, NoTail>,
                   std::conditional_t<EPI == EPI_F32, PrefetchMap, NoPrefetch> {};

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
// 16 lanes x 32 columns: thread t gets, for i = 0..3, lane t / 4 columns 8 i + 2 (t % 4) + {0, 1} in r[4 i],
// r[4 i + 1] and lane t / 4 + 8 of the same columns in r[4 i + 2], r[4 i + 3].
__device__ __forceinline__ void tmem_ld_16x256b_x4(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
// 32 lanes x 8 columns: thread t gets its lane's
__device__ __forceinline__ void tmem_ld_32x32b_x8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld_wait_for(uint32_t (&r)[8]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7])::"memory");
}
__device__ __forceinline__ void tmem_ld_wait_for(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])::"memory");
}
// Waits for this thread's tensor-memory loads; naming the registers keeps what reads them behind the wait.
__device__ __forceinline__ void tmem_ld_wait_for(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]),
                 "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])::"memory");
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

// Joins the values of a column over the 8 lanes (t / 4) that hold it: of 8 columns
// each lane keeps half at every step and ends with one, column_of_lane.
template <typename F>
__device__ __forceinline__ float fold_columns(const float (&x)[8], int lane, F&& op) {
  float a[4], b[2];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float r = __shfl_xor_sync(0xffffffffu, (lane & 16) ? x[i] : x[i + 4], 16);
    a[i] = op((lane & 16) ? x[i + 4] : x[i], r);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float r = __shfl_xor_sync(0xffffffffu, (lane & 8) ? a[i] : a[i + 2], 8);
    b[i] = op((lane & 8) ? a[i + 2] : a[i], r);
  }
  const float r = __shfl_xor_sync(0xffffffffu, (lane & 4) ? b[0] : b[1], 4);
  return op((lane & 4) ? b[1] : b[0], r);
}
// The way back: every lane gets its 8 columns' values from the lanes that hold them.
__device__ __forceinline__ void unfold_columns(float own, int lane, float (&x)[8]) {
  float b[2], a[4];
  const float o = __shfl_xor_sync(0xffffffffu, own, 4);
  b[0] = (lane & 4) ? o : own;
  b[1] = (lane & 4) ? own : o;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float r = __shfl_xor_sync(0xffffffffu, b[i], 8);
    a[i] = (lane & 8) ? r : b[i];
    a[i + 2] = (lane & 8) ? b[i] : r;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float r = __shfl_xor_sync(0xffffffffu, a[i], 16);
    x[i] = (lane & 16) ? r : a[i];
    x[i + 4] = (lane & 16) ? a[i] : r;
  }
}
__device__ __forceinline__ int column_of_lane(int lane) {
  return 16 * ((lane >> 4) & 1) + 8 * ((lane >> 3) & 1) + 2 * (lane & 3) + ((lane >> 2) & 1);
}

// ---- joins a maximum and the sum of exponentials relative to it, (top, sum), with another, (m, s): one of the two
// factors is 1, exactly
constexpr float kLog2e = 1.4426950408889634f;
__device__ __forceinline__ void ce_join(float& top, float& sum, float m, float s) {
  const float d = m == top ? 0.f : m - top;   // (infinities of one sign: not their difference)
  const float e = ptx::ex2(-fabsf(d) * kLog2e);
  sum = m > top ? fmaf(sum, e, s) : fmaf(s, e, sum);
  top = fmaxf(top, m);
}

// ---- rows of X with the tokens' weights: row t times c_t / s with c_t = alpha dloss_t (0 for ignored tokens) and
// s = max |c_t|, or 1 where that maximum (which leaves NaN out) is no scale: with s = 0 or infinite the product of the
// row and s would not be c_t's, and a weight that is not a number has to reach dW.  Rows of ignored tokens are zeros
// whatever they hold: their g is 0, but 0 times a padded position's NaN is not.
__device__ __forceinline__ float ce_scale(float top) { return top > 0.f && top < INFINITY ? top : 1.f; }
__device__ __forceinline__ float ce_weight(int t, int vocab, const long long* labels, const float* dloss, float alpha) {
  const long long y = __ldcg(labels + t);
  const float d = __ldcg(dloss + t);
  return (y >= 0 && y < vocab) ? alpha * d : 0.f;
}
// One row, by a warp.
__device__ __forceinline__ void ce_weighted_row(int t, int lane, int vocab, int hidden, const uint16_t* X, size_t ldx,
                                                const long long* labels, const float* dloss, float alpha, float s,
                                                uint16_t* out) {
  const long long y = __ldcg(labels + t);
  const bool kept = y >= 0 && y < vocab;
  const float w = __fdiv_rn(ce_weight(t, vocab, labels, dloss, alpha), s);
  const uint4* src = reinterpret_cast<const uint4*>(X + size_t(t) * ldx);
  uint4* dst = reinterpret_cast<uint4*>(out + size_t(t) * size_t(hidden));
  const int vec = hidden / 8;
  for (int c0 = lane; c0 < vec; c0 += 128) {
    uint4 v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      v[j] = kept && c0 + 32 * j < vec ? __ldcg(src + c0 + 32 * j) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (w != 1.f) {
        uint32_t* u = reinterpret_cast<uint32_t*>(&v[j]);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          u[i] = ptx::pack_bf16x2(__uint_as_float(u[i] << 16) * w, __uint_as_float(u[i] & 0xffff0000u) * w);
      }
      if (c0 + 32 * j < vec) dst[c0 + 32 * j] = v[j];
    }
  }
}

constexpr int kTrainBN = 256;         // widest tile
constexpr int kTrainMaxStages = 12;

template <bool A_MN, bool B_MN, int EPI, int GRP, int SHAPE>
struct TrainConfig {
  static constexpr bool kNarrow = SHAPE == SHAPE_NARROW, kDual = SHAPE == SHAPE_DUAL;
  static constexpr int kBN = kNarrow ? 128 : kTrainBN;     // columns of an accumulator, and widest MMA
  static constexpr int kSubs = kDual ? 2 : 1;              // accumulators of a tile
  static constexpr int kEpiWarps = kNarrow ? 4 : (kDual ? 8 : 16);
  static constexpr int kChunks = kBN / 32 / (kEpiWarps / 4);   // 32-column chunks of an accumulator per epilogue warp
  // DUAL: stages at a tile's start and end in which the first accumulator runs ahead of the second
  static constexpr int kSkew = 2;
  static constexpr bool kSums = kNarrow || SHAPE == SHAPE_SUMS;   // sums longer than one accumulator takes
  static constexpr int kThreads = 32 * (4 + kEpiWarps);
  static constexpr int kAcc = 2;
  static constexpr int kABytes = 128 * 128;
  static constexpr int kEpiBufBytes = 32 * 64;      // 32 rows x 32 BF16 (or 16 FP32)
  // LOSS: two buffers of (maximum, sum) per quadrant and column; others: a staging box per warp
  static constexpr int kEpiBytes = EPI == EPI_LOSS ? 2 * 4 * kBN * 8 : kEpiWarps * kEpiBufBytes;
  static constexpr int kTailBars = GRP == GRP_K ? kTrainMaxStages : 0;
  static constexpr int kNumBars = 2 * kTrainMaxStages + 2 * kAcc + 2 + 4 + 4 + kTailBars;
  // groups by rank: first row, rows, the group (a byte each); GRP_ROWS: first tile, and the tile count
  static constexpr int kTabInts =
      GRP == GRP_NONE ? 0 : 2 * kMaxGroups + kMaxGroups / 4 + (GRP == GRP_ROWS ? kMaxGroups + 1 : 0);
  // epilogue buffers, barriers, two scheduler answers, table, 1024-byte alignment; the rest is the ring's
  static constexpr int kFixedBytes = kEpiBytes + kNumBars * 8 + 2 * 16 + 16 + kTabInts * 4 + 1024;
  // all an SM gives a block, or two blocks, less the two static words
  static constexpr int kSmemBytes = (kNarrow ? 116736 - 1024 : 232448) - 16;
  static constexpr int kRingBytes = (kSmemBytes - kFixedBytes) / 1024 * 1024;
  static_assert(kRingBytes >= (SHAPE == SHAPE_WIDE || SHAPE == SHAPE_SUMS ? 6 : 4) * (kABytes + kSubs * kBN / 2 * 128),
                "four or six stages of the widest tiles");
  static_assert(!kDual || (B_MN && (EPI == EPI_BF16 || EPI == EPI_F32) && GRP != GRP_ROWS), "not built");
  static constexpr bool kClc = GRP != GRP_ROWS;     // GRP_ROWS: the tile count is known on the device only
  // readers of a scheduler answer: producer, warp 3 where it has tiles' work, epilogue warps; MMA issuer and scheduler
  static constexpr int kClcConsumers = 2 * ((GRP == GRP_K || EPI == EPI_DLOGITS ? 2 : 1) + kEpiWarps) + 2;
  static constexpr uint32_t kIdesc = idesc_f16(256, kBN) | (A_MN ? 1u << 15 : 0u) | (B_MN ? 1u << 16 : 0u);
};

// Width of the tiles that `n` columns are cut into.
__host__ __device__ constexpr int train_n_tile(int n, int multiple) {
  const int tiles = (n + kTrainBN - 1) / kTrainBN;
  const int w = tiles > 0 ? (n + tiles - 1) / tiles : multiple;
  return (w + multiple - 1) / multiple * multiple;
}

struct TrainTile {
  int mb, nb;
  int a0;            // this CTA's first m of A
  int n0, n_end;     // the tile's first column, and where its columns (or its group's) end
  int nt;            // MMA width
  int subs;          // accumulators
  int z;             // k part (GRP_NONE) or group
  int k0;            // GRP_K: the group's first row
  int ks0, nks;      // first k stage (from k0) and number of stages
  int k_end;         // contraction stops here (from k0)
};

template <bool A_MN, bool B_MN, int EPI, int GRP, int SHAPE>
__global__ void __launch_bounds__(TrainConfig<A_MN, B_MN, EPI, GRP, SHAPE>::kThreads, SHAPE == SHAPE_NARROW ? 2 : 1)
    train_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                 const __grid_constant__ CUtensorMap tmD, const TrainParams p,
                 const __grid_constant__ ExtraMaps<EPI, GRP> extra) {
  using C = TrainConfig<A_MN, B_MN, EPI, GRP, SHAPE>;
  constexpr int CG = 2;
  constexpr int ACC = C::kAcc;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint32_t s_tmem_base;
  __shared__ int s_abort;

  ptx::pdl_launch_dependents();
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = ptx::cluster_ctarank();
  const bool leader = rank == 0;
  const uint32_t nstages = uint32_t(p.stages);

  const uint32_t raw = ptx::smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  auto stage_a = [&](uint32_t s) { return base + s * p.stage_bytes; };
  auto stage_b = [&](uint32_t s) { return base + s * p.stage_bytes + uint32_t(C::kABytes); };
  const uint32_t epi_base = base + uint32_t(C::kRingBytes);
  const uint32_t bars = epi_base + uint32_t(C::kEpiBytes);
  auto full_bar = [&](uint32_t s) { return bars + 8u * s; };
  auto empty_bar = [&](uint32_t s) { return bars + 8u * (uint32_t(kTrainMaxStages) + s); };
  auto accf_bar = [&](uint32_t a) { return bars + 8u * (uint32_t(2 * kTrainMaxStages) + a); };
  auto acce_bar = [&](uint32_t a) { return bars + 8u * (uint32_t(2 * kTrainMaxStages + ACC) + a); };
  const uint32_t drain_bar = bars + uint32_t(8 * (2 * kTrainMaxStages + 2 * ACC));
  const uint32_t never_bar = drain_bar + 8;
  auto clc_full = [&](uint32_t i) { return never_bar + 8u + 8u * i; };
  auto clc_empty = [&](uint32_t i) { return never_bar + 24u + 8u * i; };
  auto stat_bar = [&](uint32_t h) { return never_bar + 40u + 8u * h; };   // LOSS: a quarter's four warps have written
  auto tail_go = [&](uint32_t s) { return never_bar + 72u + 8u * s; };     // GRP_K: stage s is warp 3's to fill
  auto clc_resp = [&](uint32_t i) { return ((never_bar + 72u + 8u * uint32_t(C::kTailBars) + 15u) & ~15u) + 16u * i; };
  int* s_tab = reinterpret_cast<int*>(smem_raw + (clc_resp(2) - raw));
  float2* s_stat = reinterpret_cast<float2*>(smem_raw + (epi_base - raw));   // LOSS: [buffer][quadrant][column]
  enum : int { kTabRow0 = 0, kTabRows = kMaxGroups, kTabGroup = 2 * kMaxGroups, kTabTile = kTabGroup + kMaxGroups / 4 };
  [[maybe_unused]] uint8_t* s_group = reinterpret_cast<uint8_t*>(s_tab + kTabGroup);

  auto coords = [&](int t) {
    TrainTile tc;
    if constexpr (GRP == GRP_ROWS) {
      // last place whose first tile is <= t (groups without rows have none)
      int lo = 0, hi = p.groups;
#pragma unroll 1
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_tab[kTabTile + mid] <= t) lo = mid; else hi = mid;
      }
      const int rows = s_tab[kTabRows + lo], row0 = s_tab[kTabRow0 + lo];
      tile_coords(t - s_tab[kTabTile + lo], p.tiles_m, (rows + kTrainBN - 1) / kTrainBN, p.raster_group, tc.mb, tc.nb);
      tc.nt = train_n_tile(rows, 16);
      tc.subs = 1;
      tc.n0 = row0 + tc.nb * tc.nt;
      tc.n_end = min(tc.n0 + tc.nt, row0 + rows);
      tc.z = s_group[lo];
      tc.k0 = 0;
      tc.ks0 = 0;
      tc.nks = p.kstages;
      tc.k_end = p.k;
    } else {
      const int per = p.tiles_m * p.tiles_n;
      const int z = t / per;
      tile_coords(t - z * per, p.tiles_m, p.tiles_n, p.raster_group, tc.mb, tc.nb);
      tc.nt = C::kDual ? kTrainBN : p.n_tile;
      tc.n0 = tc.nb * p.n_tile;
      tc.n_end = min(tc.n0 + p.n_tile, p.n);
      tc.subs = C::kDual && tc.n_end - tc.n0 > kTrainBN ? 2 : 1;
      tc.k0 = 0;
      if constexpr (GRP == GRP_K) {   // the groups with most rows first
        tc.z = s_group[z];
        tc.k0 = s_tab[kTabRow0 + z];
        tc.k_end = s_tab[kTabRows + z];
        tc.ks0 = 0;
        tc.nks = (tc.k_end + 63) >> 6;
      } else {
        tc.z = z;
        tc.ks0 = z * p.split_stages;
        tc.nks = min(p.split_stages, p.kstages - tc.ks0);
        tc.k_end = p.k;
      }
    }
    tc.a0 = tc.mb * 256 + int(rank) * 128;
    return tc;
  };
  // MMA width of a tile's accumulator (the last of a DUAL tile as wide as it has columns, in store boxes), this
  // CTA's first n of B in it, and the boxes it is loaded in: GRP_ROWS 32 rows each (tiles differ in width),
  // K-major otherwise one, MN-major 64 columns each (GRP_K: always two)
  auto width = [&](const TrainTile& tc, int sub) {
    return C::kDual ? min(kTrainBN, (tc.n_end - tc.n0 - sub * kTrainBN + 31) & ~31) : tc.nt;
  };
  auto first_n = [&](const TrainTile& tc, int sub) {
    return tc.n0 + sub * kTrainBN + int(rank) * (width(tc, sub) >> 1);
  };
  auto boxes = [&](const TrainTile& tc, int sub) {
    if (GRP == GRP_K) return 2;
    return (GRP == GRP_ROWS || B_MN) ? ((width(tc, sub) >> 1) + (B_MN ? 63 : 31)) / (B_MN ? 64 : 32) : 1;
  };

  if (threadIdx.x == 0) {
    s_abort = 0;
    for (uint32_t s = 0; s < nstages; ++s) {
      ptx::mbar_init(full_bar(s), 1);
      ptx::mbar_init(empty_bar(s), 1);
      if (GRP == GRP_K) ptx::mbar_init(tail_go(s), 1);
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
    for (uint32_t i = 0; i < 4; ++i) ptx::mbar_init(stat_bar(i), 4);
    ptx::fence_mbar_init();
    ptx::prefetch_tmap(&tmA);
    ptx::prefetch_tmap(&tmB);
    if (EPI != EPI_LOSS) ptx::prefetch_tmap(&tmD);
  }
  // Two narrow blocks share an SM, one of them perhaps of the next kernel: it takes tensor memory only once the
  // previous kernel is done, as a block that holds some while it waits could keep that kernel from getting its own
  if (C::kNarrow) ptx::pdl_wait();
  if (warp == 2) {
    ptx::tmem_alloc<CG>(ptx::smem_u32(&s_tmem_base), uint32_t(2 * C::kBN));
    ptx::tmem_relinquish<CG>();
  }
  ptx::tc_fence_before();
  __syncthreads();
  // see gemm_kernel.cuh: the barriers' initialisation is published by its fence
  ptx::cluster_sync_relaxed();
  ptx::tc_fence_after();
  const uint32_t tmem = s_tmem_base;

  // Dependency wait: the roles that read global memory or hand out work wait for
  // the previous grid, as in gemm_kernel.cuh; with group sizes the whole CTA.
  int num_tiles = p.num_tiles;
  if constexpr (GRP != GRP_NONE) {
    ptx::pdl_wait();
    // Row ranges: sums stop at the capacity, so that rows past it are cut off and nothing leaves 32 bits.
    // s_end: where each group ends (in the epilogue's buffers, not in use yet).  The sizes may have been cached by this SM before the
    // previous grid wrote them: they are read through L2.
    int* s_end = reinterpret_cast<int*>(smem_raw + (epi_base - raw));
    [[maybe_unused]] int* s_rows = s_end + kMaxGroups;
    const int g = threadIdx.x;
    if (warp == 3) {
      const uint32_t cap = uint32_t(GRP == GRP_ROWS ? p.n : p.k);
      uint32_t carry = 0;
#pragma unroll 1
      for (int g0 = 0; g0 < p.groups; g0 += 32) {
        uint32_t sr = g0 + lane < p.groups ? min(uint32_t(max(__ldcg(p.sizes + g0 + lane), 0)), cap) : 0u;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t x = __shfl_up_sync(0xffffffffu, sr, o);
          if (lane >= o) sr = min(sr + x, cap);
        }
        sr = min(sr + carry, cap);
        if (g0 + lane < p.groups) s_end[g0 + lane] = int(sr);
        carry = __shfl_sync(0xffffffffu, sr, 31);
      }
    }
    __syncthreads();
    // Places.  GRP_K: by falling row count, so that the long sums go out first and what is left at the end is
    // small.  GRP_ROWS: as they come; its tiles are within a factor of two of one another, and a mixture of
    // experts that are bound by reading their matrices (few rows) and by their products keeps both busy (by falling
    // width 64 uneven experts of 2048 x 2048 took 130 us, as they come 128).
    const int row0 = g > 0 && g < p.groups ? s_end[g - 1] : 0;
    const int rows = g < p.groups ? s_end[g] - row0 : 0;
    int place = g;
    if constexpr (GRP == GRP_K) {
      if (g < p.groups) s_rows[g] = rows;
      __syncthreads();
      if (g < p.groups) {
        place = 0;
#pragma unroll 4
        for (int o = 0; o < p.groups; ++o) place += (s_rows[o] > rows || (s_rows[o] == rows && o < g)) ? 1 : 0;
      }
    }
    if (g < p.groups) {
      s_group[place] = uint8_t(g);
      s_tab[kTabRow0 + place] = row0;
      s_tab[kTabRows + place] = rows;
    }
    __syncthreads();
    if constexpr (GRP == GRP_ROWS) {
      if (warp == 3) {
        int carry = 0;
#pragma unroll 1
        for (int g0 = 0; g0 < p.groups; g0 += 32) {
          const int r = g0 + lane < p.groups ? s_tab[kTabRows + g0 + lane] : 0;
          const int mine = ((r + kTrainBN - 1) / kTrainBN) * p.tiles_m;
          int tl = mine;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, tl, o);
            if (lane >= o) tl += x;
          }
          if (g0 + lane < p.groups) s_tab[kTabTile + g0 + lane] = carry + tl - mine;
          carry += __shfl_sync(0xffffffffu, tl, 31);
        }
        if (lane == 0) s_tab[kTabTile + p.groups] = carry;
      }
      __syncthreads();
      num_tiles = s_tab[kTabTile + p.groups];
    }
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
      // The read is over before the arrival (see clc_read_done).  Without that the role that
      // arrives last, the MMA issuer, now and then read the answer after next, missed a tile, and the kernel ran
      // into its wait limit.  (A proxy fence by every reader cost 0.5 us a tile; the scheduler has the one.)
      if constexpr (WARP) __syncwarp();
      if (!WARP || lane == 0) {
        const uint32_t bar = ptx::clc_read_done(clc_empty(cslot), x);
        if (leader)
          ptx::mbar_arrive(bar);
        else
          ptx::mbar_arrive_relaxed_cluster(ptx::map_to_rank(bar, 0));
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
      const uint32_t lead_full0 = ptx::map_to_rank(full_bar(0), 0);
      uint32_t stage = 0, phase = 0;
      uint32_t armed = 0, armed_par = 0;   // stages whose last arming is not yet known complete, and its parity
      bool ok = true;
      uint32_t cslot = 0, cphase = 0;
      if (GRP == GRP_NONE && !C::kNarrow) ptx::pdl_wait();
#pragma unroll 1
      for (int t = first_tile; t >= 0 && ok;) {
        const TrainTile tc = coords(t);
        const void* mA = &tmA;
        const void* mB = &tmB;
        if constexpr (EPI == EPI_F32) {
          // what the epilogue will add to, two tiles or so ahead of it: the additions then find their lines in L2
          if (p.accumulate && tc.nks > 0) {
#pragma unroll 1
            for (int r = 0; r < 128 && tc.a0 + r < p.m; r += 32)
              for (int sub = 0; sub < tc.subs; ++sub)
                ptx::tma_prefetch_3d(&extra.d, tc.n0 + sub * kTrainBN, tc.a0 + r, tc.z);
          }
        }
        const int all_boxes = boxes(tc, 0) + (tc.subs == 2 ? boxes(tc, 1) : 0);
        const uint32_t txb = p.tx_a + uint32_t(all_boxes) * p.tx_box;
#pragma unroll 1
        for (int it = 0; it < tc.nks; ++it) {
          const int k0 = (tc.ks0 + it) * 64;
          if (!wait_bar<false>(empty_bar(stage), phase ^ 1u, ctl)) {
            ok = false;
            break;
          }
          armed &= ~(1u << stage);
          const uint32_t fb = lead_full0 + 8u * stage;
          // GRP_K: rows of this stage, when the group ends in it
          const int last = GRP == GRP_K ? tc.k_end - it * 64 : 64;
          if (leader) {
            // (the rows there are and those up to the MMA's 16, of A's and B's chunks in each CTA)
            ptx::mbar_arrive_expect_tx(full_bar(stage), last < 64 ? uint32_t(2 * (2 + all_boxes) * 128) *
                                                                        ((uint32_t(last) + 15u) & ~15u)
                                                                  : txb);
            armed |= 1u << stage;
            armed_par = (armed_par & ~(1u << stage)) | (phase << stage);
          }
          // a tile of this launch, a ring slot, 16-byte aligned x (TMA's rule), the box inside the stage
          if (invariant(t < num_tiles && stage < nstages && tc.z >= 0 && (!A_MN || tc.a0 % 8 == 0) &&
                            (!B_MN || first_n(tc, 0) % 8 == 0) && tc.nt >= 16 && tc.nt <= C::kBN,
                        p.status)) {
            if (GRP == GRP_K && last < 64) {
              ptx::mbar_arrive(tail_go(stage));   // the stage is free and armed: warp 3 loads it
            } else {
              if constexpr (A_MN) {
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                  const uint32_t dst = stage_a(stage) + uint32_t(c * kTrainChunk);
                  if constexpr (GRP == GRP_ROWS)
                    ptx::tma_load_3d<CG>(dst, mA, tc.a0 + c * 64, k0, tc.z, fb, pol_a);
                  else
                    ptx::tma_load_2d<CG>(dst, mA, tc.a0 + c * 64, tc.k0 + k0, fb, pol_a);
                }
              } else {
                ptx::tma_load_2d<CG>(stage_a(stage), mA, k0, tc.a0, fb, pol_a);
              }
#pragma unroll 1
              for (int sub = 0; sub < tc.subs; ++sub) {
                const uint32_t dst = stage_b(stage) + uint32_t(sub * kTrainBN / 2 * 128);
                const int b0 = first_n(tc, sub), nbox = boxes(tc, sub);
#pragma unroll 1
                for (int c = 0; c < nbox; ++c) {
                  if constexpr (B_MN)
                    ptx::tma_load_2d<CG>(dst + uint32_t(c * kTrainChunk), mB, b0 + c * 64, tc.k0 + k0, fb, pol_b);
                  else
                    ptx::tma_load_2d<CG>(dst + uint32_t(c * 32 * 128), mB, k0, b0 + c * 32, fb, pol_b);
                }
              }
            }
          }
          if (++stage == nstages) {
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
        for (uint32_t s = 0; s < nstages; ++s)
          if (armed & (1u << s)) wait_bar<false>(full_bar(s), (armed_par >> s) & 1u, quiet);
      }
    }
    __syncwarp();
  }
  // ------------------------------------------------------------------ MMA issuer
  else if (warp == 1) {
    if (leader && ptx::elect_one()) {
      uint32_t stage = 0, phase = 0, acc = 0;
      uint32_t accbits = 0;           // parity of each accumulator's next use
      uint32_t uses0 = 0, uses1 = 0;
      bool ok = true;
      if (p.inject_stall) ok = wait_bar<false>(never_bar, 0u, ctl);
      const uint16_t mask = 0x3;
      uint32_t cslot = 0, cphase = 0;
      // the four MMAs of stage s (the tile's stage `it`) into one accumulator, whose sum starts at stage `from`
      auto issue = [&](const TrainTile& tc, uint32_t s, int it, uint32_t acc, uint32_t sub, int from = 0) {
        const uint64_t adesc = A_MN ? sdesc_mn_sw128(stage_a(s)) : sdesc_sw128(stage_a(s));
        const uint32_t b = stage_b(s) + sub * uint32_t(kTrainBN / 2 * 128);
        const uint64_t bdesc = B_MN ? sdesc_mn_sw128(b) : sdesc_sw128(b);
        const uint32_t idesc = idesc_with_n(C::kIdesc, width(tc, int(sub)));
        const int left = tc.k_end - (tc.ks0 + it) * 64;   // k past it are zero, or not there
        const bool stage_ok = invariant(s < nstages && acc < uint32_t(ACC) && tc.nt <= C::kBN, p.status);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (j * 16 >= left || !stage_ok) break;
          // 16 k: 32 bytes along K-major rows, two 8-k groups of 1024 bytes in MN-major chunks
          const uint64_t aoff = A_MN ? uint64_t((j * 2048) >> 4) : uint64_t((j * 32) >> 4);
          const uint64_t boff = B_MN ? uint64_t((j * 2048) >> 4) : uint64_t((j * 32) >> 4);
          ptx::mma_f16<CG>(tmem + acc * uint32_t(C::kBN), adesc + aoff, bdesc + boff, idesc, (it > from || j > 0) ? 1u : 0u);
        }
      };
      auto acc_free = [&](uint32_t acc) {   // the epilogue has handed it back
        if (!wait_bar<true>(acce_bar(acc), ((accbits >> acc) & 1u) ^ 1u, ctl)) return false;
        accbits ^= 1u << acc;
        if (acc) ++uses1; else ++uses0;
        ptx::tc_fence_after();
        return true;
      };
      auto advance = [&](uint32_t& s) {
        if (++s == nstages) s = 0;
        return s == 0;
      };
#pragma unroll 1
      for (int t = first_tile; t >= 0 && ok;) {
        const TrainTile tc = coords(t);
        if constexpr (!C::kDual) {
          int it = 0;
#pragma unroll 1
          do {   // (one turn, but for long sums)
            if (!acc_free(acc)) {
              ok = false;
              break;
            }
            const int from = it, to = C::kSums ? min(it + p.sum_stages, tc.nks) : tc.nks;
#pragma unroll 1
            for (; it < to; ++it) {
              if (!wait_bar<false>(full_bar(stage), phase, ctl)) {
                ok = false;
                break;
              }
              issue(tc, stage, it, acc, 0, from);
              ptx::tc_commit<CG>(empty_bar(stage), mask);
              if (advance(stage)) phase ^= 1u;
            }
            if (!ok) break;
            ptx::tc_commit<CG>(accf_bar(acc), mask);
            acc ^= 1u;
          } while (it < tc.nks);
          if (!ok) break;
        } else {
          // Both accumulators take every stage, but the first runs kSkew stages ahead at the start, while the
          // second is still being read out, and finishes kSkew stages early, so that its read-out begins under
          // the second's last MMAs.  A stage is given back when the second has used it.
          const bool two = tc.subs == 2;
          const int lead = two ? min(C::kSkew, tc.nks) : 0, trail = two ? min(C::kSkew, tc.nks - lead) : 0;
          ok = acc_free(0);
          uint32_t behind = stage;      // the second accumulator's next stage
#pragma unroll 1
          for (int it = 0; it < tc.nks && ok; ++it) {
            if (!wait_bar<false>(full_bar(stage), phase, ctl)) {
              ok = false;
              break;
            }
            if (it == lead && two) {    // catch up
              if (!acc_free(1)) {
                ok = false;
                break;
              }
              for (int i = 0; i < lead; ++i) {
                issue(tc, behind, i, 1, 1);
                ptx::tc_commit<CG>(empty_bar(behind), mask);
                advance(behind);
              }
            }
            issue(tc, stage, it, 0, 0);
            if (!two || (it >= lead && it < tc.nks - trail)) {
              if (two) issue(tc, stage, it, 1, 1);
              ptx::tc_commit<CG>(empty_bar(stage), mask);
              advance(behind);
            }
            if (advance(stage)) phase ^= 1u;
          }
          if (!ok) break;
          ptx::tc_commit<CG>(accf_bar(0), mask);
          if (two) {
            if (tc.nks <= lead && !acc_free(1)) {   // no stage came after the lead: it has not caught up
              ok = false;
              break;
            }
            for (int i = tc.nks <= lead ? 0 : tc.nks - trail; i < tc.nks; ++i) {
              issue(tc, behind, i, 1, 1);
              ptx::tc_commit<CG>(empty_bar(behind), mask);
              advance(behind);
            }
            ptx::tc_commit<CG>(accf_bar(1), mask);
          }
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
        if (uses0) wait_bar<true>(acce_bar(0), (uses0 & 1u) ^ 1u, quiet);
        if (uses1) wait_bar<true>(acce_bar(1), (uses1 & 1u) ^ 1u, quiet);
      }
    }
    __syncwarp();
  }
  // ------------------------------------------------------------------ producer of the stages where groups end
  // The group's last rows, and zeros (rows past the capacity) up to the MMA's 16: what follows in memory is the
  // next group's and may hold anything.  Boxes of 16, 8, 4, 2 and 1 rows, up to 40 copies a stage, beside the main
  // producer, which goes on with the next tile (issued by that one too they made 8 experts of 2048 rows, 4096 x
  // 7168, 6% longer).  One lane issues them in a short loop: one copy per lane, or the loop with its bounds computed
  // inside, took 106 us in place of 80 on 8 experts of few rows.  The 128-byte swizzle goes by the shared-memory
  // address, so a box may start at any row of a chunk.
  else if (warp == 3) {
    if constexpr (GRP == GRP_K) {
      const uint64_t pol = ptx::policy_evict_normal();
      const uint32_t lead_full0 = ptx::map_to_rank(full_bar(0), 0);
      uint32_t stage = 0;
      uint32_t turns = 0;   // parity of each stage's next hand-over
      uint32_t cslot = 0, cphase = 0;
#pragma unroll 1
      for (int t = first_tile; t >= 0;) {
        const TrainTile tc = coords(t);
        stage = (stage + uint32_t(tc.k_end >> 6)) % nstages;   // past the tile's whole stages
        const int last = tc.k_end & 63;
        if (last) {
          // (a stage is handed over again only after this load has been consumed)
          if (!wait_bar_warp<false>(tail_go(stage), (turns >> stage) & 1u, ctl)) break;
          turns ^= 1u << stage;
          const uint32_t fb = lead_full0 + 8u * stage;
          const int n0 = first_n(tc, 0), n1 = first_n(tc, 1), y0 = tc.k0 + tc.k_end - last, up = (last + 15) & ~15;
          if (ptx::elect_one()) {
            int r = 0;
#pragma unroll 1
            while (r < up) {
              const int left = (r < last ? last : up) - r;
              const int i = left >= 16 ? 0 : (left >= 8 ? 1 : (left >= 4 ? 2 : (left >= 2 ? 3 : 4)));
              const int y = r < last ? y0 + r : p.k;
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                const uint32_t off = uint32_t(c * kTrainChunk + r * 128);
                ptx::tma_load_2d<CG>(stage_a(stage) + off, &extra.a[i], tc.a0 + c * 64, y, fb, pol);
                ptx::tma_load_2d<CG>(stage_b(stage) + off, &extra.b[i], n0 + c * 64, y, fb, pol);
              }
              if (C::kDual && tc.subs == 2) {
#pragma unroll
                for (int c = 0; c < 2; ++c)
                  ptx::tma_load_2d<CG>(stage_b(stage) + uint32_t(kTrainBN / 2 * 128 + c * kTrainChunk + r * 128), &extra.b[i],
                                       n1 + c * 64, y, fb, pol);
              }
              r += 16 >> i;
            }
          }
          __syncwarp();
          if (++stage == nstages) stage = 0;
        }
        t = __shfl_sync(0xffffffffu, next_tile(Warp{}, t, cslot, cphase), 0);
      }
    }
    if constexpr (EPI == EPI_DLOGITS) {
      // The weighted rows of X for dW, dealt over the tiles (a launch before this one cost 5 us of the 98 that the
      // gradient of 128 tokens x 32768 x 2048 takes)
      ptx::pdl_wait();
      float top = 0.f;
      if (p.rows) {
#pragma unroll 4
        for (int t = lane; t < p.n; t += 32) top = fmaxf(top, fabsf(ce_weight(t, p.vocab, p.labels, p.dloss, p.alpha)));
#pragma unroll
        for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      }
      const float s = ce_scale(top);
      uint32_t cslot = 0, cphase = 0;
#pragma unroll 1
      for (int t = first_tile; t >= 0;) {
        if (p.rows) {
          const int begin = int((long long)p.n * t / num_tiles), end = int((long long)p.n * (t + 1) / num_tiles);
#pragma unroll 1
          for (int row = begin + int(rank); row < end; row += 2)
            ce_weighted_row(row, lane, p.vocab, p.k, p.x, p.ldx, p.labels, p.dloss, p.alpha, s, p.rows);
          if (t == 0 && leader && lane == 0) *p.rows_scale = s;
        }
        t = __shfl_sync(0xffffffffu, next_tile(Warp{}, t, cslot, cphase), 0);
      }
    }
    __syncwarp();
  }
  // ------------------------------------------------------------------ tile scheduler
  else if (warp == 2) {
    if constexpr (C::kClc) {
      if (GRP == GRP_NONE && !C::kNarrow) ptx::pdl_wait();
      if (leader && ptx::elect_one()) {
        uint32_t slot = 0, ph = 0;
#pragma unroll 1
        while (true) {
          if (!wait_bar<true>(clc_empty(slot), ph ^ 1u, ctl)) break;
          ptx::fence_proxy_async_smem();   // the readers' loads, then the answer's store
          ptx::mbar_arrive_expect_tx(clc_full(slot), 16u);
          ptx::mbar_expect_tx_relaxed_cluster(ptx::map_to_rank(clc_full(slot), 1), 16u);
          ptx::clc_try_cancel<true>(clc_resp(slot), clc_full(slot));
          if (!wait_bar<false>(clc_full(slot), ph, ctl)) break;
          uint32_t x = 0;
          const bool got = ptx::clc_read(clc_resp(slot), x);
          ptx::mbar_arrive(ptx::clc_read_done(clc_empty(slot), x));
          if (++slot == 2) {
            slot = 0;
            ph ^= 1u;
          }
          if (!got) {
            // both CTAs' roles have read the last two answers: no arrival from the other CTA is in flight when
            // this one leaves and its shared memory goes to the next kernel
            for (int i = 0; i < 2; ++i) {
              if (!wait_bar<true>(clc_empty(slot), ph ^ 1u, ctl)) break;
              if (++slot == 2) {
                slot = 0;
                ph ^= 1u;
              }
            }
            break;
          }
        }
      }
    }
    __syncwarp();
  }
  // ------------------------------------------------------------------ epilogue
  else if (warp >= 4) {
    const int e = warp - 4;
    const int q = warp & 3;              // accumulator lane quadrant this warp may read
    const int h = e >> 2;                // which of the tile's chunks: kChunks from h kChunks
    const uint32_t my_buf = epi_base + uint32_t(e * C::kEpiBufBytes);
    const uint32_t acce_lead0 = ptx::map_to_rank(acce_bar(0), 0);
    if (GRP == GRP_NONE && !C::kNarrow) ptx::pdl_wait();
    const float alpha = p.scale ? p.alpha * __ldcg(p.scale) : p.alpha;
    uint32_t acc = 0;
    uint32_t accbits = 0;                // parity of each accumulator's next use
    uint32_t cslot = 0, cphase = 0;
    bool alive = true;
    [[maybe_unused]] uint32_t turn = 0;  // LOSS: tiles so far
    // Stores go through the warp's 2 KB of shared memory: wait until the store that used it last has read it,
    // fill, send.  Rows are written 128 bytes at a time (a lane each, 16 rows to a box): with 64-byte rows a
    // bandwidth-bound weight gradient took 84 us in place of 79 (8 experts, 128 rows, 4096 x 7168).  (g leaves in rows
    // of 64, which free 16 registers: 4096 x 50000 x 256 307 us in place of 316.)
    auto stage_box = [&](auto&& fill, auto&& send) {
      if (lane == 0) ptx::bulk_wait_group_read<0>();
      __syncwarp();
      fill(my_buf);
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        send(my_buf);
        ptx::bulk_commit_group();
      }
    };
    [[maybe_unused]] auto store_rows = [&](const uint32_t (&w)[32], int row0, auto&& send) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        if (row0 + half * 16 >= p.m) break;
        stage_box(
            [&](uint32_t buf) {
              if ((lane >> 4) == half) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                  ptx::st_shared_v4(buf + uint32_t((lane & 15) * 128) + ((uint32_t(j) ^ (uint32_t(lane) & 7u)) << 4),
                                    w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
              }
            },
            [&](uint32_t buf) { send(buf, row0 + half * 16); });
      }
    };
    // Cross entropy: of the tile's columns col0 + 32 c + lane, the labels (-1: ignored, or no such column) and
    // for DLOGITS lse; read one tile ahead
    int label[C::kChunks], label_next[C::kChunks];
    float lse[C::kChunks] = {}, lse_next[C::kChunks] = {};
    auto read_columns = [&](int t, int (&lab)[C::kChunks], float (&ls)[C::kChunks]) {
      if constexpr (EPI == EPI_LOSS || EPI == EPI_DLOGITS) {
        const TrainTile tc = coords(t);
#pragma unroll
        for (int c = 0; c < C::kChunks; ++c) {
          const int col = tc.n0 + h * C::kChunks * 32 + c * 32 + lane;
          lab[c] = -1;
          if (col < tc.n_end) {
            const long long y = __ldcg(p.labels + col);
            lab[c] = (y >= 0 && y < p.vocab) ? int(y) : -1;
            if constexpr (EPI == EPI_DLOGITS) ls[c] = __ldcg(p.lse + col);
          }
        }
      }
    };
    if (first_tile >= 0) read_columns(first_tile, label_next, lse_next);
#pragma unroll 1
    for (int t = first_tile; t >= 0 && alive;) {
      const TrainTile tile = coords(t);
      const int t_next = __shfl_sync(0xffffffffu, next_tile(Warp{}, t, cslot, cphase), 0);
      if (t_next == -2) break;
#pragma unroll
      for (int c = 0; c < C::kChunks; ++c) {
        label[c] = label_next[c];
        lse[c] = lse_next[c];
      }
      if (t_next >= 0) read_columns(t_next, label_next, lse_next);
#pragma unroll 1
      for (int sub = 0; sub < (C::kDual ? tile.subs : 1); ++sub) {
        TrainTile tc = tile;               // the columns of one accumulator
        if constexpr (C::kDual) {
          acc = uint32_t(sub);
          tc.nt = width(tile, sub);
          tc.n0 += sub * kTrainBN;
          tc.n_end = min(tile.n_end, tc.n0 + kTrainBN);
        }
        const int nch = min(max(((tc.nt + 31) >> 5) - C::kChunks * h, 0), C::kChunks);   // this warp's chunks
        const int row0 = tc.a0 + q * 32;                                     // its rows of D
        const int col0 = tc.n0 + h * C::kChunks * 32;                        // and its first column
        // (selects: an array indexed at run time would live in local memory)
        [[maybe_unused]] auto pick = [](const int (&x)[C::kChunks], int c) {
          int r = x[0];
#pragma unroll
          for (int i = 1; i < C::kChunks; ++i) r = c == i ? x[i] : r;
          return r;
        };
        // columns whose label is among this warp's rows (uniform), and each lane's label as such a row
        [[maybe_unused]] auto among_rows = [&](int lab, int& off) {
          off = lab - p.vocab0 - row0;
          return __ballot_sync(0xffffffffu, lab >= 0 && off >= 0 && off < 32 && row0 + off < p.m);
        };
        auto acc_ready = [&]() {
          if (!wait_bar_warp<false>(accf_bar(acc), (accbits >> acc) & 1u, ctl)) return false;
          ptx::tc_fence_after();
          return true;
        };
        if (!acc_ready()) {
          alive = false;
          break;
        }
        const bool idle = !invariant(acc < uint32_t(ACC) && t < num_tiles && tc.nt <= C::kBN, p.status);
        const uint32_t tq = tmem + (uint32_t(q * 32) << 16) + uint32_t(h * C::kChunks * 32);
        [[maybe_unused]] const uint32_t tbase = tq + acc * uint32_t(C::kBN);
        auto hand_back = [&]() {   // every load of this tile has completed
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if (leader)
              ptx::mbar_arrive(acce_bar(acc));
            else
              ptx::mbar_arrive_relaxed_cluster(acce_lead0 + 8u * acc);
          }
          accbits ^= 1u << acc;
          if (!C::kDual) acc ^= 1u;
        };
        // SUMS: this warp's sums gather in registers, and each accumulator goes back as soon as it is read.  (From 0:
        // taking the first as it is selects for every register, and spilled.)
        [[maybe_unused]] auto gather = [&](int n, auto&& read, float (&x)[C::kChunks][32]) {
#pragma unroll
          for (int c = 0; c < C::kChunks; ++c)
#pragma unroll
            for (int j = 0; j < 32; ++j) x[c][j] = 0.f;
#pragma unroll 1
          for (int done = 0;;) {
#pragma unroll
            for (int c = 0; c < C::kChunks; ++c)
              if (c < n) read(c, acc, false, x[c]);
            hand_back();
            done += p.sum_stages;
            if (done >= tc.nks) return true;
            if (!acc_ready()) return false;
          }
        };
        // 32 columns of this lane's row, alone or added to x: 8 at a time, as there are no registers for 32 more
        [[maybe_unused]] auto read_row = [&](int c, uint32_t a, bool first, float (&x)[32]) {
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            uint32_t v[8];
            ptx::tmem_ld_32x32b_x8(tq + a * uint32_t(C::kBN) + uint32_t(c * 32 + u * 8), v);
            ptx::tmem_ld_wait_for(v);
#pragma unroll
            for (int j = 0; j < 8; ++j)
              x[8 * u + j] = first ? __uint_as_float(v[j]) : x[8 * u + j] + __uint_as_float(v[j]);
          }
        };
        // NARROW: a tile's two sums lie in the two accumulators
        [[maybe_unused]] const bool two = C::kNarrow && p.sum_stages < tc.nks;
        if (two) {
          acc ^= 1u;
          if (!acc_ready()) {
            alive = false;
            break;
          }
          acc ^= 1u;
        }
        if constexpr (EPI == EPI_LOSS) {
          float2* stat = s_stat + (turn & 1u) * uint32_t(4 * C::kBN) + h * C::kChunks * 32;
          const uint32_t stat_phase = (turn & 1u);
          ++turn;
          const float c2 = fabsf(p.c2);
          const int rows_there = p.m - row0 - (lane >> 2);   // of rows 0, 8, 16, 24 past this lane's first
          const bool edge = row0 + 32 > p.m;
          const int n = idle ? 0 : nch;
          // x[4 i + 2 k + e]: column 8 i + 2 (t % 4) + e, row t / 4 + 8 k (k = 0, 1), and, from x[16] on, 16 rows on
          auto read = [&](int c, uint32_t a, bool first, float (&x)[32]) {
            const uint32_t from = tq + a * uint32_t(C::kBN) + uint32_t(c * 32);
            uint32_t v[2][16];
            ptx::tmem_ld_16x256b_x4(from, v[0]);
            if (SHAPE != SHAPE_SUMS) ptx::tmem_ld_16x256b_x4(from + (16u << 16), v[1]);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              // (SUMS has no registers for both halves beside the sums)
              if (SHAPE == SHAPE_SUMS && u == 1) ptx::tmem_ld_16x256b_x4(from + (16u << 16), v[1]);
              ptx::tmem_ld_wait_for(v[u]);
#pragma unroll
              for (int j = 0; j < 16; ++j)
                x[16 * u + j] = first ? __uint_as_float(v[u][j]) : x[16 * u + j] + __uint_as_float(v[u][j]);
            }
          };
          auto reduce = [&](int c, float (&x)[32]) {
            // labels among these 32 rows: about one column in vocab / 32
            int off;
#pragma unroll 1
            for (uint32_t left = among_rows(pick(label, c), off); left; left &= left - 1) {
              const int j = __ffs(int(left)) - 1;
              const int row = __shfl_sync(0xffffffffu, off, j);
              const int at = 4 * (j >> 3) + 2 * ((row >> 3) & 1) + (j & 1) + 16 * (row >> 4);
              float z = x[0];
#pragma unroll
              for (int i = 1; i < 32; ++i) z = at == i ? x[i] : z;
              if (lane == 4 * (row & 7) + ((j >> 1) & 3)) p.zlabel[col0 + c * 32 + j] = z * alpha;
            }
            if (p.c2 < 0.f) {
              asm volatile("");   // (a branch, not 32 selects)
#pragma unroll
              for (int j = 0; j < 32; ++j) x[j] = -x[j];
            }
            if (edge) {   // rows past the vocabulary's end
              asm volatile("");
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (((j >> 1) & 1) * 8 + (j >> 4) * 16 >= rows_there) x[j] = -INFINITY;
            }
            float top[8], sum[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int j = 4 * (i >> 1) + (i & 1);
              top[i] = fmaxf(fmaxf(x[j], x[j + 2]), fmaxf(x[j + 16], x[j + 18]));
            }
            const float own = fold_columns(top, lane, [](float a, float b) { return fmaxf(a, b); });
            unfold_columns(own, lane, top);
            // Differences first: the largest logit then counts as exactly 1, and a sum of at least 1 with that logit
            // beside it gives an lse that is not below any logit
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int j = 4 * (i >> 1) + (i & 1);
              const float sub = fabsf(top[i]) == INFINITY ? 0.f : top[i];   // no inf - inf
              sum[i] = (ptx::ex2((x[j] - sub) * c2) + ptx::ex2((x[j + 2] - sub) * c2)) +
                       (ptx::ex2((x[j + 16] - sub) * c2) + ptx::ex2((x[j + 18] - sub) * c2));
            }
            if (c2 == 0.f && edge) {   // scale 0: 0 * -inf is not a number
#pragma unroll
              for (int i = 0; i < 8; ++i)
                sum[i] = float(rows_there > 0) + float(rows_there > 8) + float(rows_there > 16) +
                         float(rows_there > 24);
            }
            const float s = fold_columns(sum, lane, [](float a, float b) { return a + b; });
            stat[q * C::kBN + c * 32 + column_of_lane(lane)] =
                make_float2(own == -INFINITY ? own : own * fabsf(alpha), s);
          };
          if constexpr (SHAPE != SHAPE_SUMS) {
#pragma unroll 1
            for (int c = 0; c < n; ++c) {
              float x[32];
              read(c, acc, true, x);
              if (two) read(c, acc ^ 1u, false, x);
              if (c + 1 == n) {
                hand_back();
                if (two) hand_back();
              }
              reduce(c, x);
            }
            if (n == 0) {
              hand_back();
              if (two) hand_back();
            }
          } else {
            float x[C::kChunks][32];
            if (!gather(n, read, x)) {
              alive = false;
              break;
            }
#pragma unroll
            for (int c = 0; c < C::kChunks; ++c)
              if (c < n) reduce(c, x[c]);
          }
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(stat_bar(h));
          if (!wait_bar_warp<false>(stat_bar(h), stat_phase, ctl)) {
            alive = false;
            break;
          }
          // the four warps' 32 rows each: warp q joins chunk q
          const int col = col0 + q * 32 + lane;
          if (q < nch && !idle && col < tc.n_end && tc.a0 < p.m) {
            float m = -INFINITY, s = 0.f;
            float2 x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              x[i] = stat[i * C::kBN + q * 32 + lane];
              m = fmaxf(m, x[i].x);
            }
            const float sub = fabsf(m) == INFINITY ? 0.f : m;
#pragma unroll
            for (int i = 0; i < 4; ++i) s += x[i].y * ptx::ex2((x[i].x - sub) * kLog2e);
            p.part[size_t(tc.a0 >> 7) * size_t(p.n) + col] = make_float2(m, s);
          }
        } else if constexpr (EPI == EPI_DLOGITS) {
          const int n = idle ? 0 : nch;
          auto read = [&](int c, uint32_t a, bool first, float (&x)[32]) {
            if constexpr (SHAPE == SHAPE_WIDE) {
              uint32_t v[32];
              ptx::tmem_ld_32x32b_x32(tq + a * uint32_t(C::kBN) + uint32_t(c * 32), v);
              ptx::tmem_ld_wait_for(v);
#pragma unroll
              for (int j = 0; j < 32; ++j) x[j] = __uint_as_float(v[j]);
            } else {
              read_row(c, a, first, x);
            }
          };
          auto write = [&](int c, float (&g)[32]) {
            // The logit rounded as the loss has it (__fmul_rn: not fused), and then its difference: the label's
            // exp(z - lse) - 1 is 0 where lse is that logit, and the rounding of z log2(e) (2^-24 of the logit's
            // size) stays out of every g
#pragma unroll
            for (int j = 0; j < 32; ++j)
              g[j] = ptx::ex2((__fmul_rn(g[j], alpha) - __shfl_sync(0xffffffffu, lse[c], j)) * kLog2e);
            int off;
            const uint32_t hits = among_rows(label[c], off);
            if (hits) {
              asm volatile("");   // (a branch, not 32 selects)
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (((hits >> j) & 1u) && lane == __shfl_sync(0xffffffffu, off, j)) g[j] -= 1.f;
            }
            const uint32_t gone = __ballot_sync(0xffffffffu, label[c] < 0);
            if (gone) {   // ignored tokens, whatever their logits and lse are (and columns that are not there)
              asm volatile("");
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if ((gone >> j) & 1u) g[j] = 0.f;
            }
            uint32_t w[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) w[j] = ptx::pack_bf16x2(g[2 * j], g[2 * j + 1]);
            const int at = h * C::kChunks * 32 + c * 32, col = tc.n0 + at;
            if (col >= tc.n_end || row0 >= p.m) return;
            if (at + 32 <= tc.nt) {
              stage_box(
                  [&](uint32_t buf) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                      ptx::st_shared_v4(buf + uint32_t(lane * 64) + ((uint32_t(j) ^ ((uint32_t(lane) >> 1) & 3u)) << 4),
                                        w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
                  },
                  [&](uint32_t buf) {
                    ptx::tma_store_3d(&tmD, buf, col, row0, 0);
                    if (row0 + 16 < p.m) ptx::tma_store_3d(&tmD, buf + 1024u, col, row0 + 16, 0);
                  });
            } else if (row0 + lane < p.m) {   // the tile ends within the 32: its 16 columns (a 32-byte sector)
              uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.d) + size_t(row0 + lane) * p.ldd + col);
              dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
              dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
            }
          };
          if constexpr (SHAPE != SHAPE_SUMS) {
#pragma unroll
            for (int c = 0; c < C::kChunks; ++c) {
              if (c >= n) break;
              float x[32];
              read(c, acc, true, x);
              if (two) read(c, acc ^ 1u, false, x);
              if (c + 1 == n) {
                hand_back();
                if (two) hand_back();
              }
              write(c, x);
            }
            if (n == 0) {
              hand_back();
              if (two) hand_back();
            }
          } else {
            float x[C::kChunks][32];
            if (!gather(n, read, x)) {
              alive = false;
              break;
            }
#pragma unroll
            for (int c = 0; c < C::kChunks; ++c)
              if (c < n) write(c, x[c]);
          }
        } else if constexpr (EPI == EPI_BF16) {   // tiles are a multiple of 64 wide: chunks in pairs
          const int n = idle ? 0 : nch;
          const bool nothing = GRP == GRP_K && tc.nks == 0;   // no rows: the sum is empty, the accumulator undefined
#pragma unroll 1
          for (int c0 = 0; c0 < n; c0 += 2) {
            uint32_t w[32];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              uint32_t v[32];
              ptx::tmem_ld_32x32b_x32(tbase + uint32_t((c0 + c) * 32), v);
              ptx::tmem_ld_wait_for(v);
#pragma unroll
              for (int j = 0; j < 16; ++j)
                w[16 * c + j] = nothing ? 0u
                                        : ptx::pack_bf16x2(__uint_as_float(v[2 * j]) * alpha,
                                                           __uint_as_float(v[2 * j + 1]) * alpha);
            }
            if (c0 + 2 >= n) hand_back();
            const int col = col0 + c0 * 32;
            if (col < tc.n_end && row0 < p.m)
              store_rows(w, row0, [&](uint32_t buf, int r) {
                ptx::tma_store_3d(&tmD, buf, col, r, GRP == GRP_K ? tc.z : 0);
              });
          }
          if (n == 0) hand_back();
        } else {
          const int n = idle ? 0 : nch;
          [[maybe_unused]] const bool nothing = GRP == GRP_K && tc.nks == 0;
          auto write = [&](int c, uint32_t (&v)[32]) {
            const int col = col0 + c * 32;
            if (col >= tc.n_end || row0 >= p.m) return;
            if constexpr (EPI == EPI_BF16_T) {
              // even lanes take column j for rows (lane, lane + 1), odd lanes column j + 1 for rows (lane - 1, lane)
              uint32_t w[16];
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                const float x0 = __uint_as_float(v[2 * j]) * alpha, x1 = __uint_as_float(v[2 * j + 1]) * alpha;
                const float r = __shfl_xor_sync(0xffffffffu, (lane & 1) ? x0 : x1, 1);
                w[j] = (lane & 1) ? ptx::pack_bf16x2(r, x1) : ptx::pack_bf16x2(x0, r);
              }
              const int there = tc.n_end - col;   // columns of the chunk that are the tile's
              if (there >= 16) {
                stage_box(
                    [&](uint32_t buf) {
#pragma unroll
                      for (int j = 0; j < 16; ++j) {
                        const uint32_t r = uint32_t(2 * j + (lane & 1));
                        const uint32_t chunk = (uint32_t(lane) >> 3) ^ ((r >> 1) & 3u);
                        asm volatile("st.shared.b32 [%0], %1;" ::"r"(buf + r * 64u + chunk * 16u +
                                                                     ((uint32_t(lane) >> 1) & 3u) * 4u),
                                     "r"(w[j])
                                     : "memory");
                      }
                    },
                    [&](uint32_t buf) {
                      ptx::tma_store_3d(&tmD, buf, row0, col, 0);
                      if (there >= 32) ptx::tma_store_3d(&tmD, buf + 1024u, row0, col + 16, 0);
                    });
              }
              // fewer than 16 before the tile's or group's end
              if ((there & 15) && there < 32 && row0 + (lane & ~1) < p.m) {
                uint16_t* dst = static_cast<uint16_t*>(p.d) + row0 + (lane & ~1);
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                  const int r = 2 * j + (lane & 1);
                  if (r >= (there & 16) && r < there)
                    *reinterpret_cast<uint32_t*>(dst + size_t(col + r) * p.ldd) = w[j];
                }
              }
            } else {   // F32: tiles are a multiple of 32 wide
              if (nothing && p.accumulate) return;   // adding nothing
#pragma unroll
              for (int j = 0; j < 32; ++j) v[j] = nothing ? 0u : __float_as_uint(__uint_as_float(v[j]) * alpha);
              store_rows(v, row0, [&](uint32_t buf, int r) {
                if (p.accumulate)
                  ptx::tma_add_3d(&tmD, buf, col, r, tc.z);
                else
                  ptx::tma_store_3d(&tmD, buf, col, r, tc.z);
              });
            }
          };
          if constexpr (SHAPE != SHAPE_SUMS) {
#pragma unroll 1
            for (int c = 0; c < n; ++c) {
              uint32_t v[32];
              ptx::tmem_ld_32x32b_x32(tbase + uint32_t(c * 32), v);
              ptx::tmem_ld_wait_for(v);
              if (c + 1 == n) hand_back();
              write(c, v);
            }
            if (n == 0) hand_back();
          } else {
            float x[C::kChunks][32];
            if (!gather(n, read_row, x)) {
              alive = false;
              break;
            }
#pragma unroll
            for (int c = 0; c < C::kChunks; ++c) {
              if (c < n) {
                uint32_t v[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(x[c][j]);
                write(c, v);
              }
            }
          }
        }
      }
      t = t_next;
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
  ptx::cluster_sync_relaxed();
  if (warp == 2) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc<CG>(tmem, uint32_t(2 * C::kBN));
  }
}

}  // namespace tkg
