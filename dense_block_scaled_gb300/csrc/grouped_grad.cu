// grouped_grad.cu -- gradients of the expert-grouped products (row counts in
// device memory): dA = alpha dD B_g per group of rows, dB_g = alpha dD_g^T A_g.
#include "train_host.cuh"

namespace tkg {
namespace {

tkg_status check_groups(int groups, const int* sizes, int capacity, int n, int k) {
  if (groups < 1 || !sizes || capacity < 0 || n < 0 || k < 0) return TKG_ERR_INVALID_ARG;
  if (groups > kMaxGroups || capacity > kMaxSize || n > kMaxSize || k > kMaxSize) return TKG_ERR_UNSUPPORTED;
  if (!aligned_to(sizes, 4) || n % 8 != 0 || k % 8 != 0) return TKG_ERR_ALIGNMENT;
  return TKG_OK;
}

}  // namespace
}  // namespace tkg

using namespace tkg;

extern "C" {

tkg_status tkg_gemm_grouped_dev_bf16_dgrad(int groups, const int* m_sizes_dev, int m_capacity, int n, int k,
                                           const void* dD, const void* B, void* dA, float alpha,
                                           cudaStream_t stream) {
  tkg_status st = check_groups(groups, m_sizes_dev, m_capacity, n, k);
  if (st != TKG_OK || m_capacity == 0 || k == 0) return st;
  if (n == 0) return TKG_ERR_UNSUPPORTED;   // the rows to zero are known only on the device
  if (!dD || !B || !dA) return TKG_ERR_INVALID_ARG;
  if (!aligned_to(dD, 16) || !aligned_to(B, 16) || !aligned_to(dA, 16)) return TKG_ERR_ALIGNMENT;
  CUtensorMap tmA, tmB, tmD;
  // B as groups x n x k, so that rows past n of one expert arrive as zeros
  if ((st = encode_3d_swizzled(&tmA, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, B, uint64_t(k), uint64_t(n), uint64_t(groups),
                               uint64_t(k) * 2, uint64_t(n) * uint64_t(k) * 2, 64, mn_box_rows(n), 1,
                               CU_TENSOR_MAP_SWIZZLE_128B)) != TKG_OK)
    return st;
  if ((st = encode_2d(&tmB, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, dD, uint64_t(n), uint64_t(m_capacity), uint64_t(n) * 2, 64,
                      32, CU_TENSOR_MAP_SWIZZLE_128B)) != TKG_OK)
    return st;
  if ((st = map_out(&tmD, dA, m_capacity, k, 1, size_t(k) * 2, size_t(m_capacity) * size_t(k) * 2, false, true)) != TKG_OK)
    return st;
  TrainParams p{};
  p.m = k;
  p.n = m_capacity;
  p.k = n;
  p.n_tile = m_capacity < kTrainBN ? train_n_tile(m_capacity, kTileTokens) : kTrainBN;   // the widest there can be
  p.alpha = alpha;
  p.sizes = m_sizes_dev;
  p.groups = groups;
  p.d = dA;
  p.ldd = size_t(k);
  return launch_train<true, false, EPI_BF16_T, GRP_ROWS>(tmA, tmB, tmD, p, stream);
}

tkg_status tkg_gemm_grouped_dev_bf16_wgrad(int groups, const int* m_sizes_dev, int m_capacity, int n, int k,
                                           const void* dD, const void* A, void* dB, tkg_grad_type type, float alpha,
                                           cudaStream_t stream) {
  tkg_status st = check_groups(groups, m_sizes_dev, m_capacity, n, k);
  if (st != TKG_OK) return st;
  if (type != TKG_GRAD_BF16 && type != TKG_GRAD_F32 && type != TKG_GRAD_F32_ADD) return TKG_ERR_INVALID_ARG;
  if (n == 0 || k == 0) return TKG_OK;
  if (!dB) return TKG_ERR_INVALID_ARG;
  if (!aligned_to(dB, 16)) return TKG_ERR_ALIGNMENT;
  const size_t es = type == TKG_GRAD_BF16 ? 2 : 4;
  if (m_capacity == 0) {   // empty sums
    if (type == TKG_GRAD_F32_ADD) return TKG_OK;
    return cudaMemsetAsync(dB, 0, size_t(groups) * size_t(n) * size_t(k) * es, stream) == cudaSuccess ? TKG_OK
                                                                                                       : TKG_ERR_CUDA;
  }
  if (!dD || !A) return TKG_ERR_INVALID_ARG;
  if (!aligned_to(dD, 16) || !aligned_to(A, 16)) return TKG_ERR_ALIGNMENT;
  // 64-row boxes whatever the capacity (the groups' rows are not known here), and smaller ones for their ends
  CUtensorMap tmA, tmB, tmD;
  TailMaps tail;
  if ((st = map_mn_major(&tmA, dD, n, m_capacity, size_t(n) * 2, 64)) != TKG_OK) return st;
  if ((st = map_mn_major(&tmB, A, k, m_capacity, size_t(k) * 2, 64)) != TKG_OK) return st;
  for (int i = 0; i < kTailMaps; ++i) {
    if ((st = map_mn_major(&tail.a[i], dD, n, m_capacity, size_t(n) * 2, 16 >> i)) != TKG_OK) return st;
    if ((st = map_mn_major(&tail.b[i], A, k, m_capacity, size_t(k) * 2, 16 >> i)) != TKG_OK) return st;
  }
  if ((st = map_out(&tmD, dB, n, k, groups, size_t(k) * es, size_t(n) * size_t(k) * es, es == 4)) != TKG_OK) return st;
  TrainParams p{};
  p.m = n;
  p.n = k;
  p.k = m_capacity;
  p.alpha = alpha;
  p.sizes = m_sizes_dev;
  p.groups = groups;
  p.accumulate = type == TKG_GRAD_F32_ADD;
  // by the rows an expert has on average; additions stay on the narrower tiles, whose epilogues overlap more (8
  // experts of 1024 and 2048 rows, 4096 x 7168: 446 and 715 us against 473 and 728)
  const bool dual = type != TKG_GRAD_F32_ADD && train_dual(n, k, groups, ceil_div(ceil_div(m_capacity, groups), 64));
  if (type == TKG_GRAD_BF16) {
    ExtraMaps<EPI_BF16, GRP_K> extra{};
    static_cast<TailMaps&>(extra) = tail;
    p.n_tile = train_n_tile(k, kTileBF16);
    return dual ? launch_train<true, true, EPI_BF16, GRP_K, SHAPE_DUAL>(tmA, tmB, tmD, p, stream, extra)
                : launch_train<true, true, EPI_BF16, GRP_K>(tmA, tmB, tmD, p, stream, extra);
  }
  ExtraMaps<EPI_F32, GRP_K> extra{};
  static_cast<TailMaps&>(extra) = tail;
  if ((st = map_prefetch(&extra.d, dB, n, k, groups, size_t(k) * 4, size_t(n) * size_t(k) * 4)) != TKG_OK) return st;
  p.n_tile = train_n_tile(k, kTileF32);
  p.sum_stages = kSumStages;
  // A group's sum may be longer than one accumulator takes (16384 positive terms in one were off by 6.7e-5 of the sum,
  // in parts by 2.6e-6).  8 experts of 2048 rows, 4096 x 7168: stored 656 us in place of 633 (in 512-wide tiles), added 696
  // of 686; 64 experts of 250 rows, 2048 x 2048: 187 of 206 and 409 of 404.
  if (m_capacity > 64 * kSumStages)
    return launch_train<true, true, EPI_F32, GRP_K, SHAPE_SUMS>(tmA, tmB, tmD, p, stream, extra);
  return dual ? launch_train<true, true, EPI_F32, GRP_K, SHAPE_DUAL>(tmA, tmB, tmD, p, stream, extra)
              : launch_train<true, true, EPI_F32, GRP_K>(tmA, tmB, tmD, p, stream, extra);
}

}  // extern "C"
