// grouped_grad.cu -- gradients of the expert-grouped products (row counts in
// device memory): dA = alpha dD B_g per group of rows, dB_g = alpha dD_g^T A_g;
// the latter also with A's rows saved in 8 bits.
#include "mxfp8.cuh"
#include "train_host.cuh"

namespace tkg {
namespace {

tkg_status check_groups(int groups, const int* sizes, int capacity, int n, int k) {
  if (groups < 1 || !sizes || capacity < 0 || n < 0 || k < 0) return TKG_ERR_INVALID_ARG;
  if (groups > kMaxGroups || capacity > kMaxSize || n > kMaxSize || k > kMaxSize) return TKG_ERR_UNSUPPORTED;
  if (!aligned_to(sizes, 4) || n % 8 != 0 || k % 8 != 0) return TKG_ERR_ALIGNMENT;
  return TKG_OK;
}

// Rows saved in 8 bits, in the groups' order, as BF16 (exactly: a code's 4 significant bits and a power of two): row r is
// that of token slots[r] / topk, or r.  2^split warps to a row, 512 columns each in turn, 16 codes to a lane.
// Bound by what it writes: 16384 rows x 7168 take 36 us before a product of 515, 16000 x 2048 16 before 378, 128 x 7168 3
// before 79.  (Pieces of 256 columns with their stores side by side, and one to four loads at once, took the same; stores
// that ask to stay in L2 made 395 of all 16000 rows 414, as what the product adds to then misses.)
constexpr int kUnpackWarps = 4;
__global__ void __launch_bounds__(32 * kUnpackWarps) unpack_rows_kernel(int rows, int k, int tokens, int topk, int split,
                                                                        const uint8_t* __restrict__ Q,
                                                                        const uint8_t* __restrict__ sf,
                                                                        const int* __restrict__ slots,
                                                                        uint16_t* __restrict__ out) {
  ptx::pdl_launch_dependents();
  const long long task = (long long)blockIdx.x * kUnpackWarps + (threadIdx.x >> 5);
  const int r = int(task >> split), part = int(task) & ((1 << split) - 1);
  if (r >= rows) return;
  ptx::pdl_wait();
  int t = r;
  if (slots) {
    const int s = __ldcg(slots + r);
    t = s < 0 ? -1 : int(unsigned(s) / unsigned(topk));
  }
  const bool there = t >= 0 && t < tokens;
  const uint8_t* q_row = Q + size_t(there ? t : 0) * size_t(k);
  const uint8_t* sf_row = sf + size_t(there ? t : 0) * size_t(k / 32);
  uint16_t* out_row = out + size_t(r) * size_t(k);
  const int step = 512 << split;
  constexpr int kAtOnce = 2;
#pragma unroll 1
  for (int c0 = part * 512 + int(threadIdx.x & 31) * 16; c0 < k; c0 += kAtOnce * step) {
    uint4 q[kAtOnce];
    uint32_t scale[kAtOnce];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const int c = c0 + i * step;
      q[i] = make_uint4(0, 0, 0, 0);
      scale[i] = 127;
      if (there && c < k) {
        q[i] = __ldcg(reinterpret_cast<const uint4*>(q_row + c));
        scale[i] = __ldcg(sf_row + c / 32);
      }
    }
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const int c = c0 + i * step;
      if (c >= k) break;
      const float s = e8m0_value(scale[i]);
      const uint32_t u[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
      uint32_t o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float2 v = e4m3x2_values(u[j / 2] >> (16 * (j & 1)));
        o[j] = ptx::pack_bf16x2(v.x * s, v.y * s);
      }
      uint4* dst = reinterpret_cast<uint4*>(out_row + c);
      dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
      dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
  }
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

size_t tkg_gemm_grouped_dev_mxfp8_wgrad_workspace_bytes(int m_capacity, int k) {
  if (m_capacity < 0 || k < 0 || m_capacity > kMaxSize || k > kMaxSize) return 0;
  return size_t(m_capacity) * size_t(k) * 2 + 16;
}

tkg_status tkg_gemm_grouped_dev_mxfp8_wgrad(int groups, const int* m_sizes_dev, int m_capacity, int n, int k,
                                            const void* dD, int tokens, const void* Q, const void* sf, const int* slots,
                                            int topk, void* dB, tkg_grad_type type, float alpha, void* workspace,
                                            size_t workspace_bytes, cudaStream_t stream) {
  tkg_status st = check_groups(groups, m_sizes_dev, m_capacity, n, k);
  if (st != TKG_OK) return st;
  if (tokens < 0 || topk < 1) return TKG_ERR_INVALID_ARG;
  if (tokens > kMaxSize) return TKG_ERR_UNSUPPORTED;
  if (k % 32 != 0 || !aligned_to(Q, 16) || !aligned_to(slots, 4) || !aligned_to(workspace, 16)) return TKG_ERR_ALIGNMENT;
  const bool some = m_capacity > 0 && n > 0 && k > 0;
  if (some) {
    if (!dD || (tokens > 0 && (!Q || !sf)) || !dB || !workspace ||
        workspace_bytes < tkg_gemm_grouped_dev_mxfp8_wgrad_workspace_bytes(m_capacity, k) ||
        (type != TKG_GRAD_BF16 && type != TKG_GRAD_F32 && type != TKG_GRAD_F32_ADD))
      return TKG_ERR_INVALID_ARG;
    if (!aligned_to(dD, 16) || !aligned_to(dB, 16)) return TKG_ERR_ALIGNMENT;
    int split = 0;   // (log2) as many warps per row as it has columns for, while the rows leave SMs idle
    while (((long long)m_capacity << split) < kSMs * 32 && (512 << split) < k) ++split;
    const long long blocks = (((long long)m_capacity << split) + kUnpackWarps - 1) / kUnpackWarps;
    if (blocks > kMaxSize) return TKG_ERR_UNSUPPORTED;
    st = launch_small(unpack_rows_kernel, dim3(unsigned(blocks)), dim3(32 * kUnpackWarps), stream, 0u, m_capacity, k, tokens,
                      topk, split, static_cast<const uint8_t*>(Q), static_cast<const uint8_t*>(sf), slots,
                      static_cast<uint16_t*>(workspace));
    if (st != TKG_OK) return st;
  }
  return tkg_gemm_grouped_dev_bf16_wgrad(groups, m_sizes_dev, m_capacity, n, k, dD, workspace, dB, type, alpha, stream);
}

}  // extern "C"
