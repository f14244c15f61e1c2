// grouped_grad.cu -- gradients of the expert-grouped products (row counts in
// device memory): dA = alpha dD B_g per group of rows, dB_g = alpha dD_g^T A_g.
#include "train_host.cuh"

namespace tkg {
namespace {

// One warp per group: the group's rows (counts past the capacity cut off) and
// tensor maps of its rows of dD and A.  A map covers only the group's own rows,
// so what a 64-row box holds past the group's end arrives as zeros: the next
// group's rows (or the capacity's unused ones, whatever they hold) never enter
// the sum.  Also lists the groups by falling row count: with one tile list for
// all of them the long sums start first and the short ones fill the gaps.
__global__ void __launch_bounds__(kMaxGroups)
    group_maps_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                      const int* sizes, int groups, int capacity, const uint8_t* a, const uint8_t* b,
                      unsigned long long a_row_bytes, unsigned long long b_row_bytes, uint8_t* maps) {
  __shared__ int s_end[kMaxGroups];
  ptx::pdl_launch_dependents();
  ptx::pdl_wait();
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const uint32_t cap = uint32_t(capacity);
  uint32_t sr = t < groups ? min(uint32_t(max(__ldcg(sizes + t), 0)), cap) : 0u;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t x = __shfl_up_sync(0xffffffffu, sr, o);
    if (lane >= o) sr = min(sr + x, cap);
  }
  s_end[t] = int(sr);
  __syncthreads();
  uint32_t end = 0;
  for (int w = 0; w < warp; ++w) end = min(end + uint32_t(s_end[w * 32 + 31]), cap);
  end = min(end + sr, cap);
  __syncthreads();
  s_end[t] = int(end);
  __syncthreads();
  const int g = blockIdx.x;
  const int row0 = g ? s_end[g - 1] : 0, rows = s_end[g] - row0;
  if (warp == 0) {
    // this group's maps
    uint8_t* dst = maps + size_t(g) * 256;
    reinterpret_cast<uint32_t*>(dst)[lane] = reinterpret_cast<const uint32_t*>(&tmA)[lane];
    reinterpret_cast<uint32_t*>(dst + 128)[lane] = reinterpret_cast<const uint32_t*>(&tmB)[lane];
    __syncwarp();
    if (lane == 0 && rows > 0) {
      const uint8_t* base[2] = {a + a_row_bytes * (unsigned long long)row0, b + b_row_bytes * (unsigned long long)row0};
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint64_t m = __cvta_generic_to_global(dst + i * 128);
        asm volatile("tensormap.replace.tile.global_address.global.b1024.b64 [%0], %1;" ::"l"(m), "l"(base[i])
                     : "memory");
        asm volatile("tensormap.replace.tile.global_dim.global.b1024.b32 [%0], 1, %1;" ::"l"(m), "r"(rows) : "memory");
      }
    }
    __syncwarp();
    asm volatile("fence.proxy.tensormap::generic.release.gpu;" ::: "memory");
  } else if (t == 32) {
    // this group's place by falling row count
    int place = 0;
    for (int o = 0; o < groups; ++o) {
      const int ro = s_end[o] - (o ? s_end[o - 1] : 0);
      place += (ro > rows || (ro == rows && o < g)) ? 1 : 0;
    }
    int* tab = reinterpret_cast<int*>(maps + size_t(groups) * 256);
    tab[place] = g;
    tab[kMaxGroups + place] = rows;
  }
}

tkg_status check_groups(int groups, const int* sizes, int capacity, int n, int k) {
  if (groups < 1 || !sizes || capacity < 0 || n < 0 || k < 0) return TKG_ERR_INVALID_ARG;
  if (groups > kMaxGroups) return TKG_ERR_UNSUPPORTED;
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
  if ((st = map_k_major(&tmA, dD, m_capacity, n, size_t(n) * 2, 128)) != TKG_OK) return st;
  // B as groups x n x k, so that rows past n of one expert arrive as zeros
  if ((st = encode_3d_swizzled(&tmB, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, B, uint64_t(k), uint64_t(n), uint64_t(groups),
                               uint64_t(k) * 2, uint64_t(n) * uint64_t(k) * 2, 64, mn_box_rows(n), 1,
                               CU_TENSOR_MAP_SWIZZLE_128B)) != TKG_OK)
    return st;
  if ((st = map_out(&tmD, dA, m_capacity, k, 1, size_t(k) * 2, size_t(m_capacity) * size_t(k) * 2, false)) != TKG_OK)
    return st;
  TrainParams p{};
  p.m = m_capacity;
  p.n = k;
  p.k = n;
  p.splits = 1;
  p.split_stages = ceil_div(n, 64);
  p.alpha = alpha;
  p.sizes = m_sizes_dev;
  p.groups = groups;
  p.d = dA;
  const int cg = option(TKG_OPT_CTA_GROUP);
  // no group can exceed one 128-row tile: single CTAs, as in the forward product
  if (cg == 1 || (cg == 0 && m_capacity <= 128))
    return launch_train<false, true, EPI_BF16, 1, GRP_ROWS>(tmA, tmB, tmD, p, stream);
  return launch_train<false, true, EPI_BF16, 2, GRP_ROWS>(tmA, tmB, tmD, p, stream);
}

size_t tkg_gemm_grouped_dev_bf16_wgrad_workspace_bytes(int groups) {
  if (groups < 1 || groups > kMaxGroups) return 0;
  return size_t(groups) * 256 + 2 * kMaxGroups * sizeof(int);
}

tkg_status tkg_gemm_grouped_dev_bf16_wgrad(int groups, const int* m_sizes_dev, int m_capacity, int n, int k,
                                           const void* dD, const void* A, void* dB, tkg_grad_type type, float alpha,
                                           void* workspace, size_t workspace_bytes, cudaStream_t stream) {
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
  if (!dD || !A || !workspace || workspace_bytes < tkg_gemm_grouped_dev_bf16_wgrad_workspace_bytes(groups))
    return TKG_ERR_INVALID_ARG;
  if (!aligned_to(dD, 16) || !aligned_to(A, 16) || !aligned_to(workspace, 128)) return TKG_ERR_ALIGNMENT;
  CUtensorMap tmA, tmB, tmD;
  // templates of the groups' maps: 64-row boxes whatever the capacity, as the groups' rows are not known here
  if ((st = encode_2d(&tmA, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, dD, uint64_t(n), uint64_t(m_capacity), uint64_t(n) * 2, 64,
                      64, CU_TENSOR_MAP_SWIZZLE_128B)) != TKG_OK)
    return st;
  if ((st = encode_2d(&tmB, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, A, uint64_t(k), uint64_t(m_capacity), uint64_t(k) * 2, 64,
                      64, CU_TENSOR_MAP_SWIZZLE_128B)) != TKG_OK)
    return st;
  if ((st = map_out(&tmD, dB, n, k, groups, size_t(k) * es, size_t(n) * size_t(k) * es, es == 4)) != TKG_OK) return st;
  uint8_t* maps = static_cast<uint8_t*>(workspace);
  if ((st = launch_small(group_maps_kernel, dim3(groups), dim3(kMaxGroups), stream, tmA, tmB, m_sizes_dev, groups,
                         m_capacity, static_cast<const uint8_t*>(dD), static_cast<const uint8_t*>(A),
                         (unsigned long long)n * 2, (unsigned long long)k * 2, maps)) != TKG_OK)
    return st;
  TrainParams p{};
  p.m = n;
  p.n = k;
  p.k = m_capacity;
  p.splits = 1;
  p.alpha = alpha;
  p.groups = groups;
  p.maps = maps;
  p.accumulate = type == TKG_GRAD_F32_ADD;
  if (type == TKG_GRAD_BF16) return launch_train<true, true, EPI_BF16, 2, GRP_K>(tmA, tmB, tmD, p, stream);
  return launch_train<true, true, EPI_F32, 2, GRP_K>(tmA, tmB, tmD, p, stream);
}

}  // extern "C"
