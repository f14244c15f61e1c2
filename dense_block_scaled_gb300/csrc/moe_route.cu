// moe_route.cu -- routing of tokens to experts: scores, choice, weights, and each choice's row in expert order.
//
//   s = softmax(z) or sigmoid(z)  (a row of logits per token),  c = s + bias
//   the topk_groups groups (consecutive experts) with the largest sum of their two largest c stay; of their experts the
//   topk with the largest c are chosen, in falling order, ties to the lowest index
//   w_j = scale s_j, or scale s_j / sum_i s_i over the chosen
//   sizes_e = tokens that chose e;  rows(t, j) = place of (t, j) among all choices ordered by expert, then by token;
//   slots(rows(t, j)) = t topk + j
//
// Two kernels.  The first (moe_choose.cuh) chooses; within a block of tokens, the rank of (t, e) is the number of earlier
// tokens that chose e: a population count of one bit per token and expert.  The block leaves its ranks (in `rows`) and its
// count per expert.  The second adds what earlier blocks and experts have.  For a few tokens (route_blocks) one block or a
// cluster does both at once, its counts exchanged through shared memory.
// Nothing depends on the order of atomics: those are bit sets.
#include "moe_route.cuh"

namespace tkg {
namespace {

constexpr int kPlaceThreads = 512, kPlaceEach = 7;
constexpr int kPlaceEntries = 1024;        // choices that a placing block takes, about

// Block b places the choices of the blocks of tokens [b each, (b + 1) each).  It adds up all counts itself: 16-byte loads
// of 8 experts, all of a thread's on their way at once.
__global__ void __launch_bounds__(kPlaceThreads) route_place_kernel(const __grid_constant__ RouteParams p, int each) {
  // sums of a thread's counts: of all blocks, and of the earlier ones; then [each][experts]: first row of an expert's
  // choices of a block of tokens
  __shared__ __align__(16) int s_part[2][kPlaceThreads * 8];
  __shared__ int s_warp[kPlaceThreads / 32];
  int* s_base = s_part[0];
  static_assert(kMaxRouteExperts <= kPlaceThreads, "a thread per expert");
  static_assert(kPlaceEach * kMaxRouteExperts <= 2 * kPlaceThreads * 8, "the first rows fit in the sums' place");
  ptx::pdl_launch_dependents();
  const int first = blockIdx.x * each, mine = min(each, p.blocks - first);
  const int lane = threadIdx.x & 31;
  const int vecs = (p.experts + 7) / 8, groups = kPlaceThreads / vecs;
  const int vec = threadIdx.x % vecs, group = threadIdx.x / vecs;
  int total[8] = {}, before[8] = {};
  const long long begin = (long long)first * p.per_block * p.topk;
  const long long end = min((long long)p.tokens, (long long)(first + mine) * p.per_block) * p.topk;
  const int per = p.per_block * p.topk;
  ptx::pdl_wait();
  // a thread's first choices and its expert's counts in the block's own blocks of tokens, on their way with the rest
  constexpr int kAhead = 4;
  int ahead_id[kAhead], ahead_rank[kAhead], own[kPlaceEach];
#pragma unroll
  for (int a = 0; a < kAhead; ++a) {
    const long long i = begin + threadIdx.x + a * kPlaceThreads;
    ahead_id[a] = i < end ? __ldcg(p.ids + i) : -1;
    ahead_rank[a] = i < end ? __ldcg(p.rows + i) : 0;
  }
  const int mine_e = threadIdx.x;
#pragma unroll
  for (int b = 0; b < kPlaceEach; ++b)
    own[b] = b < mine && mine_e < p.experts ? int(__ldcg(p.counts + size_t(first + b) * (vecs * 8) + mine_e)) : 0;
  if (group < groups) {
#pragma unroll 8
    for (int b = group; b < p.blocks; b += groups) {
      const uint4 v = __ldcg(reinterpret_cast<const uint4*>(p.counts) + size_t(b) * vecs + vec);
      const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int lo = int(u[i] & 0xffffu), hi = int(u[i] >> 16);
        total[2 * i] += lo;
        total[2 * i + 1] += hi;
        before[2 * i] += b < first ? lo : 0;
        before[2 * i + 1] += b < first ? hi : 0;
      }
    }
    int4* to = reinterpret_cast<int4*>(&s_part[0][(group * vecs + vec) * 8]);
    to[0] = make_int4(total[0], total[1], total[2], total[3]);
    to[1] = make_int4(total[4], total[5], total[6], total[7]);
    to = reinterpret_cast<int4*>(&s_part[1][(group * vecs + vec) * 8]);
    to[0] = make_int4(before[0], before[1], before[2], before[3]);
    to[1] = make_int4(before[4], before[5], before[6], before[7]);
  }
  __syncthreads();
  // a thread per expert
  int all_of = 0, earlier = 0;
  if (mine_e < p.experts) {
#pragma unroll 8
    for (int g = 0; g < groups; ++g) {
      all_of += s_part[0][g * vecs * 8 + mine_e];
      earlier += s_part[1][g * vecs * 8 + mine_e];
    }
  }
  int upto = all_of;   // of this and the warp's earlier experts
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += y;
  }
  if (lane == 31) s_warp[threadIdx.x >> 5] = upto;
  __syncthreads();
  int row = upto - all_of + earlier, sum = 0;
#pragma unroll
  for (int w = 0; w < kPlaceThreads / 32; ++w) {
    row += w < int(threadIdx.x >> 5) ? s_warp[w] : 0;
    sum += s_warp[w];
  }
  if (mine_e < p.experts) {
    if (blockIdx.x == 0) p.sizes[mine_e] = all_of;
#pragma unroll
    for (int b = 0; b < kPlaceEach; ++b) {
      if (b < mine) s_base[b * p.experts + mine_e] = row;
      row += own[b];
    }
  }
  const int s_all = sum;
  __syncthreads();
  auto place = [&](long long i, int e, int rank) {
    if (e >= 0) {
      const int row = s_base[int(i - begin) / per * p.experts + e] + rank;
      p.rows[i] = row;
      if (invariant(unsigned(row) < unsigned(p.tokens * p.topk), p.status)) p.slots[row] = int(i);
    }
    if (i >= s_all) p.slots[i] = -1;
  };
#pragma unroll
  for (int a = 0; a < kAhead; ++a) {
    const long long i = begin + threadIdx.x + a * kPlaceThreads;
    if (i < end) place(i, ahead_id[a], ahead_rank[a]);
  }
#pragma unroll 1
  for (long long i = begin + threadIdx.x + kAhead * kPlaceThreads; i < end; i += kPlaceThreads)
    place(i, __ldcg(p.ids + i), __ldcg(p.rows + i));
}

}  // namespace
}  // namespace tkg

using namespace tkg;

extern "C" {

size_t tkg_moe_route_workspace_bytes(int tokens, int experts) {
  if (tokens < 0 || experts < 1 || experts > kMaxRouteExperts || tokens > kMaxSize) return 0;
  return size_t(route_most_blocks(tokens)) * size_t((experts + 7) / 8 * 8) * 2 + 16;
}

tkg_status tkg_moe_route(int tokens, int experts, int topk, const void* logits, tkg_type type, int ld,
                         const tkg_route_rule* rule, const float* bias, const unsigned char* keep, int* ids,
                         float* weights, int* sizes, int* rows, int* slots, void* workspace, size_t workspace_bytes,
                         cudaStream_t stream) {
  if (!rule) return TKG_ERR_INVALID_ARG;
  tkg_status st = check_route(tokens, experts, topk, logits, type, ld, rule->scores);
  if (st != TKG_OK) return st;
  const int groups = rule->groups, stay = rule->topk_groups;
  if (groups < 1 || stay < 1 || stay > groups || experts % groups != 0 || topk > experts / groups * stay ||
      (rule->renormalise != 0 && rule->renormalise != 1))
    return TKG_ERR_INVALID_ARG;
  if (groups > kMaxRouteGroups) return TKG_ERR_UNSUPPORTED;
  if (!sizes) return TKG_ERR_INVALID_ARG;
  if (!aligned_to(sizes, 4)) return TKG_ERR_ALIGNMENT;
  if (tokens == 0)
    return cudaMemsetAsync(sizes, 0, size_t(experts) * 4, stream) == cudaSuccess ? TKG_OK : TKG_ERR_CUDA;
  if (!ids || !weights || !rows || !slots || !workspace ||
      workspace_bytes < tkg_moe_route_workspace_bytes(tokens, experts))
    return TKG_ERR_INVALID_ARG;
  if (!aligned_to(bias, 4) || !aligned_to(ids, 4) || !aligned_to(weights, 4) || !aligned_to(rows, 4) ||
      !aligned_to(slots, 4) || !aligned_to(workspace, 16))
    return TKG_ERR_ALIGNMENT;
  RouteParams p{};
  p.tokens = tokens;
  p.experts = experts;
  p.topk = topk;
  p.groups = groups;
  p.per_group = experts / groups;
  p.topk_groups = stay;
  p.sigmoid = rule->scores == TKG_SCORES_SIGMOID;
  p.renormalise = rule->renormalise;
  p.scale = rule->scale;
  p.logits = logits;
  p.ld = size_t(ld);
  p.bias = bias;
  p.keep = keep;
  p.ids = ids;
  p.weights = weights;
  p.sizes = sizes;
  p.rows = rows;
  p.slots = slots;
  p.counts = static_cast<uint16_t*>(workspace);
  p.inverse = uint32_t((0x100000000ull + unsigned(p.per_group) - 1) / unsigned(p.per_group));
  if (TKG_CHECK && (st = device_status_word(&p.status)) != TKG_OK) return st;
  st = type == TKG_TYPE_F32 ? launch_choose_f32(p, stream) : launch_choose_bf16(p, stream);
  if (st != TKG_OK || p.blocks == p.cluster) return st;
  int each = kPlaceEntries / (p.per_block * p.topk);
  each = each < 1 ? 1 : (each > kPlaceEach ? kPlaceEach : each);
  return launch_small(route_place_kernel, dim3(unsigned(ceil_div(p.blocks, each))), dim3(kPlaceThreads), stream, 0u, p,
                      each);
}

}  // extern "C"
