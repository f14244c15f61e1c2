// moe_route.cu -- routing of tokens to experts: scores, choice, weights, and each choice's row in expert order; and the
// weights' gradient to the router's logits.
//
//   s = softmax(z) or sigmoid(z)  (a row of logits per token),  c = s + bias
//   the topk_groups groups (consecutive experts) with the largest sum of their two largest c stay; of their experts the
//   topk with the largest c are chosen, in falling order, ties to the lowest index
//   w_j = scale s_j, or scale s_j / sum_i s_i over the chosen
//   sizes_e = tokens that chose e;  rows(t, j) = place of (t, j) among all choices ordered by expert, then by token;
//   slots(rows(t, j)) = t topk + j
//
// Two kernels.  route_choose_kernel: a warp per token, each lane a run of consecutive experts, so that the lowest lane
// with a value also has the lowest index.  A choice is one integer maximum over the warp (redux) of keys that are
// ordered as the values are.  Within a block of tokens, the rank of (t, e) is the number of earlier tokens that chose e:
// a population count of one bit per token and expert.  The block leaves its ranks (in `rows`) and its count per expert.
// route_place_kernel: adds what earlier blocks and experts have.  A single block of tokens does both at once.
// Nothing depends on the order of atomics: those are integer sums and bit sets.
//
// Without bias and groups the logits themselves decide (both scores rise with them).  Otherwise FP32 scores decide,
// whose error is below the `near` of each value; where two neighbours around a choice are closer than that, and not of
// the same logit and bias, the token is chosen again in 64 bits, so that the choice is that of the exact scores.
#include "train_host.cuh"

namespace tkg {
namespace {

constexpr int kRouteWarps = 16;            // per block
constexpr int kRouteTokens = 32;           // tokens ranked at a time: one bit each
constexpr int kMaxRouteExperts = 512, kMaxTopk = 32, kMaxRouteGroups = 32;
constexpr int kRouteBlocks = 608;          // blocks of tokens at most (four per SM)
constexpr int kPlaceBlocks = 64, kPlaceThreads = 512;
constexpr int kPlaceEach = (kRouteBlocks + kPlaceBlocks - 1) / kPlaceBlocks;   // blocks of tokens per placing block

struct RouteParams {
  int tokens, experts, topk;
  int groups, per_group, topk_groups;
  int sigmoid, renormalise;
  float scale;
  const void* logits;
  size_t ld;                  // elements
  const float* bias;          // may be null
  const uint8_t* keep;        // may be null
  int* ids;
  float* weights;
  int* sizes;
  int* rows;
  int* slots;
  int* counts;                // [blocks][experts]
  int per_block;              // tokens, a multiple of kRouteTokens
  int blocks;
};

// Keys that are ordered as the values: NaN below every number, 0 is no value at all.  (x + 0: -0 is 0.)
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
  return x != x ? 1u : ((u & 0x80000000u) ? ~u : u | 0x80000000u);
}
__device__ __forceinline__ unsigned long long key_of(double x) {
  const unsigned long long u = (unsigned long long)__double_as_longlong(x + 0.0);
  return x != x ? 1ull : ((u >> 63) ? ~u : u | (1ull << 63));
}
__device__ __forceinline__ uint32_t warp_max(uint32_t k) { return __reduce_max_sync(0xffffffffu, k); }
__device__ __forceinline__ unsigned long long warp_max(unsigned long long k) {
  const uint32_t hi = __reduce_max_sync(0xffffffffu, uint32_t(k >> 32));
  const uint32_t lo = __reduce_max_sync(0xffffffffu, uint32_t(k >> 32) == hi ? uint32_t(k) : 0u);
  return ((unsigned long long)hi << 32) | lo;
}
template <typename F>
__device__ __forceinline__ F warp_sum(F x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
__device__ __forceinline__ float warp_fmax(float x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}
__device__ __forceinline__ float exp_of(float x) { return expf(x); }
__device__ __forceinline__ double exp_of(double x) { return exp(x); }

// A lane's run of logits, in FP32; -inf past the end.  WIDE: rows allow loads of the whole run.
template <int PER, typename L, bool WIDE>
__device__ __forceinline__ void load_run(const L* row, int lane, int experts, float (&z)[PER]) {
  constexpr int kBytes = PER * int(sizeof(L));
  const int e0 = lane * PER;
  if constexpr (WIDE) {   // experts is a multiple of PER
    constexpr int kWords = kBytes / 4;
    uint32_t w[kWords > 0 ? kWords : 1] = {};
    if (e0 < experts) {
      if constexpr (kBytes >= 16) {
#pragma unroll
        for (int i = 0; i < kBytes / 16; ++i) {
          const uint4 v = __ldcg(reinterpret_cast<const uint4*>(row + e0) + i);
          w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
        }
      } else if constexpr (kBytes == 8) {
        const uint2 v = __ldcg(reinterpret_cast<const uint2*>(row + e0));
        w[0] = v.x, w[1] = v.y;
      } else {
        w[0] = __ldcg(reinterpret_cast<const unsigned int*>(row + e0));
      }
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if constexpr (sizeof(L) == 4)
        z[i] = __uint_as_float(w[i]);
      else
        z[i] = __uint_as_float((i & 1) ? (w[i / 2] & 0xffff0000u) : (w[i / 2] << 16));
      if (e0 >= experts) z[i] = -INFINITY;
    }
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      z[i] = -INFINITY;
      if (e0 + i < experts) {
        if constexpr (sizeof(L) == 4)
          z[i] = __ldcg(reinterpret_cast<const float*>(row) + e0 + i);
        else
          z[i] = __uint_as_float(uint32_t(__ldcg(reinterpret_cast<const unsigned short*>(row) + e0 + i)) << 16);
      }
    }
  }
}

// Scores of a lane's run.
template <int PER, typename F>
__device__ __forceinline__ void scores(const float (&z)[PER], int lane, int experts, bool sigmoid, F (&s)[PER]) {
  if (sigmoid) {
#pragma unroll
    for (int i = 0; i < PER; ++i) s[i] = F(1) / (F(1) + exp_of(-F(z[i])));
  } else {
    float top = z[0];
#pragma unroll
    for (int i = 1; i < PER; ++i) top = fmaxf(top, z[i]);
    top = warp_fmax(top);
    const F sub = top == -INFINITY ? F(0) : F(top);   // (a row of nothing but -inf has scores 0)
    F sum = F(0);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      s[i] = exp_of(F(z[i]) - sub);
      sum += lane * PER + i < experts ? s[i] : F(0);
    }
    sum = warp_sum(sum);
    if (sum == F(0)) sum = F(1);
#pragma unroll
    for (int i = 0; i < PER; ++i) s[i] /= sum;
  }
}

// What may be wrong with an FP32 score, relative to it.  sigmoid: exp's and the quotient's errors and the sum's rounding,
// a few 2^-24.  softmax: the difference to the largest logit, at most 88 where the score is not 0, is rounded to 2^-24
// of itself and stands in the exponent: 2^-17.5, and the same few.
__device__ __forceinline__ float wrong_of(bool sigmoid) { return sigmoid ? 0x1p-20f : 0x1p-16f; }
// ... and, in all, with a choice score c = s + b, whose sum is rounded.
__device__ __forceinline__ float near_of(float c, float s, bool sigmoid) {
  return s * wrong_of(sigmoid) + fabsf(c) * 0x1p-22f;
}

// The choice of a token by values c (a lane's run; NaN last): lane j < topk gets the j-th expert.  `exact` is cleared
// where FP32 values do not decide.  `box`: per warp, for the groups.
template <int PER, typename F>
__device__ __forceinline__ int choose(const RouteParams& p, const float (&z)[PER], const F (&s)[PER], const F (&c)[PER],
                                      bool by_logit, int lane, F* box, bool& exact) {
  using K = decltype(key_of(F(0)));
  constexpr bool kCheck = sizeof(F) == 4;
  K key[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) key[i] = lane * PER + i < p.experts ? key_of(c[i]) : K(0);
  if (p.topk_groups < p.groups) {
    __syncwarp();
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = lane * PER + i;
      if (e < p.experts) box[e + e / 32] = c[i];
    }
    __syncwarp();
    // lane g: its group's two largest
    F a = -INFINITY, b = -INFINITY;
    bool lost = false;   // (NaN)
    if (lane < p.groups) {
#pragma unroll 4
      for (int i = 0; i < p.per_group; ++i) {
        const int e = lane * p.per_group + i;
        const F x = box[e + e / 32];
        lost |= x != x;
        b = x > a ? a : (x > b ? x : b);
        a = x > a ? x : a;
      }
    }
    const F sum = p.per_group > 1 ? (lost ? F(NAN) : a + b) : (lost ? F(NAN) : a);
    K mine = lane < p.groups ? key_of(sum) : K(0);
    uint32_t stay = 0;
    F last = F(0);
#pragma unroll 1
    for (int g = 0; g <= p.topk_groups; ++g) {
      const K m = warp_max(mine);
      const int at = __ffs(int(__ballot_sync(0xffffffffu, mine == m))) - 1;
      const F v = __shfl_sync(0xffffffffu, sum, at);
      if (g == p.topk_groups) {
        // (the four scores in them: with a bias not known here, at most 4, or 1 of softmax)
        if constexpr (kCheck) {
          const float both = fabsf(v) + fabsf(last);
          const float sums = p.bias ? (p.sigmoid ? 4.f : 1.f) : both;
          if (fabsf(last - v) <= sums * wrong_of(p.sigmoid != 0) + both * 0x1p-21f) exact = false;
        }
        break;
      }
      last = v;
      stay |= 1u << at;
      if (lane == at) mine = K(0);
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = lane * PER + i;
      if (e < p.experts && !((stay >> (e / p.per_group)) & 1u)) key[i] = K(0);
    }
  }
  int id = 0;
  float prev_c = 0.f, prev_z = 0.f, prev_b = 0.f, prev_s = 0.f;
  K top = key[0];
#pragma unroll
  for (int i = 1; i < PER; ++i) top = key[i] > top ? key[i] : top;
  // one more than topk where neighbours are to be compared
  const int picks = kCheck && !by_logit ? p.topk + 1 : p.topk;
#pragma unroll 1
  for (int j = 0; j < picks; ++j) {
    const K m = warp_max(top);
    if (m == K(0)) break;   // (no expert is left to compare with)
    const int at = __ffs(int(__ballot_sync(0xffffffffu, top == m))) - 1;
    int which = 0;
#pragma unroll
    for (int i = PER - 1; i >= 0; --i)
      if (key[i] == m) which = i;
    const int e = __shfl_sync(0xffffffffu, lane * PER + which, at);
    if (lane == j) id = e;
    if (lane == at) {
      top = K(0);
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        if (i == which) key[i] = K(0);
        top = key[i] > top ? key[i] : top;
      }
    }
    if constexpr (kCheck) {
      if (!by_logit) {
        float cc = c[0], zz = z[0], ss = s[0];
#pragma unroll
        for (int i = 1; i < PER; ++i)
          if (which == i) cc = c[i], zz = z[i], ss = s[i];
        cc = __shfl_sync(0xffffffffu, cc, at);
        zz = __shfl_sync(0xffffffffu, zz, at);
        ss = __shfl_sync(0xffffffffu, ss, at);
        const float bb = p.bias ? __ldg(p.bias + e) : 0.f;
        if (j > 0 && !(prev_c - cc > near_of(prev_c, prev_s, p.sigmoid != 0) + near_of(cc, ss, p.sigmoid != 0)) && !(zz == prev_z && bb == prev_b))
          exact = false;
        prev_c = cc, prev_z = zz, prev_b = bb, prev_s = ss;
      }
    }
  }
  return id;
}

// The same in 64 bits: rare, and kept out of the way of the registers of the rest.
template <int PER>
__device__ __noinline__ int choose_again(const RouteParams& p, const float* z_in, int lane, double* box) {
  float z[PER];
  double s[PER], c[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) z[i] = z_in[i];
  scores(z, lane, p.experts, p.sigmoid != 0, s);
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = lane * PER + i;
    c[i] = s[i] + (p.bias && e < p.experts ? double(__ldg(p.bias + e)) : 0.0);
  }
  bool exact = true;
  return choose(p, z, s, c, false, lane, box, exact);
}

template <int PER, typename L, bool WIDE>
__global__ void __launch_bounds__(32 * kRouteWarps) route_choose_kernel(const RouteParams p) {
  extern __shared__ int s_dyn[];
  // bits of the tokens that chose an expert, how many did before, and, for the groups, a row of values per warp
  uint32_t* s_bits = reinterpret_cast<uint32_t*>(s_dyn);
  int* s_count = s_dyn + p.experts;
  int* s_first = s_count + p.experts;   // (one block of tokens: each expert's first row)
  __shared__ int s_ids[kRouteTokens * kMaxTopk];
  __shared__ int s_total;
  ptx::pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  double* box = reinterpret_cast<double*>(s_dyn + (3 * p.experts + 1) / 2 * 2) + warp * (p.experts + p.experts / 32 + 1);
  for (int e = threadIdx.x; e < p.experts; e += blockDim.x) s_count[e] = 0;
  const bool by_logit = !p.bias && p.topk_groups == p.groups;
  const int begin = blockIdx.x * p.per_block, end = min(p.tokens, begin + p.per_block);
  ptx::pdl_wait();
#pragma unroll 1
  for (int t0 = begin; t0 < end; t0 += kRouteTokens) {
    const int there = min(kRouteTokens, end - t0);
    for (int e = threadIdx.x; e < p.experts; e += blockDim.x) s_bits[e] = 0;
    __syncthreads();
#pragma unroll 1
    for (int i = warp; i < there; i += kRouteWarps) {
      const int t = t0 + i;
      const bool kept = !p.keep || __ldcg(p.keep + t) != 0;
      int id = -1;
      float w = 0.f;
      if (kept) {
        float z[PER];
        load_run<PER, L, WIDE>(static_cast<const L*>(p.logits) + size_t(t) * p.ld, lane, p.experts, z);
        bool exact = true;
        float s[PER];
        if (by_logit) {
          if (!p.renormalise || p.sigmoid) {
            scores(z, lane, p.experts, p.sigmoid != 0, s);
          } else {
#pragma unroll
            for (int k = 0; k < PER; ++k) s[k] = 0.f;   // (not needed)
          }
          id = choose(p, z, s, z, true, lane, reinterpret_cast<float*>(box), exact);
        } else {
          float c[PER];
          scores(z, lane, p.experts, p.sigmoid != 0, s);
#pragma unroll
          for (int k = 0; k < PER; ++k) {
            const int e = lane * PER + k;
            c[k] = s[k] + (p.bias && e < p.experts ? __ldg(p.bias + e) : 0.f);
          }
          id = choose(p, z, s, c, false, lane, reinterpret_cast<float*>(box), exact);
          if (!exact) {
            float again[PER];
#pragma unroll
            for (int k = 0; k < PER; ++k) again[k] = z[k];
            id = choose_again<PER>(p, again, lane, box);
          }
        }
        // lane j: its expert's logit and score, from the lane that holds them
        const int from = id / PER, which = id % PER;
        float zj = 0.f, sj = 0.f;
#pragma unroll
        for (int k = 0; k < PER; ++k) {
          const float a = __shfl_sync(0xffffffffu, z[k], from), b = __shfl_sync(0xffffffffu, s[k], from);
          if (which == k) zj = a, sj = b;
        }
        const bool mine = lane < p.topk;
        if (p.renormalise) {
          if (!p.sigmoid) {   // relative to the largest of the chosen: none of them is lost
            const float top = warp_fmax(mine ? zj : -INFINITY);
            sj = expf(zj - (top == -INFINITY ? 0.f : top));
          }
          const float sum = warp_sum(mine ? sj : 0.f);
          sj = sum == 0.f ? 0.f : __fdiv_rn(sj, sum);
        }
        w = sj * p.scale;
        if (mine) atomicOr(s_bits + id, 1u << i);
      }
      if (lane < p.topk) {
        s_ids[i * p.topk + lane] = id;
        p.ids[size_t(t) * p.topk + lane] = id;
        p.weights[size_t(t) * p.topk + lane] = w;
      }
    }
    __syncthreads();
    // ranks within the block of tokens
    if (p.blocks > 1) {
      for (int i = threadIdx.x; i < there * p.topk; i += blockDim.x) {
        const int e = s_ids[i], t = i / p.topk;
        p.rows[size_t(t0) * p.topk + i] = e < 0 ? -1 : s_count[e] + __popc(s_bits[e] & ((1u << t) - 1u));
      }
      __syncthreads();
      for (int e = threadIdx.x; e < p.experts; e += blockDim.x) s_count[e] += __popc(s_bits[e]);
    }
  }
  if (p.blocks > 1) {
    __syncthreads();
    for (int e = threadIdx.x; e < p.experts; e += blockDim.x)
      p.counts[size_t(blockIdx.x) * p.experts + e] = s_count[e];
    return;
  }
  // the only block, with all of the tokens' bits
  if (warp == 0) {
    int carry = 0;
    for (int e0 = 0; e0 < p.experts; e0 += 32) {
      const int e = e0 + lane, n = e < p.experts ? __popc(s_bits[e]) : 0;
      int x = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (e < p.experts) {
        s_first[e] = carry + x - n;
        p.sizes[e] = n;
      }
      carry += __shfl_sync(0xffffffffu, x, 31);
    }
    if (lane == 0) s_total = carry;
  }
  __syncthreads();
  const int all = p.tokens * p.topk;
  for (int i = threadIdx.x; i < all; i += blockDim.x) {
    const int e = s_ids[i], t = i / p.topk;
    const int row = e < 0 ? -1 : s_first[e] + __popc(s_bits[e] & ((1u << t) - 1u));
    p.rows[i] = row;
    if (row >= 0) p.slots[row] = i;
    if (i >= s_total) p.slots[i] = -1;
  }
}

// Block b places the choices of the blocks of tokens [b each, (b + 1) each).
__global__ void __launch_bounds__(kPlaceThreads) route_place_kernel(const RouteParams p, int each) {
  extern __shared__ int s_base[];       // [each][experts]: first row of an expert's choices of a block of tokens
  __shared__ int s_total[kMaxRouteExperts], s_before[kMaxRouteExperts];
  __shared__ int s_all;
  ptx::pdl_launch_dependents();
  const int first = blockIdx.x * each, mine = min(each, p.blocks - first);
  const int lane = threadIdx.x & 31;
  for (int e = threadIdx.x; e < p.experts; e += kPlaceThreads) s_total[e] = s_before[e] = 0;
  ptx::pdl_wait();
  __syncthreads();
  // all counts, in pieces of rows: threads of a piece take neighbouring experts
  const int width = (p.experts + 31) / 32 * 32, pieces = max(1, kPlaceThreads / width);
  for (int x = threadIdx.x; x < width * pieces; x += kPlaceThreads) {
    const int e = x % width, piece = x / width;
    if (e >= p.experts) continue;
    int total = 0, before = 0;
#pragma unroll 8
    for (int b = piece; b < p.blocks; b += pieces) {
      const int n = __ldcg(p.counts + size_t(b) * p.experts + e);
      total += n;
      before += b < first ? n : 0;
      if (b >= first && b < first + mine) s_base[(b - first) * p.experts + e] = n;
    }
    atomicAdd(s_total + e, total);
    atomicAdd(s_before + e, before);
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    int carry = 0;
    for (int e0 = 0; e0 < p.experts; e0 += 32) {
      const int e = e0 + lane, n = e < p.experts ? s_total[e] : 0;
      int x = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (e < p.experts) {
        s_before[e] += carry + x - n;
        if (blockIdx.x == 0) p.sizes[e] = n;
      }
      carry += __shfl_sync(0xffffffffu, x, 31);
    }
    if (lane == 0) s_all = carry;
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.experts; e += kPlaceThreads) {
    int row = s_before[e];
    for (int b = 0; b < mine; ++b) {
      const int n = s_base[b * p.experts + e];
      s_base[b * p.experts + e] = row;
      row += n;
    }
  }
  __syncthreads();
  const long long begin = (long long)first * p.per_block * p.topk;
  const long long end = min((long long)p.tokens, (long long)(first + mine) * p.per_block) * p.topk;
  const int per = p.per_block * p.topk;
  for (long long i = begin + threadIdx.x; i < end; i += kPlaceThreads) {
    const int e = __ldcg(p.ids + i);
    if (e >= 0) {
      const int row = s_base[int(i - begin) / per * p.experts + e] + __ldcg(p.rows + i);
      p.rows[i] = row;
      p.slots[row] = int(i);
    }
    if (i >= s_all) p.slots[i] = -1;
  }
}

// dz of one token per warp.  With a_j the chosen scores, da_j their gradients:
//   plain          da_j = scale dw_j
//   renormalised   da_j = scale / A (dw_j - sum_i dw_i a_i / A),  A = sum_i a_i
//   softmax        dz_e = s_e (da_e - sum_j da_j a_j);  renormalised that sum is 0 and
//                  dz_j = scale p_j (dw_j - sum_i dw_i p_i) with p the softmax of the chosen alone
//   sigmoid        dz_e = da_e s_e (1 - s_e)
template <int PER, typename L, bool WIDE>
__global__ void __launch_bounds__(256) route_grad_kernel(const RouteParams p, const float* dweights, void* dlogits,
                                                         size_t ldd) {
  ptx::pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = blockIdx.x * 8 + warp;
  if (t >= p.tokens) return;
  ptx::pdl_wait();
  const bool mine = lane < p.topk;
  const int id = mine ? __ldcg(p.ids + size_t(t) * p.topk + lane) : -1;
  const bool chosen = id >= 0 && id < p.experts;
  const L* row = static_cast<const L*>(p.logits) + size_t(t) * p.ld;
  const float dw = chosen ? __ldcg(dweights + size_t(t) * p.topk + lane) : 0.f;
  float zj = -INFINITY;
  if (chosen) {
    if constexpr (sizeof(L) == 4)
      zj = __ldcg(reinterpret_cast<const float*>(row) + id);
    else
      zj = __uint_as_float(uint32_t(__ldcg(reinterpret_cast<const unsigned short*>(row) + id)) << 16);
  }
  const bool full = !p.sigmoid && !p.renormalise && __any_sync(0xffffffffu, chosen);   // every logit has a gradient
  float out[PER];
  float dz = 0.f;   // lane j: of the j-th choice
#pragma unroll
  for (int i = 0; i < PER; ++i) out[i] = 0.f;
  if (full) {
    float z[PER], top;
    load_run<PER, L, WIDE>(row, lane, p.experts, z);
    top = z[0];
#pragma unroll
    for (int i = 1; i < PER; ++i) top = fmaxf(top, z[i]);
    top = warp_fmax(top);
    const float sub = top == -INFINITY ? 0.f : top;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      out[i] = expf(z[i] - sub);
      sum += lane * PER + i < p.experts ? out[i] : 0.f;
    }
    sum = warp_sum(sum);
    if (sum == 0.f) sum = 1.f;
    const float inv = __fdiv_rn(1.f, sum);
    const float a = chosen ? expf(zj - sub) * inv : 0.f;
    const float da = dw * p.scale;
    const float dot = warp_sum(chosen ? da * a : 0.f);
#pragma unroll
    for (int i = 0; i < PER; ++i) out[i] = -(out[i] * inv) * dot;
    dz = a * (da - dot);
  } else if (!p.sigmoid) {
    const float top = warp_fmax(zj);
    const float e = chosen ? expf(zj - (top == -INFINITY ? 0.f : top)) : 0.f;
    const float sum = warp_sum(e);
    const float pj = sum == 0.f ? 0.f : __fdiv_rn(e, sum);
    const float dot = warp_sum(chosen ? pj * dw : 0.f);
    dz = p.scale * pj * (dw - dot);
  } else {
    const float a = chosen ? __fdiv_rn(1.f, 1.f + expf(-zj)) : 0.f;
    const float b = chosen ? __fdiv_rn(1.f, 1.f + expf(zj)) : 0.f;   // 1 - a, also where a rounds to 1
    float da = dw * p.scale;
    if (p.renormalise) {
      const float sum = warp_sum(a);
      const float pj = sum == 0.f ? 0.f : __fdiv_rn(a, sum);
      const float dot = warp_sum(chosen ? pj * dw : 0.f);
      dz = p.scale * pj * (dw - dot) * b;
    } else {
      dz = da * a * b;
    }
  }
  const uint32_t who = __ballot_sync(0xffffffffu, chosen);
#pragma unroll 1
  for (uint32_t left = who; left; left &= left - 1) {
    const int j = __ffs(int(left)) - 1;
    const int e = __shfl_sync(0xffffffffu, id, j);
    const float v = __shfl_sync(0xffffffffu, dz, j);
    if (e / PER == lane) {
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (e % PER == i) out[i] = v;
    }
  }
  L* dst = static_cast<L*>(dlogits) + size_t(t) * ldd + lane * PER;
  if constexpr (WIDE) {
    if (lane * PER >= p.experts) return;
    constexpr int kBytes = PER * int(sizeof(L)), kWords = kBytes >= 4 ? kBytes / 4 : 1;
    uint32_t w[kWords];
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      if constexpr (sizeof(L) == 4)
        w[i] = __float_as_uint(out[i]);
      else
        w[i] = ptx::pack_bf16x2(out[2 * i], out[(2 * i + 1) % PER]);
    }
    if constexpr (kBytes >= 16) {
#pragma unroll
      for (int i = 0; i < kBytes / 16; ++i)
        reinterpret_cast<uint4*>(dst)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    } else if constexpr (kBytes == 8) {
      *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
    } else {
      *reinterpret_cast<uint32_t*>(dst) = w[0];
    }
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (lane * PER + i < p.experts) {
        if constexpr (sizeof(L) == 4)
          reinterpret_cast<float*>(dst)[i] = out[i];
        else
          reinterpret_cast<unsigned short*>(dst)[i] = (unsigned short)(ptx::pack_bf16x2(out[i], 0.f) & 0xffffu);
      }
  }
}

struct F32 {
  float v;
};
struct BF16 {
  unsigned short v;
};

// Calls f with a lane's run length and whether rows allow loads of whole runs: runs divide the row, and each starts on
// a multiple of its bytes (of 16 past that).
template <typename L, typename F>
tkg_status with_run(int experts, const void* a, size_t lda, const void* b, size_t ldb, F&& f) {
  auto pick = [&](auto per) {
    constexpr int PER = decltype(per)::value;
    constexpr int kBytes = PER * int(sizeof(L));
    constexpr size_t kAlign = kBytes > 16 ? 16 : kBytes;
    if constexpr (kBytes >= 4) {
      if (experts % PER == 0 && aligned_to(a, kAlign) && aligned_to(b, kAlign) && lda * sizeof(L) % kAlign == 0 &&
          ldb * sizeof(L) % kAlign == 0)
        return f(per, std::true_type{});
    }
    return f(per, std::false_type{});
  };
  const int need = ceil_div(experts, 32);
  if (need <= 1) return pick(std::integral_constant<int, 1>{});
  if (need <= 2) return pick(std::integral_constant<int, 2>{});
  if (need <= 4) return pick(std::integral_constant<int, 4>{});
  if (need <= 8) return pick(std::integral_constant<int, 8>{});
  return pick(std::integral_constant<int, 16>{});
}

void route_blocks(int tokens, int* blocks, int* per_block) {
  const int chunks = ceil_div(tokens, kRouteTokens);
  *per_block = ceil_div(chunks, kRouteBlocks) * kRouteTokens;
  *blocks = ceil_div(tokens, *per_block);
}

tkg_status check_route(int tokens, int experts, int topk, const void* logits, tkg_type type, int ld, tkg_scores sc) {
  if (tokens < 0 || experts < 1 || topk < 1 || topk > experts || ld < experts) return TKG_ERR_INVALID_ARG;
  if (type != TKG_TYPE_BF16 && type != TKG_TYPE_F32) return TKG_ERR_INVALID_ARG;
  if (sc != TKG_SCORES_SOFTMAX && sc != TKG_SCORES_SIGMOID) return TKG_ERR_INVALID_ARG;
  if (experts > kMaxRouteExperts || topk > kMaxTopk || (long long)tokens * topk > kMaxSize) return TKG_ERR_UNSUPPORTED;
  if (tokens > 0 && !logits) return TKG_ERR_INVALID_ARG;
  if (!aligned_to(logits, type == TKG_TYPE_F32 ? 4 : 2)) return TKG_ERR_ALIGNMENT;
  return TKG_OK;
}

template <typename L>
tkg_status launch_route(RouteParams p, cudaStream_t stream) {
  return with_run<L>(p.experts, p.logits, p.ld, p.logits, p.ld, [&](auto per, auto wide) {
    constexpr int PER = decltype(per)::value;
    unsigned smem = unsigned((3 * p.experts + 1) / 2 * 2) * 4u;
    // values of the groups' choice, one row per warp, as large as its second time in 64 bits needs
    if (p.topk_groups < p.groups) smem += unsigned(kRouteWarps * (p.experts + p.experts / 32 + 1)) * 8u;
    auto kern = route_choose_kernel<PER, L, decltype(wide)::value>;
    if (smem > 40000) {
      static bool set[64] = {};   // per instantiation and device
      int dev = 0;
      if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return TKG_ERR_CUDA;
      if (!set[dev]) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 81920) != cudaSuccess) {
          cudaGetLastError();
          return TKG_ERR_CUDA;
        }
        set[dev] = true;
      }
    }
    tkg_status st = launch_small(kern, dim3(unsigned(p.blocks)), dim3(32 * kRouteWarps), stream, smem, p);
    if (st != TKG_OK || p.blocks == 1) return st;
    const int each = ceil_div(p.blocks, kPlaceBlocks);
    return launch_small(route_place_kernel, dim3(unsigned(ceil_div(p.blocks, each))), dim3(kPlaceThreads), stream,
                        unsigned(each * p.experts) * 4u, p, each);
  });
}
static_assert(kPlaceEach * kMaxRouteExperts * 4 + 2 * kMaxRouteExperts * 4 + 16 <= 49152, "shared memory of the placing blocks");

}  // namespace
}  // namespace tkg

using namespace tkg;

extern "C" {

size_t tkg_moe_route_workspace_bytes(int tokens, int experts) {
  if (tokens < 0 || experts < 1 || experts > kMaxRouteExperts || tokens > kMaxSize) return 0;
  int blocks = 0, per_block = 0;
  if (tokens > 0) route_blocks(tokens, &blocks, &per_block);
  return size_t(blocks > 1 ? blocks : 0) * size_t(experts) * 4 + 16;
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
  p.counts = static_cast<int*>(workspace);
  route_blocks(tokens, &p.blocks, &p.per_block);
  return type == TKG_TYPE_F32 ? launch_route<F32>(p, stream) : launch_route<BF16>(p, stream);
}

tkg_status tkg_moe_route_grad(int tokens, int experts, int topk, const void* logits, tkg_type type, int ld,
                              const tkg_route_rule* rule, const int* ids, const float* dweights, void* dlogits, int lddz,
                              cudaStream_t stream) {
  if (!rule) return TKG_ERR_INVALID_ARG;
  tkg_status st = check_route(tokens, experts, topk, logits, type, ld, rule->scores);
  if (st != TKG_OK) return st;
  if (lddz < experts || (rule->renormalise != 0 && rule->renormalise != 1)) return TKG_ERR_INVALID_ARG;
  if (tokens == 0) return TKG_OK;
  if (!ids || !dweights || !dlogits) return TKG_ERR_INVALID_ARG;
  if (!aligned_to(ids, 4) || !aligned_to(dweights, 4) || !aligned_to(dlogits, type == TKG_TYPE_F32 ? 4 : 2))
    return TKG_ERR_ALIGNMENT;
  RouteParams p{};
  p.tokens = tokens;
  p.experts = experts;
  p.topk = topk;
  p.sigmoid = rule->scores == TKG_SCORES_SIGMOID;
  p.renormalise = rule->renormalise;
  p.scale = rule->scale;
  p.logits = logits;
  p.ld = size_t(ld);
  p.ids = const_cast<int*>(ids);
  auto go = [&](auto type_tag) {
    using L = decltype(type_tag);
    return with_run<L>(experts, logits, size_t(ld), dlogits, size_t(lddz), [&](auto per, auto wide) {
      return launch_small(route_grad_kernel<decltype(per)::value, L, decltype(wide)::value>,
                          dim3(unsigned(ceil_div(tokens, 8))), dim3(256), stream, 0u, p, dweights, dlogits, size_t(lddz));
    });
  };
  return type == TKG_TYPE_F32 ? go(F32{}) : go(BF16{});
}

}  // extern "C"
