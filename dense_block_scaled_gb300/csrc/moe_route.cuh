// moe_route.cuh -- what routing (moe_route.cu, moe_choose.cuh) and its gradient (moe_route_grad.cu) share: a warp has a token's row of
// logits, each lane a run of consecutive experts.
#pragma once
#include "train_host.cuh"

namespace tkg {

constexpr int kMaxRouteExperts = 512, kMaxTopk = 32, kMaxRouteGroups = 32;

// Types of the logits.
struct LogitF32 {
  float v;
};
struct LogitBF16 {
  unsigned short v;
};

struct RouteParams {
  int tokens, experts, topk;
  int groups, per_group, topk_groups;
  int lanes_per_group, whole_runs;   // a group is that many lanes' runs; otherwise that many lanes read it
  uint32_t inverse;           // ceil(2^32 / per_group): e / per_group is the high word of e * inverse (e < 512)
  __device__ __forceinline__ int group_of(int e) const {
    return per_group == 1 ? e : int(__umulhi(uint32_t(e), inverse));
  }
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
  uint16_t* counts;           // [blocks][experts, rounded up to 8]
  int per_block;              // tokens
  int blocks;
  int cluster;                // blocks of a cluster: all of them, or 1
  unsigned int* status;       // check builds
};

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
// Sigmas of the chosen (a lane each).  Where a logit is below kFarLogit sigma(z) is e^z, subnormal or less, and 1 / (1 +
// exp(-z)) is 0 from -88.7 on.  Where they are divided by their sum, they are made relative to e^top, top the largest of the
// logits where that is negative (else 0), so that they keep their ratios: e^(z - top) / (1 + e^z).  (A function of its own: in
// place it cost routing by softmax, which has none of it, 2%.)
constexpr float kFarLogit = -87.f;
static __device__ __noinline__ float chosen_sigmoids(float z, bool chosen, bool renormalise) {
  if (!__any_sync(0xffffffffu, chosen && z < kFarLogit)) return 1.f / (1.f + expf(-z));
  float top = fminf(warp_fmax(chosen ? z : -INFINITY), 0.f);
  if (!renormalise || top == -INFINITY) top = 0.f;
  return top < 0.f || z < kFarLogit ? expf(z - top) / (1.f + expf(z)) : 1.f / (1.f + expf(-z));
}
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

// What is subtracted from a row's logits (their maximum, or 0 for a row of nothing but -inf).
template <int PER>
__device__ __forceinline__ float softmax_top(const float (&z)[PER]) {
  float top = z[0];
#pragma unroll
  for (int i = 1; i < PER; ++i) top = fmaxf(top, z[i]);
  top = warp_fmax(top);
  return top == -INFINITY ? 0.f : top;
}
template <typename L>
__device__ __forceinline__ float logit_at(const RouteParams& p, int t, int e) {
  const L* row = static_cast<const L*>(p.logits) + size_t(t) * p.ld;
  if constexpr (sizeof(L) == 4)
    return __ldcg(reinterpret_cast<const float*>(row) + e);
  else
    return __uint_as_float(uint32_t(__ldcg(reinterpret_cast<const unsigned short*>(row) + e)) << 16);
}
// ---- host
// How tokens are cut into blocks.  Choosing is spread over the SMs, but each block of tokens has a row of counts that
// the second kernel's blocks all read.  So: one block up to 16 tokens; a cluster of 8, which needs no second kernel, up to
// 256 (by BF16 logits alone; other choices take several times the instructions: 128); then blocks of T / 64 tokens, but 8 to
// 32 (16) of them; and no more blocks than `most`, nor tokens in one than 16 bits can count.
// From a graph, us, 128 experts by BF16 softmax / 256 by FP32 sigmoid with a bias in groups:
//     16 tokens: one block 2.9 / 6.1, cluster 3.4 / 6.9        64: cluster of 8 3.6 / 6.6, of 2 4.7 / 9.7
//    256: cluster 5.0 / 10.2, two kernels 5.1 / 8.1 (2 more from the host)
//    512: blocks of 8 5.5 / 9.1, of 16 5.6 / 9.5, of 32 6.2 / 11.3     1024: of 8 6.8 / 10.6, of 16 6.4 / 10.2
//   2048: of 8 7.3 / 13.6, of 16 6.8 / 14.2, of 32 6.6 / -             4096: of 14 10.6, of 32 8.6 / of 27 16.7, of 32 17.3
constexpr int kMaxCluster = 8, kRouteAlone = 16, kRouteLeast = 8;
inline void route_blocks(RouteParams& p, int most, bool packed) {
  const int t = p.tokens, in_cluster = packed ? 256 : 128, widest = packed ? 32 : 16;
  p.cluster = 1;
  if (t <= kRouteAlone) {
    p.per_block = t;
  } else if (t <= in_cluster) {
    p.per_block = ceil_div(t, kMaxCluster);
    p.cluster = ceil_div(t, p.per_block);
  } else {
    int least = ceil_div(t, 64);
    least = least < kRouteLeast ? kRouteLeast : (least > widest ? widest : least);
    p.per_block = ceil_div(t, most);
    if (p.per_block < least) p.per_block = least;
    if (p.per_block > 65504) p.per_block = 65504;
  }
  p.blocks = ceil_div(t, p.per_block);
}
// Blocks at most, for any kind of choice.
inline int route_most_blocks(int tokens) {
  const int at_least = ceil_div(tokens, 2 * kSMs);
  const int per_block = at_least < kRouteLeast ? kRouteLeast : (at_least > 65504 ? 65504 : at_least);
  return ceil_div(tokens, per_block);
}

// moe_choose_bf16.cu, moe_choose_f32.cu: the choices of all tokens; sets p's blocks of tokens.
tkg_status launch_choose_bf16(RouteParams& p, cudaStream_t stream);
tkg_status launch_choose_f32(RouteParams& p, cudaStream_t stream);

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

inline tkg_status check_route(int tokens, int experts, int topk, const void* logits, tkg_type type, int ld, tkg_scores sc) {
  if (tokens < 0 || experts < 1 || topk < 1 || topk > experts || ld < experts) return TKG_ERR_INVALID_ARG;
  if (type != TKG_TYPE_BF16 && type != TKG_TYPE_F32) return TKG_ERR_INVALID_ARG;
  if (sc != TKG_SCORES_SOFTMAX && sc != TKG_SCORES_SIGMOID) return TKG_ERR_INVALID_ARG;
  if (experts > kMaxRouteExperts || topk > kMaxTopk || (long long)tokens * topk > kMaxSize) return TKG_ERR_UNSUPPORTED;
  if (tokens > 0 && !logits) return TKG_ERR_INVALID_ARG;
  if (!aligned_to(logits, type == TKG_TYPE_F32 ? 4 : 2)) return TKG_ERR_ALIGNMENT;
  return TKG_OK;
}

}  // namespace tkg
