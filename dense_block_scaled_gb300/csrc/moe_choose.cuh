// moe_choose.cuh -- routing's first kernel: each token's choice of experts, its weights, and the choices' ranks within a
// block of tokens.
//
// A warp per token, each lane a run of consecutive experts.  The topk-th largest of the lanes' largest values bounds the
// topk-th value from below; what is not below that, about topk + 1 candidates, is gathered, one to a lane, and ranked by
// comparing all with all.  (BF16 logits that decide by themselves: value and index share a word, each lane sorts its run,
// and every choice is one integer maximum over the warp.)
//
// Without bias and groups the logits themselves decide (both scores rise with them).  Otherwise FP32 scores decide
// wherever they are further apart than they can be wrong; where two around a choice are closer, and not of the same logit
// and bias, the candidates are ordered again in 64 bits, so that the choice is that of c in 64 bits.
#pragma once
#include <cfloat>

#include "exp64.cuh"
#include "moe_route.cuh"

namespace tkg {
namespace {

// Warps per block: as many as the registers of a lane's run allow, for a token's choice is a long chain of short steps;
// and the blocks of an SM: two where BF16 logits decide by themselves (16384 x 128 15 us, with one 19; 65536 35 and 63;
// the others' FP32 choice takes 64 registers, and 16384 x 256 in groups 29 us with one, 35 in twice as many blocks).
template <int PER, bool PACKED>
constexpr int kRouteWarps = PER <= 8 || PACKED ? 32 : 16;
template <int PER, bool PACKED>
constexpr int kRouteOnSM = PACKED && PER <= 4 ? 2 : 1;
constexpr int kRouteWords = 4;             // 32 tokens each, ranked at a time
constexpr int kRouteTokens = 32 * kRouteWords;
constexpr int kFewTopk = 16;               // choices for which the candidates are hardly ever more than 32

// Keys that are ordered as the values: NaN below every number, 0 is no value at all.  (x + 0: -0 is 0.)
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
  return x != x ? 1u : ((u & 0x80000000u) ? ~u : u | 0x80000000u);
}
__device__ __forceinline__ unsigned long long key_of(double x) {
  const unsigned long long u = (unsigned long long)__double_as_longlong(x + 0.0);
  return x != x ? 1ull : ((u >> 63) ? ~u : u | (1ull << 63));
}
// The value of a key (0 for -0).
__device__ __forceinline__ float value_of(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : (k == 1u ? 0x7fc00000u : ~k));
}
__device__ __forceinline__ uint32_t warp_max(uint32_t k) { return __reduce_max_sync(0xffffffffu, k); }
__device__ __forceinline__ unsigned long long warp_max(unsigned long long k) {
  const uint32_t hi = __reduce_max_sync(0xffffffffu, uint32_t(k >> 32));
  const uint32_t lo = __reduce_max_sync(0xffffffffu, uint32_t(k >> 32) == hi ? uint32_t(k) : 0u);
  return ((unsigned long long)hi << 32) | lo;
}
// (of numbers that are not negative)
__device__ __forceinline__ float warp_most(float x) {
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(x)));
}
// The exponentials of a lane's run and their sum over the row: 1 where all of them are 0.
template <int PER, typename F, typename E>
__device__ __forceinline__ F softmax_sum(const float (&z)[PER], int lane, int experts, float top, F (&e)[PER], E&& exponential) {
  F sum = F(0);
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    e[i] = exponential(F(z[i]) - F(top));
    sum += lane * PER + i < experts ? e[i] : F(0);
  }
  sum = warp_sum(sum);
  return sum == F(0) ? F(1) : sum;
}
__device__ __forceinline__ double sigmoid64(double z) { return 1.0 / (1.0 + exp64(-z)); }

// Choice scores c = s + b of a lane's run, for the choice alone: in FP32 by approximate exponentials and quotients (a
// correctly rounded quotient and exp took 20 instructions each).  `wrong`: what each may be off by.
//   sigmoid, absolute, in units of 2^-24: 1 - s times s (at most 1/4) of ex2's 4 and of its argument's rounding, |z| s (1 - s)
//     < 1/4; the sum's 1, the reciprocal's 2: together below 2^-21.
//   softmax, in the same units of the largest score: ex2's 4 and, with x the distance to the largest logit, its argument's
//     two roundings, 2 x e^-x < 1; of the sum, weighted by the scores, the same with sum 2 p x <= 2 log 512 < 13, and 21
//     additions; the reciprocal's and the product's 3: together below 2^-18.
//   The sum s + b is rounded (infinite biases are not).
template <int PER>
__device__ __forceinline__ void choice_scores(const RouteParams& p, const float (&z)[PER], const float* s_bias, int lane,
                                              float most_bias, float (&c)[PER], float& wrong) {
  float most, b[PER];
  if constexpr (PER >= 4) {
#pragma unroll
    for (int i = 0; i < PER / 4; ++i) {
      const float4 v = reinterpret_cast<const float4*>(s_bias)[lane * (PER / 4) + i];
      b[4 * i] = v.x, b[4 * i + 1] = v.y, b[4 * i + 2] = v.z, b[4 * i + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) b[i] = s_bias[lane * PER + i];
  }
  auto reciprocal = [](float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
  };
  if (p.sigmoid) {
#pragma unroll
    for (int i = 0; i < PER; ++i) c[i] = reciprocal(1.f + ptx::ex2(z[i] * -kLog2e)) + b[i];
    most = 1.f;
    wrong = 0x1p-21f;
  } else {
    float e[PER];
    const float sum = softmax_sum(z, lane, p.experts, softmax_top(z), e, [](float x) { return ptx::ex2(x * kLog2e); });
    most = reciprocal(sum);
#pragma unroll
    for (int i = 0; i < PER; ++i) c[i] = fmaf(e[i], most, b[i]);
    wrong = most * 0x1p-18f;
  }
  wrong += (most + most_bias) * 0x1p-24f;
}
template <int PER>
__device__ __forceinline__ void choice_scores(const RouteParams& p, const float (&z)[PER], const float (&bias)[PER], int lane,
                                              double (&c)[PER]) {
  if (p.sigmoid) {
#pragma unroll
    for (int i = 0; i < PER; ++i) c[i] = sigmoid64(double(z[i])) + double(bias[i]);
  } else {
    const double sum = softmax_sum(z, lane, p.experts, softmax_top(z), c, [](double x) { return exp64(x); });
#pragma unroll
    for (int i = 0; i < PER; ++i) c[i] = c[i] / sum + double(bias[i]);
  }
}

// The larger and the smaller of two keys with their indices (ties: the lower index is the larger).
template <typename K>
__device__ __forceinline__ void order_two(K& a, int& ia, K& b, int& ib) {
  const bool swap = b > a || (b == a && ib < ia);
  const K k = swap ? a : b;
  const int i = swap ? ia : ib;
  a = swap ? b : a;
  ia = swap ? ib : ia;
  b = k;
  ib = i;
}
// Batcher's odd-even merge sort: calls order(a, b) for places a < b of a lane's run.
template <int PER, typename O>
__device__ __forceinline__ void sort_places(O&& order) {
#pragma unroll
  for (int p = 1; p < PER; p *= 2)
#pragma unroll
    for (int k = p; k >= 1; k /= 2)
#pragma unroll
      for (int j = k % p; j + k < PER; j += 2 * k)
#pragma unroll
        for (int i = 0; i < k; ++i)
          if (i + j + k < PER && (i + j) / (2 * p) == (i + j + k) / (2 * p)) order(i + j, i + j + k);
}
template <int PER, typename K>
__device__ __forceinline__ void sort_run(K (&key)[PER], int (&at)[PER]) {
  sort_places<PER>([&](int a, int b) { order_two(key[a], at[a], key[b], at[b]); });
}
template <int PER>
__device__ __forceinline__ void sort_run(uint32_t (&key)[PER]) {
  sort_places<PER>([&](int a, int b) {
    const uint32_t x = max(key[a], key[b]);
    key[b] = min(key[a], key[b]);
    key[a] = x;
  });
}

__device__ __forceinline__ float bias_at(const RouteParams& p, int e) { return p.bias ? __ldcg(p.bias + e) : 0.f; }

// Candidates' scores (lane j < n: logit z) are made again in 64 bits.  These are slow here (16 cycles for an instruction of
// an SM), and softmax has a sum over the row: that is first made of FP32 exponentials, whose arguments' roundings are put
// back, added in 64 bits, so that it is off by little more than exp's 2 ulp, `kSumWrong` of itself.  It scales all
// scores alike, so the order of two values c = s + b is that of the exact sum if they differ by more than that share of
// their scores' difference and what the sums with b are rounded by; only else all of its terms are made in 64 bits.
constexpr double kSumWrong = 0x1p-21;
struct Again {
  double score;
  bool exact;
};
template <int PER, typename L>
__device__ __forceinline__ Again score_again(const RouteParams& p, int t, float zj, int lane, bool exact) {
  if (p.sigmoid) return {sigmoid64(double(zj)), true};
  float z[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) z[i] = lane * PER + i < p.experts ? logit_at<L>(p, t, lane * PER + i) : -INFINITY;
  const float top = softmax_top(z);
  double sum = 0.0;
  if (exact) {
#pragma unroll
    for (int i = 0; i < PER; ++i) sum += exp64(double(z[i]) - double(top));
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const float x = z[i] - top, back = z[i] - x, lost = (z[i] - (x + back)) + (back - top);
      const float e = expf(x);
      sum += z[i] == -INFINITY ? 0.0 : double(fmaf(e, lost, e));
    }
  }
  sum = warp_sum(sum);
  return {exp64(double(zj) - double(top)) / (sum == 0.0 ? 1.0 : sum), exact};
}
// `size`: the sum of sizes of what was rounded on the way to c0 and c1, a unit of whose last places each may differ.
__device__ __forceinline__ bool in_order(const Again& by, double c0, double s0, double c1, double s1, double size) {
  return by.exact || fabs(c0 - c1) > fabs(s0 - s1) * kSumWrong + size * 0x1p-52;
}

// The order of n candidates (lane j < n: expert id) by their exact scores; lane j gets the j-th.  Rare: kept out of the
// way of the registers of the rest.
template <int PER, typename L>
__device__ __noinline__ int order_again(const RouteParams& p, int t, int n, int id, int lane) {
  const float z = lane < n ? logit_at<L>(p, t, id) : 0.f;
  const float b = lane < n ? bias_at(p, id) : 0.f;
  int out = 0;
#pragma unroll 1
  for (int turn = 0; turn < 2; ++turn) {
    const Again by = score_again<PER, L>(p, t, z, lane, turn > 0);
    const double c = by.score + double(b);
    const unsigned long long mine = key_of(c);
    int rank = 0, from = 0;
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
      const unsigned long long other = __shfl_sync(0xffffffffu, mine, i);
      const int e = __shfl_sync(0xffffffffu, id, i);
      rank += other > mine || (other == mine && e < id) ? 1 : 0;
    }
#pragma unroll 4
    for (int i = 0; i < n; ++i)
      if (__shfl_sync(0xffffffffu, rank, i) == lane) from = i;
    out = __shfl_sync(0xffffffffu, id, from);
    // lane j has the j-th: neighbours, but those of the same logit and bias, have to be in order
    const double cj = __shfl_sync(0xffffffffu, c, from), sj = __shfl_sync(0xffffffffu, by.score, from);
    const float zj = __shfl_sync(0xffffffffu, z, from), bj = __shfl_sync(0xffffffffu, b, from);
    const double cn = __shfl_down_sync(0xffffffffu, cj, 1), sn = __shfl_down_sync(0xffffffffu, sj, 1);
    const float zn = __shfl_down_sync(0xffffffffu, zj, 1), bn = __shfl_down_sync(0xffffffffu, bj, 1);
    const bool fine = lane + 1 >= n || in_order(by, cj, sj, cn, sn, fabs(cj) + fabs(cn)) || (zj == zn && bj == bn);
    if (by.exact || __all_sync(0xffffffffu, fine)) break;
  }
  return out;
}

// Which groups stay, where FP32 does not tell: `open` of those that the n candidates for their two largest scores (lane j <
// n: expert id) are of.  Returns a bit per group's first lane.
template <int PER, typename L>
__device__ __noinline__ uint32_t groups_again(const RouteParams& p, int t, int n, int id, int open, int shift, int lane) {
  const float z = lane < n ? logit_at<L>(p, t, id) : 0.f;
  const double b = lane < n ? double(bias_at(p, id)) : 0.0;
  const int g = p.group_of(id);
  uint32_t stay = 0;
#pragma unroll 1
  for (int turn = 0; turn < 2; ++turn) {
    const Again by = score_again<PER, L>(p, t, z, lane, turn > 0);
    const double c = by.score + b;
    const unsigned long long mine = key_of(c);
    int rank = 0;   // within its group
    bool fine = true;
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      const unsigned long long other = __shfl_sync(0xffffffffu, mine, i);
      const double ci = __shfl_sync(0xffffffffu, c, i), si = __shfl_sync(0xffffffffu, by.score, i);
      const int gi = __shfl_sync(0xffffffffu, g, i), e = __shfl_sync(0xffffffffu, id, i);
      if (gi == g && e != id) {
        rank += other > mine || (other == mine && e < id) ? 1 : 0;
        fine &= in_order(by, c, by.score, ci, si, fabs(c) + fabs(ci));
      }
    }
    const bool counts = lane < n && rank < 2, leads = lane < n && rank == 0;
    double two = 0.0, scores = 0.0, size = 0.0;   // of the group
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      const double ci = __shfl_sync(0xffffffffu, counts ? c : 0.0, i);
      const double si = __shfl_sync(0xffffffffu, counts ? by.score : 0.0, i);
      if (__shfl_sync(0xffffffffu, g, i) == g) {
        two += ci;
        scores += si;
        size += 2.0 * fabs(ci);   // (c, and the sum of two)
      }
    }
    const unsigned long long whole = key_of(two);
    int before = 0;   // groups before its group
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      const int gi = __shfl_sync(0xffffffffu, leads ? g : -1, i);
      const unsigned long long other = __shfl_sync(0xffffffffu, whole, i);
      const double ti = __shfl_sync(0xffffffffu, two, i), si = __shfl_sync(0xffffffffu, scores, i);
      const double zi = __shfl_sync(0xffffffffu, size, i);
      if (gi >= 0 && gi != g) {
        before += other > whole || (other == whole && gi < g) ? 1 : 0;
        fine &= in_order(by, two, scores, ti, si, size + zi);
      }
    }
    stay = __reduce_or_sync(0xffffffffu, leads && before < open ? 1u << (g << shift) : 0u);
    if (by.exact || __all_sync(0xffffffffu, fine || lane >= n)) break;
  }
  return stay;
}

// Which of a lane's run are in the best groups (a bit each); `clear` is false where that is not decided, or a value is not
// a number.  Each group has some lanes, its first holds its value: they are its runs' own, or read it from `box` (a row per
// warp).  `few`: places for candidates, or null.
template <int PER, typename L, typename F>
__device__ __forceinline__ uint32_t keep_groups(const RouteParams& p, int t, const F (&c)[PER], float wrong, int lane, F* box,
                                                float2* few, bool& clear) {
  using K = decltype(key_of(F(0)));
  const int per = p.lanes_per_group, shift = __popc(per - 1);
  const int g = lane >> shift;
  F a = -INFINITY, b = -INFINITY;   // the two largest
  int lost = 0;                     // (NaN)
  auto take = [&](F x) {
    lost |= x != x;
    if constexpr (sizeof(F) == 4) {
      b = fmaxf(b, fminf(a, x));
      a = fmaxf(a, x);
    } else {   // (64-bit minima and maxima are calls)
      const F low = x > a ? a : x;
      a = x > a ? x : a;
      b = low > b ? low : b;
    }
  };
  if (p.whole_runs) {
#pragma unroll
    for (int i = 0; i < PER; ++i) take(c[i]);
    if (g >= p.groups) lost = 0;
  } else {
    __syncwarp();
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = lane * PER + i;
      if (e < p.experts) box[e + e / 32] = c[i];
    }
    __syncwarp();
    if (g < p.groups) {
      const int end = (g + 1) * p.per_group;
#pragma unroll 4
      for (int e = g * p.per_group + (lane & (per - 1)); e < end; e += per) take(box[e + e / 32]);
    }
  }
#pragma unroll 1
  for (int o = 1; o < per; o *= 2) {
    const F c2 = __shfl_xor_sync(0xffffffffu, a, o), d2 = __shfl_xor_sync(0xffffffffu, b, o);
    lost |= __shfl_xor_sync(0xffffffffu, lost, o);
    const F low = c2 > a ? a : c2, high = d2 > b ? d2 : b;
    a = c2 > a ? c2 : a;
    b = low > high ? low : high;
  }
  const bool holds = g < p.groups && (lane & (per - 1)) == 0;
  const F sum = lost ? F(NAN) : (p.per_group > 1 ? a + b : a);
  const K mine = holds ? key_of(sum) : K(0);
  int rank = 0;   // groups before this one
#pragma unroll 4
  for (int o = 0; o < p.groups; ++o) {
    const K other = __shfl_sync(0xffffffffu, mine, o << shift);
    rank += other > mine || (other == mine && o < g) ? 1 : 0;
  }
  uint32_t stay = __ballot_sync(0xffffffffu, holds && rank < p.topk_groups);
  // the last group that stays and the first that goes: each sum of two is off by both's error and its rounding
  const uint32_t in = __ballot_sync(0xffffffffu, holds && rank == p.topk_groups - 1);
  const uint32_t out = __ballot_sync(0xffffffffu, holds && rank == p.topk_groups);
  const F last = __shfl_sync(0xffffffffu, sum, __ffs(int(in)) - 1), first = __shfl_sync(0xffffffffu, sum, __ffs(int(out)) - 1);
  const float margin = 4.f * wrong + (fabsf(float(last)) + fabsf(float(first))) * 0x1p-23f;
  clear = float(last - first) > margin;
  if constexpr (sizeof(F) == 4) {
    if (!clear && p.whole_runs && few && fabsf(last) < INFINITY && fabsf(first) < INFINITY &&
        !__any_sync(0xffffffffu, lost != 0)) {
      // groups that are clearly above the first that goes stay, those clearly below the last that stays go; the others'
      // candidates for their two largest are made again
      const uint32_t sure = __ballot_sync(0xffffffffu, holds && sum - first > margin);
      const uint32_t near = __ballot_sync(0xffffffffu, holds && !(sum - first > margin) && !(last - sum > margin));
      const bool mine_near = (near >> (g << shift)) & 1u;
      const float least = (p.per_group > 1 ? b : a) - 2.f * wrong;
      int count = 0;
#pragma unroll
      for (int i = 0; i < PER; ++i) count += mine_near && c[i] >= least ? 1 : 0;
      const int n = __reduce_add_sync(0xffffffffu, count);
      if (n <= 32) {
        int upto = count;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, upto, o);
          if (lane >= o) upto += y;
        }
        float2* to = few + (upto - count);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < PER; ++i)
          if (mine_near && c[i] >= least) *to++ = make_float2(0.f, __int_as_float(lane * PER + i));
        __syncwarp();
        const int id = lane < n ? __float_as_int(few[lane].y) : 0;
        stay = sure | groups_again<PER, L>(p, t, n, id, p.topk_groups - __popc(sure), shift, lane);
        clear = true;
      }
    }
  }
  if (p.whole_runs) return (stay >> (g << shift)) & 1u ? 0xffffffffu : 0u;
  uint32_t kept = 0;
  int in_group = p.group_of(lane * PER), left = (in_group + 1) * p.per_group - lane * PER;   // a run's groups
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (left == 0) {
      ++in_group;
      left = p.per_group;
    }
    --left;
    if (lane * PER + i < p.experts) kept |= ((stay >> (in_group << shift)) & 1u) << i;
  }
  return kept;
}

// Whether two experts have the same logit and bias, so the same score.
template <typename L>
__device__ __forceinline__ bool same_score(const RouteParams& p, int t, int a, int b) {
  return logit_at<L>(p, t, a) == logit_at<L>(p, t, b) && bias_at(p, a) == bias_at(p, b);
}

// The choice of token t by values c (a lane's run), each off by at most `wrong` (negative: exact): lane j < topk gets the
// j-th expert and, where the values are its logits, `value` its logit.  -1 in all lanes where there are more than 32
// candidates, or values among them that are no number above -infinity.  `few`: 32 places per warp.
template <int PER, typename L>
__device__ __forceinline__ int choose_few(const RouteParams& p, int t, const float (&c)[PER], float wrong, int lane,
                                          float2* few, float& value) {
  // the topk-th largest of the lanes' largest values, or -infinity (of equal ones all go at once: then it is less)
  float most = c[0];
#pragma unroll
  for (int i = 1; i < PER; ++i) most = fmaxf(most, c[i]);
  uint32_t mine = key_of(fmaxf(most, -INFINITY)), bound = 0;
#pragma unroll 1
  for (int j = 0; j < p.topk; ++j) {
    bound = warp_max(mine);
    if (mine == bound) mine = 0;
  }
  const float margin = wrong > 0.f ? 2.f * wrong : 0.f;
  // (no lower than the least finite number, which the difference may pass: what is -infinity -- lanes past the last expert,
  // experts of groups that go -- is no candidate)
  const float least = bound > key_of(-INFINITY) ? fmaxf(value_of(bound) - margin, -FLT_MAX) : -FLT_MAX;
  auto candidate = [&](int i) { return c[i] >= least && invariant(lane * PER + i < p.experts, p.status); };
  int count = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) count += candidate(i) ? 1 : 0;
  int upto = count;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += y;
  }
  const int n = __shfl_sync(0xffffffffu, upto, 31);
  if (n > 32 || n < p.topk) return -1;
  float2* to = few + (upto - count);
  __syncwarp();
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (candidate(i)) *to++ = make_float2(c[i], __int_as_float(lane * PER + i));
  __syncwarp();
  const float2 own = few[lane];   // (past n: whatever is there)
  int rank = 0;
#pragma unroll 4
  for (int i = 0; i < n; ++i) {
    const float2 o = few[i];
    rank += o.x > own.x || (o.x == own.x && __float_as_int(o.y) < __float_as_int(own.y)) ? 1 : 0;
  }
  __syncwarp();
  if (lane < n) few[rank] = own;
  __syncwarp();
  const float2 me = few[lane], next = few[lane < 31 ? lane + 1 : 31];
  int id = lane < n ? __float_as_int(me.y) : 0;
  value = me.x;
  if (wrong >= 0.f) {
    // neighbours that are too near, as far as they may belong before the last of the chosen
    const bool near = lane + 1 < n && next.x >= few[p.topk - 1].x - margin && !(me.x - next.x > margin);
    if (__any_sync(0xffffffffu, near)) {
      // (the same logit and bias give the same value)
      const bool close = near && (me.x != next.x || !same_score<L>(p, t, id, __float_as_int(next.y)));
      if (__any_sync(0xffffffffu, close)) id = order_again<PER, L>(p, t, n, id, lane);
    }
  }
  return id;
}

// The same for any values (NaN last) and number of candidates, in FP32 or by exact ones in 64 bits (`wrong` negative): a
// choice at a time.  -1 in all lanes where FP32 does not decide between more than 32 candidates.
template <int PER, typename L, typename F>
__device__ __forceinline__ int choose_any(const RouteParams& p, int t, const F (&c)[PER], uint32_t kept, float wrong,
                                          int lane) {
  using K = decltype(key_of(F(0)));
  const bool sure = wrong < 0.f;
  K key[PER];
  int at[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    key[i] = lane * PER + i < p.experts && ((kept >> i) & 1u) ? key_of(c[i]) : K(0);
    at[i] = lane * PER + i;
  }
  sort_run(key, at);
  int id = 0, j = 0, picks = p.topk;
  K last = K(0);
  bool close = false;   // two of the chosen are too near, or (below) one of the rest is to the last of them
  int e = 0;
#pragma unroll 1
  for (;;) {
#pragma unroll 1
    for (; j < picks; ++j) {
      const K m = warp_max(key[0]);
      const int before = e;
      e = int(__reduce_min_sync(0xffffffffu, key[0] == m ? uint32_t(at[0]) : 0xffffffffu));
      if (lane == j) id = e;
      if (!sure && j > 0) {
        if constexpr (sizeof(K) == 4)
          if (!(value_of(last) - value_of(m) > 2.f * wrong) && !same_score<L>(p, t, before, e)) close = true;
      }
      last = m;
      const bool step = at[0] == e && key[0] == m;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        key[i] = step ? (i + 1 < PER ? key[i + 1 < PER ? i + 1 : 0] : K(0)) : key[i];
        at[i] = step && i + 1 < PER ? at[i + 1 < PER ? i + 1 : 0] : at[i];
      }
    }
    if (sure || picks > p.topk) break;
    if constexpr (sizeof(K) == 4) {
      // Of the rest, those near the last of the chosen may belong before it.  (One of the same logit and bias as the
      // last does not, unless the chosen are ordered again.)
      const K least = key_of(value_of(last) - 2.f * wrong);
      if (!__any_sync(0xffffffffu, key[0] != K(0) && key[0] >= least)) break;
      int near = 0;
      bool other = close;
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (key[i] != K(0) && key[i] >= least) {
          ++near;
          other |= !same_score<L>(p, t, e, at[i]);
        }
      if (!__any_sync(0xffffffffu, other)) break;
      close = true;
      picks = p.topk + __reduce_add_sync(0xffffffffu, near);
      if (picks > 32) return -1;
    }
  }
  if constexpr (sizeof(K) == 4)
    if (close) id = order_again<PER, L>(p, t, j, id, lane);
  return id;
}

// The choice by BF16 logits: key and index share a word, so that one maximum gives both.
template <int PER>
__device__ __forceinline__ int choose_packed(const RouteParams& p, const float (&z)[PER], int lane, float& value) {
  uint32_t key[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = lane * PER + i;
    const uint32_t k = z[i] != z[i] ? 1u : key_of(z[i]) >> 16;   // (-inf has 0x7f)
    key[i] = e < p.experts ? (k << 16) | uint32_t(0xffff - e) : 0u;
  }
  sort_run(key);
  int id = 0;
  uint32_t mine = 0;
#pragma unroll 1
  for (int j = 0; j < p.topk; ++j) {
    const uint32_t m = warp_max(key[0]);
    if (lane == j) mine = m;
    const bool step = key[0] == m;
#pragma unroll
    for (int i = 0; i < PER; ++i) key[i] = step ? (i + 1 < PER ? key[i + 1 < PER ? i + 1 : 0] : 0u) : key[i];
  }
  id = lane < p.topk ? int(0xffffu - (mine & 0xffffu)) : 0;
  const uint32_t k = mine >> 16;
  value = __uint_as_float((k & 0x8000u) ? (k & 0x7fffu) << 16 : (k == 1u ? 0x7fc00000u : (~k & 0xffffu) << 16));
  return id;
}

// The choice where choose_few does not apply: rare, and kept out of the way of the registers of the rest.
template <int PER, typename L>
__device__ __noinline__ int choose_slowly(const RouteParams& p, int t, bool by_logit, const float* s_bias, float most_bias,
                                          int lane, double* box, float2* few) {
  float z[PER];
  bool clear = true;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = lane * PER + i;
    z[i] = e < p.experts ? logit_at<L>(p, t, e) : -INFINITY;
  }
  if (by_logit) return choose_any<PER, L>(p, t, z, 0xffffffffu, -1.f, lane);
  const bool limited = p.topk_groups < p.groups;
  {
    float c[PER], wrong;
    uint32_t kept = 0xffffffffu;
    choice_scores(p, z, s_bias, lane, most_bias, c, wrong);
    if (limited) kept = keep_groups<PER, L>(p, t, c, wrong, lane, reinterpret_cast<float*>(box), few, clear);
    const int id = clear ? choose_any<PER, L>(p, t, c, kept, wrong, lane) : -1;
    if (__shfl_sync(0xffffffffu, id, 0) >= 0) return id;
  }
  double c[PER];
  uint32_t kept = 0xffffffffu;
  float bias[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) bias[i] = s_bias[lane * PER + i];
  choice_scores(p, z, bias, lane, c);
  if (limited) kept = keep_groups<PER, L>(p, t, c, 0.f, lane, box, nullptr, clear);
  return choose_any<PER, L>(p, t, c, kept, -1.f, lane);
}

// BY_LOGIT: no bias and no limit to groups.
template <int PER, typename L, bool WIDE, bool BY_LOGIT>
__global__ void __launch_bounds__(32 * kRouteWarps<PER, BY_LOGIT && sizeof(L) == 2>)
    route_choose_kernel(const __grid_constant__ RouteParams p) {
  constexpr bool kPacked = BY_LOGIT && sizeof(L) == 2;
  extern __shared__ int s_dyn[];
  // bits of the tokens that chose an expert, how many did before, each expert's first row (one block of tokens or cluster),
  // the choices, and, for the groups, a row of values per warp
  uint32_t* s_bits = reinterpret_cast<uint32_t*>(s_dyn);   // [experts][kRouteWords]
  int* s_count = s_dyn + p.experts * kRouteWords;
  __shared__ int s_warp[32];
  ptx::pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __shared__ __align__(16) float s_bias[BY_LOGIT ? 4 : 32 * PER];
  __shared__ float2 s_few[kPacked ? 1 : kRouteWarps<PER, kPacked>][32];
  int* s_first = s_count + p.experts;
  int* s_ids = s_first + p.experts;                          // [kRouteTokens][topk]
  const int tokens_there = min(kRouteTokens, p.per_block), warps = blockDim.x >> 5;
  double* box = reinterpret_cast<double*>(s_dyn + (p.experts * (kRouteWords + 2) + tokens_there * p.topk + 1) / 2 * 2) +
                warp * (p.experts + p.experts / 32 + 1);
  for (int e = threadIdx.x; e < p.experts; e += blockDim.x) s_count[e] = 0;
  const int begin = blockIdx.x * p.per_block, end = min(p.tokens, begin + p.per_block);
  float most_bias = 0.f;   // the largest that takes a rounding
  if constexpr (!BY_LOGIT) {
    ptx::pdl_wait();
    // (through shared memory: 32 warps' runs straight from L2 are 32 times its sectors, all the same ones, 20 us)
    for (int e = threadIdx.x; e < 32 * PER; e += blockDim.x) s_bias[e] = e < p.experts ? bias_at(p, e) : 0.f;
    __syncthreads();
    for (int e = lane; e < p.experts; e += 32) {
      const float b = fabsf(s_bias[e]);
      if (b < INFINITY) most_bias = fmaxf(most_bias, b);
    }
    most_bias = warp_most(most_bias);
  }
  ptx::pdl_wait();
  auto rank_of = [&](int e, int i) {   // tokens of this chunk before i that chose e
    int n = __popc(s_bits[e * kRouteWords + (i >> 5)] & ((1u << (i & 31)) - 1u));
    for (int w = 0; w < (i >> 5); ++w) n += __popc(s_bits[e * kRouteWords + w]);
    return n;
  };
  auto count_of = [&](int e) {
    int n = 0;
#pragma unroll
    for (int w = 0; w < kRouteWords; ++w) n += __popc(s_bits[e * kRouteWords + w]);
    return n;
  };
#pragma unroll 1
  for (int t0 = begin; t0 < end; t0 += kRouteTokens) {
    const int there = min(kRouteTokens, end - t0);
    for (int e = threadIdx.x; e < p.experts * kRouteWords; e += blockDim.x) s_bits[e] = 0;
    __syncthreads();
#pragma unroll 1
    for (int i = warp; i < there; i += warps) {
      const int t = t0 + i;
      const bool kept = !p.keep || __ldcg(p.keep + t) != 0;
      int id = -1;
      float w = 0.f;
      if (kept) {
        float z[PER], zj = 0.f, sub = 0.f, sum = 1.f;
        load_run<PER, L, WIDE>(static_cast<const L*>(p.logits) + size_t(t) * p.ld, lane, p.experts, z);
        if (!p.sigmoid && !p.renormalise) {
          float e[PER];
          sub = softmax_top(z);
          sum = softmax_sum(z, lane, p.experts, sub, e, [](float x) { return expf(x); });
        }
        if constexpr (kPacked) {
          id = choose_packed(p, z, lane, zj);
        } else {
          float c[PER], wrong = -1.f;
          bool clear = true;
#pragma unroll
          for (int k = 0; k < PER; ++k) c[k] = z[k];
          if constexpr (!BY_LOGIT) {
            choice_scores(p, z, s_bias, lane, most_bias, c, wrong);
            uint32_t kept = 0xffffffffu;
            if (p.topk_groups < p.groups)
              kept = keep_groups<PER, L>(p, t, c, wrong, lane, reinterpret_cast<float*>(box), s_few[warp], clear);
            if (WIDE && lane * PER >= p.experts) kept = 0;   // (whole runs)
#pragma unroll
            for (int k = 0; k < PER; ++k)
              if ((!WIDE && lane * PER + k >= p.experts) || !(kept & (1u << k))) c[k] = -INFINITY;
          }
          id = clear && p.topk <= kFewTopk ? choose_few<PER, L>(p, t, c, wrong, lane, s_few[warp], zj) : -1;
          const bool slow = __shfl_sync(0xffffffffu, id, 0) < 0;
          if (slow) id = choose_slowly<PER, L>(p, t, BY_LOGIT, s_bias, most_bias, lane, box, s_few[warp]);
          if (!invariant(unsigned(id) < unsigned(p.experts), p.status)) id = 0;
          if (!BY_LOGIT || slow) zj = logit_at<L>(p, t, id);
        }
        // lane j: its expert's score
        const bool mine = lane < p.topk;
        if (p.sigmoid) {
          w = chosen_sigmoids(zj, mine, p.renormalise);
        } else {
          if (p.renormalise) {   // relative to the largest of the chosen: none of them is lost
            sub = warp_fmax(mine ? zj : -INFINITY);
            if (sub == -INFINITY) sub = 0.f;
          }
          w = expf(zj - sub);
          if (!p.renormalise) w = __fdiv_rn(w, sum);
        }
        if (p.renormalise) {
          const float all = warp_sum(mine ? w : 0.f);
          w = all == 0.f ? 0.f : __fdiv_rn(w, all);
        }
        w *= p.scale;
        if (mine && invariant(unsigned(id) < unsigned(p.experts), p.status))
          atomicOr(s_bits + id * kRouteWords + (i >> 5), 1u << (i & 31));
      }
      if (lane < p.topk) {
        s_ids[i * p.topk + lane] = id;
        p.ids[size_t(t) * p.topk + lane] = id;
        p.weights[size_t(t) * p.topk + lane] = w;
      }
    }
    __syncthreads();
    // ranks within the block of tokens
    if (p.blocks > p.cluster) {
      for (int i = threadIdx.x; i < there * p.topk; i += blockDim.x) {
        const int e = s_ids[i];
        p.rows[size_t(t0) * p.topk + i] = e < 0 ? -1 : s_count[e] + rank_of(e, i / p.topk);
      }
      __syncthreads();
      for (int e = threadIdx.x; e < p.experts; e += blockDim.x) s_count[e] += count_of(e);
      __syncthreads();
    }
  }
  if (p.blocks > p.cluster) {
    const int width = (p.experts + 7) / 8 * 8;
    for (int e = threadIdx.x; e < width; e += blockDim.x)
      p.counts[size_t(blockIdx.x) * width + e] = uint16_t(e < p.experts ? s_count[e] : 0);
    return;
  }
  // One block, or a cluster of them, has all of the tokens' bits: each adds up the others' counts through their shared
  // memory, a thread per expert.
  if (p.cluster > 1) {
    for (int e = threadIdx.x; e < p.experts; e += blockDim.x) s_count[e] = count_of(e);
    __syncthreads();
    ptx::cluster_sync();
  }
  int carry = 0;
  for (int e0 = 0; e0 < p.experts; e0 += blockDim.x) {   // (one turn but for a few tokens and many experts)
    const int e = e0 + threadIdx.x;
    int n = 0, before = 0;
    if (e < p.experts) {
      if (p.cluster == 1) {
        n = count_of(e);
      } else {
        const uint32_t mine = ptx::smem_u32(s_count + e);
        int of[kMaxCluster];
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r)
          of[r] = r < p.cluster ? ptx::ld_cluster(ptx::map_to_rank(mine, uint32_t(r))) : 0;
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r) {
          n += of[r];
          before += r < int(blockIdx.x) ? of[r] : 0;
        }
      }
    }
    int upto = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += y;
    }
    if (lane == 31) s_warp[warp] = upto;
    __syncthreads();
    int sum = 0, below = 0;
    const int used = min(warps, (p.experts - e0 + 31) / 32);   // warps that have experts
#pragma unroll 4
    for (int w = 0; w < used; ++w) {
      below += w < warp ? s_warp[w] : 0;
      sum += s_warp[w];
    }
    if (e < p.experts) {
      s_first[e] = carry + below + upto - n + before;
      if (blockIdx.x == 0) p.sizes[e] = n;
    }
    carry += sum;
    __syncthreads();
  }
  const int base = begin * p.topk, all = (end - begin) * p.topk;
  for (int i = threadIdx.x; i < all; i += blockDim.x) {
    const int e = s_ids[i];
    const int row = e < 0 ? -1 : s_first[e] + rank_of(e, i / p.topk);
    p.rows[base + i] = row;
    if (row >= 0 && invariant(row < p.tokens * p.topk, p.status)) p.slots[row] = base + i;
    if (base + i >= carry) p.slots[base + i] = -1;
  }
  if (p.cluster > 1) {   // no block leaves while another reads its counts
    __syncthreads();
    ptx::cluster_sync();
  }
}

template <typename L>
tkg_status launch_choose(RouteParams& p, cudaStream_t stream) {
  return with_run<L>(p.experts, p.logits, p.ld, p.logits, p.ld, [&](auto per, auto wide) {
    constexpr int PER = decltype(per)::value;
    // groups of whole runs, a power of two of them: their lanes need no shared memory
    const int runs = p.per_group / PER;
    p.whole_runs = p.per_group % PER == 0 && (runs & (runs - 1)) == 0;
    p.lanes_per_group = 1;
    if (p.whole_runs)
      p.lanes_per_group = runs;
    else
      while (2 * p.lanes_per_group * p.groups <= 32) p.lanes_per_group *= 2;
    const bool by_logit = !p.bias && p.topk_groups == p.groups;
    const bool packed = by_logit && sizeof(L) == 2;
    const int most_warps = packed ? kRouteWarps<PER, true> : kRouteWarps<PER, false>;
    route_blocks(p, kSMs * (packed ? kRouteOnSM<PER, true> : kRouteOnSM<PER, false>), packed);
    const int there = p.per_block < kRouteTokens ? p.per_block : kRouteTokens;
    unsigned smem = unsigned((p.experts * (kRouteWords + 2) + there * p.topk + 1) / 2 * 2) * 4u;
    // values of the groups' choice, one row per warp, as large as its second time in 64 bits needs
    if (p.topk_groups < p.groups && !p.whole_runs) smem += unsigned(most_warps * (p.experts + p.experts / 32 + 1)) * 8u;
    auto kern = by_logit ? route_choose_kernel<PER, L, decltype(wide)::value, true>
                         : route_choose_kernel<PER, L, decltype(wide)::value, false>;
    if (smem > 36000) {   // (beside 10 KB of its own)
      static std::atomic<bool> sets[2][64] = {};   // per instantiation and device (set twice alike if two threads race)
      std::atomic<bool>* set = sets[by_logit];
      int dev = 0;
      if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return TKG_ERR_CUDA;
      if (!set[dev]) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 102400) != cudaSuccess) {
          cudaGetLastError();
          return TKG_ERR_CUDA;
        }
        set[dev] = true;
      }
    }
    const int warps = p.per_block < 4 ? 4 : (p.per_block < most_warps ? p.per_block : most_warps);
    return launch_small_cluster(kern, dim3(unsigned(p.blocks)), dim3(32u * unsigned(warps)), unsigned(p.cluster), stream,
                                smem, p);
  });
}

}  // namespace
}  // namespace tkg
