// moe_route_grad.cu -- the gradient of the routing weights to the router's logits, the choice being fixed.
//
// With a_j the chosen scores and da_j their gradients:
//   plain          da_j = scale dw_j
//   renormalised   da_j = scale / A (dw_j - sum_i dw_i a_i / A),  A = sum_i a_i
//   softmax        dz_e = s_e (da_e - sum_j da_j a_j);  renormalised that sum is 0 and
//                  dz_j = scale p_j (dw_j - sum_i dw_i p_i) with p the softmax of the chosen alone
//   sigmoid        dz_e = da_e s_e (1 - s_e)
// A warp per token.  Only softmax without renormalisation reads the whole row; the others read the chosen logits and
// write zeros between them.  10007 x 60 without renormalisation 4.1 us from a graph (7.7 from the host, whose work bounds
// it): 2.7 MB, which is two rounds of latency and a launch.
#include "moe_route.cuh"

namespace tkg {
namespace {

template <int PER, typename L, bool WIDE>
__global__ void __launch_bounds__(256) route_grad_kernel(const __grid_constant__ RouteParams p,
                                                         const float* dweights, void* dlogits, size_t ldd) {
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
    float a = chosen_sigmoids(zj, chosen, p.renormalise);   // (renormalised: their ratios count)
    if (!chosen) a = 0.f;
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

}  // namespace
}  // namespace tkg

using namespace tkg;

extern "C" {

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
  return type == TKG_TYPE_F32 ? go(LogitF32{}) : go(LogitBF16{});
}

}  // extern "C"
