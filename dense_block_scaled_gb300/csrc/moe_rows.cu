// moe_rows.cu -- tokens' rows into expert order and back, by the rows that tkg_moe_route wrote.
//
//   dispatch  out[rows(t, j)] = X[t]
//   combine   Y[t] = sum_j w(t, j) O[rows(t, j)]     (FP32 sums in the order of j, rounded once)
//
// Each is the other's gradient (combine with weights 1).  A place outside [0, capacity), such as the -1 of a token that is
// not routed, is left out: dispatch writes nothing for it, combine reads nothing.  (Dispatch reads every token's row, on
// its way beside the places.)
//
// Both are bound by HBM.  Threads go by token and, within its row, by 16 bytes, without a gap between tokens, so that X's
// row is read once and sent to all its places, and all of a token's rows of O are on their way together.  Dispatch of 8192
// tokens x 8 x 4096 92 us (604 MB, 89 at the copy rate); combine of 5003 x 8 x 4096 58 us (54), of 5003 x 6 x 2056 with 30%
// of the tokens padding 20 us (16).
#include "rows.cuh"
#include "train_host.cuh"

namespace tkg {
namespace {

constexpr int kRowThreads = 128;
constexpr int kMaxChoices = 32;

// A thread's token and 16 bytes of its row; false past the last token.
__device__ __forceinline__ bool place_of(int tokens, int vecs, int& t, int& v) {
  int t0, v0;
  divide((unsigned long long)blockIdx.x * kRowThreads, unsigned(vecs), t0, v0);
  const unsigned x = unsigned(v0) + threadIdx.x, more = x / unsigned(vecs);
  t = t0 + int(more);
  v = int(x - more * unsigned(vecs));
  return t < tokens;
}

__global__ void __launch_bounds__(kRowThreads) dispatch_kernel(int tokens, int vecs, int topk, int capacity,
                                                               const uint16_t* X, size_t ldx, const int* rows,
                                                               uint16_t* out, size_t ldo) {
  ptx::pdl_launch_dependents();
  int t, v;
  if (!place_of(tokens, vecs, t, v)) return;
  ptx::pdl_wait();
  const uint4 x = __ldcg(reinterpret_cast<const uint4*>(X + size_t(t) * ldx) + v);
  rows += size_t(t) * topk;
#pragma unroll 1
  for (int j0 = 0; j0 < topk; j0 += 8) {
    int r[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) r[j] = j0 + j < topk ? __ldcg(rows + j0 + j) : -1;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (r[j] >= 0 && r[j] < capacity) reinterpret_cast<uint4*>(out + size_t(r[j]) * ldo)[v] = x;
  }
}

// 16 bytes where `there`, else zeros.  (Volatile, so that the loads of all choices stand together in the order written.)
__device__ __forceinline__ uint4 load_if(bool there, const uint4* from) {
  uint4 x = make_uint4(0, 0, 0, 0);
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %5, 0;\n\t"
      "@p ld.global.cg.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
      : "+r"(x.x), "+r"(x.y), "+r"(x.z), "+r"(x.w)
      : "l"(from), "r"(uint32_t(there)));
  return x;
}

// K: the number of choices, up to 8 (0: any number, 8 at a time).  With a number not known to the compiler the loads did
// not stand together: 5003 x 8 x 4096 took 72 us in place of 58.
template <int K, bool WEIGHTED>
__global__ void __launch_bounds__(kRowThreads) combine_kernel(int tokens, int vecs, int topk, int capacity,
                                                              const uint16_t* O, size_t ldo, const int* rows,
                                                              const float* weights, uint16_t* Y, size_t ldy) {
  constexpr int kAtOnce = K > 0 ? K : 8;
  ptx::pdl_launch_dependents();
  int t, v;
  if (!place_of(tokens, vecs, t, v)) return;
  ptx::pdl_wait();
  float sum[8] = {};
  rows += size_t(t) * topk;
  if (WEIGHTED) weights += size_t(t) * topk;
#pragma unroll 1
  for (int j0 = 0; j0 < (K > 0 ? 1 : topk); j0 += 8) {
    int r[kAtOnce];
    float w[kAtOnce];
    uint4 x[kAtOnce];
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) r[j] = K > 0 || j0 + j < topk ? __ldcg(rows + j0 + j) : -1;
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) w[j] = WEIGHTED && (K > 0 || j0 + j < topk) ? __ldcg(weights + j0 + j) : 1.f;
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      const bool there = unsigned(r[j]) < unsigned(capacity);
      x[j] = load_if(there, reinterpret_cast<const uint4*>(O + size_t(there ? r[j] : 0) * ldo) + v);
      w[j] = there ? w[j] : 0.f;
    }
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      const uint32_t u[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        sum[2 * i] = fmaf(w[j], __uint_as_float(u[i] << 16), sum[2 * i]);
        sum[2 * i + 1] = fmaf(w[j], __uint_as_float(u[i] & 0xffff0000u), sum[2 * i + 1]);
      }
    }
  }
  reinterpret_cast<uint4*>(Y + size_t(t) * ldy)[v] =
      make_uint4(ptx::pack_bf16x2(sum[0], sum[1]), ptx::pack_bf16x2(sum[2], sum[3]), ptx::pack_bf16x2(sum[4], sum[5]),
                 ptx::pack_bf16x2(sum[6], sum[7]));
}

long long row_blocks(int tokens, int hidden) { return ((long long)tokens * (hidden / 8) + kRowThreads - 1) / kRowThreads; }

tkg_status check_rows(int tokens, int topk, int hidden, int capacity, const void* a, int lda, const int* rows,
                      const void* b, int ldb) {
  if (tokens < 0 || topk < 1 || hidden < 0 || capacity < 0 || lda < hidden || ldb < hidden) return TKG_ERR_INVALID_ARG;
  if (topk > kMaxChoices || (long long)tokens * topk > kMaxSize || capacity > kMaxSize || hidden > kMaxSize ||
      row_blocks(tokens, hidden) > kMaxSize)
    return TKG_ERR_UNSUPPORTED;
  if (hidden > 0 && (hidden % 8 != 0 || lda % 8 != 0 || ldb % 8 != 0 || !aligned_to(a, 16) || !aligned_to(b, 16) || !aligned_to(rows, 4)))
    return TKG_ERR_ALIGNMENT;
  return TKG_OK;
}

}  // namespace
}  // namespace tkg

using namespace tkg;

extern "C" {

tkg_status tkg_moe_dispatch(int tokens, int topk, int hidden, const void* X, int ldx, const int* rows, int capacity,
                            void* out, int ldo, cudaStream_t stream) {
  tkg_status st = check_rows(tokens, topk, hidden, capacity, X, ldx, rows, out, ldo);
  if (st != TKG_OK || tokens == 0 || hidden == 0 || capacity == 0) return st;
  if (!X || !rows || !out) return TKG_ERR_INVALID_ARG;
  const int vecs = hidden / 8;
  return launch_small(dispatch_kernel, dim3(unsigned(row_blocks(tokens, hidden))), dim3(kRowThreads), stream, 0u, tokens,
                      vecs, topk, capacity, static_cast<const uint16_t*>(X), size_t(ldx), rows,
                      static_cast<uint16_t*>(out), size_t(ldo));
}

tkg_status tkg_moe_combine(int tokens, int topk, int hidden, const void* O, int ldo, int capacity, const int* rows,
                           const float* weights, void* Y, int ldy, cudaStream_t stream) {
  tkg_status st = check_rows(tokens, topk, hidden, capacity, O, ldo, rows, Y, ldy);
  if (st != TKG_OK) return st;
  if (!aligned_to(weights, 4)) return TKG_ERR_ALIGNMENT;
  if (tokens == 0 || hidden == 0) return TKG_OK;
  if ((!O && capacity > 0) || !rows || !Y) return TKG_ERR_INVALID_ARG;
  const int vecs = hidden / 8;
  auto go = [&](auto kern) {
    return launch_small(kern, dim3(unsigned(row_blocks(tokens, hidden))), dim3(kRowThreads), stream, 0u, tokens, vecs, topk,
                        capacity, static_cast<const uint16_t*>(O), size_t(ldo), rows, weights, static_cast<uint16_t*>(Y),
                        size_t(ldy));
  };
  auto pick = [&](auto k) { return weights ? go(combine_kernel<decltype(k)::value, true>) : go(combine_kernel<decltype(k)::value, false>); };
  switch (topk) {
    case 1: return pick(std::integral_constant<int, 1>{});
    case 2: return pick(std::integral_constant<int, 2>{});
    case 3: return pick(std::integral_constant<int, 3>{});
    case 4: return pick(std::integral_constant<int, 4>{});
    case 5: return pick(std::integral_constant<int, 5>{});
    case 6: return pick(std::integral_constant<int, 6>{});
    case 7: return pick(std::integral_constant<int, 7>{});
    case 8: return pick(std::integral_constant<int, 8>{});
    default: return pick(std::integral_constant<int, 0>{});
  }
}

}  // extern "C"
