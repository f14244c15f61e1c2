// moe_rows.cu -- tokens' rows into expert order and back, by the rows that tkg_moe_route wrote.
//
//   dispatch  out[rows(t, j)] = X[t]
//   combine   Y[t] = sum_j w(t, j) O[rows(t, j)]     (FP32 sums in the order of j, rounded once)
//
// Each is the other's gradient (combine with weights 1).  A place outside [0, capacity), such as the -1 of a token that is
// not routed, is left out: nothing is written for it, nothing is read.
//
// Both are bound by HBM.  Blocks go by token, so that X's row is read once and sent to all its places, and all of a
// token's rows of O are on their way together; a thread takes 16 bytes of a row.
#include "train_host.cuh"

namespace tkg {
namespace {

constexpr int kRowThreads = 128;
constexpr int kMaxChoices = 32;

__global__ void __launch_bounds__(kRowThreads) dispatch_kernel(int vecs, int topk, int capacity,
                                                               const uint16_t* __restrict__ X, size_t ldx,
                                                               const int* __restrict__ rows, uint16_t* __restrict__ out,
                                                               size_t ldo) {
  ptx::pdl_launch_dependents();
  const size_t t = blockIdx.x;
  const int v = blockIdx.y * kRowThreads + threadIdx.x;
  if (v >= vecs) return;
  ptx::pdl_wait();
  const uint4 x = __ldcg(reinterpret_cast<const uint4*>(X + t * ldx) + v);
#pragma unroll 4
  for (int j = 0; j < topk; ++j) {
    const int r = __ldcg(rows + t * topk + j);
    if (r >= 0 && r < capacity) reinterpret_cast<uint4*>(out + size_t(r) * ldo)[v] = x;
  }
}

__global__ void __launch_bounds__(kRowThreads) combine_kernel(int vecs, int topk, int capacity,
                                                              const uint16_t* __restrict__ O, size_t ldo,
                                                              const int* __restrict__ rows,
                                                              const float* __restrict__ weights,
                                                              uint16_t* __restrict__ Y, size_t ldy) {
  ptx::pdl_launch_dependents();
  const size_t t = blockIdx.x;
  const int v = blockIdx.y * kRowThreads + threadIdx.x;
  if (v >= vecs) return;
  ptx::pdl_wait();
  float sum[8] = {};
#pragma unroll 1
  for (int j0 = 0; j0 < topk; j0 += 8) {
    uint4 x[8];
    float w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      x[j] = make_uint4(0, 0, 0, 0);
      w[j] = 0.f;
      if (j0 + j < topk) {
        const int r = __ldcg(rows + t * topk + j0 + j);
        if (r >= 0 && r < capacity) {
          x[j] = __ldcg(reinterpret_cast<const uint4*>(O + size_t(r) * ldo) + v);
          w[j] = weights ? __ldcg(weights + t * topk + j0 + j) : 1.f;
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t u[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        sum[2 * i] = fmaf(w[j], __uint_as_float(u[i] << 16), sum[2 * i]);
        sum[2 * i + 1] = fmaf(w[j], __uint_as_float(u[i] & 0xffff0000u), sum[2 * i + 1]);
      }
    }
  }
  reinterpret_cast<uint4*>(Y + t * ldy)[v] =
      make_uint4(ptx::pack_bf16x2(sum[0], sum[1]), ptx::pack_bf16x2(sum[2], sum[3]), ptx::pack_bf16x2(sum[4], sum[5]),
                 ptx::pack_bf16x2(sum[6], sum[7]));
}

tkg_status check_rows(int tokens, int topk, int hidden, int capacity, const void* a, int lda, const int* rows,
                      const void* b, int ldb) {
  if (tokens < 0 || topk < 1 || hidden < 0 || capacity < 0 || lda < hidden || ldb < hidden) return TKG_ERR_INVALID_ARG;
  if (topk > kMaxChoices || (long long)tokens * topk > kMaxSize || capacity > kMaxSize || hidden > kMaxSize ||
      hidden > 65535ll * 8 * kRowThreads)
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
  return launch_small(dispatch_kernel, dim3(unsigned(tokens), unsigned(ceil_div(vecs, kRowThreads))), dim3(kRowThreads),
                      stream, 0u, vecs, topk, capacity, static_cast<const uint16_t*>(X), size_t(ldx), rows,
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
  return launch_small(combine_kernel, dim3(unsigned(tokens), unsigned(ceil_div(vecs, kRowThreads))), dim3(kRowThreads),
                      stream, 0u, vecs, topk, capacity, static_cast<const uint16_t*>(O), size_t(ldo), rows, weights,
                      static_cast<uint16_t*>(Y), size_t(ldy));
}

}  // extern "C"
