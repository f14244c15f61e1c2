// linear_ce_logits.cu -- the head's logits z = alpha X W^T with the cross-entropy epilogues (train_kernel.cuh).
#include "linear_ce.cuh"

namespace tkg {

template <int EPI>
static tkg_status launch_logits(const void* X, size_t x_bytes, const void* W, size_t w_bytes, TrainParams& p,
                                cudaStream_t stream) {
  CUtensorMap tmA, tmB, tmD;
  tkg_status st;
  p.n_tile = train_n_tile(p.n, kTileTokens);
  if ((st = map_k_major(&tmA, W, p.m, p.k, w_bytes, 128)) != TKG_OK) return st;
  if ((st = map_k_major(&tmB, X, p.n, p.k, x_bytes, p.n_tile / 2)) != TKG_OK) return st;
  tmD = tmA;
  if (EPI == EPI_DLOGITS &&
      (st = map_out(&tmD, p.d, p.m, p.n, 1, p.ldd * 2, size_t(p.m) * p.ldd * 2, false, true)) != TKG_OK)
    return st;
  p.splits = 1;
  p.split_stages = ceil_div(p.k, 64);
  const int sums = ceil_div(p.split_stages, kSumStages);
  p.sum_stages = ceil_div(p.split_stages, sums);
  // the narrow form has no registers for more sums than its two accumulators
  const int tiles = ceil_div(p.m, 256);
  if ((EPI == EPI_LOSS ? train_narrow(p.n, tiles) : train_narrow_gradient(p.n, p.k, tiles)) && sums <= 2)
    return launch_train<false, false, EPI, GRP_NONE, SHAPE_NARROW>(tmA, tmB, tmD, p, stream);
  if (sums > 1) return launch_train<false, false, EPI, GRP_NONE, SHAPE_SUMS>(tmA, tmB, tmD, p, stream);
  return launch_train<false, false, EPI, GRP_NONE>(tmA, tmB, tmD, p, stream);
}

tkg_status launch_ce_loss(const void* X, size_t x_bytes, const void* W, size_t w_bytes, TrainParams p,
                          cudaStream_t stream) {
  return launch_logits<EPI_LOSS>(X, x_bytes, W, w_bytes, p, stream);
}

tkg_status launch_ce_dlogits(const void* X, size_t x_bytes, const void* W, size_t w_bytes, TrainParams p,
                             cudaStream_t stream) {
  return launch_logits<EPI_DLOGITS>(X, x_bytes, W, w_bytes, p, stream);
}

}  // namespace tkg
