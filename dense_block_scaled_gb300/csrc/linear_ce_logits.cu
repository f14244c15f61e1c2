// linear_ce_logits.cu -- the head's logits z = alpha X W^T with the cross-entropy epilogues (train_kernel.cuh).
#include "linear_ce.cuh"

namespace tkg {

template <int EPI, int CG>
static tkg_status launch_logits(const void* X, size_t x_bytes, const void* W, size_t w_bytes, void* G, size_t g_bytes,
                                TrainParams& p, cudaStream_t stream) {
  using C = TrainConfig<false, false, EPI, CG, GRP_NONE>;
  CUtensorMap tmA, tmB, tmD;
  tkg_status st;
  if ((st = map_k_major(&tmA, X, p.m, p.k, x_bytes, 128)) != TKG_OK) return st;
  if ((st = map_k_major(&tmB, W, p.n, p.k, w_bytes, C::kBRows)) != TKG_OK) return st;
  tmD = tmA;
  if (EPI == EPI_DLOGITS && (st = map_out(&tmD, G, p.m, p.n, 1, g_bytes, size_t(p.m) * g_bytes, false)) != TKG_OK)
    return st;
  p.splits = 1;
  p.split_stages = ceil_div(p.k, 64);
  return launch_train<false, false, EPI, CG, GRP_NONE>(tmA, tmB, tmD, p, stream);
}

tkg_status launch_ce_loss(const void* X, size_t x_bytes, const void* W, size_t w_bytes, TrainParams p,
                          cudaStream_t stream) {
  if (ce_single_cta(p.m)) return launch_logits<EPI_LOSS, 1>(X, x_bytes, W, w_bytes, nullptr, 0, p, stream);
  return launch_logits<EPI_LOSS, 2>(X, x_bytes, W, w_bytes, nullptr, 0, p, stream);
}

tkg_status launch_ce_dlogits(const void* X, size_t x_bytes, const void* W, size_t w_bytes, void* G, size_t g_bytes,
                             TrainParams p, cudaStream_t stream) {
  if (ce_single_cta(p.m)) return launch_logits<EPI_DLOGITS, 1>(X, x_bytes, W, w_bytes, G, g_bytes, p, stream);
  return launch_logits<EPI_DLOGITS, 2>(X, x_bytes, W, w_bytes, G, g_bytes, p, stream);
}

}  // namespace tkg
