// linear_ce.cuh -- the head's products, instantiated in linear_ce_logits.cu and linear_ce_grad.cu.
#pragma once
#include "train_host.cuh"

namespace tkg {

// Logits of `n` vocabulary rows with the loss or the gradient epilogue; p.m, n, k, c2 and the
// epilogue's fields set.  Single CTAs when one 128-row tile holds all tokens.
tkg_status launch_ce_loss(const void* X, size_t x_bytes, const void* W, size_t w_bytes, TrainParams p,
                          cudaStream_t stream);
tkg_status launch_ce_dlogits(const void* X, size_t x_bytes, const void* W, size_t w_bytes, void* G, size_t g_bytes,
                             TrainParams p, cudaStream_t stream);
inline bool ce_single_cta(int tokens) {
  const int cg = option(TKG_OPT_CTA_GROUP);
  return cg == 1 || (cg == 0 && tokens <= 128);
}

}  // namespace tkg
