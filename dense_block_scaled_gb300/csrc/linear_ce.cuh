// linear_ce.cuh -- the head's products, instantiated in linear_ce_logits.cu.
#pragma once
#include "train_host.cuh"

namespace tkg {

// Logits of p.m vocabulary rows (at W) and p.n tokens with the loss or the gradient
// epilogue (g: [vocabulary][token], row pitch p.ldd); p.m, n, k, c2 and the epilogue's fields set.
tkg_status launch_ce_loss(const void* X, size_t x_bytes, const void* W, size_t w_bytes, TrainParams p,
                          cudaStream_t stream);
tkg_status launch_ce_dlogits(const void* X, size_t x_bytes, const void* W, size_t w_bytes, TrainParams p,
                             cudaStream_t stream);

}  // namespace tkg
