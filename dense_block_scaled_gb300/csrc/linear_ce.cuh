// linear_ce.cuh -- the head's products, instantiated in linear_ce_logits.cu, and the loss of a few tokens
// (linear_ce_few.cu).
#pragma once
#include "train_host.cuh"

namespace tkg {

// Logits of p.m vocabulary rows (at W) and p.n tokens with the loss or the gradient
// epilogue (g: [vocabulary][token], row pitch p.ldd); p.m, n, k, c2 and the epilogue's fields set.
tkg_status launch_ce_loss(const void* X, size_t x_bytes, const void* W, size_t w_bytes, TrainParams p,
                          cudaStream_t stream);
tkg_status launch_ce_dlogits(const void* X, size_t x_bytes, const void* W, size_t w_bytes, TrainParams p,
                             cudaStream_t stream);

// The loss of at most kFewTokens tokens on FP32 multiply-adds, when X fits shared memory in FP32 twice per SM: the
// blocks to launch (each leaves one part per token), or 0 when it does not apply.  ldx, ldw in elements.
constexpr int kFewTokens = 4, kFewElements = 16384, kFewMaxBlocks = 4 * kPairs;
int ce_few_blocks(int tokens, int vocab, int hidden);
tkg_status launch_ce_few(const void* X, size_t ldx, const void* W, size_t ldw, const TrainParams& p, int blocks,
                         cudaStream_t stream);

}  // namespace tkg
