// linear_ce.cu -- softmax cross entropy of a linear head over a large vocabulary
// and its gradient, without the logits ever being kept.
//
//   z = alpha X W^T,  lse_t = log sum_v exp z_tv,  loss_t = lse_t - z_t,y(t)
//   g_tv = exp(z_tv - lse_t) - [v = y(t)],  c_t = alpha dloss_t (0 for ignored t)
//   dX = diag(c) g W,  dW = g^T diag(c) X
//
// Loss: one pass over W (of at most 4 tokens perhaps without tensor cores, linear_ce_few.cu).
// Each 128 logits of a token leave their maximum and sum (8 bytes), which a second kernel joins: (M, S) of parts (m_i, s_i) is M = max m_i,
// S = sum s_i e^(m_i - M), all in FP32.  The maxima stay logits as they are and only differences go to base 2, so
// lse = M + log S has S >= 1 and is the label's own logit where that one dominates: a loss is never below 0 (with
// maxima kept in base 2 the losses of such tokens were off by up to 1e-7 of the logit, either way).
//
// Gradient: the vocabulary in pieces.  Per piece the logits are computed again
// (2 T V H flops, against reading T V logits back), g goes to a BF16 workspace of
// one piece, and two products take it from there: dW's rows of the piece are
// final, dX grows by one FP32 addition per piece.  dX's product splits its long
// axis (the vocabulary) over clusters when T x H has too few tiles; every part has
// its own FP32 buffer and the buffers are added in order.
//
// The tokens' weights c stay out of g: with a mean over T tokens every label's
// term would be -c (1 - p), all rounded the same way (up to 2^-8 of the whole
// gradient when p is small).  dX's rows are multiplied by c in FP32; for dW the
// rows of X are multiplied by c / max |c| and rounded (exactly X's own rows when
// the weights are equal, as for a mean), and the sums by max |c| in FP32.
#include <cmath>

#include "linear_ce.cuh"

namespace tkg {
namespace {

// ---------------------------------------------------------------- joining the loss's parts
// 8 tokens per block (64 contiguous bytes of a part) and 128 threads per token,
// which read the parts in batches of 4 with the loads in flight together.
constexpr int kJoinTokens = 8;
__global__ void __launch_bounds__(1024)
    ce_join_kernel(int tokens, int vocab, int parts, const float2* __restrict__ part, const float* __restrict__ zlabel,
                   const long long* __restrict__ labels, float* __restrict__ loss, float* __restrict__ lse) {
  __shared__ float2 s_part[32][kJoinTokens];
  ptx::pdl_launch_dependents();
  ptx::pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = blockIdx.x * kJoinTokens + (lane & 7);
  float top = -INFINITY, sum = 0.f;
  if (t < tokens) {
#pragma unroll 1
    for (int i = threadIdx.x >> 3; i < parts; i += 512) {
      float2 x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        x[j] = i + 128 * j < parts ? __ldcg(part + size_t(i + 128 * j) * size_t(tokens) + t)
                                   : make_float2(-INFINITY, 0.f);
      const float up = fmaxf(fmaxf(x[0].x, x[1].x), fmaxf(x[2].x, x[3].x));
      const float base = fabsf(up) == INFINITY ? 0.f : up;   // no inf - inf
      float s = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) s += x[j].y * ptx::ex2((x[j].x - base) * kLog2e);
      ce_join(top, sum, up, s);
    }
  }
#pragma unroll
  for (int o = 8; o < 32; o <<= 1) {
    const float m = __shfl_xor_sync(0xffffffffu, top, o), s = __shfl_xor_sync(0xffffffffu, sum, o);
    ce_join(top, sum, m, s);
  }
  if (lane < kJoinTokens) s_part[warp][lane] = make_float2(top, sum);
  __syncthreads();
  if (warp == 0) {
    // 4 lanes per token, 8 warps' results each
    top = -INFINITY;
    sum = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      const float2 x = s_part[(lane >> 3) * 8 + w][lane & 7];
      ce_join(top, sum, x.x, x.y);
    }
#pragma unroll
    for (int o = 8; o < 32; o <<= 1) {
      const float m = __shfl_xor_sync(0xffffffffu, top, o), s = __shfl_xor_sync(0xffffffffu, sum, o);
      ce_join(top, sum, m, s);
    }
    if (lane < kJoinTokens && t < tokens) {
      const float l = top + logf(sum);
      const long long y = __ldcg(labels + t);
      lse[t] = l;
      loss[t] = (y >= 0 && y < vocab) ? l - __ldcg(zlabel + t) : 0.f;
    }
  }
}

// ---------------------------------------------------------------- rows of X with the tokens' weights
// ce_weighted_row for every token, and s.  Every block finds s again from the T
// weights (T x 12 bytes from L2 for each of at most two blocks per SM, against one
// more launch), then takes a row per warp.  For heads with too few tiles to deal
// the rows over, or too many weights (see rows_on_the_side).
__global__ void __launch_bounds__(256)
    ce_rows_kernel(int tokens, int vocab, int hidden, const uint16_t* __restrict__ X, size_t ldx,
                   const long long* __restrict__ labels, const float* __restrict__ dloss, float alpha,
                   uint16_t* __restrict__ out, float* __restrict__ scale) {
  __shared__ float s_max[8];
  ptx::pdl_launch_dependents();
  ptx::pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  float top = 0.f;
#pragma unroll 8
  for (int t = tid; t < tokens; t += 256) top = fmaxf(top, fabsf(ce_weight(t, vocab, labels, dloss, alpha)));
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (lane == 0) s_max[warp] = top;
  __syncthreads();
  top = s_max[lane & 7];
#pragma unroll
  for (int o = 4; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  const float s = ce_scale(top);
  if (blockIdx.x == 0 && tid == 0) *scale = s;
  for (int t = blockIdx.x * 8 + warp; t < tokens; t += gridDim.x * 8)
    ce_weighted_row(t, lane, vocab, hidden, X, ldx, labels, dloss, alpha, s, out);
}

// ---------------------------------------------------------------- dX from its FP32 parts
// Parts are [hidden][token] (pitch a multiple of 64); dX is [token][hidden].  A
// block adds the parts of 64 tokens x 16 hidden, in order and eight parts' loads in
// flight together, turns them in shared memory and multiplies by the tokens' weights.
// With SPLIT = 2 (few blocks) each half of its threads adds half of the parts.  Rows past
// the 65535 blocks of the grid's second dimension are in its third.
template <int SPLIT>
__global__ void __launch_bounds__(256 * SPLIT)
    ce_dx_kernel(int tokens, int vocab, int hidden, int parts, const float* __restrict__ part, size_t pitch,
                 const long long* __restrict__ labels, const float* __restrict__ dloss, float alpha,
                 uint16_t* __restrict__ dX, size_t lddx) {
  __shared__ float s_t[SPLIT][16][65];
  ptx::pdl_launch_dependents();
  ptx::pdl_wait();
  const int t0 = blockIdx.x * 64, h0 = (blockIdx.z * gridDim.y + blockIdx.y) * 16, tid = threadIdx.x;
  const int tq = (tid & 15) * 4, hr = (tid >> 4) & 15, half = tid >> 8;   // four tokens of one row
  const int share = SPLIT == 2 ? (parts + 1) / 2 : parts, first = half * share, end = min(parts, first + share);
  const float* src = part + size_t(h0 + hr) * pitch + t0 + tq;
  const size_t part_len = size_t(hidden) * pitch;
  const bool row = h0 + hr < hidden;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (int p0 = first; p0 < end; p0 += 8) {
    float4 x[8];
#pragma unroll
    for (int p = 0; p < 8; ++p)
      x[p] = p0 + p < end && row ? __ldcg(reinterpret_cast<const float4*>(src + size_t(p0 + p) * part_len))
                                 : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      s.x += x[p].x;
      s.y += x[p].y;
      s.z += x[p].z;
      s.w += x[p].w;
    }
  }
  s_t[half][hr][tq] = s.x;
  s_t[half][hr][tq + 1] = s.y;
  s_t[half][hr][tq + 2] = s.z;
  s_t[half][hr][tq + 3] = s.w;
  __syncthreads();
  // 2 threads per token, 8 hidden (16 bytes) each
  const int c = tid >> 1, t = t0 + c, hh = (tid & 1) * 8;
  if (tid < 128 && t < tokens && h0 + hh < hidden) {
    const long long y = __ldcg(labels + t);
    const float w = alpha * __ldcg(dloss + t);
    auto sum = [&](int h) { return SPLIT == 2 ? s_t[0][h][c] + s_t[SPLIT - 1][h][c] : s_t[0][h][c]; };
    uint32_t o[4] = {0, 0, 0, 0};
    if (y >= 0 && y < vocab) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        o[i] = ptx::pack_bf16x2(sum(hh + 2 * i) * w, sum(hh + 2 * i + 1) * w);
    }
    *reinterpret_cast<uint4*>(dX + size_t(t) * lddx + h0 + hh) = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

inline size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// ---------------------------------------------------------------- plans and workspaces
// The plans go by the GB300's 76 pairs of SMs, so that a workspace's size depends
// on the problem alone; on fewer SMs they are only less well balanced.

struct GradPlan {
  int piece;          // vocabulary entries per piece
  int pieces;
  int parts;          // k parts of dX's product
  bool dx_dual;       // on 256 x 512 tiles
  size_t tokens_up;   // row pitch of g and of dX's parts, in elements
  size_t g_off, part_off, scale_off, bytes;   // the weighted rows of X come first
};

// Vocabulary entries per piece: g (piece x T BF16) of up to 512 MB, a multiple of 256, at least 4096.
int default_piece(int tokens, int vocab) {
  long long piece = (512ll << 20) / (2ll * tokens) / 256 * 256;
  if (piece < 4096) piece = 4096;
  return piece < vocab ? int(piece) : vocab;
}

// Parts of dX's long axis and its tiles' shape: what takes least time, a part at
// least 8 stages (512 vocabulary entries) long, and 32 at most.  dX with at least 4, 8 and 16 stages: 1 token x 1500 x
// 256 10.5, 11.0 and 14.3 us, 1 x 6000 x 1024 18.2, 16.4 and 17.2; with at most 32 and 64 parts: 1 x 32768 x 256 18.5
// and 20.9, 64 x 131072 x 256 42.5 and 38.5.  More parts, or the wide tiles, have to gain 3%, as the time leaves out
// adding the parts: without that 64 x 131072 x 2048 takes 195 us in place of 169, 777 x 131072 x 1024 340 of 295.
void plan_dx(int tokens, int hidden, int k, int* parts, bool* dual) {
  const int stages = ceil_div(k, 64);
  const int forced = option(TKG_OPT_BF16_TILE_N);
  double best = 1e300;
  for (int d = 0; d < 2; ++d) {
    if ((forced == 256 && d) || (forced == 512 && !d)) continue;
    const int tiles = ceil_div(hidden, 256) * ceil_div(tokens, d ? 512 : 256);
    for (int s = 1; s <= 32 && (s == 1 || stages / s >= 8); ++s) {
      const int per = ceil_div(stages, s);
      if (ceil_div(stages, per) != s) continue;
      const double time = train_rounds(double(tiles) * s) * train_tile_time(per, d != 0);
      if (time < 0.97 * best) {
        best = time;
        *parts = s;
        *dual = d != 0;
      }
    }
  }
}

GradPlan grad_plan(int tokens, int vocab, int hidden, int piece) {
  GradPlan pl{};
  pl.piece = piece > 0 ? (piece < vocab ? piece : vocab) : default_piece(tokens, vocab);
  pl.pieces = ceil_div(vocab, pl.piece);
  plan_dx(tokens, hidden, pl.piece, &pl.parts, &pl.dx_dual);
  pl.tokens_up = round_up(size_t(tokens), 64);
  pl.g_off = round_up(size_t(tokens) * size_t(hidden) * 2, 256);
  pl.part_off = pl.g_off + round_up(size_t(pl.piece) * pl.tokens_up * 2, 256);
  pl.scale_off = pl.part_off + size_t(pl.parts) * size_t(hidden) * pl.tokens_up * 4;
  pl.bytes = pl.scale_off + 16;
  return pl;
}

// Whether a spare warp of the logits' blocks writes the weighted rows of X, and not a kernel before them.  Its rows and
// the search for the largest of the T weights, which every such warp makes, have to stay behind the tiles' products:
// dW of 128 tokens x 16384 x 1024 takes 22.6 us (26.9 with the kernel), 2048 x 32768 x 256 78.8 (80.9), 6000 x 32768 x
// 2048 994 (1008); but with many rows to a tile 8192 x 8000 x 256 125.8 (103.5), and with many weights and short products
// 4096 x 32768 x 256 152.7 (148.5), 16384 x 65536 x 256 1143 (1117).
bool rows_on_the_side(int tokens, int piece, int hidden) {
  const double tiles = double(ceil_div(piece, 256)) * ceil_div(tokens, kTrainBN);
  return tokens / tiles <= 4.0 && tokens <= (hidden >= 2048 ? 16384 : 2048);
}

// One (maximum, sum) per token and 128 vocabulary rows, or per block of the kernel for few tokens.
size_t loss_part_bytes(int tokens, int vocab) {
  int parts = ceil_div(vocab, 128);
  if (tokens <= kFewTokens && parts < kFewMaxBlocks) parts = kFewMaxBlocks;
  return round_up(size_t(parts) * size_t(tokens) * sizeof(float2), 256);
}

tkg_status check_head(int tokens, int vocab, int hidden, const void* X, int ldx, const void* W, int ldw,
                      const long long* labels, bool* empty) {
  *empty = false;
  if (tokens < 0 || vocab < 0 || hidden < 0) return TKG_ERR_INVALID_ARG;
  if (vocab == 0 || hidden == 0) return TKG_ERR_UNSUPPORTED;   // a softmax over nothing; an empty product
  if (tokens > kMaxSize || vocab > kMaxSize || hidden > kMaxSize) return TKG_ERR_UNSUPPORTED;
  if (hidden % 8 != 0) return TKG_ERR_ALIGNMENT;
  if (tokens == 0) {
    *empty = true;
    return TKG_OK;
  }
  if (!X || !W || !labels || ldx < hidden || ldw < hidden) return TKG_ERR_INVALID_ARG;
  if (!aligned_to(X, 16) || !aligned_to(W, 16) || ldx % 8 != 0 || ldw % 8 != 0 || !aligned_to(labels, 8))
    return TKG_ERR_ALIGNMENT;
  return TKG_OK;
}

}  // namespace
}  // namespace tkg

using namespace tkg;

extern "C" {

size_t tkg_linear_ce_loss_workspace_bytes(int tokens, int vocab) {
  if (tokens < 0 || vocab < 0 || tokens > kMaxSize || vocab > kMaxSize) return 0;
  return loss_part_bytes(tokens, vocab) + size_t(tokens) * 4;
}

tkg_status tkg_linear_ce_loss(int tokens, int vocab, int hidden, const void* X, int ldx, const void* W, int ldw,
                              const long long* labels, float alpha, float* loss, float* lse, void* workspace,
                              size_t workspace_bytes, cudaStream_t stream) {
  bool empty;
  tkg_status st = check_head(tokens, vocab, hidden, X, ldx, W, ldw, labels, &empty);
  if (st != TKG_OK || empty) return st;
  if (!loss || !lse || !workspace || workspace_bytes < tkg_linear_ce_loss_workspace_bytes(tokens, vocab))
    return TKG_ERR_INVALID_ARG;
  if (!aligned_to(loss, 4) || !aligned_to(lse, 4) || !aligned_to(workspace, 16)) return TKG_ERR_ALIGNMENT;
  const int few = option(TKG_OPT_CTA_GROUP) ? 0 : ce_few_blocks(tokens, vocab, hidden);
  const int parts = few ? few : ceil_div(vocab, 128);
  TrainParams p{};
  p.m = vocab;
  p.n = tokens;
  p.k = hidden;
  p.alpha = alpha;
  p.c2 = alpha * kLog2e;
  p.vocab = vocab;
  p.labels = labels;
  p.part = static_cast<float2*>(workspace);
  p.zlabel = reinterpret_cast<float*>(static_cast<char*>(workspace) + loss_part_bytes(tokens, vocab));
  st = few ? launch_ce_few(X, size_t(ldx), W, size_t(ldw), p, few, stream)
           : launch_ce_loss(X, size_t(ldx) * 2, W, size_t(ldw) * 2, p, stream);
  if (st != TKG_OK) return st;
  return launch_small(ce_join_kernel, dim3(unsigned(ceil_div(tokens, kJoinTokens))), dim3(1024), stream, 0u, tokens, vocab,
                      parts, p.part, p.zlabel, labels, loss, lse);
}

size_t tkg_linear_ce_grad_workspace_bytes(int tokens, int vocab, int hidden, int piece) {
  if (tokens < 0 || vocab < 0 || hidden < 0 || piece < 0) return 0;
  if (tokens == 0 || vocab == 0 || hidden == 0) return 0;
  if (tokens > kMaxSize || vocab > kMaxSize || hidden > kMaxSize) return 0;
  return grad_plan(tokens, vocab, hidden, piece).bytes;
}

tkg_status tkg_linear_ce_grad(int tokens, int vocab, int hidden, const void* X, int ldx, const void* W, int ldw,
                              const long long* labels, float alpha, const float* lse, const float* dloss, void* dX,
                              int lddx, void* dW, int lddw, tkg_grad_type dw_type, int piece, void* workspace,
                              size_t workspace_bytes, cudaStream_t stream) {
  bool empty;
  tkg_status st = check_head(tokens, vocab, hidden, X, ldx, W, ldw, labels, &empty);
  if (st != TKG_OK) return st;
  if (piece < 0 || (dw_type != TKG_GRAD_BF16 && dw_type != TKG_GRAD_F32 && dw_type != TKG_GRAD_F32_ADD))
    return TKG_ERR_INVALID_ARG;
  const size_t es = dw_type == TKG_GRAD_BF16 ? 2 : 4;
  if (dW) {
    if (lddw < hidden) return TKG_ERR_INVALID_ARG;
    if (!aligned_to(dW, 16) || size_t(lddw) * es % 16 != 0) return TKG_ERR_ALIGNMENT;
  }
  if (empty) {   // no tokens: dW is an empty sum
    if (!dW || dw_type == TKG_GRAD_F32_ADD) return TKG_OK;
    return cudaMemset2DAsync(dW, size_t(lddw) * es, 0, size_t(hidden) * es, size_t(vocab), stream) == cudaSuccess
               ? TKG_OK
               : TKG_ERR_CUDA;
  }
  if (dX) {
    if (lddx < hidden) return TKG_ERR_INVALID_ARG;
    if (!aligned_to(dX, 16) || lddx % 8 != 0) return TKG_ERR_ALIGNMENT;
  }
  if (!dX && !dW) return TKG_OK;
  const GradPlan pl = grad_plan(tokens, vocab, hidden, piece);
  if (!lse || !dloss || !workspace || workspace_bytes < pl.bytes) return TKG_ERR_INVALID_ARG;
  if (!aligned_to(lse, 4) || !aligned_to(dloss, 4) || !aligned_to(workspace, 16)) return TKG_ERR_ALIGNMENT;
  char* ws = static_cast<char*>(workspace);
  uint16_t* rows = reinterpret_cast<uint16_t*>(ws);
  void* G = ws + pl.g_off;
  float* part = reinterpret_cast<float*>(ws + pl.part_off);
  float* scale = reinterpret_cast<float*>(ws + pl.scale_off);
  CUtensorMap tmA, tmB, tmD;

  const bool on_the_side = dW && rows_on_the_side(tokens, pl.piece, hidden);
  if (dW && !on_the_side) {
    const int blocks = ceil_div(tokens, 8) < 4 * kPairs ? ceil_div(tokens, 8) : 4 * kPairs;
    if ((st = launch_small(ce_rows_kernel, dim3(unsigned(blocks)), dim3(256), stream, 0u, tokens, vocab, hidden,
                           static_cast<const uint16_t*>(X), size_t(ldx), labels, dloss, alpha, rows, scale)) != TKG_OK)
      return st;
  }
  for (int i = 0; i < pl.pieces; ++i) {
    const int v0 = i * pl.piece, nv = vocab - v0 < pl.piece ? vocab - v0 : pl.piece;
    const char* Wp = static_cast<const char*>(W) + size_t(v0) * size_t(ldw) * 2;
    TrainParams p{};
    p.m = nv;
    p.n = tokens;
    p.k = hidden;
    p.alpha = alpha;
    p.c2 = alpha * kLog2e;
    p.vocab0 = v0;
    p.vocab = vocab;
    p.labels = labels;
    p.lse = lse;
    p.d = G;
    p.ldd = pl.tokens_up;
    if (on_the_side && i == 0) {
      p.x = static_cast<const uint16_t*>(X);
      p.ldx = size_t(ldx);
      p.dloss = dloss;
      p.rows = rows;
      p.rows_scale = scale;
    }
    if ((st = launch_ce_dlogits(X, size_t(ldx) * 2, Wp, size_t(ldw) * 2, p, stream)) != TKG_OK) return st;
    if (dX) {
      // (parts of) W^T g of this piece: hidden x tokens
      TrainParams q{};
      q.m = hidden;
      q.n = tokens;
      q.k = nv;
      q.n_tile = train_n_tile(tokens, kTileF32);
      q.alpha = 1.f;
      q.split_stages = ceil_div(ceil_div(nv, 64), pl.parts);
      q.splits = ceil_div(ceil_div(nv, 64), q.split_stages);
      q.accumulate = i > 0;
      if ((st = map_mn_major(&tmA, Wp, hidden, nv, size_t(ldw) * 2)) != TKG_OK) return st;
      if ((st = map_mn_major(&tmB, G, tokens, nv, pl.tokens_up * 2)) != TKG_OK) return st;
      if ((st = map_out(&tmD, part, hidden, tokens, pl.parts, pl.tokens_up * 4, size_t(hidden) * pl.tokens_up * 4,
                        true)) != TKG_OK)
        return st;
      ExtraMaps<EPI_F32, GRP_NONE> extra{};
      if ((st = map_prefetch(&extra.d, part, hidden, tokens, pl.parts, pl.tokens_up * 4,
                             size_t(hidden) * pl.tokens_up * 4)) != TKG_OK)
        return st;
      st = pl.dx_dual ? launch_train<true, true, EPI_F32, GRP_NONE, SHAPE_DUAL>(tmA, tmB, tmD, q, stream, extra)
                      : launch_train<true, true, EPI_F32, GRP_NONE>(tmA, tmB, tmD, q, stream, extra);
      if (st != TKG_OK) return st;
    }
    if (dW) {
      // rows [v0, v0 + nv) of dW = g (c / s X)
      TrainParams q{};
      q.m = nv;
      q.n = hidden;
      q.k = tokens;
      q.n_tile = train_n_tile(hidden, es == 2 ? kTileBF16 : kTileF32);
      q.alpha = 1.f;
      q.scale = scale;
      q.splits = 1;
      q.split_stages = ceil_div(tokens, 64);
      q.accumulate = dw_type == TKG_GRAD_F32_ADD;
      if ((st = map_k_major(&tmA, G, nv, tokens, pl.tokens_up * 2, 128)) != TKG_OK) return st;
      if ((st = map_mn_major(&tmB, rows, hidden, tokens, size_t(hidden) * 2)) != TKG_OK) return st;
      if ((st = map_out(&tmD, static_cast<char*>(dW) + size_t(v0) * size_t(lddw) * es, nv, hidden, 1, size_t(lddw) * es,
                        size_t(nv) * size_t(lddw) * es, es == 4)) != TKG_OK)
        return st;
      if (es == 2) {
        st = train_dual(nv, hidden, 1, ceil_div(tokens, 64))
                 ? launch_train<false, true, EPI_BF16, GRP_NONE, SHAPE_DUAL>(tmA, tmB, tmD, q, stream)
                 : launch_train<false, true, EPI_BF16, GRP_NONE>(tmA, tmB, tmD, q, stream);
      } else {
        ExtraMaps<EPI_F32, GRP_NONE> extra{};
        if ((st = map_prefetch(&extra.d, static_cast<float*>(dW) + size_t(v0) * size_t(lddw), nv, hidden, 1,
                               size_t(lddw) * 4, size_t(nv) * size_t(lddw) * 4)) != TKG_OK)
          return st;
        const int sums = ceil_div(q.split_stages, kSumStages);
        q.sum_stages = ceil_div(q.split_stages, sums);
        st = sums > 1 ? launch_train<false, true, EPI_F32, GRP_NONE, SHAPE_SUMS>(tmA, tmB, tmD, q, stream, extra)
                      : launch_train<false, true, EPI_F32, GRP_NONE>(tmA, tmB, tmD, q, stream, extra);
      }
      if (st != TKG_OK) return st;
    }
  }
  if (!dX) return TKG_OK;
  // Half of the parts per thread where there are few blocks: 40 tokens x 21648 x 1024 (64 blocks) 43.0 us in place of
  // 46.1, 200 x 5000 x 768 (192) 27.4 of 28.8, but 128 x 32768 x 2048 (256) 95.0 of 92.3 (from a graph); dX alone of 777
  // x 32768 x 256 (208) 45.8 of 47.5, of 16 x 32768 x 4096 (256) 104 of 96
  const int across = ceil_div(tokens, 64), down = ceil_div(hidden, 16), deep = ceil_div(down, 65535);
  const bool few = (long long)across * down <= 3 * kPairs;
  const dim3 grid(unsigned(across), unsigned(ceil_div(down, deep)), unsigned(deep));
  return launch_small(few ? ce_dx_kernel<2> : ce_dx_kernel<1>, grid, dim3(few ? 512 : 256), stream, 0u, tokens, vocab,
                      hidden, pl.parts, part, pl.tokens_up, labels, dloss, alpha, static_cast<uint16_t*>(dX),
                      size_t(lddx));
}

}  // extern "C"
