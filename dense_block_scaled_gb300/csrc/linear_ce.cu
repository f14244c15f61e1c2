// linear_ce.cu -- softmax cross entropy of a linear head over a large vocabulary
// and its gradient, without the logits ever being kept.
//
//   z = alpha X W^T,  lse_t = log sum_v exp z_tv,  loss_t = lse_t - z_t,y(t)
//   g_tv = alpha dloss_t (exp(z_tv - lse_t) - [v = y(t)]),  dX = g W,  dW = g^T X
//
// Loss: one pass over W.  Each 128 logits of a row leave their maximum and sum
// (8 bytes), which a second kernel joins: (M, S) of parts (m_i, s_i) is M = max m_i,
// S = sum s_i 2^(m_i - M), in base 2, all in FP32.
//
// Gradient: the vocabulary in pieces.  Per piece the logits are computed again
// (2 T V H flops, against reading T V logits back), g goes to a BF16 workspace of
// one piece, and two products take it from there: dW's rows of the piece are
// final, dX grows by one FP32 addition per piece.  dX's product splits its long
// axis (the vocabulary) over CTAs when T x H has too few tiles; every part has
// its own FP32 buffer and the buffers are added in order.
#include <cmath>

#include "linear_ce.cuh"

namespace tkg {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// ---------------------------------------------------------------- joining the loss's parts
// 32 tokens per block; warp w reads parts w, w + 32, ... of its 32 tokens (256
// contiguous bytes a part), then the block's warps are joined in shared memory.
__global__ void __launch_bounds__(1024)
    ce_join_kernel(int tokens, int vocab, int parts, const float2* __restrict__ part, const float* __restrict__ zlabel,
                   const long long* __restrict__ labels, float* __restrict__ loss, float* __restrict__ lse) {
  __shared__ float s_top[32][33], s_sum[32][33];
  ptx::pdl_launch_dependents();
  ptx::pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int t = blockIdx.x * 32 + lane;
  float top = -INFINITY, sum = 0.f;
  if (t < tokens) {
#pragma unroll 4
    for (int i = warp; i < parts; i += warps) {
      const float2 x = __ldcg(part + size_t(i) * size_t(tokens) + t);
      const float m = fmaxf(top, x.x);
      const float base = fabsf(m) == INFINITY ? 0.f : m;   // no inf - inf
      sum = sum * ptx::ex2(top - base) + x.y * ptx::ex2(x.x - base);
      top = m;
    }
  }
  s_top[warp][lane] = top;
  s_sum[warp][lane] = sum;
  __syncthreads();
  if (warp == 0 && t < tokens) {
    for (int w = 1; w < warps; ++w) {
      const float m = fmaxf(top, s_top[w][lane]);
      const float base = fabsf(m) == INFINITY ? 0.f : m;
      sum = sum * ptx::ex2(top - base) + s_sum[w][lane] * ptx::ex2(s_top[w][lane] - base);
      top = m;
    }
    const float l = (top + log2f(sum)) * kLn2;
    const long long y = __ldcg(labels + t);
    lse[t] = l;
    loss[t] = (y >= 0 && y < vocab) ? l - __ldcg(zlabel + t) : 0.f;
  }
}

// ---------------------------------------------------------------- rows of X, ignored ones cleared
// dW = g^T X sums over rows whose g is 0 too; a row that is not a number (a padded
// position of an attention with nothing to attend to) would make 0 * NaN of it.
__global__ void __launch_bounds__(256)
    ce_rows_kernel(int tokens, int vocab, int hidden, const uint16_t* __restrict__ X, size_t ldx,
                   const long long* __restrict__ labels, uint16_t* __restrict__ out) {
  ptx::pdl_launch_dependents();
  ptx::pdl_wait();
  const int vec = hidden / 8;   // 16-byte pieces of a row
  const size_t total = size_t(tokens) * size_t(vec);
  for (size_t i = size_t(blockIdx.x) * blockDim.x + threadIdx.x; i < total; i += size_t(gridDim.x) * blockDim.x) {
    const size_t t = i / size_t(vec), c = i - t * size_t(vec);
    const long long y = __ldcg(labels + t);
    uint4 v = make_uint4(0, 0, 0, 0);
    if (y >= 0 && y < vocab) v = __ldcg(reinterpret_cast<const uint4*>(X + t * ldx) + c);
    reinterpret_cast<uint4*>(out)[i] = v;
  }
}

// ---------------------------------------------------------------- dX from its FP32 parts
__global__ void __launch_bounds__(256)
    ce_dx_kernel(int tokens, int hidden, int parts, const float* __restrict__ part, uint16_t* __restrict__ dX,
                 size_t lddx) {
  ptx::pdl_launch_dependents();
  ptx::pdl_wait();
  const int vec = hidden / 8;
  const size_t total = size_t(tokens) * size_t(vec);
  for (size_t i = size_t(blockIdx.x) * blockDim.x + threadIdx.x; i < total; i += size_t(gridDim.x) * blockDim.x) {
    const size_t t = i / size_t(vec), c = i - t * size_t(vec);
    float s[8] = {};
#pragma unroll 4
    for (int p = 0; p < parts; ++p) {
      const float4* src = reinterpret_cast<const float4*>(part + (size_t(p) * size_t(tokens) * size_t(hidden))) + 2 * i;
      const float4 a = __ldcg(src), b = __ldcg(src + 1);
      s[0] += a.x; s[1] += a.y; s[2] += a.z; s[3] += a.w;
      s[4] += b.x; s[5] += b.y; s[6] += b.z; s[7] += b.w;
    }
    *(reinterpret_cast<uint4*>(dX + t * lddx) + c) =
        make_uint4(ptx::pack_bf16x2(s[0], s[1]), ptx::pack_bf16x2(s[2], s[3]), ptx::pack_bf16x2(s[4], s[5]),
                   ptx::pack_bf16x2(s[6], s[7]));
  }
}

inline size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// ---------------------------------------------------------------- plans and workspaces
// The plans go by the GB300's 152 SMs, so that a workspace's size depends on the
// problem alone; on fewer SMs they are only less well balanced.
constexpr int kSms = 152;

struct GradPlan {
  int piece;          // vocabulary entries per piece
  int pieces;
  int parts;          // k parts of dX's product
  bool dx_f32;        // dX through FP32 parts
  size_t g_row;       // bytes of one row of g
  size_t rows_off, g_off, part_off, bytes;
};

// Vocabulary entries per piece: g (T x piece BF16) of up to 512 MB, a multiple of 256, at least 4096.
int default_piece(int tokens, int vocab) {
  long long piece = (512ll << 20) / (2ll * tokens) / 256 * 256;
  if (piece < 4096) piece = 4096;
  return piece < vocab ? int(piece) : vocab;
}

// Parts of dX's long axis: the number whose rounds of tiles take least, a part
// at least 8 stages (512 vocabulary entries) long.
int dx_parts(int tokens, int hidden, int k) {
  const int cg = tokens <= 128 ? 1 : 2;
  const int slots = kSms / cg;
  const int tiles = ceil_div(tokens, 128 * cg) * ceil_div(hidden, 256);
  const int stages = ceil_div(k, 64);
  int best = 1;
  double best_time = 1e300;
  for (int s = 1; s <= 32 && (s == 1 || stages / s >= 8); ++s) {
    const int per = ceil_div(stages, s);
    if (ceil_div(stages, per) != s) continue;
    const double time = double(ceil_div(tiles * s, slots)) * (per + 12);   // about 12 stages' time to start and drain
    if (time < 0.95 * best_time) {
      best = s;
      best_time = time;
    }
  }
  return best;
}

GradPlan grad_plan(int tokens, int vocab, int hidden, int piece) {
  GradPlan pl{};
  pl.piece = piece > 0 ? (piece < vocab ? piece : vocab) : default_piece(tokens, vocab);
  pl.pieces = ceil_div(vocab, pl.piece);
  pl.parts = dx_parts(tokens, hidden, pl.piece);
  pl.dx_f32 = pl.pieces > 1 || pl.parts > 1;
  pl.g_row = round_up(size_t(pl.piece) * 2, 128);
  pl.rows_off = 0;
  pl.g_off = round_up(size_t(tokens) * size_t(hidden) * 2, 256);
  pl.part_off = pl.g_off + round_up(size_t(tokens) * pl.g_row, 256);
  pl.bytes = pl.part_off + (pl.dx_f32 ? size_t(pl.parts) * size_t(tokens) * size_t(hidden) * 4 : 0);
  return pl;
}

tkg_status check_head(int tokens, int vocab, int hidden, const void* X, int ldx, const void* W, int ldw,
                      const long long* labels, bool* empty) {
  *empty = false;
  if (tokens < 0 || vocab < 0 || hidden < 0) return TKG_ERR_INVALID_ARG;
  if (vocab == 0 || hidden == 0) return TKG_ERR_UNSUPPORTED;   // a softmax over nothing; an empty product
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

tkg_status run_rows(int tokens, int vocab, int hidden, const void* X, int ldx, const long long* labels, void* out,
                    cudaStream_t stream) {
  const size_t pieces = size_t(tokens) * size_t(hidden / 8);
  const unsigned blocks = unsigned(pieces / 256 + 1 < size_t(kSms) * 8 ? pieces / 256 + 1 : size_t(kSms) * 8);
  return launch_small(ce_rows_kernel, dim3(blocks), dim3(256), stream, tokens, vocab, hidden,
                      static_cast<const uint16_t*>(X), size_t(ldx), labels, static_cast<uint16_t*>(out));
}

}  // namespace
}  // namespace tkg

using namespace tkg;

extern "C" {

size_t tkg_linear_ce_loss_workspace_bytes(int tokens, int vocab) {
  if (tokens < 0 || vocab < 0) return 0;
  return round_up(size_t(ceil_div(vocab, 256)) * 2 * size_t(tokens) * sizeof(float2), 256) + size_t(tokens) * 4;
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
  const int parts = ceil_div(vocab, 256) * 2;
  TrainParams p{};
  p.m = tokens;
  p.n = vocab;
  p.k = hidden;
  p.alpha = alpha;
  p.c2 = alpha * kLog2e;
  p.vocab = vocab;
  p.labels = labels;
  p.part = static_cast<float2*>(workspace);
  p.zlabel = reinterpret_cast<float*>(static_cast<char*>(workspace) +
                                      round_up(size_t(parts) * size_t(tokens) * sizeof(float2), 256));
  if ((st = launch_ce_loss(X, size_t(ldx) * 2, W, size_t(ldw) * 2, p, stream)) != TKG_OK) return st;
  const int warps = parts < 32 ? parts : 32;
  return launch_small(ce_join_kernel, dim3(unsigned(ceil_div(tokens, 32))), dim3(unsigned(32 * warps)), stream, tokens,
                      vocab, parts, p.part, p.zlabel, labels, loss, lse);
}

size_t tkg_linear_ce_grad_workspace_bytes(int tokens, int vocab, int hidden, int piece) {
  if (tokens < 0 || vocab < 0 || hidden < 0 || piece < 0) return 0;
  if (tokens == 0 || vocab == 0 || hidden == 0) return 0;
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
  void* rows = ws + pl.rows_off;
  void* G = ws + pl.g_off;
  float* part = reinterpret_cast<float*>(ws + pl.part_off);
  const bool single = ce_single_cta(tokens);
  CUtensorMap tmA, tmB, tmD;

  if (dW && (st = run_rows(tokens, vocab, hidden, X, ldx, labels, rows, stream)) != TKG_OK) return st;
  for (int i = 0; i < pl.pieces; ++i) {
    const int v0 = i * pl.piece, nv = vocab - v0 < pl.piece ? vocab - v0 : pl.piece;
    const char* Wp = static_cast<const char*>(W) + size_t(v0) * size_t(ldw) * 2;
    TrainParams p{};
    p.m = tokens;
    p.n = nv;
    p.k = hidden;
    p.alpha = alpha;
    p.c2 = alpha * kLog2e;
    p.vocab0 = v0;
    p.vocab = vocab;
    p.labels = labels;
    p.lse = lse;
    p.dloss = dloss;
    if ((st = launch_ce_dlogits(X, size_t(ldx) * 2, Wp, size_t(ldw) * 2, G, pl.g_row, p, stream)) != TKG_OK) return st;
    if (dX) {
      // (parts of) g W of this piece
      TrainParams q{};
      q.m = tokens;
      q.n = hidden;
      q.k = nv;
      q.alpha = 1.f;
      q.split_stages = ceil_div(ceil_div(nv, 64), pl.parts);
      q.splits = ceil_div(ceil_div(nv, 64), q.split_stages);
      q.accumulate = i > 0;
      if ((st = map_k_major(&tmA, G, tokens, nv, pl.g_row, 128)) != TKG_OK) return st;
      if ((st = map_mn_major(&tmB, Wp, hidden, nv, size_t(ldw) * 2)) != TKG_OK) return st;
      if (pl.dx_f32)
        st = map_out(&tmD, part, tokens, hidden, pl.parts, size_t(hidden) * 4, size_t(tokens) * size_t(hidden) * 4, true);
      else
        st = map_out(&tmD, dX, tokens, hidden, 1, size_t(lddx) * 2, size_t(tokens) * size_t(lddx) * 2, false);
      if (st != TKG_OK) return st;
      if (pl.dx_f32)
        st = single ? launch_train<false, true, EPI_F32, 1, GRP_NONE>(tmA, tmB, tmD, q, stream)
                    : launch_train<false, true, EPI_F32, 2, GRP_NONE>(tmA, tmB, tmD, q, stream);
      else
        st = single ? launch_train<false, true, EPI_BF16, 1, GRP_NONE>(tmA, tmB, tmD, q, stream)
                    : launch_train<false, true, EPI_BF16, 2, GRP_NONE>(tmA, tmB, tmD, q, stream);
      if (st != TKG_OK) return st;
    }
    if (dW) {
      // rows [v0, v0 + nv) of dW = g^T X
      TrainParams q{};
      q.m = nv;
      q.n = hidden;
      q.k = tokens;
      q.alpha = 1.f;
      q.splits = 1;
      q.split_stages = ceil_div(tokens, 64);
      q.accumulate = dw_type == TKG_GRAD_F32_ADD;
      if ((st = map_mn_major(&tmA, G, nv, tokens, pl.g_row)) != TKG_OK) return st;
      if ((st = map_mn_major(&tmB, rows, hidden, tokens, size_t(hidden) * 2)) != TKG_OK) return st;
      if ((st = map_out(&tmD, static_cast<char*>(dW) + size_t(v0) * size_t(lddw) * es, nv, hidden, 1, size_t(lddw) * es,
                        size_t(nv) * size_t(lddw) * es, es == 4)) != TKG_OK)
        return st;
      st = es == 2 ? launch_train<true, true, EPI_BF16, 2, GRP_NONE>(tmA, tmB, tmD, q, stream)
                   : launch_train<true, true, EPI_F32, 2, GRP_NONE>(tmA, tmB, tmD, q, stream);
      if (st != TKG_OK) return st;
    }
  }
  if (dX && pl.dx_f32) {
    const size_t pieces = size_t(tokens) * size_t(hidden / 8);
    const unsigned blocks = unsigned(pieces / 256 + 1 < size_t(kSms) * 8 ? pieces / 256 + 1 : size_t(kSms) * 8);
    return launch_small(ce_dx_kernel, dim3(blocks), dim3(256), stream, tokens, hidden, pl.parts, part,
                        static_cast<uint16_t*>(dX), size_t(lddx));
  }
  return TKG_OK;
}

}  // extern "C"
