// linear_ce_few.cu -- the loss of a few tokens (1 to 4): the head's matrix is
// read once and every other cost has to hide behind that read.
//
// A tensor-core tile has 256 vocabulary rows to a pair of SMs, so a vocabulary of
// a few thousand leaves most SMs idle.  Here every warp takes the same number of
// rows, and the products are FP32 multiply-adds: per W element one conversion and
// one FMA per token.  A warp works on four rows at a time: each X value (FP32 in
// shared memory) serves four rows, and up to four pieces of 256 columns of all
// four are on their way (16 warps per SM with 8 KB each; 45 KB per SM cover HBM's
// latency at full rate, half of that measured 31 us where this takes 26).  The
// 4 x T sums are joined over the lanes by exchanging halves (16 shuffles for the 16
// sums of four tokens, against 80 in butterflies: 4000 x 2112 9.8 us against 10.9),
// each pair (row, token) then belongs to one lane, which keeps its running maximum and sum; a block leaves one
// (maximum, sum) per token.
//
// Bound by HBM: 1 token x 32768 x 2048 takes 25.9 us (134 MB, 19.8 us at the
// copy rate; 26.8 on tensor-core tiles), x 131072 x 4096 156 us (6.9 TB/s), x 4000
// x 2048 9.2 us (13.9 on tiles).
#include "linear_ce.cuh"

namespace tkg {
namespace {

constexpr int kFewThreads = 256;
constexpr int kFewRows = 4;

template <int TT, int DEPTH>
__global__ void __launch_bounds__(kFewThreads, 2)
    ce_few_kernel(int tokens, int vocab, int hidden, const uint16_t* __restrict__ X, size_t ldx,
                  const uint16_t* __restrict__ W, size_t ldw, const long long* __restrict__ labels, float alpha,
                  float2* __restrict__ part, float* __restrict__ zlabel) {
  // 256 columns at a time: [columns / 256][token][half of a lane's 8 columns][lane][4], so that a quarter of a
  // warp reads 128 contiguous bytes
  extern __shared__ float s_x[];
  __shared__ float2 s_part[kFewThreads / 32][TT];
  ptx::pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int blocks = (hidden + 255) / 256;
  const long long warps = (long long)gridDim.x * (kFewThreads / 32);
  const long long id = (long long)blockIdx.x * (kFewThreads / 32) + warp;
  const int first = int((long long)vocab * id / warps), end = int((long long)vocab * (id + 1) / warps);
  // this warp's first pieces of W on their way to L2 while the previous kernel may still run (nothing is read back)
#pragma unroll
  for (int d = 0; d < DEPTH; ++d)
#pragma unroll
    for (int r = 0; r < kFewRows; ++r)
      if (first + r < end && d * 256 + lane * 8 < hidden && (lane & 3) == 0)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(W + size_t(first + r) * ldw + d * 256 + lane * 8));
  ptx::pdl_wait();
  for (int i = threadIdx.x; i < blocks * 32 * TT; i += kFewThreads) {
    const int q = i / (32 * TT), t = (i / 32) % TT, l = i & 31, col = q * 256 + l * 8;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (t < tokens && col < hidden) v = __ldcg(reinterpret_cast<const uint4*>(X + size_t(t) * ldx + col));
    float4* lo = reinterpret_cast<float4*>(s_x + size_t((q * TT + t) * 2) * 128 + l * 4);
    lo[0] = make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u), __uint_as_float(v.y << 16),
                        __uint_as_float(v.y & 0xffff0000u));
    lo[32] = make_float4(__uint_as_float(v.z << 16), __uint_as_float(v.z & 0xffff0000u), __uint_as_float(v.w << 16),
                         __uint_as_float(v.w & 0xffff0000u));
  }
  // lane (r TT + t) (32 / kSums) keeps the running maximum and sum of rows r (mod 4) and token t
  constexpr int kSums = kFewRows * TT, kApart = 32 / kSums;
  const int my_t = lane / kApart % TT, my_r = lane / kApart / TT;
  const bool mine = lane % kApart == 0 && my_t < tokens;
  const long long label = mine ? __ldcg(labels + my_t) : -1;
  __syncthreads();

  float top = -INFINITY, sum = 0.f;   // largest logit, and the sum of exponentials relative to it

  // DEPTH pieces of 256 columns in flight; a group of four rows takes a multiple of DEPTH steps (the ones past its
  // columns are zeros)
  const int steps = (blocks + DEPTH - 1) / DEPTH * DEPTH;
  auto load = [&](int row, int q, uint4 (&w)[kFewRows]) {
    const int col = q * 256 + lane * 8;
#pragma unroll
    for (int r = 0; r < kFewRows; ++r)
      w[r] = row + r < end && col < hidden ? __ldcg(reinterpret_cast<const uint4*>(W + size_t(row + r) * ldw + col))
                                           : make_uint4(0, 0, 0, 0);
  };
  uint4 next[DEPTH][kFewRows];
#pragma unroll
  for (int d = 0; d < DEPTH; ++d) load(first, d, next[d]);
#pragma unroll 1
  for (int row = first; row < end; row += kFewRows) {
    float acc[kFewRows][TT] = {};
#pragma unroll 1
    for (int q0 = 0; q0 < steps; q0 += DEPTH) {
#pragma unroll
      for (int d = 0; d < DEPTH; ++d) {
        float f[kFewRows][8];
#pragma unroll
        for (int r = 0; r < kFewRows; ++r) {
          const uint32_t u[4] = {next[d][r].x, next[d][r].y, next[d][r].z, next[d][r].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            f[r][2 * i] = __uint_as_float(u[i] << 16);
            f[r][2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
          }
        }
        // the piece DEPTH further on, of these rows or the next ones
        const bool wraps = q0 + DEPTH >= steps;
        load(wraps ? row + kFewRows : row, wraps ? d : q0 + DEPTH + d, next[d]);
        if (q0 + d < blocks) {
#pragma unroll
          for (int t = 0; t < TT; ++t) {
            const float4* x = reinterpret_cast<const float4*>(s_x + size_t(((q0 + d) * TT + t) * 2) * 128) + lane;
            const float4 a = x[0], b = x[32];
#pragma unroll
            for (int r = 0; r < kFewRows; ++r) {
              float s = acc[r][t];
              s = fmaf(f[r][0], a.x, s);
              s = fmaf(f[r][1], a.y, s);
              s = fmaf(f[r][2], a.z, s);
              s = fmaf(f[r][3], a.w, s);
              s = fmaf(f[r][4], b.x, s);
              s = fmaf(f[r][5], b.y, s);
              s = fmaf(f[r][6], b.z, s);
              acc[r][t] = fmaf(f[r][7], b.w, s);
            }
          }
        }
      }
    }
    // the sums over the lanes: each step exchanges halves while a lane has more than one sum, so that lane l ends
    // with sum l / (32 / kSums)
    float v[kSums];
#pragma unroll
    for (int i = 0; i < kSums; ++i) v[i] = acc[i / TT][i % TT];
#pragma unroll
    for (int n = kSums / 2, o = 16; o; n >>= 1, o >>= 1) {
      if (n) {
#pragma unroll
        for (int i = 0; i < n; ++i) {
          const float r = __shfl_xor_sync(0xffffffffu, (lane & o) ? v[i] : v[i + n], o);
          v[i] = ((lane & o) ? v[i + n] : v[i]) + r;
        }
      } else {
        v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
      }
    }
    const float z = v[0];
    if (mine && row + my_r < end) {
      const float y = z * alpha;
      if (label == row + my_r) zlabel[my_t] = y;
      ce_join(top, sum, y, 1.f);
    }
  }
  // over the four rows' lanes, then over the block's warps
#pragma unroll
  for (int o = TT * kApart; o < 32; o <<= 1) {
    const float m = __shfl_xor_sync(0xffffffffu, top, o), s = __shfl_xor_sync(0xffffffffu, sum, o);
    ce_join(top, sum, m, s);
  }
  if (lane % kApart == 0 && my_r == 0) s_part[warp][my_t] = make_float2(top, sum);
  __syncthreads();
  if (threadIdx.x < TT && int(threadIdx.x) < tokens) {
    top = -INFINITY;
    sum = 0.f;
    for (int w = 0; w < kFewThreads / 32; ++w) ce_join(top, sum, s_part[w][threadIdx.x].x, s_part[w][threadIdx.x].y);
    part[size_t(blockIdx.x) * size_t(tokens) + threadIdx.x] = make_float2(top, sum);
  }
}

template <int TT, int DEPTH>
tkg_status launch_few(int blocks, int smem, const TrainParams& p, const void* X, size_t ldx, const void* W, size_t ldw,
                      cudaStream_t stream) {
  auto kern = ce_few_kernel<TT, DEPTH>;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return TKG_ERR_CUDA;
  static std::atomic<bool> attr_set[64] = {};   // per instantiation and device (set twice alike if two threads race)
  if (!attr_set[dev]) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kFewElements * 4) != cudaSuccess) {
      cudaGetLastError();
      return TKG_ERR_CUDA;
    }
    attr_set[dev] = true;
  }
  return launch_small(kern, dim3(unsigned(blocks)), dim3(kFewThreads), stream, unsigned(smem), p.n, p.m, p.k,
                      static_cast<const uint16_t*>(X), ldx, static_cast<const uint16_t*>(W), ldw, p.labels, p.alpha,
                      p.part, p.zlabel);
}

inline int few_width(int tokens) { return tokens <= 1 ? 1 : (tokens <= 2 ? 2 : 4); }

}  // namespace

int ce_few_blocks(int tokens, int vocab, int hidden) {
  const int tt = few_width(tokens);
  if (tokens > kFewTokens || tt * ((hidden + 255) / 256) * 256 > kFewElements) return 0;
  // One token at any vocabulary; with more the multiply-adds cost more than idle SMs do, past 16384 entries for
  // two (hidden 2112, replayed from a graph: 32768 entries 32.9 us against 26.9 on tiles; 16384 at hidden 512 6.4)
  // and past 8192 for four (8000 entries 10.7 us, 10457 16.4 against 13.5 on tiles; hidden 512 5.9, 7.2 against 7.8).
  if (tt > 1 && (long long)vocab * tt > 32768) return 0;
  const int blocks = ceil_div(vocab, kFewRows * (kFewThreads / 32));   // four rows a warp at least
  return blocks < kFewMaxBlocks ? blocks : kFewMaxBlocks;
}

tkg_status launch_ce_few(const void* X, size_t ldx, const void* W, size_t ldw, const TrainParams& p, int blocks,
                         cudaStream_t stream) {
  const int tt = few_width(p.n), pieces = (p.k + 255) / 256;
  const int smem = tt * pieces * 256 * 4;
  if (tt == 4) return launch_few<4, 2>(blocks, smem, p, X, ldx, W, ldw, stream);
  if (pieces < 3) {
    if (tt == 1) return launch_few<1, 2>(blocks, smem, p, X, ldx, W, ldw, stream);
    return launch_few<2, 2>(blocks, smem, p, X, ldx, W, ldw, stream);
  }
  if (tt == 1) return launch_few<1, 4>(blocks, smem, p, X, ldx, W, ldw, stream);
  return launch_few<2, 4>(blocks, smem, p, X, ldx, W, ldw, stream);
}

}  // namespace tkg
