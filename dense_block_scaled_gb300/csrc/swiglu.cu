// swiglu.cu -- the gated activation between two products, rows saved in 8 bits for the backward pass (MXFP8: E4M3
// codes and a power of two per 32 columns, both row-major), and the activation's gradient from them.
//
//   forward   h = silu(g) u of rows [g | u];  silu(x) = x sigma(x), sigma(x) = 1 / (1 + exp(-x))
//   backward  with g, u as saved, the row's router weight w and dh = the gradient to w-less h:
//             dg = w dh u sigma(g) (1 + g (1 - sigma(g))),  du = w dh silu(g),  w h (what the second product's weight
//             gradient multiplies), dw = sum dh h
//
// All of it is bound by HBM: each input byte is read once, each output byte written once.  A warp takes pieces of 256
// columns, a lane 8 of them (16 bytes of BF16, 8 of codes), four lanes a block of 32.
#include "mxfp8.cuh"
#include "train_host.cuh"

namespace tkg {
namespace {

constexpr int kWarps = 8, kPiece = 256;

__device__ __forceinline__ void unpack(const uint4& v, float (&x)[8]) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(u[i] << 16);
    x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack(const float (&x)[8]) {
  return make_uint4(ptx::pack_bf16x2(x[0], x[1]), ptx::pack_bf16x2(x[2], x[3]), ptx::pack_bf16x2(x[4], x[5]),
                    ptx::pack_bf16x2(x[6], x[7]));
}

// Codes of a lane's 8 columns, and their block's scale code (the same in its four lanes).
__device__ __forceinline__ uint2 to_codes(const float (&x)[8], uint32_t& scale) {
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) a = fmaxf(a, fabsf(x[i]));
  a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
  a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 2));
  const int e = mx_exponent(a);
  scale = uint32_t(e + 127);
  const float inv = __uint_as_float(uint32_t(127 - e) << 23);   // 2^-e: normal, as e <= 120
  uint2 q;
  q.x = cvt_e4m3x2(x[0] * inv, x[1] * inv) | (cvt_e4m3x2(x[2] * inv, x[3] * inv) << 16);
  q.y = cvt_e4m3x2(x[4] * inv, x[5] * inv) | (cvt_e4m3x2(x[6] * inv, x[7] * inv) << 16);
  return q;
}
__device__ __forceinline__ void from_codes(const uint2& q, uint32_t scale, float (&x)[8]) {
  const float s = e8m0_value(scale);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = e4m3x2_values((i < 2 ? q.x : q.y) >> (16 * (i & 1)));
    x[2 * i] = v.x * s;
    x[2 * i + 1] = v.y * s;
  }
}

// sigma: 1 ulp of the exponential's and the reciprocal's approximations; subnormal results stay
__device__ __forceinline__ float sigma(float x) {
  float e, r;
  asm("ex2.approx.f32 %0, %1;" : "=f"(e) : "f"(x * -kLog2e));
  asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return r;
}

// Walks `COUNT` consecutive pieces of the rows' pieces from the warp's first on.
template <int COUNT>
struct Pieces {
  int row[COUNT], col[COUNT];   // a lane's first column; row -1: past the end
  __device__ __forceinline__ Pieces(int rows, int width, int lane) {
    const int per_row = (width + kPiece - 1) / kPiece;
    const long long first = ((long long)blockIdx.x * kWarps + (threadIdx.x >> 5)) * COUNT;
    int r = int(first / per_row), piece = int(first - (long long)r * per_row);
#pragma unroll
    for (int i = 0; i < COUNT; ++i) {
      row[i] = r < rows ? r : -1;
      col[i] = piece * kPiece + lane * 8;
      if (++piece == per_row) {
        piece = 0;
        ++r;
      }
    }
  }
};
template <int COUNT>
long long pieces_blocks(int rows, int width) {
  return ((long long)rows * ceil_div(width, kPiece) + COUNT * kWarps - 1) / (COUNT * kWarps);
}

constexpr int kSavePieces = 4;
__global__ void __launch_bounds__(32 * kWarps) save_kernel(int rows, int k, const uint16_t* __restrict__ X, size_t ldx,
                                                           uint8_t* __restrict__ Q, uint8_t* __restrict__ sf) {
  ptx::pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const Pieces<kSavePieces> at(rows, k, lane);
  ptx::pdl_wait();
  uint4 v[kSavePieces];
#pragma unroll
  for (int i = 0; i < kSavePieces; ++i)
    v[i] = at.row[i] >= 0 && at.col[i] < k ? __ldcg(reinterpret_cast<const uint4*>(X + size_t(at.row[i]) * ldx + at.col[i]))
                                           : make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int i = 0; i < kSavePieces; ++i) {
    float x[8];
    uint32_t scale;
    unpack(v[i], x);
    const uint2 q = to_codes(x, scale);
    if (at.row[i] >= 0 && at.col[i] < k) {
      const size_t o = size_t(at.row[i]) * size_t(k) + at.col[i];
      *reinterpret_cast<uint2*>(Q + o) = q;
      if ((lane & 3) == 0) sf[o / 32] = uint8_t(scale);
    }
  }
}

constexpr int kGatePieces = 2;
template <bool SAVE>
__global__ void __launch_bounds__(32 * kWarps)
    swiglu_kernel(int rows, int inner, const uint16_t* __restrict__ GU, size_t ldgu, uint16_t* __restrict__ H, size_t ldh,
                  uint8_t* __restrict__ Q, uint8_t* __restrict__ sf) {
  ptx::pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const Pieces<kGatePieces> at(rows, inner, lane);
  ptx::pdl_wait();
  uint4 v[kGatePieces][2];
#pragma unroll
  for (int i = 0; i < kGatePieces; ++i)
#pragma unroll
    for (int b = 0; b < 2; ++b)
      v[i][b] = at.row[i] >= 0 && at.col[i] < inner
                    ? __ldcg(reinterpret_cast<const uint4*>(GU + size_t(at.row[i]) * ldgu + b * inner + at.col[i]))
                    : make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int i = 0; i < kGatePieces; ++i) {
    const bool there = at.row[i] >= 0 && at.col[i] < inner;
    float g[8], u[8], h[8];
    unpack(v[i][0], g);
    unpack(v[i][1], u);
    if constexpr (SAVE) {
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        uint32_t scale;
        const uint2 q = to_codes(b ? u : g, scale);
        if (there) {
          const size_t o = (size_t(at.row[i]) * 2 + b) * size_t(inner) + at.col[i];
          *reinterpret_cast<uint2*>(Q + o) = q;
          if ((lane & 3) == 0) sf[o / 32] = uint8_t(scale);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) h[j] = g[j] * sigma(g[j]) * u[j];
    if (there) *reinterpret_cast<uint4*>(H + size_t(at.row[i]) * ldh + at.col[i]) = pack(h);
  }
}

struct GateGrad {
  int rows, inner, choices;
  int split;                  // warps per row: 1, 2, 4 or 8
  const uint8_t* Q;
  const uint8_t* sf;
  const uint16_t* dH;
  size_t lddh;
  const int* slots;           // may be null: row r is choice r
  const float* weights;       // may be null: 1
  uint16_t* dGU;
  size_t lddgu;
  uint16_t* H;                // may be null
  size_t ldh;
  float* dweights;            // may be null
};

// The warps of a row take its pieces in turn; dw's parts are joined in a fixed order.
__global__ void __launch_bounds__(32 * kWarps) swiglu_grad_kernel(const GateGrad p) {
  __shared__ float s_part[kWarps];
  ptx::pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int part = warp & (p.split - 1);
  const long long row = (long long)blockIdx.x * (kWarps / p.split) + warp / p.split;
  ptx::pdl_wait();
  int slot = -1;
  if (row < p.rows) slot = p.slots ? __ldcg(p.slots + row) : int(row);
  const bool there = slot >= 0 && slot < p.choices;
  float dot = 0.f;
  if (there) {
    const float w = p.weights ? __ldcg(p.weights + slot) : 1.f;
    const uint8_t* q = p.Q + size_t(row) * 2 * size_t(p.inner);
    const uint8_t* sf = p.sf + size_t(row) * 2 * size_t(p.inner / 32);
    const uint16_t* dh = p.dH + size_t(row) * p.lddh;
    uint16_t* dx = p.dGU + size_t(row) * p.lddgu;
#pragma unroll 2
    for (int c = part * kPiece + lane * 8; c < p.inner; c += p.split * kPiece) {
      const uint2 qg = __ldcg(reinterpret_cast<const uint2*>(q + c));
      const uint2 qu = __ldcg(reinterpret_cast<const uint2*>(q + p.inner + c));
      const uint32_t sg = __ldcg(sf + c / 32), su = __ldcg(sf + (p.inner + c) / 32);
      const uint4 vd = __ldcg(reinterpret_cast<const uint4*>(dh + c));
      float g[8], u[8], d[8], h[8];
      from_codes(qg, sg, g);
      from_codes(qu, su, u);
      unpack(vd, d);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float s = sigma(g[j]), silu = g[j] * s;
        h[j] = silu * u[j];
        dot = fmaf(d[j], h[j], dot);
        const float wd = w * d[j];
        h[j] *= w;
        g[j] = wd * u[j] * (s * fmaf(g[j], 1.f - s, 1.f));
        u[j] = wd * silu;
      }
      *reinterpret_cast<uint4*>(dx + c) = pack(g);
      *reinterpret_cast<uint4*>(dx + p.inner + c) = pack(u);
      if (p.H) *reinterpret_cast<uint4*>(p.H + size_t(row) * p.ldh + c) = pack(h);
    }
  }
  if (!p.dweights) return;
#pragma unroll
  for (int o = 16; o; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
  if (p.split > 1) {
    if (lane == 0) s_part[warp] = dot;
    __syncthreads();
    if (part == 0 && lane == 0)
      for (int i = 1; i < p.split; ++i) dot += s_part[warp + i];
  }
  if (there && part == 0 && lane == 0) p.dweights[slot] = dot;
}

bool size_ok(long long x) { return x <= kMaxSize; }

}  // namespace
}  // namespace tkg

using namespace tkg;

extern "C" {

tkg_status tkg_checkpoint_mxfp8(int rows, int k, const void* X, int ldx, void* Q, void* sf, cudaStream_t stream) {
  if (rows < 0 || k < 0 || ldx < k) return TKG_ERR_INVALID_ARG;
  if (!size_ok(rows) || !size_ok(k)) return TKG_ERR_UNSUPPORTED;
  if (k == 0) return TKG_OK;
  if (k % 32 != 0 || ldx % 8 != 0 || !aligned_to(X, 16) || !aligned_to(Q, 16)) return TKG_ERR_ALIGNMENT;
  if (rows == 0) return TKG_OK;
  if (!X || !Q || !sf) return TKG_ERR_INVALID_ARG;
  const long long blocks = pieces_blocks<kSavePieces>(rows, k);
  if (!size_ok(blocks)) return TKG_ERR_UNSUPPORTED;
  return launch_small(save_kernel, dim3(unsigned(blocks)), dim3(32 * kWarps), stream, 0u, rows, k,
                      static_cast<const uint16_t*>(X), size_t(ldx), static_cast<uint8_t*>(Q), static_cast<uint8_t*>(sf));
}

tkg_status tkg_swiglu(int rows, int inner, const void* GU, int ldgu, void* H, int ldh, void* Q, void* sf,
                      cudaStream_t stream) {
  if (rows < 0 || inner < 0 || ldgu < 2ll * inner || ldh < inner || (Q == nullptr) != (sf == nullptr))
    return TKG_ERR_INVALID_ARG;
  if (!size_ok(rows) || !size_ok(2ll * inner)) return TKG_ERR_UNSUPPORTED;
  if (inner == 0) return TKG_OK;
  if (inner % (Q ? 32 : 8) != 0 || ldgu % 8 != 0 || ldh % 8 != 0 || !aligned_to(GU, 16) || !aligned_to(H, 16) ||
      !aligned_to(Q, 16))
    return TKG_ERR_ALIGNMENT;
  if (rows == 0) return TKG_OK;
  if (!GU || !H) return TKG_ERR_INVALID_ARG;
  const long long blocks = pieces_blocks<kGatePieces>(rows, inner);
  if (!size_ok(blocks)) return TKG_ERR_UNSUPPORTED;
  return launch_small(Q ? swiglu_kernel<true> : swiglu_kernel<false>, dim3(unsigned(blocks)), dim3(32 * kWarps), stream, 0u,
                      rows, inner, static_cast<const uint16_t*>(GU), size_t(ldgu), static_cast<uint16_t*>(H), size_t(ldh),
                      static_cast<uint8_t*>(Q), static_cast<uint8_t*>(sf));
}

tkg_status tkg_swiglu_grad(int rows, int inner, const void* Q, const void* sf, const void* dH, int lddh, const int* slots,
                           int choices, const float* weights, void* dGU, int lddgu, void* H, int ldh, float* dweights,
                           cudaStream_t stream) {
  if (rows < 0 || inner < 0 || choices < 0 || lddh < inner || lddgu < 2ll * inner || (H && ldh < inner) ||
      (dweights && !weights))
    return TKG_ERR_INVALID_ARG;
  if (!size_ok(rows) || !size_ok(choices) || !size_ok(2ll * inner)) return TKG_ERR_UNSUPPORTED;
  if (!aligned_to(slots, 4) || !aligned_to(weights, 4) || !aligned_to(dweights, 4)) return TKG_ERR_ALIGNMENT;
  if (inner > 0 && (inner % 32 != 0 || lddh % 8 != 0 || lddgu % 8 != 0 || (H && ldh % 8 != 0) || !aligned_to(Q, 16) ||
                    !aligned_to(dH, 16) || !aligned_to(dGU, 16) || !aligned_to(H, 16)))
    return TKG_ERR_ALIGNMENT;
  if (rows == 0 || (inner == 0 && !dweights)) return TKG_OK;   // (without columns dw is 0)
  if (inner > 0 && (!Q || !sf || !dH || !dGU)) return TKG_ERR_INVALID_ARG;
  GateGrad p{};
  p.rows = rows;
  p.inner = inner;
  p.choices = choices;
  p.Q = static_cast<const uint8_t*>(Q);
  p.sf = static_cast<const uint8_t*>(sf);
  p.dH = static_cast<const uint16_t*>(dH);
  p.lddh = size_t(lddh);
  p.slots = slots;
  p.weights = weights;
  p.dGU = static_cast<uint16_t*>(dGU);
  p.lddgu = size_t(lddgu);
  p.H = static_cast<uint16_t*>(H);
  p.ldh = size_t(ldh);
  p.dweights = dweights;
  p.split = 1;
  // as many warps per row as it has pieces for, while the rows leave SMs idle
  while (p.split < kWarps && (long long)rows * p.split < 152 * 32 && p.split * kPiece < inner) p.split *= 2;
  return launch_small(swiglu_grad_kernel, dim3(unsigned(ceil_div(rows, kWarps / p.split))), dim3(32 * kWarps), stream, 0u, p);
}

}  // extern "C"
