// swiglu.cu -- the gated activation between two products, rows saved in 8 bits for the backward pass (MXFP8: E4M3
// codes and a power of two per 32 columns, both row-major), and the activation's gradient from them.
//
//   forward   h = silu(g) u of rows [g | u];  silu(x) = x sigma(x), sigma(x) = 1 / (1 + exp(-x))
//   backward  with g, u as saved, the row's router weight w and dh = the gradient to w-less h:
//             dg = w dh u sigma(g) (1 + g (1 - sigma(g))),  du = w dh silu(g),  w h (what the second product's weight
//             gradient multiplies), dw = sum dh h
//
// All of it is bound by HBM: each input byte is read once, each output byte written once.  A warp takes pieces of 256
// columns, a lane 8 of them (16 bytes of BF16, 8 of codes), four lanes a block of 32.  65536 rows of 2 x 2048 with their
// checkpoint 154 us (1082 MB, 159 at the copy rate), without 112 (118); 8192 x 4096 to 8 bits 16.6 us (15.0); the
// gradient of 16004 rows x 1408, 30% of them padding, 28.8 us (23.4), of 65536 rows 103 (96).
#include "mxfp8.cuh"
#include "rows.cuh"
#include "train_host.cuh"

namespace tkg {
namespace {

// Columns of a piece; warps of a block and pieces of a warp, one after another.  Blocks go out at about 1000 a us, so they
// may not be too small (8192 x 4096 to 8 bits, 131072 pieces: with 2 warps of 2 pieces 34 us, with 8 warps 16.5), and a
// warp that takes more pieces leaves a longer last round (4 pieces: 17.5).
constexpr int kPiece = 256, kSaveWarps = 8, kGateWarps = 8;

__device__ __forceinline__ void unpack(const uint4& v, float (&x)[8]) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(u[i] << 16);
    x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
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

// Two FP32 values in one register pair, and the instructions that take such pairs: the activation is bound by how many
// instructions its arithmetic takes as soon as HBM is not.
struct Two {
  unsigned long long v;
};
__device__ __forceinline__ Two two(float a, float b) {
  Two r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ Two two(float a) { return two(a, a); }
__device__ __forceinline__ float2 both(Two x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x.v));
  return r;
}
__device__ __forceinline__ Two operator*(Two a, Two b) {
  Two r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ Two operator+(Two a, Two b) {
  Two r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ Two fma2(Two a, Two b, Two c) {
  Two r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ uint32_t pack(Two x) {
  const float2 f = both(x);
  return ptx::pack_bf16x2(f.x, f.y);
}

// sigma by the approximations of the exponential and the reciprocal, for x from kFar on.  (They flush subnormals: a sigma
// below 2^-126 is 0.  The forms that keep them take four instructions more each; gates below kFar are rare, and where a
// lane has one, it makes those again.)
constexpr float kFar = -87.f;
__device__ __forceinline__ Two sigma(Two x) {
  const float2 y = both(x * two(-kLog2e));
  const float2 z = both(two(ptx::ex2(y.x), ptx::ex2(y.y)) + two(1.f));
  float a, b;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(a) : "f"(z.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(b) : "f"(z.y));
  return two(a, b);
}
__device__ __forceinline__ Two two_of(uint32_t bf16x2) {
  return two(__uint_as_float(bf16x2 << 16), __uint_as_float(bf16x2 & 0xffff0000u));
}
__device__ __forceinline__ Two two_of_codes(uint32_t codes, Two scale) {
  const float2 f = e4m3x2_values(codes);
  return two(f.x, f.y) * scale;
}

// Gates below kFar.  There sigma(x) is exp(x), and 1 - sigma(x) is 1, to FP32's last bit.  exp(x) = t^4 with t = exp(x / 4),
// x / 4 being exact: t is normal down to x = -349, and a product with large numbers between its factors is right where
// exp(x) itself would be below FP32's numbers.  A lane that has one of them among its eight columns makes these again, out
// of the way of the registers of the rest: the 65536 rows above take 154 us (152 without it; 170 where it stood in the
// loop), with one gate of 100 far 232 and with all of them 383.
__device__ __forceinline__ float far_gate(float g, float u) {   // silu(g) u
  const float t = expf(0.25f * g);
  return (((u * t) * (g * t)) * t) * t;
}
__device__ __forceinline__ uint16_t bf16_of(float x) { return uint16_t(ptx::pack_bf16x2(x, 0.f)); }
// The largest of eight BF16 taken as unsigned numbers, two at a time: the farthest below 0 (or NaN), if any is.
__device__ __forceinline__ bool any_far(const uint4& v) {
  const uint32_t m = __vmaxu2(__vmaxu2(v.x, v.y), __vmaxu2(v.z, v.w));
  constexpr uint32_t kBits = 0xc2aeu;   // kFar
  return (m & 0xffffu) > kBits || (m >> 16) > kBits;
}
__device__ __forceinline__ uint32_t pick(const uint4& v, int i) { return i == 0 ? v.x : (i == 1 ? v.y : (i == 2 ? v.z : v.w)); }
__device__ __forceinline__ float bf16_at(const uint4& v, int i) {
  const uint32_t two = pick(v, i >> 1);
  return __uint_as_float((i & 1) ? (two & 0xffff0000u) : (two << 16));
}
// (The inputs come in registers: the output may stand in their place.)
__device__ __noinline__ void far_gates(uint4 g, uint4 u, uint16_t* h) {
#pragma unroll 1
  for (int i = 0; i < 8; ++i)
    if (bf16_at(g, i) < kFar) h[i] = bf16_of(far_gate(bf16_at(g, i), bf16_at(u, i)));
}

constexpr int kSavePieces = 2;
using SavePieces = Pieces<kSavePieces, kSaveWarps, kPiece>;
__global__ void __launch_bounds__(32 * kSaveWarps) save_kernel(int rows, int k, const uint16_t* __restrict__ X,
                                                               size_t ldx, uint8_t* __restrict__ Q,
                                                               uint8_t* __restrict__ sf) {
  ptx::pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  SavePieces at(rows, k);
#pragma unroll
  for (int i = 0; i < kSavePieces; ++i) at.col[i] += lane * 8;
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

constexpr int kGatePieces = 1;
using GatePieces = Pieces<kGatePieces, kGateWarps, kPiece>;
template <bool SAVE>
__global__ void __launch_bounds__(32 * kGateWarps)
    swiglu_kernel(int rows, int inner, const uint16_t* __restrict__ GU, size_t ldgu, uint16_t* __restrict__ H, size_t ldh,
                  uint8_t* __restrict__ Q, uint8_t* __restrict__ sf) {
  ptx::pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  GatePieces at(rows, inner);
#pragma unroll
  for (int i = 0; i < kGatePieces; ++i) at.col[i] += lane * 8;
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
    const bool there = at.row[i] >= 0 && at.col[i] < inner, far = any_far(v[i][0]);
    if constexpr (SAVE) {
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        float x[8];
        uint32_t scale;
        unpack(v[i][b], x);
        const uint2 q = to_codes(x, scale);
        if (there) {
          const size_t o = (size_t(at.row[i]) * 2 + b) * size_t(inner) + at.col[i];
          *reinterpret_cast<uint2*>(Q + o) = q;
          if ((lane & 3) == 0) sf[o / 32] = uint8_t(scale);
        }
      }
    }
    const uint32_t g[4] = {v[i][0].x, v[i][0].y, v[i][0].z, v[i][0].w}, u[4] = {v[i][1].x, v[i][1].y, v[i][1].z, v[i][1].w};
    uint32_t h[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const Two x = two_of(g[j]);
      h[j] = pack(x * sigma(x) * two_of(u[j]));
    }
    if (there) {
      *reinterpret_cast<uint4*>(H + size_t(at.row[i]) * ldh + at.col[i]) = make_uint4(h[0], h[1], h[2], h[3]);
      if (far) far_gates(v[i][0], v[i][1], H + size_t(at.row[i]) * ldh + at.col[i]);
    }
  }
}

constexpr int kGradWarps = 8, kGradLeast = 4;   // warps of a block: at most, and at least
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

// The same of the gradients; returns what these columns add to the sum of dh silu(g) u.
__device__ __noinline__ float far_gradients(const GateGrad& p, long long row, int c, float w, uint4 dh) {
  const uint8_t* q = p.Q + size_t(row) * 2 * size_t(p.inner) + c;
  const uint8_t* sf = p.sf + size_t(row) * 2 * size_t(p.inner / 32);
  const float scale_g = e8m0_value(__ldcg(sf + c / 32)), scale_u = e8m0_value(__ldcg(sf + (p.inner + c) / 32));
  float dots = 0.f;
#pragma unroll 1
  for (int i = 0; i < 8; ++i) {
    const float g = e4m3x2_values(__ldcg(q + i)).x * scale_g;
    if (!(g < kFar)) continue;
    const float u = e4m3x2_values(__ldcg(q + p.inner + i)).x * scale_u, d = bf16_at(dh, i);
    const float h = far_gate(g, u), t = expf(0.25f * g), wd = w * d;
    dots = fmaf(d, h, dots);
    uint16_t* dx = p.dGU + size_t(row) * p.lddgu + c + i;
    dx[0] = bf16_of(((u * t) * ((1.f + g) * t)) * ((wd * t) * t));   // sigma (1 + g (1 - sigma)) is exp(g) (1 + g)
    dx[p.inner] = bf16_of((((wd * t) * (g * t)) * t) * t);
    if (p.H) p.H[size_t(row) * p.ldh + c + i] = bf16_of(h * w);
  }
  return dots;
}

// The warps of a row take its pieces in turn; dw's parts are joined in a fixed order.
__global__ void __launch_bounds__(32 * kGradWarps, 4) swiglu_grad_kernel(const __grid_constant__ GateGrad p) {
  __shared__ float s_part[kGradWarps];
  ptx::pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int part = warp & (p.split - 1);
  const long long row = (long long)blockIdx.x * ((blockDim.x >> 5) / p.split) + warp / p.split;
  ptx::pdl_wait();
  int slot = -1;
  if (row < p.rows) slot = p.slots ? __ldcg(p.slots + row) : int(row);
  const bool there = slot >= 0 && slot < p.choices;
  Two dots = two(0.f);
  if (there) {
    const Two w = two(p.weights ? __ldcg(p.weights + slot) : 1.f);
    const uint8_t* q = p.Q + size_t(row) * 2 * size_t(p.inner);
    const uint8_t* sf = p.sf + size_t(row) * 2 * size_t(p.inner / 32);
    const uint16_t* dh = p.dH + size_t(row) * p.lddh;
    uint16_t* dx = p.dGU + size_t(row) * p.lddgu;
    uint16_t* ho = p.H ? p.H + size_t(row) * p.ldh : nullptr;
    // two pieces on their way at a time
#pragma unroll 1
    for (int c0 = part * kPiece + lane * 8; c0 < p.inner; c0 += 2 * p.split * kPiece) {
      uint2 qg[2], qu[2];
      uint32_t sg[2], su[2];
      uint4 vd[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int c = c0 + i * p.split * kPiece;
        if (c < p.inner) {
          qg[i] = __ldcg(reinterpret_cast<const uint2*>(q + c));
          qu[i] = __ldcg(reinterpret_cast<const uint2*>(q + p.inner + c));
          sg[i] = __ldcg(sf + c / 32);
          su[i] = __ldcg(sf + (p.inner + c) / 32);
          vd[i] = __ldcg(reinterpret_cast<const uint4*>(dh + c));
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int c = c0 + i * p.split * kPiece;
        if (c >= p.inner) break;
        const Two scale_g = two(e8m0_value(sg[i])), scale_u = two(e8m0_value(su[i]));
        const uint32_t dv[4] = {vd[i].x, vd[i].y, vd[i].z, vd[i].w};
        uint32_t og[4], ou[4], oh[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const Two g = two_of_codes((j < 2 ? qg[i].x : qg[i].y) >> (16 * (j & 1)), scale_g);
          const Two u = two_of_codes((j < 2 ? qu[i].x : qu[i].y) >> (16 * (j & 1)), scale_u);
          const Two d = two_of(dv[j]), s = sigma(g), silu = g * s, wd = w * d;
          const Two h = silu * u;
          dots = fma2(d, h, dots);
          oh[j] = pack(h * w);
          // sigma (1 + g (1 - sigma)) = sigma + silu (1 - sigma), times u first: w dh u alone may be past FP32's range
          og[j] = pack(wd * (u * fma2(silu, fma2(s, two(-1.f), two(1.f)), s)));
          ou[j] = pack(wd * silu);
        }
        *reinterpret_cast<uint4*>(dx + c) = make_uint4(og[0], og[1], og[2], og[3]);
        *reinterpret_cast<uint4*>(dx + p.inner + c) = make_uint4(ou[0], ou[1], ou[2], ou[3]);
        if (ho) *reinterpret_cast<uint4*>(ho + c) = make_uint4(oh[0], oh[1], oh[2], oh[3]);
        // a block with room for them, as 448 x 2^-3 is above kFar (what they added to the dots is 0)
        if (sg[i] >= 125u) dots = dots + two(far_gradients(p, row, c, both(w).x, vd[i]), 0.f);
      }
    }
  }
  if (!p.dweights) return;
  float dot = both(dots).x + both(dots).y;
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
  const long long blocks = SavePieces::blocks(rows, k);
  if (!size_ok(blocks)) return TKG_ERR_UNSUPPORTED;
  return launch_small(save_kernel, dim3(unsigned(blocks)), dim3(32 * kSaveWarps), stream, 0u, rows, k,
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
  const long long blocks = GatePieces::blocks(rows, inner);
  if (!size_ok(blocks)) return TKG_ERR_UNSUPPORTED;
  return launch_small(Q ? swiglu_kernel<true> : swiglu_kernel<false>, dim3(unsigned(blocks)), dim3(32 * kGateWarps), stream, 0u,
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
  // As many warps per row as it has pieces for, while the rows leave SMs idle (a piece to each warp, 6 of them, whatever the
  // rows: 16004 rows x 1408 43 us in place of 28).  Blocks of 4 warps: of 8 the last round is longer (34 us).
  while (p.split < kGradWarps && (long long)rows * p.split < kSMs * 32 && p.split * kPiece < inner) p.split *= 2;
  const int warps = p.split > kGradLeast ? p.split : kGradLeast;
  return launch_small(swiglu_grad_kernel, dim3(unsigned(ceil_div(rows, warps / p.split))), dim3(unsigned(32 * warps)), stream, 0u, p);
}

}  // extern "C"
