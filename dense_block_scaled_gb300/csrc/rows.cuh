// rows.cuh -- how kernels that go over rows of a matrix find their place.
#pragma once
#include <cstdint>

namespace tkg {

// x = quotient * d + remainder, in 32 bits where x fits (a 64-bit division takes some 70 instructions).
__device__ __forceinline__ void divide(unsigned long long x, unsigned d, int& quotient, int& remainder) {
  if ((x >> 32) == 0) {
    const unsigned q = unsigned(x) / d;
    quotient = int(q);
    remainder = int(unsigned(x) - q * d);
  } else {
    const unsigned long long q = x / d;
    quotient = int(q);
    remainder = int(x - q * d);
  }
}

// Walks `COUNT` consecutive pieces, of PIECE columns each, of the rows' pieces, from the warp's first on.
template <int COUNT, int WARPS, int PIECE>
struct Pieces {
  int row[COUNT], col[COUNT];   // the piece's first column; row -1: past the end
  __device__ __forceinline__ Pieces(int rows, int width) {
    const int per_row = (width + PIECE - 1) / PIECE;
    int r, piece;
    divide(((unsigned long long)blockIdx.x * WARPS + (threadIdx.x >> 5)) * COUNT, unsigned(per_row), r, piece);
#pragma unroll
    for (int i = 0; i < COUNT; ++i) {
      row[i] = r < rows ? r : -1;
      col[i] = piece * PIECE;
      if (++piece == per_row) {
        piece = 0;
        ++r;
      }
    }
  }
  static long long blocks(int rows, int width) {
    return ((long long)rows * ((width + PIECE - 1) / PIECE) + COUNT * WARPS - 1) / (COUNT * WARPS);
  }
};

}  // namespace tkg
