// exp64 of n numbers, for tests/test_exp64_gpu.py.
#include <cuda_runtime.h>

#include "exp64.cuh"

__global__ void values(const double* x, double* y, long long n) {
  const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  if (i < n) y[i] = tkg::exp64(x[i]);
}

extern "C" int exp64_values(const double* x, double* y, long long n, cudaStream_t stream) {
  if (n < 1 || n > (1ll << 30)) return -1;
  values<<<unsigned((n + 255) / 256), 256, 0, stream>>>(x, y, n);
  return int(cudaGetLastError());
}
