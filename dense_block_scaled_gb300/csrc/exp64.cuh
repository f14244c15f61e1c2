// exp64.cuh -- the exponential in 64 bits that decides between near ties of routing.
#pragma once

namespace tkg {

// exp in 64 bits, without a branch, so that several run side by side (CUDA's took 1 us each in the choice of experts, one
// after the other), by the reduction of Cody and Waite, log 2 in two parts, and the Taylor series:
// x = n log 2 + r with |r| <= log(2) / 2, the series of e^r to r^13, and 2^n in two halves, as a subnormal result takes two
// steps.  Infinities and NaN come out as they should: n is kept within what the halves can hold.
// Off by less than 2 units in the last place: the series' rest is r^14 / 14!, at most 4.2e-18 and 2^-57.2 of e^r (0.03
// units), r is off by 2^-54 (0.35), the steps' roundings come to one unit.  (0.85 units at most were seen.)
__device__ __forceinline__ double exp64(double x) {
  const double top = 6755399441055744.0;   // 1.5 2^52: adding it rounds to a whole number
  const double y = fma(fmin(fmax(x, -800.0), 800.0), 1.4426950408889634, top);
  const int n = __double2loint(y);
  const double m = y - top;
  const double r = fma(m, -2.3190468138462996e-17, fma(m, -0.6931471805599453, fmin(fmax(x, -800.0), 800.0)));
  double e = 1.0 / 6227020800.0;
  e = fma(e, r, 1.0 / 479001600.0);
  e = fma(e, r, 1.0 / 39916800.0);
  e = fma(e, r, 1.0 / 3628800.0);
  e = fma(e, r, 1.0 / 362880.0);
  e = fma(e, r, 1.0 / 40320.0);
  e = fma(e, r, 1.0 / 5040.0);
  e = fma(e, r, 1.0 / 720.0);
  e = fma(e, r, 1.0 / 120.0);
  e = fma(e, r, 1.0 / 24.0);
  e = fma(e, r, 1.0 / 6.0);
  e = fma(e, r, 0.5);
  e = fma(e, r, 1.0);
  e = fma(e, r, 1.0);
  const int h = n >> 1;
  e = e * __hiloint2double((1023 + h) << 20, 0) * __hiloint2double((1023 + n - h) << 20, 0);
  return x != x ? x : e;
}

}  // namespace tkg
