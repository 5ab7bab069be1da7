// mrr_quotient.h -- 64-bit numbers on their way to few bits by way of 32, so that the last
// rounding is that of the exact number. No HIP header: the tests run it on the host as well.
#pragma once

#include <stdint.h>

#if defined(__HIP__)
#define MRR_ANYWHERE __host__ __device__ inline
#else
#define MRR_ANYWHERE inline
#endif

namespace mrr {

// The nearer of 32 bits' neighbours towards 0, its last bit set, where d is none of them: a
// rounding of it to fewer bits is then that of d.
MRR_ANYWHERE float to_odd(double d) {
  const float f = static_cast<float>(d);
  const double back = static_cast<double>(f);
  if (back == d || !(__builtin_fabsf(f) < __builtin_inff())) return f;
  uint32_t b;
  __builtin_memcpy(&b, &f, 4);
  b = (b - (__builtin_fabs(back) > __builtin_fabs(d) ? 1u : 0u)) | 1u;
  float odd;
  __builtin_memcpy(&odd, &b, 4);
  return odd;
}

// The same of a number that lies off a finite d towards the sign of `rest`, by less than d's
// neighbours in 64 bits do.
MRR_ANYWHERE float to_odd(double d, double rest) {
  const float f = static_cast<float>(d);
  if (rest == 0.0 || static_cast<double>(f) != d) return to_odd(d);
  uint32_t b;
  __builtin_memcpy(&b, &f, 4);
  b = (b - ((d < 0.0) == (rest > 0.0) ? 1u : 0u)) | 1u;
  float odd;
  __builtin_memcpy(&odd, &b, 4);
  return odd;
}

// full p / most, of products p and most (|p| <= most, inverse = 1 / most), where full p is exact in
// 64 bits and no quotient lies off a border between two roundings by less than 64 bits hold: of
// products of 46 bits by 127, and of two 32-bit numbers' 48 by 448, whose e4m3 borders have 5
// bits, so that what is off one is off by more than 2^-53 of it.
MRR_ANYWHERE float short_quotient_to_odd(double p, double most, double inverse, double full) {
  const double q0 = full * p * inverse;
  return to_odd(__builtin_fma(__builtin_fma(-q0, most, full * p), inverse, q0));
}

// Of products of two 32-bit numbers 127 p has up to 55 bits and is taken in two parts. With
// most's 48 bits every remainder is exact, so the last one has the sign of what q lacks of the
// exact quotient, and is 0 where q is that: a quotient on a border, or next to one by less than
// 64 bits hold, is on the side where it belongs. (8192 x 4096 fp32 rows with their sum to int8
// 83.8 us, with one part 82.5.)
MRR_ANYWHERE float quotient_to_odd(double p, double most, double inverse, double full) {
  const double hi = full * p, lo = __builtin_fma(full, p, -hi);
  const double q0 = hi * inverse;
  const double q = __builtin_fma(__builtin_fma(-q0, most, hi) + lo, inverse, q0);
  return to_odd(q, __builtin_fma(-q, most, hi) + lo);
}

}  // namespace mrr
