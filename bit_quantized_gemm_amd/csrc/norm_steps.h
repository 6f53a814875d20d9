// Steps of the norm's exact codes: plain arithmetic, shared by the kernel (rmsnorm.hip) and by a host test.
#pragma once

#include <stdint.h>

#ifdef __HIPCC__
#define NORM_FN __host__ __device__ inline __attribute__((always_inline))
#else
#define NORM_FN static inline
#endif

namespace rms {

// a / b rounded once, from r = 1 / b rounded once, where nothing on the way overflows or underflows (a zero loses its sign).  The
// product is within two units in the last place; the first step brings it within one, and from there the second rounds
// the quotient itself (Markstein, Computation of Elementary Functions on the IBM RISC System/6000 Processor, 1990).  A row's
// divisors are few; a division of its own for each value costs three times as much (2048 x 11008 with a residual to MXFP4 41.7 us so).
NORM_FN double divided(double a, double b, double r) {
  double q = a * r;
  q = __builtin_fma(__builtin_fma(-q, b, a), r, q);
  return __builtin_fma(__builtin_fma(-q, b, a), r, q);
}

// Distance of an fp32 number (as bits) from the nearest border of two MXFP4 codes, or of two exponents (4 and 8): in units of its last
// place, offset by 4, so that up to four below to three above are 0 to 7.  All of these have 21 zeros at the end of their
// significands; smaller numbers than the lowest border, 0.25, are none whatever their bits: zeros, above all.
NORM_FN uint32_t border_distance(uint32_t bits) {
  const uint32_t a = bits & 0x7FFFFFFFu;
  return a < 0x3E000000u ? 0x1FFFFFu : (a + 4) & 0x1FFFFFu;
}

}  // namespace rms
