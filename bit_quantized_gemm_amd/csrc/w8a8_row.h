// Pieces of the W8A8 row quantize shared by its kernel and by the product of very few tokens, which quantizes them itself.
#pragma once

#include "serve_internal.h"

namespace atom {
namespace w8a8 {

// 16 bytes at any address of a 16-bit element: gfx950 loads them in one instruction (two cache lines at most).
typedef u32x4 Unaligned __attribute__((aligned(2)));

// Elements 8 c .. 8 c + 7 of a row of K, zeros behind K.  kWide: the row is 16-byte aligned and K a multiple of 8.
template <bool kWide>
__device__ __forceinline__ u32x4 load8(const uint16_t* x, int c, int K) {
  u32x4 w = {0, 0, 0, 0};
  if (kWide) {
    if (8 * c < K) w = *reinterpret_cast<const u32x4*>(x + 8 * c);
  } else if (8 * c + 8 <= K) {
    w = *reinterpret_cast<const Unaligned*>(x + 8 * c);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int e = 8 * c + 2 * j;
      w[j] = (e < K ? (uint32_t)x[e] : 0u) | (e + 1 < K ? (uint32_t)x[e + 1] << 16 : 0u);
    }
  }
  return w;
}

// max |x| of eight elements as bits: the order of the bits is the order of the values.
__device__ __forceinline__ uint32_t max8(u32x4 w, uint32_t m) {
#pragma unroll
  for (int j = 0; j < 4; ++j) m = max(m, max(w[j] & 0x7FFFu, (w[j] >> 16) & 0x7FFFu));
  return m;
}

// The codes of eight elements as bytes.  s = fl32(max / 127), r = fl32(1 / s) (0 for s = 0).  |x| is at most the row's
// maximum, so a code is within +-127 by itself; next to fp32's smallest numbers (bf16 rows below 2^-93) the
// reciprocal overflows and the scale's own rounding can carry a code further: the plain divide, clamped.
template <class T>
__device__ __forceinline__ u32x2 codes8(u32x4 w, float s, float r) {
  const bool tiny = s < 0x1p-100f;
  u32x2 o;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    uint32_t b[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float v = elem<T>(w[2 * half + j / 2], j & 1);
      const float u = tiny ? __builtin_fminf(__builtin_fmaxf(s > 0.0f ? v / s : 0.0f, -127.0f), 127.0f) : quotient(v, s, r);
      b[j] = __builtin_bit_cast(uint32_t, u + 12582912.0f);     // 1.5 * 2^23: the integer (ties to even) in the low byte
    }
    o[half] = __builtin_amdgcn_perm(b[1], b[0], 0x0C0C0400u) | __builtin_amdgcn_perm(b[3], b[2], 0x04000C0Cu);
  }
  return o;
}

}  // namespace w8a8
}  // namespace atom
