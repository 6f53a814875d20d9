// Pieces of the MXFP4 row quantizer (atom_mxfp4.h), shared by its kernel, the norm in front of it and the product of
// very few tokens, which quantizes them itself.  Eight elements a lane, four lanes a block, 32 lanes a group.
#pragma once

#include "serve_internal.h"
#include "w8a8_row.h"

namespace atom {
namespace mx {

constexpr int kBlock = 32, kGroup = 256;
constexpr uint32_t kNanScale = 255;

__host__ __device__ inline int padded(int K) { return (K + kGroup - 1) / kGroup * kGroup; }

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, false);
}
// max over the four lanes of a block, of values whose order is that of their bits.
__device__ __forceinline__ uint32_t block_max(uint32_t m) {
  m = max(m, dpp<0xB1>(m));                             // lane ^ 1
  return max(m, dpp<0x4E>(m));                          // lane ^ 2
}

// The scale bytes of four neighbouring blocks as a word, in each lane that holds one of them.
__device__ __forceinline__ uint32_t gather_scales(uint32_t byte, int lane) {
  uint32_t w = byte << (8 * ((lane >> 2) & 3));
  w |= dpp<0x128>(w);                                   // lane + 8 (mod 16) of each row of 16
  return w | dpp<0x124>(w);                             // lane + 4
}

// The scale byte of a block with the largest magnitude `top` (fp32 bits, no sign): floor(log2) - 2 and the bias.  The
// bits of fp32's smallest numbers have the exponent 0, which is clamped like theirs.
__device__ __forceinline__ uint32_t scale_byte(uint32_t top) {
  const int e = (int)(top >> 23);
  return e == 255 ? kNanScale : (uint32_t)max(e - 2, 0);
}
// 1 / 2^e of a scale byte below 253, exact: 2^127 for byte 0 (2^-127).
__device__ __forceinline__ float inverse_scale(uint32_t byte) { return __builtin_bit_cast(float, (254u - byte) << 23); }

// The codes of eight values in units of their scale: nearest, ties to the even code, saturating (the conversion's
// own rounding; walked over all fp16 values and the borders' neighbours by a test).
__device__ __forceinline__ uint32_t codes8(const float (&u)[8]) {
  uint32_t c = 0;
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, u[0], u[1], 1.0f, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, u[2], u[3], 1.0f, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, u[4], u[5], 1.0f, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, u[6], u[7], 1.0f, 3);
}

// Codes and scale byte of a lane's eight 16-bit elements; all lanes of the wave call it.  x * 2^-e is exact but for
// values below 2^-125 of the block's largest, which round to zero either way.
template <class T>
__device__ __forceinline__ uint32_t quantize8(u32x4 w, uint32_t& byte) {
  byte = scale_byte(__builtin_bit_cast(uint32_t, T::load(block_max(w8a8::max8(w, 0)))));
  const bool nan = byte == kNanScale;
  const float inv = nan ? 0.0f : inverse_scale(byte);
  float u[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) u[j] = elem<T>(w[j / 2], j & 1) * inv;
  const uint32_t c = codes8(u);
  return nan ? 0u : c;
}

}  // namespace mx
}  // namespace atom
