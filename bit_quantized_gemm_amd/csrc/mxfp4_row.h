// Pieces of the MXFP4 row quantizer (atom_mxfp4.h), shared by its kernel, the norm in front of it and the product that
// quantizes its tokens itself.  Eight elements a lane, four lanes a block, 32 lanes a group.
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

// The codes of eight values in units of their scale: nearest, ties to the even code, saturating (the conversion's
// own rounding; walked over all fp16 values and the borders' neighbours by a test).
__device__ __forceinline__ uint32_t codes8(const float (&u)[8]) {
  uint32_t c = 0;
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, u[0], u[1], 1.0f, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, u[2], u[3], 1.0f, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, u[4], u[5], 1.0f, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, u[6], u[7], 1.0f, 3);
}

// Elements 8 c .. 8 c + 7 of a row of K >= 8 that may begin at any element, in two steps, so that nothing waits between loads: past
// the row's end its last eight are loaded, and `behind` moves those that are wanted into place, zeros behind them.
__device__ __forceinline__ u32x4 load8_any(const uint16_t* x, int c, int K) {
  return *reinterpret_cast<const w8a8::Unaligned*>(x + min(8 * c, K - 8));
}
__device__ __forceinline__ u32x4 behind(u32x4 w, int c, int K) {
  const int s = 8 * c + 8 - K;                          // elements of the eight that are not there
  if (s <= 0) return w;
  uint64_t lo = (uint64_t)w[1] << 32 | w[0], hi = (uint64_t)w[3] << 32 | w[2];
  if (s & 4) lo = hi, hi = 0;
  const int b = 16 * (s & 3);
  lo = lo >> b | (hi << 1) << (63 - b);
  hi >>= b;
  return s < 8 ? u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)} : u32x4{0, 0, 0, 0};
}

// Stores the first `left` of eight 16-bit elements, at any address of an element (one instruction where all are there; eight stores
// of an element each take four times as long: a product's 1275 x 19836 x 128 57 us, 23 so).
__device__ __forceinline__ void store8(uint16_t* dst, u32x4 v, int left) {
  if (left >= 8) {
    *reinterpret_cast<w8a8::Unaligned*>(dst) = v;
  } else {
#pragma unroll
    for (int e = 0; e < 7; ++e)
      if (e < left) dst[e] = (uint16_t)(v[e / 2] >> (16 * (e & 1)));
  }
}

// The largest magnitude of eight 16-bit elements, as bits.
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t max8(u32x4 w) {
  u16x2 m[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) m[j] = __builtin_bit_cast(u16x2, w[j] & 0x7FFF7FFFu);
  const u16x2 t = __builtin_elementwise_max(__builtin_elementwise_max(m[0], m[1]), __builtin_elementwise_max(m[2], m[3]));
  return max((uint32_t)t[0], (uint32_t)t[1]);
}

// The codes of two elements into byte J of c: elements / scale, of which the conversion takes the exponent alone.
template <int J>
__device__ __forceinline__ uint32_t codes2(Fp16, uint32_t c, uint32_t w, float scale) {
  typedef _Float16 h2 __attribute__((ext_vector_type(2)));
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(h2, w), scale, J);
}
template <int J>
__device__ __forceinline__ uint32_t codes2(Bf16, uint32_t c, uint32_t w, float scale) {
  typedef __bf16 b2 __attribute__((ext_vector_type(2)));
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(b2, w), scale, J);
}

// Codes and scale byte of a lane's eight 16-bit elements; all lanes of the wave call it.  The conversion takes the elements as
// they are and rounds once; byte << 23 is 2^(byte - 127) as it reads a scale, with byte 0 as well.
template <class T>
__device__ __forceinline__ uint32_t quantize8(u32x4 w, uint32_t& byte) {
  byte = scale_byte(__builtin_bit_cast(uint32_t, T::load(block_max(max8(w)))));
  const float scale = __builtin_bit_cast(float, byte << 23);
  const uint32_t c = codes2<3>(T{}, codes2<2>(T{}, codes2<1>(T{}, codes2<0>(T{}, 0, w[0], scale), w[1], scale), w[2], scale), w[3], scale);
  return byte == kNanScale ? 0u : c;
}

}  // namespace mx
}  // namespace atom
