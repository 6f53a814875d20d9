// MXFP4 row quantize for gfx950, and its inverse (formats: atom_mxfp4.h).
//
// What bounds it: HBM, 2 K bytes in and K / 2 + K / 32 out for a row.  A block's scale needs its own 32 values alone, so a
// row needs no barrier: a lane loads eight elements (16 bytes), four lanes join their maxima by two DPP moves, and the
// 16 lanes of four blocks gather a word of scale bytes.  Codes leave as 4 bytes a lane, whole lines a wave.
//
// Scales lie group by group ([groups, rows, 8]), so a line of them belongs to 16 rows: a workgroup takes neighbouring rows,
// whose pieces of it meet in one L2.
//
// Measured: 8192 x 8192 37.8 us from HBM (4.5 TB/s; a copy of memory reaches 5.1), 2048 x 11008 14.4, with operands and codes in the
// last-level cache 26.6 and 10.1, 16 x 4096 1.9 to 2.1 us, of which the launch is most; back to values 8192 x 8192 42 and 30 us.  With the
// elements multiplied in fp32 before the conversion a tenth more (2048 x 11008 14.6 for 13.3, three sets in turn).
#include "mxfp4_row.h"

namespace atom {
namespace {

constexpr int kThreads = 256;
// Workgroup (x, y): rows 4 RW x .., elements 512 CW y .. + 512 CW - 1 of each; a wave takes one row in four.
template <class T, bool VEC, int RW, int CW>
__global__ __launch_bounds__(kThreads) void quantize_kernel(const uint16_t* __restrict__ X, int64_t ldx, int rows, int K,
                                                            int Kp, uint8_t* __restrict__ Xq, uint8_t* __restrict__ sx) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  auto row_of = [&](int i) { return (int)blockIdx.x * 4 * RW + 4 * i + wave; };
  auto chunk_of = [&](int j) { return ((int)blockIdx.y * CW + j) * 64 + lane; };   // of eight elements
  u32x4 w[RW][CW];
#pragma unroll
  for (int i = 0; i < RW; ++i)
#pragma unroll
    for (int j = 0; j < CW; ++j) w[i][j] = w8a8::load8<VEC>(X + (int64_t)min(row_of(i), rows - 1) * ldx, chunk_of(j), K);
#pragma unroll
  for (int i = 0; i < RW; ++i)
#pragma unroll
    for (int j = 0; j < CW; ++j) {
      const int row = row_of(i), c = chunk_of(j);
      uint32_t byte;
      const uint32_t code = mx::quantize8<T>(w[i][j], byte);
      const uint32_t four = mx::gather_scales(byte, lane);
      if (row < rows && 8 * c < Kp) {
        *reinterpret_cast<uint32_t*>(Xq + (int64_t)row * (Kp / 2) + 4 * c) = code;
        if ((lane & 15) == 0)
          *reinterpret_cast<uint32_t*>(sx + ((int64_t)(c >> 5) * rows + row) * 8 + ((c >> 4) & 1) * 4) = four;
      }
    }
}

// One thread per eight elements of each of ROWS / 4 rows.
template <class T, bool VEC, int ROWS>
__global__ __launch_bounds__(kThreads) void dequantize_kernel(const uint8_t* __restrict__ Xq, const uint8_t* __restrict__ sx,
                                                              int rows, int K, int Kp, uint16_t* __restrict__ X) {
  const int c = blockIdx.y * 64 + (threadIdx.x & 63), wave = threadIdx.x >> 6;
  if (8 * c >= K) return;
  uint32_t code[ROWS / 4], byte[ROWS / 4];
#pragma unroll
  for (int i = 0; i < ROWS / 4; ++i) {
    const int64_t row = min((int)blockIdx.x * ROWS + 4 * i + wave, rows - 1);
    code[i] = *reinterpret_cast<const uint32_t*>(Xq + row * (Kp / 2) + 4 * c);
    byte[i] = sx[((int64_t)(c >> 5) * rows + row) * 8 + ((c >> 2) & 7)];
  }
#pragma unroll
  for (int i = 0; i < ROWS / 4; ++i) {
    const int row = blockIdx.x * ROWS + 4 * i + wave;
    if (row >= rows) return;
    // 2^e; 2^-127 is one of fp32's subnormal numbers, and all products with a code are exact
    const float scale = __builtin_bit_cast(float, byte[i] == mx::kNanScale ? 0x7FC00000u : byte[i] ? byte[i] << 23 : 0x00400000u);
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t q = code[i] >> (4 * j), m = q & 7;
      // 0, 0.5, 1, 1.5 in halves, then 1 or 1.5 times 2 and 4
      const float a = m < 4 ? 0.5f * (float)m : (float)(2 + (m & 1)) * (m < 6 ? 1.0f : 2.0f);
      v[j] = (q & 8 ? -a : a) * scale;
    }
    mx::store8(X + (int64_t)row * K + 8 * c, u32x4{pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]), pack2<T>(v[4], v[5]), pack2<T>(v[6], v[7])},
               VEC ? 8 : K - 8 * c);
  }
}

// Whether there are workgroups enough for several rows each.
bool many(int rows, int Kp, int per, int columns, int64_t enough) {
  return (int64_t)((rows + per - 1) / per) * ((Kp + columns - 1) / columns) >= enough;
}

}  // namespace

// (rows <= 2^24: at most 2^22 workgroups of 2^8 threads in x.)
hipError_t launch_quantize_mxfp4(const uint16_t* X, int64_t ldx, bool bf16, int rows, int K, uint8_t* Xq, uint8_t* sx,
                                 hipStream_t stream) {
  const int Kp = mx::padded(K);
  const bool vec = K % 8 == 0 && (rows == 1 || ldx % 8 == 0) && (reinterpret_cast<uintptr_t>(X) & 15) == 0;
  auto go = [&](auto kernel, int per, int columns) {
    hipLaunchKernelGGL(kernel, dim3((rows + per - 1) / per, (Kp + columns - 1) / columns), dim3(kThreads), 0, stream, X, ldx, rows, K,
                       Kp, Xq, sx);
  };
  // (us, rows x columns of a workgroup 4 x 512, 16 x 512, 8 x 1024: 512 x 4096 2.9, 3.2, 3.2; 1024 x 4096 3.6, 3.9, 4.0; 2048 x 4096 6.8, 6.2, 6.2;
  // 2048 x 11008 16.2, 14.3, 14.2; 8192 x 8192 36.3, 38.3, 37.8; unaligned 333 x 1155 2.3, 3.5, 3.2, 3000 x 1155 4.4, 5.5, 5.1)
  auto pick = [&](auto type) {
    using T = decltype(type);
    if (many(rows, Kp, 4, 512, 4096)) vec ? go(quantize_kernel<T, true, 2, 2>, 8, 1024) : go(quantize_kernel<T, false, 2, 2>, 8, 1024);
    else vec ? go(quantize_kernel<T, true, 1, 1>, 4, 512) : go(quantize_kernel<T, false, 1, 1>, 4, 512);
  };
  bf16 ? pick(Bf16{}) : pick(Fp16{});
  return hipGetLastError();
}

hipError_t launch_dequantize_mxfp4(const uint8_t* Xq, const uint8_t* sx, int rows, int K, bool bf16, uint16_t* X,
                                   hipStream_t stream) {
  const int Kp = mx::padded(K);
  const bool vec = K % 8 == 0;
  auto go = [&](auto kernel, int per) {
    hipLaunchKernelGGL(kernel, dim3((rows + per - 1) / per, (Kp + 511) / 512), dim3(kThreads), 0, stream, Xq, sx, rows, K, Kp, X);
  };
  auto pick = [&](auto type) {
    using T = decltype(type);
    // (us, 4 and 16 rows: 16 x 4096 2.0 and 3.3, 8192 x 8192 49 and 38: a line of scales is read once for 16 rows)
    if (many(rows, Kp, 16, 512, 2048)) vec ? go(dequantize_kernel<T, true, 16>, 16) : go(dequantize_kernel<T, false, 16>, 16);
    else vec ? go(dequantize_kernel<T, true, 4>, 4) : go(dequantize_kernel<T, false, 4>, 4);
  };
  bf16 ? pick(Bf16{}) : pick(Fp16{});
  return hipGetLastError();
}

}  // namespace atom
