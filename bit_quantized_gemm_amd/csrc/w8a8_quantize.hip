// Row quantize of the W8A8 layer for gfx950: one fp32 scale and K int8 codes for each row of an
// fp16 or bf16 matrix, codes = clamp(rint(fl32(x / s)), -127, 127), s = fl32(max|x| / 127).
//
// What bounds it: HBM, 2 K bytes in and K + 4 out for a row (3 K in all).  The scale needs the whole row before the first
// code, so a row is read once into registers by the threads that share it, its maximum is joined
// (in a wave by DPP-free shuffles, across waves through LDS) and the codes are made from the registers.
// The threads of a row follow its length: a wave for short rows (four rows a workgroup, no
// barrier), 256 or 512 threads up to 16384 elements, 1024 beyond; few rows, which leave units idle, take more (us, with the
// other count: 256 x 2048 2.7 and 3.3, 1024 x 2048 3.8 and 3.5, 4096 x 2048 8.7 and 5.3; 512 x 8192 3.7 and 4.1, 1024 x 8192 5.3
// and 5.3, 2048 x 8192 10.1 and 9.4).  The counts cross at 250 rows of 1024 elements and 700 of 2048, at 700 of 5120 and 1000 of
// 8192; the borders, 384 and 1024, lie between and cost at most 10% next to them.
// Rows whose elements no aligned 16-byte load fits (odd K or stride, shifted views) are read by unaligned ones, the last few
// elements one by one.
//
// The codes are those of an IEEE divide, without its dozen instructions an element: see quotient().
//
// Measured: 2048 x 11008 12.8 us and 4096 x 8192 16.7 us (5.3 and 5.9 TB/s with the input in the caches, a copy of memory reaches 5.1),
// 16 x 4096 2.9 us, of which the launch is most, 333 x 1155 (unaligned rows) 3.3 us.
#include "w8a8_row.h"
#include "w8a8_rows.h"

namespace atom {
namespace {

template <class T, int THREADS, int CH, bool VEC>
__global__ __launch_bounds__(w8a8::block_threads(THREADS)) void quantize_kernel(const uint16_t* __restrict__ X, int64_t ldx,
                                                                               int rows, int K, int Kp,
                                                                               int8_t* __restrict__ Xq,
                                                                               float* __restrict__ sx) {
  constexpr int kBlock = w8a8::block_threads(THREADS);
  constexpr int kRows = kBlock / THREADS;               // rows of one workgroup
  const int t = threadIdx.x % THREADS;
  const int row = blockIdx.x * kRows + threadIdx.x / THREADS;
  if (kRows > 1 && row >= rows) return;                 // whole waves: no barrier follows
  const uint16_t* x = X + (size_t)row * ldx;

  u32x4 w[CH];                                          // chunk c = t + i * THREADS: elements 8 c .. 8 c + 7
#pragma unroll
  for (int i = 0; i < CH; ++i) w[i] = w8a8::load8<VEC>(x, t + i * THREADS, K);
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < CH; ++i) m = w8a8::max8(w[i], m);
#pragma unroll
  for (int d = 32; d; d >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d));
  if constexpr (THREADS > 64) {
    __shared__ uint32_t wave_max[THREADS / 64];
    if ((threadIdx.x & 63) == 0) wave_max[threadIdx.x >> 6] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < THREADS / 64; ++i) m = max(m, wave_max[i]);
  }
  const float s = T::load(m) / 127.0f;
  if (t == 0) sx[row] = s;
  const float r = s > 0.0f ? 1.0f / s : 0.0f;
  int8_t* q = Xq + (size_t)row * Kp;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = t + i * THREADS;
    if (8 * c < Kp) *reinterpret_cast<u32x2*>(q + 8 * c) = w8a8::codes8<T>(w[i], s, r);
  }
}

template <class T, int THREADS, int CH>
void launch(const uint16_t* X, int64_t ldx, bool vec, int rows, int K, int Kp, int8_t* Xq, float* sx, hipStream_t st) {
  constexpr int kBlock = w8a8::block_threads(THREADS), kRows = kBlock / THREADS;
  for (int64_t r = 0; r < rows; r += w8a8::launch_rows(THREADS)) {
    const int n = (int)(rows - r < w8a8::launch_rows(THREADS) ? rows - r : w8a8::launch_rows(THREADS));
    const dim3 grid((n + kRows - 1) / kRows);
    if (vec)
      hipLaunchKernelGGL((quantize_kernel<T, THREADS, CH, true>), grid, dim3(kBlock), 0, st, X + r * ldx, ldx, n, K, Kp,
                         Xq + r * Kp, sx + r);
    else
      hipLaunchKernelGGL((quantize_kernel<T, THREADS, CH, false>), grid, dim3(kBlock), 0, st, X + r * ldx, ldx, n, K, Kp,
                         Xq + r * Kp, sx + r);
  }
}

template <class T>
void dispatch(const uint16_t* X, int64_t ldx, int rows, int K, int8_t* Xq, float* sx, hipStream_t st) {
  const int Kp = (K + 127) / 128 * 128;
  const bool vec = K % 8 == 0 && (rows == 1 || ldx % 8 == 0) && (reinterpret_cast<uintptr_t>(X) & 15) == 0;
  const w8a8::RowShape s = w8a8::row_shape(rows, Kp);
  if (s.threads == 64 && s.chunks == 1) launch<T, 64, 1>(X, ldx, vec, rows, K, Kp, Xq, sx, st);
  else if (s.threads == 64) launch<T, 64, 4>(X, ldx, vec, rows, K, Kp, Xq, sx, st);
  else if (s.threads == 256 && s.chunks == 1) launch<T, 256, 1>(X, ldx, vec, rows, K, Kp, Xq, sx, st);
  else if (s.threads == 256 && s.chunks == 2) launch<T, 256, 2>(X, ldx, vec, rows, K, Kp, Xq, sx, st);
  else if (s.threads == 256) launch<T, 256, 4>(X, ldx, vec, rows, K, Kp, Xq, sx, st);
  else if (s.threads == 512 && s.chunks == 2) launch<T, 512, 2>(X, ldx, vec, rows, K, Kp, Xq, sx, st);
  else if (s.threads == 512) launch<T, 512, 4>(X, ldx, vec, rows, K, Kp, Xq, sx, st);
  else launch<T, 1024, 8>(X, ldx, vec, rows, K, Kp, Xq, sx, st);
}

}  // namespace

hipError_t launch_quantize_w8a8(const uint16_t* X, int64_t ldx, bool bf16, int rows, int K, int8_t* Xq, float* sx,
                                hipStream_t stream) {
  if (bf16)
    dispatch<Bf16>(X, ldx, rows, K, Xq, sx, stream);
  else
    dispatch<Fp16>(X, ldx, rows, K, Xq, sx, stream);
  return hipGetLastError();
}

}  // namespace atom
