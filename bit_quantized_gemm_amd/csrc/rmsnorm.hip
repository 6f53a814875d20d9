// Root-mean-square norm with the residual's addition in front and the quantized layers' row formats behind it, for gfx950
// (formulas: atom_norm.h).
//
// What bounds it: HBM.  A row is read once (twice its bytes with a residual, and once out again), kept in registers by
// the threads that share it, and leaves as codes.  With a residual, graph replays over rows from HBM: 8192 x 8192 to int8 84.7 us, to
// MXFP4 81.3 us (5.6 and 5.4 TB/s; a copy of memory reaches 5.1; 96 us where calls lie apart), 2048 x 11008 30.1 and 31.7 us (34 and 35
// over 800 MB of outputs too), 16 x 4096 3.1 and 3.2 us, of which the launch is more than half.
//
// Exact codes.  p = h * w is exact in fp32 (two 8- or 11-bit significands), so y = p / root, root = sqrt(mean + eps), is one
// row's number away from exact: the sum of squares and the root are fp64, and each code is made from p times one factor in
// fp32.  Its error is two roundings (three for int8) of 2^-24, so only values that close to the border of two codes can come out
// wrong: they are seen by their distance to it, and the wave makes that chunk's codes again in fp64.  A factor puts a value that
// lies on a border (a row of +-3 has whole halves) a step of 2^-53 beside it: what even fp64 leaves that near is made by the
// formula's own divisions, behind everything else.  (A norm rounded to 32 bits gives other codes for one value in about 2^16,
// and for a block's exponent the whole block's.)
#include "mxfp4_row.h"
#include "norm_steps.h"
#include "w8a8_rows.h"

namespace atom {
namespace {

using rms::divided;

struct Norm {
  const uint16_t *X, *R, *W;
  int64_t ldx, ldr, ldh;
  double eps, inv_k;
  int first, end, rows, K;      // rows of this launch, and of the whole matrix
  uint16_t* H;
  uint8_t* Xq;
  void* sx;
};

// v of the lane that CTRL names, within rows of 16 lanes.
template <int CTRL>
__device__ __forceinline__ double moved(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  return __builtin_bit_cast(double, (uint64_t)mx::dpp<CTRL>((uint32_t)(b >> 32)) << 32 | mx::dpp<CTRL>((uint32_t)b));
}
// Sum and maximum over a wave, in every lane: lane ^ 1, ^ 2, 7 - lane of 8, 15 - lane of 16, then across rows.
__device__ __forceinline__ double wave_sum(double v) {
  v += moved<0xB1>(v);
  v += moved<0x4E>(v);
  v += moved<0x141>(v);
  v += moved<0x140>(v);
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}
__device__ __forceinline__ float wave_top(float v) {
  uint32_t b = __builtin_bit_cast(uint32_t, v);          // not negative: the order of the bits
  b = max(b, mx::dpp<0xB1>(b));
  b = max(b, mx::dpp<0x4E>(b));
  b = max(b, mx::dpp<0x141>(b));
  b = max(b, mx::dpp<0x140>(b));
  b = max(b, (uint32_t)__shfl_xor((int)b, 16));
  return __builtin_bit_cast(float, max(b, (uint32_t)__shfl_xor((int)b, 32)));
}

// Code of one magnitude in fp64 units of its scale: nearest, ties to the even code, saturating.
__device__ __forceinline__ uint32_t fp4_code(double a) {
  return (a > 0.25) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0);
}
// Whether a number is within eight units in the last place of one with `zeros` zeros at the end of its significand.
__device__ __forceinline__ bool beside(double a, int zeros) {
  return ((__builtin_bit_cast(uint64_t, a) + 8) & (((uint64_t)1 << zeros) - 1)) < 16;
}

// The scale of a block whose largest |y| this is: its byte, and 1 / scale.
struct Block {
  uint32_t byte;
  double unit;
  __device__ __forceinline__ explicit Block(double y) {
    const int e = (int)(__builtin_bit_cast(uint64_t, y) >> 52);
    byte = e == 2047 ? mx::kNanScale : (uint32_t)min(max(e - 1023 - 2 + 127, 0), 252);
    unit = __builtin_bit_cast(double, (uint64_t)(1023 + 127 - (int)byte) << 52);
  }
};

// The wave's chunks of `which` again, by the formula's own steps.  Rare, and so behind everything else: a loop over h and w as they
// are in memory, which leaves the common way its registers and its code (inside it, 4096 x 4097 to int8 takes 32.0 us, 29.4 so).
template <class T, int THREADS, bool VEC, bool MX>
__device__ __forceinline__ void again(const Norm& a, int row, int t, uint32_t which, float top, double root, double rstd) {
  const uint16_t* from = a.R ? a.H + (size_t)row * a.ldh : a.X + (size_t)row * a.ldx;
  const int lane = threadIdx.x & 63;
#pragma unroll 1
  for (; which; which &= which - 1) {
    const int c = t + __builtin_ctz(which) * THREADS;
    const u32x4 h = w8a8::load8<VEC>(from, c, a.K), w = w8a8::load8<VEC>(a.W, c, a.K);
    float p[8];
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      p[j] = elem<T>(h[j / 2], j & 1) * elem<T>(w[j / 2], j & 1);
      m = max(m, __builtin_bit_cast(uint32_t, p[j]) & 0x7FFFFFFFu);
    }
    if constexpr (!MX) {
      const int Kp = (a.K + 127) / 128 * 128;
      const float s = (float)divided(divided((double)top, root, rstd), 127.0, 1.0 / 127.0);
      const double per = s > 0.0f ? 1.0 / (double)s : 0.0;
      u32x2 o = {0, 0};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const double u = divided(divided((double)p[j], root, rstd), (double)s, per);
        o[j / 4] |= ((uint32_t)(int)__builtin_fmin(__builtin_fmax(__builtin_rint(u), -127.0), 127.0) & 0xFFu) << (8 * (j & 3));
      }
      if (8 * c < Kp) *reinterpret_cast<u32x2*>(a.Xq + (size_t)row * Kp + 8 * c) = o;
    } else {
      const int Kp = mx::padded(a.K);
      const Block k(divided((double)__builtin_bit_cast(float, mx::block_max(m)), root, rstd));
      uint32_t code = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        code |= (fp4_code(divided((double)__builtin_fabsf(p[j]), root, rstd) * k.unit) | __builtin_bit_cast(uint32_t, p[j]) >> 31 << 3)
                << (4 * j);
      if (k.byte == mx::kNanScale) code = 0;
      const uint32_t four = mx::gather_scales(k.byte, lane);
      if (8 * c < Kp) {
        *reinterpret_cast<uint32_t*>(a.Xq + (size_t)row * (Kp / 2) + 4 * c) = code;
        if ((lane & 15) == 0)
          *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(a.sx) + ((int64_t)(c >> 5) * a.rows + row) * 8 + ((c >> 4) & 1) * 4) = four;
      }
    }
  }
}

template <class T, int THREADS, int CH, bool VEC, bool MX>
__global__ __launch_bounds__(w8a8::block_threads(THREADS)) void norm_kernel(Norm a) {
  constexpr int kBlock = w8a8::block_threads(THREADS);
  constexpr int kRows = kBlock / THREADS;               // rows of one workgroup
  const int t = threadIdx.x % THREADS, lane = threadIdx.x & 63;
  const int row = a.first + blockIdx.x * kRows + threadIdx.x / THREADS;
  if (kRows > 1 && row >= a.end) return;                // whole waves: no barrier follows
  const uint16_t* x = a.X + (size_t)row * a.ldx;

  u32x4 h[CH], w[CH];                                   // chunk c = t + i * THREADS: elements 8 c .. 8 c + 7
#pragma unroll
  for (int i = 0; i < CH; ++i) h[i] = w8a8::load8<VEC>(x, t + i * THREADS, a.K);
  if (a.R) {
    const uint16_t* from = a.R + (size_t)row * a.ldr;
    uint16_t* dst = a.H + (size_t)row * a.ldh;
    u32x4 r[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) r[i] = w8a8::load8<VEC>(from, t + i * THREADS, a.K);
#pragma unroll
    for (int i = 0; i < CH; ++i) w[i] = w8a8::load8<VEC>(a.W, t + i * THREADS, a.K);
    __builtin_amdgcn_sched_barrier(0);                  // all loads are on their way before the first sum
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = t + i * THREADS;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float lo = elem<T>(h[i][j], 0) + elem<T>(r[i][j], 0), hi = elem<T>(h[i][j], 1) + elem<T>(r[i][j], 1);
        asm("" : "+v"(lo), "+v"(hi));                   // two roundings, as two steps have them: never one fused one
        h[i][j] = pack2<T>(lo, hi);
      }
      if (!VEC || 8 * c < a.K) mx::store8(dst + 8 * c, h[i], VEC ? 8 : a.K - 8 * c);
    }
  } else {
#pragma unroll
    for (int i = 0; i < CH; ++i) w[i] = w8a8::load8<VEC>(a.W, t + i * THREADS, a.K);
  }

  double sum[2] = {};
  float top = 0.0f;                                     // largest |p| (int8: the row's scale)
#pragma unroll
  for (int i = 0; i < CH; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float v = elem<T>(h[i][j / 2], j & 1);
      sum[j & 1] = __builtin_fma((double)v, (double)v, sum[j & 1]);
      if (!MX) top = __builtin_fmaxf(top, __builtin_fabsf(v * elem<T>(w[i][j / 2], j & 1)));
    }
  double total = wave_sum(sum[0] + sum[1]);
  if (!MX) top = wave_top(top);
  if constexpr (THREADS > 64) {
    __shared__ double sums[THREADS / 64];
    __shared__ float tops[THREADS / 64];
    if (lane == 0) {
      sums[threadIdx.x >> 6] = total;
      tops[threadIdx.x >> 6] = top;
    }
    __syncthreads();
    total = 0.0;
#pragma unroll
    for (int i = 0; i < THREADS / 64; ++i) {            // the same order in every wave
      total += sums[i];
      if (!MX) top = __builtin_fmaxf(top, tops[i]);
    }
  }
  const double root = __builtin_sqrt(divided(total, (double)a.K, a.inv_k) + a.eps), rstd = 1.0 / root;
  uint32_t undecided = 0;                               // the wave's chunks (bit i) with a value next to a border in 64 bits too

  if constexpr (!MX) {
    const int Kp = (a.K + 127) / 128 * 128;
    const float s = (float)divided(divided((double)top, root, rstd), 127.0, 1.0 / 127.0);
    if (t == 0) static_cast<float*>(a.sx)[row] = s;
    // y / s without the norm, which cancels but for s's own rounding: no code waits for the sum of squares
    const float f32 = 127.0f / top;
    // a factor beyond fp32, or a scale whose own rounding can carry a code past 127
    const bool extreme = !(f32 < 0x1p100f) || s < 0x1p-100f;
    uint8_t* q = a.Xq + (size_t)row * Kp;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = t + i * THREADS;
      uint32_t b[8];
      float far = 0.0f;                                 // largest distance to an integer
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float u = elem<T>(h[i][j / 2], j & 1) * elem<T>(w[i][j / 2], j & 1) * f32;
        const float k = u + 12582912.0f;                // 1.5 * 2^23: the integer (ties to even) in the low byte
        far = __builtin_fmaxf(far, __builtin_fabsf(u - (k - 12582912.0f)));
        b[j] = __builtin_bit_cast(uint32_t, k);
      }
      // three roundings (of the factor, of u and of s) of at most 127: u is within 381 x 2^-24 of the exact value, 2.27e-5
      if (__builtin_amdgcn_ballot_w64(extreme || far >= 0.5f - 0x1.9p-16f)) {
        const double f = divided(rstd, (double)s, (double)f32 * root);   // (from 2^-22 by two steps: 2^-52)
        double beside = 0.0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const double u = (double)(elem<T>(h[i][j / 2], j & 1) * elem<T>(w[i][j / 2], j & 1)) * f, k = __builtin_rint(u);
          beside = __builtin_fmax(beside, __builtin_fabs(u - k));
          b[j] = (uint32_t)(int)k;
        }
        if (__builtin_amdgcn_ballot_w64(extreme || beside >= 0.5 - 0x1p-40)) undecided |= 1u << i;
      }
      if (8 * c < Kp) {
        u32x2 o;
#pragma unroll
        for (int k = 0; k < 2; ++k)
          o[k] = __builtin_amdgcn_perm(b[4 * k + 1], b[4 * k], 0x0C0C0400u) |
                 __builtin_amdgcn_perm(b[4 * k + 3], b[4 * k + 2], 0x04000C0Cu);
        *reinterpret_cast<u32x2*>(q + 8 * c) = o;
      }
    }
  } else {
    const int Kp = mx::padded(a.K);
    uint8_t* q = a.Xq + (size_t)row * (Kp / 2);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = t + i * THREADS;
      float p[8];
      uint32_t m = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        p[j] = elem<T>(h[i][j / 2], j & 1) * elem<T>(w[i][j / 2], j & 1);
        m = max(m, __builtin_bit_cast(uint32_t, p[j]) & 0x7FFFFFFFu);
      }
      m = mx::block_max(m);
      const double y = (double)__builtin_bit_cast(float, m) * rstd;
      const Block k(y);
      const double f = rstd * k.unit;
      const float f32 = m ? (float)f : 0.0f;            // a block of zeros, as behind K: any factor
      float u[8];
      uint32_t near = 8;                                // distance to a border, in units of the last place
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        u[j] = p[j] * f32;
        // within 2 units in the last place of the exact value; all borders (0.25, 0.75, 1.25, ... 5) have 21 zeros at the
        // end of their significands
        near = min(near, (__builtin_bit_cast(uint32_t, u[j]) + 4) & 0x1FFFFFu);
      }
      uint32_t code = mx::codes8(u);
      // (the last: a factor beyond fp32)
      if (__builtin_amdgcn_ballot_w64(near < 8 || !(f32 < 0x1p100f))) {
        near = 8;                                       // (zeros come as far as here: sums that cancel are one in 10^4 of fp16 rows)
#pragma unroll
        for (int j = 0; j < 8; ++j) near = min(near, rms::border_distance(__builtin_bit_cast(uint32_t, u[j])));
        if (__builtin_amdgcn_ballot_w64(near < 8 || !(f32 < 0x1p100f))) {
          bool tie = m != 0 && beside(y, 52);           // the exponent's: a power of two is 4 or 8 of the scale, a border here too
          code = 0;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const double v = __builtin_fabs((double)p[j] * f);
            tie |= v >= 0.125 && beside(v, 50);
            code |= (fp4_code(v) | __builtin_bit_cast(uint32_t, p[j]) >> 31 << 3) << (4 * j);
          }
          if (__builtin_amdgcn_ballot_w64(tie)) undecided |= 1u << i;
        }
      }
      if (k.byte == mx::kNanScale) code = 0;
      const uint32_t four = mx::gather_scales(k.byte, lane);
      if (8 * c < Kp) {
        *reinterpret_cast<uint32_t*>(q + 4 * c) = code;
        if ((lane & 15) == 0)
          *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(a.sx) + ((int64_t)(c >> 5) * a.rows + row) * 8 +
                                       ((c >> 4) & 1) * 4) = four;
      }
    }
  }
  if (undecided) again<T, THREADS, VEC, MX>(a, row, t, undecided, top, root, rstd);
}

template <class T, bool MX, int THREADS, int CH>
void launch(const Norm& a, bool vec, hipStream_t st) {
  constexpr int kBlock = w8a8::block_threads(THREADS), kRows = kBlock / THREADS;
  const dim3 grid((a.end - a.first + kRows - 1) / kRows);
  if (vec)
    hipLaunchKernelGGL((norm_kernel<T, THREADS, CH, true, MX>), grid, dim3(kBlock), 0, st, a);
  else
    hipLaunchKernelGGL((norm_kernel<T, THREADS, CH, false, MX>), grid, dim3(kBlock), 0, st, a);
}

template <class T, bool MX>
void dispatch(const Norm& a, hipStream_t st) {
  const int Kp = MX ? mx::padded(a.K) : (a.K + 127) / 128 * 128;
  auto wide = [&](const void* p, int64_t ld) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (a.rows == 1 || ld % 8 == 0); };
  const bool vec = a.K % 8 == 0 && wide(a.X, a.ldx) && wide(a.W, 0) && (!a.R || (wide(a.R, a.ldr) && wide(a.H, a.ldh)));
  const w8a8::RowShape s = w8a8::row_shape(a.rows, Kp);
  if (s.threads == 64 && s.chunks == 1) launch<T, MX, 64, 1>(a, vec, st);
  else if (s.threads == 64) launch<T, MX, 64, 4>(a, vec, st);
  else if (s.threads == 256 && s.chunks == 1) launch<T, MX, 256, 1>(a, vec, st);
  else if (s.threads == 256 && s.chunks == 2) launch<T, MX, 256, 2>(a, vec, st);
  else if (s.threads == 256) launch<T, MX, 256, 4>(a, vec, st);
  else if (s.threads == 512 && s.chunks == 2) launch<T, MX, 512, 2>(a, vec, st);
  else if (s.threads == 512) launch<T, MX, 512, 4>(a, vec, st);
  else launch<T, MX, 1024, 8>(a, vec, st);
}

// What int8 rows stand for: one thread per eight elements.
template <class T, bool VEC>
__global__ __launch_bounds__(256) void dequantize_kernel(const int8_t* __restrict__ Xq, const float* __restrict__ sx, int rows,
                                                         int K, int Kp, uint16_t* __restrict__ X) {
  const int c = blockIdx.y * 64 + (threadIdx.x & 63), row = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (row >= rows || 8 * c >= K) return;
  const u32x2 q = *reinterpret_cast<const u32x2*>(Xq + (size_t)row * Kp + 8 * c);
  const float s = sx[row];
  float v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    v[j] = (float)(int8_t)(q[j / 4] >> (8 * (j & 3))) * s;
    asm("" : "+v"(v[j]));
  }
  mx::store8(X + (size_t)row * K + 8 * c, u32x4{pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]), pack2<T>(v[4], v[5]), pack2<T>(v[6], v[7])},
             VEC ? 8 : K - 8 * c);
}

}  // namespace

hipError_t launch_rmsnorm(const NormCall& n, bool mx, hipStream_t stream) {
  const w8a8::RowShape s = w8a8::row_shape(n.rows, mx ? mx::padded(n.K) : (n.K + 127) / 128 * 128);
  const int64_t most = w8a8::launch_rows(s.threads);    // rows of one launch, which has less than 2^32 threads
  for (int64_t r = 0; r < n.rows; r += most) {
    const Norm a = {n.X, n.R, n.W, n.ldx, n.ldr, n.ldh, n.eps, 1.0 / n.K, (int)r, (int)(n.rows - r < most ? n.rows : r + most),
                    n.rows, n.K, n.H, n.Xq, n.sx};
    if (n.bf16)
      mx ? dispatch<Bf16, true>(a, stream) : dispatch<Bf16, false>(a, stream);
    else
      mx ? dispatch<Fp16, true>(a, stream) : dispatch<Fp16, false>(a, stream);
  }
  return hipGetLastError();
}

hipError_t launch_dequantize_w8a8(const int8_t* Xq, const float* sx, int rows, int K, bool bf16, uint16_t* X,
                                  hipStream_t stream) {
  const int Kp = (K + 127) / 128 * 128;
  const dim3 grid((rows + 3) / 4, (K + 511) / 512);
  auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, dim3(256), 0, stream, Xq, sx, rows, K, Kp, X); };
  if (bf16) K % 8 == 0 ? go(dequantize_kernel<Bf16, true>) : go(dequantize_kernel<Bf16, false>);
  else K % 8 == 0 ? go(dequantize_kernel<Fp16, true>) : go(dequantize_kernel<Fp16, false>);
  return hipGetLastError();
}

}  // namespace atom
