// Writing and reading the 4-bit KV cache on gfx950 (layout and quantizer: atom_kv4.h).
//
// Both kernels are bound by HBM (a row of D channels: 2 D bytes on one side, D/2 + 4 on the other).  A
// row is one lane per 8 channels: the append joins its extremes over D/8 lanes, so the codes are
// made from the registers that the one 16-byte load filled.  Keys leave as 4 bytes a lane, values as two
// 2-byte pieces 8 bytes apart (four tokens interleaved, the order that attention's matrix operands read).
#include "kv4_layout.h"
#include "serve_internal.h"

namespace atom {
namespace {

constexpr int kThreads = 256;

struct Pool {
  uint8_t *k, *v;
  uint32_t *k_par, *v_par;      // zero point in the low half, scale in the high half
  int pages, log_page, heads;
};

Pool pool_of(const atom_kv4_cache& c) {
  return Pool{(uint8_t*)c.k, (uint8_t*)c.v, (uint32_t*)c.k_par, (uint32_t*)c.v_par, c.pages, __builtin_ctz(c.page),
              c.heads};
}

// Joins the minimum and maximum of the LANES lanes that share a row.
template <int LANES>
__device__ __forceinline__ void extremes(float& lo, float& hi) {
#pragma unroll
  for (int d = LANES / 2; d; d >>= 1) {
    lo = __builtin_fminf(lo, __shfl_xor(lo, d));
    hi = __builtin_fmaxf(hi, __shfl_xor(hi, d));
  }
}

// One row per D / 8 lanes; blockIdx.y: 0 keys, 1 values.
template <class T, int D>
__global__ __launch_bounds__(kThreads) void append_kernel(const uint16_t* __restrict__ K, int64_t k_stride,
                                                          const uint16_t* __restrict__ V, int64_t v_stride,
                                                          const int64_t* __restrict__ slots, int64_t rows, Pool c) {
  constexpr int kLanes = D / 8;
  const int64_t row = (int64_t)blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes;
  if (row >= rows) return;                             // whole groups of lanes leave together
  const int lane = threadIdx.x % kLanes;
  const bool values = blockIdx.y != 0;
  const int64_t token = row / c.heads;
  const int head = (int)(row - token * c.heads);
  const int64_t slot = slots[token];
  if (!kv4::valid_slot(slot, c.pages, c.log_page)) return;
  const uint16_t* src = (values ? V + token * v_stride : K + token * k_stride) + (int64_t)head * D + 8 * lane;
  const u32x4 w = *reinterpret_cast<const u32x4*>(src);
  float x[8], lo = 0.0f, hi = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[i] = elem<T>(w[i / 2], i & 1);
    lo = __builtin_fminf(lo, x[i]);
    hi = __builtin_fmaxf(hi, x[i]);
  }
  extremes<kLanes>(lo, hi);
  const float s = (float)(_Float16)__builtin_fminf((hi - lo) / 15.0f, 65504.0f);
  const bool some = s > 0.0f;
  const float r = some ? 1.0f / s : 0.0f;
  const float zero = some && lo < 0.0f ? __builtin_fminf(__builtin_rintf(-lo / s), 15.0f) : 0.0f;   // never -0
  uint32_t q = 0;                                      // nibble i: the code of channel i
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float u = __builtin_rintf(quotient(x[i], s, r)) + zero;
    q |= (uint32_t)(int)__builtin_fminf(__builtin_fmaxf(u, 0.0f), 15.0f) << (4 * i);
  }
  const int64_t page = slot >> c.log_page;
  const int t = (int)(slot & ((1 << c.log_page) - 1));
  const int64_t at = kv4::row_index(page, head, c.heads, c.log_page, t);
  if (!values) {
    *reinterpret_cast<uint32_t*>(c.k + at * (D / 2) + 4 * lane) = q;
  } else {
    uint8_t* b = c.v + kv4::value_block(page, head, c.heads, c.log_page, D, t >> 2);
    *reinterpret_cast<uint16_t*>(b + kv4::value_in_block(2 * lane, t & 3)) = (uint16_t)q;
    *reinterpret_cast<uint16_t*>(b + kv4::value_in_block(2 * lane + 1, t & 3)) = (uint16_t)(q >> 16);
  }
  if (lane == 0) (values ? c.v_par : c.k_par)[at] = pack2<Fp16>(zero, s);
}

template <class T, int D>
__global__ __launch_bounds__(kThreads) void read_kernel(Pool c, const int64_t* __restrict__ slots, int64_t rows,
                                                        uint16_t* __restrict__ K, uint16_t* __restrict__ V) {
  constexpr int kLanes = D / 8;
  const int64_t row = (int64_t)blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes;
  if (row >= rows) return;
  const int lane = threadIdx.x % kLanes;
  const bool values = blockIdx.y != 0;
  const int64_t token = row / c.heads;
  const int head = (int)(row - token * c.heads);
  const int64_t slot = slots[token];
  uint16_t* dst = (values ? V : K) + row * D + 8 * lane;
  if (!kv4::valid_slot(slot, c.pages, c.log_page)) {
    *reinterpret_cast<u32x4*>(dst) = u32x4{0, 0, 0, 0};
    return;
  }
  const int64_t page = slot >> c.log_page;
  const int t = (int)(slot & ((1 << c.log_page) - 1));
  const int64_t at = kv4::row_index(page, head, c.heads, c.log_page, t);
  uint32_t q;
  if (!values) {
    q = *reinterpret_cast<const uint32_t*>(c.k + at * (D / 2) + 4 * lane);
  } else {
    const uint8_t* b = c.v + kv4::value_block(page, head, c.heads, c.log_page, D, t >> 2);
    q = *reinterpret_cast<const uint16_t*>(b + kv4::value_in_block(2 * lane, t & 3)) |
        (uint32_t)*reinterpret_cast<const uint16_t*>(b + kv4::value_in_block(2 * lane + 1, t & 3)) << 16;
  }
  const uint32_t par = (values ? c.v_par : c.k_par)[at];
  const float zero = elem<Fp16>(par, 0), s = elem<Fp16>(par, 1);
  u32x4 o;
#pragma unroll
  for (int i = 0; i < 4; ++i) {     // an integer below 16 times 11 bits: exact until the one rounding
    const float a = ((float)((q >> (8 * i)) & 15) - zero) * s, b = ((float)((q >> (8 * i + 4)) & 15) - zero) * s;
    o[i] = pack2<T>(a, b);
  }
  *reinterpret_cast<u32x4*>(dst) = o;
}

template <class T, int D>
void append(const uint16_t* K, int64_t ks, const uint16_t* V, int64_t vs, const int64_t* slots, int64_t rows,
            const Pool& p, hipStream_t st) {
  constexpr int kRows = kThreads / (D / 8);
  hipLaunchKernelGGL((append_kernel<T, D>), dim3((unsigned)((rows + kRows - 1) / kRows), 2), dim3(kThreads), 0, st, K,
                     ks, V, vs, slots, rows, p);
}
template <class T, int D>
void read(const Pool& p, const int64_t* slots, int64_t rows, uint16_t* K, uint16_t* V, hipStream_t st) {
  constexpr int kRows = kThreads / (D / 8);
  hipLaunchKernelGGL((read_kernel<T, D>), dim3((unsigned)((rows + kRows - 1) / kRows), 2), dim3(kThreads), 0, st, p,
                     slots, rows, K, V);
}

}  // namespace

hipError_t launch_kv4_append(const uint16_t* K, int64_t ks, const uint16_t* V, int64_t vs, const int64_t* slots,
                             int tokens, bool bf16, const atom_kv4_cache& c, hipStream_t st) {
  const Pool p = pool_of(c);
  const int64_t rows = (int64_t)tokens * c.heads;
  if (bf16) {
    if (c.dim == 64) append<Bf16, 64>(K, ks, V, vs, slots, rows, p, st);
    else if (c.dim == 128) append<Bf16, 128>(K, ks, V, vs, slots, rows, p, st);
    else append<Bf16, 256>(K, ks, V, vs, slots, rows, p, st);
  } else {
    if (c.dim == 64) append<Fp16, 64>(K, ks, V, vs, slots, rows, p, st);
    else if (c.dim == 128) append<Fp16, 128>(K, ks, V, vs, slots, rows, p, st);
    else append<Fp16, 256>(K, ks, V, vs, slots, rows, p, st);
  }
  return hipGetLastError();
}

hipError_t launch_kv4_read(const atom_kv4_cache& c, const int64_t* slots, int tokens, bool bf16, uint16_t* K,
                           uint16_t* V, hipStream_t st) {
  const Pool p = pool_of(c);
  const int64_t rows = (int64_t)tokens * c.heads;
  if (bf16) {
    if (c.dim == 64) read<Bf16, 64>(p, slots, rows, K, V, st);
    else if (c.dim == 128) read<Bf16, 128>(p, slots, rows, K, V, st);
    else read<Bf16, 256>(p, slots, rows, K, V, st);
  } else {
    if (c.dim == 64) read<Fp16, 64>(p, slots, rows, K, V, st);
    else if (c.dim == 128) read<Fp16, 128>(p, slots, rows, K, V, st);
    else read<Fp16, 256>(p, slots, rows, K, V, st);
  }
  return hipGetLastError();
}

}  // namespace atom
