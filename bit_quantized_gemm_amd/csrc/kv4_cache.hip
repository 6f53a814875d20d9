// Writing and reading the 4-bit KV cache on gfx950 (layout and quantizer: atom_kv4.h).
//
// Both kernels are bound by HBM (a row of D channels: 2 D bytes on one side, D/2 + 4 on the other).  A row is one
// lane per 8 channels: the append joins its extremes over D/8 lanes, so the codes are made from the registers that the
// one 16-byte load filled.  Keys leave as 4 bytes a lane, values as two 2-byte pieces 8 bytes apart (four tokens
// interleaved, the order that attention's matrix operands read).
//
// A workgroup takes consecutive tokens of one head, 2048 / D at a time: the pieces of a line that neighbouring tokens
// share then meet in one L2 (rows dealt out head by head put them into different XCDs' caches), and no thread divides an
// index.  8192 tokens x 32 heads x 128: 45 us to append, 35 us to read (169 MB each: 3.8 and 4.8 TB/s; a copy reaches 5.1).  With
// two divides of 64-bit indices a row, IEEE divides for the quotients and rows dealt head by head it took 60 and 38 us.
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

template <int C>
struct Ctrl {
  static constexpr int value = C;
};
// max over the LANES lanes (a power of two, 8 to 32) that share a row.
template <int LANES>
__device__ __forceinline__ float row_max(float x) {
  auto step = [](float v, auto ctrl) {
    return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), decltype(ctrl)::value, 0xF, 0xF, false));
  };
  x = __builtin_fmaxf(x, step(x, Ctrl<0xB1>{}));       // lane ^ 1
  x = __builtin_fmaxf(x, step(x, Ctrl<0x4E>{}));       // lane ^ 2
  x = __builtin_fmaxf(x, step(x, Ctrl<0x141>{}));      // 7 - lane in each 8
  if (LANES >= 16) x = __builtin_fmaxf(x, step(x, Ctrl<0x140>{}));   // 15 - lane in each 16
  if (LANES >= 32) x = __builtin_fmaxf(x, __shfl_xor(x, 16));
  return x;
}

// Adding 1.5 * 2^23 rounds to an integer (ties to even) and leaves it in the low bits; far larger values keep their
// order as integers, so a clamp of the bits clamps the value.
constexpr float kRound = 12582912.0f;
constexpr int kRoundBits = 0x4B400000;

// blockIdx.x: `span` tokens, blockIdx.y: head, blockIdx.z: 0 keys, 1 values.
template <class T, int D>
__global__ __launch_bounds__(kThreads) void append_kernel(const uint16_t* __restrict__ K, int64_t k_stride,
                                                          const uint16_t* __restrict__ V, int64_t v_stride,
                                                          const int64_t* __restrict__ slots, int tokens, int span, Pool c) {
  constexpr int kLanes = D / 8, kRows = kThreads / kLanes;
  const int lane = threadIdx.x % kLanes, head = blockIdx.y;
  const bool values = blockIdx.z != 0;
  const int first = blockIdx.x * span, last = min(first + span, tokens);
  const int64_t stride = values ? v_stride : k_stride;
  const uint16_t* src = (values ? V : K) + (int64_t)head * D + 8 * lane;
  for (int token = first + threadIdx.x / kLanes; token < last; token += kRows) {   // whole groups of lanes leave together
    const int64_t slot = slots[token];
    const u32x4 w = *reinterpret_cast<const u32x4*>(src + token * stride);
    float x[8], lo = 0.0f, hi = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i] = elem<T>(w[i / 2], i & 1);
      lo = __builtin_fmaxf(lo, -x[i]);
      hi = __builtin_fmaxf(hi, x[i]);
    }
    lo = row_max<kLanes>(lo);                            // -min(x, 0)
    hi = row_max<kLanes>(hi);
    // fl32((hi - lo) / 15): two corrected steps, as in quotient(); an infinite range ends in the largest scale
    const float range = hi + lo, r15 = 1.0f / 15.0f, d0 = range * r15;
    const float d1 = __builtin_fmaf(__builtin_fmaf(-d0, 15.0f, range), r15, d0);
    const float d2 = __builtin_fmaf(__builtin_fmaf(-d1, 15.0f, range), r15, d1);
    const float s = (float)(_Float16)__builtin_fminf(d2, 65504.0f);
    // the correctly rounded reciprocal of a positive fp16 value: the hardware's, refined once
    const float r0 = __builtin_amdgcn_rcpf(s);
    const float r = s > 0.0f ? __builtin_fmaf(__builtin_fmaf(-s, r0, 1.0f), r0, r0) : 0.0f;
    const float zero = s > 0.0f ? __builtin_fminf(__builtin_rintf(quotient(lo, s, r)), 15.0f) : 0.0f;
    const int least = kRoundBits - (int)zero;            // code 0
    uint32_t q = 0;                                      // nibble i: the code of channel i, `least` too large
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int bits = __builtin_bit_cast(int, quotient(x[i], s, r) + kRound);
      q += (uint32_t)min(max(bits, least), least + 15) << (4 * i);
    }
    q -= (uint32_t)least * 0x11111111u;
    if (!kv4::valid_slot(slot, c.pages, c.log_page)) continue;
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
}

template <class T, int D>
__global__ __launch_bounds__(kThreads) void read_kernel(Pool c, const int64_t* __restrict__ slots, int tokens, int span,
                                                        uint16_t* __restrict__ K, uint16_t* __restrict__ V) {
  constexpr int kLanes = D / 8, kRows = kThreads / kLanes;
  const int lane = threadIdx.x % kLanes, head = blockIdx.y;
  const bool values = blockIdx.z != 0;
  const int first = blockIdx.x * span, last = min(first + span, tokens);
  for (int token = first + threadIdx.x / kLanes; token < last; token += kRows) {
    const int64_t slot = slots[token];
    uint16_t* dst = (values ? V : K) + ((int64_t)token * c.heads + head) * D + 8 * lane;
    if (!kv4::valid_slot(slot, c.pages, c.log_page)) {
      *reinterpret_cast<u32x4*>(dst) = u32x4{0, 0, 0, 0};
      continue;
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
}

// Tokens of a workgroup: one pass of its threads when the grid is small, four when it fills the GPU anyway.
template <int D>
int span_of(int tokens, int heads) {
  constexpr int kRows = kThreads / (D / 8);
  return (int64_t)tokens * heads >= (int64_t)kRows * 4096 ? 4 * kRows : kRows;
}
template <class T, int D>
void append(const uint16_t* K, int64_t ks, const uint16_t* V, int64_t vs, const int64_t* slots, int tokens,
            const Pool& p, hipStream_t st) {
  const int span = span_of<D>(tokens, p.heads);
  hipLaunchKernelGGL((append_kernel<T, D>), dim3((unsigned)((tokens + span - 1) / span), p.heads, 2), dim3(kThreads), 0, st,
                     K, ks, V, vs, slots, tokens, span, p);
}
template <class T, int D>
void read(const Pool& p, const int64_t* slots, int tokens, uint16_t* K, uint16_t* V, hipStream_t st) {
  const int span = span_of<D>(tokens, p.heads);
  hipLaunchKernelGGL((read_kernel<T, D>), dim3((unsigned)((tokens + span - 1) / span), p.heads, 2), dim3(kThreads), 0, st, p,
                     slots, tokens, span, K, V);
}

}  // namespace

hipError_t launch_kv4_append(const uint16_t* K, int64_t ks, const uint16_t* V, int64_t vs, const int64_t* slots,
                             int tokens, bool bf16, const atom_kv4_cache& c, hipStream_t st) {
  const Pool p = pool_of(c);
  if (bf16) {
    if (c.dim == 64) append<Bf16, 64>(K, ks, V, vs, slots, tokens, p, st);
    else if (c.dim == 128) append<Bf16, 128>(K, ks, V, vs, slots, tokens, p, st);
    else append<Bf16, 256>(K, ks, V, vs, slots, tokens, p, st);
  } else {
    if (c.dim == 64) append<Fp16, 64>(K, ks, V, vs, slots, tokens, p, st);
    else if (c.dim == 128) append<Fp16, 128>(K, ks, V, vs, slots, tokens, p, st);
    else append<Fp16, 256>(K, ks, V, vs, slots, tokens, p, st);
  }
  return hipGetLastError();
}

hipError_t launch_kv4_read(const atom_kv4_cache& c, const int64_t* slots, int tokens, bool bf16, uint16_t* K,
                           uint16_t* V, hipStream_t st) {
  const Pool p = pool_of(c);
  if (bf16) {
    if (c.dim == 64) read<Bf16, 64>(p, slots, tokens, K, V, st);
    else if (c.dim == 128) read<Bf16, 128>(p, slots, tokens, K, V, st);
    else read<Bf16, 256>(p, slots, tokens, K, V, st);
  } else {
    if (c.dim == 64) read<Fp16, 64>(p, slots, tokens, K, V, st);
    else if (c.dim == 128) read<Fp16, 128>(p, slots, tokens, K, V, st);
    else read<Fp16, 256>(p, slots, tokens, K, V, st);
  }
  return hipGetLastError();
}

}  // namespace atom
