// Causal attention over the 4-bit KV cache for gfx950 (layout: atom_kv4.h).
//
// With codes k, v, zero points a, b and scales s, u of a token,
//   score = c * s * (sum_d q_d k_d - a * sum_d q_d),      c = scale * log2(e)
//   out_d = sum_t w_t (v_td - b_t) / sum_t p_t,           p = 2^(score - max), w = p * u,
// so the matrix cores multiply the codes themselves and the scales meet one score or one weight a
// token.  A code goes into the fp16 operand as the bits it has: a half-precision number whose low eleven bits are b is b 2^-24
// exactly (below 2^-14 a subnormal, which the gfx950 matrix cores keep).  Shifted by three, a half-word's nibbles stand there as 8 q and
// 128 q: unpacking eight codes is two shifts and four ands, and the factor 16 of every other nibble is taken out of the query (keys) or the
// result (values), exactly.  The place matters: the matrix cores line up the products of a sum by their operands' exponent
// fields, which for every subnormal is that of 2^-14, and drop what lies some 2^-24 below the largest.  With q and 16 q (one shift less)
// sums of 32 products were off by up to 2^-11.5 codes of the largest factor, always downwards; with 8 q it is 2^-14.5, with
// prompt_kernel's normal numbers 2^-18.  (Error against 64 bits of 16 x 2048 tokens, fp16, queries 64 times as large: 2.09e-4 of the norm
// with q, 1.87e-4 with 8 q or all 128 q, 1.86e-4 in 32 bits; all 128 q, four shifts, takes 3% more time.)
//
// Both products have the tokens (keys) or channels (values) as rows and the queries as columns: a
// lane's scores belong to one query, and as the contraction over tokens may run in any order, the
// weights feed the second product from the registers the first one left them in.  The values'
// four-token blocks in the cache are the operand order of that product.
//
// Ranges.  The queries are scaled by a power of two so that the largest element lies in [2^13, 2^14): of a row, or in prompt_kernel
// of a workgroup's rows while the rows' own largest elements are within 2^12 of each other.  fp16 then holds fp16 and bf16 queries exactly down to 2^-24 of that element.  The
// weights w are rounded to fp16: 2^-11 of each, as fp16's own rounding of the output.  Sums of w (v - b) and of p carry the same power
// of two, so it leaves the quotient; it is the row's own and follows the largest *weight* (score and value scale together): a token
// of large values and no weight costs the others nothing.  The zero points multiply the rounded weights too, so a
// rounding error acts on (v - b), not on v and b apart.  Scores, maxima and all sums are held in fp32.
//
// Reference: weights are 2^(score - ref) u with ref such that the largest of a row lies in [2^4, 2^15.1] from the row's first tile
// on: fp16 then holds whatever is above 2^-18 of it to 11 bits, and the rest to steps of 2^-28.  When some weight of
// a wave passes the limit (decode_kernel's twice the largest so far, prompt_kernel's 2^15), ref is raised so that the row's
// largest is 2^4 to 2^5 and the sums are rescaled, in a wave-uniform branch that random data take in the first tiles only.  ref counts
// tokens that the row sees, no others, and goes by their scales' exponents: the score that sets it is then a whole power of two and
// its weight, a fp16 number times that, not rounded at all.  (Error against 64 bits of a decode step over 2048 tokens of 128 channels,
// fp16: 2.7e-4 of the norm, 3.0e-4 with a reference that is not whole, 2.1e-4 with weights in 32 bits, the output's rounding alone;
// raised at every new largest weight it is no less and takes 3% more time.)
#include "atom_internal.h"
#include "kv4_layout.h"
#include "serve_internal.h"

namespace atom {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNegInf = -__builtin_inff();

struct Args {
  const uint16_t* q;
  int64_t q_stride;
  const uint8_t *k, *v;
  const uint32_t *k_par, *v_par;
  const int32_t *table, *lens, *q_start;
  int pages, log_page, heads, width, total_q, q_heads, group, batch, max_q, max_len;
  int row_tiles, chunks, chunk_tokens;
  float scale;
  uint16_t* out;
  float* part;          // [chunks][total_q * q_heads][D], then (M, l) pairs [chunks][total_q * q_heads][2]
};

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }   // 1 ulp; 2^-inf = 0
__device__ __forceinline__ float max3(float a, float b, float c) { return __builtin_fmaxf(__builtin_fmaxf(a, b), c); }

template <int B>
struct Half {
  static constexpr int value = B;
};

// A value that all lanes hold, in a scalar register.
__device__ __forceinline__ float uniform(float x) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(uint32_t, x)));
}

// max over lanes l, l ^ 32 and (kAll) l ^ 16 of a wave
template <bool kAll>
__device__ __forceinline__ float join_max(float x) {
  if (kAll) x = __builtin_fmaxf(x, __shfl_xor(x, 16));
  return __builtin_fmaxf(x, __shfl_xor(x, 32));
}
template <bool kAll>
__device__ __forceinline__ float join_sum(float x) {
  if (kAll) x += __shfl_xor(x, 16);
  return x + __shfl_xor(x, 32);
}

// Eight codes of a word -> fp16 operand, halves (n0, n4, 16 n1, 16 n5, n2, n6, 16 n3, 16 n7) * 2^-21.
constexpr int kCodeBits = 21;
__device__ __forceinline__ h8v unpack_keys(uint32_t w) {
  const uint32_t x = w << 3, y = w >> 5;
  const u32x4 o = {x & 0x00780078u, x & 0x07800780u, y & 0x00780078u, y & 0x07800780u};
  return __builtin_bit_cast(h8v, o);
}

// The query operand of the same word: the row's eight channels in that order, the odd ones times g, the others times f.
__device__ __forceinline__ h8v query_operand(const float (&x)[8], float f, float g) {
  return h8v{(_Float16)(x[0] * f), (_Float16)(x[4] * f), (_Float16)(x[1] * g), (_Float16)(x[5] * g),
             (_Float16)(x[2] * f), (_Float16)(x[6] * f), (_Float16)(x[3] * g), (_Float16)(x[7] * g)};
}

// The exponent that brings a row whose largest element has these bits to [2^13, 2^14): 2^-114 for bf16's largest, at most 2^100.
__device__ __forceinline__ int query_exponent(float top) {
  return min(100, 140 - (int)(__builtin_bit_cast(uint32_t, top) >> 23));
}
// c1 of queries scaled by 2^e and codes scaled by 2^-bits.  Positive, and at most 2^90: scores / c1 are whole multiples of 2^-69
// (codes 2^-21, queries 2^-24, a scale 2^-24 at least), so beyond that the largest score alone has weight either way, and
// no product of it with a scale and a sum overflows.
__device__ __forceinline__ float score_factor(float scale, int e, int bits) {
  return __builtin_fminf(__builtin_fmaxf(__builtin_ldexpf(scale * kLog2e, bits - e), 1e-37f), 0x1p90f);
}

// A query row spread over the lanes that share column l: its operands, and the constants of its scores.
template <class T, int WORDS>
__device__ __forceinline__ void load_query(const uint16_t* src, float scale, h8v (&op)[WORDS], float& sum, float& c1) {
  u32x4 raw[WORDS];
#pragma unroll
  for (int w = 0; w < WORDS; ++w) raw[w] = *reinterpret_cast<const u32x4*>(src + 8 * w);
  float top = 0.0f;
#pragma unroll
  for (int w = 0; w < WORDS; ++w)
#pragma unroll
    for (int i = 0; i < 8; ++i) top = __builtin_fmaxf(top, __builtin_fabsf(elem<T>(raw[w][i / 2], i & 1)));
  top = join_max<true>(top);
  const int e = top == __builtin_inff() ? 0 : query_exponent(top);
  const float f = __builtin_ldexpf(1.0f, e);
  float s = 0.0f;
#pragma unroll
  for (int w = 0; w < WORDS; ++w) {
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = elem<T>(raw[w][i / 2], i & 1);
    op[w] = query_operand(x, f, f * 0.0625f);
#pragma unroll
    for (int i = 0; i < 8; ++i) s += x[i] * f;
  }
  sum = join_sum<true>(s) * 0x1p-21f;
  c1 = score_factor(scale, e, kCodeBits);
}

__device__ __forceinline__ float low_half(uint32_t w) { return elem<Fp16>(w, 0); }
__device__ __forceinline__ float high_half(uint32_t w) { return elem<Fp16>(w, 1); }

constexpr float kTarget = 4.0f, kLimit = 15.0f;   // log2 of a row's largest weight: after ref is raised (at least), and at most

// How far ref rises for a row whose largest weight is 2^top (its scale's exponent alone): at the row's first tokens wherever that
// is, later only upwards.  Beyond 2^22, where the scores' own steps come near the target, to that weight's score itself, so that
// no weight is left above its value scale.
__device__ __forceinline__ float rise(float top, bool first) {
  const float to = __builtin_fabsf(top) < 0x1p22f ? top - kTarget : top;
  if (first) return top == kNegInf ? 0.0f : to;
  return __builtin_fmaxf(to, 0.0f);
}

// 47 + log2 of the scale in the high half of a parameter word, to 0.09 below: fp16's exponent and mantissa bits, read as a
// fraction of 32 (the fifteen bits times 2^-10), and up to 2^-10 of the zero point's.  Scales below 2^-14, zero among them, count as
// 2^-15 to 2^-14.  exponent(): the same rounded down to a whole number.
constexpr float kLogBias = 47.0f;
__device__ __forceinline__ float log_scale(uint32_t word) {
  return __builtin_bit_cast(float, __builtin_amdgcn_alignbit(0x42u, word, 8));
}
__device__ __forceinline__ float exponent(uint32_t word) {
  return __builtin_bit_cast(float, __builtin_amdgcn_alignbit(0x42u, word, 8) & 0xFFFC0000u);
}

// ------------------------------------------------------------------ few query rows: bound by the cache's bytes
// One workgroup: a chunk of one sequence's tokens in one kv head against 16 query rows.  Its WAVES waves
// take turns at units of 32 tokens, loaded straight into registers (16 bytes a lane), and join their sums at the end
// through LDS.  A unit's keys are replaced by the next unit's as soon as the score product has read them, its values
// after theirs: one unit of registers, so that four waves fit a SIMD (D = 128) and hide each other's latency.
//
// Measured (GPU time): 16 sequences of up to 2048 tokens, 32 kv heads of 128 channels: 21.8 us, 4.7 TB/s of codes and parameters (a
// plain read of as many bytes takes 17); 4 of up to 32768, 8 kv heads, 64 query heads: 26.5 us and 4 to join, 4.8 TB/s.  There the
// vector ALUs' some 200 instructions a unit take half the time and do not hide wholly behind the loads.  Two units of
// registers (half the waves) and 16 chunks instead of 8 gained nothing.
template <class T, int D, int WAVES>
__global__ __launch_bounds__(64 * WAVES) __attribute__((amdgpu_waves_per_eu(D == 256 ? 2 : 4))) void decode_kernel(Args a) {
  constexpr int W = D / 32;                  // words of codes a lane holds of a 16-token tile: keys and values
  constexpr int NT = D / 16;                 // 16-channel tiles of the output
  __shared__ float sm[WAVES][16], sl[WAVES][16];
  __shared__ __attribute__((aligned(16))) f32x4 so[WAVES / 2][NT][64];

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, h = lane >> 4;
  int lin = blockIdx.x;
  const int chunk = lin % a.chunks;
  lin /= a.chunks;
  const int tile = lin % a.row_tiles, bh = lin / a.row_tiles;
  const int b = bh / a.heads, head = bh - b * a.heads;
  const kv4::Sequence seq = kv4::sequence(a.q_start[b], a.q_start[b + 1], a.lens[b], a.total_q, a.max_q, a.max_len,
                                          a.width << a.log_page);
  const int rows = seq.queries * a.group, r0 = tile * 16;
  if (r0 >= rows) return;
  const int last = min(r0 + 16, rows) - 1;
  const int begin = chunk * a.chunk_tokens;
  const int end = min(begin + a.chunk_tokens, kv4::visible(seq, last / a.group));
  if (chunk > 0 && begin >= end) return;     // the joining kernel leaves such chunks out
  const int all = min(kv4::visible(seq, r0 / a.group), seq.tokens);   // tokens every row of the tile sees

  // Addresses: row of the first token of each 16-token tile of a unit (units start at multiples of 32 tokens).
  const int32_t* table = a.table + (int64_t)b * a.width;
  auto row_of = [&](int tok) __attribute__((always_inline)) {
    const int page = kv4::page_id(table[kv4::table_column(tok, a.log_page, a.width)], a.pages);
    return kv4::row_index(page, head, a.heads, a.log_page, tok & ((1 << a.log_page) - 1));
  };
  struct Rows {
    int64_t r[2];
  };
  auto rows_of = [&](int base) __attribute__((always_inline)) {
    Rows x;
    x.r[0] = row_of(base);
    x.r[1] = a.log_page >= 5 ? x.r[0] + 16 : row_of(base + 16);
    return x;
  };
  uint32_t k[2][W], v[2][W];
  u32x4 kp[2], vp[2];
  auto words = [&](uint32_t (&x)[W], const uint32_t* src) __attribute__((always_inline)) {
    if constexpr (W == 2) {
      const u32x2 y = *reinterpret_cast<const u32x2*>(src);
      x[0] = y[0], x[1] = y[1];
    } else {
#pragma unroll
      for (int g = 0; g < W; g += 4) {
        const u32x4 y = *reinterpret_cast<const u32x4*>(src + g);
#pragma unroll
        for (int j = 0; j < 4; ++j) x[g + j] = y[j];
      }
    }
  };
  const int k_off = l16 * (D / 8) + h * W, v_off = h * (D / 2) + l16 * W;
  auto load_keys = [&](const Rows& r) __attribute__((always_inline)) {
#pragma unroll
    for (int t = 0; t < 2; ++t) words(k[t], reinterpret_cast<const uint32_t*>(a.k + r.r[t] * (D / 2)) + k_off);
  };
  auto load_key_parameters = [&](const Rows& r) __attribute__((always_inline)) {
#pragma unroll
    for (int t = 0; t < 2; ++t) kp[t] = *reinterpret_cast<const u32x4*>(a.k_par + r.r[t] + 4 * h);
  };
  auto load_values = [&](const Rows& r) __attribute__((always_inline)) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      words(v[t], reinterpret_cast<const uint32_t*>(a.v + r.r[t] * (D / 2)) + v_off);
      vp[t] = *reinterpret_cast<const u32x4*>(a.v_par + r.r[t] + 4 * h);
    }
  };
  int base = begin + 32 * wave;
  if (base < end) {
    const Rows r = rows_of(base);
    load_keys(r);
    load_key_parameters(r);
    load_values(r);
  }

  h8v q[W];
  float qs, c1;
  const int row = min(r0 + l16, rows - 1), qi = row / a.group;
  load_query<T, W>(a.q + (int64_t)(seq.first + qi) * a.q_stride + (int64_t)(head * a.group + row - qi * a.group) * D + 8 * W * h,
                   a.scale, q, qs, c1);
  const int limit = kv4::visible(seq, qi);

  f32x4 o[NT], zs = {};
  float ref = 0.0f, l = 0.0f;                // l: this lane's part of sum 2^(score - ref)
  bool first = true;
#pragma unroll
  for (int i = 0; i < NT; ++i) o[i] = f32x4{};

  for (; base < end; base += 32 * WAVES) {
    const Rows next = rows_of(min(base + 32 * WAVES, end - 1) & ~31);    // behind the last unit: in the chunk, unused
    f32x4 s[2] = {};
#pragma unroll
    for (int w = 0; w < W; ++w)
#pragma unroll
      for (int t = 0; t < 2; ++t) s[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(unpack_keys(k[t][w]), q[w], s[t], 0, 0, 0);
    load_keys(next);
    if (base + 32 > all) {                   // what lies behind the sequence's end is no number
      const int there = seq.tokens - base - 4 * h;
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (16 * t + r >= there) kp[t][r] = vp[t][r] = 0;
    }

    float y[8], top = kNegInf;               // score - ref
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t par = kp[j >> 2][j & 3];
      y[j] = __builtin_fmaf(__builtin_fmaf(-low_half(par), qs, s[j >> 2][j & 3]) * high_half(par), c1, -ref);
    }
    load_key_parameters(next);
    if (base + 32 > all) {
      const int seen = limit - base - 4 * h;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (16 * (j >> 2) + (j & 3) >= seen) y[j] = kNegInf;
    }
#pragma unroll
    for (int j = 0; j < 8; j += 2)
      top = max3(top, y[j] + log_scale(vp[j >> 2][j & 3]), y[j + 1] + log_scale(vp[j >> 2][(j & 3) + 1]));
    if (first || __any(top > kTarget + 1.0f + kLogBias)) {
      top = kNegInf;
#pragma unroll
      for (int j = 0; j < 8; ++j) top = __builtin_fmaxf(top, y[j] + exponent(vp[j >> 2][j & 3]));
      const float delta = rise(join_max<true>(top) - kLogBias, first), f = first ? 0.0f : exp2_fast(-delta);
      first = false;
      ref += delta;
      l *= f;
      zs *= f;
#pragma unroll
      for (int i = 0; i < NT; ++i) o[i] *= f;
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] -= delta;
    }
    h8v p;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float e = exp2_fast(y[j]);
      l += e;
      p[j] = (_Float16)(e * high_half(vp[j >> 2][j & 3]));
    }

    // zero points: rows of the first operand all alike, so every register of zs holds the same sum
    u32x4 zp;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int r = 0; r < 2; ++r)
        zp[2 * t + r] = __builtin_amdgcn_perm(vp[t][2 * r + 1], vp[t][2 * r], 0x05040100u);
    zs = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8v, zp), p, zs, 0, 0, 0);
#pragma unroll
    for (int u = 0; u < W / 2; ++u) {
      const u32x4 lo = {v[0][2 * u], v[0][2 * u + 1], v[1][2 * u], v[1][2 * u + 1]};
      const u32x4 x = lo << 3, z = lo >> 5;
      const u32x4 op[4] = {x & 0x00780078u, x & 0x07800780u, z & 0x00780078u, z & 0x07800780u};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        o[4 * u + i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8v, op[i]), p, o[4 * u + i], 0, 0, 0);
    }
    load_values(next);
  }

  // Join the waves: everything to the largest reference (log2), then a tree over the sums.
  l = join_sum<true>(l);
  if (h == 0) {
    sm[wave][l16] = l > 0.0f || l != l ? ref : kNegInf;
    sl[wave][l16] = l;
  }
  __syncthreads();
  float M = kNegInf;
  l = 0.0f;
#pragma unroll
  for (int x = 0; x < WAVES; ++x) M = __builtin_fmaxf(M, sm[x][l16]);
#pragma unroll
  for (int x = 0; x < WAVES; ++x)
    if (M != kNegInf) l += sl[x][l16] * exp2_fast(sm[x][l16] - M);
  const float f = M == kNegInf ? 0.0f : exp2_fast(sm[wave][l16] - M);
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) o[i][r] = f * __builtin_fmaf(o[i][r], i & 1 ? 0x1p17f : 0x1p21f, -zs[0]);
  for (int half = WAVES / 2; half; half >>= 1) {
    if (half < WAVES / 2) __syncthreads();   // the step before has read its buffers
    if (wave >= half && wave < 2 * half) {
#pragma unroll
      for (int i = 0; i < NT; ++i) so[wave - half][i][lane] = o[i];
    }
    __syncthreads();
    if (wave < half) {
#pragma unroll
      for (int i = 0; i < NT; ++i) o[i] += so[wave][i][lane];
    }
  }
  if (wave > 0 || r0 + l16 >= rows) return;
  // register g of o[j]: channel NT * (4 h + g) + j
  const int64_t id = (int64_t)(seq.first + qi) * a.q_heads + head * a.group + row - qi * a.group;
  if (a.chunks == 1) {
    const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
#pragma unroll
    for (int g = 0; g < 4; ++g)
#pragma unroll
      for (int j = 0; j < NT; j += 4)
        *reinterpret_cast<u32x2*>(a.out + id * D + NT * (4 * h + g) + j) =
            u32x2{pack2<T>(o[j][g] * inv, o[j + 1][g] * inv), pack2<T>(o[j + 2][g] * inv, o[j + 3][g] * inv)};
    return;
  }
  const int64_t all_rows = (int64_t)a.total_q * a.q_heads;
  float* dst = a.part + (chunk * all_rows + id) * D;
#pragma unroll
  for (int g = 0; g < 4; ++g)
#pragma unroll
    for (int j = 0; j < NT; j += 4)
      *reinterpret_cast<f32x4*>(dst + NT * (4 * h + g) + j) = f32x4{o[j][g], o[j + 1][g], o[j + 2][g], o[j + 3][g]};
  if (h == 0) {
    float* ml = a.part + a.chunks * all_rows * D + (chunk * all_rows + id) * 2;
    ml[0] = M;
    ml[1] = l;
  }
}

// ------------------------------------------------------------------ many query rows: bound by the vector ALUs and matrix cores
// One workgroup of four waves: 128 query rows of one sequence and kv head, 32 a wave, against a chunk of the tokens in
// tiles of 64.  A tile is unpacked once for all waves on its way into LDS, as fp16 operands with the zero point already
// taken off (q 2^-24 or 16 q 2^-24, as the bits lie, times a power of two less the zero point, in one instruction for two codes: a small
// integer's multiple of 2^-9, a normal number), two buffers, the next tile's loads in registers
// meanwhile.  That leaves a wave per score one fma (scale and running maximum), half a maximum, the exponential, the
// sum, the value scale and half a conversion.
//
// LDS.  Keys: row of a token, 16-byte chunk c (a word's eight channels) at position c ^ (token & 15), D = 64: c ^ (token / 2 & 7).  Values: row of a
// channel, 64 tokens in the order in which a lane of the score product holds them (16 at a time: 0-3, 8-11 for
// lanes 0-31, 4-7, 12-15 for the others); chunk c at position c ^ (d & 7) ^ (d / 8 & 7).  Sixteen lanes of a 16-byte read hit all banks.
//
// The scale of the queries (a power of two) is one for the workgroup, so that a token's factor c1 * s can be made when it
// is staged.  A row 2^12 below the largest one then still has its queries to 2^-25 of its own largest element.  Where rows lie further
// apart (or one is far out), each has a scale of its own, c1 stands for one half way between the ends, and each row's sums are
// multiplied by its own factor over that one before they are scaled: 16 products a half tile in a branch of the whole workgroup.
//
// Reference: a half tile's largest score and the largest value scale of the wave so far bound its weights; only where that bound
// passes 2^15 are the weights themselves looked at.
//
// Measured: 2 prompts of up to 4096 tokens, 32 heads of 128 channels: 279-299 us (0.81-0.87 PFLOP/s of the visible half; the matrix cores' rate
// alone would take 177).  The vector ALUs are busy 60% of the time (counters), the matrix cores 40%, and the clock gives way to
// the power drawn: the same call takes 334 us on normal data of full length, 281 on zeros.  Rows with scales of their own 294 us
// where one scale takes 284.  Of a workgroup's time 8 us are its start, first tile and end.  64 rows a wave with one wave a SIMD (half the LDS reads and unpacking a row) took 499 us, eight waves a
// workgroup no less than four, and a schedule pinned to the products 4% more.
template <class T, int D>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(D == 256 ? 1 : 2))) void prompt_kernel(Args a) {
  constexpr int NW = 4;                      // waves
  constexpr int S = D / 16;                  // K = 16 slices of the key product
  constexpr int NT = D / 32;                 // 32-channel tiles of the output
  constexpr int kTile = 64;
  constexpr int kStageBits = 9;              // codes in LDS are multiples of 2^-9
  constexpr int W = D / (8 * NW);            // words of key codes, and of value codes, that a thread stages: 2, 4 or 8
  constexpr int kLds = kTile * D * 2;        // bytes of a tile's keys, or values, in LDS
  __shared__ __attribute__((aligned(16))) uint8_t lds[2][2][kLds];
  __shared__ __attribute__((aligned(16))) float lf[2][2][kTile];           // c1 * key scale, value scale
  __shared__ int lexp[2][NW];                // a wave's least and largest exponent of a row

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l32 = lane & 31, h = lane >> 5;
  int lin = blockIdx.x;
  const int chunk = lin % a.chunks;
  lin /= a.chunks;
  const int bh = lin % (a.batch * a.heads);
  const int tile = a.row_tiles - 1 - lin / (a.batch * a.heads);   // the rows that see most first
  const int b = bh / a.heads, head = bh - b * a.heads;
  const kv4::Sequence seq = kv4::sequence(a.q_start[b], a.q_start[b + 1], a.lens[b], a.total_q, a.max_q, a.max_len,
                                          a.width << a.log_page);
  const int rows = seq.queries * a.group, r0 = tile * (32 * NW);
  if (r0 >= rows) return;
  const int begin = chunk * a.chunk_tokens;
  const int end = min(begin + a.chunk_tokens, kv4::visible(seq, (min(r0 + 32 * NW, rows) - 1) / a.group));
  if (chunk > 0 && begin >= end) return;

  const int row = min(r0 + 32 * wave + l32, rows - 1), qi = row / a.group;
  const int limit = kv4::visible(seq, qi);
  // the tokens that all of this wave's rows see
  const int all = min(kv4::visible(seq, min(r0 + 32 * wave, rows - 1) / a.group), seq.tokens);

  auto key_swizzle = [](int t) { return D == 64 ? (t >> 1) & 7 : t & 15; };   // D = 64: two rows cover the banks
  // ---- staging: thread t carries words W (t % NW) .. of token t / NW's keys, and words W (t % 4 NW) .. of 4-token
  // block t / (4 NW)'s values
  const int32_t* table = a.table + (int64_t)b * a.width;
  auto row_of = [&](int tok) __attribute__((always_inline)) {
    const int page = kv4::page_id(table[kv4::table_column(tok, a.log_page, a.width)], a.pages);
    return kv4::row_index(page, head, a.heads, a.log_page, tok & ((1 << a.log_page) - 1));
  };
  const int kt = tid / NW, kp = tid % NW, vb = tid / (4 * NW), vp = tid % (4 * NW);
  uint32_t gk[W], gv[W], gkp;
  u32x4 gvp;
  auto get = [&](uint32_t (&x)[W], const uint32_t* src) __attribute__((always_inline)) {
    if constexpr (W >= 4) {
#pragma unroll
      for (int g = 0; g < W; g += 4) {
        const u32x4 v = *reinterpret_cast<const u32x4*>(src + g);
#pragma unroll
        for (int j = 0; j < 4; ++j) x[g + j] = v[j];
      }
    } else {
      const u32x2 v = *reinterpret_cast<const u32x2*>(src);
      x[0] = v[0], x[1] = v[1];
    }
  };
  // Pages of 64 tokens or more hold a whole tile: one page for all threads, its id read a tile ahead.
  const bool whole = a.log_page >= 6;
  auto page_of = [&](int tok) __attribute__((always_inline)) {
    return table[kv4::table_column(tok, a.log_page, a.width)];
  };
  int entry = whole ? page_of(begin) : 0;
  auto fetch = [&](int base) __attribute__((always_inline)) {
    if (whole) {
      const int64_t row = kv4::row_index(kv4::page_id(__builtin_amdgcn_readfirstlane(entry), a.pages), head, a.heads, a.log_page,
                                         base & ((1 << a.log_page) - 1));
      get(gk, reinterpret_cast<const uint32_t*>(a.k + row * (D / 2)) + (kt * (D / 8) + W * kp));
      get(gv, reinterpret_cast<const uint32_t*>(a.v + row * (D / 2)) + (vb * (D / 2) + W * vp));
      gkp = (a.k_par + row)[kt];
      gvp = *reinterpret_cast<const u32x4*>(a.v_par + row + 4 * vb);
      entry = page_of(base + kTile);
    } else {
      const int64_t kr = row_of(base + kt), vr = row_of(base + 4 * vb);
      int wk = W * kp, wv = W * vp;          // kept from being added to the arrays' addresses ahead of the loop: no registers for that
      asm("" : "+v"(wk), "+v"(wv));
      get(gk, reinterpret_cast<const uint32_t*>(a.k + kr * (D / 2)) + wk);
      get(gv, reinterpret_cast<const uint32_t*>(a.v + vr * (D / 2)) + wv);
      gkp = a.k_par[kr];
      gvp = *reinterpret_cast<const u32x4*>(a.v_par + vr);
    }
  };
  if (begin < end) fetch(begin);             // on its way while the queries are read and scaled

  // ---- queries: lane half h holds words 2 s + h of its row
  h8v q[S];
  float c1, rel;                             // rel: this row's factor over c1
  bool apart;
  {
    const uint16_t* src = a.q + (int64_t)(seq.first + qi) * a.q_stride + (int64_t)(head * a.group + row - qi * a.group) * D + 8 * h;
    u32x4 raw[S];
#pragma unroll
    for (int w = 0; w < S; ++w) raw[w] = *reinterpret_cast<const u32x4*>(src + 16 * w);
    float top = 0.0f;
#pragma unroll
    for (int w = 0; w < S; ++w)
#pragma unroll
      for (int i = 0; i < 8; ++i) {          // the row's largest finite element
        const float x = __builtin_fabsf(elem<T>(raw[w][i / 2], i & 1));
        top = x < __builtin_inff() ? __builtin_fmaxf(top, x) : top;
      }
    top = join_max<false>(top);
    const int own = query_exponent(top);
    int least = own, most = top > 0.0f ? own : -114;     // a row of zeros keeps no distance
#pragma unroll
    for (int d = 16; d; d >>= 1) {
      least = min(least, __shfl_xor(least, d));
      most = max(most, __shfl_xor(most, d));
    }
    if (lane == 0) lexp[0][wave] = least, lexp[1][wave] = most;
    __syncthreads();
#pragma unroll
    for (int v = 0; v < NW; ++v) {
      least = min(least, lexp[0][v]);
      most = max(most, lexp[1][v]);
    }
    least = __builtin_amdgcn_readfirstlane(least);
    most = __builtin_amdgcn_readfirstlane(most);
    apart = most - least > 12;
    const int e = apart ? own : least;
    const float f = __builtin_ldexpf(1.0f, e);
#pragma unroll
    for (int w = 0; w < S; ++w) {
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = elem<T>(raw[w][i / 2], i & 1);
      q[w] = query_operand(x, f, f);
    }
    c1 = score_factor(a.scale, apart ? (least + most) >> 1 : least, kStageBits);
    rel = score_factor(a.scale, e, kStageBits) / c1;
  }

  auto half2 = [](uint32_t w) { return __builtin_bit_cast(h2v, w); };
  const h2v kUnit = {(_Float16)0x1p-9f, (_Float16)0x1p-9f}, kLow = {(_Float16)0x1p15f, (_Float16)0x1p15f},
            kHigh = {(_Float16)0x1p11f, (_Float16)0x1p11f};
  // the pairs of halves (q - zero) 2^-9 of the codes in the two low nibbles of each half-word
  auto unpack = [&](uint32_t w, h2v z) __attribute__((always_inline)) {
    return u32x2{__builtin_bit_cast(uint32_t, __builtin_elementwise_fma(half2(w & 0x000F000Fu), kLow, -z)),
                 __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(half2(w & 0x00F000F0u), kHigh, -z))};
  };
  // Staging in steps that fill the gaps between matrix products: parameters and keys first, then the values.
  uint8_t* const skeys = &lds[0][0][0] + kt * (D * 2);
  uint8_t* const svals = &lds[0][1][0] + 8 * ((vb >> 1) & 1);
  const int vchunk = 2 * (vb >> 2) + (vb & 1);           // 16-byte chunk of a channel's row that holds the block's tokens
  h2v kz, vz[2];
  auto stage_parameters = [&](int buf, int base) __attribute__((always_inline)) {
    uint32_t par = gkp;
    u32x4 vpar = gvp;
    if (base + kTile > seq.tokens) {                     // what lies behind the sequence's end is no number
      if (base + kt >= seq.tokens) par = 0;
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (base + 4 * vb + r >= seq.tokens) vpar[r] = 0;
    }
    kz = half2(__builtin_amdgcn_perm(par, par, 0x01000100u)) * kUnit;
    lf[buf][0][kt] = c1 * high_half(par);                // the same from every thread of the token
    vz[0] = half2(__builtin_amdgcn_perm(vpar[1], vpar[0], 0x05040100u)) * kUnit;
    vz[1] = half2(__builtin_amdgcn_perm(vpar[3], vpar[2], 0x05040100u)) * kUnit;
    *reinterpret_cast<f32x4*>(&lf[buf][1][4 * vb]) =
        f32x4{high_half(vpar[0]), high_half(vpar[1]), high_half(vpar[2]), high_half(vpar[3])};
  };
  auto stage_keys = [&](int buf, int w) __attribute__((always_inline)) {           // w < W
    const u32x2 lo = unpack(gk[w], kz), hi = unpack(gk[w] >> 8, kz);
    *reinterpret_cast<u32x4*>(skeys + buf * (2 * kLds) + (((W * kp + w) ^ key_swizzle(kt)) << 4)) =
        u32x4{lo[0], lo[1], hi[0], hi[1]};
  };
  auto stage_values = [&](int buf, int n) __attribute__((always_inline)) {         // n < W: two channels of a quad
    auto place = [&](int d) __attribute__((always_inline)) {
      return svals + buf * (2 * kLds) + d * 128 + ((vchunk ^ (d & 7) ^ ((d >> 3) & 7)) << 4);
    };
    const int g = n >> 1, i = 2 * (n & 1), d = 4 * (W / 2 * vp + g) + i;
    const u32x2 x = unpack(gv[2 * g] >> (4 * i), vz[0]), z = unpack(gv[2 * g + 1] >> (4 * i), vz[1]);
    *reinterpret_cast<u32x2*>(place(d)) = u32x2{x[0], z[0]};
    *reinterpret_cast<u32x2*>(place(d + 1)) = u32x2{x[1], z[1]};
  };

  f32x16 o[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) o[i] = f32x16{};
  float ref = 0.0f, l = 0.0f;
  float most = 0x1p-40f, room = kLimit + 40.0f;          // a power of two that no value scale so far exceeds, kLimit - log2 of it
  bool first = true;

  // LDS addresses of this lane's operands in buffer 0; other buffers, halves and channels are constants further.
  const uint8_t* const base0 = &lds[0][0][0];
  int ka[S], va[4];
#pragma unroll
  for (int w = 0; w < S; ++w) ka[w] = l32 * (D * 2) + (((2 * w + h) ^ key_swizzle(l32)) << 4);
#pragma unroll
  for (int x = 0; x < 4; ++x) va[x] = kLds + l32 * 128 + (((2 * x + h) ^ (l32 & 7) ^ (l32 >> 3)) << 4);
  // key operand of slice w of half t; value operand n: 16 tokens n / NT of half t, channels 32 (n % NT) + l32
  auto key = [&](int buf, int t, int w) __attribute__((always_inline)) {
    return *reinterpret_cast<const h8v*>(base0 + ka[w] + (buf * 2 * kLds + t * 32 * D * 2));
  };
  auto value = [&](int buf, int t, int n) __attribute__((always_inline)) {
    const int x = n / NT, i = n % NT;
    return *reinterpret_cast<const h8v*>(base0 + va[2 * (t ^ (i & 1)) + x] + (buf * 2 * kLds + i * 4096));
  };

  float y[16];
  h8v p[2], ring[4];
  f32x16 s;
  f32x4 u[4];                                // value scales of the half tile whose weights come next (see read)
  // Masks, and raises the reference where it has to be raised; base: the half tile's first token.
  auto settle = [&](int buf, int t, int base) __attribute__((always_inline)) {
    if (base + 32 > all) {
      const int seen = limit - base - 4 * h;
#pragma unroll
      for (int j = 0; j < 16; ++j)
        if (8 * (j >> 2) + (j & 3) >= seen) y[j] = kNegInf;
    }
    float big = lf[buf][1][32 * t + l32];    // a value scale: of any token
    float top = max3(y[0], y[1], y[2]);
#pragma unroll
    for (int j = 3; j < 15; j += 2) top = max3(top, y[j], y[j + 1]);
    top = __builtin_fmaxf(top, y[15]);
    if (first || __any(top > room || big > most)) {
#pragma unroll
      for (int d = 16; d; d >>= 1) big = __builtin_fmaxf(big, __shfl_xor(big, d));
      most = __builtin_bit_cast(float, (__builtin_bit_cast(uint32_t, __builtin_fmaxf(big, most)) + 0x7FFFFFu) & 0x7F800000u);
      room = uniform(kLimit + 127.0f - (float)(__builtin_bit_cast(uint32_t, most) >> 23));
      most = uniform(most);
      top = kNegInf;
#pragma unroll
      for (int j = 0; j < 16; ++j) {         // a scale of zero counts as 2^-40: its p stays in fp32's range
        const float v = lf[buf][1][32 * t + 4 * h + 8 * (j >> 2) + (j & 3)];
        top = __builtin_fmaxf(top, y[j] + (float)(__builtin_amdgcn_frexp_expf(__builtin_fmaxf(v, 0x1p-40f)) - 1));
      }
      const float delta = rise(join_max<false>(top), first), f = first ? 0.0f : exp2_fast(-delta);
      first = false;
      ref += delta;
      l *= f;
#pragma unroll
      for (int i = 0; i < NT; ++i) o[i] *= f;
#pragma unroll
      for (int j = 0; j < 16; ++j) y[j] -= delta;
    }
  };
  auto weigh = [&]() __attribute__((always_inline)) {      // s of rows with scales of their own
    if (apart) {
#pragma unroll
      for (int j = 0; j < 16; ++j) s[j] *= rel;
    }
  };
  auto scale4 = [&](const f32x4& f, int g) __attribute__((always_inline)) {
#pragma unroll
    for (int r = 0; r < 4; ++r) y[4 * g + r] = __builtin_fmaf(s[4 * g + r], f[r], -ref);
  };
  // Scores of (buf, t) on the matrix cores while the vector ALUs turn y into the weights of (wbuf, wt).  Every product is a
  // scheduling region of its own with its share of the rest, operands are read four products ahead; the last reads
  // are the first operands of the product with the values that follows.
  // The first reads of scores_and_weights, made before the masks and the reference of the half tile in front (D = 256
  // has no registers for that).
  auto read = [&](int buf, int t, int wbuf, int wt) __attribute__((always_inline)) {
#pragma unroll
    for (int w = 0; w < 4; ++w) ring[w] = key(buf, t, w);
#pragma unroll
    for (int g = 0; g < 4; ++g) u[g] = *reinterpret_cast<const f32x4*>(&lf[0][0][0] + (2 * wbuf + 1) * kTile + 32 * wt + 8 * g + 4 * h);
    __builtin_amdgcn_sched_barrier(0);
  };
  auto read_ahead = [&](int buf, int t, int wbuf, int wt) __attribute__((always_inline)) {
    if (D < 256) read(buf, t, wbuf, wt);
  };
  auto scores_and_weights = [&](int buf, int t, int wbuf, int wt) __attribute__((always_inline)) {
    if (D == 256) read(buf, t, wbuf, wt);
    s = f32x16{};
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int w = 0; w < S; ++w) {
      s = __builtin_amdgcn_mfma_f32_32x32x16_f16(ring[w & 3], q[w], s, 0, 0, 0);
      ring[w & 3] = w + 4 < S ? key(buf, t, w + 4 < S ? w + 4 : 0) : value(wbuf, wt, w + 4 - S < 0 ? 0 : w + 4 - S);
#pragma unroll
      for (int j = 16 * w / S; j < 16 * (w + 1) / S; ++j) {
        const float e = exp2_fast(y[j]);
        l += e;
        p[j >> 3][j & 7] = (_Float16)(e * u[j >> 2][j & 3]);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // The product of the weights with the values of (wbuf, wt) while s is scaled (factors of (buf, t)) and `fill(n)` runs.
  auto product_and_scale = [&](int wbuf, int wt, int buf, int t, auto fill) __attribute__((always_inline)) {
    weigh();
    f32x4 f[4];
#pragma unroll
    for (int g = 0; g < 4; ++g) f[g] = *reinterpret_cast<const f32x4*>(&lf[0][0][0] + 2 * buf * kTile + 32 * t + 8 * g + 4 * h);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int n = 0; n < 2 * NT; ++n) {
      o[n % NT] = __builtin_amdgcn_mfma_f32_32x32x16_f16(ring[n & 3], p[n / NT], o[n % NT], 0, 0, 0);
      if (n + 4 < 2 * NT) ring[n & 3] = value(wbuf, wt, n + 4 < 2 * NT ? n + 4 : 0);
      fill(n);
      if (n >= 2 * NT - 4) scale4(f[n - (2 * NT - 4)], n - (2 * NT - 4));
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  // Half tiles in a pipeline: while the matrix cores make the scores of one, the vector ALUs make the weights of the
  // one before; while its product with the values runs, the next scores are scaled and the next tile is unpacked.
  if (begin < end) {
    stage_parameters(0, begin);
#pragma unroll
    for (int w = 0; w < W; ++w) {
      stage_keys(0, w);
      stage_values(0, w);
    }
  }
  __syncthreads();
  if (begin + kTile < end) fetch(begin + kTile);
  if (begin < end) {
    s = f32x16{};
#pragma unroll
    for (int w = 0; w < S; ++w) s = __builtin_amdgcn_mfma_f32_32x32x16_f16(key(0, 0, w), q[w], s, 0, 0, 0);
    weigh();
#pragma unroll
    for (int g = 0; g < 4; ++g) scale4(*reinterpret_cast<const f32x4*>(&lf[0][0][8 * g + 4 * h]), g);
    read_ahead(0, 1, 0, 0);
    settle(0, 0, begin);
  }
  // One tile in buffer B.  What is staged or multiplied behind the last tile repeats what is there and is not used.
  auto step = [&](auto which, int base) __attribute__((always_inline)) {
    constexpr int B = decltype(which)::value;
    scores_and_weights(B, 1, B, 0);
    product_and_scale(B, 0, B, 1, [&](int n) __attribute__((always_inline)) {
      if (n == 0) stage_parameters(B ^ 1, base + kTile);
#pragma unroll
      for (int w = 0; w < W; ++w)
        if (n == w + 1) stage_keys(B ^ 1, w);
    });
    __syncthreads();                         // the next tile's keys are there
    read_ahead(B ^ 1, 0, B, 1);
    settle(B, 1, base + 32);
    scores_and_weights(B ^ 1, 0, B, 1);
    product_and_scale(B, 1, B ^ 1, 0, [&](int n) __attribute__((always_inline)) {
#pragma unroll
      for (int w = 0; w < W; ++w)
        if (n == w + 1) stage_values(B ^ 1, w);
    });
    read_ahead(B ^ 1, 1, B ^ 1, 0);
    if (base + kTile < end) settle(B ^ 1, 0, base + kTile);
    if (base + 2 * kTile < end) fetch(base + 2 * kTile);
    __syncthreads();                         // its values too, and every wave has read this tile
  };
  for (int base = begin; base < end; base += 2 * kTile) {
    step(Half<0>{}, base);
    if (base + kTile < end) step(Half<1>{}, base + kTile);
  }

  // Register 4 g + r of o[i]: channel 32 i + 8 g + 4 h + r.
  l = join_sum<false>(l);
  const int64_t id = (int64_t)(seq.first + qi) * a.q_heads + head * a.group + row - qi * a.group;
  const int64_t all_rows = (int64_t)a.total_q * a.q_heads;
  const bool live = r0 + 32 * wave + l32 < rows;
  if (a.chunks > 1) {
    if (!live) return;
    if (h == 0) {
      float* ml = a.part + a.chunks * all_rows * D + (chunk * all_rows + id) * 2;
      ml[0] = l > 0.0f || l != l ? ref : kNegInf;
      ml[1] = l;
    }
    float* dst = a.part + (chunk * all_rows + id) * D;
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int g = 0; g < 4; ++g)
        *reinterpret_cast<f32x4*>(dst + 32 * i + 8 * g + 4 * h) =
            f32x4{o[i][4 * g] * 0x1p9f, o[i][4 * g + 1] * 0x1p9f, o[i][4 * g + 2] * 0x1p9f, o[i][4 * g + 3] * 0x1p9f};
    return;
  }
  // Out through LDS, a wave's rows in a part of its own, so that rows leave whole (eight-byte pieces of 32 rows a
  // multiple of 4 KB apart would all go to one channel of the L2).  Piece of 16 bytes c of row r at c ^ (r & 7).
  const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
  uint8_t* own = lds[0][0] + wave * (32 * D * 2);
  static_assert(NW * 32 * D * 2 <= sizeof(lds), "the output rows fit the tile buffers");
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const float e = inv * 0x1p9f;
      *reinterpret_cast<u32x2*>(own + l32 * (D * 2) + (((4 * i + g) ^ (l32 & 7)) << 4) + 8 * h) =
          u32x2{pack2<T>(o[i][4 * g] * e, o[i][4 * g + 1] * e), pack2<T>(o[i][4 * g + 2] * e, o[i][4 * g + 3] * e)};
    }
  constexpr int kLanes = D / 8;              // lanes of a row
  for (int r = lane / kLanes; r < 32; r += 64 / kLanes) {
    const int gr = r0 + 32 * wave + r;
    if (gr < rows) {
      const int i = gr / a.group;
      const int64_t rid = (int64_t)(seq.first + i) * a.q_heads + head * a.group + gr - i * a.group;
      *reinterpret_cast<u32x4*>(a.out + rid * D + 8 * (lane % kLanes)) =
          *reinterpret_cast<const u32x4*>(own + r * (D * 2) + (((lane % kLanes) ^ (r & 7)) << 4));
    }
  }
}

// ------------------------------------------------------------------ joining the chunks of a divided sequence
// SPLIT waves a query row: its chunks' sums, each scaled to the largest reference.  Wave v of them adds chunks v, v + SPLIT,
// ... in order, then the waves' sums are added in order.  Sums are read beside the statistics, eight in flight, also of
// chunks that hold no token of the row (whatever is there, left out below): one memory latency less.  Four waves a row
// are for few rows of many chunks (64 rows of 64 chunks 18.0 us in all, 19.4 with one; 8192 rows of 8: 75.8 and 65.1).
template <class T, int D, int SPLIT>
__global__ __launch_bounds__(256) void join_kernel(Args a) {
  constexpr int C = D / 64;
  __shared__ float part[SPLIT > 1 ? 4 : 1][D];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int most = a.max_q * a.group, at = SPLIT > 1 ? (int)blockIdx.x : (int)blockIdx.x * 4 + wave, v = SPLIT > 1 ? wave : 0;
  const int bh = at / most, r = at - bh * most;
  if (bh >= a.batch * a.heads) return;       // (SPLIT = 1: the last workgroup's waves past the rows)
  const int b = bh / a.heads, head = bh - b * a.heads;
  const kv4::Sequence seq = kv4::sequence(a.q_start[b], a.q_start[b + 1], a.lens[b], a.total_q, a.max_q, a.max_len,
                                          a.width << a.log_page);
  if (r >= seq.queries * a.group) return;
  const int i = r / a.group, n = kv4::visible(seq, i);
  const int64_t id = (int64_t)(seq.first + i) * a.q_heads + head * a.group + r - i * a.group;
  const int64_t all_rows = (int64_t)a.total_q * a.q_heads;
  const int chunks = (n + a.chunk_tokens - 1) / a.chunk_tokens;          // those that hold a token of this row
  const float* ml = a.part + a.chunks * all_rows * D + id * 2;
  const float* src = a.part + id * D + lane * C;
  float x[8][C];
  auto load = [&](int c0) __attribute__((always_inline)) {
#pragma unroll
    for (int k = 0; k < 8; ++k)
#pragma unroll
      for (int j = 0; j < C; ++j) x[k][j] = src[min(c0 + SPLIT * k, a.chunks - 1) * all_rows * D + j];
  };
  load(v);
  const float2 st = *reinterpret_cast<const float2*>(ml + min(lane, a.chunks - 1) * all_rows * 2);
  const float M = lane < chunks ? st.x : kNegInf;
  float l = lane < chunks ? st.y : 0.0f;
  float top = M;
#pragma unroll
  for (int d = 32; d; d >>= 1) top = __builtin_fmaxf(top, __shfl_xor(top, d));
  const float f = M == kNegInf ? 0.0f : exp2_fast(M - top);
  l *= f;
#pragma unroll
  for (int d = 32; d; d >>= 1) l += __shfl_xor(l, d);
  float sum[C] = {};
  for (int c0 = v; c0 < chunks; c0 += 8 * SPLIT) {
    if (c0 > v) load(c0);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float g = __shfl(f, min(c0 + SPLIT * k, 63));
      if (c0 + SPLIT * k < chunks)
#pragma unroll
        for (int j = 0; j < C; ++j) sum[j] += g * x[k][j];
    }
  }
  const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
  if constexpr (SPLIT == 1) {
#pragma unroll
    for (int j = 0; j < C; ++j) a.out[id * D + lane * C + j] = T::store(sum[j] * inv);
  } else {
#pragma unroll
    for (int j = 0; j < C; ++j) part[wave][lane * C + j] = sum[j];
    __syncthreads();
    if (threadIdx.x < D) {
      const int d = threadIdx.x;
      a.out[id * D + d] = T::store((part[0][d] + part[1][d] + part[2][d] + part[3][d]) * inv);
    }
  }
}

template <class T, int D>
void launch(const Args& a, int kind, hipStream_t st) {
  const dim3 grid((unsigned)((int64_t)a.batch * a.heads * a.row_tiles * a.chunks));
  if (kind == kv4::kFour)
    hipLaunchKernelGGL((decode_kernel<T, D, 4>), grid, dim3(256), 0, st, a);
  else if (kind == kv4::kEight)
    hipLaunchKernelGGL((decode_kernel<T, D, 8>), grid, dim3(512), 0, st, a);
  else
    hipLaunchKernelGGL((prompt_kernel<T, D>), grid, dim3(256), 0, st, a);
  if (a.chunks > 1) {
    const int64_t rows = (int64_t)a.batch * a.heads * a.max_q * a.group;
    if (rows >= 1024 || a.chunks <= 8)
      hipLaunchKernelGGL((join_kernel<T, D, 1>), dim3((unsigned)((rows + 3) / 4)), dim3(256), 0, st, a);
    else
      hipLaunchKernelGGL((join_kernel<T, D, 4>), dim3((unsigned)rows), dim3(256), 0, st, a);
  }
}

}  // namespace

Kv4Plan kv4_plan(int q_heads, int heads, int dim, int batch, int max_q, int max_len) {
  return kv4::plan(q_heads, heads, dim, batch, max_q, max_len, compute_units());
}

int64_t kv4_workspace_bytes(const Kv4Plan& p, int total_q, int q_heads, int dim) {
  return p.chunks > 1 ? (int64_t)p.chunks * total_q * q_heads * (dim + 2) * 4 : 0;
}

hipError_t launch_kv4_attention(const Kv4Attention& x, const Kv4Plan& plan, float* work, hipStream_t st) {
  Args a;
  a.q = x.q;
  a.q_stride = x.q_stride;
  a.k = (const uint8_t*)x.cache.k;
  a.v = (const uint8_t*)x.cache.v;
  a.k_par = (const uint32_t*)x.cache.k_par;
  a.v_par = (const uint32_t*)x.cache.v_par;
  a.table = x.table;
  a.lens = x.lens;
  a.q_start = x.q_start;
  a.pages = x.cache.pages;
  a.log_page = __builtin_ctz(x.cache.page);
  a.heads = x.cache.heads;
  a.width = x.width;
  a.total_q = x.total_q;
  a.q_heads = x.q_heads;
  a.group = x.q_heads / x.cache.heads;
  a.batch = x.batch;
  a.max_q = x.max_q;
  a.max_len = x.max_len;
  a.row_tiles = plan.row_tiles;
  a.chunks = plan.chunks;
  a.chunk_tokens = plan.chunk_tokens;
  a.scale = x.scale;
  a.out = x.out;
  a.part = work;
  if (x.bf16) {
    if (x.cache.dim == 64) launch<Bf16, 64>(a, plan.kind, st);
    else if (x.cache.dim == 128) launch<Bf16, 128>(a, plan.kind, st);
    else launch<Bf16, 256>(a, plan.kind, st);
  } else {
    if (x.cache.dim == 64) launch<Fp16, 64>(a, plan.kind, st);
    else if (x.cache.dim == 128) launch<Fp16, 128>(a, plan.kind, st);
    else launch<Fp16, 256>(a, plan.kind, st);
  }
  return hipGetLastError();
}

}  // namespace atom
