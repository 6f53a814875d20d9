// Causal attention over the 4-bit KV cache for gfx950 (layout: atom_kv4.h).
//
// With codes k, v, zero points a, b and scales s, u of a token,
//   score = c * s * (sum_d q_d k_d - a * sum_d q_d),      c = scale * log2(e)
//   out_d = sum_t w_t (v_td - b_t) / sum_t p_t,           p = 2^(score - max), w = p * u,
// so the matrix cores multiply the codes themselves and the scales meet one score or one weight a
// token.  A code goes into the fp16 operand as the bits it has: the half-precision number with
// mantissa q is q * 2^-24 exactly (a subnormal, which the gfx950 matrix cores keep), and with the
// nibble one place up 16 q * 2^-24.  Unpacking eight codes is one shift and four ands; the factor 16 of every
// other nibble is taken out of the query (keys) or the result (values), exactly.
//
// Both products have the tokens (keys) or channels (values) as rows and the queries as columns: a
// lane's scores belong to one query, and as the contraction over tokens may run in any order, the
// weights feed the second product from the registers the first one left them in.  The values'
// four-token blocks in the cache are the operand order of that product.
//
// Ranges.  A query row is scaled by a power of two so that its largest element lies in [2^13, 2^14):
// fp16 then holds fp16 and bf16 queries exactly down to 2^-24 of that largest element.  Weights are rounded to fp16
// (relative 2^-12 each, as the output's own rounding) after a power of two, 2^-E >= 1 / (largest u so
// far), keeps them in [0, 1]: both the weights and the sum of p carry it, so it leaves the quotient.  The
// zero points multiply the rounded weights too (one more matrix product), so a rounding error acts on (v - b), not
// on v and b apart.  Scores, maxima and all sums are fp32.
//
// Running maximum: m is raised, and the sums rescaled, only when some score of the wave lies above it (or
// some u above 2^E): a wave-uniform branch that random data take in the first few tiles only.
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

// Eight codes of a word -> fp16 operand, halves (n0, n4, 16 n1, 16 n5, n2, n6, 16 n3, 16 n7) * 2^-24.
__device__ __forceinline__ h8v unpack_keys(uint32_t w) {
  const uint32_t v = w >> 8;
  const u32x4 o = {w & 0x000F000Fu, w & 0x00F000F0u, v & 0x000F000Fu, v & 0x00F000F0u};
  return __builtin_bit_cast(h8v, o);
}

// The query operand of the same word: the row's eight channels in that order, the odd ones / 16.
__device__ __forceinline__ h8v query_operand(const float (&x)[8], float f) {
  const float g = f * 0.0625f;
  return h8v{(_Float16)(x[0] * f), (_Float16)(x[4] * f), (_Float16)(x[1] * g), (_Float16)(x[5] * g),
             (_Float16)(x[2] * f), (_Float16)(x[6] * f), (_Float16)(x[3] * g), (_Float16)(x[7] * g)};
}

// A query row spread over the lanes that share column l: its operands, and the constants of its scores.
template <class T, int WORDS, bool kAll>
__device__ __forceinline__ void load_query(const uint16_t* src, float scale, h8v (&op)[WORDS], float& sum, float& c1) {
  u32x4 raw[WORDS];
#pragma unroll
  for (int w = 0; w < WORDS; ++w) raw[w] = *reinterpret_cast<const u32x4*>(src + 8 * w);
  float top = 0.0f;
#pragma unroll
  for (int w = 0; w < WORDS; ++w)
#pragma unroll
    for (int i = 0; i < 8; ++i) top = __builtin_fmaxf(top, __builtin_fabsf(elem<T>(raw[w][i / 2], i & 1)));
  top = join_max<kAll>(top);
  const int ex = (int)(__builtin_bit_cast(uint32_t, top) >> 23) - 127;   // floor(log2 top); -127 for 0, 128 for inf
  const int e = max(-100, min(100, ex == 128 ? 0 : 13 - ex));
  const float f = __builtin_ldexpf(1.0f, e);
  float s = 0.0f;
#pragma unroll
  for (int w = 0; w < WORDS; ++w) {
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = elem<T>(raw[w][i / 2], i & 1);
    op[w] = query_operand(x, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) s += x[i] * f;
  }
  sum = join_sum<kAll>(s) * 0x1p-24f;
  // positive and finite, so that it keeps the scores' order and -inf stays -inf
  c1 = __builtin_fminf(__builtin_fmaxf(__builtin_ldexpf(scale * kLog2e, 24 - e), 1e-37f), 3e38f);
}

// Running statistics of one column's sums.
struct Stat {
  float m;       // the largest y = score / c1 seen (or -inf)
  float ref;     // what is subtracted in the exponent: c1 * m + E (0 while m = -inf)
  float l;       // this lane's part of sum p 2^-E
};

__device__ __forceinline__ float low_half(uint32_t w) { return elem<Fp16>(w, 0); }
__device__ __forceinline__ float high_half(uint32_t w) { return elem<Fp16>(w, 1); }
// E for a word whose high half is the largest scale: scale <= 2^E
__device__ __forceinline__ float exponent_of(uint32_t word) {
  const float s = high_half(word);
  return (float)max(-24, (int)(__builtin_bit_cast(uint32_t, s) >> 23) - 126);
}

// ------------------------------------------------------------------ few query rows: bound by the cache's bytes
// One workgroup: a chunk of one sequence's tokens in one kv head against NR * 16 query rows.  Its four
// waves take turns at units of 32 tokens, loaded straight into registers (16 bytes a lane), the next
// unit's while the current one is multiplied, and join their sums at the end through LDS.
template <class T, int D, int NR>
__global__ __launch_bounds__(256) void decode_kernel(Args a) {
  constexpr int W = D / 32;                  // words of codes a lane holds of a 16-token tile: keys and values
  constexpr int NT = D / 16;                 // 16-channel tiles of the output
  __shared__ float sm[4][NR * 16], sl[4][NR * 16];
  __shared__ __attribute__((aligned(16))) f32x4 so[2][NT][64];

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, h = lane >> 4;
  int lin = blockIdx.x;
  const int chunk = lin % a.chunks;
  lin /= a.chunks;
  const int tile = lin % a.row_tiles, bh = lin / a.row_tiles;
  const int b = bh / a.heads, head = bh - b * a.heads;
  const kv4::Sequence seq = kv4::sequence(a.q_start[b], a.q_start[b + 1], a.lens[b], a.total_q, a.max_q, a.max_len,
                                          a.width << a.log_page);
  const int rows = seq.queries * a.group, r0 = tile * NR * 16;
  if (r0 >= rows) return;
  const int last = min(r0 + NR * 16, rows) - 1;
  const int begin = chunk * a.chunk_tokens;
  const int end = min(begin + a.chunk_tokens, kv4::visible(seq, last / a.group));
  if (chunk > 0 && begin >= end) return;     // the joining kernel leaves such chunks out
  const int all = min(kv4::visible(seq, r0 / a.group), seq.tokens);   // tokens every row of the tile sees

  h8v q[NR][W];
  float qs[NR], c1[NR];
  int limit[NR];
#pragma unroll
  for (int n = 0; n < NR; ++n) {
    const int r = min(r0 + 16 * n + l16, rows - 1), i = r / a.group;
    const uint16_t* src = a.q + (int64_t)(seq.first + i) * a.q_stride + (int64_t)(head * a.group + r - i * a.group) * D;
    load_query<T, W, true>(src + 8 * W * h, a.scale, q[n], qs[n], c1[n]);
    limit[n] = kv4::visible(seq, i);
  }

  struct Raw {
    uint32_t k[2][W], v[2][W];
    u32x4 kp[2], vp[2];
  };
  const int32_t* table = a.table + (int64_t)b * a.width;
  auto load = [&](Raw& x, int base) __attribute__((always_inline)) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int tok = base + 16 * t;
      const int page = kv4::page_id(table[kv4::table_column(tok, a.log_page, a.width)], a.pages);
      const int64_t row = kv4::row_index(page, head, a.heads, a.log_page, tok & ((1 << a.log_page) - 1));
      const uint32_t* k = reinterpret_cast<const uint32_t*>(a.k + row * (D / 2)) + l16 * (D / 8) + h * W;
      const uint32_t* v = reinterpret_cast<const uint32_t*>(a.v + row * (D / 2)) + h * (D / 2) + l16 * W;
      if constexpr (W == 2) {
        const u32x2 kk = *reinterpret_cast<const u32x2*>(k), vv = *reinterpret_cast<const u32x2*>(v);
#pragma unroll
        for (int j = 0; j < 2; ++j) x.k[t][j] = kk[j], x.v[t][j] = vv[j];
      } else {
#pragma unroll
        for (int g = 0; g < W / 4; ++g) {
          const u32x4 kk = *reinterpret_cast<const u32x4*>(k + 4 * g), vv = *reinterpret_cast<const u32x4*>(v + 4 * g);
#pragma unroll
          for (int j = 0; j < 4; ++j) x.k[t][4 * g + j] = kk[j], x.v[t][4 * g + j] = vv[j];
        }
      }
      x.kp[t] = *reinterpret_cast<const u32x4*>(a.k_par + row + 4 * h);
      x.vp[t] = *reinterpret_cast<const u32x4*>(a.v_par + row + 4 * h);
    }
  };

  f32x4 o[NR][NT], zs[NR];
  Stat st[NR];
  uint32_t top_v = 0;                        // parameter word of the largest value scale so far (E of its high half)
  float E = -24.0f;
#pragma unroll
  for (int n = 0; n < NR; ++n) {
    zs[n] = f32x4{};
#pragma unroll
    for (int i = 0; i < NT; ++i) o[n][i] = f32x4{};
    st[n] = Stat{kNegInf, 0.0f, 0.0f};
  }

  Raw cur, next;
  int base = begin + 32 * wave;
  if (base < end) load(cur, base);
  for (; base < end; base += 128) {
    if (base + 128 < end) load(next, base + 128);
    uint32_t word = 0;
    if (base + 32 > seq.tokens) {            // what lies behind the sequence's end is no number
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (base + 16 * t + 4 * h + r >= seq.tokens) cur.kp[t][r] = cur.vp[t][r] = 0;
    }
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) word = max(word, cur.vp[t][r]);
    const bool raise_v = __any(word > (top_v | 0xFFFFu));
    if (raise_v) {
      word = max(word, (uint32_t)__shfl_xor((int)word, 16));
      word = max(word, (uint32_t)__shfl_xor((int)word, 32));
      top_v = max(top_v, word);
    }
    const float newE = raise_v ? exponent_of(top_v) : E;

    h8v p[NR];
    const bool masked = base + 32 > all;
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      f32x4 s[2] = {};
#pragma unroll
      for (int w = 0; w < W; ++w)
#pragma unroll
        for (int t = 0; t < 2; ++t)
          s[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(unpack_keys(cur.k[t][w]), q[n][w], s[t], 0, 0, 0);
      float y[8], top = kNegInf;
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const uint32_t par = cur.kp[t][r];
          y[4 * t + r] = __builtin_fmaf(-low_half(par), qs[n], s[t][r]) * high_half(par);
        }
      if (masked) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (base + 16 * (j >> 2) + 4 * h + (j & 3) >= limit[n]) y[j] = kNegInf;
      }
#pragma unroll
      for (int j = 0; j < 8; j += 2) top = max3(top, y[j], y[j + 1]);
      if (__any(top > st[n].m) || raise_v) {
        const float m = __builtin_fmaxf(st[n].m, join_max<true>(top));
        const float ref = m == kNegInf ? 0.0f : __builtin_fmaf(c1[n], m, newE);
        const float f = st[n].m == kNegInf ? 0.0f : exp2_fast(st[n].ref - ref);
        st[n].m = m;
        st[n].ref = ref;
        st[n].l *= f;
        zs[n] *= f;
#pragma unroll
        for (int i = 0; i < NT; ++i) o[n][i] *= f;
      }
      float w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float e = exp2_fast(__builtin_fmaf(y[j], c1[n], -st[n].ref));
        st[n].l += e;
        w[j] = e * high_half(cur.vp[j >> 2][j & 3]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) p[n][j] = (_Float16)w[j];
    }
    E = newE;

    // zero points: rows of the first operand all alike, so every register of zs holds the same sum
    u32x4 zp;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int r = 0; r < 2; ++r)
        zp[2 * t + r] = __builtin_amdgcn_perm(cur.vp[t][2 * r + 1], cur.vp[t][2 * r], 0x05040100u);
#pragma unroll
    for (int n = 0; n < NR; ++n)
      zs[n] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8v, zp), p[n], zs[n], 0, 0, 0);
#pragma unroll
    for (int u = 0; u < W / 2; ++u) {
      const u32x4 lo = {cur.v[0][2 * u], cur.v[0][2 * u + 1], cur.v[1][2 * u], cur.v[1][2 * u + 1]};
      const u32x4 hi = lo >> 8;
      const u32x4 op[4] = {lo & 0x000F000Fu, lo & 0x00F000F0u, hi & 0x000F000Fu, hi & 0x00F000F0u};
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int n = 0; n < NR; ++n)
          o[n][4 * u + i] =
              __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8v, op[i]), p[n], o[n][4 * u + i], 0, 0, 0);
    }
    cur = next;
  }

  // Join the waves: everything to the largest reference (log2), then a tree over the sums.
#pragma unroll
  for (int n = 0; n < NR; ++n) {
    const float l = join_sum<true>(st[n].l);
    if (h == 0) {
      sm[wave][16 * n + l16] = st[n].m == kNegInf ? kNegInf : st[n].ref;
      sl[wave][16 * n + l16] = l;
    }
  }
  __syncthreads();
#pragma unroll
  for (int n = 0; n < NR; ++n) {
    float M = kNegInf, l = 0.0f;
#pragma unroll
    for (int v = 0; v < 4; ++v) M = __builtin_fmaxf(M, sm[v][16 * n + l16]);
#pragma unroll
    for (int v = 0; v < 4; ++v)
      if (M != kNegInf) l += sl[v][16 * n + l16] * exp2_fast(sm[v][16 * n + l16] - M);
    const float f = M == kNegInf ? 0.0f : exp2_fast(sm[wave][16 * n + l16] - M);
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        o[n][i][r] = f * __builtin_fmaf(o[n][i][r], i & 1 ? 0x1p20f : 0x1p24f, -zs[n][0]);
    if (n > 0) __syncthreads();              // the buffers of the row tile before
    if (wave >= 2)
#pragma unroll
      for (int i = 0; i < NT; ++i) so[wave - 2][i][lane] = o[n][i];
    __syncthreads();
    if (wave < 2)
#pragma unroll
      for (int i = 0; i < NT; ++i) o[n][i] += so[wave][i][lane];
    __syncthreads();
    if (wave == 1)
#pragma unroll
      for (int i = 0; i < NT; ++i) so[0][i][lane] = o[n][i];
    __syncthreads();
    if (wave == 0) {
#pragma unroll
      for (int i = 0; i < NT; ++i) o[n][i] += so[0][i][lane];
      const int r = r0 + 16 * n + l16;
      if (r < rows) {
        const int i = r / a.group;
        const int64_t id = (int64_t)(seq.first + i) * a.q_heads + head * a.group + r - i * a.group;
        if (a.chunks == 1) {
          const float inv = l > 0.0f ? 1.0f / l : 0.0f;
#pragma unroll
          for (int g = 0; g < 4; ++g)        // register g: channels NT * (4 h + g) .. + NT - 1
#pragma unroll
            for (int j = 0; j < NT; j += 4)
              *reinterpret_cast<u32x2*>(a.out + id * D + NT * (4 * h + g) + j) =
                  u32x2{pack2<T>(o[n][j][g] * inv, o[n][j + 1][g] * inv),
                        pack2<T>(o[n][j + 2][g] * inv, o[n][j + 3][g] * inv)};
        } else {
          const int64_t all_rows = (int64_t)a.total_q * a.q_heads;
          float* dst = a.part + (chunk * all_rows + id) * D;
#pragma unroll
          for (int g = 0; g < 4; ++g)
#pragma unroll
            for (int j = 0; j < NT; j += 4)
              *reinterpret_cast<f32x4*>(dst + NT * (4 * h + g) + j) =
                  f32x4{o[n][j][g], o[n][j + 1][g], o[n][j + 2][g], o[n][j + 3][g]};
          if (h == 0) {
            float* ml = a.part + a.chunks * all_rows * D + (chunk * all_rows + id) * 2;
            ml[0] = M;
            ml[1] = l;
          }
        }
      }
    }
  }
}

// ------------------------------------------------------------------ many query rows: bound by the vector ALUs and matrix cores
// One workgroup: 128 query rows of one sequence and kv head, 32 a wave, against a chunk of the tokens in
// tiles of 64.  The packed tile is staged in LDS once for the four waves (two buffers, the next tile's
// loads in registers meanwhile); each wave unpacks it for itself.
template <class T, int D>
__global__ __launch_bounds__(256) void prompt_kernel(Args a) {
  constexpr int S = D / 16;                  // K = 16 slices of the key product; a lane's words of a token row
  constexpr int NT = D / 32;                 // 32-channel tiles of the output
  constexpr int kRow = D / 2 + 16;           // staged key row: an odd number of 16-byte slots
  constexpr int PW = D / 32;                 // words of keys, and of values, that a thread stages
  constexpr int kTile = 64;
  __shared__ __attribute__((aligned(16))) uint8_t lk[2][kTile * kRow];
  __shared__ __attribute__((aligned(16))) uint8_t lv[2][kTile * D / 2];
  __shared__ __attribute__((aligned(16))) uint32_t lp[2][2][kTile];        // key, then value parameters

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
  const int rows = seq.queries * a.group, r0 = tile * 128;
  if (r0 >= rows) return;
  const int begin = chunk * a.chunk_tokens;
  const int end = min(begin + a.chunk_tokens, kv4::visible(seq, (min(r0 + 128, rows) - 1) / a.group));
  if (chunk > 0 && begin >= end) return;

  const int row = r0 + 32 * wave + l32, qi = min(row, rows - 1) / a.group;
  const int64_t id = (int64_t)(seq.first + qi) * a.q_heads + head * a.group + min(row, rows - 1) - qi * a.group;
  h8v q[S];
  float qs, c1;
  load_query<T, S, false>(a.q + (int64_t)(seq.first + qi) * a.q_stride +
                              (int64_t)(head * a.group + min(row, rows - 1) - qi * a.group) * D + 8 * S * h,
                          a.scale, q, qs, c1);
  const int limit = kv4::visible(seq, qi);
  // of this wave's rows: the tokens that all of them see, and that any of them sees
  const int w0 = min(r0 + 32 * wave, rows - 1), w1 = min(r0 + 32 * wave + 31, rows - 1);
  const int all = min(kv4::visible(seq, w0 / a.group), seq.tokens);
  const int any = r0 + 32 * wave < rows ? min(end, kv4::visible(seq, w1 / a.group)) : 0;

  // staging: thread t carries PW words of token t / 4's keys, PW words of 4-token block t / 16's values, and
  // (t < 128) one parameter word
  const int32_t* table = a.table + (int64_t)b * a.width;
  auto row_of = [&](int tok) __attribute__((always_inline)) {
    const int page = kv4::page_id(table[kv4::table_column(tok, a.log_page, a.width)], a.pages);
    return kv4::row_index(page, head, a.heads, a.log_page, tok & ((1 << a.log_page) - 1));
  };
  uint32_t gk[PW], gv[PW], gp = 0;
  auto copy = [&](uint32_t* dst, const uint32_t* src) __attribute__((always_inline)) {
    if constexpr (PW == 2) {
      *reinterpret_cast<u32x2*>(dst) = *reinterpret_cast<const u32x2*>(src);
    } else {
#pragma unroll
      for (int g = 0; g < PW; g += 4) *reinterpret_cast<u32x4*>(dst + g) = *reinterpret_cast<const u32x4*>(src + g);
    }
  };
  auto fetch = [&](int base) __attribute__((always_inline)) {
    const uint32_t* k = reinterpret_cast<const uint32_t*>(a.k + row_of(base + tid / 4) * (D / 2)) + (tid & 3) * PW;
    const uint32_t* v = reinterpret_cast<const uint32_t*>(a.v + row_of(base + tid / 16 * 4) * (D / 2)) + (tid & 15) * PW;
#pragma unroll
    for (int g = 0; g < PW; g += PW == 2 ? 2 : 4) {
      if constexpr (PW == 2) {
        const u32x2 kk = *reinterpret_cast<const u32x2*>(k), vv = *reinterpret_cast<const u32x2*>(v);
        gk[0] = kk[0], gk[1] = kk[1], gv[0] = vv[0], gv[1] = vv[1];
      } else {
        const u32x4 kk = *reinterpret_cast<const u32x4*>(k + g), vv = *reinterpret_cast<const u32x4*>(v + g);
#pragma unroll
        for (int j = 0; j < 4; ++j) gk[g + j] = kk[j], gv[g + j] = vv[j];
      }
    }
    if (tid < 128) {
      const int tok = base + (tid & 63);
      gp = (tid < 64 ? a.k_par : a.v_par)[row_of(tok)];
      if (tok >= seq.tokens) gp = 0;         // what lies behind the sequence's end is no number
    }
  };
  auto store = [&](int buf) __attribute__((always_inline)) {
    copy(reinterpret_cast<uint32_t*>(&lk[buf][(tid / 4) * kRow]) + (tid & 3) * PW, gk);
    copy(reinterpret_cast<uint32_t*>(&lv[buf][0]) + tid * PW, gv);
    if (tid < 128) lp[buf][tid >> 6][tid & 63] = gp;
  };

  f32x16 o[NT], zs = {};
#pragma unroll
  for (int i = 0; i < NT; ++i) o[i] = f32x16{};
  Stat st{kNegInf, 0.0f, 0.0f};
  uint32_t top_v = 0;
  float E = -24.0f;

  if (begin < end) {
    fetch(begin);
    store(0);
  }
  __syncthreads();
  int buf = 0;
  for (int base = begin; base < end; base += kTile, buf ^= 1) {
    if (base + kTile < end) fetch(base + kTile);
    if (base < any) {
      const uint32_t word = lp[buf][1][lane];
      const bool raise_v = __any(word > (top_v | 0xFFFFu));
      if (raise_v) {
        uint32_t w = word;
#pragma unroll
        for (int d = 32; d; d >>= 1) w = max(w, (uint32_t)__shfl_xor((int)w, d));
        top_v = max(top_v, w);
      }
      const float newE = raise_v ? exponent_of(top_v) : E;
      float y[32];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        f32x16 s = {};
        const uint32_t* k = reinterpret_cast<const uint32_t*>(&lk[buf][(32 * t + l32) * kRow]) + h * S;
#pragma unroll
        for (int w = 0; w < S; w += 4) {
          const u32x4 kk = *reinterpret_cast<const u32x4*>(k + w);
#pragma unroll
          for (int j = 0; j < 4; ++j) s = __builtin_amdgcn_mfma_f32_32x32x16_f16(unpack_keys(kk[j]), q[w + j], s, 0, 0, 0);
        }
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const u32x4 par = *reinterpret_cast<const u32x4*>(&lp[buf][0][32 * t + 8 * g + 4 * h]);
#pragma unroll
          for (int r = 0; r < 4; ++r)
            y[16 * t + 4 * g + r] = __builtin_fmaf(-low_half(par[r]), qs, s[4 * g + r]) * high_half(par[r]);
        }
      }
      if (base + kTile > all) {
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (base + 32 * (j >> 4) + 8 * ((j >> 2) & 3) + 4 * h + (j & 3) >= limit) y[j] = kNegInf;
      }
      float top = kNegInf;
#pragma unroll
      for (int j = 0; j < 32; j += 2) top = max3(top, y[j], y[j + 1]);
      if (__any(top > st.m) || raise_v) {
        const float m = __builtin_fmaxf(st.m, join_max<false>(top));
        const float ref = m == kNegInf ? 0.0f : __builtin_fmaf(c1, m, newE);
        const float f = st.m == kNegInf ? 0.0f : exp2_fast(st.ref - ref);
        st.m = m;
        st.ref = ref;
        st.l *= f;
        zs *= f;
#pragma unroll
        for (int i = 0; i < NT; ++i) o[i] *= f;
      }
      E = newE;
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int x = 0; x < 2; ++x) {        // 16 tokens: blocks 4 x + h and 4 x + 2 + h of the 32
          h8v p;
          u32x4 zp;
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            const u32x4 par = *reinterpret_cast<const u32x4*>(&lp[buf][1][32 * t + 16 * x + 8 * g + 4 * h]);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const float e = exp2_fast(__builtin_fmaf(y[16 * t + 8 * x + 4 * g + r], c1, -st.ref));
              st.l += e;
              p[4 * g + r] = (_Float16)(e * high_half(par[r]));
            }
            zp[2 * g] = __builtin_amdgcn_perm(par[1], par[0], 0x05040100u);
            zp[2 * g + 1] = __builtin_amdgcn_perm(par[3], par[2], 0x05040100u);
          }
          zs = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(h8v, zp), p, zs, 0, 0, 0);
          const uint8_t* b0 = &lv[buf][(8 * t + 4 * x + h) * 2 * D];
          const uint8_t* b1 = b0 + 4 * D;
          if constexpr (D == 64) {           // half a quad a lane: channels 2 l32, 2 l32 + 1
            const u32x2 v0 = *reinterpret_cast<const u32x2*>(b0 + 8 * (l32 >> 1));
            const u32x2 v1 = *reinterpret_cast<const u32x2*>(b1 + 8 * (l32 >> 1));
            const u32x4 w = u32x4{v0[0], v0[1], v1[0], v1[1]} >> (8 * (l32 & 1));
            o[0] = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(h8v, w & 0x000F000Fu), p, o[0], 0, 0, 0);
            o[1] = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(h8v, w & 0x00F000F0u), p, o[1], 0, 0, 0);
          } else {
#pragma unroll
            for (int u = 0; u < NT / 4; ++u) {
              const u32x2 v0 = *reinterpret_cast<const u32x2*>(b0 + 8 * ((NT / 4) * l32 + u));
              const u32x2 v1 = *reinterpret_cast<const u32x2*>(b1 + 8 * ((NT / 4) * l32 + u));
              const u32x4 lo = {v0[0], v0[1], v1[0], v1[1]}, hi = lo >> 8;
              const u32x4 op[4] = {lo & 0x000F000Fu, lo & 0x00F000F0u, hi & 0x000F000Fu, hi & 0x00F000F0u};
#pragma unroll
              for (int i = 0; i < 4; ++i)
                o[4 * u + i] =
                    __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(h8v, op[i]), p, o[4 * u + i], 0, 0, 0);
            }
          }
        }
    }
    if (base + kTile < end) store(buf ^ 1);
    __syncthreads();
  }

  const float l = join_sum<false>(st.l);
  if (row >= rows) return;
  const int64_t all_rows = (int64_t)a.total_q * a.q_heads;
  if (a.chunks > 1 && h == 0) {
    float* ml = a.part + a.chunks * all_rows * D + (chunk * all_rows + id) * 2;
    ml[0] = st.m == kNegInf ? kNegInf : st.ref;
    ml[1] = l;
  }
  const float inv = a.chunks > 1 ? 1.0f : l > 0.0f ? 1.0f / l : 0.0f;
#pragma unroll
  for (int g = 0; g < 16; ++g) {             // register g: channels NT * (8 (g / 4) + 4 h + g % 4) .. + NT - 1
    const int d = NT * (8 * (g >> 2) + 4 * h + (g & 3));
    float x[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) x[i] = inv * __builtin_fmaf(o[i][g], i & 1 ? 0x1p20f : 0x1p24f, -zs[0]);
    if (a.chunks > 1) {
      float* dst = a.part + (chunk * all_rows + id) * D + d;
#pragma unroll
      for (int i = 0; i < NT; i += 2) *reinterpret_cast<float2*>(dst + i) = float2{x[i], x[i + 1]};
    } else {
#pragma unroll
      for (int i = 0; i < NT; i += 2) *reinterpret_cast<uint32_t*>(a.out + id * D + d + i) = pack2<T>(x[i], x[i + 1]);
    }
  }
}

// ------------------------------------------------------------------ joining the chunks of a divided sequence
// One wave per query row: the chunks' sums, each scaled to the largest reference, in chunk order.
template <class T, int D>
__global__ __launch_bounds__(256) void join_kernel(Args a) {
  constexpr int C = D / 64;
  const int lane = threadIdx.x & 63;
  const int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int most = a.max_q * a.group;
  const int bh = (int)(w / most), r = (int)(w - (int64_t)bh * most);
  if (bh >= a.batch * a.heads) return;
  const int b = bh / a.heads, head = bh - b * a.heads;
  const kv4::Sequence seq = kv4::sequence(a.q_start[b], a.q_start[b + 1], a.lens[b], a.total_q, a.max_q, a.max_len,
                                          a.width << a.log_page);
  if (r >= seq.queries * a.group) return;
  const int i = r / a.group, n = kv4::visible(seq, i);
  const int64_t id = (int64_t)(seq.first + i) * a.q_heads + head * a.group + r - i * a.group;
  const int64_t all_rows = (int64_t)a.total_q * a.q_heads;
  const int chunks = (n + a.chunk_tokens - 1) / a.chunk_tokens;          // those that hold a token of this row
  const float* ml = a.part + a.chunks * all_rows * D + id * 2;
  float M = kNegInf, l = 0.0f;
  if (lane < chunks) {
    M = ml[lane * all_rows * 2];
    l = ml[lane * all_rows * 2 + 1];
  }
  float top = M;
#pragma unroll
  for (int d = 32; d; d >>= 1) top = __builtin_fmaxf(top, __shfl_xor(top, d));
  const float f = M == kNegInf ? 0.0f : exp2_fast(M - top);
  l *= f;
#pragma unroll
  for (int d = 32; d; d >>= 1) l += __shfl_xor(l, d);
  float x[C] = {};
  for (int c = 0; c < chunks; ++c) {
    const float g = __shfl(f, c);
    const float* src = a.part + (c * all_rows + id) * D + lane * C;
#pragma unroll
    for (int j = 0; j < C; ++j) x[j] += g * src[j];
  }
  const float inv = l > 0.0f ? 1.0f / l : 0.0f;
#pragma unroll
  for (int j = 0; j < C; ++j) a.out[id * D + lane * C + j] = T::store(x[j] * inv);
}

constexpr int kMaxChunks = 64;               // one lane of the joining wave each

template <class T, int D>
void launch(const Args& a, int kind, hipStream_t st) {
  const dim3 grid((unsigned)((int64_t)a.batch * a.heads * a.row_tiles * a.chunks));
  if (kind == 1)
    hipLaunchKernelGGL((decode_kernel<T, D, 1>), grid, dim3(256), 0, st, a);
  else if (kind == 2)
    hipLaunchKernelGGL((decode_kernel<T, D, 2>), grid, dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL((prompt_kernel<T, D>), grid, dim3(256), 0, st, a);
  if (a.chunks > 1) {
    const int64_t waves = (int64_t)a.batch * a.heads * a.max_q * a.group;
    hipLaunchKernelGGL((join_kernel<T, D>), dim3((unsigned)((waves + 3) / 4)), dim3(256), 0, st, a);
  }
}

}  // namespace

// kind 1, 2: decode_kernel with one or two tiles of 16 rows; 3: prompt_kernel.
Kv4Plan kv4_plan(int total_q, int q_heads, int heads, int dim, int batch, int max_q, int max_len) {
  const int64_t rows = (int64_t)max_q * (q_heads / heads);
  Kv4Plan p;
  p.kind = rows <= 16 ? 1 : rows <= 32 ? 2 : 3;
  const int per = p.kind == 3 ? 128 : 16 * p.kind;
  p.row_tiles = (int)((rows + per - 1) / per);
  // workgroups without division, against four (two) a compute unit
  const int64_t groups = (int64_t)batch * heads * p.row_tiles;
  const int64_t want = p.kind == 3 ? 512 : 1024;
  const int step = 128;
  int64_t chunks = (want + groups - 1) / groups;
  chunks = chunks < 1 ? 1 : chunks > kMaxChunks ? kMaxChunks : chunks;
  const int64_t tokens = (max_len + chunks - 1) / chunks;
  p.chunk_tokens = (int)((tokens + step - 1) / step * step);
  p.chunks = max_len < 1 ? 1 : (max_len + p.chunk_tokens - 1) / p.chunk_tokens;
  return p;
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
