/*
 * atom_kv4.h -- C ABI of the 4-bit KV cache on MI355X (gfx950): appending keys and values to its
 * pages, reading them back, and causal attention over it.
 *
 * The cache is four device arrays over `pages` pages of `page` tokens, for H kv heads of D channels:
 *   k     : uint8 [pages, H, page, D/2]         codes of the keys, channel 2j in the low nibble of byte j
 *   v     : uint8 [pages, H, page/4, D/4, 8]    codes of the values, four tokens interleaved: channel d of
 *                                               token t is in byte 4 ((t % 4) / 2) + 2 (t % 2) + (d % 4) / 2
 *                                               of [t / 4, d / 4], the low nibble for even d
 *   k_par, v_par : fp16 [pages, H, page, 2]     (zero point, scale) of a token's key / value in one head
 * A code q stands for scale * (q - zero).  For a head's D channels x of one token,
 *   lo = min(min x, 0), hi = max(max x, 0), scale = fp16_rne(fl32(min((hi - lo) / 15, 65504))),
 *   zero = clamp(rint_even(fl32(-lo / scale)), 0, 15), q = clamp(rint_even(fl32(x / scale)) + zero, 0, 15),
 *   and all three are 0 where scale = 0.
 * Whoever fills the arrays without the append below keeps to that: zero points are whole numbers from 0 to 15, scales finite
 * and not negative.  Attention's results for other parameters are unspecified (no fault).
 *
 * Shapes: D is 64, 128 or 256; page is a power of two from 16 to 256; 1 <= H <= 1024;
 * 1 <= pages < 2^31 / page; fp16 or bf16 keys, values and queries (`dtype`, as in atom_w8a8.h).  The
 * conventions of atom.h hold: device pointers of the caller, 16-byte aligned (table, lens, q_start and
 * slots: aligned to their elements), no allocation, no synchronization, ATOM_E_* from checks on the host.
 */
#ifndef ATOM_KV4_H_
#define ATOM_KV4_H_

#include <stdint.h>

#include "atom_w8a8.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The cache's arrays and sizes. */
typedef struct {
  void *k, *k_par, *v, *v_par;
  int32_t pages, page, heads, dim;
} atom_kv4_cache;

/*
 * Append: the key and value of token i go to slot slots[i] = page index * page + place in the page.
 * A slot outside the cache (such as -1) skips its token, so padded batches need no second shape.
 * Two tokens of one call must not share a slot.  Rows that hold an inf or NaN get unspecified codes.
 *   K, V  : const fp16 / bf16 [tokens, H, D]; rows of H * D contiguous elements, k_stride / v_stride
 *           elements apart (multiples of 8)
 *   slots : const int64 [tokens]
 */
int atom_kv4_append(const void *K, int64_t k_stride, const void *V, int64_t v_stride, const int64_t *slots,
                    int32_t tokens, int32_t dtype, const atom_kv4_cache *cache, void *stream);

/*
 * Read back: what the codes in slots[i] stand for, rounded once, contiguous; zeros for a slot outside
 * the cache.
 *   K, V : fp16 / bf16 [tokens, H, D]                                         (outputs)
 */
int atom_kv4_read(const atom_kv4_cache *cache, const int64_t *slots, int32_t tokens, int32_t dtype, void *K, void *V,
                  void *stream);

/*
 * Causal attention of the last tokens of each of `batch` sequences over their pages.
 *   Q       : const fp16 / bf16 [total_q, Hq, D], rows q_stride elements apart (a multiple of 8); Hq is a
 *             multiple of H, query head j reads kv head j / (Hq / H)
 *   table   : const int32 [batch, width]: page of the sequence's tokens page * i .. page * i + page - 1
 *   lens    : const int32 [batch]: tokens of the sequence in the cache, its queries' own included
 *   q_start : const int32 [batch + 1]: sequence b's queries are rows q_start[b] .. q_start[b + 1] - 1
 *   out     : fp16 / bf16 [total_q, Hq, D] contiguous                         (output)
 * Query i of n sees the tokens 0 .. lens[b] - n + i; one that sees none gets zeros.  Rows outside every
 * sequence are left as they were.  out = softmax(scale * q . k) v with fp32 statistics and sums; scale > 0.
 * A token's weight times its value scale is rounded to fp16 with the largest such product that the query sees as its unit
 * (2^-11 of it; products below 2^-18 of the largest: to steps of 2^-28 of the largest; a scale below 2^-14 counts as 2^-14
 * in that unit).
 * max_q and max_len bound the sequences' queries and tokens on the host.  Queries behind max_q are left out (their rows
 * stay as they were; the others see what they would).  A length above max_len, or above what `width` pages hold, is taken as
 * that: the sequence ends there, and its last query sees its last token.  batch * H * ceil(max_q * Hq / H / 128) must stay
 * below 2^24, the largest launch.  Entries of lens, q_start and table outside their ranges are clamped into them (garbage out,
 * no fault).  What lies in the pages behind a sequence's end is never used in a result.
 * workspace: atom_kv4_attention_workspace_bytes(...) bytes (0 when none is needed) let long sequences be
 * divided among workgroups; with less (or NULL) they run undivided.  Contents on entry do not matter;
 * calls that may overlap in time need one each.
 */
int64_t atom_kv4_attention_workspace_bytes(int32_t total_q, int32_t q_heads, int32_t heads, int32_t dim,
                                           int32_t batch, int32_t max_q, int32_t max_len);
int atom_kv4_attention(const void *Q, int64_t q_stride, const atom_kv4_cache *cache, const int32_t *table,
                       int32_t width, const int32_t *lens, const int32_t *q_start, int32_t total_q, int32_t q_heads,
                       int32_t batch, int32_t max_q, int32_t max_len, float scale, int32_t dtype, void *out,
                       void *workspace, int64_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* ATOM_KV4_H_ */
