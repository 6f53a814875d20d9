// Addresses in the 4-bit KV cache (atom_kv4.h), and the clamps that keep every access inside it
// whatever the block tables, lengths and slots hold.  Plain arithmetic, shared by the kernels and
// by a host test that walks it over bad inputs.
#pragma once

#include <stdint.h>

#ifdef __HIPCC__
#define KV4_FN __host__ __device__ inline __attribute__((always_inline))
#else
#define KV4_FN static inline
#endif

namespace kv4 {

// Row (page, head, token in page) of the cache for a slot: the index of its (zero, scale) pair, and
// in units of D/2 bytes that of its key codes.
KV4_FN int64_t row_index(int64_t page_id, int head, int heads, int log_page, int in_page) {
  return ((page_id * heads + head) << log_page) + in_page;
}
// Whether a slot lies in the cache.
KV4_FN bool valid_slot(int64_t slot, int pages, int log_page) {
  return slot >= 0 && (slot >> log_page) < pages;
}
// Byte of the value codes of 4-token block `block` (of its page) in one (page, head).
KV4_FN int64_t value_block(int64_t page_id, int head, int heads, int log_page, int dim, int block) {
  return (((page_id * heads + head) << log_page) + 4 * (int64_t)block) * (dim / 2);
}
// Within a block: byte of the two bytes that hold channels 4 quad .. 4 quad + 3 of token t (0 .. 3).
KV4_FN int value_in_block(int quad, int t) { return 8 * quad + 4 * (t >> 1) + 2 * (t & 1); }

// Page id from a table entry, clamped into the pool.
KV4_FN int page_id(int entry, int pages) { return entry < 0 ? 0 : entry >= pages ? pages - 1 : entry; }
// Table column of a token, clamped into the table's width.
KV4_FN int table_column(int token, int log_page, int width) {
  const int c = token >> log_page;
  return c < width ? c : width - 1;
}

// A sequence's queries and tokens after clamping: rows first .. first + queries - 1 of Q, tokens in [0, limit].
struct Sequence {
  int first, queries, tokens;
  int behind;   // queries of the sequence before clamping to max_q: query i sees tokens 0 .. tokens - behind + i
};
KV4_FN Sequence sequence(int start, int end, int len, int total_q, int max_q, int max_len, int capacity) {
  Sequence s;
  s.first = start < 0 ? 0 : start > total_q ? total_q : start;
  int e = end < s.first ? s.first : end > total_q ? total_q : end;
  s.behind = e - s.first;
  s.queries = s.behind < max_q ? s.behind : max_q;
  const int most = max_len < capacity ? max_len : capacity;
  s.tokens = len < 0 ? 0 : len > most ? most : len;
  return s;
}
// Tokens that query i sees (0 when it sees none).
KV4_FN int visible(const Sequence& s, int i) {
  const int n = s.tokens - s.behind + i + 1;
  return n < 0 ? 0 : n;
}

}  // namespace kv4
