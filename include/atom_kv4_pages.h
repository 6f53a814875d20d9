/*
 * atom_kv4_pages.h -- C ABI of the 4-bit KV cache's bookkeeping on MI355X (gfx950): block tables, slots
 * and a pool of free pages, kept on the device, so that a captured step can admit tokens and
 * finish sequences without the host.
 *
 * State of `batch` sequences: lens int32 [batch] (tokens in the cache), table int32 [batch, width] (their pages, as
 * atom_kv4_attention reads it) and a pool of free pages: free int32 [capacity], the first state[0] of
 * which are free, the next one to be taken last; state int32 [2] = (free pages, pages missing).
 *
 * Values are clamped into range before use, so that no content faults: lengths into [0, width * page], new
 * tokens to at least 0, state[0] into [0, capacity], page ids below 0 give no slots.
 *
 * The conventions of atom.h hold; pointers are aligned to their elements.  page is a power of two from 16 to
 * 256, width * page at most 2^30, batch and capacity at most 2^20 and 2^27.  Calls on one state follow each other on
 * one stream (or are ordered by its events).
 */
#ifndef ATOM_KV4_PAGES_H_
#define ATOM_KV4_PAGES_H_

#include <stdint.h>

#include "atom_kv4.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Extend: sequence b gains new[b] tokens.  The tokens of all sequences lie one sequence behind the other in
 * `total` rows; what does not fit into them is not taken (start[b] = min(sum of new[0 .. b-1], total)).
 * Pages are taken for tokens that no page of the sequence holds yet, in the order of the sequences, and
 * written behind the table's last ones.  Where the pool holds too few, nothing is taken at all: every slot is
 * -1, lengths, table and pool stay, and the number of pages missing is written to state_out[1] (0 otherwise).
 *   new       : const int32 [batch]
 *   slots     : int64 [total]      slot of each new token, as atom_kv4_append takes them; -1 for rows behind
 *                                  the last one and for tokens behind width * page            (output)
 *   start     : int32 [batch + 1]  first row of each sequence, as atom_kv4_attention's q_start  (output)
 *   lens_out  : int32 [batch]      lengths with the new tokens, at most width * page            (output)
 *   state_out : int32 [2]          (free pages left, pages missing)                             (output)
 * lens_out may be lens and state_out may be state; other outputs overlap nothing.
 */
int atom_kv4_extend(const int32_t *lens, const int32_t *new_tokens, int32_t *table, int32_t batch, int32_t width, int32_t page,
                    const int32_t *free_pages, int32_t capacity, const int32_t *state, int64_t *slots, int32_t total,
                    int32_t *start, int32_t *lens_out, int32_t *state_out, void *stream);

/*
 * Release: the pages of every sequence with done[b] != 0 return to the pool, in the order of the sequences
 * and of their tables, and its length becomes 0.  Pages beyond the pool's capacity (given back twice) are dropped.
 *   done      : const uint8 [batch]
 *   lens_out, state_out : as above; free_pages is written from state[0] on        (outputs)
 */
int atom_kv4_release(const uint8_t *done, const int32_t *lens, const int32_t *table, int32_t batch, int32_t width,
                     int32_t page, int32_t *free_pages, int32_t capacity, const int32_t *state, int32_t *lens_out,
                     int32_t *state_out, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* ATOM_KV4_PAGES_H_ */
