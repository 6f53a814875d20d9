// Host side of the C ABI declared in include/atom_kv4_pages.h: argument validation (all of it before any HIP call),
// then the launches on the caller's stream.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "atom_kv4_pages.h"
#include "host_checks.h"
#include "serve_internal.h"

namespace {

using namespace atom::check;

bool valid_state(int32_t batch, int32_t width, int32_t page, int32_t capacity) {
  return batch >= 1 && batch <= (1 << 20) && width >= 1 && page >= 16 && page <= 256 && (page & (page - 1)) == 0 &&
         (uint64_t)width * (uint64_t)page <= ((uint64_t)1 << 30) && capacity >= 1 && capacity <= (1 << 27);
}

}  // namespace

extern "C" {

int atom_kv4_extend(const int32_t* lens, const int32_t* new_tokens, int32_t* table, int32_t batch, int32_t width, int32_t page,
                    const int32_t* free_pages, int32_t capacity, const int32_t* state, int64_t* slots, int32_t total,
                    int32_t* start, int32_t* lens_out, int32_t* state_out, void* stream) {
  if (!lens || !new_tokens || !table || !free_pages || !state || !slots || !start || !lens_out || !state_out) return ATOM_E_NULL;
  if (!valid_state(batch, width, page, capacity) || !valid_rows(total)) return ATOM_E_SHAPE;
  if (!aligned(lens, 4) || !aligned(new_tokens, 4) || !aligned(table, 4) || !aligned(free_pages, 4) || !aligned(state, 4) ||
      !aligned(slots, 8) || !aligned(start, 4) || !aligned(lens_out, 4) || !aligned(state_out, 4))
    return ATOM_E_ALIGN;
  const uint64_t b = (uint64_t)batch * 4;
  const Range in[4] = {range_of(new_tokens, b), range_of(free_pages, (uint64_t)capacity * 4),
                       range_of(lens, lens_out == lens ? 0 : b), range_of(state, state_out == state ? 0 : 8)};
  const Range out[5] = {range_of(table, b * (uint64_t)width), range_of(slots, (uint64_t)total * 8), range_of(start, b + 4),
                        range_of(lens_out, b), range_of(state_out, 8)};
  if (int s = check_overlap(in, 4, out, 5)) return s;
  const atom::Kv4Extend a = {lens, new_tokens, table, batch, width, __builtin_ctz(page), free_pages, capacity, state, slots,
                             total, start, lens_out, state_out};
  return hip_status(atom::launch_kv4_extend(a, static_cast<hipStream_t>(stream)));
}

int atom_kv4_release(const uint8_t* done, const int32_t* lens, const int32_t* table, int32_t batch, int32_t width,
                     int32_t page, int32_t* free_pages, int32_t capacity, const int32_t* state, int32_t* lens_out,
                     int32_t* state_out, void* stream) {
  if (!done || !lens || !table || !free_pages || !state || !lens_out || !state_out) return ATOM_E_NULL;
  if (!valid_state(batch, width, page, capacity)) return ATOM_E_SHAPE;
  if (!aligned(lens, 4) || !aligned(table, 4) || !aligned(free_pages, 4) || !aligned(state, 4) || !aligned(lens_out, 4) ||
      !aligned(state_out, 4))
    return ATOM_E_ALIGN;
  const uint64_t b = (uint64_t)batch * 4;
  const Range in[4] = {range_of(done, (uint64_t)batch), range_of(table, b * (uint64_t)width),
                       range_of(lens, lens_out == lens ? 0 : b), range_of(state, state_out == state ? 0 : 8)};
  const Range out[3] = {range_of(free_pages, (uint64_t)capacity * 4), range_of(lens_out, b), range_of(state_out, 8)};
  if (int s = check_overlap(in, 4, out, 3)) return s;
  const atom::Kv4Release a = {done, lens, table, batch, width, __builtin_ctz(page), free_pages, capacity, state, lens_out,
                              state_out};
  return hip_status(atom::launch_kv4_release(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
