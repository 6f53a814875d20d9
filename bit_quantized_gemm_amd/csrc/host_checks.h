// Argument checks shared by the host APIs of the serving operators; all of them run before any HIP call.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "atom_w8a8.h"

namespace atom {
namespace check {

struct Range {
  uintptr_t lo, hi;   // [lo, hi)
};

inline Range range_of(const void* p, uint64_t bytes) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return Range{a, a + (uintptr_t)bytes};
}

inline bool overlap(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi; }

// Every output must be disjoint from every input and from the other outputs.
inline int check_overlap(const Range* in, int n_in, const Range* out, int n_out) {
  for (int o = 0; o < n_out; ++o) {
    for (int i = 0; i < n_in; ++i)
      if (overlap(out[o], in[i])) return ATOM_E_OVERLAP;
    for (int p = o + 1; p < n_out; ++p)
      if (overlap(out[o], out[p])) return ATOM_E_OVERLAP;
  }
  return ATOM_OK;
}

inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline bool aligned16(const void* p) { return aligned(p, 16); }
inline bool valid_dtype(int32_t t) { return t == ATOM_FP16 || t == ATOM_BF16; }
inline bool valid_rows(int32_t r) { return r >= 1 && r <= ATOM_MAX_ROWS; }
inline int hip_status(hipError_t e) { return e == hipSuccess ? ATOM_OK : ATOM_E_HIP; }
inline uint64_t up16(uint64_t n) { return (n + 15) & ~(uint64_t)15; }

// ---- 16-bit rows of any K, ldx elements apart
inline bool valid_k8(int32_t K) { return K >= 1 && K <= ATOM_MAX_K; }
inline uint64_t row_bytes8(int32_t K) { return ((uint64_t)K + 127) / 128 * 128; }
inline bool valid_gemm8(int32_t M, int32_t N, int32_t K) {
  if (!valid_k8(K) || !valid_rows(M) || !valid_rows(N)) return false;
  return (uint64_t)((M + 127) / 128) * (uint64_t)((N + 127) / 128) <= ATOM_MAX_TILES;
}
inline bool valid_x(const void* X, int64_t ldx, int32_t rows, int32_t K) {
  return aligned(X, 2) && (rows == 1 || (ldx >= K && ldx <= ((int64_t)1 << 40)));
}
inline uint64_t x_bytes(int64_t ldx, int32_t rows, int32_t K) {
  return rows == 1 ? (uint64_t)K * 2 : ((uint64_t)(rows - 1) * (uint64_t)ldx + (uint64_t)K) * 2;
}

}  // namespace check
}  // namespace atom
