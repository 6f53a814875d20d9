// How the W8A8 row quantize is launched: plain arithmetic, shared by the host code and by a host test.
#pragma once

#include <stdint.h>

namespace atom {
namespace w8a8 {

// Threads that share a row, and the chunks of eight elements that each of them holds.
struct RowShape {
  int threads, chunks;
};
inline RowShape row_shape(int64_t rows, int Kp) {
  if (Kp <= 512) return {64, 1};
  if (Kp <= 2048) return rows <= 384 ? RowShape{256, 1} : RowShape{64, 4};
  if (Kp <= 4096) return {256, 2};
  if (Kp <= 8192) return rows <= 1024 ? RowShape{512, 2} : RowShape{256, 4};
  if (Kp <= 16384) return {512, 4};
  return {1024, 8};
}

constexpr int block_threads(int threads) { return threads <= 64 ? 256 : threads; }
// Rows of one launch, which has less than 2^32 threads: more rows take more launches.
constexpr int64_t launch_rows(int threads) {
  return (((int64_t)1 << 32) - 1) / block_threads(threads) * (block_threads(threads) / threads);
}

}  // namespace w8a8
}  // namespace atom
