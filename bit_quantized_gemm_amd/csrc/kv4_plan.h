// How attention over the 4-bit KV cache is launched: plain arithmetic on a call's sizes, shared by the host code and
// by a host test that pins the kernel each shape takes.
#pragma once

#include <stdint.h>

#include <initializer_list>

namespace kv4 {

enum Kind { kFour = 1, kEight = 2, kPrompt = 3 };
constexpr int kMaxChunks = 64;               // one lane of the joining wave each
constexpr int kMaxGroups = 1 << 24;          // workgroups that no launch reaches: it has less than 2^32 threads, 256 each

// Query rows (query tokens x query heads of one kv head) tiles of a sequence and kv head, and the tokens of one chunk of a
// sequence; chunks > 1 need scratch.
struct Plan {
  int kind, row_tiles, chunks, chunk_tokens;
};

// How a call is run: decode_kernel (16 rows a workgroup) or prompt_kernel (128), and in how many chunks a sequence is divided
// (joined by a second kernel; not below 256 tokens a chunk).
//
// Up to 16 rows a sequence and kv head: decode_kernel in eight waves (kEight), four (kFour) from 512 workgroups on; divided until
// there are 256 workgroups, but not up to 1024 tokens, which eight waves walk through in four steps.  Measured (one call,
// 256 compute units): 16 sequences of 2048 tokens, 32 kv heads: 26.0 us whole in four waves, 26.1 in eight, 29.6 divided in two; 4
// of 32768, 8 kv heads: 30.1 in 8 chunks, 30.7 in 16, 36.3 in 24; 16 of 4096 with 16 heads of 64 channels: 17.8 whole in eight
// waves, 22.8 in four; one of 700: 6.9 whole, 9.1 divided.
//
// More rows: the least of these estimates (us; a round fills the compute units with four workgroups of decode_kernel or two of
// prompt_kernel, half as many of 256 channels):
//   decode_kernel: 2, 5 a round, and for each 128 tokens (a unit a wave) 2.0, 1.2 or 0.85 with the units full, half or a quarter full
//   prompt_kernel: 3.5, 5 a round, and for each 64 tokens 2.45 or 1.55 with the units full or half full; 1.55 for the longest
//   joining: 4, 0.4 for 1000 rows, and the partial sums' way through memory.
// Measured (us), decode_kernel and prompt_kernel whole, and the best of both divided: 16 sequences of 2048 tokens, 8 kv heads of 128
// channels, 80 rows each: 36, 56, 38; 256 rows: 72, 58, 68; one sequence of 8192, 512 rows: 50, 189, 42; prompts of 2 x 1600 tokens, 32
// heads: 115, 76, 124; 4 x 1000, 4 kv heads of 256 channels, 400 rows: 24, 58, 36.  Over 37 shapes the choice is within 11% of the
// best of all kinds and divisions, within 5% on 32.
inline Plan plan(int q_heads, int heads, int dim, int batch, int max_q, int max_len, int cus) {
  const int64_t rows = (int64_t)max_q * (q_heads / heads);
  auto make = [&](int kind, int64_t chunks) {
    Plan p;
    p.kind = kind;
    const int per = kind == kPrompt ? 128 : 16;
    p.row_tiles = (int)((rows + per - 1) / per);
    const int64_t tokens = (max_len + chunks - 1) / chunks;
    p.chunk_tokens = (int)((tokens + 255) / 256 * 256);
    p.chunks = (max_len + p.chunk_tokens - 1) / p.chunk_tokens;
    return p;
  };
  const int64_t pairs = (int64_t)batch * heads;
  if (rows <= 16) {
    const int64_t chunks = pairs >= 512 || max_len <= 1024 ? 1 : (256 + pairs - 1) / pairs;
    return make(pairs >= 512 ? kFour : kEight, chunks > kMaxChunks ? kMaxChunks : chunks);
  }
  const double all = (double)pairs * rows;
  const double seen = max_len > max_q ? max_len - 0.5 * max_q : 0.5 * max_len;   // tokens that a row sees, on average
  Plan best = make(kPrompt, 1);
  double least = -1.0;
  for (int kind : {kFour, kPrompt}) {
    const int slots = (kind == kFour ? 4 : 2) / (dim == 256 ? 2 : 1);
    const double narrow = dim > 64 ? 1.0 : kind == kFour ? 0.55 : 0.75, wide = kind == kPrompt && dim == 256 ? 2.0 : 1.0;
    for (int64_t want = 1; want <= kMaxChunks; want += want < 8 ? 1 : want / 4) {
      const Plan p = make(kind, want);
      if (p.chunks > 1 && all >= 1 << 24) continue;        // more rows than a launch of the joining kernel has workgroups
      const double groups = (double)pairs * p.row_tiles * p.chunks;
      if (groups >= kMaxGroups) continue;
      const double full = (double)(int64_t)(groups / (slots * cus)), rest = (groups - full * slots * cus) / cus;
      double time;
      if (kind == kFour) {
        const double last = rest == 0.0 ? 0.0 : 4 * rest <= slots ? 0.85 : 2 * rest <= slots ? 1.2 : 2.0;
        time = 2.0 + 5.0 * (full + (rest > 0.0)) + narrow * (seen / p.chunks / 128 + 0.5) * (full * 2.0 + last);
      } else {
        const double last = rest == 0.0 ? 0.0 : 2 * rest <= slots || slots == 1 ? 1.55 : 2.45;
        const double steps = seen / p.chunks / 64 + 0.5, most = (double)max_len / p.chunks / 64 * 1.55;
        time = steps * (full * (slots == 1 ? 1.55 : 2.45) + last);
        time = 3.5 + 5.0 * (full + (rest > 0.0)) + narrow * wide * (time > most ? time : most);
      }
      if (p.chunks > 1) time += 4.0 + 0.4e-3 * all + all * p.chunks * dim * 8 / 5e6;
      if (least < 0.0 || time < least) {
        least = time;
        best = p;
      }
    }
  }
  return best;
}

}  // namespace kv4
