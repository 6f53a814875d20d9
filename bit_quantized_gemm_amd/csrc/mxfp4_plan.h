// How MXFP4 products are run: plain arithmetic on a call's sizes, shared by the host code and by a host test that pins the
// kernel each shape takes.
#pragma once

#include <stdint.h>

namespace atom {
namespace mx {

constexpr int kBatch = 4;        // groups of K whose loads a wave of the few-rows kernels has in flight
constexpr int kTokens = 16;      // tokens of a workgroup that quantizes them itself

// The kinds of kernel: few rows, then the tiled kernel's tile sizes, smallest first.
constexpr int kRowKinds = 2, kKinds = 7;
constexpr int kDividedKind = 2;  // the tile size whose plans may divide K
constexpr int kBM[kKinds] = {16, 32, 64, 64, 128, 256, 256}, kBN[kKinds] = {16, 16, 64, 128, 128, 128, 256};

// Waves of a few-rows workgroup, which divide K's groups: as few turns of whole batches as possible, then as little behind
// the ranges' ends.  (1 x 4096 x 4096, 16 groups: 4 waves 4.0 us, 8 5.0, 16 5.8; 1 x 4096 x 11008, 43 groups: 4 8.6, 8 8.6, 11 7.2, 16 8.3.)
inline int rows_waves(int groups) {
  int best = 4, turns = 1 << 30, loaded = 1 << 30;
  for (int w = 4; w <= 16; ++w) {
    const int t = ((groups + w - 1) / w + kBatch - 1) / kBatch;
    if (t < turns || (t == turns && w * t * kBatch < loaded)) {
      best = w;
      turns = t;
      loaded = w * t * kBatch;
    }
  }
  return best;
}

// `tiles` workgroups; `splits` of them divide K for each output tile (their fp32 parts are added by a second kernel).
struct Plan {
  int kind, tiles, splits;
};

// The plan of a shape: the kernel whose estimated time (us) is least.
//   Few rows: a start, and for each 16 columns of a compute unit a rate for K's groups and its end.
//   Tiles: a round of the grid takes `fixed` us (first stages, epilogue) and `full` us for each group of K when every unit
//     holds `slots` workgroups, `one` us when it holds one, and `far` us where that one waits for HBM: operands past 5 MB (measured
//     over sets of 40 products in turn: smaller ones were still in the last-level cache); reading the weights sets a floor (`read`
//     bytes a us).
//   64 x 64 tiles with K divided two to four ways, at least four groups each: the second kernel's 2.3 us and the parts' way
//     through memory on top.
// Fitted on 256 units to 137 shapes of products alone (1 to 4096 rows, 64 to 28672 columns, K 256 to 11008), `far` to 130 more with K up to
// 28672: over these and 45 of the others the choice is 1.7% slower than the best kernel on average, over 10% on ten, most (47%) on
// 512 x 260 x 2048, a little more than one round of 32-token workgroups.  Measured (us), few rows and the tiles from
// 64 x 64 up (M x N x K): 16 x 4096 x 4096 5.0, 10.5, 12.5, 13.6, 17.4, 25.4; 16 x 28672 x 8192 37, 28, 30, 31, 39, 48; 32 x 4096 x 4096
// 7.0 (16 rows at a time), 6.3 (32), 10.7, 12.8, 13.9; 256 x 11008 x 4096 18.6, 19.3, 17.0, 21.8, 32 (tiles); 1024 x 11008 x 4096 56, 47, 38, 43, 35;
// 2048 x 4096 x 11008 97, 76, 57, 53, 72; 4096 x 28672 x 8192 925, 760, 537, 535, 449.  64 x 4096 x 11008 whole, two, three and four ways 24.7,
// 17.9, 16.3 and 15.6; 777 x 777 x 8192 21.3, 17, 15.7 and 17.
inline Plan plan(int M, int N, int K, int cus, bool divide = true) {
  auto tiles = [&](int kind) {
    return (int64_t)((M + kBM[kind] - 1) / kBM[kind]) * ((N + kBN[kind] - 1) / kBN[kind]);
  };
  struct Rows {
    double start, group, end;
  };
  constexpr Rows rows[kRowKinds] = {{2.1, 0.118, 0.515}, {1.6, 0.155, 1.4}};
  struct Cost {
    int slots;
    double full, one, far, fixed, read;
  };
  constexpr Cost cost[kKinds] = {{}, {}, {3, 0.91, 0.38, 0.52, 2.8, 3.6e6}, {2, 0.88, 0.55, 0.55, 3.3, 4.6e6},
                                 {2, 1.25, 0.70, 0.70, 4.1, 4.5e6}, {1, 0.90, 0.90, 0.90, 6.8, 3.4e6}, {1, 1.45, 1.45, 1.45, 12.8, 5.7e6}};
  const int groups = (K + 255) / 256;
  const bool hbm = ((int64_t)M + N) * groups * 136 > 5000000;
  Plan best = {0, 0, 1};
  double least = -1.0;
  // (a launch has less than 2^32 threads, and at most 65535 workgroups in y)
  auto offer = [&](int kind, int64_t t, int splits, double time) {
    if ((least >= 0.0 && time >= least) || t * splits * (kind < kRowKinds ? 1024 : 256) >= (int64_t)1 << 32) return;
    if (kind < kRowKinds && M > 65535 * kBM[kind]) return;
    least = time;
    best = Plan{kind, (int)t, splits};
  };
  for (int kind = 0; kind < kRowKinds; ++kind) {
    const double per = (double)tiles(kind) / cus, r = per > 1.0 ? per : 1.0;
    offer(kind, tiles(kind), 1, rows[kind].start + r * (groups * rows[kind].group + rows[kind].end));
  }
  for (int kind = kRowKinds; kind < kKinds; ++kind) {
    const Cost& c = cost[kind];
    const int64_t t = tiles(kind);
    for (int splits = 1; splits <= (divide && kind == kDividedKind ? 4 : 1); ++splits) {
      if (splits > 1 && (groups < 4 * splits || t * splits > c.slots * cus)) break;
      const int64_t per = (t * splits + cus - 1) / cus;    // workgroups of the busiest unit
      const int64_t full = per / c.slots, rest = per % c.slots;
      const double one = hbm ? c.far : c.one;
      const double part = rest ? one + (c.full - one) * (rest - 1) / (c.slots > 1 ? c.slots - 1 : 1) : 0.0;
      const double multiply = (groups + splits - 1) / splits * (full * c.full + part);
      const double read = (double)N * groups * 136 / (splits > 1 ? 5.6e6 : c.read);
      double time = 0.3 + (multiply > read ? multiply : read) + (full + (rest ? 1 : 0)) * c.fixed;
      if (splits > 1) time += 2.3 + (double)t * splits * kBM[kind] * kBN[kind] * 8 / 4.0e6;
      offer(kind, t, splits, time);
    }
  }
  return best;
}

// Bytes of a plan's parts, and the plan of a shape for as much scratch memory: where that is too little for the parts, the one of
// least time that has none, which is often another kernel than the divided one (us, divided, its kernel whole, and so: 333 x 512 x
// 28672 22.5, 61, 46; 200 x 1024 x 14336 15.0, 31.6, 25.6; 64 x 4096 x 8192 13.2, 19.9, 15.8).
inline int64_t part_bytes(const Plan& p) { return p.splits > 1 ? (int64_t)p.splits * p.tiles * kBM[p.kind] * kBN[p.kind] * 4 : 0; }
inline Plan plan_within(int M, int N, int K, int cus, int64_t scratch) {
  const Plan p = plan(M, N, K, cus);
  return part_bytes(p) > scratch ? plan(M, N, K, cus, false) : p;
}

// Whether one launch quantizes the tokens, 16 in every workgroup, and multiplies: where their codes leave room in LDS and one round of
// workgroups of at most 64 columns holds all outputs, or one and a half of 48, of which a unit holds two if rows are short (or
// there are few tokens).  One launch and two (us, M x N x K): 1 x 4096 x 4096 4.4 and 6.3, 1 x 28672 x 8192 23.9 and 31.8, 4 x 11008 x 1155 5.2 and 8.4,
// 8 x 4096 x 4096 5.7 and 6.6, 16 x 11008 x 2048 6.1 and 10.8, 8 x 8192 x 8192 12.4 and 12.4, 64 x 4096 x 2048 6.3 and 8.4, 256 x 1024 x 2048 6.1 and 8.0,
// 250 x 777 x 1155 6.4 and 10.4, 333 x 777 x 2048 8.1 and 9.1.  Against two where 16 long tokens meet few columns: 16 x 4096 x 4096 7.8 and 7.0, 17 x 256 x 4096
// 6.6 and 6.4, 333 x 777 x 1155 8.3 and 8.0; called one by one from Python these are 7.8 and 8.9, 6.6 and 8.9, 8.3 and 9.4, since the second
// launch is 4 us of the host's time.  So it is for few tokens of long rows: 8 x 4096 x 8192 9.3 and 8.8, 4 x 16384 x 8192 19.5 and 18.8.  Past that: 16 x 28672 x 1155 10.9 and 9.3, 16 x 28672 x 4096 18.9 and 17.5, 128 x 4096 x 2048 9.1 and 8.5, 512 x 1024 x 1155
// 8.9 and 7.2.
inline bool rows_fit(int M, int N, int K, int cus) {
  const int64_t tokens = M < kTokens ? M : kTokens, blocks = (M + kTokens - 1) / kTokens;
  return M == 1 || (tokens * K <= 65536 && (M <= 8 || ((int64_t)N + 63) / 64 * blocks <= cus ||
                                            (K <= 2048 && ((int64_t)N + 47) / 48 * blocks * 2 <= 3 * cus)));
}

// Its workgroups: `columns` times 16 columns each, K's groups divided among `waves`.
//   Columns: as few as give each unit one workgroup (the tokens are quantized once for all of them); one for long rows of one or two
//     tokens, whose weights take longer than the quantizing (us, one and three: 1 x 11008 x 4096 7.3 and 7.9, 4 x 11008 x 4096 8.5 and 8.2).
//   Waves: what each costs its unit, how often each waits for weights and how many units of 512 elements it quantizes.  Where several
//     workgroups come to a unit these wait for each other's weights: four (us, 4, 8 and 12: 8 x 28672 x 8192 30.0, 31.5, 34.2).
// On 256 units, over 245 shapes (1 to 512 tokens, 300 to 28672 columns, K 512 to 11008): the choice is 0.8% slower than the best of one to
// four columns and 4 to 16 waves on average, and two launches take 1.27 times its time.
struct RowsPlan {
  int columns, waves;
};
inline RowsPlan rows_plan(int M, int N, int K, int cus) {
  const int tokens = M < kTokens ? M : kTokens, groups = (K + 255) / 256, units = tokens * ((groups + 1) / 2);
  const int64_t tiles = (N + 15) / 16, blocks = (M + kTokens - 1) / kTokens;
  int columns = 1;
  if (K < 4096 || M > 2)
    while (columns < 4 && (tiles + columns - 1) / columns * blocks > cus) ++columns;
  if (M > 8 && (tiles + columns - 1) / columns * blocks > cus) columns = 3;   // one and a half rounds
  const double full = (double)((tiles + columns - 1) / columns * blocks) / cus, each = full > 1.0 ? full : 1.0;
  RowsPlan best = {columns, 4};
  double least = -1.0;
  for (int w = 4; w <= (each > 1.5 ? 4 : 16); w += 4) {
    const int flight = kBatch / columns, turns = ((groups + w - 1) / w + flight - 1) / flight;
    const double time = 4.0 * w * each + 16.0 * turns + 3.0 * ((units + w - 1) / w);
    if (least < 0.0 || time < least) {
      least = time;
      best.waves = w;
    }
  }
  return best;
}

}  // namespace mx
}  // namespace atom
