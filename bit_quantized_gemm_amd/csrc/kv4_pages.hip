// Bookkeeping of the 4-bit KV cache on gfx950 (atom_kv4_pages.h): the tokens that a step adds to its sequences, and the pages of
// finished ones.
//
// What bounds it: latency.  Every workgroup scans the sequences for itself (a tile of as many as it has threads at a
// time), which costs less than a launch that does it once, and then takes its own rows: a row's sequence is found by
// bisection in LDS, its page is an entry of the table or of the pool.  Measured: 64 sequences, a token each 3.1 us, 256 sequences,
// 230528 tokens 4.3 us; pages of 64 and 1024 sequences given back 3.1 and 4.3 us (a launch alone is 1.8).  In place, where a second launch
// commits, the 230528 tokens take 6.7 us and the 1024 sequences 7.3.
//
// Sums saturate where they no longer matter (behind the last row, behind the pool's end), so 32 bits hold them.
#include "kv4_layout.h"
#include "serve_internal.h"

namespace atom {
namespace {

__device__ __forceinline__ uint32_t plus(uint32_t a, uint32_t b, uint32_t most) { return min(a + b, most); }

// Exclusive sums over a workgroup's threads, each at most `most` (below 2^31); `all`: the sum of all.
template <int THREADS>
__device__ __forceinline__ uint32_t exclusive(uint32_t v, uint32_t most, uint32_t* waves, uint32_t& all) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint32_t s = min(v, most);
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t o = (uint32_t)__shfl_up((int)s, d);
    if (lane >= d) s = plus(s, o, most);
  }
  __syncthreads();                                      // `waves` may still be read from the last call
  if (lane == 63) waves[wave] = s;
  __syncthreads();
  uint32_t before = 0;
  all = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 64; ++w) {
    if (w == wave) before = all;
    all = plus(all, waves[w], most);
  }
  const uint32_t left = (uint32_t)__shfl_up((int)s, 1);
  return lane ? plus(before, left, most) : before;
}

__device__ __forceinline__ int clamped(int x, int most) { return min(max(x, 0), most); }

// One sequence's part of a step: its first row, its length before and behind it, pages before, the first of its fresh ones.
struct Sequence {
  uint32_t start, first;
  int tokens, after, have, need;
};

// Rows span * blockIdx.x .. of `total` a workgroup.  commit: workgroup 0 writes the lengths and the pool's state (not while
// other workgroups may still read the same arrays).
template <int THREADS>
__global__ __launch_bounds__(THREADS) void extend_kernel(Kv4Extend a, int span, int commit) {
  __shared__ uint32_t waves[THREADS / 64];
  __shared__ uint32_t s_start[THREADS + 1], s_first[THREADS];
  __shared__ int s_tokens[THREADS];
  const int tid = threadIdx.x;
  const int most = a.width << a.log_page, mask = (1 << a.log_page) - 1;
  const uint32_t total = (uint32_t)a.total, kMost = 1u << 30;
  const int pool = clamped(a.state[0], a.capacity);

  uint32_t row = 0, page = 0;                           // in front of the tile
  auto tile = [&](int b0) __attribute__((always_inline)) {
    const int b = b0 + tid;
    const bool in = b < a.batch;
    Sequence s;
    s.tokens = in ? clamped(a.lens[b], most) : 0;
    const uint32_t more = in ? (uint32_t)max(a.more[b], 0) : 0;
    uint32_t rows, pages;
    s.start = plus(row, exclusive<THREADS>(more, total, waves, rows), total);
    const uint32_t taken = plus(s.start, min(more, total), total) - s.start;
    s.after = (int)min((uint32_t)s.tokens + taken, (uint32_t)most);
    s.have = (s.tokens + mask) >> a.log_page;
    s.need = ((s.after + mask) >> a.log_page) - s.have;
    s.first = page + exclusive<THREADS>((uint32_t)s.need, kMost, waves, pages);
    row = plus(row, rows, total);
    page = min(page + pages, kMost);
    return s;
  };
  Sequence s = tile(0);
  for (int b0 = THREADS; b0 < a.batch; b0 += THREADS) tile(b0);
  const uint32_t end = row, needed = page;              // rows taken, pages needed
  const bool fits = needed <= (uint32_t)pool;

  const uint32_t lo = (uint32_t)blockIdx.x * (uint32_t)span, hi = min(lo + (uint32_t)span, total);
  const bool first = blockIdx.x == 0;
  row = page = 0;
  for (int b0 = 0; b0 < a.batch; b0 += THREADS) {
    const uint32_t begin = row;
    if (a.batch > THREADS) s = tile(b0);
    else row = end;
    __syncthreads();                                    // the last tile's rows are done
    s_start[tid] = s.start;
    s_first[tid] = s.first;
    s_tokens[tid] = s.tokens;
    if (tid == 0) s_start[THREADS] = row;
    __syncthreads();
    if (first) {
      const int b = b0 + tid;
      if (b < a.batch) {
        if (!commit || span) a.start[b] = (int)s.start;
        if (commit) a.lens_out[b] = fits ? s.after : s.tokens;
      }
    }
    if (fits) {
      for (uint32_t r = max(lo, begin) + tid; r < min(hi, row); r += THREADS) {
        int at = 0;                                     // the last sequence of the tile that starts at r or before it
#pragma unroll
        for (int d = THREADS / 2; d; d >>= 1)
          if (s_start[at + d] <= r) at += d;
        const int b = b0 + at;
        const int tokens = s_tokens[at], t = tokens + (int)(r - s_start[at]);
        int64_t slot = -1;
        if (t < most) {
          const int have = (tokens + mask) >> a.log_page, col = t >> a.log_page;
          int32_t* entry = a.table + (int64_t)b * a.width + col;
          int id;
          if (col < have) {
            id = *entry;
          } else {
            id = a.free_pages[pool - 1 - (int)(s_first[at] + (uint32_t)(col - have))];
            if ((t & mask) == 0) *entry = id;           // a page's first token
          }
          if (id >= 0) slot = (int64_t)id << a.log_page | (t & mask);
        }
        a.slots[r] = slot;
      }
    }
  }
  for (uint32_t r = max(lo, fits ? end : 0) + tid; r < hi; r += THREADS) a.slots[r] = -1;
  if (first && tid == 0) {
    if (!commit || span) a.start[a.batch] = (int)end;
    if (commit) {
      a.state_out[0] = fits ? pool - (int)needed : pool;
      a.state_out[1] = fits ? 0 : (int)(needed - (uint32_t)pool);
    }
  }
}

// A wave takes sequences blockIdx.x * waves + wave, then those a grid further.
template <int THREADS>
__global__ __launch_bounds__(THREADS) void release_kernel(Kv4Release a, int copy, int commit) {
  __shared__ uint32_t waves[THREADS / 64];
  __shared__ uint32_t s_first[THREADS];
  __shared__ int s_pages[THREADS];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int most = a.width << a.log_page, mask = (1 << a.log_page) - 1;
  const uint32_t capacity = (uint32_t)a.capacity;
  const uint32_t pool = (uint32_t)clamped(a.state[0], a.capacity);
  uint32_t given = 0;                                   // pages in front of the tile
  for (int b0 = 0; b0 < a.batch; b0 += THREADS) {
    const int b = b0 + tid;
    const bool in = b < a.batch;
    const int tokens = in ? clamped(a.lens[b], most) : 0;
    const bool done = in && a.done[b] != 0;
    const int pages = done ? (tokens + mask) >> a.log_page : 0;
    uint32_t all;
    const uint32_t at = plus(given, exclusive<THREADS>((uint32_t)pages, capacity, waves, all), capacity);
    given = plus(given, all, capacity);
    s_first[tid] = pool + at;
    s_pages[tid] = pages;
    __syncthreads();
    if (commit && blockIdx.x == 0 && in) a.lens_out[b] = done ? 0 : tokens;
    if (copy) {
      const int n = min(a.batch - b0, THREADS);
      for (int i = blockIdx.x * (THREADS / 64) + wave; i < n; i += gridDim.x * (THREADS / 64)) {
        const int32_t* from = a.table + (int64_t)(b0 + i) * a.width;
        const uint32_t to = s_first[i];
        for (int c = lane; c < s_pages[i] && to + c < capacity; c += 64) a.free_pages[to + c] = from[c];
      }
    }
  }
  __syncthreads();
  if (commit && blockIdx.x == 0 && tid == 0) {
    a.state_out[0] = (int)plus(pool, given, capacity);
    a.state_out[1] = 0;
  }
}

}  // namespace

hipError_t launch_kv4_extend(const Kv4Extend& a, hipStream_t stream) {
  // A row a thread, and at most 512 workgroups where each has many sequences to scan.  Us, by rows of a workgroup of 256 threads (64
  // sequences): 288 rows in all 3.3 (256), 3.9 (512); 4096 rows 3.5, 4.0 and 11.8 (4096); 256 sequences, 230528 rows 4.3 and 4.5; 1024 sequences,
  // 262144 rows in workgroups of 1024 threads 5.2 (1024), 5.8 (2048).  In place one workgroup takes up to 1024 rows (5.4
  // us) rather than a second launch.
  const int threads = a.batch <= 256 ? 256 : 1024;
  const bool in_place = a.lens_out == a.lens || a.state_out == a.state;
  int span = threads;
  if (in_place && a.total <= 1024) span = 1024;
  if (a.batch > 1024 && a.total > 512 * span) span = (a.total + 511) / 512;
  const int groups = (a.total + span - 1) / span;
  const bool later = groups > 1 && in_place;
  auto go = [&](int g, int n, int commit) {
    if (threads == 256)
      hipLaunchKernelGGL((extend_kernel<256>), dim3(g), dim3(256), 0, stream, a, n, commit);
    else
      hipLaunchKernelGGL((extend_kernel<1024>), dim3(g), dim3(1024), 0, stream, a, n, commit);
  };
  go(groups, span, !later);
  if (later) go(1, 0, 1);
  return hipGetLastError();
}

hipError_t launch_kv4_release(const Kv4Release& a, hipStream_t stream) {
  // A sequence a wave; in place one workgroup takes up to 64 sequences rather than a second launch.
  const bool in_place = a.lens_out == a.lens || a.state_out == a.state;
  const int groups = in_place && a.batch <= 64 ? 1 : a.batch < 1024 ? (a.batch + 15) / 16 : 64;
  const bool later = groups > 1 && in_place;
  auto go = [&](int g, int copy, int commit) {
    hipLaunchKernelGGL((release_kernel<1024>), dim3(g), dim3(1024), 0, stream, a, copy, commit);
  };
  go(groups, 1, !later);
  if (later) go(1, 0, 1);
  return hipGetLastError();
}

}  // namespace atom
