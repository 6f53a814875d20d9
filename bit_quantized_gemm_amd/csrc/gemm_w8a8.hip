// W8A8 GEMM for gfx950: Y[m,n] = round(sx[m] * sw[n] * sum_k qx[m,k] * qw[n,k] + bias[n]) from
// int8 codes with one fp32 scale a row on both sides, on v_mfma_i32_{32x32x32,16x16x64}_i8.
//
// The whole sum over K is one exact int32 (127^2 * 65536 < 2^31), so the scales are applied once
// in the epilogue, and K may be divided among waves or workgroups without changing a bit.
//
// Operand layout.  Both operands are rows of K bytes; in a K = 32 slice lane l supplies row
// l & 31 and bytes 16 (l >> 5) .. + 15.  The weights are the first operand, so a 32x32 accumulator
// holds its tile transposed: lane l owns token l & 31, element r is column
// (r >> 2) * 8 + (l >> 5) * 4 + (r & 3): four runs of four columns.
//
// Kernels.
//   gemm_tile_kernel: bound by the matrix cores, and at the largest sizes by the power they draw (4096 x 28672 x 8192 at
//     2.5 POP/s on quantized normal data, 3.0 on zeros).  The workgroup's four waves each own a quarter of a BM x BN tile.
//     Stages of 128 bytes of K are copied from global memory straight into a ring of LDS buffers (LDS-DMA): whole
//     cache lines, because a line fetched in two halves by two stages came twice from the L2 (256 x 256 tiles, 64-byte
//     stages: 1000 us instead of 935).  Stage rows are unpadded, 16-byte chunks at swizzled positions: the 16 lanes of a
//     16-byte read hit distinct bank groups.  A stage is four K slices; a wave multiplies one slice while the next one's
//     operands are read, one read or copy between two products.
//     2048 x 4096 x 11008 (M x N x K) takes 86.5 us, 2.13 POP/s; the library's int8 product reaches 2.05.
//   gemm_rows_kernel (few tokens, or few outputs): bound by reading the weights.  A workgroup owns 16 columns, its
//     waves divide K, and each wave loads its operands straight into registers, a batch of
//     16-byte loads in flight at once; the waves' integer sums meet in LDS.  Weights from HBM: 1 x 4096 x 4096 5.9 us,
//     1 x 28672 x 8192 43 us (5.5 TB/s), 16 x 11008 x 4096 14.3 us (3.2 TB/s, and as many bytes of codes from the L2).
//     48 columns a workgroup (a third of those) took 13.2 us there, more elsewhere.
//   linear_rows_kernel: the same for at most four tokens with the quantizer in front, one launch for two: 1 x 4096 x 4096
//     6.2 us against 2.6 + 5.9.
#include "lds_ring.h"
#include "atom_internal.h"
#include "gemm_tile.h"
#include "w8a8_row.h"

namespace atom {
namespace {

__device__ __forceinline__ i32x16 mma(i32x4 w, i32x4 x, i32x16 c) {
  return __builtin_amdgcn_mfma_i32_32x32x32_i8(w, x, c, 0, 0, 0);
}

// One output: (acc * sx) * sw + bias, each step in fp32.  acc converts to fp32 with one rounding
// (relative 2^-24); Y's own rounding is 2^-11 or 2^-8.  The empty asm keeps the compiler from folding the fma and
// Y's conversion into one instruction with one rounding in some kernels and not in others.
__device__ __forceinline__ float scaled(int acc, float sx, float sw, float bias) {
  float y = __builtin_fmaf((float)acc * sx, sw, bias);
  asm("" : "+v"(y));
  return y;
}

// Eight outputs of a row, `left` of them inside it; wide: the row's start is 16-byte aligned.
template <class T>
__device__ __forceinline__ void store8(uint16_t* dst, const float (&y)[8], int left, bool wide) {
  if (wide && left >= 8) {
    *reinterpret_cast<u32x4*>(dst) =
        u32x4{pack2<T>(y[0], y[1]), pack2<T>(y[2], y[3]), pack2<T>(y[4], y[5]), pack2<T>(y[6], y[7])};
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < left) dst[e] = T::store(y[e]);
  }
}

// BM x BN output tile of four waves (2 x 2), RING stage buffers.  kDivided (K may be divided): with splits > 1 piece p of tile t is
// workgroup p * tiles + t and writes its int32 tile to part[(p * tiles + t) * BM * BN].
template <class T, int BM, int BN, int RING, int WAVES, bool kDivided>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(WAVES))) void gemm_tile_kernel(
    const int8_t* __restrict__ Xq, const float* __restrict__ sx, const int8_t* __restrict__ Wq,
    const float* __restrict__ sw, const uint16_t* __restrict__ bias, int M, int N, int Kp, uint16_t* __restrict__ Y,
    int tiles, int splits, int32_t* __restrict__ part) {
  constexpr int WM = BM / 2, WN = BN / 2, TM = WM / 32, TN = WN / 32;
  constexpr int kDmaA = BM / 32, kDmaB = BN / 32;        // LDS-DMA instructions per wave and stage
  constexpr int kPer = kDmaA + kDmaB;
  constexpr int kA = BM * kStage, kB = BN * kStage;
  // each stage buffer its own object: the compiler knows that a copy into one does not write another
  __shared__ __attribute__((aligned(16))) uint8_t la0[kA], la1[kA], la2[kA];
  __shared__ __attribute__((aligned(16))) uint8_t lb0[kB], lb1[kB], lb2[kB];   // (buffers past RING take no LDS)
  auto LA = [&](int p) -> uint8_t* { return p == 0 ? la0 : p == 1 ? la1 : la2; };
  auto LB = [&](int p) -> uint8_t* { return p == 0 ? lb0 : p == 1 ? lb1 : lb2; };

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1, l32 = lane & 31, kh = lane >> 5;
  const int tiles_m = (M + BM - 1) / BM, tiles_n = (N + BN - 1) / BN;
  int lin = (int)blockIdx.x, piece = 0;
  if (kDivided && splits > 1) {
    piece = lin / tiles;
    lin -= piece * tiles;
  } else {
    // workgroups go to the 8 XCDs in turn: give each a contiguous run of the tile order, so that
    // the tiles of one L2 share their operands
    const int per = tiles / 8, more = tiles % 8, x = lin % 8;
    lin = x * per + min(x, more) + lin / 8;
  }
  const int2 tc = tile_coords(lin, tiles_m, tiles_n);
  const int m0 = tc.x * BM, n0 = tc.y * BN;
  const int stages = Kp / kStage;
  const int sa = kDivided ? (int)((int64_t)stages * piece / splits) : 0;
  const int sb = kDivided ? (int)((int64_t)stages * (piece + 1) / splits) : stages;

  // Stage copies: wave w copies rows [w B / 4, (w + 1) B / 4) of both operands, 8 rows an
  // instruction: lane i lands at row i / 8, position i % 8, and loads the chunk that lies there.
  // Rows past M / N repeat the last one (their results are never stored).
  const int rows_a = min(BM, M - m0), rows_b = min(BN, N - n0);
  const __amdgpu_buffer_rsrc_t ra =
      __builtin_amdgcn_make_buffer_rsrc((void*)(Xq + (size_t)m0 * Kp), (short)0, rows_a * Kp, 0x00020000);
  const __amdgpu_buffer_rsrc_t rb =
      __builtin_amdgcn_make_buffer_rsrc((void*)(Wq + (size_t)n0 * Kp), (short)0, rows_b * Kp, 0x00020000);
  int va[kDmaA], vb[kDmaB];
#pragma unroll
  for (int h = 0; h < kDmaA; ++h) {
    const int r = wave * (BM / 4) + 8 * h + lane / 8;
    va[h] = min(r, rows_a - 1) * Kp + pos(r, lane & 7) * 16;
  }
#pragma unroll
  for (int h = 0; h < kDmaB; ++h) {
    const int r = wave * (BN / 4) + 8 * h + lane / 8;
    vb[h] = min(r, rows_b - 1) * Kp + pos(r, lane & 7) * 16;
  }
  // Copies of stages behind the last repeat it (never read).
  auto dma = [&](int p, int s) __attribute__((always_inline)) {
    const int off = min(s, stages - 1) * kStage;
#pragma unroll
    for (int h = 0; h < kDmaA; ++h) lds_dma16(ra, LA(p) + (wave * (BM / 4) + 8 * h) * kStage, va[h], off);
#pragma unroll
    for (int h = 0; h < kDmaB; ++h) lds_dma16(rb, LB(p) + (wave * (BN / 4) + 8 * h) * kStage, vb[h], off);
  };
  const int swz = (l32 >> 1) & 7;
  auto read = [&](const uint8_t* buf, int row, int t) __attribute__((always_inline)) {   // slice t of a tile row
    return *reinterpret_cast<const i32x4*>(buf + row * kStage + (((2 * t + kh) ^ swz) << 4));
  };

  i32x16 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = i32x16{};
  i32x4 a0[TM], b0[TN], a1[TM], b1[TN];
  auto load = [&](int p, int t, i32x4 (&a)[TM], i32x4 (&b)[TN]) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < TM; ++i) a[i] = read(LA(p), wm * WM + 32 * i + l32, t);
#pragma unroll
    for (int j = 0; j < TN; ++j) b[j] = read(LB(p), wn * WN + 32 * j + l32, t);
  };
  auto multiply = [&](const i32x4 (&a)[TM], const i32x4 (&b)[TN]) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[i][j] = mma(b[j], a[i], acc[i][j]);
  };

  // Ring.  Stage t lives in buffer (t - sa) % RING.  On entry of stage s its first slice is in registers and its
  // copy is visible to every wave; stages s+1 .. s+RING-1 are in flight.  The barrier comes once this wave's reads
  // of stage s are done and its copy of stage s+1 has landed: behind it the last slice is multiplied while the
  // next stage's first is read and stage s+RING is copied into the buffer that stage s has left.
#pragma unroll
  for (int p = 0; p < RING; ++p) dma(p, sa + p);
  __builtin_amdgcn_s_waitcnt(wait_vm_lgkm0((RING - 1) * kPer));
  wg_barrier();
  load(0, 0, a0, b0);
  auto stage = [&](auto ring, int s) __attribute__((always_inline)) {
    constexpr int p = decltype(ring)::kCur, p1 = decltype(ring)::kNext;
    load(p, 1, a1, b1);
    multiply(a0, b0);
    interleave<TM * TN, TM + TN, 0>();
    __builtin_amdgcn_sched_barrier(0);
    load(p, 2, a0, b0);
    multiply(a1, b1);
    interleave<TM * TN, TM + TN, 0>();
    __builtin_amdgcn_sched_barrier(0);
    load(p, 3, a1, b1);
    multiply(a0, b0);
    interleave<TM * TN, TM + TN, 0>();
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(wait_vm_lgkm0((RING - 2) * kPer));
    wg_barrier();
    load(p1, 0, a0, b0);      // behind the last stage: a repeated copy, unused
    dma(p, s + RING);
    multiply(a1, b1);
    interleave<TM * TN, TM + TN, kPer>();
    __builtin_amdgcn_sched_barrier(0);
  };
  {
    int s = sa;
    for (; s + RING <= sb; s += RING) ring_turn<0, RING>(stage, s);
    ring_tail<0, RING>(stage, s, sb);
  }
  __builtin_amdgcn_s_waitcnt(0);                          // no copy into LDS outlives the workgroup

  if (kDivided && splits > 1) {
    int32_t* tile = part + ((size_t)piece * tiles + lin) * (BM * BN);
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *reinterpret_cast<i32x4*>(tile + (wm * WM + 32 * i + l32) * BN + wn * WN + 32 * j + 8 * q + 4 * kh) =
              i32x4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
    return;
  }
  // Epilogue through LDS, 32 rows of a wave at a time: the accumulators' columns lie four to a lane and 32 rows to an
  // instruction, and stores of that shape send 16 bytes each to rows a multiple of 4 KB apart, all in one channel of the L2
  // (4096 x 28672 outputs of K = 256: 236 us so, 114 us row by row; of K = 8192: 935 and 762 us).  Chunk c of 4 columns of row r lies at position
  // c ^ (r & 15): both the writes (16 rows of one chunk) and the reads (a row's chunks) cover all banks.
  wg_barrier();                                           // every wave has read its last stage
  constexpr int kLanes = WN / 8;                          // lanes of a row: 8 columns each
  i32x4* own = reinterpret_cast<i32x4*>(wave == 0 ? la0 : wave == 1 ? la1 : RING == 2 ? (wave == 2 ? lb0 : lb1)
                                                                                      : (wave == 2 ? la2 : lb0));
  static_assert(32 * WN * 4 <= kA && 32 * WN * 4 <= kB, "a wave's rows fit a stage buffer");
  const int c8 = lane % kLanes, n = n0 + wn * WN + 8 * c8;
  float w[8], b[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int c = min(n + e, N - 1);
    w[e] = sw[c];
    b[e] = bias ? T::load(bias[c]) : 0.0f;
  }
#pragma unroll
  for (int i = 0; i < TM; ++i) {
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        own[l32 * (WN / 4) + ((8 * j + 2 * q + kh) ^ (l32 & 15))] =
            i32x4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
#pragma unroll
    for (int r = lane / kLanes; r < 32; r += 64 / kLanes) {
      const int m = m0 + wm * WM + 32 * i + r;
      const i32x4 lo = own[r * (WN / 4) + ((2 * c8) ^ (r & 15))], hi = own[r * (WN / 4) + ((2 * c8 + 1) ^ (r & 15))];
      const float x = sx[min(m, M - 1)];
      float y[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        y[e] = scaled(lo[e], x, w[e], b[e]);
        y[e + 4] = scaled(hi[e], x, w[e + 4], b[e + 4]);
      }
      if (m < M) store8<T>(Y + (size_t)m * N + n, y, N - n, (N & 7) == 0);
    }
  }
}

// Adds the integer pieces of a split product and writes Y.  One thread per four columns of a tile row.
template <class T, int BM, int BN>
__global__ __launch_bounds__(256) void finish_kernel(const int32_t* __restrict__ part, const float* __restrict__ sx,
                                                     const float* __restrict__ sw, const uint16_t* __restrict__ bias,
                                                     int M, int N, uint16_t* __restrict__ Y, int tiles, int splits) {
  constexpr int kPerTile = BM * BN / 4 / 256;             // workgroups per tile
  const int lin = blockIdx.x / kPerTile;
  const int2 tc = tile_coords(lin, (M + BM - 1) / BM, (N + BN - 1) / BN);
  const int e4 = (blockIdx.x % kPerTile) * 256 + threadIdx.x;
  const int r = e4 / (BN / 4), c = e4 % (BN / 4) * 4;
  const int m = tc.x * BM + r, n = tc.y * BN + c;
  if (m >= M || n >= N) return;
  i32x4 a = {};
  for (int p = 0; p < splits; ++p)
    a += *reinterpret_cast<const i32x4*>(part + ((size_t)p * tiles + lin) * (BM * BN) + r * BN + c);
  const float x = sx[m];
  uint16_t* dst = Y + (size_t)m * N + n;
  float y[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int cc = min(n + e, N - 1);
    y[e] = scaled(a[e], x, sw[cc], bias ? T::load(bias[cc]) : 0.0f);
  }
  if (n + 4 <= N && (N & 3) == 0) {
    *reinterpret_cast<u32x2*>(dst) = u32x2{pack2<T>(y[0], y[1]), pack2<T>(y[2], y[3])};
  } else {
    for (int e = 0; e < 4; ++e)
      if (n + e < N) dst[e] = T::store(y[e]);
  }
}

// 16 RT tokens (blockIdx.y) against 16 columns (blockIdx.x) a workgroup.  Lane l of a K = 64 slice supplies row l & 15, bytes
// 16 (l >> 4) .. + 15 of both operands; an accumulator holds token l & 15, columns 4 (l >> 4) .. + 3.
constexpr int kBatch = 4;        // units of 128 bytes of K whose loads a wave has in flight
template <class T, int RT>
__global__ __launch_bounds__(1024) void gemm_rows_kernel(const int8_t* __restrict__ Xq, const float* __restrict__ sx,
                                                         const int8_t* __restrict__ Wq, const float* __restrict__ sw,
                                                         const uint16_t* __restrict__ bias, int M, int N, int Kp,
                                                         uint16_t* __restrict__ Y) {
  extern __shared__ __attribute__((aligned(16))) int32_t sums[];   // [waves][RT][16 tokens][16 columns]
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
  const int l16 = lane & 15, q = lane >> 4, n0 = blockIdx.x * 16, m0 = blockIdx.y * (16 * RT);
  const int units = Kp / 128;
  const int ua = units * wave / waves, ub = units * (wave + 1) / waves;
  const int8_t* w = Wq + (size_t)min(n0 + l16, N - 1) * Kp + 16 * q;
  const int8_t* x[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) x[i] = Xq + (size_t)min(m0 + 16 * i + l16, M - 1) * Kp + 16 * q;
  i32x4 acc[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) acc[i] = i32x4{};
  for (int u = ua; u < ub; u += kBatch) {
    i32x4 b[kBatch][2], a[RT][kBatch][2];
#pragma unroll
    for (int k = 0; k < kBatch; ++k)      // past the range's end: the last unit again, not multiplied
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int off = min(u + k, ub - 1) * 128 + 64 * t;
        b[k][t] = *reinterpret_cast<const i32x4*>(w + off);
#pragma unroll
        for (int i = 0; i < RT; ++i) a[i][k][t] = *reinterpret_cast<const i32x4*>(x[i] + off);
      }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (u + k < ub) {
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int i = 0; i < RT; ++i) acc[i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(b[k][t], a[i][k][t], acc[i], 0, 0, 0);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < RT; ++i)
    *reinterpret_cast<i32x4*>(sums + ((wave * RT + i) * 16 + l16) * 16 + 4 * q) = acc[i];
  __syncthreads();
  for (int e = threadIdx.x; e < RT * 256; e += blockDim.x) {
    const int m = m0 + (e >> 4), n = n0 + (e & 15);
    if (m >= M || n >= N) continue;
    int s = 0;
    for (int v = 0; v < waves; ++v) s += sums[v * RT * 256 + e];
    Y[(size_t)m * N + n] = T::store(scaled(s, sx[m], sw[n], bias ? T::load(bias[n]) : 0.0f));
  }
}

// The layer for at most MR <= 4 tokens in one launch: every workgroup quantizes the tokens for itself, into LDS, while its
// first weights are on their way; then as above.  Each wave's weights are read as in gemm_rows_kernel.
template <class T, int MR, int CH>
__global__ __launch_bounds__(1024) void linear_rows_kernel(const uint16_t* __restrict__ X, int64_t ldx,
                                                           const int8_t* __restrict__ Wq, const float* __restrict__ sw,
                                                           const uint16_t* __restrict__ bias, int M, int N, int K, int Kp,
                                                           uint16_t* __restrict__ Y) {
  extern __shared__ __attribute__((aligned(16))) int32_t shared[];   // sums [waves][16 tokens][16 columns], then the codes
  __shared__ uint32_t wave_max[MR][16];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
  const int l16 = lane & 15, q = lane >> 4, n0 = blockIdx.x * 16;
  const int units = Kp / 128;
  const int ua = units * wave / waves, ub = units * (wave + 1) / waves;
  const int8_t* w = Wq + (size_t)min(n0 + l16, N - 1) * Kp + 16 * q;
  i32x4 b[kBatch][2];
  auto load = [&](int u) __attribute__((always_inline)) {      // past the range's end: the last unit again, not multiplied
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
#pragma unroll
      for (int t = 0; t < 2; ++t) b[k][t] = *reinterpret_cast<const i32x4*>(w + min(u + k, max(ub, 1) - 1) * 128 + 64 * t);
  };
  load(ua);
  __builtin_amdgcn_sched_barrier(0);

  int8_t* codes = reinterpret_cast<int8_t*>(shared + waves * 256);
  u32x4 x[MR][CH];
#pragma unroll
  for (int m = 0; m < MR; ++m) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      x[m][i] = w8a8::load8<false>(X + (int64_t)min(m, M - 1) * ldx, threadIdx.x + i * blockDim.x, K);
      top = w8a8::max8(x[m][i], top);
    }
#pragma unroll
    for (int d = 32; d; d >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, d));
    if (lane == 0) wave_max[m][wave] = top;
  }
  __syncthreads();
  float s[MR];
#pragma unroll
  for (int m = 0; m < MR; ++m) {
    uint32_t top = 0;
    for (int v = 0; v < waves; ++v) top = max(top, wave_max[m][v]);
    s[m] = T::load(top) / 127.0f;
    const float r = s[m] > 0.0f ? 1.0f / s[m] : 0.0f;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = threadIdx.x + i * blockDim.x;
      if (8 * c < Kp) *reinterpret_cast<u32x2*>(codes + m * Kp + 8 * c) = w8a8::codes8<T>(x[m][i], s[m], r);
    }
  }
  __syncthreads();

  const int8_t* row = codes + min(l16, MR - 1) * Kp + 16 * q;
  i32x4 acc = {};
  for (int u = ua; u < ub; u += kBatch) {
    if (u > ua) load(u);
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (u + k < ub) {
#pragma unroll
        for (int t = 0; t < 2; ++t)
          acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(
              b[k][t], *reinterpret_cast<const i32x4*>(row + (u + k) * 128 + 64 * t), acc, 0, 0, 0);
      }
    }
  }
  *reinterpret_cast<i32x4*>(shared + (wave * 16 + l16) * 16 + 4 * q) = acc;
  __syncthreads();
  const int m = threadIdx.x >> 4, n = n0 + (threadIdx.x & 15);
  if (m < M && n < N) {
    int sum = 0;
    for (int v = 0; v < waves; ++v) sum += shared[v * 256 + threadIdx.x];
    float sx = s[0];
#pragma unroll
    for (int i = 1; i < MR; ++i) sx = m == i ? s[i] : sx;
    Y[(size_t)m * N + n] = T::store(scaled(sum, sx, sw[n], bias ? T::load(bias[n]) : 0.0f));
  }
}

// The kinds of kernel: few rows, then the tiled kernel's tile sizes, smallest first.
constexpr int kKinds = 5;
constexpr int kDividedKind = 1;  // the tile size whose plans may divide K
constexpr int kBM[kKinds] = {16, 64, 128, 256, 256}, kBN[kKinds] = {16, 128, 128, 128, 256};

// Waves of a workgroup that divide units of 128 bytes of K.  A wave loads whole batches, so the count (8 to 16, four
// units each where there are fewer; at least one for 1024 bytes, which linear_rows_kernel's quantizer needs) is the
// one that loads least behind the ranges' ends: 16 x 4096 x 11008 with 11 waves of at most 8 units 15.0 us, with 8 of 11 14.9, with 16 of
// 6 17.6.
int rows_waves(int Kp) {
  const int units = Kp / 128;
  if (units <= 32) return max(4, (units + kBatch - 1) / kBatch);
  int best = 16, least = 1 << 30;
  for (int w = min(16, max(8, (units + 7) / 8)); w <= 16; ++w) {
    const int loaded = w * (((units + w - 1) / w + kBatch - 1) / kBatch * kBatch);
    if (loaded < least) {
      least = loaded;
      best = w;
    }
  }
  return best;
}

template <class T>
void launch(const int8_t* Xq, const float* sx, const int8_t* Wq, const float* sw, const uint16_t* bias, int M, int N,
            int K, uint16_t* Y, int32_t* part, const W8Plan& p, hipStream_t st) {
  const int Kp = (K + 127) / 128 * 128;
  if (p.kind == 0) {
    const int waves = rows_waves(Kp);
    if (M <= 16)
      hipLaunchKernelGGL((gemm_rows_kernel<T, 1>), dim3(p.tiles), dim3(64 * waves), waves * 1024, st, Xq, sx, Wq, sw,
                         bias, M, N, Kp, Y);
    else
      hipLaunchKernelGGL((gemm_rows_kernel<T, 2>), dim3(p.tiles, (M + 31) / 32), dim3(64 * waves), waves * 2048, st, Xq, sx, Wq, sw,
                         bias, M, N, Kp, Y);
    return;
  }
  const dim3 grid(p.tiles * p.splits);
#define ATOM_TILE(KIND, BM, BN, RING, W)                                                                             \
  if (p.kind == KIND)                                                                                                \
    hipLaunchKernelGGL((gemm_tile_kernel<T, BM, BN, RING, W, KIND == kDividedKind>), grid, dim3(256), 0, st, Xq, sx, \
                       Wq, sw, bias, M, N, Kp, Y, p.tiles, p.splits, part);
  ATOM_TILE(1, 64, 128, 3, 2)
  ATOM_TILE(2, 128, 128, 2, 2)
  ATOM_TILE(3, 256, 128, 3, 1)
  ATOM_TILE(4, 256, 256, 2, 1)
#undef ATOM_TILE
  if (p.splits > 1)
    hipLaunchKernelGGL((finish_kernel<T, kBM[kDividedKind], kBN[kDividedKind]>),
                       dim3(p.tiles * (kBM[kDividedKind] * kBN[kDividedKind] / 1024)), dim3(256), 0, st, part, sx, sw, bias, M,
                       N, Y, p.tiles, p.splits);
}

template <class T, int MR>
void launch_linear_rows(const uint16_t* X, int64_t ldx, const int8_t* Wq, const float* sw, const uint16_t* bias, int M,
                        int N, int K, uint16_t* Y, hipStream_t st) {
  const int Kp = (K + 127) / 128 * 128, waves = rows_waves(Kp), chunks = (Kp / 8 + 64 * waves - 1) / (64 * waves);
  const dim3 grid((N + 15) / 16), block(64 * waves);
  const size_t lds = waves * 1024 + (size_t)MR * Kp;
#define ATOM_ROWS(CH)                                                                                                   \
  if (chunks <= CH) {                                                                                                  \
    hipLaunchKernelGGL((linear_rows_kernel<T, MR, CH>), grid, block, lds, st, X, ldx, Wq, sw, bias, M, N, K, Kp, Y);   \
    return;                                                                                                            \
  }
  ATOM_ROWS(1)
  ATOM_ROWS(2)
#undef ATOM_ROWS
}

}  // namespace

// The plan of a shape: the kernel whose estimated time (us) is least.
//   Few rows: a start, and for each round of a workgroup a compute unit a rate for K (up to 16 tokens a unit reads its 16
//     columns and as much again of the tokens' codes, beyond that 32 tokens in a second tile of rows).
//   Tiles: a round of the grid takes `fixed` us (first stages, epilogue) and `full` ns for each element of K when every
//     unit holds `slots` workgroups, `one` ns when it holds one; reading the weights sets a floor.
//   64 x 128 tiles with K divided two to four ways, at least eight stages each and at most one workgroup a unit: the
//     second kernel's 2.5 us and the pieces' way through memory on top (and 4%: with weights that stay in the caches
//     undivided tiles gain more, 256 x 4096 x 4096 18.8 and 19.1 us from HBM, 14.3 and 18 not).
// Fitted on 256 units to weights that come from HBM, products alone.  Measured (M x N x K): few rows and undivided tiles 16 x 4096 x
// 4096 6.8 and 17.5, 16 x 12288 x 4096 15.2 and 19.2, 16 x 28672 x 8192 62 and 58, 32 x 4096 x 4096 8.8 and 18.0, 128 x 1024 x 4096 8.3
// and 18.4, 300 x 300 x 300 3.8 and 6.0, 64 x 4096 x 1024 8.0 and 6.3; undivided, two, three and four ways 64 x 5120 x 5120 25.7, 19.2,
// 16.4 and 15.4, 64 x 11008 x 4096 20.6, 17.4, 23.0 and 21.8 (the last two on more than 256 workgroups).
W8Plan w8_plan(int M, int N, int K) {
  auto tiles = [&](int kind) {
    return (int)((int64_t)((M + kBM[kind] - 1) / kBM[kind]) * ((N + kBN[kind] - 1) / kBN[kind]));
  };
  struct Cost {
    int slots;
    double full, one, fixed;
  };
  constexpr Cost cost[kKinds] = {{}, {2, 5.3, 4.0, 3.0}, {2, 8.1, 6.2, 5.0}, {1, 7.6, 7.6, 7.0}, {1, 13.5, 13.5, 12.0}};
  const int cus = compute_units(), stages = (K + 127) / 128;
  W8Plan best = {0, (N + 15) / 16, 1};
  const int64_t rounds = ((int64_t)best.tiles * (M <= 16 ? 1 : (M + 31) / 32) + cus - 1) / cus;
  double least = M <= 16 ? 2.9 + rounds * K * (M <= 4 ? 0.70e-3 : 0.97e-3) : 2.4 + rounds * (1.0 + 1.45e-3 * K);
  for (int kind = 1; kind < kKinds; ++kind) {
    const Cost& c = cost[kind];
    const int t = tiles(kind);
    for (int splits = 1; splits <= (kind == kDividedKind ? 4 : 1); ++splits) {
      if (splits > 1 && (stages < 8 * splits || t * splits > cus)) break;
      const int64_t per = ((int64_t)t * splits + cus - 1) / cus;    // workgroups of the busiest unit
      const int64_t full = per / c.slots, rest = per % c.slots;
      const double k = splits == 1 ? K : (stages + splits - 1) / splits * 128;
      const double multiply = 1e-3 * k * (full * c.full + (rest ? c.one : 0.0));
      const double read = (double)N * K / (splits > 1 ? 6e6 : 4.2e6);
      double time = (multiply > read ? multiply : read) + (full + (rest ? 1 : 0)) * c.fixed;
      if (splits > 1) time = 1.04 * (time + 2.5 + (double)t * splits * kBM[kind] * kBN[kind] * 8 / 3.3e6);
      if (time < least) {
        least = time;
        best = W8Plan{kind, t, splits};
      }
    }
  }
  return best;
}

int64_t w8_workspace_bytes(const W8Plan& p) {
  return p.splits > 1 ? (int64_t)p.splits * p.tiles * kBM[p.kind] * kBN[p.kind] * 4 : 0;
}

hipError_t launch_gemm_w8a8(const int8_t* Xq, const float* sx, const int8_t* Wq, const float* sw, const uint16_t* bias,
                            int M, int N, int K, bool bf16, uint16_t* Y, int32_t* part, const W8Plan& plan,
                            hipStream_t stream) {
  if (bf16)
    launch<Bf16>(Xq, sx, Wq, sw, bias, M, N, K, Y, part, plan, stream);
  else
    launch<Fp16>(Xq, sx, Wq, sw, bias, M, N, K, Y, part, plan, stream);
  return hipGetLastError();
}

bool linear_rows_fits(int M, int N, int K) {
  const int64_t work = (int64_t)M * K * (((N + 15) / 16 + compute_units() - 1) / compute_units());
  return M <= 4 && work <= 16384;
}

hipError_t launch_linear_rows(const uint16_t* X, int64_t ldx, const int8_t* Wq, const float* sw, const uint16_t* bias,
                              int M, int N, int K, bool bf16, uint16_t* Y, hipStream_t stream) {
  if (bf16)
    M == 1 ? launch_linear_rows<Bf16, 1>(X, ldx, Wq, sw, bias, M, N, K, Y, stream)
           : launch_linear_rows<Bf16, 4>(X, ldx, Wq, sw, bias, M, N, K, Y, stream);
  else
    M == 1 ? launch_linear_rows<Fp16, 1>(X, ldx, Wq, sw, bias, M, N, K, Y, stream)
           : launch_linear_rows<Fp16, 4>(X, ldx, Wq, sw, bias, M, N, K, Y, stream);
  return hipGetLastError();
}

}  // namespace atom
