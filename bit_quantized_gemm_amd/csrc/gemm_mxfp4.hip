// MXFP4 GEMM for gfx950: Y[m,n] = round(sum over blocks of 2^(ex + ew) * (32 products of 4-bit floats) + bias[n]) on
// v_mfma_scale_f32_{32x32x64,16x16x128}_f8f6f4, which take the blocks' scale bytes as they are: twice the operations of the
// int8 product a cycle, from half its bytes.
//
// Operand layout.  A stage is a group of 256 values: 128 bytes, a cache line, of each row, eight blocks of 16 bytes.  An
// instruction takes one block of each row from each lane, and which block of K that is is free as long as both operands
// agree: lane l of the 32x32x64 supplies row l & 31 and, in slice t of a stage, block 4 (l >> 5) + t, so the scale bytes
// of its four slices are one word of the group's eight, chosen by the instruction's byte select.  The weights are the
// first operand, so a 32x32 accumulator holds its tile transposed: lane l owns token l & 31, element r is column
// (r >> 2) * 8 + (l >> 5) * 4 + (r & 3): four runs of four columns.
//
// Precision.  A block's 32 products and their sum are exact; instructions add blocks' sums to the fp32 accumulator, aligned to
// the largest of them (errors of 2^-23 of the magnitudes, measured on operands of very different scales).
//
// Kernels.
//   gemm_tile_kernel: the workgroup's four waves each own a quarter of a BM x BN tile; stages are copied from global memory
//     straight into LDS (LDS-DMA).  At the largest sizes the power that random operands draw bounds it: 4096 x 28672 x 8192
//     (M x N x K) takes 449 us, 4.3 PFLOP/s, with zeros 348 us; the same kernel without copies and LDS reads 327 and 266 us (the
//     matrix cores alone at the clock that power leaves), without its stores 416 and 308.  The library's product reaches 3.0 PFLOP/s
//     there.  Below that it is bound by how fast a compute unit gets lines that miss its L2: 2048 x 4096 x 11008 50.5 us (3.7
//     PFLOP/s; 48 to 50 where the operands are in the last-level cache), 47 with zeros, 46 the copies alone.
//     On the way there (4096 x 28672 x 8192 and 2048 x 4096 x 11008): 485 and 61 us with each wave's scale words loaded into
//     registers and a stage's copies issued in one slice; 478 and 62 with all of a stage's operands in registers after its first slice
//     (256 x 256 tiles); 449 and 53 with scales through LDS and copies spread over the slices.
//   gemm_rows_kernel (few tokens, or few outputs): bound by reading the weights and the launch.  A workgroup owns 16 columns, its
//     waves divide K, each loads its operands straight into registers, all of them at once where K is short; the waves' sums
//     meet in LDS.  Weights from HBM: 16 x 4096 x 4096 5.0 us, 16 x 11008 x 4096 9.2 us (2.6 TB/s; as many bytes of codes from
//     the L2), 1 x 11008 x 4096 7.0 us.
//   linear_rows_kernel: the same with the quantizer in front, where one round of workgroups holds all outputs: one launch for two (us,
//     weights from HBM), 1 x 4096 x 4096 4.7 and 6.3, 4 x 11008 x 4096 8.2 and 10.1, 16 x 11008 x 4096 10.2 and 11.3, 16 x 4096 x 4096
//     7.8 to 8.3 and 7.0, 256 x 1024 x 2048 6.1 and 8.0.
#include "lds_ring.h"
#include "atom_internal.h"
#include "gemm_tile.h"
#include "mxfp4_plan.h"
#include "mxfp4_row.h"

namespace atom {
namespace {

typedef int32_t i32x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ i32x8 operand(i32x4 v) { return i32x8{v[0], v[1], v[2], v[3], 0, 0, 0, 0}; }
constexpr int kFp4 = 4;          // the instructions' number of the E2M1 format

// One slice: byte TB of both scale words.
template <int TB>
__device__ __forceinline__ f32x16 mma32(i32x4 w, i32x4 x, f32x16 c, int sw, int sx) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(operand(w), operand(x), c, kFp4, kFp4, TB, sw, TB, sx);
}
template <int TB>
__device__ __forceinline__ f32x4 mma16(i32x4 w, i32x4 x, f32x4 c, int sw, int sx) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand(w), operand(x), c, kFp4, kFp4, TB, sw, TB, sx);
}

// The sum and the bias in fp32.  The empty asm keeps the compiler from folding the sum and Y's conversion into one
// instruction with one rounding in some kernels and not in others.
__device__ __forceinline__ float biased(float acc, float bias) {
  float y = acc + bias;
  asm("" : "+v"(y));
  return y;
}

// Tile order: bands of tile rows, the rows fastest inside a band, so that the tiles that share an L2 form a block.  Four rows of
// 256 tokens a band: 2048 x 4096 x 11008 51.3 us, with eight 52.2; eight of 128: 2048 x 11008 x 4096 65.4 us, with four 66.5.
template <int BM>
__device__ __forceinline__ int2 tile_at(int lin, int tiles_m, int tiles_n) {
  constexpr int kBand = BM == 256 ? 4 : 8;
  const int band = lin / (kBand * tiles_n), first = band * kBand, rows = min(tiles_m - first, kBand);
  const int in_band = lin - band * kBand * tiles_n;
  return int2{first + in_band % rows, in_band / rows};
}

// BM x BN output tile of four waves (2 x 2), RING stage buffers.  kDivided (K may be divided): with splits > 1 piece p of tile t is
// workgroup p * tiles + t and writes its fp32 tile to part[(p * tiles + t) * BM * BN].
template <class T, int BM, int BN, int RING, int WAVES, bool kDivided, bool kEarly, bool kBias>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(WAVES))) void gemm_tile_kernel(
    const uint8_t* __restrict__ Xq, const uint8_t* __restrict__ sx, const uint8_t* __restrict__ Wq,
    const uint8_t* __restrict__ sw, const uint16_t* __restrict__ bias, int M, int N, int stages, uint16_t* __restrict__ Y,
    int tiles, int splits, float* __restrict__ part) {
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
  const int2 tc = tile_at<BM>(lin, tiles_m, tiles_n);
  const int m0 = tc.x * BM, n0 = tc.y * BN;
  const int sa = kDivided ? (int)((int64_t)stages * piece / splits) : 0;
  const int sb = kDivided ? (int)((int64_t)stages * (piece + 1) / splits) : stages;

  // The tile's bias, for the epilogue (the first barrier comes before it).
  __shared__ __attribute__((aligned(16))) uint16_t l_bias[kBias ? BN : 4];
  if (kBias && tid < BN) l_bias[tid] = bias[min(n0 + tid, N - 1)];

  // Stage copies: wave w copies rows [w B / 4, (w + 1) B / 4) of both operands, 8 rows an
  // instruction: lane i lands at row i / 8, position i % 8, and loads the chunk that lies there.
  // Rows past M / N repeat the last one (their results are never stored).
  const int rows_a = min(BM, M - m0), rows_b = min(BN, N - n0), bytes = stages * kStage;
  const __amdgpu_buffer_rsrc_t ra =
      __builtin_amdgcn_make_buffer_rsrc((void*)(Xq + (size_t)m0 * bytes), (short)0, rows_a * bytes, 0x00020000);
  const __amdgpu_buffer_rsrc_t rb =
      __builtin_amdgcn_make_buffer_rsrc((void*)(Wq + (size_t)n0 * bytes), (short)0, rows_b * bytes, 0x00020000);
  int va[kDmaA], vb[kDmaB];
#pragma unroll
  for (int h = 0; h < kDmaA; ++h) {
    const int r = wave * (BM / 4) + 8 * h + lane / 8;
    va[h] = min(r, rows_a - 1) * bytes + pos(r, lane & 7) * 16;
  }
#pragma unroll
  for (int h = 0; h < kDmaB; ++h) {
    const int r = wave * (BN / 4) + 8 * h + lane / 8;
    vb[h] = min(r, rows_b - 1) * bytes + pos(r, lane & 7) * 16;
  }
  // Instructions [from, to) of a stage's copies.  Stages behind the last repeat it (never read).
  auto dma = [&](int p, int s, int from, int to) __attribute__((always_inline)) {
    const int off = min(s, stages - 1) * kStage;
#pragma unroll
    for (int h = 0; h < kDmaA; ++h)
      if (h >= from && h < to) lds_dma16(ra, LA(p) + (wave * (BM / 4) + 8 * h) * kStage, va[h], off);
#pragma unroll
    for (int h = 0; h < kDmaB; ++h)
      if (kDmaA + h >= from && kDmaA + h < to) lds_dma16(rb, LB(p) + (wave * (BN / 4) + 8 * h) * kStage, vb[h], off);
  };
  const int swz = (l32 >> 1) & 7;
  auto read = [&](const uint8_t* buf, int row, int t) __attribute__((always_inline)) {   // slice t of a tile row
    return *reinterpret_cast<const i32x4*>(buf + row * kStage + (((4 * kh + t) ^ swz) << 4));
  };
  // Scales of a stage: 8 bytes a row, loaded once by the workgroup (thread t: row t of the two operands' rows, and row 256 + t)
  // and read from LDS as words.  Each wave loading its own words takes four times the instructions, which stand in line
  // with the copies: 4096 x 28672 x 8192 of zeros 371 us so, 330 us without any scales, 348 us through LDS.
  constexpr int kRows = (BM + BN + 255) / 256;
  __shared__ __attribute__((aligned(16))) u32x2 ls0[kRows * 256], ls1[kRows * 256];
  const uint8_t* from[kRows];
  size_t step[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int e = tid + 256 * i;
    const bool is_a = e < BM;
    from[i] = (is_a ? sx : sw) + (size_t)(is_a ? min(m0 + e, M - 1) : min(n0 + e - BM, N - 1)) * 8;
    step[i] = (size_t)(is_a ? M : N) * 8;
  }
  struct Rows {
    u32x2 v[kRows];
  };
  auto fetch = [&](int s, Rows& r) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < kRows; ++i) r.v[i] = *reinterpret_cast<const u32x2*>(from[i] + min(s, stages - 1) * step[i]);
  };
  auto put = [&](int odd, const Rows& r) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < kRows; ++i) (odd ? ls1 : ls0)[tid + 256 * i] = r.v[i];
  };
  struct Scales {
    int a[TM], b[TN];
  };
  auto scales = [&](int odd, Scales& q) __attribute__((always_inline)) {
    const uint8_t* l = reinterpret_cast<const uint8_t*>(odd ? ls1 : ls0) + l32 * 8 + 4 * kh;
#pragma unroll
    for (int i = 0; i < TM; ++i) q.a[i] = *reinterpret_cast<const int*>(l + (wm * WM + 32 * i) * 8);
#pragma unroll
    for (int j = 0; j < TN; ++j) q.b[j] = *reinterpret_cast<const int*>(l + (BM + wn * WN + 32 * j) * 8);
  };

  f32x16 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = f32x16{};
  struct Slice {
    i32x4 a[TM], b[TN];
  };
  auto load = [&](int p, int t, Slice& r) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < TM; ++i) r.a[i] = read(LA(p), wm * WM + 32 * i + l32, t);
#pragma unroll
    for (int j = 0; j < TN; ++j) r.b[j] = read(LB(p), wn * WN + 32 * j + l32, t);
  };
  auto multiply = [&](auto t, const Slice& r, const Scales& q) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[i][j] = mma32<decltype(t)::kCur>(r.b[j], r.a[i], acc[i][j], q.b[j], q.a[i]);
  };

  // Ring.  Stage t lives in buffer (t - sa) % RING, its scales in ls0 or ls1 by its parity.  A CU takes 64 bytes of copies a
  // cycle and a wave waits at a copy that it does not take, so a stage's copies are spread over the slices.  Waits
  // count copies alone: loads of scales lie among them, but where the last stages need none the compiler leaves
  // them out or moves them, and a count that included them would let a copy be late.
  constexpr int kReads = TM + TN, kMmas = TM * TN;
  Rows rows;
  Scales now, next;
  fetch(sa, rows);
  put(0, rows);
  fetch(sa + 1, rows);
  if constexpr (kEarly) {
    // Two buffers.  All operands of a stage are in registers after its first slice; behind that slice's barrier stage s+2
    // is copied into the buffer, and it has six slices to arrive.
    constexpr int kHalf = kPer / 2;
    Slice r0, r1, r2, r3;
#pragma unroll
    for (int p = 0; p < 2; ++p) dma(p, sa + p, 0, kPer);
    __builtin_amdgcn_s_waitcnt(wait_vm_lgkm0(kPer));
    wg_barrier();
    load(0, 0, r0);
    load(0, 1, r1);
    scales(0, now);
    auto stage = [&](auto ring, int s) __attribute__((always_inline)) {
      constexpr int p = decltype(ring)::kCur, p1 = decltype(ring)::kNext;
      load(p, 2, r2);
      load(p, 3, r3);
      multiply(Ring<0, 4>{}, r0, now);
      interleave<kMmas, 2 * kReads, 0>();
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_waitcnt(wait_vm_lgkm0(63));
      wg_barrier();             // every wave has read stage s
      put(p1, rows);
      fetch(s + 2, rows);
      dma(p, s + 2, 0, kHalf);
      multiply(Ring<1, 4>{}, r1, now);
      interleave<kMmas, 0, kHalf + kRows>();
      __builtin_amdgcn_sched_barrier(0);
      dma(p, s + 2, kHalf, kPer);
      multiply(Ring<2, 4>{}, r2, now);
      interleave<kMmas, 0, kPer - kHalf>();
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_waitcnt(wait_vm_lgkm0(kPer));
      wg_barrier();             // stage s+1 and its scales are there
      load(p1, 0, r0);          // behind the last stage: a repeated copy, unused
      load(p1, 1, r1);
      scales(p1, next);
      multiply(Ring<3, 4>{}, r3, now);
      interleave<kMmas, 3 * kReads, 0>();
      now = next;
      __builtin_amdgcn_sched_barrier(0);
    };
    int s = sa;
    for (; s + RING <= sb; s += RING) ring_turn<0, RING>(stage, s);
    ring_tail<0, RING>(stage, s, sb);
  } else {
    // Three buffers.  On entry of stage s its first slice and its scales are in registers and its copy is visible to every
    // wave; stage s+1 and a quarter of s+2 are in flight.  The barrier comes once this wave's reads of stage s are
    // done and its copy of stage s+1 has landed: behind it the last slice is multiplied while the next stage's first is
    // read and the copy of stage s+3 begins in the buffer that stage s has left.
    constexpr int kQ1 = (kPer + 3) / 4, kQ2 = (kPer + 1) / 2, kQ3 = (3 * kPer + 3) / 4;
    Slice r0, r1;
    dma(0, sa, 0, kPer);
    dma(1, sa + 1, 0, kPer);
    dma(2, sa + 2, 0, kQ1);
    __builtin_amdgcn_s_waitcnt(wait_vm_lgkm0(kPer));
    wg_barrier();
    load(0, 0, r0);
    scales(0, now);
    auto stage = [&](auto ring, int s, int odd) __attribute__((always_inline)) {
      constexpr int p = decltype(ring)::kCur, p1 = decltype(ring)::kNext, p2 = decltype(ring)::kAfterNext;
      load(p, 1, r1);
      dma(p2, s + 2, kQ1, kQ2);
      multiply(Ring<0, 4>{}, r0, now);
      interleave<kMmas, kReads, kQ2 - kQ1>();
      __builtin_amdgcn_sched_barrier(0);
      put(!odd, rows);
      load(p, 2, r0);
      dma(p2, s + 2, kQ2, kQ3);
      multiply(Ring<1, 4>{}, r1, now);
      interleave<kMmas, kReads, kQ3 - kQ2>();
      __builtin_amdgcn_sched_barrier(0);
      fetch(s + 2, rows);
      load(p, 3, r1);
      dma(p2, s + 2, kQ3, kPer);
      multiply(Ring<2, 4>{}, r0, now);
      interleave<kMmas, kReads, kPer - kQ3 + kRows>();
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_waitcnt(wait_vm_lgkm0(kPer));
      wg_barrier();
      load(p1, 0, r0);          // behind the last stage: a repeated copy, unused
      scales(!odd, next);
      dma(p, s + 3, 0, kQ1);
      multiply(Ring<3, 4>{}, r1, now);
      interleave<kMmas, 2 * kReads, kQ1>();
      now = next;
      __builtin_amdgcn_sched_barrier(0);
    };
    int s = sa;
    auto turn = [&](int odd) __attribute__((always_inline)) {
      stage(Ring<0, 3>{}, s, odd);
      stage(Ring<1, 3>{}, s + 1, !odd);
      stage(Ring<2, 3>{}, s + 2, odd);
      s += 3;
    };
    for (; s + 6 <= sb;) {
      turn(0);
      turn(1);
    }
    if (s + 3 <= sb) {
      turn(0);
      if (s < sb) stage(Ring<0, 3>{}, s, 1);
      if (s + 1 < sb) stage(Ring<1, 3>{}, s + 1, 0);
    } else {
      if (s < sb) stage(Ring<0, 3>{}, s, 0);
      if (s + 1 < sb) stage(Ring<1, 3>{}, s + 1, 1);
    }
  }
  __builtin_amdgcn_s_waitcnt(0);                          // no copy into LDS outlives the workgroup

  if (kDivided && splits > 1) {
    float* tile = part + ((size_t)piece * tiles + lin) * (BM * BN);
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *reinterpret_cast<f32x4*>(tile + (wm * WM + 32 * i + l32) * BN + wn * WN + 32 * j + 8 * q + 4 * kh) =
              f32x4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
    return;
  }
  // Epilogue: a wave's tile in Y's type through LDS (it fits a stage buffer), so that whole rows of it are stored.  A lane has
  // four neighbouring columns of a row: half a chunk of 16 bytes.  Chunk c of row r lies at position c ^ r (modulo the
  // row's chunks), its halves swapped in rows 16 to 31 of 32, so that 32 rows' halves cover all banks.
  wg_barrier();                                           // every wave has read its last stage
  constexpr int kChunks = WN / 8;                         // 16-byte chunks of a row: one lane's store
  static_assert(WM * WN * 2 <= kA && WM * WN * 2 <= kB, "a wave's tile fits a stage buffer");
  uint8_t* own = wave == 0 ? la0 : wave == 1 ? la1 : RING == 2 ? (wave == 2 ? lb0 : lb1) : (wave == 2 ? la2 : lb0);
#pragma unroll
  for (int j = 0; j < TN; ++j)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      u32x2 b = {0, 0};
      if (kBias) b = *reinterpret_cast<const u32x2*>(l_bias + wn * WN + 32 * j + 8 * q + 4 * kh);
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        float y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = biased(acc[i][j][4 * q + e], elem<T>(b[e / 2], e & 1));
        const int chunk = (4 * j + q) ^ (l32 & (kChunks - 1));
        *reinterpret_cast<u32x2*>(own + ((32 * i + l32) * kChunks + chunk) * 16 + 8 * (kh ^ (l32 >> 4))) =
            u32x2{pack2<T>(y[0], y[1]), pack2<T>(y[2], y[3])};
      }
    }
  const int c = lane % kChunks, n = n0 + wn * WN + 8 * c;
#pragma unroll
  for (int it = 0; it < WM * kChunks / 64; ++it) {
    const int r = it * (64 / kChunks) + lane / kChunks, m = m0 + wm * WM + r;
    u32x4 v = *reinterpret_cast<const u32x4*>(own + (r * kChunks + (c ^ (r & (kChunks - 1)))) * 16);
    if ((it * (64 / kChunks)) & 16) v = u32x4{v[2], v[3], v[0], v[1]};
    if (m < M) mx::store8(Y + (size_t)m * N + n, v, N - n);
  }
}

// Adds the pieces of a split product in their order and writes Y.  One thread per four columns of a tile row.
template <class T, int BM, int BN>
__global__ __launch_bounds__(256) void finish_kernel(const float* __restrict__ part, const uint16_t* __restrict__ bias, int M,
                                                     int N, uint16_t* __restrict__ Y, int tiles, int splits) {
  constexpr int kPerTile = BM * BN / 4 / 256;             // workgroups per tile
  const int lin = blockIdx.x / kPerTile;
  const int2 tc = tile_at<BM>(lin, (M + BM - 1) / BM, (N + BN - 1) / BN);
  const int e4 = (blockIdx.x % kPerTile) * 256 + threadIdx.x;
  const int r = e4 / (BN / 4), c = e4 % (BN / 4) * 4;
  const int m = tc.x * BM + r, n = tc.y * BN + c;
  if (m >= M || n >= N) return;
  f32x4 a = {};
  for (int p = 0; p < splits; ++p)
    a += *reinterpret_cast<const f32x4*>(part + ((size_t)p * tiles + lin) * (BM * BN) + r * BN + c);
  uint16_t* dst = Y + (size_t)m * N + n;
  float y[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) y[e] = biased(a[e], bias ? T::load(bias[min(n + e, N - 1)]) : 0.0f);
  if (n + 4 <= N) {
    typedef u32x2 Unaligned __attribute__((aligned(2)));
    *reinterpret_cast<Unaligned*>(dst) = u32x2{pack2<T>(y[0], y[1]), pack2<T>(y[2], y[3])};
  } else {
    for (int e = 0; e < 4; ++e)
      if (n + e < N) dst[e] = T::store(y[e]);
  }
}

// Few rows: 16 RT tokens (blockIdx.y) against 16 columns (blockIdx.x) a workgroup on the 16x16x128, K's groups divided among
// its waves, operands straight into registers.  In slice t (0, 1) of a group lane l supplies row l & 15 and block 2 (l >> 4) + t
// of both operands: its two scale bytes are one 16-bit word.  An accumulator holds token l & 15, columns 4 (l >> 4) .. + 3.
struct Operand {                 // a lane's rows of one operand
  const uint8_t *codes, *scales;
  size_t step;                   // bytes of the scales of one group
  __device__ __forceinline__ Operand(const uint8_t* q, const uint8_t* s, int rows, int row, int quarter, int groups)
      : codes(q + (size_t)row * groups * kStage + 32 * quarter), scales(s + (size_t)row * 8 + 2 * quarter), step((size_t)rows * 8) {}
  __device__ __forceinline__ i32x4 block(int g, int t) const {
    return *reinterpret_cast<const i32x4*>(codes + (size_t)g * kStage + 16 * t);
  }
  __device__ __forceinline__ int scale(int g) const { return *reinterpret_cast<const uint16_t*>(scales + g * step); }
};

using mx::kBatch;
template <class T, int RT>
__global__ __launch_bounds__(1024) void gemm_rows_kernel(const uint8_t* __restrict__ Xq, const uint8_t* __restrict__ sx,
                                                         const uint8_t* __restrict__ Wq, const uint8_t* __restrict__ sw,
                                                         const uint16_t* __restrict__ bias, int M, int N, int groups,
                                                         uint16_t* __restrict__ Y) {
  extern __shared__ __attribute__((aligned(16))) float sums[];   // [waves][RT][16 tokens][16 columns]
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
  const int l16 = lane & 15, q = lane >> 4, n0 = blockIdx.x * 16, m0 = blockIdx.y * (16 * RT);
  const int ua = groups * wave / waves, ub = groups * (wave + 1) / waves;
  const Operand w(Wq, sw, N, min(n0 + l16, N - 1), q, groups);
  f32x4 acc[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) acc[i] = f32x4{};
  for (int u = ua; u < ub; u += kBatch) {
    i32x4 b[kBatch][2], a[RT][kBatch][2];
    int eb[kBatch], ea[RT][kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {    // past the range's end: the last group again, not multiplied
      const int g = min(u + k, ub - 1);
#pragma unroll
      for (int t = 0; t < 2; ++t) b[k][t] = w.block(g, t);
      eb[k] = w.scale(g);
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        const Operand x(Xq, sx, M, min(m0 + 16 * i + l16, M - 1), q, groups);
#pragma unroll
        for (int t = 0; t < 2; ++t) a[i][k][t] = x.block(g, t);
        ea[i][k] = x.scale(g);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (u + k < ub) {
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          acc[i] = mma16<0>(b[k][0], a[i][k][0], acc[i], eb[k], ea[i][k]);
          acc[i] = mma16<1>(b[k][1], a[i][k][1], acc[i], eb[k], ea[i][k]);
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < RT; ++i)
    *reinterpret_cast<f32x4*>(sums + ((wave * RT + i) * 16 + l16) * 16 + 4 * q) = acc[i];
  __syncthreads();
  for (int e = threadIdx.x; e < RT * 256; e += blockDim.x) {
    const int m = m0 + (e >> 4), n = n0 + (e & 15);
    if (m >= M || n >= N) continue;
    float s = 0.0f;
    for (int v = 0; v < waves; ++v) s += sums[v * RT * 256 + e];
    Y[(size_t)m * N + n] = T::store(biased(s, bias ? T::load(bias[n]) : 0.0f));
  }
}

// The layer of few outputs in one launch: every workgroup quantizes its 16 tokens (blockIdx.y) for itself, into LDS, then as above,
// against 16 CT columns.  Its first loads of tokens are under way before those of its weights, since loads arrive in order, and its weights
// while it quantizes.  Addresses are a wave's, in scalar registers, and rows of LDS whole units, so that a unit takes few
// instructions besides the quantizer's own: 16 x 4096 x 4096 (M x N x K) 9.2 us with an index a lane, 8.2 so, 7.7 without
// conditions on the stores.  Rows in LDS lie 16 bytes (their scales 4) apart beyond their units, so that their reads do not meet in one bank.
__host__ __device__ constexpr int lds_codes(int pairs) { return pairs * 2 * kStage + 16; }
__host__ __device__ constexpr int lds_scales(int pairs) { return pairs * 16 + 4; }

template <class T, int CT, bool VEC>
__global__ __launch_bounds__(1024) void linear_rows_kernel(const uint16_t* __restrict__ X, int64_t ldx,
                                                           const uint8_t* __restrict__ Wq, const uint8_t* __restrict__ sw,
                                                           const uint16_t* __restrict__ bias, int rows, int N, int K,
                                                           int groups, uint16_t* __restrict__ Y) {
  const int m0 = blockIdx.y * mx::kTokens, M = min(rows - m0, mx::kTokens);   // this workgroup's tokens
  X += m0 * ldx;
  Y += (size_t)m0 * N;
  constexpr int kUnits = 8, kFlight = kBatch / CT;             // units of tokens and groups of weights in flight
  extern __shared__ __attribute__((aligned(16))) uint8_t shared[];   // codes and scales; sums [waves][CT][16 tokens][16 columns]
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
  const int l16 = lane & 15, q = lane >> 4, n0 = blockIdx.x * (16 * CT);
  const int ua = groups * wave / waves, ub = groups * (wave + 1) / waves;

  // A unit is 512 elements of a token, two groups: a wave's load.
  const int per = (groups + 1) / 2;
  struct At {
    int row, col;
  };
  const At step = {waves / per, waves % per};
  auto next = [&](At& a) __attribute__((always_inline)) {
    const int col = a.col + step.col, over = col >= per;
    a = At{a.row + step.row + over, col - (over ? per : 0)};
  };
  u32x4 x[kUnits];
  auto tokens = [&](At a) __attribute__((always_inline)) {
#pragma unroll
    for (int k = 0; k < kUnits; ++k, next(a)) {
      if (a.row >= M) continue;
      if constexpr (VEC) {
        const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc((void*)(X + a.row * ldx), (short)0, K * 2, 0x00020000);
        x[k] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, a.col * 1024 + lane * 16, 0, 0));
      } else {
        x[k] = K < 8 ? w8a8::load8<false>(X + a.row * ldx, a.col * 64 + lane, K) : mx::load8_any(X + a.row * ldx, a.col * 64 + lane, K);
      }
    }
  };
  At at = {wave / per, wave % per};
  tokens(at);
  __builtin_amdgcn_sched_barrier(0);

  i32x4 b[kFlight][CT][2];
  int eb[kFlight][CT];
  const int columns = min(16 * CT, N - n0), bytes = groups * kStage;
  const __amdgpu_buffer_rsrc_t rw = __builtin_amdgcn_make_buffer_rsrc((void*)(Wq + (size_t)n0 * bytes), (short)0, columns * bytes, 0x00020000);
  int vw[CT], vs[CT];
#pragma unroll
  for (int j = 0; j < CT; ++j) {
    const int r = min(16 * j + l16, columns - 1);
    vw[j] = r * bytes + 32 * q;
    vs[j] = r * 8 + 2 * q;
  }
  auto load = [&](int u) __attribute__((always_inline)) {      // past the range's end: the last group again, not multiplied
#pragma unroll
    for (int k = 0; k < kFlight; ++k) {
      const int g = min(u + k, max(ub, 1) - 1);
      const __amdgpu_buffer_rsrc_t rs =
          __builtin_amdgcn_make_buffer_rsrc((void*)(sw + ((size_t)g * N + n0) * 8), (short)0, columns * 8, 0x00020000);
#pragma unroll
      for (int j = 0; j < CT; ++j) {
#pragma unroll
        for (int t = 0; t < 2; ++t) b[k][j][t] = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(rw, vw[j] + 16 * t, g * kStage, 0));
        eb[k][j] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(rs, vs[j], 0, 0);
      }
    }
  };
  load(ua);
  __builtin_amdgcn_sched_barrier(0);

  uint8_t* codes = shared;
  uint8_t* scales = codes + M * lds_codes(per);
  auto quantize = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int k = 0; k < kUnits; ++k, next(at)) {
      if (at.row >= M) continue;
      uint32_t byte;
      const int c = at.col * 64 + lane;
      if (!VEC && K >= 8 && at.col == per - 1) x[k] = mx::behind(x[k], c, K);
      const uint32_t code = mx::quantize8<T>(x[k], byte);
      *reinterpret_cast<uint32_t*>(codes + at.row * lds_codes(per) + 4 * c) = code;
      scales[at.row * lds_scales(per) + (c >> 2)] = (uint8_t)byte;       // (the same from a block's four lanes)
    }
  };
  quantize();
  while (at.row < M) {
    tokens(at);
    quantize();
  }
  __syncthreads();

  const uint8_t* own = codes + min(l16, M - 1) * lds_codes(per) + 32 * q;
  const uint8_t* own_scales = scales + min(l16, M - 1) * lds_scales(per) + 2 * q;
  f32x4 acc[CT];
#pragma unroll
  for (int j = 0; j < CT; ++j) acc[j] = f32x4{};
  for (int u = ua; u < ub; u += kFlight) {
    if (u > ua) load(u);
#pragma unroll
    for (int k = 0; k < kFlight; ++k) {
      if (u + k < ub) {
        const i32x4 a0 = *reinterpret_cast<const i32x4*>(own + (u + k) * kStage);
        const i32x4 a1 = *reinterpret_cast<const i32x4*>(own + (u + k) * kStage + 16);
        const int ea = *reinterpret_cast<const uint16_t*>(own_scales + (u + k) * 8);
#pragma unroll
        for (int j = 0; j < CT; ++j) {
          acc[j] = mma16<0>(b[k][j][0], a0, acc[j], eb[k][j], ea);
          acc[j] = mma16<1>(b[k][j][1], a1, acc[j], eb[k][j], ea);
        }
      }
    }
  }
  __syncthreads();                                             // the sums take the codes' place
  float* sums = reinterpret_cast<float*>(shared);
#pragma unroll
  for (int j = 0; j < CT; ++j) *reinterpret_cast<f32x4*>(sums + ((wave * CT + j) * 16 + l16) * 16 + 4 * q) = acc[j];
  __syncthreads();
  for (int e = threadIdx.x; e < M * 16 * CT; e += blockDim.x) {
    const int m = e / (16 * CT), j = e / 16 % CT, n = n0 + e % (16 * CT);
    if (n < N) {
      float sum = 0.0f;
      for (int v = 0; v < waves; ++v) sum += sums[((v * CT + j) * 16 + m) * 16 + (e & 15)];
      Y[(size_t)m * N + n] = T::store(biased(sum, bias ? T::load(bias[n]) : 0.0f));
    }
  }
}

using mx::kBM;
using mx::kBN;
using mx::kDividedKind;
using mx::rows_waves;

template <class T>
void launch(const uint8_t* Xq, const uint8_t* sx, const uint8_t* Wq, const uint8_t* sw, const uint16_t* bias, int M, int N,
            int K, uint16_t* Y, float* part, const MxPlan& p, hipStream_t st) {
  const int groups = mx::padded(K) / mx::kGroup;
#define ATOM_ROWS(KIND, RT)                                                                                              \
  if (p.kind == KIND) {                                                                                                  \
    const int waves = rows_waves(groups);                                                                                \
    hipLaunchKernelGGL((gemm_rows_kernel<T, RT>), dim3((N + 15) / 16, (M + 16 * RT - 1) / (16 * RT)), dim3(64 * waves),  \
                       waves * RT * 1024, st, Xq, sx, Wq, sw, bias, M, N, groups, Y);                                    \
    return;                                                                                                              \
  }
  ATOM_ROWS(0, 1)
  ATOM_ROWS(1, 2)
#undef ATOM_ROWS
  const dim3 grid(p.tiles * p.splits);
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(256), 0, st, Xq, sx, Wq, sw, bias, M, N, groups, Y, p.tiles, p.splits, part);
  };
#define ATOM_TILE(KIND, BM, BN, RING, W, E)                                                  \
  if (p.kind == KIND) {                                                                      \
    constexpr bool kDivided = KIND == kDividedKind;                                          \
    bias && p.splits == 1 ? go(gemm_tile_kernel<T, BM, BN, RING, W, kDivided, E, true>)      \
                          : go(gemm_tile_kernel<T, BM, BN, RING, W, kDivided, E, false>);    \
  }
  ATOM_TILE(2, 64, 64, 3, 3, false)
  ATOM_TILE(3, 64, 128, 3, 2, false)
  ATOM_TILE(4, 128, 128, 2, 2, true)
  ATOM_TILE(5, 256, 128, 3, 1, false)
  ATOM_TILE(6, 256, 256, 2, 1, true)
#undef ATOM_TILE
  if (p.splits > 1)
    hipLaunchKernelGGL((finish_kernel<T, kBM[kDividedKind], kBN[kDividedKind]>),
                       dim3(p.tiles * (kBM[kDividedKind] * kBN[kDividedKind] / 1024)), dim3(256), 0, st, part, bias, M,
                       N, Y, p.tiles, p.splits);
}

template <class T, bool VEC>
void launch_rows(const uint16_t* X, int64_t ldx, const uint8_t* Wq, const uint8_t* sw, const uint16_t* bias, int M,
                 int N, int K, uint16_t* Y, hipStream_t st) {
  const int groups = mx::padded(K) / mx::kGroup, pairs = (groups + 1) / 2;
  const mx::RowsPlan p = mx::rows_plan(M, N, K, compute_units());
  const int lds = max(p.waves * p.columns * 1024, min(M, mx::kTokens) * (lds_codes(pairs) + lds_scales(pairs)));
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((N + 16 * p.columns - 1) / (16 * p.columns), (M + mx::kTokens - 1) / mx::kTokens), dim3(64 * p.waves),
                       lds, st, X, ldx, Wq, sw, bias, M, N, K, groups, Y);
  };
  switch (p.columns) {
    case 1: return go(linear_rows_kernel<T, 1, VEC>);
    case 2: return go(linear_rows_kernel<T, 2, VEC>);
    case 3: return go(linear_rows_kernel<T, 3, VEC>);
    default: return go(linear_rows_kernel<T, 4, VEC>);
  }
}

}  // namespace

MxPlan mx_plan(int M, int N, int K, int64_t scratch) { return mx::plan_within(M, N, K, compute_units(), scratch); }
bool mx_one_launch(int M, int N, int K) { return mx::rows_fit(M, N, K, compute_units()); }

int64_t mx_workspace_bytes(const MxPlan& p) { return mx::part_bytes(p); }

hipError_t launch_gemm_mxfp4(const uint8_t* Xq, const uint8_t* sx, const uint8_t* Wq, const uint8_t* sw, const uint16_t* bias,
                             int M, int N, int K, bool bf16, uint16_t* Y, float* part, const MxPlan& plan,
                             hipStream_t stream) {
  if (bf16)
    launch<Bf16>(Xq, sx, Wq, sw, bias, M, N, K, Y, part, plan, stream);
  else
    launch<Fp16>(Xq, sx, Wq, sw, bias, M, N, K, Y, part, plan, stream);
  return hipGetLastError();
}

hipError_t launch_linear_rows_mxfp4(const uint16_t* X, int64_t ldx, const uint8_t* Wq, const uint8_t* sw, const uint16_t* bias,
                                    int M, int N, int K, bool bf16, uint16_t* Y, hipStream_t stream) {
  const bool vec = K % 8 == 0 && (M == 1 || ldx % 8 == 0) && (reinterpret_cast<uintptr_t>(X) & 15) == 0;
  if (bf16)
    vec ? launch_rows<Bf16, true>(X, ldx, Wq, sw, bias, M, N, K, Y, stream)
        : launch_rows<Bf16, false>(X, ldx, Wq, sw, bias, M, N, K, Y, stream);
  else
    vec ? launch_rows<Fp16, true>(X, ldx, Wq, sw, bias, M, N, K, Y, stream)
        : launch_rows<Fp16, false>(X, ldx, Wq, sw, bias, M, N, K, Y, stream);
  return hipGetLastError();
}

}  // namespace atom
