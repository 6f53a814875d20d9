// Pieces that the tiled GEMM kernels with stages of whole cache lines share (gemm_w8a8.hip, gemm_mxfp4.hip).
#pragma once

#include "serve_internal.h"

namespace atom {

constexpr int kStage = 128;   // bytes of K of one stage: a cache line of each row

// Position of 16-byte chunk c of staged row r: two rows cover the banks once, and the next bits of the row
// choose one of the eight positions.
__device__ __forceinline__ int pos(int r, int c) { return c ^ ((r >> 1) & 7); }

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

// Order of a slice: NM products, each followed by its share of ND LDS reads and NV copies.  Left to itself the
// compiler puts the reads behind the products, so that every slice ends in a wait for LDS.
template <int NM, int ND, int NV>
__device__ __forceinline__ void interleave() {
  if constexpr (NM > 0) {
    constexpr int nd = (ND + NM - 1) / NM, nv = (NV + NM - 1) / NM;
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    if constexpr (nd > 0) __builtin_amdgcn_sched_group_barrier(0x100, nd, 0);
    if constexpr (nv > 0) __builtin_amdgcn_sched_group_barrier(0x020, nv, 0);
    interleave<NM - 1, ND - nd, NV - nv>();
  }
}

}  // namespace atom
