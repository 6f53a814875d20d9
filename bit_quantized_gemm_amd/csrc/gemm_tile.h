// Pieces that the tiled GEMM kernels with stages of whole cache lines share (gemm_w8a8.hip, gemm_mxfp4.hip).
#pragma once

#include <hip/hip_runtime.h>

namespace atom {

constexpr int kStage = 128;   // bytes of K of one stage: a cache line of each row

// Position of 16-byte chunk c of staged row r: two rows cover the banks once, and the next bits of the row
// choose one of the eight positions.
__device__ __forceinline__ int pos(int r, int c) { return c ^ ((r >> 1) & 7); }

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
