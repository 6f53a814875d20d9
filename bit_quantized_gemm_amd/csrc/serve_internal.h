// Internal declarations of the W8A8 layer and the 4-bit KV cache, shared by their host APIs and
// kernels.  Every launcher enqueues on `stream` and returns hipGetLastError() after its launches;
// arguments are validated by the caller before any launcher runs.
#pragma once

#include <hip/hip_runtime.h>
#include <hip/hip_fp16.h>
#include <stdint.h>

#include "atom_kv4.h"
#include "atom_mxfp4.h"
#include "atom_norm.h"
#include "atom_w8a8.h"
#include "kv4_plan.h"
#include "mxfp4_plan.h"

namespace atom {

// ---- 16-bit element types: fp16 and bf16 as template parameters of the kernels
typedef _Float16 h2v __attribute__((ext_vector_type(2)));
typedef _Float16 h8v __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

struct Fp16 {
  static __device__ __forceinline__ float load(uint32_t bits) { return (float)__builtin_bit_cast(_Float16, (uint16_t)bits); }
  static __device__ __forceinline__ uint16_t store(float f) { return __builtin_bit_cast(uint16_t, (_Float16)f); }
};
struct Bf16 {
  static __device__ __forceinline__ float load(uint32_t bits) { return __builtin_bit_cast(float, (bits & 0xFFFFu) << 16); }
  static __device__ __forceinline__ uint16_t store(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }   // RNE
};
// Elements 0 and 1 of a 32-bit word.
template <class T>
__device__ __forceinline__ float elem(uint32_t w, int i) { return T::load(i ? w >> 16 : w & 0xFFFFu); }
template <class T>
__device__ __forceinline__ uint32_t pack2(float a, float b) { return (uint32_t)T::store(a) | (uint32_t)T::store(b) << 16; }

// A quotient with the nearest integer of fl32(x / s): the product with the correctly rounded reciprocal r, corrected once.
// For 8- and 11-bit x against the scales of both quantizers (fl32(max / 127); any fp16 value) this was walked over every pair of
// significands (tests/test_serve_arith.py): fl32(x / s) lies exactly on a border between two codes for common x, such
// as max / 2, and an uncorrected product falls on either side of it.  s = 0: r = 0, and 0 for x = 0.
__device__ __forceinline__ float quotient(float x, float s, float r) {
  const float q = x * r;
  return __builtin_fmaf(__builtin_fmaf(-q, s, x), r, q);
}

// ---- W8A8
hipError_t launch_quantize_w8a8(const uint16_t* X, int64_t ldx, bool bf16, int rows, int K, int8_t* Xq, float* sx,
                                hipStream_t stream);

// How a W8A8 product is run: kind 0 is the few-rows kernel, 1.. the tiled kernels' tile sizes;
// `splits` workgroups divide K for each output tile (their integer parts are added by a second
// kernel from scratch).
struct W8Plan {
  int kind, tiles, splits;
};
W8Plan w8_plan(int M, int N, int K);
int64_t w8_workspace_bytes(const W8Plan& plan);
hipError_t launch_gemm_w8a8(const int8_t* Xq, const float* sx, const int8_t* Wq, const float* sw, const uint16_t* bias,
                            int M, int N, int K, bool bf16, uint16_t* Y, int32_t* part, const W8Plan& plan,
                            hipStream_t stream);

// The whole layer in one launch, for so few tokens that every workgroup may quantize them for itself.
bool linear_rows_fits(int M, int N, int K);
hipError_t launch_linear_rows(const uint16_t* X, int64_t ldx, const int8_t* Wq, const float* sw, const uint16_t* bias,
                              int M, int N, int K, bool bf16, uint16_t* Y, hipStream_t stream);

hipError_t launch_dequantize_w8a8(const int8_t* Xq, const float* sx, int rows, int K, bool bf16, uint16_t* X,
                                  hipStream_t stream);

// ---- MXFP4
hipError_t launch_quantize_mxfp4(const uint16_t* X, int64_t ldx, bool bf16, int rows, int K, uint8_t* Xq, uint8_t* sx,
                                 hipStream_t stream);
hipError_t launch_dequantize_mxfp4(const uint8_t* Xq, const uint8_t* sx, int rows, int K, bool bf16, uint16_t* X,
                                   hipStream_t stream);
using MxPlan = mx::Plan;
MxPlan mx_plan(int M, int N, int K, int64_t scratch);   // for this device's compute units and as much scratch memory
bool mx_one_launch(int M, int N, int K);                 // whether launch_linear_rows_mxfp4 takes the layer
int64_t mx_workspace_bytes(const MxPlan& plan);
hipError_t launch_gemm_mxfp4(const uint8_t* Xq, const uint8_t* sx, const uint8_t* Wq, const uint8_t* sw, const uint16_t* bias,
                             int M, int N, int K, bool bf16, uint16_t* Y, float* part, const MxPlan& plan,
                             hipStream_t stream);
hipError_t launch_linear_rows_mxfp4(const uint16_t* X, int64_t ldx, const uint8_t* Wq, const uint8_t* sw, const uint16_t* bias,
                                    int M, int N, int K, bool bf16, uint16_t* Y, hipStream_t stream);

// ---- norm in front of the quantized layers; R and H are null together
struct NormCall {
  const uint16_t* X;
  int64_t ldx;
  const uint16_t* R;
  int64_t ldr;
  const uint16_t* W;
  double eps;
  bool bf16;
  int rows, K;
  uint16_t* H;
  int64_t ldh;
  uint8_t* Xq;
  void* sx;
};
hipError_t launch_rmsnorm(const NormCall& n, bool mx, hipStream_t stream);

// ---- KV cache's bookkeeping
struct Kv4Extend {
  const int32_t *lens, *more;
  int32_t* table;
  int batch, width, log_page;
  const int32_t* free_pages;
  int capacity;
  const int32_t* state;
  int64_t* slots;
  int total;
  int32_t *start, *lens_out, *state_out;
};
hipError_t launch_kv4_extend(const Kv4Extend& a, hipStream_t stream);
struct Kv4Release {
  const uint8_t* done;
  const int32_t *lens, *table;
  int batch, width, log_page;
  int32_t* free_pages;
  int capacity;
  const int32_t* state;
  int32_t *lens_out, *state_out;
};
hipError_t launch_kv4_release(const Kv4Release& a, hipStream_t stream);

// ---- KV cache
hipError_t launch_kv4_append(const uint16_t* K, int64_t k_stride, const uint16_t* V, int64_t v_stride,
                             const int64_t* slots, int tokens, bool bf16, const atom_kv4_cache& c, hipStream_t stream);
hipError_t launch_kv4_read(const atom_kv4_cache& c, const int64_t* slots, int tokens, bool bf16, uint16_t* K,
                           uint16_t* V, hipStream_t stream);

struct Kv4Attention {
  const uint16_t* q;
  int64_t q_stride;
  atom_kv4_cache cache;
  const int32_t *table, *lens, *q_start;
  int width, total_q, q_heads, batch, max_q, max_len;
  float scale;
  bool bf16;
  uint16_t* out;
};
using Kv4Plan = kv4::Plan;
Kv4Plan kv4_plan(int q_heads, int heads, int dim, int batch, int max_q, int max_len);   // for this device's compute units
int64_t kv4_workspace_bytes(const Kv4Plan& plan, int total_q, int q_heads, int dim);
hipError_t launch_kv4_attention(const Kv4Attention& a, const Kv4Plan& plan, float* work, hipStream_t stream);

}  // namespace atom
