/*
 * atom_w8a8.h -- C ABI of the W8A8 linear layer on MI355X (gfx950): 8-bit integer codes on both
 * sides, one scale for each token and one for each output channel.
 *
 * For layers that do not stand the 4-bit codes of atom.h.  With x a row of X, w a row of W:
 *   sx = fl32(max|x| / 127),   qx = clamp(rint_even(fl32(x / sx)), -127, 127),  0 where sx = 0,
 *   likewise (sw, qw) for w;   Y[m,n] = round(acc * sx[m] * sw[n] + bias[n]),  acc = sum_k qx * qw.
 * acc is an exact 32-bit integer (127 * 127 * ATOM_MAX_K < 2^31); the scaling and the bias are
 * fp32, acc * sx[m] first (which therefore has to be below 2^128), and Y is rounded once.
 *
 * The conventions of atom.h hold (device pointers owned by the caller, no allocation, no
 * synchronization, arguments checked on the host first, ATOM_E_* returned), except that
 *   - X and Y are fp16 or bf16 (`dtype`), scales are fp32;
 *   - any K with 1 <= K <= ATOM_MAX_K: packed rows are atom_w8a8_row_bytes(K) bytes long, the
 *     codes behind K are zero;
 *   - rows of X lie ldx elements apart (ldx >= K) and need only the alignment of their elements;
 *     16-byte aligned rows are read with wide loads.  Every other pointer is 16-byte aligned.
 */
#ifndef ATOM_W8A8_H_
#define ATOM_W8A8_H_

#include <stdint.h>

#include "atom.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { ATOM_FP16 = 0, ATOM_BF16 = 1 };

/* Bytes of one packed row: K rounded up to a multiple of 128; -ATOM_E_SHAPE for an invalid K. */
int64_t atom_w8a8_row_bytes(int32_t K);

/*
 * Codes and scales of the rows of X: activations at run time, weights offline (rows = output
 * channels).  A row that holds an inf or NaN gets unspecified codes and scale (no fault).
 *   X  : const fp16 / bf16 [rows, K], row stride ldx
 *   Xq : int8 [rows, row bytes]      sx : float [rows]                        (outputs)
 */
int atom_quantize_w8a8(const void *X, int64_t ldx, int32_t dtype, int32_t rows, int32_t K, void *Xq, float *sx,
                       void *stream);

/*
 * Y from packed operands.  bias (of `dtype`, [N]) may be NULL.
 *   Xq : const int8 [M, row bytes]   sx : const float [M]
 *   Wq : const int8 [N, row bytes]   sw : const float [N]
 *   Y  : fp16 / bf16 [M, N]                                                   (output)
 * workspace: atom_gemm_w8a8_workspace_bytes(M, N, K) bytes let a grid of few output tiles divide
 * K among workgroups; with less (or NULL) it runs undivided, with the same result bit for bit:
 * the parts are integers.  Contents on entry do not matter.
 */
int64_t atom_gemm_w8a8_workspace_bytes(int32_t M, int32_t N, int32_t K);
int atom_gemm_w8a8(const void *Xq, const float *sx, const void *Wq, const float *sw, const void *bias, int32_t M,
                   int32_t N, int32_t K, int32_t dtype, void *Y, void *workspace, int64_t workspace_bytes,
                   void *stream);

/*
 * The layer in one call: quantizes X into the workspace, then Y as above; the few tokens that take one launch need none
 * (0 bytes, NULL).  The workspace holds at least atom_linear_w8a8_workspace_bytes(M, N, K) bytes (ATOM_E_SHAPE
 * otherwise); its contents on entry do not matter, and calls that may overlap in time need one each.
 */
int64_t atom_linear_w8a8_workspace_bytes(int32_t M, int32_t N, int32_t K);
int atom_linear_w8a8(const void *X, int64_t ldx, int32_t dtype, const void *Wq, const float *sw, const void *bias,
                     int32_t M, int32_t N, int32_t K, void *Y, void *workspace, int64_t workspace_bytes,
                     void *stream);

#ifdef __cplusplus
}
#endif

#endif /* ATOM_W8A8_H_ */
