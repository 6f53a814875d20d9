/*
 * atom_mxfp4.h -- C ABI of the MXFP4 linear layer on MI355X (gfx950): microscaled 4-bit floating
 * point (the OCP Microscaling Formats specification's MXFP4: E2M1 elements, E8M0 scales) on both
 * sides.
 *
 * A row is cut into blocks of 32 values.  With a = max |x| of a block, its scale is 2^e,
 *   e = clamp(floor(log2 a) - 2, -127, 125), -127 for a block of zeros, held as the byte e + 127;
 * a value's code is the 4-bit float (sign, two bits of exponent, one of mantissa: 0, 0.5, 1, 1.5, 2, 3,
 * 4, 6) nearest to x / 2^e, ties to the even code, above 6 the code of 6; the sign of a value that rounds
 * to zero is kept.  A block that holds an inf or NaN gets the scale byte 255 (NaN) and codes of zero.
 * Y[m,n] = round(sum_k x[m,k] * w[n,k] + bias[n]) over what the codes stand for: the sum is taken
 * by the matrix cores in fp32 (each block's 32 products exactly), Y is rounded once.  A scale of NaN makes its
 * row of X (column of Y, for weights) NaN.
 *
 * Packed rows: K is padded with zeros (codes 0, scale bytes 0) to Kp, a multiple of 256.
 *   codes  : uint8 [rows, Kp / 2], value 2j of a row in the low nibble of byte j
 *   scales : uint8 [Kp / 256, rows, 8]: the eight blocks of each group of 256 values
 *
 * The conventions of atom.h hold (device pointers owned by the caller, no allocation, no synchronization,
 * arguments checked on the host first, ATOM_E_* returned), with those of atom_w8a8.h for X, Y, bias and
 * `dtype`: fp16 or bf16, any K with 1 <= K <= ATOM_MAX_K, rows of X ldx elements apart and aligned
 * to their elements; every other pointer is 16-byte aligned.
 */
#ifndef ATOM_MXFP4_H_
#define ATOM_MXFP4_H_

#include <stdint.h>

#include "atom_w8a8.h"

#ifdef __cplusplus
extern "C" {
#endif

#define ATOM_MX_BLOCK 32   /* values that share a scale */
#define ATOM_MX_GROUP 256  /* values whose eight scales lie together; K is padded to whole groups */

/* Bytes of the codes of one row (Kp / 2), and its groups (Kp / 256); -ATOM_E_SHAPE for an invalid K. */
int64_t atom_mxfp4_row_bytes(int32_t K);
int32_t atom_mxfp4_groups(int32_t K);

/*
 * Codes and scales of the rows of X: activations at run time, weights offline (rows = output channels).
 *   X  : const fp16 / bf16 [rows, K], row stride ldx
 *   Xq : uint8 [rows, row bytes]     sx : uint8 [groups, rows, 8]            (outputs)
 */
int atom_quantize_mxfp4(const void *X, int64_t ldx, int32_t dtype, int32_t rows, int32_t K, void *Xq, void *sx,
                        void *stream);

/*
 * What packed rows stand for, rounded once to `dtype` (MXFP4 values between that type's smallest and
 * largest numbers are exact).
 *   X : fp16 / bf16 [rows, K] contiguous                                      (output)
 */
int atom_dequantize_mxfp4(const void *Xq, const void *sx, int32_t rows, int32_t K, int32_t dtype, void *X,
                          void *stream);

/*
 * Y from packed operands.  bias (of `dtype`, [N]) may be NULL.
 *   Xq : const uint8 [M, row bytes]   sx : const uint8 [groups, M, 8]
 *   Wq : const uint8 [N, row bytes]   sw : const uint8 [groups, N, 8]
 *   Y  : fp16 / bf16 [M, N]                                                   (output)
 * workspace: atom_gemm_mxfp4_workspace_bytes(M, N, K) bytes let a grid of few output tiles divide K
 * among workgroups (fp32 parts added in a fixed order: repeated calls agree bit for bit); with less (or
 * NULL) the fastest kernel that needs none takes the call, in up to twice the time where K is long.  Contents on entry do not matter.
 */
int64_t atom_gemm_mxfp4_workspace_bytes(int32_t M, int32_t N, int32_t K);
int atom_gemm_mxfp4(const void *Xq, const void *sx, const void *Wq, const void *sw, const void *bias, int32_t M,
                    int32_t N, int32_t K, int32_t dtype, void *Y, void *workspace, int64_t workspace_bytes,
                    void *stream);

/*
 * The layer in one call: quantizes X into the workspace, then Y as above; few tokens, or few outputs, take
 * one launch that needs none (0 bytes, NULL).  The workspace holds at least atom_linear_mxfp4_workspace_bytes(M, N, K) bytes
 * (ATOM_E_SHAPE otherwise); its contents on entry do not matter, and calls that may overlap in time need one each.
 */
int64_t atom_linear_mxfp4_workspace_bytes(int32_t M, int32_t N, int32_t K);
int atom_linear_mxfp4(const void *X, int64_t ldx, int32_t dtype, const void *Wq, const void *sw, const void *bias,
                      int32_t M, int32_t N, int32_t K, void *Y, void *workspace, int64_t workspace_bytes,
                      void *stream);

#ifdef __cplusplus
}
#endif

#endif /* ATOM_MXFP4_H_ */
