/*
 * atom_norm.h -- C ABI of the root-mean-square norm in front of the quantized layers on MI355X
 * (gfx950): the residual's addition, the norm and the rows' quantization in one pass.
 *
 * For a row x (and r) of K elements, weights w and eps > 0:
 *   h = round(fl32(x + r)) in the rows' own type (h = x without a residual),
 *   y = h * w / sqrt(mean(h^2) + eps), not rounded,
 * and y's codes and scales are those of atom_quantize_w8a8 (s = fl32(max|y| / 127), code = clamp(
 * rint_even(y / s), -127, 127)) or of atom_quantize_mxfp4.  The products h * w are taken in fp32 (exact for fp16; for
 * bf16 while they lie between 2^-110 and 2^127), everything else in 64 bits with one rounding a step: the sum of squares (in an
 * order of the kernel's own), its division by K, the root, the division by it and by s.  Codes and scales are those of these
 * steps bit for bit: a value on the border of two codes goes the formulas' way wherever the sum of squares is exact, and
 * else one within a few 2^-53 of a border may go either way.
 * A row that holds an inf or NaN, or an h * w beyond fp32, gets unspecified codes and scales (no fault).
 *
 * The conventions of atom.h hold, with those of atom_w8a8.h for `dtype` and rows: X, residual and H rows
 * lie ldx, ldr, ldh elements apart (at least K) and need only the alignment of their elements, as does `weight`; every
 * other pointer is 16-byte aligned.
 */
#ifndef ATOM_NORM_H_
#define ATOM_NORM_H_

#include <stdint.h>

#include "atom_mxfp4.h"
#include "atom_w8a8.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 *   X, residual : const fp16 / bf16 [rows, K]; residual may be NULL, H then too
 *   weight      : const fp16 / bf16 [K]
 *   H           : fp16 / bf16 [rows, K] (output); may be the residual or X itself (the same address and
 *                 stride), which is then replaced by the sum
 *   Xq, sx      : as atom_quantize_w8a8 / atom_quantize_mxfp4 write them       (outputs)
 */
int atom_rmsnorm_w8a8(const void *X, int64_t ldx, const void *residual, int64_t ldr, const void *weight, double eps,
                      int32_t dtype, int32_t rows, int32_t K, void *H, int64_t ldh, void *Xq, float *sx, void *stream);
int atom_rmsnorm_mxfp4(const void *X, int64_t ldx, const void *residual, int64_t ldr, const void *weight, double eps,
                       int32_t dtype, int32_t rows, int32_t K, void *H, int64_t ldh, void *Xq, void *sx, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* ATOM_NORM_H_ */
