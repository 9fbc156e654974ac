/*
 * layer_norm -- the layer norm of a matrix's rows on AMD Instinct MI355X
 * (gfx950), and its backward pass.
 *
 *   m = sum x / n    v = sum (x - m)^2 / n    r = 1 / sqrt(v + eps)    h = (x - m) r
 *   Y = h * weight + bias
 *
 *   X, Y  [rows, cols]   rows ldx, ldy apart      weight, bias  [cols], or NULL for 1 and 0
 *
 * X and Y are binary16 (type LAYER_NORM_F16), bfloat16 (LAYER_NORM_BF16) or
 * binary32 (LAYER_NORM_F32); weight and bias both of that type or both binary32
 * (param_type).  The elements of a row are adjacent.  Sums and statistics are in
 * 32 bits, the variance about the mean (two passes over a row held in
 * registers); Y is rounded once, to nearest even.
 *
 * Backward pass, for the gradient dY of Y, with g = dY * weight:
 *
 *   dX = r (g - mean(g) - h mean(g h))    dweight = sum_rows dY * h    dbias = sum_rows dY
 *
 * from X and the m and r that the forward pass kept in `saved` ([rows, 2],
 * binary32).  dX, dweight and dbias are rounded once; the sums over rows are in
 * 32 bits, in an order that the sizes fix: results repeat bit for bit.
 * dweight or dbias may be NULL: it is then not computed.
 *
 * Ownership, concurrency, errors and capture are those of gemm_nt_f16.h: the
 * caller owns every buffer, calls enqueue on `stream` and return a hipError_t
 * as int.  The backward call takes its workspace from the caller (16-byte
 * aligned); it may be reused or freed by work enqueued later on the same stream.
 *
 * hipErrorInvalidValue before anything is enqueued: a negative size or one
 * above 2^31 - 1, cols above 2^24, a row pitch below the row or above 2^31 - 1,
 * a matrix that spans 2^58 elements or more, an unknown type or a param_type
 * that is neither the type nor binary32, eps negative or NaN, a null or
 * misaligned pointer with a non-zero extent (elements on their size; `saved` on
 * 8 bytes), an output whose first-to-last-element range meets an input's,
 * another output's or the workspace's, a workspace that is too small.
 *
 * rows == 0 writes no Y and zeros to dweight and dbias; cols == 0 writes nothing.
 * Any pointers aligned to their elements and any pitches are accepted.
 */
#ifndef LAYER_NORM_H
#define LAYER_NORM_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct ihipStream_t* hipStream_t;

#define LAYER_NORM_VERSION 1

enum { LAYER_NORM_F16 = 0, LAYER_NORM_BF16 = 1, LAYER_NORM_F32 = 2 };

/* Y, and `saved` for the backward pass unless it is NULL. */
int layer_norm(const void* X, const void* weight, const void* bias, void* Y, void* saved, int64_t rows, int64_t cols,
               int64_t ldx, int64_t ldy, int32_t type, int32_t param_type, double eps, hipStream_t stream);

/* dX (rows lddx apart), dweight and dbias (of param_type) from dY (lddy), the
 * forward pass's X and weight and what it saved. */
int layer_norm_backward(const void* dY, const void* X, const void* weight, const void* saved, void* dX, void* dweight,
                        void* dbias, int64_t rows, int64_t cols, int64_t lddy, int64_t ldx, int64_t lddx, int32_t type,
                        int32_t param_type, void* workspace, int64_t workspace_bytes, hipStream_t stream);

/* Bytes of the backward call's workspace (sums of the columns, 256 MB at most, and 8 bytes
 * to a row of more than 8192 elements); -1 for invalid sizes.  Host-only. */
int64_t layer_norm_backward_workspace(int64_t rows, int64_t cols);

/* LAYER_NORM_VERSION of the built library. */
int layer_norm_version(void);

#ifdef __cplusplus
}
#endif

#endif /* LAYER_NORM_H */
