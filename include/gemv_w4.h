/*
 * gemv_w4 -- products of a few rows with 4-bit weights on AMD Instinct MI355X
 * (gfx950): the serving form of a linear layer.
 *
 *   Y = X W^T      W[n][k] = (Q[n][k] - zero[n][k / group]) * scale[n][k / group]
 *
 *   X       [M, K]          binary16 or bfloat16, rows ldx elements apart
 *   Q       [N, K / 2]      bytes: the low half holds the code of even k, the
 *                           high half that of the odd k after it (0 .. 15);
 *                           rows ldq bytes apart
 *   scale   [N, K / group]  of X's type, rows adjacent
 *   zero    [N, K / group]  of X's type (any value of it), or NULL: 8
 *   Y       [M, N]          of X's type, rows ldy elements apart
 *
 * Codes enter the matrix cores as whole numbers, which both types hold
 * exactly (binary16: code - 8; bfloat16: code + 128); a group's sum is
 * multiplied by its scale in 32 bits, and zero points, with the offset, enter
 * as (zero + offset) * (sum of the group's x).  Y is rounded once, to nearest
 * even.  The order of the additions is fixed for given sizes.
 *
 * Infinities and NaN in X, scale and zero give what the definition gives,
 * and large finite X do not overflow on the way: results that are not finite
 * are computed again term by term in 64 bits, unless their row of X begins
 * with a NaN.  That costs time where rows hold infinities or a later NaN (one
 * such row: 57 us for 8192 x 4096 weights instead of 9).
 *
 * M may be any number of rows: one to sixteen cost the same, since reading
 * the weights is all the work; further on each 32 rows (small results) or 64
 * read the weights again.
 *
 * Ownership, concurrency, errors and capture are those of gemm_nt_f16.h; no
 * workspace is needed.
 *
 * hipErrorInvalidValue before anything is enqueued: a negative size or one of
 * 2^31 or more, K no multiple of 32 or of group, K of 2^21 or more, a group
 * that is neither a power of two from 32 on nor K itself, a pitch below the
 * row, ldx or ldq above 2^23, ldq no multiple of 16, Q not 16-byte aligned,
 * an unknown type, a null or odd pointer with a non-zero extent, Y meeting an
 * input, more tiles than a launch can hold (N of 2^27 or more; 2^22 tiles of
 * 64 x 64).  M == 0 or N == 0 writes nothing; K == 0 writes +0.
 *
 * Any 2-byte aligned X is accepted, but rows of it that do not start on 16
 * bytes are read element by element, 16 at a time (4096 x 4096 weights, 16
 * and 64 rows: 21 and 77 us, and 8 and 11 for aligned ones).
 */
#ifndef GEMV_W4_H
#define GEMV_W4_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct ihipStream_t* hipStream_t;

#define GEMV_W4_VERSION 1

enum { GEMV_W4_F16 = 0, GEMV_W4_BF16 = 1 };

int gemv_w4(const void* X, const void* Q, const void* scale, const void* zero, void* Y, int64_t M, int64_t N,
            int64_t K, int64_t group, int64_t ldx, int64_t ldq, int64_t ldy, int32_t type, hipStream_t stream);

/* GEMV_W4_VERSION of the built library. */
int gemv_w4_version(void);

#ifdef __cplusplus
}
#endif

#endif /* GEMV_W4_H */
