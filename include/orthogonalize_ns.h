/*
 * orthogonalize_ns -- Newton-Schulz orthogonalisation of an update matrix on
 * AMD Instinct MI355X (gfx950), as the Muon optimiser applies it to the
 * momentum of a weight.
 *
 *   X <- G / (|G|_F + eps)
 *   steps times, with (a, b, c) of that step:  X <- a X + (b S + c S S) X,  S = X X^T
 *
 * The polynomial acts on the singular values alone, so it is the same from
 * either side: the kernels work on the side with the shorter rows count.
 *
 *   G    [batch, rows, cols]  binary16, bfloat16 or 32-bit floats; rows ldg
 *                             elements apart, matrices stride_g apart
 *   out  [batch, rows, cols]  bfloat16; ldo, stride_o
 *
 * |G|_F is summed in 64 bits, the products' sums are in 32 bits.  X, S and
 * the polynomial aI + bS + cSS are held in binary16 between the products,
 * which is 8 times finer than the bfloat16 that the update is usually computed
 * in; what rounding takes from the polynomial's diagonal, its largest part, is
 * put back into the product's rows.  The result is therefore bfloat16,
 * whatever G's type.
 *
 * Error, |out - exact|_F over |exact|_F, as a multiple of what rounding the
 * exact result alone leaves (1.66e-3), five steps:
 *   noise, sides from 1 to 9000                           1.05 to 1.4
 *   256 x 1024, singular values that fall evenly in the
 *   logarithm from 1 to 10^-1, 10^-2, 10^-4, 10^-6        1.2, 2.4, 5.6, 7.4
 * The steps amplify small singular values by up to 3.4 each, and with them the
 * rounding of the X that they are part of.
 *
 * X, S and the polynomial are held times powers of two that use binary16's
 * range: entries of X (at first G's over |G|_F) lose bits below 2^-28 and are
 * lost below 2^-38.  Of 256 x 1024 of noise rows and columns 10^-6 of the others
 * are as near the exact result as those, 10^-7 0.7% off; of 4096 x 4096 10^-5 as
 * near, 10^-6 0.5% and 10^-7 5% off.  With polynomials that blow values up past 65504
 * the result is not finite.
 *
 * With steps > 0 a matrix that holds an infinity or a NaN gives NaN; with none,
 * G / inf.  The zero matrix gives zeros, and 0 / 0 with eps = 0.
 *
 * Ownership, concurrency, errors and capture are those of gemm_nt_f16.h.  The
 * workspace (orthogonalize_ns_workspace bytes, 16-byte aligned) is the
 * caller's and may be reused by work enqueued later on the same stream.
 *
 * hipErrorInvalidValue before anything is enqueued: a negative size, a size
 * above 2^21 - 64 in rows or cols, batch of 2^16 or more, a pitch below the
 * row, ldo of 2^21 or more, matrices of out that do not lie one after
 * another, an unknown type, steps below 0 or above 64, null coefficients with
 * steps > 0, eps below 0 or NaN, a null or misaligned pointer with a non-zero
 * extent, out or the workspace meeting G or each other, a workspace that is
 * too small, more tiles than a launch can hold (2^24 of 64 x 64).
 */
#ifndef ORTHOGONALIZE_NS_H
#define ORTHOGONALIZE_NS_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct ihipStream_t* hipStream_t;

#define ORTHOGONALIZE_NS_VERSION 1

enum { ORTHOGONALIZE_NS_F16 = 0, ORTHOGONALIZE_NS_BF16 = 1, ORTHOGONALIZE_NS_F32 = 2 };

/* coefficients: 3 * steps doubles in host memory, (a, b, c) of each step;
 * read before the call returns. */
int orthogonalize_ns(const void* G, void* out, int64_t batch, int64_t rows, int64_t cols, int64_t ldg,
                     int64_t stride_g, int64_t ldo, int64_t stride_o, int32_t type, int32_t steps,
                     const double* coefficients, double eps, void* workspace, int64_t workspace_bytes,
                     hipStream_t stream);

/* Bytes of the workspace; -1 for invalid sizes.  Host-only. */
int64_t orthogonalize_ns_workspace(int64_t batch, int64_t rows, int64_t cols);

/* ORTHOGONALIZE_NS_VERSION of the built library. */
int orthogonalize_ns_version(void);

#ifdef __cplusplus
}
#endif

#endif /* ORTHOGONALIZE_NS_H */
