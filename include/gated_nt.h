/*
 * gated_nt -- the gated linear layer of a feed-forward block on AMD Instinct
 * MI355X (gfx950): both projections, the activation and the product in one
 * kernel, and its backward pass.
 *
 *   g = X Wg^T    u = X Wu^T    H = act(g) * u
 *
 *   X  [T, D]   rows ldx elements apart      Wg, Wu [F, D]   ldg, ldu apart
 *   H  [T, F]   rows ldh apart
 *
 * All are binary16 (type GATED_NT_F16) or bfloat16 (GATED_NT_BF16), the
 * elements of a row adjacent.  Sums, the activation and the product are in
 * 32 bits; H is rounded once, to nearest even.
 *
 *   act(g) = g * sigmoid(z),  z = g                                  (GATED_NT_SILU)
 *                             z = 2 sqrt(2/pi) (g + 0.044715 g^3)    (GATED_NT_GELU_TANH)
 *
 * Backward pass, for the gradient dH of H:
 *
 *   dG = dH * u * act'(g)     dU = dH * act(g)      (each rounded once to the type)
 *   dX = dG Wg + dU Wu        dWg = dG^T X          dWu = dU^T X
 *
 * with sums in 32 bits.  It reads what the forward pass kept in `saved`:
 * u * act'(g) and act(g) in 32 bits, in a layout of the library's own,
 * gated_nt_saved_bytes(T, F) bytes.  Kept in 32 bits they add nothing to the
 * gradients' error; in the operands' type each would add as much as the
 * final rounding does.
 *
 * The rounding of dG and dU adds about as much to a gradient's error as its own
 * rounding (sqrt 2 of it in all).  In binary16 they are held times a power of
 * two that follows dH's largest finite entry, so this holds for dH of any size;
 * entries of dG and dU below 2^-10 of dH's largest lose bits, and ones above
 * 2^19 times it overflow.
 *
 * Ownership, concurrency, errors and capture are those of gemm_nt_f16.h: the
 * caller owns every buffer, calls enqueue on `stream` and return a hipError_t
 * as int.  A call that needs a workspace takes it from the caller
 * (gated_nt_workspace, gated_nt_backward_workspace; 16-byte aligned); it may
 * be reused or freed by work enqueued later on the same stream.
 *
 * hipErrorInvalidValue before anything is enqueued: a negative size, T above
 * 2^31 - 257 (2^21 - 64 in the backward pass, whose sums run over T), D above
 * 2^21 - 64, F above 2^20 - 64, a result of more tiles than a launch can hold
 * (2^23 of 256 x 128), a row pitch below the row or of 2^21 or more, an
 * unknown type or activation, a null or odd pointer with a non-zero extent, `saved`
 * not 16-byte aligned, an output whose first-to-last-element range meets an
 * input's, another output's or the workspace's, a workspace that is too small.
 *
 * T == 0 or F == 0 writes no H; a sum over nothing (D == 0, or T == 0 and
 * F == 0 in the gradients) is +0.
 *
 * Any 2-byte aligned pointers and any sizes are accepted.  The kernels read
 * 16 bytes at a time: an operand whose pointer is not 16-byte aligned or
 * whose pitch or D is no multiple of 8 is first copied into the workspace
 * (all such in one launch; 160 x 539 x 1434: 14 us, and 10 with D = 544).
 * Copied weights cross memory three times, which is most of the time of a few
 * rows: one row by 8192 x 4097 takes 87 us and a workspace of 136 MB, by 8192 x
 * 4096 30 us and none.  The backward pass lays out both weights anew whatever T
 * is (one row by 8192 x 4096: 136 us).
 */
#ifndef GATED_NT_H
#define GATED_NT_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct ihipStream_t* hipStream_t;

#define GATED_NT_VERSION 1

enum { GATED_NT_F16 = 0, GATED_NT_BF16 = 1 };
enum { GATED_NT_SILU = 0, GATED_NT_GELU_TANH = 1 };

/* H, and `saved` for the backward pass unless it is NULL. */
int gated_nt(const void* X, const void* Wg, const void* Wu, void* H, void* saved,
             int64_t T, int64_t D, int64_t F, int64_t ldx, int64_t ldg, int64_t ldu, int64_t ldh,
             int32_t type, int32_t activation, void* workspace, int64_t workspace_bytes,
             hipStream_t stream);

/* dX [T, D], dWg and dWu [F, D] (rows lddx, lddg, lddu apart) from dH [T, F]
 * (lddh), the forward pass's operands and what it saved. */
int gated_nt_backward(const void* dH, const void* X, const void* Wg, const void* Wu, const void* saved,
                      void* dX, void* dWg, void* dWu, int64_t T, int64_t D, int64_t F,
                      int64_t lddh, int64_t ldx, int64_t ldg, int64_t ldu,
                      int64_t lddx, int64_t lddg, int64_t lddu, int32_t type,
                      void* workspace, int64_t workspace_bytes, hipStream_t stream);

/* Bytes of `saved`; of the forward call's workspace for these operands (0 if
 * they can be read as they are); of the backward call's workspace.  -1 for
 * invalid sizes.  Host-only. */
int64_t gated_nt_saved_bytes(int64_t T, int64_t F);
int64_t gated_nt_workspace(const void* X, const void* Wg, const void* Wu, int64_t T, int64_t D, int64_t F,
                           int64_t ldx, int64_t ldg, int64_t ldu);
int64_t gated_nt_backward_workspace(int64_t T, int64_t D, int64_t F);

/* GATED_NT_VERSION of the built library. */
int gated_nt_version(void);

#ifdef __cplusplus
}
#endif

#endif /* GATED_NT_H */
