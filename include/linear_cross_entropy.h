/*
 * linear_cross_entropy -- the softmax cross entropy of a linear layer's outputs
 * over a large vocabulary on AMD Instinct MI355X (gfx950), without keeping the
 * outputs, and its gradients.
 *
 *   l = X W^T    loss[t] = log sum_v exp(l[t, v]) - l[t, target[t]]
 *
 *   X  [T, D]   rows ldx elements apart      W  [V, D]   ldw apart
 *   target  [T] 64-bit whole numbers, target_stride apart      loss  [T] binary32
 *
 * X and W are binary16 (type LINEAR_CROSS_ENTROPY_F16) or bfloat16
 * (LINEAR_CROSS_ENTROPY_BF16), the elements of a row adjacent.  The outputs l
 * are 32-bit sums that never leave the chip unrounded or rounded: of each row and
 * piece of the vocabulary only the largest l and the sum of exp(l - largest) are
 * kept, in 32 bits, and joined in a fixed order.
 *
 * A token whose target is ignore_index has loss 0 and adds nothing to the
 * gradients, whatever its row of X holds (NaN and infinities too).  A target
 * that is neither that nor in 0 .. V - 1 gives NaN, in its loss, its row of dX and all of dW.
 *
 * Backward pass, for the gradient dloss [T] (binary32, dloss_stride apart; 0
 * repeats one number) of loss:
 *
 *   dl[t, v] = softmax(l)[t, v] - (v == target[t])
 *   dX[t] = dloss[t] sum_v dl[t, v] W[v]       dW[v] = sum_t (dloss[t] dl[t, v]) X[t]
 *
 * with sums in 32 bits.  It reads what the forward pass kept in `saved` ([T, 3]
 * binary32: the largest l, the sum, the target's l) and computes l again, a piece
 * of the vocabulary at a time.  dl is rounded once to the type for dX, and once,
 * times dloss over dloss' largest finite magnitude, for dW, to be the operand of
 * one matrix product each; for dX what rounding takes from the target's dl is put
 * back.  This adds at most about as much to a gradient's error as its own
 * rounding (sqrt 2 of it in all: 2.4e-4 off for 1000 x 1032 x 32001 in binary16, 2.1e-4
 * with dl in 32 bits; 1.8e-3 and 1.7e-3 for 8192 x 4096 x 131072 in bfloat16).  A high
 * and a low part of dl would keep its bits for both products a second time, about 47%
 * of that large step.  In binary16 both are held times 2^15: probabilities down to
 * 2^-29 keep all bits, and dloss may have any size.
 *
 * Ownership, concurrency, errors and capture are those of gemm_nt_f16.h: the
 * caller owns every buffer, calls enqueue on `stream` and return a hipError_t
 * as int.  Workspaces come from the caller (16-byte aligned); they may be reused
 * or freed by work enqueued later on the same stream.
 *
 * hipErrorInvalidValue before anything is enqueued: a negative size, V == 0, T
 * above 2^27 (2^21 - 64 in the backward pass, whose sums run over T), V above
 * 2^31 - 257, D above 2^21 - 64, a result or operands of more tiles than a launch
 * can hold, a row pitch below the row or of 2^21 or more, a negative stride or
 * one above 2^31, an unknown type, a null or misaligned pointer with a non-zero
 * extent (elements on their size), an output whose first-to-last-element range
 * meets an input's, another output's or the workspace's, a workspace that is
 * too small.
 *
 * T == 0 writes no loss and zeros to dW; D == 0 makes every l zero.  Any 2-byte
 * aligned X, W, dX and dW and any sizes are accepted.  The kernels read 16 bytes at
 * a time: of more than 16 tokens an X or W whose pointer is not 16-byte aligned or
 * whose pitch or D is no multiple of 8 is first copied into the workspace (181
 * tokens by 109366 x 333: 70 us of a step's 322).
 *
 * Up to 16 tokens have kernels of their own, which read W where it lies, hold dl
 * in 32 bits and never round it (the gradients' only rounding is their own).
 */
#ifndef LINEAR_CROSS_ENTROPY_H
#define LINEAR_CROSS_ENTROPY_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct ihipStream_t* hipStream_t;

#define LINEAR_CROSS_ENTROPY_VERSION 1

enum { LINEAR_CROSS_ENTROPY_F16 = 0, LINEAR_CROSS_ENTROPY_BF16 = 1 };

/* loss, and `saved` for the backward pass unless it is NULL. */
int linear_cross_entropy(const void* X, const void* W, const int64_t* target, float* loss, float* saved, int64_t T,
                         int64_t D, int64_t V, int64_t ldx, int64_t ldw, int64_t target_stride, int32_t type,
                         int64_t ignore_index, void* workspace, int64_t workspace_bytes, hipStream_t stream);

/* dX [T, D] and dW [V, D] (rows lddx, lddw apart) from dloss, the forward
 * pass's operands and what it saved. */
int linear_cross_entropy_backward(const float* dloss, const void* X, const void* W, const int64_t* target,
                                  const float* saved, void* dX, void* dW, int64_t T, int64_t D, int64_t V,
                                  int64_t dloss_stride, int64_t ldx, int64_t ldw, int64_t target_stride, int64_t lddx,
                                  int64_t lddw, int32_t type, int64_t ignore_index, void* workspace,
                                  int64_t workspace_bytes, hipStream_t stream);

/* Bytes of the calls' workspaces for these operands; -1 for invalid sizes.  Host-only.
 *
 * Above 16 tokens, forward: 8 bytes for each token and 32 words (64, of more than 2^26
 * outputs), what is copied of X and W, and 32 MB from D 505 on.  Backward: dl of a piece
 * of the vocabulary twice, each of up to 2^27 elements of 2 bytes, or 1024 to a token if
 * that is more; X transposed, what is copied of X and of a piece of W, a transpose of the
 * piece where the products run faster on one (some thousand tokens of long rows), 4 D
 * bytes to a token where there are several pieces, and 32 MB.  (1000 x 4096 x 131072:
 * 48 MB and 546 MB.) */
int64_t linear_cross_entropy_workspace(const void* X, const void* W, int64_t T, int64_t D, int64_t V, int64_t ldx,
                                       int64_t ldw);
int64_t linear_cross_entropy_backward_workspace(const void* X, const void* W, int64_t T, int64_t D, int64_t V,
                                                int64_t ldx, int64_t ldw);

/* LINEAR_CROSS_ENTROPY_VERSION of the built library. */
int linear_cross_entropy_version(void);

#ifdef __cplusplus
}
#endif

#endif /* LINEAR_CROSS_ENTROPY_H */
