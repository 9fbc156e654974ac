/*
 * dropout -- dropout on AMD Instinct MI355X (gfx950) whose mask is computed, not
 * stored, with the sum of a residual.
 *
 *   Y[r, c] = keep(r cols + c) ? X[r, c] s : 0,  + residual[r, c] if given
 *
 *   X, residual, Y  [rows, cols]   rows ldx, ldr, ldy apart, the elements of a row adjacent
 *
 * All are binary16 (type DROPOUT_F16), bfloat16 (DROPOUT_BF16) or binary32
 * (DROPOUT_F32); product and sum are in 32 bits, rounded once, to nearest even.
 * What is dropped is chosen, not multiplied: a NaN or an infinity there is gone.
 *
 * The mask.  Element e = r cols + c draws 16 bits u(e) and is kept if
 * u(e) >= d, d = p 65536 to the nearest whole number: p is held to 2^-17, and
 * s = 65536 / (65536 - d) is the inverse of the share that is kept.  (p == 1
 * keeps nothing.)  The bits are those of Philox 4x32 with ten rounds (Salmon,
 * Moraes, Dror, Shaw: Parallel random numbers: as easy as 1, 2, 3, 2011): key =
 * seed (low word first), counter = (block low, block high, offset low, offset high)
 * with block = e / 8; u(e) is half e % 8 of the four words, low halves first.
 * Different offsets give independent masks: number the calls with them.  The
 * mask depends on seed, offset, p and the element's number alone, not on type,
 * pitch or device.
 *
 * The backward pass is the same call on the gradient of Y, without a residual,
 * whose own gradient is that of Y.
 *
 * `state`, unless NULL, is two 64-bit numbers in device memory, read when the
 * call runs: seed = state[0], offset = state[1] + `offset` (modulo 2^64), and
 * the argument `seed` is not used.  A captured graph then draws new masks on each
 * replay.
 *
 * Ownership, concurrency, errors and capture are those of gemm_nt_f16.h: the
 * caller owns every buffer, calls enqueue on `stream` and return a hipError_t
 * as int.  No workspace.
 *
 * hipErrorInvalidValue before anything is enqueued: a negative size or one
 * above 2^31 - 1, a row pitch below the row or above 2^31 - 1, a matrix that
 * spans 2^58 elements or more, an unknown type, p outside 0 .. 1 or NaN, a null
 * or misaligned pointer with a non-zero extent (elements on their size, state on
 * 8 bytes), a Y whose first-to-last-element range meets an input's, unless that
 * input is Y itself (same pointer and pitch: in place).
 *
 * rows == 0 or cols == 0 writes nothing.  Any pointers aligned to their elements
 * and any pitches are accepted.
 */
#ifndef DROPOUT_H
#define DROPOUT_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct ihipStream_t* hipStream_t;

#define DROPOUT_VERSION 1

enum { DROPOUT_F16 = 0, DROPOUT_BF16 = 1, DROPOUT_F32 = 2 };

int dropout(const void* X, const void* residual, void* Y, int64_t rows, int64_t cols, int64_t ldx, int64_t ldr, int64_t ldy,
            int32_t type, double p, uint64_t seed, uint64_t offset, const uint64_t* state, hipStream_t stream);

/* DROPOUT_VERSION of the built library. */
int dropout_version(void);

#ifdef __cplusplus
}
#endif

#endif /* DROPOUT_H */
