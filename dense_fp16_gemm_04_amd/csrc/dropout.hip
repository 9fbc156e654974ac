// Dropout with a mask that is computed, and the sum of a residual, for gfx950:
// include/dropout.h.
//
// Bound by its bytes.  Ten rounds of Philox 4x32 are 20 products of 32 by 32
// bits, at a quarter of the rate of other instructions; its 128 bits therefore
// serve eight elements, 16 each, not four.  8192 x 8192 in bfloat16: 71 us with a
// residual, 5.6 TB/s, and 46 without, 5.9.
#include "dropout.h"

#include <math.h>

#include <algorithm>

#include "abi.h"
#include "cus.h"
#include "rows.h"

namespace {

using namespace rows;

constexpr int kBlock = 8;  // elements to a block of random bits
constexpr int kThreads = 256;

typedef uint32_t Words __attribute__((ext_vector_type(4)));

__device__ __forceinline__ Words philox(Words c, uint32_t k0, uint32_t k1)
{
#pragma unroll
    for (int i = 0; i < 10; ++i) {
        const uint64_t a = (uint64_t)c[0] * 0xD2511F53u, b = (uint64_t)c[2] * 0xCD9E8D57u;
        c = Words{(uint32_t)(b >> 32) ^ c[1] ^ k0, (uint32_t)b, (uint32_t)(a >> 32) ^ c[3] ^ k1, (uint32_t)a};
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return c;
}

template <class E>
struct Dropout {
    const E *X, *residual;  // residual null: none
    E* Y;
    const uint64_t* state;  // null: the two numbers here
    uint64_t seed, offset;
    int64_t cols, ldx, ldr, ldy, elements;  // (dense matrices: one row of them all)
    uint32_t drop;
    float scale;
};

// A block of eight elements to a thread.  A block inside a row (all of them, but
// one, in dense matrices) is read and written whole, any other element by element.
template <class E, bool RESIDUAL>
__global__ void __launch_bounds__(kThreads) dropout_blocks(const Dropout<E> f)
{
    typedef Vec<E, kBlock> V;
    const uint64_t seed = f.state ? f.state[0] : f.seed, offset = f.state ? f.state[1] + f.offset : f.offset;
    const uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32), o0 = (uint32_t)offset, o1 = (uint32_t)(offset >> 32);
    const int64_t blocks = (f.elements + kBlock - 1) / kBlock;
    for (int64_t b = (int64_t)blockIdx.x * kThreads + threadIdx.x; b < blocks; b += (int64_t)gridDim.x * kThreads) {
        const int64_t e0 = b * kBlock;
        int64_t row = 0, col = e0;
        if (f.cols != f.elements) {
            row = (uint64_t)f.elements >> 32 ? e0 / f.cols : (int64_t)((uint32_t)e0 / (uint32_t)f.cols);
            col = e0 - row * f.cols;
        }
        const bool whole = col + kBlock <= f.cols;
        V x, r;
        const E *px = f.X + row * f.ldx + col, *pr = RESIDUAL ? f.residual + row * f.ldr + col : nullptr;
        if (whole) {
            x = load<E, kBlock>(px, kBlock);
            if (RESIDUAL) r = load<E, kBlock>(pr, kBlock);
        }
        const Words bits = philox(Words{(uint32_t)b, (uint32_t)(b >> 32), o0, o1}, k0, k1);
        auto value = [&](int i, E xi, E ri) __attribute__((always_inline)) {
            const uint32_t u = i & 1 ? bits[i / 2] >> 16 : bits[i / 2] & 0xffffu;
            const float add = RESIDUAL ? (float)ri : 0.0f;
            return (E)(u >= f.drop ? __builtin_fmaf((float)xi, f.scale, add) : add);
        };
        if (whole) {
            V y;
#pragma unroll
            for (int i = 0; i < kBlock; ++i) y[i] = value(i, x[i], RESIDUAL ? r[i] : (E)0.0f);
            store<E, kBlock>(f.Y + row * f.ldy + col, kBlock, y);
        } else {
            const int n = (int)std::min<int64_t>(kBlock, f.elements - e0);
#pragma unroll
            for (int i = 0; i < kBlock; ++i) {
                if (i < n)
                    f.Y[row * f.ldy + col] = value(i, f.X[row * f.ldx + col], RESIDUAL ? f.residual[row * f.ldr + col] : (E)0.0f);
                if (++col == f.cols) {
                    col = 0;
                    ++row;
                }
            }
        }
    }
}

template <class E>
int launch(const Dropout<E>& f, hipStream_t stream)
{
    const int64_t blocks = (f.elements + kBlock - 1) / kBlock;
    const int64_t n = std::min<int64_t>((blocks + kThreads - 1) / kThreads, (int64_t)1 << 20);
    if (f.residual)
        hipLaunchKernelGGL((dropout_blocks<E, true>), dim3((unsigned)n), dim3(kThreads), 0, stream, f);
    else
        hipLaunchKernelGGL((dropout_blocks<E, false>), dim3((unsigned)n), dim3(kThreads), 0, stream, f);
    return (int)hipGetLastError();
}

}  // namespace

extern "C" {

int dropout_version(void) { return DROPOUT_VERSION; }

int dropout(const void* X, const void* residual, void* Y, int64_t rows, int64_t cols, int64_t ldx, int64_t ldr, int64_t ldy,
            int32_t type, double p, uint64_t seed, uint64_t offset, const uint64_t* state, hipStream_t stream)
{
    using namespace abi;
    if (type < DROPOUT_F16 || type > DROPOUT_F32 || !(p >= 0 && p <= 1)) return hipErrorInvalidValue;
    if (!good_span(rows, cols, ldx) || !good_span(rows, cols, ldy) || (residual && !good_span(rows, cols, ldr)))
        return hipErrorInvalidValue;
    if (rows == 0 || cols == 0) return hipSuccess;
    const int64_t es = type == DROPOUT_F32 ? 4 : 2;
    if (!good_pointer(X, rows, cols, es) || !good_pointer(Y, rows, cols, es) || (uintptr_t)residual % es || (uintptr_t)state % 8)
        return hipErrorInvalidValue;
    const bool one = rows == 1;  // whose pitch says nothing
    const Range y(Y, rows, cols, ldy, es), x(X, rows, cols, ldx, es), s(state, 1, state ? 2 : 0, 0, 8);
    const Range r(residual, residual ? rows : 0, cols, ldr, es);
    if ((y.meets(x) && !(X == Y && (one || ldx == ldy))) || (y.meets(r) && !(residual == Y && (one || ldr == ldy))) || y.meets(s))
        return hipErrorInvalidValue;
    const uint32_t drop = (uint32_t)floor(p * 65536 + 0.5);
    const float scale = drop < 65536 ? 65536.0f / (float)(65536 - drop) : 0.0f;
    const bool dense = one || (ldx == cols && ldy == cols && (!residual || ldr == cols));
#define DROPOUT(E)                                                                                                          \
    launch<E>({(const E*)X, (const E*)residual, (E*)Y, state, seed, offset, dense ? rows * cols : cols, ldx, ldr, ldy, rows * cols, \
               drop, scale},                                                                                                \
              stream)
    return type == DROPOUT_F16 ? DROPOUT(_Float16) : type == DROPOUT_BF16 ? DROPOUT(__bf16) : DROPOUT(float);
#undef DROPOUT
}

}  // extern "C"
