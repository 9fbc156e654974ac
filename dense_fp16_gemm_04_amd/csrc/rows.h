// What the row-wise operators share: a row in chunks of 16 bytes, whatever its
// alignment, and sums over the lanes that hold a row.
#ifndef DENSE_FP16_GEMM_ROWS_H
#define DENSE_FP16_GEMM_ROWS_H

#include <hip/hip_runtime.h>

#include <stdint.h>

#include "cus.h"

namespace rows {

constexpr int kWave = 64;

template <class T, int N>
using Vec = T __attribute__((ext_vector_type(N)));

// Elements of a type to a chunk of 16 bytes.
template <class E>
constexpr int kChunk = 16 / (int)sizeof(E);

// N elements from p on, of which `left` exist (at least one); zeros after them.
// The whole ones need no alignment but their elements' (gfx950 loads and stores
// any address; 16 bytes over a cache line's end cost two accesses).  Single
// elements are loaded whether there or not, the last one instead: with branches
// around them the compiler waits for each.  (`left` is new to the compiler
// there: it would compute the elements' addresses and comparisons before a loop
// over rows and keep them, in more registers than there are.)
template <class T, int N>
__device__ __forceinline__ Vec<T, N> load(const T* p, int left)
{
    typedef Vec<T, N> Any __attribute__((aligned(sizeof(T))));
    if (left >= N) return *(const Any*)p;
    asm volatile("" : "+v"(left));
    Vec<T, N> v;
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] = p[min(e, left - 1)];
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] = e < left ? v[e] : (T)0.0f;
    return v;
}

template <class T, int N>
__device__ __forceinline__ void store(T* p, int left, const Vec<T, N>& v)
{
    typedef Vec<T, N> Any __attribute__((aligned(sizeof(T))));
    if (left >= N) {
        *(Any*)p = v;
        return;
    }
    asm volatile("" : "+v"(left));
#pragma unroll
    for (int e = 0; e < N; ++e)
        if (e < left) p[e] = v[e];
}

// Sum over groups of G adjacent lanes (a power of two), the same bits in all of
// them: each step adds two equal halves, in either order.
template <int CTRL>
__device__ __forceinline__ float add_dpp(float v)
{
    return v + __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}
template <int G>
__device__ __forceinline__ float group_sum(float v)
{
    if constexpr (G >= 2) v = add_dpp<0xb1>(v);   // quad_perm 1, 0, 3, 2
    if constexpr (G >= 4) v = add_dpp<0x4e>(v);   // quad_perm 2, 3, 0, 1
    if constexpr (G >= 8) v = add_dpp<0x141>(v);  // row_half_mirror
    if constexpr (G >= 16) v = add_dpp<0x140>(v);  // row_mirror
    if constexpr (G >= 32) v += __shfl_xor(v, 16);
    if constexpr (G >= 64) v += __shfl_xor(v, 32);
    return v;
}

// LDS of `sums`: two sets of what each wave adds.
template <int G, int K>
struct Parts {
    float at[2][G > kWave ? K * (G / kWave) : 1];
};

// K sums over groups of G adjacent lanes: parts of a wave, or (G above 64) the
// whole workgroup, whose waves meet once.  `turn` alternates from call to call:
// who writes a set again has met the others since they read it.
template <int G, int K>
__device__ __forceinline__ void sums(float (&v)[K], Parts<G, K>& parts, int turn)
{
    constexpr int W = G / kWave;
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = group_sum<G < kWave ? G : kWave>(v[k]);
    if constexpr (W > 1) {
        float* p = parts.at[turn & 1];
        if (threadIdx.x % kWave == 0)
#pragma unroll
            for (int k = 0; k < K; ++k) p[k * W + threadIdx.x / kWave] = v[k];
        __syncthreads();
#pragma unroll
        for (int k = 0; k < K; ++k) {
            v[k] = 0.0f;
#pragma unroll
            for (int w = 0; w < W; ++w) v[k] += p[k * W + w];
        }
    }
}

// Sums of columns over `parts` rows `step` apart, C columns to a workgroup of 1024
// threads, which take every (1024 / C)th row each and meet in LDS.  `at`: the
// thread's column in the first row; null: it has none.  The first C threads get
// their columns' sums.
constexpr int kSumThreads = 1024;
template <int C>
__device__ __forceinline__ float columns_sum(const float* at, int64_t step, int parts)
{
    constexpr int S = kSumThreads / C;
    __shared__ float meet[S][C];
    const int c = threadIdx.x % C, share = threadIdx.x / C;
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (at) {
        int p = share;
        for (; p + 3 * S < parts; p += 4 * S)
#pragma unroll
            for (int k = 0; k < 4; ++k) s[k] += at[(p + k * S) * step];
#pragma unroll
        for (int k = 0; k < 3; ++k)
            if (p + k * S < parts) s[k] += at[(p + k * S) * step];
    }
    meet[share][c] = (s[0] + s[1]) + (s[2] + s[3]);
#pragma unroll
    for (int half = S / 2; half > 0; half /= 2) {
        __syncthreads();
        if (share < half) meet[share][c] += meet[share + half][c];
    }
    return meet[0][c];
}
// 64 columns are whole cache lines, 16 four times the workgroups: where 64 are too
// few for half the chip.  (1 row of 1024 columns from 1000 parts: 7.4 us by 64 and
// 4.6 by 16; 8 of 2048 from 500 11.7 and 12.9.)
inline bool wide_sums(int64_t columns, int64_t rows) { return (columns + 63) / 64 * rows >= cus::kCus / 2; }

// Bytes [first, last] of a matrix stay far from where 64 bits end.
inline bool good_span(int64_t rows, int64_t cols, int64_t ld)
{
    constexpr int64_t most = ((int64_t)1 << 31) - 1;
    return rows >= 0 && cols >= 0 && rows <= most && cols <= most && ld >= cols && ld <= most &&
           (rows == 0 || (rows - 1) * ld + cols < ((int64_t)1 << 58));
}

}  // namespace rows

#endif
