// Copies that bring an operand into the form the tiled products read: rows
// on 16 bytes or more, padded with zeros to a multiple of eight elements, as they are
// or transposed.
#ifndef DENSE_FP16_GEMM_RELAYOUT_H
#define DENSE_FP16_GEMM_RELAYOUT_H

#include "cdna4.h"

namespace relayout {

using namespace cdna4;

constexpr int kTile = 64;       // a workgroup moves a 64 x 64 tile
constexpr int kThreads = 256;   // as 16 columns of four elements by 16 rows, four times
constexpr int kPitch = 68;      // LDS row pitch in elements: 8-byte aligned, 34 banks apart

template <class E>
using Four = E __attribute__((ext_vector_type(4)));

// Four elements of a row, columns c .. c + 3 of `cols` (at least one), zero
// past the end.  One by one they are loaded whether there or not, the last
// element instead: with branches around them the compiler waits for each.
template <class E>
__device__ __forceinline__ Four<E> load4(const E* row, int c, int cols, bool vec)
{
    Four<E> v;
    if (vec && c + 3 < cols) {
        v = *(const Four<E>*)(row + c);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = row[min(c + e, cols - 1)];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = c + e < cols ? v[e] : (E)0.0f;
    }
    return v;
}

// A matrix's elements by fours, workgroup `block` of `blocks` of 256 threads
// taking its share: `each(v)` of all fours of a thread's (zeros past a row's
// end), four loads in flight.
template <class E, class Each>
__device__ __forceinline__ void each_four(const E* src, int64_t lds_, int rows, int cols, bool vec, int block, int blocks,
                                          Each each)
{
    // a workgroup takes pieces of 256 groups of a row, or several short rows
    const int per = (int)(((int64_t)cols + 3) / 4), lanes = min(per, 256), step = 256 / lanes, pieces = (per + 255) / 256;
    const int lane = threadIdx.x % lanes, first = threadIdx.x / lanes;
    const int64_t units = first < step ? (int64_t)rows * pieces : 0;
    const int64_t stride = (int64_t)blocks * step;
    for (int64_t u0 = (int64_t)block * step + first; u0 < units; u0 += 4 * stride) {
        Four<E> v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t u = u0 + i * stride;
            const int64_t r = pieces == 1 ? u : u / pieces;
            const int c = ((int)(u - r * pieces) * 256 + lane) * 4;
            v[i] = Four<E>{};
            if (u < units) v[i] = load4(src + r * lds_, c, cols, vec);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) each(v[i]);
    }
}

// Writes a 64 x 64 tile that LDS holds row-major (pitch kPitch) transposed:
// dst[c][r] for tile row r and column c, whole rows of `rows` in groups of
// eight bytes (dst's pitch is a multiple of 8; rows past `rows_valid` hold
// zeros in LDS, and `rows` is a multiple of eight from it on).
template <class E>
__device__ __forceinline__ void store_transposed(const E* tile, E* dst, int64_t ldd, int r0, int c0, int rows, int cols)
{
    const int x = threadIdx.x & 15, y = threadIdx.x >> 4;
#pragma unroll
    for (int it = 0; it < 4; ++it) {
        const int c = it * 16 + y, r = x * 4;
        if (c0 + c >= cols || r0 + r >= rows) continue;
        typename Elem<E>::x4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = tile[(r + e) * kPitch + c];
        *(typename Elem<E>::x4*)(dst + (int64_t)(c0 + c) * ldd + r0 + r) = v;
    }
}

// Up to three operands of one width in one launch, one to each blockIdx.y:
// dst[r][c] = src[r][c] for c < cols, 0 for cols <= c < ldd.
template <class E>
struct Copies {
    struct Job {
        const E* src;
        E* dst;
        int64_t lds_, rows;
    } job[3];
    int jobs;
};

template <class E>
__global__ void __launch_bounds__(kThreads) copy_rows(const Copies<E> copies, int cols, int ldd)
{
    const typename Copies<E>::Job j = copies.job[blockIdx.y];
    const uint32_t per = (uint32_t)ldd / 4;
    const int64_t groups = j.rows * per;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < groups; i += (int64_t)gridDim.x * kThreads) {
        const int64_t r = groups >> 32 ? i / per : (uint32_t)i / per;
        const int c = (int)(i - r * per) * 4;
        *(typename Elem<E>::x4*)(j.dst + r * ldd + c) = load4(j.src + r * j.lds_, c, cols, false);
    }
}

// dst[c][r] = src[r][c] for r < rows, 0 for rows <= r < padded: tile number
// `id` of tiles().
template <class E>
struct Transpose {
    const E* src;
    E* dst;
    int64_t lds_, ldd;
    int rows, cols, padded, vec;

    __host__ __device__ int64_t tiles() const
    {
        return (int64_t)((padded + kTile - 1) / kTile) * ((cols + kTile - 1) / kTile);
    }
    __device__ __forceinline__ void run(int id, E* tile) const
    {
        const int tiles_c = (cols + kTile - 1) / kTile;
        const int r0 = id / tiles_c * kTile, c0 = id % tiles_c * kTile;
        const int x = threadIdx.x & 15, y = threadIdx.x >> 4;
#pragma unroll
        for (int it = 0; it < 4; ++it) {
            const int r = it * 16 + y;
            typename Elem<E>::x4 v = {};
            if (r0 + r < rows) v = load4(src + (int64_t)(r0 + r) * lds_, c0 + x * 4, cols, vec);
            *(typename Elem<E>::x4*)(tile + r * kPitch + x * 4) = v;
        }
        __syncthreads();
        store_transposed(tile, dst, ldd, r0, c0, padded, cols);
    }
};

}  // namespace relayout

#endif
