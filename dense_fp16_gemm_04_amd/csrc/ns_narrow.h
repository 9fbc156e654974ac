// The iteration for matrices X [m, n] of at most 64 rows, one launch to a step.
//
// In three launches a step of such a matrix is all latency: about 4.5 us each,
// whatever they compute.  Here a workgroup has `cw` chunks of 64 columns of X
// and adds up its share of S = X X^T; the next step's workgroups each sum all
// shares (in a fixed order), compute P from S, which for 64 rows is little
// work to repeat, and P times their own columns, from which the next share
// follows.  X is kept as X^T [n, 64] only, in place: no other workgroup
// touches those columns.  Shares are 32-bit, 16 KiB to a workgroup, and
// alternate between two buffers.
//
// A wave has 16 rows of S and P and, of a chunk, 16 columns of X.  Shares lie
// in memory in the order of a wave's lanes.  Rows m .. 63 are zero throughout
// (P's are not, but meet rows of zeros).
//
// Five steps of 64 x 64, 256, 1024, 4096 and 8192, one matrix: 34, 34, 41, 60
// and 82 us, as three launches a step 64, 66, 74, 126 and 105; of 32 x 64: 32
// and 58.  Longer ones, 64 x 16384, 65536, 262144 and 1048576: 100, 183, 422 and
// 962, and 117, 228, 646 and 4116; sixteen of 64 x 16384 193 and 293, 64 of 64 x
// 65536 2847 and 3901.  With 128 rows the same scheme took 64 us for 256 columns
// and 87 for 1024, the three launches 65 and 78: repeating P costs what the launches did.
#ifndef DENSE_FP16_GEMM_NS_NARROW_H
#define DENSE_FP16_GEMM_NS_NARROW_H

#include <algorithm>
#include <cmath>

#include "nt_core.h"

namespace narrow {

using namespace cdna4;

typedef _Float16 half;
using half4 = Elem<half>::x4;
using half8 = Elem<half>::x8;

struct Args {
    half* xt;
    const float* from;  // shares of S
    float* to;
    __bf16* out;
    int m, n, shares, chunks, cw, tall, vec;  // tall: out (and G) are X^T
    int64_t ldo, stride_o;
    // S = alpha * sum; P = a + b S + c S S; X' (or out) = next * P X, with X, S
    // and P times their powers of two
    float alpha, a, b, c, next;
};

constexpr int kRows = 64, kThreads = kRows * 4, kBlocks = kRows / 16, kFragments = kRows / 32;
constexpr int kPitch = kRows + 8;           // of LDS rows: 16 rows' 16 bytes fall on 64 banks
constexpr int64_t kShare = kRows * kRows;   // floats
typedef half Image[kRows * kPitch];

// acc[j] += rows 16 wave .. of x times rows 16 j .. of x, sums over 64 columns.
__device__ __forceinline__ void gram(f32x4 (&acc)[kBlocks], const half* x, int lane, int wave)
{
    const half* at = x + (lane & 15) * kPitch + 8 * (lane >> 4);
#pragma unroll
    for (int k = 0; k < kFragments; ++k) {
        const half8 fa = *(const half8*)(at + wave * 16 * kPitch + k * 32);
#pragma unroll
        for (int j = 0; j < kBlocks; ++j)
            acc[j] = Elem<half>::mfma(*(const half8*)(at + j * 16 * kPitch + k * 32), fa, acc[j]);
    }
}

__device__ __forceinline__ void store_share(const f32x4 (&acc)[kBlocks], float* to, int lane, int wave)
{
    float* at = to + blockIdx.x * kShare + wave * (16 * kRows) + lane * 4;
#pragma unroll
    for (int j = 0; j < kBlocks; ++j) *(f32x4*)(at + j * 256) = acc[j];
}

// An entry of G to one of X: times scale / (norm + eps), the norm from four
// partial sums of squares.  As a power of two and a rest: in 32 bits the
// factor alone would overflow for norms below 2^-112 and lose bits above 2^140.
struct Factor {
    float rest;
    int bits = 0;
    __device__ __forceinline__ Factor(const double* part, double eps, double scale)
    {
        const double norm = sqrt(part[0] + part[1] + part[2] + part[3]) + eps;
        double f = scale / norm;
        // (an eps of next to nothing and the zero matrix: zeros)
        if (norm > 0 && f > 0x1p1000) f = 0x1p1000;
        if (f > 0 && f <= 0x1p1000) {
            bits = ilogb(f);
            f = ldexp(f, -bits);
        }
        rest = (float)f;
    }
    __device__ __forceinline__ half operator()(float g) const { return (half)(ldexpf(g, bits) * rest); }
};

// X^T and the shares of S from G: `partial` holds the sums of its squares.
template <class E>
__global__ void __launch_bounds__(kThreads)
ns_narrow_begin(const Args a, const E* __restrict__ G, int64_t ldg, int64_t stride_g,
                const double* __restrict__ partial, double eps, double scale)
{
    __shared__ __attribute__((aligned(16))) Image x;
    __shared__ double part[4];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid / 64);
    const int b = blockIdx.x / a.shares, share = blockIdx.x % a.shares;
    static_assert(kThreads == 256, "one partial sum per thread");
    double s = partial[b * 256 + tid];
    for (int d = 32; d > 0; d >>= 1) s += __shfl_xor(s, d);
    if (lane == 0) part[wave] = s;
    __syncthreads();
    const Factor f(part, eps, scale);
    const E* g = G + b * stride_g;
    half* xt = a.xt + (int64_t)b * a.chunks * kRows * kRows;
    f32x4 acc[kBlocks] = {};
    const int last = min((share + 1) * a.cw, a.chunks);
    for (int chunk = share * a.cw; chunk < last; ++chunk) {
        const int n0 = chunk * kRows;
        E v[kRows / 4];
#pragma unroll
        for (int i = 0; i < kRows / 4; ++i) {
            const int at = i * kThreads + tid, slow = at / kRows, fast = at % kRows;
            const int row = a.tall ? n0 + slow : slow, col = a.tall ? fast : n0 + fast;  // of G
            v[i] = (E)0.0f;
            if (row < (a.tall ? a.n : a.m) && col < (a.tall ? a.m : a.n)) v[i] = g[row * ldg + col];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kRows / 4; ++i) {
            const int at = i * kThreads + tid, slow = at / kRows, fast = at % kRows;
            x[a.tall ? fast * kPitch + slow : slow * kPitch + fast] = f((float)v[i]);
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kBlocks; ++i) {
            const int at = i * kThreads + tid, n = at / (kRows / 4), m = at % (kRows / 4) * 4;
            half4 w;
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = x[(m + e) * kPitch + n];
            *(half4*)(xt + (int64_t)(n0 + n) * kRows + m) = w;
        }
        gram(acc, x, lane, wave);
    }
    store_share(acc, a.to, lane, wave);
}

// One step.  LAST: the result instead of X^T and the next shares.
template <bool LAST>
__global__ void __launch_bounds__(kThreads) ns_narrow_step(const Args a)
{
    __shared__ __attribute__((aligned(16))) Image s, p, x;
    __shared__ __attribute__((aligned(16))) float ratio[kRows];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid / 64);
    const int r = lane & 15, h = lane >> 4;
    const int b = blockIdx.x / a.shares, share = blockIdx.x % a.shares;
    half* xt = a.xt + (int64_t)b * a.chunks * kRows * kRows + (wave * 16 + r) * kRows;  // the lane's column of X, of chunk 0
    const int last = min((share + 1) * a.cw, a.chunks);
    half8 fx[kFragments];
    auto fetch = [&](int chunk) __attribute__((always_inline)) {
#pragma unroll
        for (int k = 0; k < kFragments; ++k) fx[k] = *(const half8*)(xt + (int64_t)chunk * kRows * kRows + k * 32 + 8 * h);
    };
    fetch(share * a.cw);

    // S, rows 16 wave .. of it: the lane has row r, columns 16 j + 4 h ..
    f32x4 sum[kBlocks] = {};
    const float* from = a.from + (int64_t)b * a.shares * kShare + wave * (16 * kRows) + lane * 4;
#pragma unroll 8
    for (int i = 0; i < a.shares; ++i)
#pragma unroll
        for (int j = 0; j < kBlocks; ++j) sum[j] += *(const f32x4*)(from + i * kShare + j * 256);
    const int mine = (wave * 16 + r) * kPitch + 4 * h;
    half4 s16[kBlocks];
#pragma unroll
    for (int j = 0; j < kBlocks; ++j) *(half4*)(s + mine + j * 16) = s16[j] = round4<half>(sum[j] * a.alpha);
    __syncthreads();

    // P, and what rounding takes from its diagonal (left where that is
    // subnormal, and the quotient perhaps far from 1)
    f32x4 ss[kBlocks] = {};
    gram(ss, s, lane, wave);
#pragma unroll
    for (int j = 0; j < kBlocks; ++j) {
        f32x4 v = ss[j] * a.c;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[e] = __builtin_fmaf(a.b, (float)s16[j][e], v[e]);
            if (j == wave && r == 4 * h + e) {
                const float d = v[e] + a.a, d16 = (float)(half)d;
                v[e] = d;
                ratio[wave * 16 + r] = __builtin_fabsf(d16) >= 0x1p-14f ? d * __builtin_amdgcn_rcpf(d16) : 1.0f;
            }
        }
        *(half4*)(p + mine + j * 16) = round4<half>(v);
    }
    __syncthreads();

    f32x4 acc[kBlocks] = {};
    for (int chunk = share * a.cw; chunk < last; ++chunk) {
        // the lane has column 16 wave + r of the chunk, rows 16 j + 4 h ..
        f32x4 y[kBlocks] = {};
#pragma unroll
        for (int k = 0; k < kFragments; ++k)
#pragma unroll
            for (int j = 0; j < kBlocks; ++j)
                y[j] = Elem<half>::mfma(*(const half8*)(p + (j * 16 + r) * kPitch + k * 32 + 8 * h), fx[k], y[j]);
        if (chunk + 1 < last) fetch(chunk + 1);
        const int turned = (4 * h + (lane & 3)) * kPitch + wave * 16 + (lane & 12);
#pragma unroll
        for (int j = 0; j < kBlocks; ++j) {
            const f32x4 v = y[j] * (*(const f32x4*)(ratio + j * 16 + 4 * h) * a.next);
            if constexpr (LAST) {
                const Elem<__bf16>::x4 w = round4<__bf16>(v);
                typedef Elem<__bf16>::x4 out4;
                if (a.tall)
                    *(out4*)(x + mine + j * 16) = w;  // rows of X^T
                else
                    *(out4*)(x + turned + j * 16 * kPitch) = nt::quad_transposed(w, lane);
            } else {
                const half4 w = round4<half>(v);
                *(half4*)(xt + (int64_t)chunk * kRows * kRows + j * 16 + 4 * h) = w;
                *(half4*)(x + turned + j * 16 * kPitch) = nt::quad_transposed(w, lane);
            }
        }
        __syncthreads();
        if constexpr (LAST) {
            typedef Elem<__bf16>::x4 out4;
            __bf16* out = a.out + b * a.stride_o;
#pragma unroll
            for (int i = 0; i < kBlocks; ++i) {
                const int at = i * kThreads + tid, rx = at / (kRows / 4), cx = at % (kRows / 4) * 4;
                const int row = a.tall ? chunk * kRows + rx : rx, col = a.tall ? cx : chunk * kRows + cx;
                const int rows = a.tall ? a.n : a.m, cols = a.tall ? a.m : a.n;
                if (row >= rows) continue;
                const out4 w = *(const out4*)(x + rx * kPitch + cx);
                __bf16* to = out + row * a.ldo + col;
                if (a.vec && col + 3 < cols) {
                    *(out4*)to = w;
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (col + e < cols) to[e] = w[e];
                }
            }
        } else {
            gram(acc, x, lane, wave);
        }
        __syncthreads();
    }
    if constexpr (!LAST) store_share(acc, a.to, lane, wave);
}

// The layout of the work, by the sizes of one matrix.
struct Plan {
    bool used = false;  // or the tiled products, which are faster for more rows
    int64_t shares = 0, chunks = 0, cw = 1;
    Plan(int64_t m, int64_t n)
    {
        if (m > kRows) return;
        used = true;
        chunks = (n + kRows - 1) / kRows;
        // a step reads all shares and walks cw chunks, each of which takes
        // about four times as long as a share
        cw = std::max<int64_t>(1, (int64_t)std::lround(0.5 * std::sqrt((double)chunks)));
        shares = (chunks + cw - 1) / cw;
    }
};

}  // namespace narrow

#endif
