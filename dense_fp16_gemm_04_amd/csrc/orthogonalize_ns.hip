// Newton-Schulz orthogonalisation for gfx950: include/orthogonalize_ns.h.
//
// m <= n are the matrix's sides.  Per step, in NT form throughout,
//   S  = X X^T              [m, m] from X  [m, n]
//   P  = a I + b S + c S S  [m, m], S S = S S^T
//   X' = P X                [m, n] = P (X^T)^T from X^T [n, m]
// so both X and X^T are kept, and the product that makes X' writes both.  S
// and P are symmetric: only tiles on and below the diagonal are computed,
// and the others are written as their transposes.
//
// Rounding.  a is part of P: P's diagonal is then near 1 once the singular
// values are, where that of bS + cSS is near -2.7.  The diagonal is still by
// far P's largest part, so its rounding is taken back: row r of X' is
// multiplied by d / binary16(d) of P's diagonal entry d, which makes that
// entry exact and the others, small ones, off by as much.  (Relative error of
// the bfloat16 result, 54 x 1286: 2.60e-3 without, 1.94e-3 with, 1.90e-3 with
// an exact P; 40 x 4000: 3.13e-3, 2.27e-3, 2.28e-3.)
//
// Range.  X, S and P are each held times a power of two that brings the largest
// entry they can have near 2^14 (Ranges), so that small ones, of rows and
// columns far below the others, keep their bits: of 256 x 1024 of noise with a
// row 10^-5 of the others that row is 1.9e-3 off, one of 10^-7 6e-3.  (With X
// near sqrt(n) times its typical entry and S and P as they are 2.8e-2, and 1:
// it came out as zero.)
//
// Matrices of at most 64 rows take one launch a step: ns_narrow.h.
//
// 4096 x 4096, five steps: 1375 us, 1000 TFLOP/s of what symmetry leaves (1255 on
// the fastest of four MI355X): a step is S 71 + 7.5 us, P 73 + 8 (tiles, and
// joining the last wave's split sums), X' 108 and the last one 103; sums of
// squares and X 41.  256 x 256: 70 us, seventeen launches of 3 to 5.
#include "orthogonalize_ns.h"

#include <algorithm>
#include <cmath>

#include "abi.h"
#include "ns_narrow.h"
#include "nt_launch.h"
#include "relayout.h"

namespace {

using namespace nt;

typedef _Float16 half;
using half4 = Elem<half>::x4;

constexpr int kNormBlocks = 256;  // partial sums of squares per matrix

// Partial sums of squares, in 64 bits (a 32-bit sum would overflow for
// entries past 2^63 and lose small ones beside large ones).
template <class E>
__global__ void __launch_bounds__(256) ns_squares(const E* __restrict__ G, int64_t ldg, int64_t stride, int rows,
                                                  int cols, int vec, double* __restrict__ partial)
{
    const int b = blockIdx.x / kNormBlocks, k = blockIdx.x % kNormBlocks;
    double s = 0;
    relayout::each_four(G + b * stride, ldg, rows, cols, vec, k, kNormBlocks, [&](const relayout::Four<E>& v) {
#pragma unroll
        for (int e = 0; e < 4; ++e) s += (double)(float)v[e] * (double)(float)v[e];
    });
    __shared__ double part[256];
    part[threadIdx.x] = s;
    __syncthreads();
    for (int d = 128; d > 0; d >>= 1) {
        if (threadIdx.x < d) part[threadIdx.x] += part[threadIdx.x + d];
        __syncthreads();
    }
    if (threadIdx.x == 0) partial[blockIdx.x] = part[0];
}

// D1 [rows, p1] = G * scale / (norm + eps) (narrow::Factor) and D2 [cols, p2]
// its transpose, both padded with zeros to their pitches.
template <class E>
__global__ void __launch_bounds__(relayout::kThreads)
ns_start(const E* __restrict__ G, int64_t ldg, int64_t stride_g, int rows, int cols, const double* __restrict__ partial,
         double eps, double scale, half* __restrict__ D1, half* __restrict__ D2, int64_t stride_x, int p1, int p2,
         int tiles_r, int tiles_c, int vec)
{
    using namespace relayout;
    __shared__ half tile[kTile * kPitch];
    const int per = tiles_r * tiles_c, b = blockIdx.x / per, id = blockIdx.x % per;
    const int r0 = id / tiles_c * kTile, c0 = id % tiles_c * kTile;
    __shared__ double part[4];
    {
        static_assert(kNormBlocks == kThreads, "one partial sum per thread");
        double s = partial[b * kNormBlocks + threadIdx.x];
        for (int d = 32; d > 0; d >>= 1) s += __shfl_xor(s, d);
        if (threadIdx.x % 64 == 0) part[threadIdx.x / 64] = s;
    }
    __syncthreads();
    const narrow::Factor f(part, eps, scale);
    const E* g = G + b * stride_g;
    half* d1 = D1 + b * stride_x;
    const int x = threadIdx.x & 15, y = threadIdx.x >> 4;
#pragma unroll
    for (int it = 0; it < 4; ++it) {
        const int r = it * 16 + y, c = c0 + x * 4;
        half4 v = {};
        if (r0 + r < rows) {
            const Four<E> w = load4(g + (r0 + r) * ldg, c, cols, vec);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = f((float)w[e]);
            if (c < p1) *(half4*)(d1 + (int64_t)(r0 + r) * p1 + c) = v;
        }
        *(half4*)(tile + r * kPitch + x * 4) = v;
    }
    __syncthreads();
    store_transposed(tile, D2 + b * stride_x, p2, r0, c0, p2, cols);
}

// steps == 0: the normalised matrix itself.
__global__ void __launch_bounds__(256) ns_copy_out(const half* __restrict__ X, int64_t ldx, int64_t stride_x,
                                                   __bf16* __restrict__ out, int64_t ldo, int64_t stride_o, int rows,
                                                   int cols, int64_t total, float scale)
{
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t row = i / cols, c = i - row * cols, b = row / rows, r = row - b * rows;
        out[b * stride_o + r * ldo + c] = (__bf16)((float)X[b * stride_x + r * ldx + c] * scale);
    }
}

// How a tile is written: as it is, transposed, or both; in 16-byte pieces or
// element by element.
enum { kAsIs = 1, kTurned = 2, kEights = 4 };

// S (POLY false: alpha A A^T) or P (POLY true: alpha A A^T + beta A + gamma I,
// A symmetric), each times its power of two, [m, mp] with pitch ldc, tiles on
// and below the diagonal and their transposes.
template <bool POLY>
struct SymmetricOp {
    static constexpr bool kPersist = !POLY, kSplit = true;  // (P's epilogue would spill there)
    const half* A;
    half* C;
    float* diag;  // (POLY) C's diagonal before it is rounded
    int M, K, lda, ldc, mp, tiles, per;  // per: tiles of one matrix
    int64_t stride_a, stride_c;
    float alpha, beta, gamma;

    template <int BM, int BN>
    __device__ __forceinline__ void tile(int id, Tile& t) const
    {
        id = xcd_order(id, tiles);
        t.batch = id / per;
        int tm, tn;
        triangle_tile(id - t.batch * per, (M + BM - 1) / BM, BM / BN, tm, tn);
        t.m0 = tm * BM;
        t.n0 = tn * BN;
        // what a tile that reaches the diagonal mirrors is written by itself
        // or its neighbour
        t.mirror = t.n0 < t.m0;
    }
    __device__ __forceinline__ bool outside(const Tile& t) const { return t.m0 >= M || t.n0 >= M; }
    __device__ __forceinline__ const half* a_rows(const Tile& t, int row, int& n) const
    {
        return rows_from(A + t.batch * stride_a, t.m0 + row, M, lda, n);
    }
    template <int WTN>
    __device__ __forceinline__ const half* b_rows(const Tile& t, int row, int& n) const
    {
        return rows_from(A + t.batch * stride_a, t.n0 + row, M, lda, n);
    }
    template <int WTN>
    __device__ __forceinline__ int b_pitch(int) const
    {
        return lda;
    }
    template <class T>
    __device__ __forceinline__ void epilogue(const Tile& t, const f32x4 (&acc)[T::FM][T::FN], int lane, int wave,
                                             unsigned char* s0, unsigned char* s1) const
    {
        half* c = C + t.batch * stride_c;
        half4 v[T::FM][T::FN];
        const Rows direct = rows_at(c, t.m0, M, T::BM, ldc, t.n0, mp);
        if constexpr (POLY) {
            // the tile of A through LDS to the values that use it, which
            // take its place there
            static_assert(T::BM * T::BN * 2 <= T::STAGE_MAX, "the tile fits");
            const Rows old = rows_at(A + t.batch * stride_a, t.m0, M, T::BM, lda, t.n0, mp);
            const Image<T::BN> image{s0, s1};
            const int wm = wave / T::WAVES_N, wn = wave % T::WAVES_N;
            const float gamma_here = t.m0 + wm * T::WTM == t.n0 + wn * T::WTN ? gamma : 0.0f;
            f32x4 diagonal;  // of a block: row l % 16 is column 4 (l / 16) + e
#pragma unroll
            for (int e = 0; e < 4; ++e) diagonal[e] = (lane & 15) == 4 * (lane >> 4) + e ? 1.0f : 0.0f;
            auto on_diagonal = [&](int i, int j) { return t.m0 + wm * T::WTM + i * 16 == t.n0 + wn * T::WTN + j * 16; };
            float mine[T::FM];  // the lane's entry of each block row on the diagonal, if it has one
#pragma unroll
            for (int i = 0; i < T::FM; ++i) mine[i] = 0.0f;
            auto same = [](int x) { return x; };
            fill<T, T::BN, T::BM>(image, old, same, lane, wave);
            lds_barrier<0>();
            const int at_row = wm * T::WTM + (lane & 15), at_col = wn * T::WTN + 4 * (lane >> 4);
#pragma unroll
            for (int i = 0; i < T::FM; ++i)
#pragma unroll
                for (int j = 0; j < T::FN; ++j) {
                    half4* at = image.template at<half4>(at_row + i * 16, at_col + j * 16);
                    const half4 a4 = *at;
                    f32x4 w = acc[i][j] * alpha;
                    // (where a wave's part is square, only its blocks (i, i)
                    // can lie on the diagonal)
                    constexpr bool SQUARE = T::WTM == T::WTN;
                    const float on = SQUARE ? gamma_here : on_diagonal(i, j) ? gamma : 0.0f;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        w[e] = __builtin_fmaf(beta, (float)a4[e], w[e]);
                        if (!SQUARE || i == j) w[e] = __builtin_fmaf(diagonal[e], on, w[e]);
                    }
                    const half4 w16 = round4<half>(w);
                    *at = v[i][j] = w16;
                    if (!SQUARE || i == j) {
                        float d = diagonal[0] * w[0];
#pragma unroll
                        for (int e = 1; e < 4; ++e) d = __builtin_fmaf(diagonal[e], w[e], d);
                        mine[i] = SQUARE || on_diagonal(i, j) ? d : mine[i];
                    }
                }
            lds_barrier<63>();
            drain<T, T::BN, T::BM, true>(image, direct, same, lane, wave);
            lds_barrier<63>();
            // (the waves whose rows have no entry in the tile store nothing)
            const __amdgpu_buffer_rsrc_t entries =
                make_rsrc(diag + (int64_t)t.batch * mp + t.m0, (uint32_t)min(T::BM, M - t.m0) * 4u);
#pragma unroll
            for (int i = 0; i < T::FM; ++i) {
                const int m = wm * T::WTM + i * 16, n = t.m0 + m - t.n0 - wn * T::WTN;  // the entry's column in the wave's
                const uint32_t at =
                    (lane & 15) >> 2 == lane >> 4 && n >= 0 && n < T::WTN ? (uint32_t)(m + (lane & 15)) * 4u : kOob;
                __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, mine[i]), entries, at, 0, 0);
            }
        } else {
            write_rows<T, T::FN, true>([&](int i, int j) { return v[i][j] = round4<half>(acc[i][j] * alpha); }, direct,
                                       lane, wave, s0, s1);
        }
        // Rows M .. mp - 1 of the accumulator are zero: the transpose's
        // padding.
        Rows turned = rows_at(c, t.n0, M, T::BN, ldc, t.m0, mp);
        if (!(T::WAVES == 1 ? t.mirror : t.n0 < t.m0)) turned.rs = make_rsrc(c, 0);  // (a whole tile's, of a sub-tile)
        write_turned<T, true>([&](int i, int j) { return v[i][j]; }, turned, lane, wave, s0, s1);
    }
};

// X' = P X [m, n] and its transpose [n, m] in binary16, or (LAST) the result
// in bfloat16, in out's layout, each times alpha: out's rows are X's (HOW has
// kAsIs) or X^T's (kTurned).
template <bool LAST, int HOW>
struct ApplyOp {
    // (element by element, the 256 x 256 kernel would spill scalar registers)
    static constexpr bool kPersist = (HOW & kEights) != 0, kSplit = true;
    const half *P, *Xt;
    const float* diag;  // P's diagonal before it was rounded
    half *X, *XtNew;
    __bf16* out;
    int M, N, K, lda, ldb, ldx, np, tiles, tiles_m, tiles_n, ldo;  // ldb, ldx: of X^T and X
    int64_t stride_p, stride_x, stride_o;
    float alpha;

    template <int BM, int BN>
    __device__ __forceinline__ void tile(int id, Tile& t) const
    {
        const int per = tiles_m * tiles_n;
        id = xcd_order(id, tiles);  // (whole matrices of a batch to an XCD)
        t.batch = id / per;
        int tm, tn;
        grid_tile(id - t.batch * per, tiles_m, tiles_n, tm, tn);
        t.m0 = tm * BM;
        t.n0 = tn * BN;
    }
    __device__ __forceinline__ bool outside(const Tile& t) const { return t.m0 >= M || t.n0 >= N; }
    __device__ __forceinline__ const half* a_rows(const Tile& t, int row, int& n) const
    {
        return rows_from(P + t.batch * stride_p, t.m0 + row, M, lda, n);
    }
    template <int WTN>
    __device__ __forceinline__ const half* b_rows(const Tile& t, int row, int& n) const
    {
        return rows_from(Xt + t.batch * stride_x, t.n0 + row, N, ldb, n);
    }
    template <int WTN>
    __device__ __forceinline__ int b_pitch(int) const
    {
        return ldb;
    }
    template <class T>
    __device__ __forceinline__ void epilogue(const Tile& t, const f32x4 (&acc)[T::FM][T::FN], int lane, int wave,
                                             unsigned char* s0, unsigned char* s1) const
    {
        constexpr bool EIGHTS = (HOW & kEights) != 0;
        // Each row's factor: what rounding took from its diagonal entry.  (A
        // subnormal one is left as it is, its quotient may be far from 1.)
        const __amdgpu_buffer_rsrc_t entries =
            make_rsrc(diag + (int64_t)t.batch * K + t.m0, (uint32_t)min(T::BM, M - t.m0) * 4u);
        float f[T::FM];
#pragma unroll
        for (int i = 0; i < T::FM; ++i) {
            const uint32_t at = (uint32_t)(wave / T::WAVES_N * T::WTM + i * 16 + (pinned(lane) & 15)) * 4u;
            f[i] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(entries, at, 0, 0));
        }
#pragma unroll
        for (int i = 0; i < T::FM; ++i) {
            const float d16 = (float)(half)f[i];
            f[i] = __builtin_fabsf(d16) >= 0x1p-14f ? f[i] * __builtin_amdgcn_rcpf(d16) : 1.0f;
            f[i] *= alpha;
        }
        if constexpr (LAST) {
            __bf16* o = out + t.batch * stride_o;
            auto value = [&](int i, int j) { return round4<__bf16>(acc[i][j] * f[i]); };
            if constexpr (HOW & kAsIs)
                write_rows<T, T::FN, EIGHTS>(value, rows_at(o, t.m0, M, T::BM, ldo, t.n0, N), lane, wave, s0, s1);
            if constexpr (HOW & kTurned)
                write_turned<T, EIGHTS>(value, rows_at(o, t.n0, N, T::BN, ldo, t.m0, M), lane, wave, s0, s1);
        } else {
            // (columns N .. np - 1 and rows M .. K - 1 of the accumulator
            // are zero: the padding of both)
            auto value = [&](int i, int j) { return round4<half>(acc[i][j] * f[i]); };
            write_rows<T, T::FN, true>(value, rows_at(X + t.batch * stride_x, t.m0, M, T::BM, ldx, t.n0, np), lane, wave,
                                       s0, s1);
            write_turned<T, true>(value, rows_at(XtNew + t.batch * stride_x, t.n0, N, T::BN, ldb, t.m0, K), lane, wave,
                                  s0, s1);
        }
    }
};

// ------------------------------------------------------------------ host --

// Rows start on 128 bytes: the tiles that read and write them then do so by
// whole cache lines (1000 x 4001: 217 us, and 254 with 16 bytes).
constexpr int64_t kLine = 64;

struct Space {
    double* partial;
    half *x[2], *xt[2], *s, *p;
    float *diag, *sums;  // P's diagonal; of split tiles
    int64_t m, n, mp, np, lm, ln, stride_x, stride_s, bytes;
    Space(void* base, int64_t batch, int64_t rows, int64_t cols)
    {
        m = std::min(rows, cols);
        n = std::max(rows, cols);
        mp = abi::up(m, 8);
        np = abi::up(n, 8);
        lm = abi::up(m, kLine);
        ln = abi::up(n, kLine);
        stride_x = std::max(mp * ln, np * lm);
        stride_s = mp * lm;
        abi::Carve c(base);
        partial = c.take<double>(batch * kNormBlocks);
        for (int i = 0; i < 2; ++i) {
            x[i] = c.take<half>(batch * stride_x);
            xt[i] = c.take<half>(batch * stride_x);
        }
        s = c.take<half>(batch * stride_s);
        p = c.take<half>(batch * stride_s);
        diag = c.take<float>(batch * mp);
        sums = n >= kSplitK ? c.take<float>(kSplitFloats) : nullptr;
        bytes = c.used();
    }
};

struct NarrowSpace {
    double* partial;
    half* xt;
    float* shares[2];
    int64_t bytes;
    NarrowSpace(void* base, int64_t batch, const narrow::Plan& p)
    {
        abi::Carve c(base);
        partial = c.take<double>(batch * kNormBlocks);
        xt = c.take<half>(batch * p.chunks * narrow::kShare);
        for (float*& s : shares) s = c.take<float>(batch * p.shares * narrow::kShare);
        bytes = c.used();
    }
};

int64_t triangle(int64_t t) { return t * (t + 1) / 2; }

template <class OP>
int launch_symmetric(const OP& op, int64_t m, int64_t batch, float* partial, hipStream_t stream)
{
    auto per = [=](const Kind& k) { return k.bm / k.bn * triangle((m + k.bm - 1) / k.bm); };
    return launch<half>(
        op, op.K, partial, [=](const Kind& k) { return per(k) * batch; },
        [=](OP& o, const Kind& k) { o.per = (int)per(k); }, stream);
}

// The powers of two of a step.  Singular values lie in 0 .. sigma, which is 1
// at the start, |G|_F being at least the largest; no entry of X exceeds sigma,
// none of S its square, none of P the polynomial's largest value there.  Each
// is held times the 2^k that brings its bound to 2^14 at most and above 2^13:
// binary16 ends at 2^16, so rounding has room, and below at 2^-24.  Of a
// polynomial that could blow up values near 1 but is given smaller ones the
// bounds say nothing: S and P are then held as they are, and X, whose typical
// entry is 1 / sqrt(n) when it is orthonormal, times sqrt(n).
struct Ranges {
    double sigma = 1.0;
    int least, x, s = 0, p = 0;
    explicit Ranges(int64_t n) : least(std::min(12, (int)std::lround(0.5 * std::log2((double)n)))) { x = bits(sigma, least); }
    static int bits(double bound, int least)
    {
        int e = 0;
        const double m = std::frexp(std::max(bound, 1e-300), &e);
        return std::min(60, std::max(least, 14 - (m == 0.5 ? e - 1 : e)));
    }
    // S and P of the step (a, b, c); leaves sigma and x for the next one
    void step(double a, double b, double c)
    {
        const double u1 = sigma * sigma;
        auto p_at = [=](double u) { return std::fabs(a + u * (b + u * c)); };
        auto x_at = [=](double u) { return std::sqrt(u) * p_at(u); };
        // the ends, and where the derivatives in u = sigma^2 are zero
        double p_most = std::max(p_at(0), p_at(u1)), x_most = x_at(u1);
        auto inside = [=](double u) { return u > 0 && u < u1; };
        if (inside(-b / (2 * c))) p_most = std::max(p_most, p_at(-b / (2 * c)));
        if (c == 0) {
            if (inside(-a / (3 * b))) x_most = std::max(x_most, x_at(-a / (3 * b)));
        } else {
            const double root = std::sqrt(std::max(0.0, 9 * b * b - 20 * a * c));
            for (double u : {(-3 * b + root) / (10 * c), (-3 * b - root) / (10 * c)})
                if (inside(u)) x_most = std::max(x_most, x_at(u));
        }
        s = bits(u1, 0);
        p = bits(p_most, 0);
        sigma = std::min(x_most, 1e70);
        x = bits(sigma, least);
    }
};

// Factors of a step's products and sums, for X, S and P times their powers of two.
struct Factors {
    float s, c, b, a, next, out;  // S, S S, S and I in P; P X, as the next X and as the result
    Factors(Ranges& r, const double* abc)
    {
        const int x = r.x;
        r.step(abc[0], abc[1], abc[2]);
        s = (float)std::ldexp(1.0, r.s - 2 * x);
        c = (float)std::ldexp(abc[2], r.p - 2 * r.s);
        b = (float)std::ldexp(abc[1], r.p - r.s);
        a = (float)std::ldexp(abc[0], r.p);
        next = (float)std::ldexp(1.0, r.x - r.p - x);
        out = (float)std::ldexp(1.0, -r.p - x);
    }
};

template <class E>
int squares(const E* G, int64_t batch, int64_t rows, int64_t cols, int64_t ldg, int64_t stride_g, int vec, double* partial,
            hipStream_t stream)
{
    hipLaunchKernelGGL(ns_squares<E>, dim3((unsigned)(batch * kNormBlocks)), dim3(256), 0, stream, G, ldg, stride_g,
                       (int)rows, (int)cols, vec, partial);
    return (int)hipGetLastError();
}

template <class E>
int run_narrow(const narrow::Plan& plan, const E* G, __bf16* out, int64_t batch, int64_t rows, int64_t cols, int64_t ldg,
               int64_t stride_g, int64_t ldo, int64_t stride_o, int32_t steps, const double* coefficients, double eps,
               void* workspace, hipStream_t stream)
{
    const NarrowSpace w(workspace, batch, plan);
    const unsigned grid = (unsigned)(batch * plan.shares);  // (no more than 64 x 64 tiles)
    const int vec = (uintptr_t)G % (4 * sizeof(E)) == 0 && ldg % 4 == 0 && stride_g % 4 == 0;
    int rc = squares(G, batch, rows, cols, ldg, stride_g, vec, w.partial, stream);
    if (rc) return rc;
    narrow::Args a = {};
    a.xt = w.xt;
    a.out = out;
    a.m = (int)std::min(rows, cols);
    a.n = (int)std::max(rows, cols);
    a.shares = (int)plan.shares;
    a.chunks = (int)plan.chunks;
    a.cw = (int)plan.cw;
    a.tall = rows > cols;
    a.vec = (uintptr_t)out % 8 == 0 && ldo % 4 == 0 && stride_o % 4 == 0;
    a.ldo = ldo;
    a.stride_o = stride_o;
    Ranges ranges(a.n);
    const double scale = std::ldexp(1.0, ranges.x);
    a.to = w.shares[0];
    hipLaunchKernelGGL((narrow::ns_narrow_begin<E>), dim3(grid), dim3(narrow::kThreads), 0, stream, a, G, ldg,
                       stride_g, w.partial, eps, scale);
    if ((rc = (int)hipGetLastError())) return rc;
    for (int i = 0; i < steps; ++i) {
        a.from = w.shares[i & 1];
        a.to = w.shares[~i & 1];
        const Factors f(ranges, coefficients + 3 * i);
        a.alpha = f.s;
        a.a = f.a;
        a.b = f.b;
        a.c = f.c;
        a.next = i + 1 < steps ? f.next : f.out;
        if (i + 1 < steps)
            hipLaunchKernelGGL((narrow::ns_narrow_step<false>), dim3(grid), dim3(narrow::kThreads), 0, stream, a);
        else
            hipLaunchKernelGGL((narrow::ns_narrow_step<true>), dim3(grid), dim3(narrow::kThreads), 0, stream, a);
        if ((rc = (int)hipGetLastError())) return rc;
    }
    return hipSuccess;
}

template <class E>
int run(const E* G, __bf16* out, int64_t batch, int64_t rows, int64_t cols, int64_t ldg, int64_t stride_g, int64_t ldo,
        int64_t stride_o, int32_t steps, const double* coefficients, double eps, void* workspace, hipStream_t stream)
{
    const int64_t pr = abi::up(rows, kLine), pc = abi::up(cols, kLine);
    const int64_t tr = pr / 64, tc = pc / 64;
    // (no launch here has more workgroups than that)
    if (!abi::good_grid(tr * tc * batch, 256)) return hipErrorInvalidValue;
    const narrow::Plan plan(std::min(rows, cols), std::max(rows, cols));
    if (plan.used && steps > 0)
        return run_narrow(plan, G, out, batch, rows, cols, ldg, stride_g, ldo, stride_o, steps, coefficients, eps,
                                 workspace, stream);
    const Space w(workspace, batch, rows, cols);
    const bool tall = rows > cols;
    Ranges ranges(w.n);
    const double scale = std::ldexp(1.0, ranges.x);
    int rc;
    const int vec = (uintptr_t)G % (4 * sizeof(E)) == 0 && ldg % 4 == 0 && stride_g % 4 == 0;
    if ((rc = squares(G, batch, rows, cols, ldg, stride_g, vec, w.partial, stream))) return rc;
    half* d1 = tall ? w.xt[0] : w.x[0];
    half* d2 = tall ? w.x[0] : w.xt[0];
    hipLaunchKernelGGL(ns_start<E>, dim3((unsigned)(tr * tc * batch)), dim3(256), 0, stream, G, ldg, stride_g, (int)rows,
                       (int)cols, w.partial, eps, scale, d1, d2, w.stride_x, (int)pc, (int)pr, (int)tr, (int)tc, vec);
    if ((rc = (int)hipGetLastError())) return rc;
    if (steps == 0) {
        const int64_t total = batch * rows * cols;
        hipLaunchKernelGGL(ns_copy_out, dim3((unsigned)std::min<int64_t>((total + 255) / 256, 65536)), dim3(256), 0, stream,
                           d1, pc, w.stride_x, out, ldo, stride_o, (int)rows, (int)cols, total, (float)(1.0 / scale));
        return (int)hipGetLastError();
    }
    for (int i = 0; i < steps; ++i) {
        const int from = i & 1, to = from ^ 1;
        const Factors f(ranges, coefficients + 3 * i);
        SymmetricOp<false> s = {};
        s.A = w.x[from];
        s.C = w.s;
        s.M = (int)w.m;
        s.K = (int)w.np;
        s.lda = (int)w.ln;
        s.ldc = (int)w.lm;
        s.mp = (int)w.mp;
        s.stride_a = w.stride_x;
        s.stride_c = w.stride_s;
        s.alpha = f.s;
        if ((rc = launch_symmetric(s, w.m, batch, w.sums, stream))) return rc;
        SymmetricOp<true> p = {};
        p.A = w.s;
        p.C = w.p;
        p.diag = w.diag;
        p.M = (int)w.m;
        p.K = p.mp = (int)w.mp;
        p.lda = p.ldc = (int)w.lm;
        p.stride_a = p.stride_c = w.stride_s;
        p.alpha = f.c;
        p.beta = f.b;
        p.gamma = f.a;
        if ((rc = launch_symmetric(p, w.m, batch, w.sums, stream))) return rc;
        auto apply = [&](auto op) {
            op.P = w.p;
            op.diag = w.diag;
            op.Xt = w.xt[from];
            op.X = w.x[to];
            op.XtNew = w.xt[to];
            op.out = out;
            op.M = (int)w.m;
            op.N = (int)w.n;
            op.K = (int)w.mp;
            op.lda = op.ldb = (int)w.lm;
            op.ldx = (int)w.ln;
            op.np = (int)w.np;
            op.ldo = (int)ldo;
            op.stride_p = w.stride_s;
            op.stride_x = w.stride_x;
            op.stride_o = stride_o;
            op.alpha = i + 1 < steps ? f.next : f.out;
            return launch_grid<half>(op, w.m, w.n, 1, batch, op.K, w.sums, stream);
        };
        const bool eights = (uintptr_t)out % 16 == 0 && ldo % 8 == 0 && cols % 8 == 0 && stride_o % 8 == 0;
        if (i + 1 < steps)
            rc = apply(ApplyOp<false, kAsIs | kTurned | kEights>{});
        else if (tall)
            rc = eights ? apply(ApplyOp<true, kTurned | kEights>{}) : apply(ApplyOp<true, kTurned>{});
        else
            rc = eights ? apply(ApplyOp<true, kAsIs | kEights>{}) : apply(ApplyOp<true, kAsIs>{});
        if (rc) return rc;
    }
    return hipSuccess;
}

bool good_sizes(int64_t batch, int64_t rows, int64_t cols)
{
    return batch >= 0 && batch < (1 << 16) && rows >= 0 && rows <= abi::kMaxPitch - 63 && cols >= 0 &&
           cols <= abi::kMaxPitch - 63;
}

}  // namespace

extern "C" {

int orthogonalize_ns_version(void) { return ORTHOGONALIZE_NS_VERSION; }

int64_t orthogonalize_ns_workspace(int64_t batch, int64_t rows, int64_t cols)
{
    if (!good_sizes(batch, rows, cols)) return -1;
    if (batch == 0 || rows == 0 || cols == 0) return 0;
    const narrow::Plan plan(std::min(rows, cols), std::max(rows, cols));
    return std::max(Space(nullptr, batch, rows, cols).bytes, plan.used ? NarrowSpace(nullptr, batch, plan).bytes : 0);
}

int orthogonalize_ns(const void* G, void* out, int64_t batch, int64_t rows, int64_t cols, int64_t ldg, int64_t stride_g,
                     int64_t ldo, int64_t stride_o, int32_t type, int32_t steps, const double* coefficients, double eps,
                     void* workspace, int64_t workspace_bytes, hipStream_t stream)
{
    using namespace abi;
    if (!good_sizes(batch, rows, cols)) return hipErrorInvalidValue;
    if (ldg < cols || ldg > kMaxDim || ldo < cols || ldo > kMaxPitch) return hipErrorInvalidValue;
    if (type < ORTHOGONALIZE_NS_F16 || type > ORTHOGONALIZE_NS_F32) return hipErrorInvalidValue;
    if (steps < 0 || steps > 64 || (steps > 0 && !coefficients) || !(eps >= 0)) return hipErrorInvalidValue;
    if (batch == 0 || rows == 0 || cols == 0) return hipSuccess;
    const int64_t elem = type == ORTHOGONALIZE_NS_F32 ? 4 : 2;
    const int64_t span_g = (rows - 1) * ldg + cols, span_o = (rows - 1) * ldo + cols;
    const int64_t far = (int64_t)1 << 56;
    if (batch > 1 && (stride_g < 0 || stride_g > far / batch || stride_o < span_o || stride_o > far / batch))
        return hipErrorInvalidValue;
    if (!good_pointer(G, rows, cols, elem) || !good_pointer(out, rows, cols, 2) || (uintptr_t)workspace % 16)
        return hipErrorInvalidValue;
    const int64_t need = orthogonalize_ns_workspace(batch, rows, cols);
    if (!workspace || workspace_bytes < need) return hipErrorInvalidValue;
    const Range g(G, 1, (batch - 1) * (batch > 1 ? stride_g : 0) + span_g, 0, elem);
    const Range o(out, 1, (batch - 1) * (batch > 1 ? stride_o : 0) + span_o, 0, 2);
    const Range w(workspace, 1, need, 0, 1);
    if (o.meets(g) || o.meets(w) || w.meets(g)) return hipErrorInvalidValue;
    if (batch == 1) stride_g = stride_o = 0;
#define RUN(E)                                                                                                 \
    run<E>((const E*)G, (__bf16*)out, batch, rows, cols, ldg, stride_g, ldo, stride_o, steps, coefficients, eps, \
           workspace, stream)
    if (type == ORTHOGONALIZE_NS_F16) return RUN(_Float16);
    if (type == ORTHOGONALIZE_NS_BF16) return RUN(__bf16);
    return RUN(float);
#undef RUN
}

}  // extern "C"
