// Newton-Schulz orthogonalisation for gfx950: include/orthogonalize_ns.h.
//
// m <= n are the matrix's sides.  Per step, in NT form throughout,
//   S  = X X^T              [m, m] from X  [m, n]
//   P  = a I + b S + c S S  [m, m], S S = S S^T
//   X' = P X                [m, n] = P (X^T)^T from X^T [n, m]
// so both X and X^T are kept, and the product that makes X' writes both.  S
// and P are symmetric: only tiles on and below the diagonal are computed,
// and the others are written as their transposes.  a is part of P: P's
// diagonal is then near 1 once the singular values are, and its rounding
// costs a third of what the rounding of bS + cSS (diagonal near -2.7) does.
#include "orthogonalize_ns.h"

#include <algorithm>
#include <cmath>

#include "abi.h"
#include "nt_launch.h"
#include "relayout.h"

namespace {

using namespace nt;

typedef _Float16 half;
using half4 = Elem<half>::x4;

constexpr int kNormBlocks = 256;  // partial sums of squares per matrix

// Partial sums of squares, in 64 bits (a 32-bit sum would overflow for
// entries past 2^63 and lose small ones beside large ones).  Four elements of
// a row at a time; `per`: groups of four to a row.
template <class E>
__global__ void __launch_bounds__(256) ns_squares(const E* __restrict__ G, int64_t ldg, int64_t stride, int rows,
                                                  int cols, int per, int vec, double* __restrict__ partial)
{
    const int b = blockIdx.x / kNormBlocks, k = blockIdx.x % kNormBlocks;
    const E* g = G + b * stride;
    double s = 0;
    // a workgroup takes pieces of 256 groups of a row, or several short rows
    const int lanes = min(per, 256), step = 256 / lanes, pieces = (per + 255) / 256;
    const int lane = threadIdx.x % lanes, first = threadIdx.x / lanes;
    const int64_t units = first < step ? (int64_t)rows * pieces : 0;
    typedef E x4 __attribute__((ext_vector_type(4)));
    for (int64_t u = (int64_t)k * step + first; u < units; u += kNormBlocks * step) {
        const int64_t r = pieces == 1 ? u : u / pieces;
        const int c = ((int)(u - r * pieces) * 256 + lane) * 4;
        const E* at = g + r * ldg + c;
        x4 v = {};
        if (vec && c + 3 < cols) {
            v = *(const x4*)at;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (c + e < cols) v[e] = at[e];
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) s += (double)(float)v[e] * (double)(float)v[e];
    }
    __shared__ double part[256];
    part[threadIdx.x] = s;
    __syncthreads();
    for (int d = 128; d > 0; d >>= 1) {
        if (threadIdx.x < d) part[threadIdx.x] += part[threadIdx.x + d];
        __syncthreads();
    }
    if (threadIdx.x == 0) partial[blockIdx.x] = part[0];
}

// D1 [rows, p1] = G * scale / (norm + eps) and D2 [cols, p2] its transpose,
// both padded with zeros to their pitches.
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
    const float f = (float)(scale / (sqrt(part[0] + part[1] + part[2] + part[3]) + eps));
    const E* g = G + b * stride_g;
    half* d1 = D1 + b * stride_x;
    const int x = threadIdx.x & 15, y = threadIdx.x >> 4;
#pragma unroll
    for (int it = 0; it < 4; ++it) {
        const int r = it * 16 + y, c = c0 + x * 4;
        half4 v = {};
        if (r0 + r < rows) {
            const E* at = g + (r0 + r) * ldg + c;
            if (vec && c + 3 < cols) {
                typedef E x4 __attribute__((ext_vector_type(4)));
                const x4 w = *(const x4*)at;
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = (half)((float)w[e] * f);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (c + e < cols) v[e] = (half)((float)at[e] * f);
            }
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

// Where a tile goes: rows of a matrix from the tile's first one on, `pitch`
// bytes apart, and how many columns it has.
struct Rows {
    __amdgpu_buffer_rsrc_t rs;
    uint32_t pitch;
    int cols;
};
template <class E>
__device__ __forceinline__ Rows rows_at(E* base, int row, int rows, int most, int ld, int cols)
{
    Rows r;
    r.pitch = (uint32_t)ld * 2u;
    r.rs = make_rsrc(base + (int64_t)row * ld, (uint32_t)min(most, rows - row) * r.pitch);
    r.cols = cols;
    return r;
}

// How a tile is written: as it is, transposed, or both; rows in whole pieces
// (8 bytes, 16 for the transpose) or element by element.
enum { kAsIs = 1, kTurned = 2, kPieces = 4 };

// Writes the tile at (m0, n0).  The transpose goes through LDS: a lane's four values belong to
// four of its rows.  It is staged as rows n of BM columns m, ROUNDS turns of
// BN / ROUNDS rows, wave column wn's in stage[wn]; 16-byte chunk c of row n
// sits at c ^ 2 ((n / 4) % 8), so that the four rows that 64 lanes write lie
// in different banks.  It then leaves in whole rows, 16 bytes per lane.
template <class E, int HOW, class T, class Value>
__device__ __forceinline__ void write_tile(const f32x4 (&acc)[T::FM][T::FN], Value value, const Rows& direct,
                                           const Rows& turned, int m0, int n0, int lane, int wave,
                                           unsigned char* stage0, unsigned char* stage1)
{
    constexpr int FM = T::FM, FN = T::FN, WTM = T::WTM, WTN = T::WTN, ROUNDS = T::ROUNDS;
    constexpr int PITCH = T::BM * 2, CH = T::BM / 8;
    constexpr int RW = WTN / ROUNDS;  // staged rows per wave column
    constexpr int RPI = 64 / CH;      // rows per wave-wide read
    constexpr int ITERS = T::WAVES_N * RW / T::WAVES / RPI;
    static_assert(ITERS * RPI * T::WAVES == T::WAVES_N * RW, "rows split evenly over the waves");
    const int wm = wave / T::WAVES_N, wn = wave % T::WAVES_N;
    unsigned char* mine = wn ? stage1 + (wn - 1) * RW * PITCH : stage0;
#pragma unroll
    for (int h = 0; h < ROUNDS; ++h) {
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            const int ln = pinned(lane);
            const int r = wm * WTM + i * 16 + (ln & 15);
#pragma unroll
            for (int jj = 0; jj < FN / ROUNDS; ++jj) {
                const int j = h * (FN / ROUNDS) + jj;
                const int c = wn * WTN + j * 16 + 4 * (ln >> 4);
                const f32x4 v = value(r, c, acc[i][j]);
                if constexpr (HOW & kAsIs)
                    buffer_store4<E, (HOW & kPieces) != 0>(
                        direct.rs, (uint32_t)r * direct.pitch + (uint32_t)(n0 + c) * 2u, n0 + c, direct.cols, v);
                if constexpr (HOW & kTurned) {
                    const typename Elem<E>::x4 e4 = round4<E>(v);
                    const int row = jj * 16 + 4 * (ln >> 4);  // (row / 4 is the same for the four)
                    unsigned char* at = mine + row * PITCH + (((r >> 3) ^ ((2 * ((row >> 2) & 7)) & (CH - 1))) << 4) +
                                        (r & 7) * 2;
#pragma unroll
                    for (int e = 0; e < 4; ++e) *(E*)(at + e * PITCH) = e4[e];
                }
            }
        }
        if constexpr (HOW & kTurned) {
            lds_barrier<63>();
            const int ln = pinned(lane);
#pragma unroll
            for (int it = 0; it < ITERS; ++it) {
                const int row = (wave * ITERS + it) * RPI + ln / CH;  // of both wave columns'
                const int side = row / RW, local = row - side * RW, ch = ln % CH;
                const unsigned char* from = (side ? stage1 + (side - 1) * RW * PITCH : stage0) + local * PITCH +
                                            ((ch ^ ((2 * ((local >> 2) & 7)) & (CH - 1))) << 4);
                const typename Elem<E>::x8 v = *(const typename Elem<E>::x8*)from;
                const int m = m0 + ch * 8;
                const uint32_t at = (uint32_t)(side * WTN + h * RW + local) * turned.pitch + (uint32_t)m * 2u;
                if constexpr (HOW & kPieces) {
                    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), turned.rs,
                                                           m < turned.cols ? at : kOob, 0, 0);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const E one = v[e];
                        __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, one), turned.rs,
                                                              m + e < turned.cols ? at + (uint32_t)e * 2u : kOob, 0, 0);
                    }
                }
            }
            lds_barrier<63>();
        }
    }
}

// S (POLY false: alpha A A^T) or P (POLY true: alpha A A^T + beta A + gamma I,
// A symmetric), [m, m] with pitch mp, tiles on and below the diagonal and
// their transposes.
template <bool POLY>
struct SymmetricOp {
    static constexpr bool kPersist = true, kOblong = false;  // (square tiles)
    const half* A;
    half* C;
    int M, K, lda, mp, tiles, per;  // per: tiles of one matrix
    int64_t stride_a, stride_c;
    float alpha, beta, gamma;

    template <int BM, int BN>
    __device__ __forceinline__ void tile(int id, Tile& t) const
    {
        t.batch = id / per;
        id -= t.batch * per;
        // row r of the triangle holds tiles r (r + 1) / 2 .. + r
        int r = (int)((__builtin_sqrtf(8.0f * (float)id + 1.0f) - 1.0f) * 0.5f);
        while (r * (r + 1) / 2 > id) --r;
        while ((r + 1) * (r + 2) / 2 <= id) ++r;
        t.m0 = r * BM;
        t.n0 = (id - r * (r + 1) / 2) * BN;
    }
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
        const Rows direct = rows_at(c, t.m0, M, T::BM, mp, mp);
        // Rows M .. mp - 1 of the accumulator are zero: the transpose's
        // padding.  A tile on the diagonal has no mirror image to write.
        Rows turned = rows_at(c, t.n0, M, T::BN, mp, mp);
        if (t.m0 == t.n0) turned.rs = make_rsrc(c, 0);
        const Rows old = rows_at(A + t.batch * stride_a, t.m0, M, T::BM, lda, mp);
        auto value = [&](int r, int col, const f32x4& sum) __attribute__((always_inline)) {
            f32x4 v = sum * alpha;
            if constexpr (POLY) {
                const int n = t.n0 + col;
                const uint32_t at = n < mp ? (uint32_t)r * old.pitch + (uint32_t)n * 2u : kOob;
                const half4 a4 = __builtin_bit_cast(half4, __builtin_amdgcn_raw_buffer_load_b64(old.rs, at, 0, 0));
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    v[e] += __builtin_fmaf(beta, (float)a4[e], n + e == t.m0 + r ? gamma : 0.0f);
            }
            return v;
        };
        write_tile<half, kAsIs | kTurned | kPieces, T>(acc, value, direct, turned, t.m0, t.n0, lane, wave, s0, s1);
    }
};

// X' = P X [m, n] and its transpose [n, m] in binary16, or (LAST) the result
// in bfloat16, times alpha, in out's layout: out's rows are X's (HOW has
// kAsIs) or X^T's (kTurned).
template <bool LAST, int HOW>
struct ApplyOp {
    // (element by element, the 256 x 256 kernel would spill scalar registers)
    static constexpr bool kPersist = (HOW & kPieces) != 0, kOblong = true;
    const half *P, *Xt;
    half *X, *XtNew;
    __bf16* out;
    int M, N, K, lda, ldb, np, tiles, tiles_m, tiles_n, ldo;
    int64_t stride_p, stride_x, stride_o;
    float alpha;

    template <int BM, int BN>
    __device__ __forceinline__ void tile(int id, Tile& t) const
    {
        const int per = tiles_m * tiles_n;
        t.batch = id / per;
        int tm, tn;
        tile_of(id - t.batch * per, tiles_m, tiles_n, tm, tn);
        t.m0 = tm * BM;
        t.n0 = tn * BN;
    }
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
        auto value = [&](int, int, const f32x4& sum) __attribute__((always_inline)) { return LAST ? sum * alpha : sum; };
        if constexpr (LAST) {
            __bf16* o = out + t.batch * stride_o;
            Rows direct = {}, turned = {};
            if constexpr (HOW & kAsIs) direct = rows_at(o, t.m0, M, T::BM, ldo, N);
            if constexpr (HOW & kTurned) turned = rows_at(o, t.n0, N, T::BN, ldo, M);
            write_tile<__bf16, HOW, T>(acc, value, direct, turned, t.m0, t.n0, lane, wave, s0, s1);
        } else {
            // (columns N .. np - 1 and rows M .. ldb - 1 of the accumulator
            // are zero: the padding of both)
            const Rows direct = rows_at(X + t.batch * stride_x, t.m0, M, T::BM, np, np);
            const Rows turned = rows_at(XtNew + t.batch * stride_x, t.n0, N, T::BN, ldb, ldb);
            write_tile<half, HOW, T>(acc, value, direct, turned, t.m0, t.n0, lane, wave, s0, s1);
        }
    }
};

// ------------------------------------------------------------------ host --

struct Space {
    double* partial;
    half *x[2], *xt[2], *s, *p;
    int64_t m, n, mp, np, stride_x, stride_s, bytes;
    Space(void* base, int64_t batch, int64_t rows, int64_t cols)
    {
        m = std::min(rows, cols);
        n = std::max(rows, cols);
        mp = abi::up(m, 8);
        np = abi::up(n, 8);
        stride_x = mp * np;
        stride_s = mp * mp;
        abi::Carve c(base);
        partial = c.take<double>(batch * kNormBlocks);
        for (int i = 0; i < 2; ++i) {
            x[i] = c.take<half>(batch * stride_x);
            xt[i] = c.take<half>(batch * stride_x);
        }
        s = c.take<half>(batch * stride_s);
        p = c.take<half>(batch * stride_s);
        bytes = c.used();
    }
};

int64_t triangle(int64_t t) { return t * (t + 1) / 2; }

template <class OP>
int launch_symmetric(const OP& op, int64_t m, int64_t batch, hipStream_t stream)
{
    auto per = [=](const Kind& k) { return triangle((m + k.bm - 1) / k.bm); };
    return launch<half>(
        op, op.K, [=](const Kind& k) { return k.bm == k.bn ? per(k) * batch : -1; },
        [=](OP& o, const Kind& k) { o.per = (int)per(k); }, stream);
}

template <class E>
int run(const E* G, __bf16* out, int64_t batch, int64_t rows, int64_t cols, int64_t ldg, int64_t stride_g, int64_t ldo,
        int64_t stride_o, int32_t steps, const double* coefficients, double eps, void* workspace, hipStream_t stream)
{
    const Space w(workspace, batch, rows, cols);
    const bool tall = rows > cols;
    // an entry of an orthonormal X is about 1 / sqrt(n); X is held times
    // 2^k near sqrt(n), at most 2^12, so entries (at most about 1.2 before
    // the scale) neither leave binary16's range nor its full precision
    const int k = std::min(12, (int)std::lround(0.5 * std::log2((double)w.n)));
    const double scale = std::ldexp(1.0, k);
    int rc;
    const int vec = (uintptr_t)G % (4 * sizeof(E)) == 0 && ldg % 4 == 0 && stride_g % 4 == 0;
    hipLaunchKernelGGL(ns_squares<E>, dim3((unsigned)(batch * kNormBlocks)), dim3(256), 0, stream, G, ldg, stride_g,
                       (int)rows, (int)cols, (int)((cols + 3) / 4), vec, w.partial);
    if ((rc = (int)hipGetLastError())) return rc;
    const int64_t pr = abi::up(rows, 8), pc = abi::up(cols, 8);
    const int64_t tr = (pr + 63) / 64, tc = (pc + 63) / 64;
    if (tr * tc * batch > abi::kMaxDim) return hipErrorInvalidValue;
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
        SymmetricOp<false> s = {};
        s.A = w.x[from];
        s.C = w.s;
        s.M = (int)w.m;
        s.K = s.lda = (int)w.np;
        s.mp = (int)w.mp;
        s.stride_a = w.stride_x;
        s.stride_c = w.stride_s;
        s.alpha = (float)(1.0 / (scale * scale));
        if ((rc = launch_symmetric(s, w.m, batch, stream))) return rc;
        SymmetricOp<true> p = {};
        p.A = w.s;
        p.C = w.p;
        p.M = (int)w.m;
        p.K = p.lda = p.mp = (int)w.mp;
        p.stride_a = p.stride_c = w.stride_s;
        p.alpha = (float)coefficients[3 * i + 2];
        p.beta = (float)coefficients[3 * i + 1];
        p.gamma = (float)coefficients[3 * i];
        if ((rc = launch_symmetric(p, w.m, batch, stream))) return rc;
        auto apply = [&](auto op) {
            op.P = w.p;
            op.Xt = w.xt[from];
            op.X = w.x[to];
            op.XtNew = w.xt[to];
            op.out = out;
            op.M = (int)w.m;
            op.N = (int)w.n;
            op.K = op.lda = op.ldb = (int)w.mp;
            op.np = (int)w.np;
            op.ldo = (int)ldo;
            op.stride_p = w.stride_s;
            op.stride_x = w.stride_x;
            op.stride_o = stride_o;
            op.alpha = (float)(1.0 / scale);
            return launch_grid<half>(op, w.m, w.n, 1, batch, op.K, stream);
        };
        const bool eights = (uintptr_t)out % 16 == 0 && ldo % 8 == 0 && cols % 8 == 0 && stride_o % 8 == 0;
        if (i + 1 < steps)
            rc = apply(ApplyOp<false, kAsIs | kTurned | kPieces>{});
        else if (tall)
            rc = eights ? apply(ApplyOp<true, kTurned | kPieces>{}) : apply(ApplyOp<true, kTurned>{});
        else
            rc = eights ? apply(ApplyOp<true, kAsIs | kPieces>{}) : apply(ApplyOp<true, kAsIs>{});
        if (rc) return rc;
    }
    return hipSuccess;
}

bool good_sizes(int64_t batch, int64_t rows, int64_t cols)
{
    return batch >= 0 && batch < (1 << 16) && rows >= 0 && rows <= abi::kMaxPitch - 8 && cols >= 0 &&
           cols <= abi::kMaxPitch - 8;
}

}  // namespace

extern "C" {

int orthogonalize_ns_version(void) { return ORTHOGONALIZE_NS_VERSION; }

int64_t orthogonalize_ns_workspace(int64_t batch, int64_t rows, int64_t cols)
{
    if (!good_sizes(batch, rows, cols)) return -1;
    if (batch == 0 || rows == 0 || cols == 0) return 0;
    return Space(nullptr, batch, rows, cols).bytes;
}

int orthogonalize_ns(const void* G, void* out, int64_t batch, int64_t rows, int64_t cols, int64_t ldg, int64_t stride_g,
                     int64_t ldo, int64_t stride_o, int32_t type, int32_t steps, const double* coefficients, double eps,
                     void* workspace, int64_t workspace_bytes, hipStream_t stream)
{
    using namespace abi;
    if (!good_sizes(batch, rows, cols)) return hipErrorInvalidValue;
    if (ldg < cols || ldg > kMaxDim || ldo < cols || ldo > kMaxPitch) return hipErrorInvalidValue;
    if (type < ORTHOGONALIZE_NS_F16 || type > ORTHOGONALIZE_NS_F32) return hipErrorInvalidValue;
    if (steps < 0 || steps > 64 || (steps > 0 && !coefficients)) return hipErrorInvalidValue;
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
