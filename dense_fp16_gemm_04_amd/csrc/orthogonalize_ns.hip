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
#include "nt_core.h"
#include "relayout.h"

namespace {

using namespace nt;

typedef _Float16 half;
using half4 = Elem<half>::x4;

constexpr int kNormBlocks = 64;  // partial sums of squares per matrix

// Partial sums of squares, in 64 bits (a 32-bit sum would overflow for
// entries past 2^63 and lose small ones beside large ones).
template <class E>
__global__ void __launch_bounds__(256) ns_squares(const E* __restrict__ G, int64_t ldg, int64_t stride, int rows,
                                                  int cols, double* __restrict__ partial)
{
    const int b = blockIdx.x / kNormBlocks, k = blockIdx.x % kNormBlocks;
    const E* g = G + b * stride;
    double s = 0;
    const int64_t total = (int64_t)rows * cols;
    for (int64_t i = (int64_t)k * 256 + threadIdx.x; i < total; i += kNormBlocks * 256) {
        const int64_t r = i / cols;
        const double v = (double)(float)g[r * ldg + (i - r * cols)];
        s += v * v;
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
         int tiles_r, int tiles_c)
{
    using namespace relayout;
    __shared__ half tile[kTile * kPitch];
    __shared__ float factor;
    const int per = tiles_r * tiles_c, b = blockIdx.x / per, id = blockIdx.x % per;
    const int r0 = id / tiles_c * kTile, c0 = id % tiles_c * kTile;
    if (threadIdx.x == 0) {
        double s = 0;
        for (int i = 0; i < kNormBlocks; ++i) s += partial[b * kNormBlocks + i];
        factor = (float)(scale / (sqrt(s) + eps));
    }
    __syncthreads();
    const float f = factor;
    const E* g = G + b * stride_g;
    half* d1 = D1 + b * stride_x;
    const int x = threadIdx.x & 15, y = threadIdx.x >> 4;
#pragma unroll
    for (int it = 0; it < 4; ++it) {
        const int r = it * 16 + y, c = c0 + x * 4;
        half4 v = {};
        if (r0 + r < rows) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (c + e < cols) v[e] = (half)((float)g[(r0 + r) * ldg + c + e] * f);
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

// S (POLY false: alpha A A^T) or P (POLY true: alpha A A^T + beta A + gamma I,
// A symmetric), [m, m] with pitch mp, tiles on and below the diagonal and
// their transposes.
template <bool POLY>
struct SymmetricOp {
    const half* A;
    half* C;
    int M, K, lda, mp, per;  // per: tiles of one matrix
    int64_t stride_a, stride_c;
    float alpha, beta, gamma;

    template <int BM, int BN>
    __device__ __forceinline__ bool tile(int id, Tile& t) const
    {
        static_assert(BM == BN, "square tiles");
        t.batch = id / per;
        id -= t.batch * per;
        // row r of the triangle holds tiles r (r + 1) / 2 .. + r
        int r = (int)((__builtin_sqrtf(8.0f * (float)id + 1.0f) - 1.0f) * 0.5f);
        while (r * (r + 1) / 2 > id) --r;
        while ((r + 1) * (r + 2) / 2 <= id) ++r;
        t.m0 = r * BM;
        t.n0 = (id - r * (r + 1) / 2) * BN;
        return true;
    }
    __device__ __forceinline__ const half* a_rows(const Tile& t, int row, int& n) const
    {
        return rows_from(A + t.batch * stride_a, t.m0 + row, M, lda, n);
    }
    template <int BN>
    __device__ __forceinline__ const half* b_rows(const Tile& t, int row, int& n) const
    {
        return rows_from(A + t.batch * stride_a, t.n0 + row, M, lda, n);
    }
    __device__ __forceinline__ int b_pitch(int) const { return lda; }
    template <class T>
    __device__ __forceinline__ void epilogue(const Tile& t, const Acc<T>& acc, int lane, int wm, int wn,
                                             unsigned char*) const
    {
        const half* s = A + t.batch * stride_a;
        half* c = C + t.batch * stride_c;
        const bool mirror = t.m0 != t.n0;
#pragma unroll
        for (int i = 0; i < T::FM; ++i) {
            const int m = t.m0 + wm * T::WTM + i * 16 + (lane & 15);
            // rows M .. mp - 1 of the accumulator are zero: the transposed
            // tile's padding
            if (m >= mp) continue;
#pragma unroll
            for (int j = 0; j < T::FN; ++j) {
                const int n = t.n0 + wn * T::WTN + j * 16 + 4 * (lane >> 4);
                if (n >= mp) continue;
                f32x4 v = acc[i][j] * alpha;
                if constexpr (POLY) {
                    if (m < M) {
                        const half4 a4 = *(const half4*)(s + (int64_t)m * lda + n);
#pragma unroll
                        for (int e = 0; e < 4; ++e) v[e] += beta * (float)a4[e] + (n + e == m ? gamma : 0.0f);
                    }
                }
                const half4 h = round4<half>(v);
                if (m < M) *(half4*)(c + (int64_t)m * mp + n) = h;
                if (mirror)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (n + e < M) c[(int64_t)(n + e) * mp + m] = h[e];
            }
        }
    }
};

// X' = P X [m, n] and its transpose [n, m] in binary16, or (LAST) the result
// in bfloat16, times alpha, in the layout that out has.
template <bool LAST>
struct ApplyOp {
    const half *P, *Xt;
    half *X, *XtNew;
    __bf16* out;
    int M, N, K, lda, ldb, np, tiles_m, tiles_n, tall, vec, ldo;
    int64_t stride_p, stride_x, stride_o;
    float alpha;

    template <int BM, int BN>
    __device__ __forceinline__ bool tile(int id, Tile& t) const
    {
        const int per = tiles_m * tiles_n;
        t.batch = id / per;
        int tm, tn;
        tile_of(id - t.batch * per, tiles_m, tiles_n, 8, tm, tn);
        t.m0 = tm * BM;
        t.n0 = tn * BN;
        return true;
    }
    __device__ __forceinline__ const half* a_rows(const Tile& t, int row, int& n) const
    {
        return rows_from(P + t.batch * stride_p, t.m0 + row, M, lda, n);
    }
    template <int BN>
    __device__ __forceinline__ const half* b_rows(const Tile& t, int row, int& n) const
    {
        return rows_from(Xt + t.batch * stride_x, t.n0 + row, N, ldb, n);
    }
    __device__ __forceinline__ int b_pitch(int) const { return ldb; }
    template <class T>
    __device__ __forceinline__ void epilogue(const Tile& t, const Acc<T>& acc, int lane, int wm, int wn,
                                             unsigned char*) const
    {
#pragma unroll
        for (int i = 0; i < T::FM; ++i) {
            const int m = t.m0 + wm * T::WTM + i * 16 + (lane & 15);
            // (rows M .. ldb - 1: zeros, the padding of X'^T)
            if (m >= (LAST ? M : ldb)) continue;
#pragma unroll
            for (int j = 0; j < T::FN; ++j) {
                const int n = t.n0 + wn * T::WTN + j * 16 + 4 * (lane >> 4);
                if constexpr (LAST) {
                    __bf16* o = out + t.batch * stride_o;
                    const f32x4 v = acc[i][j] * alpha;
                    if (!tall) {
                        store4<__bf16>(o + (int64_t)m * ldo, n, N, v, vec);
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (n + e < N) o[(int64_t)(n + e) * ldo + m] = (__bf16)v[e];
                    }
                } else {
                    const half4 h = round4<half>(acc[i][j]);
                    if (m < M && n < np) *(half4*)(X + t.batch * stride_x + (int64_t)m * np + n) = h;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (n + e < N) XtNew[t.batch * stride_x + (int64_t)(n + e) * ldb + m] = h[e];
                }
            }
        }
    }
};

// ------------------------------------------------------------------ host --

using Tile128 = Shape<half, 128, 128, 3, 1>;
using Tile64 = Shape<half, 64, 64, 3, 2>;

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
int launch_symmetric(OP op, int64_t m, int64_t batch, hipStream_t stream)
{
    const bool big = triangle((m + 127) / 128) * batch >= 128;
    const int64_t edge = big ? 128 : 64, per = triangle((m + edge - 1) / edge);
    if (per * batch > abi::kMaxDim) return hipErrorInvalidValue;
    op.per = (int)per;
    if (big)
        hipLaunchKernelGGL((nt_tile<Tile128, OP>), dim3((unsigned)(per * batch)), dim3(256), 0, stream, op);
    else
        hipLaunchKernelGGL((nt_tile<Tile64, OP>), dim3((unsigned)(per * batch)), dim3(256), 0, stream, op);
    return (int)hipGetLastError();
}

template <class OP>
int launch_apply(OP op, int64_t m, int64_t n, int64_t batch, hipStream_t stream)
{
    const bool big = ((m + 127) / 128) * ((n + 127) / 128) * batch >= 128;
    const int64_t edge = big ? 128 : 64, tm = (m + edge - 1) / edge, tn = (n + edge - 1) / edge;
    if (tm * tn * batch > abi::kMaxDim) return hipErrorInvalidValue;
    op.tiles_m = (int)tm;
    op.tiles_n = (int)tn;
    if (big)
        hipLaunchKernelGGL((nt_tile<Tile128, OP>), dim3((unsigned)(tm * tn * batch)), dim3(256), 0, stream, op);
    else
        hipLaunchKernelGGL((nt_tile<Tile64, OP>), dim3((unsigned)(tm * tn * batch)), dim3(256), 0, stream, op);
    return (int)hipGetLastError();
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
    hipLaunchKernelGGL(ns_squares<E>, dim3((unsigned)(batch * kNormBlocks)), dim3(256), 0, stream, G, ldg, stride_g,
                       (int)rows, (int)cols, w.partial);
    if ((rc = (int)hipGetLastError())) return rc;
    const int64_t pr = abi::up(rows, 8), pc = abi::up(cols, 8);
    const int64_t tr = (pr + 63) / 64, tc = (pc + 63) / 64;
    if (tr * tc * batch > abi::kMaxDim) return hipErrorInvalidValue;
    half* d1 = tall ? w.xt[0] : w.x[0];
    half* d2 = tall ? w.x[0] : w.xt[0];
    hipLaunchKernelGGL(ns_start<E>, dim3((unsigned)(tr * tc * batch)), dim3(256), 0, stream, G, ldg, stride_g, (int)rows,
                       (int)cols, w.partial, eps, scale, d1, d2, w.stride_x, (int)pc, (int)pr, (int)tr, (int)tc);
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
            op.tall = tall;
            op.vec = (uintptr_t)out % 8 == 0 && ldo % 4 == 0 && (batch == 1 || stride_o % 4 == 0);
            op.ldo = (int)ldo;
            op.stride_p = w.stride_s;
            op.stride_x = w.stride_x;
            op.stride_o = stride_o;
            op.alpha = (float)(1.0 / scale);
            return launch_apply(op, w.m, w.n, batch, stream);
        };
        if ((rc = i + 1 < steps ? apply(ApplyOp<false>{}) : apply(ApplyOp<true>{}))) return rc;
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
    if (ldg < cols || ldg > kMaxDim || ldo < cols || ldo > kMaxDim) return hipErrorInvalidValue;
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
