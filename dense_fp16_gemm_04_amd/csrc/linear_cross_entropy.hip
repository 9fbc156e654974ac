// The softmax cross entropy of a linear layer's outputs over a vocabulary, and
// its gradients, for gfx950: include/linear_cross_entropy.h.
//
// Forward: one NT product X W^T whose epilogue reduces each row of a wave's
// sub-tile to its largest output and the sum of exponentials about it, eight
// bytes for 32 to 128 outputs; a second kernel joins them.
//
// Backward, a piece of the vocabulary at a time: the product again, whose
// epilogue turns outputs to dl = softmax - onehot and writes it row-major, and
// times dloss transposed; dX += dl W, with sums kept in 32 bits from piece to
// piece, and dW = (dloss dl)^T X in NT form on a transposed copy of X.  dX takes W
// as it lies, or (in the largest tiles) from a transposed copy of the piece.
//
// Bound by the matrix cores where K is long (8192 x 4096 x 131072: 6.1 ms for the
// loss and 18.3 for the gradients, 1437 TFLOP/s), and by the epilogues, 6 us a tile for
// the loss and 12 for dl, where it is short (1000 x 1032 x 32001: 80 and 95 us for
// 45 us of products each).
#include "linear_cross_entropy.h"

#include <algorithm>

#include "abi.h"
#include "nt_launch.h"
#include "relayout.h"

namespace {

using namespace nt;

constexpr float kLog2e = 1.44269504f;

typedef float f32x2 __attribute__((ext_vector_type(2)));

// The largest and the sum over the four groups of 16 lanes, which hold a row.
__device__ __forceinline__ float max_over_groups(float v)
{
    v = fmaxf(v, __shfl_xor(v, 16));
    return fmaxf(v, __shfl_xor(v, 32));
}
__device__ __forceinline__ float sum_over_groups(float v)
{
    v += __shfl_xor(v, 16);
    return v + __shfl_xor(v, 32);
}

// What exponentials are taken about: the largest output, or 0 where that is
// -infinity (there are none, or all are: the sum is then 0, not NaN).
__device__ __forceinline__ float about(float m) { return m == -INFINITY ? 0.0f : m; }

// A block's values, where it holds 256 accumulation registers read one by one and
// anew each time: a value that the compiler reads twice it keeps in a vector
// register from the first time on, and all of them spill.  (The kernel has
// waited for its last MFMAs before the epilogue.)
template <class T>
__device__ __forceinline__ f32x4 read(const f32x4& acc)
{
    if constexpr (T::FM * T::FN < 64) return acc;
    f32x4 v;
#pragma unroll
    for (int e = 0; e < 4; ++e) asm volatile("v_accvgpr_read_b32 %0, %1" : "=v"(v[e]) : "a"(acc[e]));
    return v;
}

// The value is computed here, not later with what it is made of kept until then.
__device__ __forceinline__ float done(float v)
{
    asm volatile("" : "+v"(v));
    return v;
}

template <class E>
struct LseOp {
    static constexpr bool kPersist = true, kSplit = true;
    const E *X, *W;
    const int64_t* target;
    float* tl;     // [M]: the target's output
    f32x2* parts;  // [segments][Mp]: (largest, sum) of WTN columns of a row
    int64_t target_stride, Mp;
    int M, N, K, lda, ldb, first, tiles, tiles_m, tiles_n;  // first: the column that W's first row is

    template <int BM, int BN>
    __device__ __forceinline__ void tile(int id, Tile& t) const
    {
        int tm, tn;
        grid_tile(xcd_order(id, tiles), tiles_m, tiles_n, tm, tn);
        t.m0 = tm * BM;
        t.n0 = tn * BN;
        t.batch = 0;
    }
    __device__ __forceinline__ bool outside(const Tile& t) const { return t.m0 >= M || t.n0 >= N; }
    __device__ __forceinline__ const E* a_rows(const Tile& t, int row, int& n) const
    {
        return rows_from(X, t.m0 + row, M, lda, n);
    }
    template <int WTN>
    __device__ __forceinline__ const E* b_rows(const Tile& t, int row, int& n) const
    {
        return rows_from(W, t.n0 + row, N, ldb, n);
    }
    template <int WTN>
    __device__ __forceinline__ int b_pitch(int) const
    {
        return ldb;
    }
    template <class T>
    __device__ __forceinline__ void epilogue(const Tile& t, const f32x4 (&acc)[T::FM][T::FN], int lane, int wave, unsigned char*,
                                             unsigned char*) const
    {
        // (One basic block up to the targets: values that live across a branch
        // are taken out of the accumulation registers before it, and spill.)
        const int ln = pinned(lane);
        const int m0 = t.m0 + wave / T::WAVES_N * T::WTM, n0 = t.n0 + wave % T::WAVES_N * T::WTN;
        // -infinity is added to columns that are not there, 0 to the others
        const int there = N - n0 - 4 * (ln >> 4);  // of the lane's columns, from its first on
        float top[T::FM], sum[T::FM];
        int64_t c[T::FM];  // (loaded while the sums are made)
#pragma unroll
        for (int i = 0; i < T::FM; ++i) {
            top[i] = -INFINITY;
            c[i] = target[min(m0 + i * 16 + (ln & 15), M - 1) * target_stride];
        }
#pragma unroll
        for (int j = 0; j < T::FN; ++j) {
            const f32x4 bias = absent(j, there);
#pragma unroll
            for (int i = 0; i < T::FM; ++i) top[i] = done(fmaxf(top[i], largest(read<T>(acc[i][j]) + bias)));
        }
#pragma unroll
        for (int i = 0; i < T::FM; ++i) {
            top[i] = max_over_groups(top[i]);
            sum[i] = 0.0f;
        }
#pragma unroll
        for (int j = 0; j < T::FN; ++j) {
            const f32x4 bias = absent(j, there);
#pragma unroll
            for (int i = 0; i < T::FM; ++i) {
                const f32x4 l = read<T>(acc[i][j]);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    sum[i] += __builtin_amdgcn_exp2f(__builtin_fmaf(l[e] - about(top[i]), kLog2e, bias[e]));
                sum[i] = done(sum[i]);
            }
        }
        __builtin_amdgcn_sched_barrier(0);
        // (sub-tiles past the last column have no part)
        const __amdgpu_buffer_rsrc_t to =
            make_rsrc(parts + (int64_t)(n0 / T::WTN) * Mp + m0, n0 < N && m0 < M ? (uint32_t)min(M - m0, T::WTM) * 8u : 0u);
        int at[T::FM];  // the target's place among the lane's columns
        bool any = false;
#pragma unroll
        for (int i = 0; i < T::FM; ++i) {
            const int row = m0 + i * 16 + (ln & 15);
            const f32x2 part = {top[i], sum_over_groups(sum[i])};
            __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, part), to, ln < 16 ? (i * 16 + ln) * 8 : kOob, 0, 0);
            const int64_t place = c[i] - first - n0;
            at[i] = row < M && place >= 0 && place < min(T::WTN, N - n0) ? (int)place - 4 * (ln >> 4) : -1;
            any |= at[i] >= 0;
        }
        if (!__any(any)) return;
        // the lane's value in the target's column: few sub-tiles have any
        float found[T::FM];
#pragma unroll
        for (int i = 0; i < T::FM; ++i) {
            bool mine = false;
            found[i] = 0.0f;
#pragma unroll
            for (int j = 0; j < T::FN; ++j) {
                const f32x4 l = read<T>(acc[i][j]);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const bool here = at[i] == j * 16 + e;
                    found[i] = here ? l[e] : found[i];
                    mine |= here;
                }
                found[i] = done(found[i]);
            }
            at[i] = mine ? 0 : -1;
        }
#pragma unroll
        for (int i = 0; i < T::FM; ++i)
            if (at[i] == 0) tl[m0 + i * 16 + (ln & 15)] = found[i];
    }
    static __device__ __forceinline__ float largest(const f32x4& v) { return fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])); }
    static __device__ __forceinline__ f32x4 absent(int j, int there)
    {
        f32x4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = j * 16 + e < there ? 0.0f : -INFINITY;
        return v;
    }
};

// Joins the parts of R rows to a workgroup: 1024 / R threads take every so many
// of a row's, and meet in LDS.
constexpr int kJoin = 1024;

struct Join {
    const f32x2* parts;
    const int64_t* target;
    const float* tl;
    float *loss, *saved;  // saved null: not kept
    int64_t target_stride, ignore, Mp;
    int M, N, segments;
};

// (largest, sum) of two parts.
__device__ __forceinline__ f32x2 joined(const f32x2& a, const f32x2& b)
{
    const float m = fmaxf(a[0], b[0]), c = about(m);
    return f32x2{m, a[1] * __builtin_amdgcn_exp2f((a[0] - c) * kLog2e) + b[1] * __builtin_amdgcn_exp2f((b[0] - c) * kLog2e)};
}

template <int R>
__global__ void __launch_bounds__(kJoin) lse_join(const Join f)
{
    constexpr int S = kJoin / R;
    __shared__ f32x2 meet[S][R];
    const int r = threadIdx.x % R, s = threadIdx.x / R;
    const int64_t row = (int64_t)blockIdx.x * R + r;
    f32x2 all = {-INFINITY, 0.0f};
    if (row < f.M) {
        const f32x2* at = f.parts + row;
        int p = s;
        for (; p + 3 * S < f.segments; p += 4 * S) {
            f32x2 v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = at[(p + k * S) * f.Mp];
            all = joined(all, joined(joined(v[0], v[1]), joined(v[2], v[3])));
        }
        for (; p < f.segments; p += S) all = joined(all, at[p * f.Mp]);
    }
    meet[s][r] = all;
#pragma unroll
    for (int half = S / 2; half > 0; half /= 2) {
        __syncthreads();
        if (s < half) meet[s][r] = joined(meet[s][r], meet[s + half][r]);
    }
    if (s > 0 || row >= f.M) return;
    all = meet[0][r];
    const int64_t c = f.target[row * f.target_stride];
    const bool there = c >= 0 && c < f.N;
    const bool ignored = c == f.ignore;
    const float tl = ignored ? 0.0f : there ? f.tl[row] : NAN;
    f.loss[row] = ignored ? 0.0f : (all[0] - tl) + logf(all[1]);
    if (f.saved) {
        f.saved[3 * row] = all[0];
        f.saved[3 * row + 1] = all[1];
        f.saved[3 * row + 2] = tl;
    }
}

// ------------------------------------------------------------- backward --

#include "loss_few.h"

// binary16 ends at 2^-24: dl is held times 2^15.  bfloat16 has the range of 32
// bits and needs no shift.
template <class E>
constexpr float kShift = 0.0f;
template <>
constexpr float kShift<_Float16> = 15.0f;

// What the backward pass needs of a row.  dl 2^shift = exp2(min(l - top, 0)
// log2 e + bias) but in the target's column, where it is `hit`; what makes dW is
// that times `weight`, dloss over its largest magnitude, which dW's product puts
// back: where all tokens have one dloss, as of a mean, its digits then are in no
// rounding (8192 x 4096 x 131072 in bfloat16: dW 3.0e-3 off with dloss itself in
// them, twice what its own rounding leaves).  A row that is ignored or not there
// has 0, -infinity, 0, 0: then the minimum, which takes the number of a number and
// NaN, makes dl zero whatever l is.  Of columns that are not there it keeps dl
// finite, and of those that are l is no larger than top but by another order of
// summation.
//
// The target's dl is most of a row's size, and its rounding most of dX's error
// where few terms are large.  Each row of dl is therefore held times what makes
// `hit` a number of the type (1 and half a step at most), which `back`, the factor
// to the row's sums, and `weight` take out again: dX (300 x 200 x 513, binary16)
// 2.28e-4 off, its own rounding, and 2.73e-4 without.
struct RowInfo {
    float top, bias, weight, hit;
};

// The rows' numbers, by one workgroup: dloss' largest magnitude has to be known first.
template <class E>
struct RowNumbers {
    const float *dloss, *saved;
    const int64_t* target;
    int64_t dloss_stride, target_stride, ignore;
    int M, Mp, N;  // Mp: rows of whole tiles
    RowInfo* info;
    int* column;    // of the target, or -1
    float* back;    // to dX's sums
    float* factor;  // to dW's sums

    __device__ __forceinline__ void run() const
    {
        __shared__ float part[relayout::kThreads / kWave];
        float most = 0.0f;
        for (int row = threadIdx.x; row < M; row += relayout::kThreads) {
            const float g = fabsf(dloss[row * dloss_stride]);
            if (target[row * target_stride] != ignore && g < INFINITY) most = fmaxf(most, g);
        }
        for (int d = 32; d > 0; d >>= 1) most = fmaxf(most, __shfl_xor(most, d));
        if (threadIdx.x % kWave == 0) part[threadIdx.x / kWave] = most;
        __syncthreads();
        most = fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3]));
        if (most == 0.0f) most = 1.0f;
        if (threadIdx.x == 0) *factor = most * exp2f(-kShift<E>);
        for (int row = threadIdx.x; row < Mp; row += relayout::kThreads) {
            RowInfo r = {0.0f, -INFINITY, 0.0f, 0.0f};
            float b = 0.0f;
            int at = -1;
            if (row < M) {
                const int64_t c = target[row * target_stride];
                if (c != ignore) {
                    const float top = saved[3 * (int64_t)row], sum = saved[3 * (int64_t)row + 1], tl = saved[3 * (int64_t)row + 2];
                    const bool there = c >= 0 && c < N;
                    const float g = dloss[row * dloss_stride], hit = (expf(tl - top) - sum) / sum * exp2f(kShift<E>);
                    r.hit = (float)(E)hit;
                    const float times = r.hit == 0.0f ? 1.0f : r.hit / hit;
                    r.top = top;
                    r.bias = there ? kShift<E> - log2f(sum) + log2f(times) : NAN;
                    r.weight = g / most / times;
                    b = g * exp2f(-kShift<E>) / times;
                    at = there ? (int)c : -1;
                }
            }
            info[row] = r;
            back[row] = b;
            column[row] = at;
        }
    }
};

// An operand's rows laid out as the products read them, by tiles of 64 x 64 read
// once: copied to rows of whole cache lines (where they cannot be read in place) and
// transposed (where a gradient sums over them), zeros past their end.  Of tokens
// that are ignored the transpose holds zeros: 0 times what they hold may be NaN.
template <class E>
struct LayOut {
    const E* src;
    E *copy, *turned;  // null: not made
    int64_t ld, ld_copy, ld_turned;
    int rows, cols;
    const int64_t* target;  // null: rows are not tokens
    int64_t target_stride, ignore;

    __host__ __device__ int64_t tiles() const
    {
        constexpr int64_t N = relayout::kTile;
        return copy || turned ? (rows + N - 1) / N * ((cols + N - 1) / N) : 0;
    }
    __device__ __forceinline__ void run(int id, E* tile) const
    {
        using namespace relayout;
        const int tiles_c = (cols + kTile - 1) / kTile;
        const int r0 = id / tiles_c * kTile, c0 = id % tiles_c * kTile;
        const int x = threadIdx.x & 15, y = threadIdx.x >> 4, c = c0 + x * 4;
#pragma unroll
        for (int it = 0; it < 4; ++it) {
            const int r = it * 16 + y;
            Four<E> v = {};
            if (r0 + r < rows && c < cols) {
                // (a row's end is loaded from four elements before it, and shifted)
                const int past = cols < 4 ? 0 : max(c + 4 - cols, 0);
                v = ::rows::load<E, 4>(src + (r0 + r) * ld + c - past, cols < 4 ? cols - c : 4);
                v = __builtin_bit_cast(Four<E>, __builtin_bit_cast(uint64_t, v) >> past * 16);
            }
            if (copy && r0 + r < rows) *(Four<E>*)(copy + (r0 + r) * ld_copy + c) = v;
            if (target && r0 + r < rows && target[(r0 + r) * target_stride] == ignore) v = Four<E>{};
            *(Four<E>*)(tile + r * kPitch + x * 4) = v;
        }
        if (!turned) return;
        __syncthreads();
        store_transposed(tile, turned, ld_turned, r0, c0, (int)ld_turned, cols);
    }
};

// What the products read, in one launch: the rows' numbers (with the first piece), X and
// a piece of W.
template <class E>
struct Prepare {
    RowNumbers<E> numbers;
    LayOut<E> x, w;
    int first, second;  // the layouts' first workgroups
};

template <class E>
__global__ void __launch_bounds__(relayout::kThreads) loss_prepare(const Prepare<E> p)
{
    __shared__ E tile[relayout::kTile * relayout::kPitch];
    const int id = blockIdx.x;
    if (id < p.first)
        p.numbers.run();
    else if (id < p.second)
        p.x.run(id - p.first, tile);
    else
        p.w.run(id - p.second, tile);
}

template <class E>
int enqueue(Prepare<E>& p, bool numbers, hipStream_t stream)
{
    p.first = numbers ? 1 : 0;
    p.second = p.first + (int)p.x.tiles();
    const int64_t groups = p.second + p.w.tiles();
    if (groups == 0) return hipSuccess;
    hipLaunchKernelGGL(loss_prepare<E>, dim3((unsigned)groups), dim3(relayout::kThreads), 0, stream, p);
    return (int)hipGetLastError();
}

// dl of a piece of the vocabulary: row-major to dl (pitch ldd), times dloss and
// transposed to dlt (pitch ldt).
template <class E>
struct DlOp {
    static constexpr bool kPersist = true, kSplit = false;
    const E *X, *W;  // W from the piece's first row on
    E *dl, *dlt;
    const RowInfo* info;
    const int* column;
    int M, N, K, lda, ldb, ldd, ldt, first, tiles, tiles_m, tiles_n;

    template <int BM, int BN>
    __device__ __forceinline__ void tile(int id, Tile& t) const
    {
        int tm, tn;
        grid_tile(xcd_order(id, tiles), tiles_m, tiles_n, tm, tn);
        t.m0 = tm * BM;
        t.n0 = tn * BN;
        t.batch = 0;
    }
    __device__ __forceinline__ const E* a_rows(const Tile& t, int row, int& n) const
    {
        return rows_from(X, t.m0 + row, M, lda, n);
    }
    template <int WTN>
    __device__ __forceinline__ const E* b_rows(const Tile& t, int row, int& n) const
    {
        return rows_from(W, t.n0 + row, N, ldb, n);
    }
    template <int WTN>
    __device__ __forceinline__ int b_pitch(int) const
    {
        return ldb;
    }
    template <class T>
    __device__ __forceinline__ void epilogue(const Tile& t, const f32x4 (&acc)[T::FM][T::FN], int lane, int wave, unsigned char* s0,
                                             unsigned char* s1) const
    {
        const int ln = pinned(lane), wm = wave / T::WAVES_N, wn = wave % T::WAVES_N;
        const RowInfo* const rows = info + t.m0 + wm * T::WTM + (ln & 15);
        float top[T::FM], bias[T::FM];
#pragma unroll
        for (int i = 0; i < T::FM; ++i) {
            top[i] = rows[i * 16].top;
            bias[i] = rows[i * 16].bias;
        }
        auto dl_of = [&](int i, int j) __attribute__((always_inline)) {
            f32x4 v = read<T>(acc[i][j]);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(fminf(v[e] - top[i], 0.0f), kLog2e, bias[i]));
            __builtin_amdgcn_sched_barrier(0);  // (block by block, for the registers' sake)
            return v;
        };
        // a row's target, if among the wave's columns, from the first of them
        int at[T::FM];
        float hit[T::FM], weight[T::FM];
#pragma unroll
        for (int i = 0; i < T::FM; ++i) {
            at[i] = column[t.m0 + wm * T::WTM + i * 16 + (ln & 15)] - first - t.n0 - wn * T::WTN;
            hit[i] = rows[i * 16].hit;
            weight[i] = rows[i * 16].weight;
        }
        // Both images at once, so that each exponential is taken once; of 256 x 256
        // tiles, whose LDS holds a quarter of both, in four rounds of 32 rows of
        // each wave.  (Row-major first, then transposed with the exponentials
        // taken again, two rounds each: 107 us for 1000 x 1032 x 32001, and 98.)
        constexpr int ROUNDS = T::BM * T::BN * 4 > T::STAGE_MAX ? 4 : 1, IR = T::FM / ROUNDS, RW = T::WTM / ROUNDS;
        constexpr int TC = T::BM / ROUNDS, TCH = TC / 8, RPI = 64 / TCH, ITERS = T::BN / RPI / T::WAVES;
        static_assert(T::BM * T::BN * 4 <= ROUNDS * T::STAGE_MAX && ITERS * RPI * T::WAVES == T::BN, "both images fit");
        constexpr int BYTES = T::BM * T::BN * 2 / ROUNDS;
        const Image<T::BN> image{s0, s0 + 32768};
        const Image<TC> turned{ROUNDS > 1 ? s1 : s0 + BYTES, s0 + BYTES + 32768};
        static_assert(ROUNDS == 1 || BYTES == 32768, "an image to a slot");
        // (columns past N, up to a chunk of eight, hold numbers, which meet zeros)
        const Rows to = rows_at(dl, t.m0, M, T::BM, ldd, t.n0, (N + 7) & ~7);
        const Rows to_t = rows_at(dlt, t.n0, N, T::BN, ldt, t.m0, (M + 7) & ~7);
#pragma unroll
        for (int h = 0; h < ROUNDS; ++h) {
            const int l = pinned(lane), r = l & 15, q = 4 * (l >> 4);
#pragma unroll
            for (int k = 0; k < IR; ++k) {
                const int i = h * IR + k, row = wm * RW + k * 16;
                float own = 0.0f;
#pragma unroll
                for (int j = 0; j < T::FN; ++j) {
                    const f32x4 v = dl_of(i, j);
                    if (j == 0) own = v[0];
                    image.put(row + r, wn * T::WTN + j * 16 + q, round4<E>(v));
                    turned.put(wn * T::WTN + j * 16 + q + (l & 3), row + (l & 12), quad_transposed(round4<E>(v * weight[i]), l));
                }
                // The target's column.  (A row without one here gets a value that it
                // has: a branch would take all accumulators out of their registers.)
                const bool here = at[i] >= 0 && at[i] < T::WTN;
                const int c = wn * T::WTN + (here ? at[i] : q);
                const float v = here ? hit[i] : own;
                image.set(row + r, c, (E)v);
                turned.set(c, row + r, (E)(v * weight[i]));
            }
            lds_barrier<63>();
            drain<T, T::BN, T::WAVES_M * RW, true>(image, to, [&](int x) { return x / RW * T::WTM + h * RW + x % RW; }, lane, wave);
            const int ch = l % TCH, m = t.m0 + ch * 8 / RW * T::WTM + h * RW + ch * 8 % RW;
            const int x0 = (int)as_vector((uint32_t)wave * (ITERS * RPI)) + l / TCH;
#pragma unroll
            for (int it = 0; it < ITERS; ++it) {
                const int x = x0 + it * RPI;
                const uint32_t at = m < to_t.cols ? (uint32_t)x * to_t.pitch + (uint32_t)m * 2u : kOob;
                __builtin_amdgcn_raw_buffer_store_b128(turned.get(x, ch), to_t.rs, at, 0, 0);
            }
            lds_barrier<63>();
        }
    }
};

// sums += A B^T, sums in blocks of 16 x 16, row of blocks by row, in the order in
// which a wave's lanes hold them (lane l: row l % 16, columns 4 (l / 16) .. + 3).
constexpr int kBlockFloats = 256;

// TURNED: B is W where it lies, `there` rows.
template <class E, bool TURNED>
struct AddOp {
    static constexpr bool kPersist = !TURNED, kSplit = true, kTurned = TURNED;
    const E *A, *B;
    float* sums;
    int M, N, K, lda, ldb, there, fresh, tiles, tiles_m, tiles_n;  // fresh: sums hold nothing yet

    template <int BM, int BN>
    __device__ __forceinline__ void tile(int id, Tile& t) const
    {
        int tm, tn;
        grid_tile(xcd_order(id, tiles), tiles_m, tiles_n, tm, tn);
        t.m0 = tm * BM;
        t.n0 = tn * BN;
        t.batch = 0;
    }
    __device__ __forceinline__ bool outside(const Tile& t) const { return t.m0 >= M || t.n0 >= N; }
    __device__ __forceinline__ const E* a_rows(const Tile& t, int row, int& n) const
    {
        return rows_from(A, t.m0 + row, M, lda, n);
    }
    template <int WTN>
    __device__ __forceinline__ const E* b_rows(const Tile& t, int row, int& n) const
    {
        return rows_from(B, t.n0 + row, N, ldb, n);
    }
    __device__ __forceinline__ const E* b_turned(const Tile& t, int& steps, int& cols) const
    {
        steps = there;
        cols = ((N + 7) & ~7) - t.n0;
        return B + t.n0;
    }
    template <int WTN>
    __device__ __forceinline__ int b_pitch(int) const
    {
        return ldb;
    }
    template <class T>
    __device__ __forceinline__ void epilogue(const Tile& t, const f32x4 (&acc)[T::FM][T::FN], int lane, int wave, unsigned char*,
                                             unsigned char*) const
    {
        const int ln = pinned(lane);
        const int bm = (t.m0 + wave / T::WAVES_N * T::WTM) / 16, bn = (t.n0 + wave % T::WAVES_N * T::WTN) / 16;
        // (what is not there is out of the buffers' range, and so are sums that
        // hold nothing yet: read as zeros, not written)
        const int rows = (M + 15) / 16 - bm, cols = (N + 15) / 16, left = max(cols - bn, 0);
#pragma unroll
        for (int i = 0; i < T::FM; ++i) {
            __builtin_amdgcn_sched_barrier(0);  // (row by row of blocks, for the registers' sake)
            const float* const at = sums + ((int64_t)(bm + i) * cols + bn) * kBlockFloats;
            const uint32_t bytes = i < rows ? (uint32_t)left * (kBlockFloats * 4u) : 0u;
            const __amdgpu_buffer_rsrc_t to = make_rsrc(at, bytes), from = make_rsrc(at, fresh ? 0u : bytes);
            u32x4 old[T::FN];
#pragma unroll
            for (int j = 0; j < T::FN; ++j)
                old[j] = __builtin_amdgcn_raw_buffer_load_b128(from, ln * 16 + j * (kBlockFloats * 4), 0, 0);
#pragma unroll
            for (int j = 0; j < T::FN; ++j) {
                const f32x4 v = acc[i][j] + __builtin_bit_cast(f32x4, old[j]);
                __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), to, ln * 16 + j * (kBlockFloats * 4), 0, 0);
            }
        }
    }
};

// write_rows for rows on any boundary: eight columns to a lane at any address but at
// a row's end, and branches around what is not there, which is why the values
// come by read().  (dW of 181 x 333 x 109366: 95 us with each element stored alone, and 73.)
template <class T, class E, class Value>
__device__ __forceinline__ void write_any(Value value, E* out, int64_t ld, int m0, int rows, int n0, int cols, int lane, int wave,
                                          unsigned char* s0, unsigned char* s1)
{
    constexpr int COLS = T::BN, ROUNDS = T::BM * COLS * 2 > T::STAGE_MAX ? 2 : 1, RW = T::WTM / ROUNDS, IR = T::FM / ROUNDS;
    constexpr int CH = COLS / 8, RPI = 64 / CH, ITERS = T::WAVES_M * RW / RPI / T::WAVES;
    static_assert(ITERS * RPI * T::WAVES == T::WAVES_M * RW, "rows split evenly over the waves");
    const Image<COLS> image{s0, s1};
    const int wm = wave / T::WAVES_N, wn = wave % T::WAVES_N;
#pragma unroll
    for (int h = 0; h < ROUNDS; ++h) {
        const int ln = pinned(lane);
#pragma unroll
        for (int i = 0; i < IR; ++i)
#pragma unroll
            for (int j = 0; j < T::FN; ++j)
                image.put(wm * RW + i * 16 + (ln & 15), wn * T::WTN + j * 16 + 4 * (ln >> 4), value(h * IR + i, j));
        lds_barrier<63>();
        const int ch = ln % CH, n = n0 + ch * 8;
        for (int it = 0; it < ITERS; ++it) {
            const int x = (wave * ITERS + it) * RPI + ln / CH, row = m0 + x / RW * T::WTM + h * RW + x % RW;
            if (row < rows && n < cols)
                ::rows::store<E, 8>(out + row * ld + n, cols - n, __builtin_bit_cast(::rows::Vec<E, 8>, image.get(x, ch)));
        }
        lds_barrier<63>();
    }
}

// The last piece's: dX[t] = back[t] (A B^T and, MORE, the sums of the pieces before),
// rounded.  EIGHTS: dX's rows take 16-byte pieces and hold a multiple of eight.
template <class E, bool TURNED, bool EIGHTS, bool MORE>
struct DxOp : AddOp<E, TURNED> {
    using Base = AddOp<E, TURNED>;
    E* dX;
    const float* back;
    int ldx, pad;

    template <class T>
    __device__ __forceinline__ void epilogue(const Tile& t, const f32x4 (&acc)[T::FM][T::FN], int lane, int wave, unsigned char* s0,
                                             unsigned char* s1) const
    {
        const int ln = pinned(lane), M = Base::M, N = Base::N;
        const int bm = (t.m0 + wave / T::WAVES_N * T::WTM) / 16, bn = (t.n0 + wave % T::WAVES_N * T::WTN) / 16;
        const int rows = (M + 15) / 16 - bm, cols = (N + 15) / 16, left = max(cols - bn, 0);
        float g[T::FM];
#pragma unroll
        for (int i = 0; i < T::FM; ++i) g[i] = back[(bm + i) * 16 + (ln & 15)];
        f32x4 old[T::FN];
        auto value = [&](int i, int j) __attribute__((always_inline)) {
            if constexpr (MORE)
                if (j == 0) {
                    const float* const at = Base::sums + ((int64_t)(bm + i) * cols + bn) * kBlockFloats;
                    const __amdgpu_buffer_rsrc_t from = make_rsrc(at, i < rows ? (uint32_t)left * (kBlockFloats * 4u) : 0u);
#pragma unroll
                    for (int k = 0; k < T::FN; ++k)
                        old[k] = __builtin_bit_cast(
                            f32x4, __builtin_amdgcn_raw_buffer_load_b128(from, ln * 16 + k * (kBlockFloats * 4), 0, 0));
                }
            const f32x4 v = EIGHTS ? acc[i][j] : read<T>(acc[i][j]);
            return round4<E>((MORE ? v + old[j] : v) * g[i]);
        };
        if constexpr (EIGHTS)
            write_rows<T, T::FN, true>(value, rows_at(dX, t.m0, M, T::BM, ldx, t.n0, N), lane, wave, s0, s1);
        else
            write_any<T>(value, dX, ldx, t.m0, M, t.n0, N, lane, wave, s0, s1);
    }
};

// A piece's rows of dW where StoreOp would store each element alone.
template <class E>
struct DwOp : StoreOp<E, false, true> {
    using Base = StoreOp<E, false, true>;
    template <class T>
    __device__ __forceinline__ void epilogue(const Tile& t, const f32x4 (&acc)[T::FM][T::FN], int lane, int wave, unsigned char* s0,
                                             unsigned char* s1) const
    {
        const float f = *Base::factor;
        auto value = [&](int i, int j) __attribute__((always_inline)) { return round4<E>(read<T>(acc[i][j]) * f); };
        write_any<T>(value, Base::C[0], Base::ldc[0], t.m0, Base::M, t.n0, Base::N, lane, wave, s0, s1);
    }
};

// ------------------------------------------------------------------ host --

bool vec8(const void* p, int64_t ld) { return (uintptr_t)p % 16 == 0 && ld % 8 == 0; }

// Rows of what is copied, transposed or kept start on 128 bytes, and are written and
// read in whole cache lines.  (Copies of rows that start on 16 bytes: steps of 4000 x
// 4001 x 32001 3520 us, and 3217; 181 x 333 x 109366 332 and 322.)
constexpr int64_t kLine = 64;

// A product over n columns of the vocabulary (by `other` rows, sums of K) may be
// made in two: whole waves of 256 x 256 tiles first, the rest in tiles that leave
// fewer CUs idle.  Returns the first one's columns, n if one is better: the
// model's times and 4 us for the launch.  (Steps of 2048 x 2048 x 50001, 1568
// tiles for 256 CUs: 1593 us in one and 1555 in two; 1000 x 768 x 50001 471 and 448.)
template <class OP>
int64_t first_of_two(int64_t other, int64_t n, int64_t K, bool partial)
{
    auto tiles = [=](int64_t m) { return [=](const Kind& k) { return (other + k.bm - 1) / k.bm * ((m + k.bn - 1) / k.bn); }; };
    const int cus = num_cus();
    const int64_t strip = (other + 255) / 256, waves = strip * ((n + 255) / 256) / cus, first = waves * cus / strip * 256;
    if (K <= 128 || first == 0 || first >= n) return n;
    const Choice one = choose<OP>(K, partial, tiles(n)), rest = choose<OP>(K, partial, tiles(n - first));
    return model_us(kKinds[0], waves * cus, K, cus) + rest.us + 4.0 < one.us ? first : n;
}

// Whether dX's product over n rows of W reads them as they lie: not in 256 x 256 tiles,
// which are faster, but without the transpose, whose bytes cross memory twice (once
// where W is copied anyway).  (Steps with it and without: 17 x 4096 x 20000 256 us and
// 163, 200 x 1024 x 32000 127 and 108, 1000 x 1032 x 32001 394 and 340, 2048 x 2048 x
// 32000 975 and 909, 8192 x 1024 x 50000 3410 and 3290; 8192 x 4096 x 32768, in 256 x 256
// tiles, 6000 and 6330.)  Which of the two a workspace has to hold too, and so by an
// MI355X's CUs, whatever device is current.
template <class E>
bool turned_for(int64_t T, int64_t n, int64_t D, bool copied)
{
    auto tiles = [=](const Kind& k) { return (T + k.bm - 1) / k.bm * ((D + k.bn - 1) / k.bn); };
    const int64_t K = abi::up(n, 8);
    const bool split = K >= kSplitK;
    const double transpose = 2.0 * n * D * (copied ? 1 : 2) / 4.9e6;
    return choose<AddOp<E, true>>(K, split, tiles, cus::kCus).us < choose<AddOp<E, false>>(K, split, tiles, cus::kCus).us + transpose;
}

// The parts of up to this many outputs may be of 32 columns, of more 64 at least
// (which leaves out the smaller tiles): 8 bytes each.
constexpr int64_t kSmall = (int64_t)1 << 26;
int64_t part_width(int64_t T, int64_t V) { return T <= kSmall / V ? 32 : 64; }

bool in_place(const void* p, int64_t D, int64_t ld) { return D % 8 == 0 && vec8(p, ld); }
// X, which every tile of the vocabulary reads anew, is copied to whole lines too where
// the products are large.  (Steps of 2000 x 1496 x 32001 848 us in place and 827,
// 8192 x 1000 x 50000 3520 and 3405; forward alone 6000 x 2632 x 4000 148 and 138, but
// 1000 x 520 x 60001 97 and 102.  W's copy costs more than it gives: 2000 x 1496 x 32001
// forward 185 and 220.)
bool in_place(const void* X, int64_t T, int64_t D, int64_t V, int64_t ldx)
{
    const bool lines = (uintptr_t)X % 128 == 0 && ldx % kLine == 0;
    return in_place(X, D, ldx) && (lines || (double)T * (double)D * (double)V < 6e10);
}

template <class E>
struct ForwardSpace {
    E *x = nullptr, *w = nullptr;  // null: read in place
    float *tl, *partial = nullptr;
    f32x2* parts;
    int64_t Mp, bytes;
    ForwardSpace(void* base, const void* X, const void* W, int64_t T, int64_t D, int64_t V, int64_t ldx, int64_t ldw)
    {
        abi::Carve c(base);
        tl = c.take<float>(T);
        if (T <= few::kTokens) {
            Mp = few::kTokens;
            parts = c.take<f32x2>((V + few::kRows - 1) / few::kRows * Mp);
        } else {
            const int64_t ld = abi::up(D, kLine), width = part_width(T, V);
            Mp = abi::up(T, 16);
            if (!in_place(X, T, D, V, ldx)) x = c.take<E>(T * ld);
            if (!in_place(W, D, ldw)) w = c.take<E>(V * ld);
            parts = c.take<f32x2>(((V + width - 1) / width + 1) * Mp);
            if (abi::up(D, 8) >= kSplitK) partial = c.take<float>(kSplitFloats);
        }
        bytes = T ? c.used() : 0;
    }
};

// Rows to a workgroup: 8, or from 2048 on 32, whose parts lie in two whole cache lines,
// not in half of one.  (The loss of D 64 by 131072 words: 1000 tokens 94.7 us with 8 and 98.6
// with 32, 1500 136 and 137, 2048 178 and 176, 6000 506 and 492; 8192 by 50000 273 and 264.)
int join(const Join& j, hipStream_t stream)
{
    auto with = [&](auto kernel, int64_t rows) {
        hipLaunchKernelGGL(kernel, dim3((unsigned)((j.M + rows - 1) / rows)), dim3(kJoin), 0, stream, j);
        return (int)hipGetLastError();
    };
    if (j.M <= few::kTokens) return with(lse_join<1>, 1);
    return j.M < 2048 ? with(lse_join<8>, 8) : with(lse_join<32>, 32);
}

template <class E>
int forward(const E* X, const E* W, const int64_t* target, float* loss, float* saved, int64_t T, int64_t D, int64_t V, int64_t ldx,
            int64_t ldw, int64_t target_stride, int64_t ignore, void* workspace, hipStream_t stream)
{
    const ForwardSpace<E> w(workspace, X, W, T, D, V, ldx, ldw);
    Join j = {w.parts, target, w.tl, loss, saved, target_stride, ignore, w.Mp, (int)T, (int)V, 0};
    int rc;
    if (T <= few::kTokens) {
        const few::Lse<E> f = {X, W, target, w.tl, w.parts, target_stride, ldx, ldw, (int)T, (int)D, (int)V};
        const int64_t n = 16 * few::blocks_of(V);
        j.segments = (int)((V + n - 1) / n);
        hipLaunchKernelGGL((n > few::kRows ? few::few_lse<E, 4> : few::few_lse<E, 2>), dim3((unsigned)std::min(j.segments, 1 << 20)),
                           dim3(few::kWaves * kWave), 0, stream, f);
        if ((rc = (int)hipGetLastError())) return rc;
        return join(j, stream);
    }
    const int64_t ld = abi::up(D, kLine);
    Prepare<E> p = {};
    if (w.x) p.x = {X, w.x, nullptr, ldx, ld, 0, (int)T, (int)D};
    if (w.w) p.w = {W, w.w, nullptr, ldw, ld, 0, (int)V, (int)D};
    if ((rc = enqueue(p, false, stream))) return rc;
    LseOp<E> op = {};
    op.X = w.x ? w.x : X;
    op.target = target;
    op.tl = w.tl;
    op.target_stride = target_stride;
    op.Mp = w.Mp;
    op.M = (int)T;
    op.K = (int)abi::up(D, 8);
    op.lda = (int)(w.x ? ld : ldx);
    op.ldb = (int)(w.w ? ld : ldw);
    const int64_t split = first_of_two<LseOp<E>>(T, V, op.K, w.partial);
    for (int64_t v0 = 0; v0 < V; v0 = v0 ? V : split) {
        const int64_t n = v0 ? V - split : split;
        op.W = (w.w ? w.w : W) + v0 * op.ldb;
        op.N = (int)n;
        op.first = (int)v0;
        op.parts = w.parts + j.segments * w.Mp;
        rc = launch<E>(
            op, op.K, w.partial,
            [&](const Kind& k) {
                const bool wide = k.bn == 256 || k.bm == 256;  // (sub-tiles of 64 columns or more)
                if (!wide && part_width(T, V) > 32) return INT64_MAX;
                return (T + k.bm - 1) / k.bm * ((n + k.bn - 1) / k.bn);
            },
            [&](LseOp<E>& o, const Kind& k) {
                o.tiles_m = (int)((T + k.bm - 1) / k.bm);
                o.tiles_n = (int)((n + k.bn - 1) / k.bn);
                const int wtn = k.bn == 256 ? 128 : k.bm == 256 ? 64 : 32;
                j.segments += (int)((n + wtn - 1) / wtn);
            },
            stream);
        if (rc) return rc;
    }
    return join(j, stream);
}

// Columns of the vocabulary to a piece: dl of 2^27 elements, 256 MB, twice, in
// rows of 2^20 at most (a pitch is below 2^21) and 1024 at least, for which more than
// 131072 tokens take more; the pieces alike, of whole tiles.
int64_t piece_of(int64_t T, int64_t V)
{
    const int64_t most = std::min<int64_t>(std::max<int64_t>(((int64_t)1 << 27) / std::max<int64_t>(T, 1), 1024), 1 << 20);
    const int64_t pieces = (V + most - 1) / most;
    return std::min(V, abi::up((V + pieces - 1) / pieces, 256));
}

// Shares of W's rows for few tokens, whose gradients' sums cross memory twice: as
// many workgroups as run at once (32000 x 2048 in 256, 512 and 1024: 1 token by 1024 columns
// 86, 68 and 63 us, 8 tokens 142, 123 and 139).
struct Shares {
    int64_t per, count, chunks;  // rows to a share, shares, pieces of D
    Shares(int64_t T, int64_t D, int64_t V)
    {
        const int64_t columns = few::kGradThreads * (T <= 8 ? 8 : 4);
        chunks = std::max<int64_t>((D + columns - 1) / columns, 1);
        const int64_t most = std::max<int64_t>((T <= 4 ? 4 : 2) * cus::kCus / chunks, 1);
        per = abi::up((V + most - 1) / most, 4);
        count = (V + per - 1) / per;
    }
};

template <class E>
struct BackwardSpace {
    E *x = nullptr, *w = nullptr;  // null: read in place
    E *xt, *wt = nullptr, *dl, *dlt;
    RowInfo* info;
    int* column;
    float *back, *sums, *factor, *partial;
    int64_t Tp, Vp, piece, rows, bytes;
    BackwardSpace(void* base, const void* X, const void* W, int64_t T, int64_t D, int64_t V, int64_t ldx, int64_t ldw)
    {
        abi::Carve c(base);
        if (T > 0 && T <= few::kTokens) {
            sums = c.take<float>(V * few::kTokens);  // dl
            partial = c.take<float>(Shares(T, D, V).count * T * D);
            bytes = c.used();
            return;
        }
        const int64_t ld = abi::up(D, kLine);
        piece = piece_of(T, V);
        Tp = abi::up(T, kLine);
        Vp = abi::up(piece, kLine);
        rows = abi::up(T, 256);
        if (!in_place(X, T, D, V, ldx)) x = c.take<E>(T * ld);
        const bool products = T > 0 && D > 0, copied = products && !in_place(W, D, ldw);  // W is read, copied first
        if (copied) w = c.take<E>(piece * ld);
        xt = c.take<E>(D * Tp);
        // (the last piece's rows of W may be fewer, and read the other way)
        const int64_t last = V - (V - 1) / piece * piece;
        if (products && !(turned_for<E>(T, piece, D, copied) && (last == piece || turned_for<E>(T, last, D, copied))))
            wt = c.take<E>(D * Vp);
        dl = c.take<E>(T * Vp);
        dlt = c.take<E>(piece * Tp);
        info = c.take<RowInfo>(rows);
        column = c.take<int>(rows);
        back = c.take<float>(rows);
        sums = piece < V ? c.take<float>((T + 15) / 16 * ((D + 15) / 16) * kBlockFloats) : nullptr;
        factor = c.take<float>(1);
        partial = T ? c.take<float>(kSplitFloats) : nullptr;
        bytes = c.used();
    }
};

template <class E>
int backward_few(const float* dloss, const E* X, const E* W, const int64_t* target, const float* saved, E* dX, E* dW, int64_t T,
                 int64_t D, int64_t V, int64_t dloss_stride, int64_t ldx, int64_t ldw, int64_t target_stride, int64_t lddx,
                 int64_t lddw, int64_t ignore, const BackwardSpace<E>& w, hipStream_t stream)
{
    if (D == 0) return hipSuccess;
    const few::Dl<E> d = {X, W, target, dloss, saved, w.sums, target_stride, dloss_stride, ignore, ldx, ldw, (int)T, (int)D, (int)V};
    const int64_t n = 16 * few::blocks_of(V), blocks = (V + n - 1) / n;
    hipLaunchKernelGGL((n > few::kRows ? few::few_dl<E, 4> : few::few_dl<E, 2>), dim3((unsigned)std::min<int64_t>(blocks, 1 << 20)),
                       dim3(few::kWaves * kWave), 0, stream, d);
    int rc = (int)hipGetLastError();
    if (rc) return rc;
    const Shares s(T, D, V);
    const few::Grads<E> g = {X,      W,   target, w.sums, dW,     w.partial, target_stride, ignore,
                             ldx,    ldw, lddw,   (int)T, (int)D, (int)V,    (int)s.per};
    auto with = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3((unsigned)s.count, (unsigned)s.chunks), dim3(few::kGradThreads), 0, stream, g);
        return (int)hipGetLastError();
    };
    if (T == 1) rc = with(few::few_grads<E, 1, 8>);
    else if (T <= 4) rc = with(few::few_grads<E, 4, 8>);
    else if (T <= 8) rc = with(few::few_grads<E, 8, 8>);
    else rc = with(few::few_grads<E, 16, 4>);
    if (rc) return rc;
    const few::Sum<E> sum = {w.partial, target, dX, target_stride, ignore, lddx, (int)T, (int)D, (int)s.count};
    const bool wide = rows::wide_sums(D, T);
    const int64_t columns = wide ? 64 : 16;
    hipLaunchKernelGGL((wide ? few::few_sum<E, 64> : few::few_sum<E, 16>), dim3((unsigned)((D + columns - 1) / columns), (unsigned)T),
                       dim3(rows::kSumThreads), 0, stream, sum);
    return (int)hipGetLastError();
}

template <class E>
int backward(const float* dloss, const E* X, const E* W, const int64_t* target, const float* saved, E* dX, E* dW, int64_t T,
             int64_t D, int64_t V, int64_t dloss_stride, int64_t ldx, int64_t ldw, int64_t target_stride, int64_t lddx,
             int64_t lddw, int64_t ignore, void* workspace, hipStream_t stream)
{
    const BackwardSpace<E> w(workspace, X, W, T, D, V, ldx, ldw);
    if (T > 0 && T <= few::kTokens)
        return backward_few<E>(dloss, X, W, target, saved, dX, dW, T, D, V, dloss_stride, ldx, ldw, target_stride, lddx, lddw,
                               ignore, w, stream);
    int rc;
    const int64_t ld = abi::up(D, kLine);
    for (int64_t v0 = 0; v0 < V; v0 += w.piece) {
        const int64_t n = std::min(w.piece, V - v0);
        const E* const W0 = W + v0 * ldw;
        Prepare<E> p = {};
        if (v0 == 0) {
            p.numbers = {dloss,  saved,       target, dloss_stride, target_stride, ignore,  (int)T,
                         (int)w.rows, (int)V, w.info, w.column,     w.back,        w.factor};
            p.x = {X, w.x, w.xt, ldx, ld, w.Tp, (int)T, (int)D, target, target_stride, ignore};
        }
        const bool turned = D > 0 && turned_for<E>(T, n, D, w.w != nullptr);
        if (T > 0) p.w = {W0, w.w, turned ? nullptr : w.wt, ldw, ld, w.Vp, (int)n, (int)D};
        if ((rc = enqueue(p, v0 == 0, stream))) return rc;
        if (T > 0) {
            DlOp<E> op = {};
            op.X = w.x ? w.x : X;
            op.info = w.info;
            op.column = w.column;
            op.M = (int)T;
            op.K = (int)abi::up(D, 8);
            op.lda = (int)(w.x ? ld : ldx);
            op.ldb = (int)(w.w ? ld : ldw);
            op.ldd = (int)w.Vp;
            op.ldt = (int)w.Tp;
            const int64_t split = first_of_two<DlOp<E>>(T, n, op.K, false);
            for (int64_t c = 0; c < n; c = c ? n : split) {
                op.W = (w.w ? w.w : W0) + c * op.ldb;
                op.dl = w.dl + c;
                op.dlt = w.dlt + c * w.Tp;
                op.first = (int)(v0 + c);
                op.N = (int)(c ? n - split : split);
                if ((rc = launch_grid<E>(op, T, op.N, 1, 1, op.K, nullptr, stream))) return rc;
            }
            if (D > 0) {
                auto product = [&](auto op) {
                    op.A = w.dl;
                    op.B = !turned ? w.wt : w.w ? w.w : W0;
                    op.sums = w.sums;
                    op.M = (int)T;
                    op.N = (int)D;
                    op.K = (int)abi::up(n, 8);
                    op.lda = (int)w.Vp;
                    op.ldb = (int)(!turned ? w.Vp : w.w ? ld : ldw);
                    op.there = (int)n;
                    op.fresh = v0 == 0;
                    return launch_grid<E>(op, T, D, 1, 1, op.K, op.K >= kSplitK ? w.partial : nullptr, stream);
                };
                auto last = [&](auto op) {
                    op.dX = dX;
                    op.back = w.back;
                    op.ldx = (int)lddx;
                    return product(op);
                };
                const bool eights = vec8(dX, lddx) && D % 8 == 0;
                auto either = [&](auto t) {
                    constexpr bool TURNED = decltype(t)::value;
                    if (v0 + n < V) return product(AddOp<E, TURNED>{});
                    if (v0 == 0) return eights ? last(DxOp<E, TURNED, true, false>{}) : last(DxOp<E, TURNED, false, false>{});
                    return eights ? last(DxOp<E, TURNED, true, true>{}) : last(DxOp<E, TURNED, false, true>{});
                };
                rc = turned ? either(Flag<true>{}) : either(Flag<false>{});
                if (rc) return rc;
            }
        }
        if (D > 0) {
            auto product = [&](auto op) {
                op.factor = w.factor;
                op.B = w.xt;
                op.N = (int)D;
                op.K = (int)abi::up(T, 8);
                op.lda = op.ldb = (int)w.Tp;
                op.ldc[0] = (int)lddw;
                float* const partial = op.K >= kSplitK ? w.partial : nullptr;
                const int64_t split = first_of_two<decltype(op)>(D, n, op.K, partial);
                for (int64_t c = 0; c < n; c = c ? n : split) {
                    op.A[0] = w.dlt + c * w.Tp;
                    op.C[0] = dW + (v0 + c) * lddw;
                    op.M = (int)(c ? n - split : split);
                    if ((rc = launch_grid<E>(op, op.M, D, 1, 1, op.K, partial, stream))) return rc;
                }
                return (int)hipSuccess;
            };
            const bool eights = vec8(dW, lddw) && D % 8 == 0;
            rc = eights ? product(StoreOp<E, true, true>{}) : product(DwOp<E>{});
            if (rc) return rc;
        }
    }
    return hipSuccess;
}

bool good_sizes(int64_t T, int64_t D, int64_t V)
{
    return T >= 0 && T <= (int64_t)1 << 27 && D >= 0 && D <= abi::kMaxPitch - 63 && V > 0 && V <= abi::kMaxDim - 256;
}
bool good_backward_sizes(int64_t T, int64_t D, int64_t V) { return good_sizes(T, D, V) && T <= abi::kMaxPitch - 63; }
// Workgroups that lay out X and V rows of W, and the one beside them.
int64_t layout_tiles(int64_t T, int64_t D, int64_t V) { return ((T + 63) / 64 + (V + 63) / 64) * ((D + 63) / 64) + 1; }
bool good_stride(int64_t s) { return s >= 0 && s <= (int64_t)1 << 31; }

}  // namespace

extern "C" {

int linear_cross_entropy_version(void) { return LINEAR_CROSS_ENTROPY_VERSION; }

int64_t linear_cross_entropy_workspace(const void* X, const void* W, int64_t T, int64_t D, int64_t V, int64_t ldx, int64_t ldw)
{
    if (!good_sizes(T, D, V)) return -1;
    return ForwardSpace<_Float16>(nullptr, X, W, T, D, V, ldx, ldw).bytes;
}

int64_t linear_cross_entropy_backward_workspace(const void* X, const void* W, int64_t T, int64_t D, int64_t V, int64_t ldx, int64_t ldw)
{
    if (!good_backward_sizes(T, D, V)) return -1;
    return BackwardSpace<_Float16>(nullptr, X, W, T, D, V, ldx, ldw).bytes;
}

int linear_cross_entropy(const void* X, const void* W, const int64_t* target, float* loss, float* saved, int64_t T, int64_t D, int64_t V,
                         int64_t ldx, int64_t ldw, int64_t target_stride, int32_t type, int64_t ignore_index, void* workspace,
                         int64_t workspace_bytes, hipStream_t stream)
{
    using namespace abi;
    if (!good_sizes(T, D, V) || !good_pitch(ldx, D) || !good_pitch(ldw, D) || !good_stride(target_stride)) return hipErrorInvalidValue;
    if (type != LINEAR_CROSS_ENTROPY_F16 && type != LINEAR_CROSS_ENTROPY_BF16) return hipErrorInvalidValue;
    if (T == 0) return hipSuccess;
    if (!nt::fits(T, V, 1) || !good_grid(layout_tiles(T, D, V), relayout::kThreads)) return hipErrorInvalidValue;
    if (!good_pointer(X, T, D, 2) || !good_pointer(W, V, D, 2) || !good_pointer(target, T, 1, 8) || !good_pointer(loss, T, 1, 4) ||
        (uintptr_t)saved % 4 || (uintptr_t)workspace % 16)
        return hipErrorInvalidValue;
    const int64_t need = linear_cross_entropy_workspace(X, W, T, D, V, ldx, ldw);
    if (!workspace || workspace_bytes < need) return hipErrorInvalidValue;
    const Range in[] = {Range(X, T, D, ldx, 2), Range(W, V, D, ldw, 2), Range(target, T, 1, target_stride, 8)};
    const Range out[] = {Range(loss, 1, T, 0, 4), Range(saved, 1, saved ? 3 * T : 0, 0, 4), Range(workspace, 1, need, 0, 1)};
    for (int i = 0; i < 3; ++i) {
        for (const Range& r : in)
            if (out[i].meets(r)) return hipErrorInvalidValue;
        for (int k = 0; k < i; ++k)
            if (out[i].meets(out[k])) return hipErrorInvalidValue;
    }
#define FORWARD(E) \
    forward<E>((const E*)X, (const E*)W, target, loss, saved, T, D, V, ldx, ldw, target_stride, ignore_index, workspace, stream)
    return type == LINEAR_CROSS_ENTROPY_F16 ? FORWARD(_Float16) : FORWARD(__bf16);
#undef FORWARD
}

int linear_cross_entropy_backward(const float* dloss, const void* X, const void* W, const int64_t* target, const float* saved, void* dX,
                                  void* dW, int64_t T, int64_t D, int64_t V, int64_t dloss_stride, int64_t ldx, int64_t ldw,
                                  int64_t target_stride, int64_t lddx, int64_t lddw, int32_t type, int64_t ignore_index, void* workspace,
                                  int64_t workspace_bytes, hipStream_t stream)
{
    using namespace abi;
    if (!good_backward_sizes(T, D, V) || !good_pitch(ldx, D) || !good_pitch(ldw, D) || !good_pitch(lddx, D) || !good_pitch(lddw, D) ||
        !good_stride(target_stride) || !good_stride(dloss_stride))
        return hipErrorInvalidValue;
    if (type != LINEAR_CROSS_ENTROPY_F16 && type != LINEAR_CROSS_ENTROPY_BF16) return hipErrorInvalidValue;
    if (!nt::fits(T, piece_of(T, V), 1) || !nt::fits(T, D, 1) || !nt::fits(piece_of(T, V), D, 1)) return hipErrorInvalidValue;
    if (!good_grid(layout_tiles(T, D, piece_of(T, V)), relayout::kThreads)) return hipErrorInvalidValue;
    if (!good_pointer(dloss, T, 1, 4) || !good_pointer(X, T, D, 2) || !good_pointer(W, V, D, 2) || !good_pointer(target, T, 1, 8) ||
        !good_pointer(saved, T, 1, 4) || !good_pointer(dX, T, D, 2) || !good_pointer(dW, V, D, 2) || (uintptr_t)workspace % 16)
        return hipErrorInvalidValue;
    const int64_t need = linear_cross_entropy_backward_workspace(X, W, T, D, V, ldx, ldw);
    if (!workspace || workspace_bytes < need) return hipErrorInvalidValue;
    const Range in[] = {Range(dloss, T, 1, dloss_stride, 4), Range(X, T, D, ldx, 2), Range(W, V, D, ldw, 2),
                        Range(target, T, 1, target_stride, 8), Range(saved, 1, 3 * T, 0, 4)};
    const Range out[] = {Range(dX, T, D, lddx, 2), Range(dW, V, D, lddw, 2), Range(workspace, 1, need, 0, 1)};
    for (int i = 0; i < 3; ++i) {
        for (const Range& r : in)
            if (out[i].meets(r)) return hipErrorInvalidValue;
        for (int k = 0; k < i; ++k)
            if (out[i].meets(out[k])) return hipErrorInvalidValue;
    }
#define BACKWARD(E)                                                                                                                  \
    backward<E>(dloss, (const E*)X, (const E*)W, target, saved, (E*)dX, (E*)dW, T, D, V, dloss_stride, ldx, ldw, target_stride, lddx, \
                lddw, ignore_index, workspace, stream)
    return type == LINEAR_CROSS_ENTROPY_F16 ? BACKWARD(_Float16) : BACKWARD(__bf16);
#undef BACKWARD
}

}  // extern "C"
