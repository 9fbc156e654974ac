// The layer norm of a matrix's rows and its backward pass for gfx950:
// include/layer_norm.h.
//
// Both passes are bound by their bytes: a row is read once, held in registers
// (as it came, in its type) through its sums, and written once.  8192 x 4096 in
// bfloat16: 29 us forward, 4.6 TB/s, and 35 backward, 5.8.  Rows that registers do not
// hold are read again: backward above 2048 chunks of 16 bytes x and dy twice (3000 x
// 16384 in bfloat16 74 us, 20000 118; in binary32 8192 62, 12000 142), forward above 4096.
#include "layer_norm.h"

#include <algorithm>
#include <type_traits>

#include "abi.h"
#include "cus.h"
#include "rows.h"

namespace {

using namespace rows;

// Chunk i of a lane is number i * G + lane of its row: adjacent lanes take
// adjacent chunks.
template <class E, class P>
struct Forward {
    const E* X;
    const P *weight, *bias;  // null: 1 and 0
    E* Y;
    float* saved;  // null: not kept
    int64_t ldx, ldy;
    int rows, cols;
    float eps;
};

__device__ __forceinline__ float deviation(float sum, int cols, float eps) { return 1.0f / __builtin_sqrtf(sum / (float)cols + eps); }

// The squares of a chunk's distances from the mean.  Only a row's last chunk
// may have elements that are not there: those lanes take the other way.  (`left`
// is new to the compiler each time: it would keep the comparisons through the
// rows, in more scalar registers than there are.)
template <class E, int N>
__device__ __forceinline__ float squares(const Vec<E, N>& v, float mean, int left, float sum)
{
    if (left >= N) {
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const float d = (float)v[e] - mean;
            sum = __builtin_fmaf(d, d, sum);
        }
    } else {
        asm volatile("" : "+v"(left));
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const float d = e < left ? (float)v[e] - mean : 0.0f;
            sum = __builtin_fmaf(d, d, sum);
        }
    }
    return sum;
}

// Where a lane's chunk `n` of a row lies.  The last one, where a row is no whole
// number of chunks, moves back to end with the row: it holds some elements that
// the chunk before holds too, which count once in the row's sums; whatever is
// computed of each is computed twice alike and stored twice.  (Loaded and stored one
// by one the row's last elements make their wave wait, and all others for it: steps
// of 1000 x 2731 in binary16 take 30 us and so 26, 20000 x 3003 212 and 161, 20000 x
// 301 in binary32 41 and 33.)  A row shorter than a chunk is loaded one by one: G of
// 8 and C of 1 alone (SHORT).  WHOLE: rows are whole chunks, and nothing else is
// there (steps of 2048 x 8192 in bfloat16 50.3 us and 48.5).
// (`twice` is new to the compiler each time: it would keep the comparisons through
// the rows, in more scalar registers than there are.)
template <int N, int G, int C, bool WHOLE>
struct Place {
    static constexpr bool SHORT = !WHOLE && G == 8 && C == 1;
    int c, twice, cols;  // the first element, how many the chunk before has too
    bool ends;           // a row may end here: in the second half of a lane's chunks
    __device__ __forceinline__ Place(int i, int lane, int cols_)
        : c((i * G + lane) * N), twice(0), cols(cols_), ends(!WHOLE && 2 * i + 1 >= C)
    {
        if (ends) {
            if (c < cols && c + N > cols && (!SHORT || cols >= N)) {
                twice = c + N - cols;
                c = cols - N;
            }
            asm volatile("" : "+v"(twice));
        }
    }
    __device__ __forceinline__ bool there() const { return c < cols; }
    __device__ __forceinline__ int left() const { return SHORT ? cols - c : N; }
    // whether element e counts in the row's sums
    __device__ __forceinline__ bool counts(int e) const { return !ends || (e >= twice && (!SHORT || e < cols - c)); }
};

// weight and bias of a chunk.
template <class P, int N>
__device__ __forceinline__ void load_params(const P* weight, const P* bias, int c, int left, Vec<P, N>& w, Vec<P, N>& b)
{
    w = (P)1.0f;
    b = (P)0.0f;
    if (left > 0 && weight) w = load<P, N>(weight + c, left);
    if (left > 0 && bias) b = load<P, N>(bias + c, left);
}

// Rows of up to G * C chunks, G lanes to a row; G below 64: several rows to a wave.
// Lanes with few chunks keep weight and bias for all their rows.
template <class E, class P, int G, int C, bool WHOLE>
__global__ void __launch_bounds__(G > 256 ? G : 256) norm_rows(const Forward<E, P> f)
{
    constexpr int N = kChunk<E>, R = (G > 256 ? G : 256) / G;
    constexpr bool KEEP = C <= 2;
    using At = Place<N, G, C, WHOLE>;
    __shared__ Parts<G, 1> parts;
    const int lane = threadIdx.x % G, mine = threadIdx.x / G, cols = f.cols;
    Vec<P, N> kw[KEEP ? C : 1], kb[KEEP ? C : 1];
    if constexpr (KEEP)
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const At at(i, lane, cols);
            load_params<P, N>(f.weight, f.bias, at.c, at.there() ? at.left() : 0, kw[i], kb[i]);
        }
    for (int64_t first = (int64_t)blockIdx.x * R; first < f.rows; first += (int64_t)gridDim.x * R) {
        const int64_t row = first + mine;
        const bool there = row < f.rows;
        Vec<E, N> v[C];
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const At at(i, lane, cols);
            v[i] = Vec<E, N>{};
            if (there && at.there()) v[i] = load<E, N>(f.X + row * f.ldx + at.c, at.left());
        }
        float s[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const At at(i, lane, cols);
#pragma unroll
            for (int e = 0; e < N; ++e) s[0] += at.counts(e) ? (float)v[i][e] : 0.0f;
        }
        sums<G, 1>(s, parts, 0);
        const float mean = s[0] / (float)cols;
        s[0] = 0.0f;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const At at(i, lane, cols);
            if (!at.there()) continue;
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const float d = at.counts(e) ? (float)v[i][e] - mean : 0.0f;
                s[0] = __builtin_fmaf(d, d, s[0]);
            }
        }
        sums<G, 1>(s, parts, 1);
        const float r = deviation(s[0], cols, f.eps);
        if (there && f.saved && lane == 0) {
            f.saved[2 * row] = mean;
            f.saved[2 * row + 1] = r;
        }
        E* y = f.Y + row * f.ldy;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const At at(i, lane, cols);
            Vec<P, N> w, b;
            if constexpr (KEEP) {
                w = kw[i];
                b = kb[i];
            } else {
                load_params<P, N>(f.weight, f.bias, at.c, at.there() ? at.left() : 0, w, b);
            }
            Vec<E, N> o;
#pragma unroll
            for (int e = 0; e < N; ++e) o[e] = (E)__builtin_fmaf(((float)v[i][e] - mean) * r, (float)w[e], (float)b[e]);
            if (there && at.there()) store<E, N>(y + at.c, at.left(), o);
        }
    }
}

// Rows of any length, a workgroup to a row that is read three times.
constexpr int kWide = 1024;

template <class E, class P>
__global__ void __launch_bounds__(kWide) norm_wide(const Forward<E, P> f)
{
    constexpr int N = kChunk<E>;
    __shared__ Parts<kWide, 1> parts;
    const int cols = f.cols;
    for (int64_t row = blockIdx.x; row < f.rows; row += gridDim.x) {
        const E* x = f.X + row * f.ldx;
        E* y = f.Y + row * f.ldy;
        float s[1] = {0.0f};
        for (int64_t c = (int64_t)threadIdx.x * N; c < cols; c += kWide * N) {
            const Vec<E, N> v = load<E, N>(x + c, cols - (int)c);
#pragma unroll
            for (int e = 0; e < N; ++e) s[0] += (float)v[e];
        }
        sums<kWide, 1>(s, parts, 0);
        const float mean = s[0] / (float)cols;
        s[0] = 0.0f;
        for (int64_t c = (int64_t)threadIdx.x * N; c < cols; c += kWide * N) {
            const Vec<E, N> v = load<E, N>(x + c, cols - (int)c);
            s[0] = squares<E, N>(v, mean, cols - (int)c, s[0]);
        }
        sums<kWide, 1>(s, parts, 1);
        const float r = deviation(s[0], cols, f.eps);
        if (f.saved && threadIdx.x == 0) {
            f.saved[2 * row] = mean;
            f.saved[2 * row + 1] = r;
        }
        for (int64_t c = (int64_t)threadIdx.x * N; c < cols; c += kWide * N) {
            const int left = cols - (int)c;
            const Vec<E, N> v = load<E, N>(x + c, left);
            Vec<P, N> w, b;
            load_params<P, N>(f.weight, f.bias, (int)c, left, w, b);
            Vec<E, N> o;
#pragma unroll
            for (int e = 0; e < N; ++e) o[e] = (E)__builtin_fmaf(((float)v[e] - mean) * r, (float)w[e], (float)b[e]);
            store<E, N>(y + c, left, o);
        }
    }
}

// Rows of sums start on cache lines.  (8192 x 4095: adding them up, 16 to a workgroup, 8.9 us, and 7.2.)
__host__ __device__ inline int64_t sum_pitch(int64_t cols) { return (cols + 31) / 32 * 32; }

template <class E, class P>
struct Backward {
    const E *dY, *X;
    const P* weight;
    const float* saved;
    E* dX;
    float* partial;  // [workgroups][2][sum_pitch(cols)]: sums of dY h and of dY; null: none
    P *dweight, *dbias;  // one workgroup's (null: not wanted)
    int64_t lddy, ldx, lddx;
    int rows, cols;
};

// Rows of up to G * C chunks: dX, and each workgroup's sums over its rows.  The
// next row's loads are in flight while a row is worked on, where registers allow.
template <class E, class P, int G, int C, bool WHOLE>
__global__ void __launch_bounds__(G > 256 ? G : 256) norm_back_rows(const Backward<E, P> f)
{
    constexpr int N = kChunk<E>, T = G > 256 ? G : 256, R = T / G;
    constexpr bool AHEAD = C * N < 32;
    using At = Place<N, G, C, WHOLE>;
    __shared__ Parts<G, 2> parts;
    __shared__ float meet[R > 1 ? R * G * C * N : 1];
    const int lane = threadIdx.x % G, mine = threadIdx.x / G, cols = f.cols;
    const int64_t step = (int64_t)gridDim.x * R;
    Vec<P, N> w[C];
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const At at(i, lane, cols);
        w[i] = (P)1.0f;
        if (at.there() && f.weight) w[i] = load<P, N>(f.weight + at.c, at.left());
    }
    float aw[C][N], ab[C][N];
#pragma unroll
    for (int i = 0; i < C; ++i)
#pragma unroll
        for (int e = 0; e < N; ++e) aw[i][e] = ab[i][e] = 0.0f;

    struct Row {
        Vec<E, N> x[C], d[C];
        float mean, r;
    };
    auto fetch = [&](int64_t row) __attribute__((always_inline)) {
        Row v;
        const bool there = row < f.rows;
        v.mean = there ? f.saved[2 * row] : 0.0f;
        v.r = there ? f.saved[2 * row + 1] : 0.0f;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const At at(i, lane, cols);
            v.x[i] = Vec<E, N>{};
            v.d[i] = Vec<E, N>{};
            if (there && at.there()) {
                v.x[i] = load<E, N>(f.X + row * f.ldx + at.c, at.left());
                v.d[i] = load<E, N>(f.dY + row * f.lddy + at.c, at.left());
            }
        }
        return v;
    };
    int turn = 0;
    int64_t first = (int64_t)blockIdx.x * R;
    Row next = {};
    if constexpr (AHEAD) next = fetch(first + mine);
    for (; first < f.rows; first += step) {
        const int64_t row = first + mine;
        Row v;
        if constexpr (AHEAD) {
            v = next;
            next = fetch(row + step);
        } else {
            v = fetch(row);
        }
        float s[2] = {0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const At at(i, lane, cols);
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const float h = ((float)v.x[i][e] - v.mean) * v.r, dy = (float)v.d[i][e];
                const float g = at.counts(e) ? dy * (float)w[i][e] : 0.0f;
                s[0] += g;
                s[1] = __builtin_fmaf(g, h, s[1]);
                aw[i][e] = __builtin_fmaf(dy, h, aw[i][e]);
                ab[i][e] += dy;
            }
        }
        sums<G, 2>(s, parts, turn++);
        const float mg = s[0] / (float)cols, mgh = s[1] / (float)cols;
        E* to = f.dX + row * f.lddx;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const At at(i, lane, cols);
            Vec<E, N> o;
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const float h = ((float)v.x[i][e] - v.mean) * v.r, g = (float)v.d[i][e] * (float)w[i][e];
                o[e] = (E)(v.r * (g - mg - h * mgh));
            }
            if (row < f.rows && at.there()) store<E, N>(to + at.c, at.left(), o);
        }
    }
    const int64_t pitch = sum_pitch(cols);
    float* const out = f.partial ? f.partial + (int64_t)blockIdx.x * 2 * pitch : nullptr;
    if (!out && !f.dweight && !f.dbias) return;
    if constexpr (R == 1) {
        // (a lane's chunks whole: one element at a time, which lie apart from lane to
        // lane, 1000 x 2728 takes 13.9 us, and 11.5)
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const At at(i, lane, cols);
            if (!at.there()) continue;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                Vec<float, N> sum;
                Vec<P, N> rounded;
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    sum[e] = k ? ab[i][e] : aw[i][e];
                    rounded[e] = (P)sum[e];
                }
                if (out) store<float, N>(out + k * pitch + at.c, at.left(), sum);
                P* const to = k ? f.dbias : f.dweight;
                if (to) store<P, N>(to + at.c, at.left(), rounded);
            }
        }
    } else {
        // the groups' sums meet in LDS, first those of dY h
        constexpr int W = G * C * N;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < C; ++i) {
                const At at(i, lane, cols);
#pragma unroll
                for (int e = 0; e < N; ++e) meet[mine * W + at.c + e] = k ? ab[i][e] : aw[i][e];
            }
            __syncthreads();
            for (int c = threadIdx.x; c < cols; c += T) {
                float sum = 0.0f;
#pragma unroll
                for (int g = 0; g < R; ++g) sum += meet[g * W + c];
                if (out) out[k * pitch + c] = sum;
                P* const to = k ? f.dbias : f.dweight;
                if (to) to[c] = (P)sum;
            }
        }
    }
}

// Rows of any length: their two means first, a workgroup to a row, then dX and
// the sums of a tile of columns over a share of the rows.
template <class E, class P>
__global__ void __launch_bounds__(kWide) norm_back_means(const Backward<E, P> f, float* means)
{
    constexpr int N = kChunk<E>;
    __shared__ Parts<kWide, 2> parts;
    const int cols = f.cols;
    int turn = 0;
    for (int64_t row = blockIdx.x; row < f.rows; row += gridDim.x) {
        const E *x = f.X + row * f.ldx, *d = f.dY + row * f.lddy;
        const float mean = f.saved[2 * row], r = f.saved[2 * row + 1];
        float s[2] = {0.0f, 0.0f};
        for (int64_t c = (int64_t)threadIdx.x * N; c < cols; c += kWide * N) {
            const int left = cols - (int)c;
            const Vec<E, N> vx = load<E, N>(x + c, left), vd = load<E, N>(d + c, left);
            Vec<P, N> w = (P)1.0f;
            if (f.weight) w = load<P, N>(f.weight + c, left);
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const float g = (float)vd[e] * (float)w[e];
                s[0] += g;
                s[1] = __builtin_fmaf(g, ((float)vx[e] - mean) * r, s[1]);
            }
        }
        sums<kWide, 2>(s, parts, turn++);
        if (threadIdx.x == 0) {
            means[2 * row] = s[0] / (float)cols;
            means[2 * row + 1] = s[1] / (float)cols;
        }
    }
}

constexpr int kTileThreads = 256;

template <class E, class P>
__global__ void __launch_bounds__(kTileThreads) norm_back_tiles(const Backward<E, P> f, const float* means)
{
    constexpr int N = kChunk<E>;
    const int cols = f.cols;
    const int64_t c = ((int64_t)blockIdx.y * kTileThreads + threadIdx.x) * N;
    if (c >= cols) return;
    const int left = cols - (int)c;
    Vec<P, N> w = (P)1.0f;
    if (f.weight) w = load<P, N>(f.weight + c, left);
    float aw[N], ab[N];
#pragma unroll
    for (int e = 0; e < N; ++e) aw[e] = ab[e] = 0.0f;
    for (int64_t row = blockIdx.x; row < f.rows; row += gridDim.x) {
        const Vec<E, N> x = load<E, N>(f.X + row * f.ldx + c, left), d = load<E, N>(f.dY + row * f.lddy + c, left);
        const float mean = f.saved[2 * row], r = f.saved[2 * row + 1], mg = means[2 * row], mgh = means[2 * row + 1];
        Vec<E, N> o;
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const float h = ((float)x[e] - mean) * r, dy = (float)d[e];
            aw[e] = __builtin_fmaf(dy, h, aw[e]);
            ab[e] += dy;
            o[e] = (E)(r * (dy * (float)w[e] - mg - h * mgh));
        }
        store<E, N>(f.dX + row * f.lddx + c, left, o);
    }
    if (!f.partial) return;
    const int64_t pitch = sum_pitch(cols);
    float* const out = f.partial + (int64_t)blockIdx.x * 2 * pitch + c;
    Vec<float, N> sw, sb;
#pragma unroll
    for (int e = 0; e < N; ++e) {
        sw[e] = aw[e];
        sb[e] = ab[e];
    }
    store<float, N>(out, left, sw);
    store<float, N>(out + pitch, left, sb);
}

// Adds the workgroups' sums.  blockIdx.y: dweight, dbias.
template <class P, int C>
__global__ void __launch_bounds__(kSumThreads) norm_columns(const float* partial, int parts, int cols, P* dweight, P* dbias)
{
    P* const to = blockIdx.y ? dbias : dweight;
    if (!to) return;
    const int64_t c = (int64_t)blockIdx.x * C + threadIdx.x % C;
    const int64_t pitch = sum_pitch(cols);
    const float sum = columns_sum<C>(c < cols ? partial + blockIdx.y * pitch + c : nullptr, 2 * pitch, parts);
    if (threadIdx.x < C && c < cols) to[c] = (P)sum;
}

// ------------------------------------------------------------------ host --

int64_t chunks_of(int64_t cols, int32_t type) { return type == LAYER_NORM_F32 ? (cols + 3) / 4 : (cols + 7) / 8; }

// Workgroups that share the rows of a backward pass, `per` rows each at a time.
int64_t sharers(int64_t rows, int64_t per, int64_t most) { return std::min((rows + per - 1) / per, most); }

// How the backward pass takes rows of so many chunks: G lanes with C chunks each
// (0: rows of any length).
struct Way {
    int g, c;
};
Way way_of(int64_t chunks)
{
    for (const Way w : {Way{8, 1}, Way{16, 1}, Way{32, 1}, Way{64, 1}, Way{64, 2}, Way{256, 1}, Way{256, 2}, Way{256, 4}, Way{512, 4}})
        if (chunks <= w.g * w.c) return w;
    return {0, 0};
}

int64_t back_groups(int64_t rows, int64_t cols, int32_t type)
{
    const Way w = way_of(chunks_of(cols, type));
    constexpr int cus = cus::kCus;
    // Rows of any length: 64 shares, but sums of 256 MB at most (2^19 columns, where that
    // begins, are 256 workgroups to a share).  (By 16, 32, 64 and 128, in bfloat16: 300 x
    // 40000 36, 36, 37 and 44 us, 3000 x 20000 194, 145, 118 and 124, 20000 x 20000 1389,
    // 952, 808 and 832.)
    if (w.g == 0) return sharers(rows, 1, std::min<int64_t>(64, ((int64_t)1 << 25) / cols));
    // Each workgroup's sums cross memory twice, and fewer workgroups hide less: steps with
    // 1, 2 and 3 for each CU take, of 500 x 16384 in bfloat16 (whose lanes hold more) 38, 50
    // and 50 us, of 1000 x 2048 (four rows to a workgroup, or two) 22.5, 24.5 and 28.4, and
    // with 2, 3 and 4 of 8192 x 4096 70, 73 and 81; the backward pass alone of 20000 x 300
    // with 1, 2 and 3 34, 21 and 17.
    // Few enough rows are one workgroup's, which needs no second launch (4 x 1024: 4.4
    // us, and 4.4 and 3.5 in two; four turns of rows take longer than that).
    const int64_t per = w.g > 256 ? 1 : 256 / w.g;
    if (rows > 0 && rows <= 2 * per) return 1;
    if (w.c == 1 && w.g <= 64) return sharers(rows, per, 4 * cus);
    return sharers(rows, per, w.c >= 4 || rows <= 4 * cus * per ? cus : 2 * cus);
}

template <class E, class P>
int forward(const Forward<E, P>& f, hipStream_t stream)
{
    const int64_t chunks = (f.cols + kChunk<E> - 1) / kChunk<E>;
    const int64_t most = cus::kCus * 8;
    auto with = [&](auto kernel, int threads, int per) {
        const int64_t n = std::min((f.rows + (int64_t)per - 1) / per, most);
        hipLaunchKernelGGL(kernel, dim3((unsigned)n), dim3(threads), 0, stream, f);
        return (int)hipGetLastError();
    };
    auto rows = [&](auto whole) {
        constexpr bool W = decltype(whole)::value;
        if (chunks <= 8) return with(norm_rows<E, P, 8, 1, W>, 256, 32);
        if (chunks <= 16) return with(norm_rows<E, P, 16, 1, W>, 256, 16);
        if (chunks <= 32) return with(norm_rows<E, P, 32, 1, W>, 256, 8);
        if (chunks <= 64) return with(norm_rows<E, P, 64, 1, W>, 256, 4);
        if (chunks <= 128) return with(norm_rows<E, P, 64, 2, W>, 256, 4);
        if (chunks <= 256) return with(norm_rows<E, P, 256, 1, W>, 256, 1);
        if (chunks <= 512) return with(norm_rows<E, P, 256, 2, W>, 256, 1);
        if (chunks <= 1024) return with(norm_rows<E, P, 256, 4, W>, 256, 1);
        if (chunks <= 2048) return with(norm_rows<E, P, 512, 4, W>, 512, 1);
        return with(norm_rows<E, P, 1024, 4, W>, 1024, 1);
    };
    if (chunks <= 4096) return f.cols % kChunk<E> ? rows(std::false_type{}) : rows(std::true_type{});
    return with(norm_wide<E, P>, kWide, 1);
}

template <class E, class P>
int backward(Backward<E, P> f, P* dweight, P* dbias, float* partial, float* means, int64_t groups, hipStream_t stream)
{
    const bool alone = groups == 1 && f.rows > 0 && way_of((f.cols + kChunk<E> - 1) / kChunk<E>).g > 0;
    if (alone) {
        f.dweight = dweight;
        f.dbias = dbias;
    } else if (dweight || dbias) {
        f.partial = partial;
    }
    const int64_t chunks = (f.cols + kChunk<E> - 1) / kChunk<E>;
    const Way w = way_of(chunks);
    int rc = hipSuccess;
    if (f.rows > 0) {
        auto with = [&](auto kernel) {
            hipLaunchKernelGGL(kernel, dim3((unsigned)groups), dim3(std::max(256, w.g)), 0, stream, f);
            return (int)hipGetLastError();
        };
        auto rows = [&](auto whole) {
            constexpr bool W = decltype(whole)::value;
            if (w.g == 8) return with(norm_back_rows<E, P, 8, 1, W>);
            if (w.g == 16) return with(norm_back_rows<E, P, 16, 1, W>);
            if (w.g == 32) return with(norm_back_rows<E, P, 32, 1, W>);
            if (w.g == 64) return w.c == 1 ? with(norm_back_rows<E, P, 64, 1, W>) : with(norm_back_rows<E, P, 64, 2, W>);
            if (w.g == 512) return with(norm_back_rows<E, P, 512, 4, W>);
            if (w.c == 1) return with(norm_back_rows<E, P, 256, 1, W>);
            return w.c == 2 ? with(norm_back_rows<E, P, 256, 2, W>) : with(norm_back_rows<E, P, 256, 4, W>);
        };
        if (w.g)
            rc = f.cols % kChunk<E> ? rows(std::false_type{}) : rows(std::true_type{});
        else {
            hipLaunchKernelGGL((norm_back_means<E, P>), dim3((unsigned)std::min<int64_t>(f.rows, 2 * cus::kCus)), dim3(kWide), 0,
                               stream, f, means);
            if ((rc = (int)hipGetLastError())) return rc;
            const int64_t tiles = (chunks + kTileThreads - 1) / kTileThreads;
            hipLaunchKernelGGL((norm_back_tiles<E, P>), dim3((unsigned)groups, (unsigned)tiles), dim3(kTileThreads), 0, stream, f,
                               (const float*)means);
            rc = (int)hipGetLastError();
        }
        if (rc) return rc;
    }
    if (!alone && (dweight || dbias)) {  // (of no rows: zeros)
        const bool wide = wide_sums(f.cols, 2);
        const int64_t columns = wide ? 64 : 16;
        hipLaunchKernelGGL((wide ? norm_columns<P, 64> : norm_columns<P, 16>), dim3((unsigned)((f.cols + columns - 1) / columns), 2),
                           dim3(kSumThreads), 0, stream, (const float*)partial, (int)groups, f.cols, dweight, dbias);
        rc = (int)hipGetLastError();
    }
    return rc;
}

struct BackwardSpace {
    float *partial, *means;
    int64_t bytes, groups;
    BackwardSpace(void* base, int64_t rows, int64_t cols, int32_t type)
    {
        abi::Carve c(base);
        groups = back_groups(rows, cols, type);
        partial = c.take<float>(groups * 2 * sum_pitch(cols));
        means = way_of(chunks_of(cols, type)).g ? nullptr : c.take<float>(2 * rows);
        bytes = c.used();
    }
};

// Rows of up to 2^24 elements: what a launch over their columns may hold.
bool good_size(int64_t rows, int64_t cols, int64_t ld) { return cols <= 1 << 24 && good_span(rows, cols, ld); }

bool good_types(int32_t type, int32_t param)
{
    return type >= LAYER_NORM_F16 && type <= LAYER_NORM_F32 && (param == type || param == LAYER_NORM_F32);
}
int64_t size_of(int32_t type) { return type == LAYER_NORM_F32 ? 4 : 2; }

}  // namespace

extern "C" {

int layer_norm_version(void) { return LAYER_NORM_VERSION; }

int64_t layer_norm_backward_workspace(int64_t rows, int64_t cols)
{
    if (!good_size(rows, cols, cols)) return -1;
    // (of either width of elements)
    return std::max(BackwardSpace(nullptr, rows, cols, LAYER_NORM_F32).bytes, BackwardSpace(nullptr, rows, cols, LAYER_NORM_F16).bytes);
}

#define FOR_TYPES(CALL)                                                                              \
    (type == LAYER_NORM_F32 ? CALL(float, float)                                                     \
     : type == LAYER_NORM_F16                                                                        \
         ? (param_type == LAYER_NORM_F32 ? CALL(_Float16, float) : CALL(_Float16, _Float16))         \
         : (param_type == LAYER_NORM_F32 ? CALL(__bf16, float) : CALL(__bf16, __bf16)))

int layer_norm(const void* X, const void* weight, const void* bias, void* Y, void* saved, int64_t rows, int64_t cols,
               int64_t ldx, int64_t ldy, int32_t type, int32_t param_type, double eps, hipStream_t stream)
{
    using namespace abi;
    if (!good_types(type, param_type) || !(eps >= 0) || !good_size(rows, cols, ldx) || !good_size(rows, cols, ldy))
        return hipErrorInvalidValue;
    if (rows == 0 || cols == 0) return hipSuccess;
    const int64_t es = size_of(type), ps = size_of(param_type);
    if (!good_pointer(X, rows, cols, es) || !good_pointer(Y, rows, cols, es) || (uintptr_t)weight % ps || (uintptr_t)bias % ps ||
        (uintptr_t)saved % 8)
        return hipErrorInvalidValue;
    const Range y(Y, rows, cols, ldy, es), s(saved, 1, saved ? 2 * rows : 0, 0, 4);
    const Range in[] = {Range(X, rows, cols, ldx, es), Range(weight, 1, weight ? cols : 0, 0, ps), Range(bias, 1, bias ? cols : 0, 0, ps)};
    for (const Range& r : in)
        if (y.meets(r) || s.meets(r)) return hipErrorInvalidValue;
    if (y.meets(s)) return hipErrorInvalidValue;
#define FORWARD(E, P)                                                                                                       \
    forward<E, P>({(const E*)X, (const P*)weight, (const P*)bias, (E*)Y, (float*)saved, ldx, ldy, (int)rows, (int)cols, (float)eps}, \
                  stream)
    return FOR_TYPES(FORWARD);
#undef FORWARD
}

int layer_norm_backward(const void* dY, const void* X, const void* weight, const void* saved, void* dX, void* dweight,
                        void* dbias, int64_t rows, int64_t cols, int64_t lddy, int64_t ldx, int64_t lddx, int32_t type,
                        int32_t param_type, void* workspace, int64_t workspace_bytes, hipStream_t stream)
{
    using namespace abi;
    if (!good_types(type, param_type) || !good_size(rows, cols, lddy) || !good_size(rows, cols, ldx) || !good_size(rows, cols, lddx))
        return hipErrorInvalidValue;
    if (cols == 0) return hipSuccess;
    const int64_t es = size_of(type), ps = size_of(param_type);
    if (!good_pointer(dY, rows, cols, es) || !good_pointer(X, rows, cols, es) || !good_pointer(dX, rows, cols, es) ||
        !good_pointer(saved, rows, cols, 8) || (uintptr_t)weight % ps || (uintptr_t)dweight % ps || (uintptr_t)dbias % ps ||
        (uintptr_t)workspace % 16)
        return hipErrorInvalidValue;
    const int64_t need = layer_norm_backward_workspace(rows, cols);
    if (need > 0 && (!workspace || workspace_bytes < need)) return hipErrorInvalidValue;
    const Range in[] = {Range(dY, rows, cols, lddy, es), Range(X, rows, cols, ldx, es), Range(weight, 1, weight ? cols : 0, 0, ps),
                        Range(saved, 1, 2 * rows, 0, 4)};
    const Range out[] = {Range(dX, rows, cols, lddx, es), Range(dweight, 1, dweight ? cols : 0, 0, ps),
                         Range(dbias, 1, dbias ? cols : 0, 0, ps), Range(workspace, 1, need, 0, 1)};
    for (int i = 0; i < 4; ++i) {
        for (const Range& r : in)
            if (out[i].meets(r)) return hipErrorInvalidValue;
        for (int k = 0; k < i; ++k)
            if (out[i].meets(out[k])) return hipErrorInvalidValue;
    }
    const BackwardSpace w(workspace, rows, cols, type);
#define BACKWARD(E, P)                                                                                                         \
    backward<E, P>({(const E*)dY, (const E*)X, (const P*)weight, (const float*)saved, (E*)dX, nullptr, nullptr, nullptr, lddy, ldx, \
                    lddx, (int)rows, (int)cols},                                                                                                \
                   (P*)dweight, (P*)dbias, w.partial, w.means, w.groups, stream)
    return FOR_TYPES(BACKWARD);
#undef BACKWARD
}

}  // extern "C"
