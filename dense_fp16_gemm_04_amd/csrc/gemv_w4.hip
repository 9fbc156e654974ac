// Products of a few rows with 4-bit weights for gfx950: include/gemv_w4.h.
//
// A workgroup of eight waves takes 16 R rows of W and 16 MB rows of X; the
// waves share K in ranges of whole chunks of 128, each adds up its own in
// registers, and the eight partial sums meet in LDS.  Per chunk a lane reads
// 16 bytes (32 codes) of one row of W, so a wave reads 64 adjacent bytes of
// each of 16 rows.  W is read once per 16 MB rows of X and x, from L2, once per
// 16 R rows of W; what counts is bytes in flight: codes are loaded WD chunks
// ahead, x XD runs of 32 k ahead.
//
// Lane l = 16 h + r holds codes 32 h .. + 31 of row r as four words.  The
// matrix cores sum over the lanes h, so a sum that one scale can be applied
// to needs words of one group in one register: the 4 x 4 words of lanes r, r
// + 16, r + 32, r + 48 are transposed (two permlane32_swap, two
// permlane16_swap), after which word j of lane h holds k = 32 j + 8 h .. + 7
// and register j is one run of 32 k.
//
// Codes become numbers by placing them in the mantissa of 2^p: 1024 + q in
// binary16 (0x6400 | q), less 1032 exactly; 128 + q in bfloat16 (0x4300 | q),
// whose 136 goes out with the zero point.  One shift and one mask give codes
// i and i + 4 of a word as a pair, so x's pairs are put in that order too.
//
// With x as the first operand of v_mfma_f32_16x16x32, lane l's four results
// belong to row l % 16 of W and rows 4 h .. 4 h + 3 of X: one scale per lane.
// The group's sum of x, for the zero points, is one more product with ones.
#include "gemv_w4.h"

#include <algorithm>

#include "abi.h"
#include "cdna4.h"

namespace {

using namespace cdna4;

constexpr int kWaves = 8, kThreads = kWaves * kWave;
constexpr int kChunk = 128;

template <class E>
struct Code;
template <>
struct Code<_Float16> {
    static constexpr uint32_t magic = 0x64006400u;
    static constexpr float bias = 8.0f;  // the codes arrive less 8
    static constexpr bool exact = true;
    static constexpr uint32_t ones = 0x3c003c00u;
};
template <>
struct Code<__bf16> {
    static constexpr uint32_t magic = 0x43004300u;
    static constexpr float bias = -128.0f;  // the codes arrive plus 128
    static constexpr bool exact = false;
    static constexpr uint32_t ones = 0x3f803f80u;
};

// The eight codes of a word as numbers (q + offset of the type), pairs (i, i + 4).
template <class E>
__device__ __forceinline__ typename Elem<E>::x8 codes(uint32_t w)
{
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t pair = ((w >> (4 * i)) & 0x000f000fu) | Code<E>::magic;
        if constexpr (Code<E>::exact) {
            typedef _Float16 h2 __attribute__((ext_vector_type(2)));
            const h2 d = __builtin_bit_cast(h2, pair) - (h2){(_Float16)1032.0f, (_Float16)1032.0f};
            pair = __builtin_bit_cast(uint32_t, d);
        }
        v[i] = pair;
    }
    return __builtin_bit_cast(typename Elem<E>::x8, v);
}

// x's eight values in the order of codes(): (0, 4), (1, 5), (2, 6), (3, 7).
__device__ __forceinline__ u32x4 pair_order(const u32x4& x)
{
    u32x4 v;
    v[0] = __builtin_amdgcn_perm(x[2], x[0], 0x05040100u);
    v[1] = __builtin_amdgcn_perm(x[2], x[0], 0x07060302u);
    v[2] = __builtin_amdgcn_perm(x[3], x[1], 0x05040100u);
    v[3] = __builtin_amdgcn_perm(x[3], x[1], 0x07060302u);
    return v;
}

// One, two or four adjacent 16-bit values, two to a register.
template <int N>
struct Few {
    uint32_t v[(N + 1) / 2];
};
// Loads the first n (the same for all lanes).
template <class E, int N>
__device__ __forceinline__ void load_few(Few<N>& f, const E* p, int n)
{
    if (n == N) {
        if constexpr (N == 1)
            f.v[0] = *(const uint16_t*)p;
        else
            __builtin_memcpy(f.v, p, 2 * N);
    } else {
#pragma unroll
        for (int i = 0; i < (N + 1) / 2; ++i) {
            const uint32_t lo = 2 * i < n ? ((const uint16_t*)p)[2 * i] : 0;
            const uint32_t hi = 2 * i + 1 < n ? ((const uint16_t*)p)[2 * i + 1] : 0;
            f.v[i] = lo | hi << 16;
        }
    }
}
template <class E, int N>
__device__ __forceinline__ float few(const Few<N>& f, int i)
{
    const uint32_t word = f.v[i / 2];
    const uint16_t bits = (uint16_t)(i % 2 ? word >> 16 : word);
    return (float)__builtin_bit_cast(E, bits);
}

// FLUSH: runs of 32 k per group sum (4: the group holds whole chunks).
template <class E, int MB, int R, int FLUSH, bool ZERO>
__global__ void __launch_bounds__(kThreads)
gemv_w4_kernel(const E* __restrict__ X, const unsigned char* __restrict__ Q, const E* __restrict__ scale,
               const E* __restrict__ zero, E* __restrict__ Y, int M, int N, int K, int shift, int groups, int64_t ldx,
               int64_t ldq, int64_t ldy)
{
    using x8 = typename Elem<E>::x8;
    constexpr bool SUM = ZERO || !Code<E>::exact;  // the group's sum of x is needed
    constexpr int SC = 4 / FLUSH;                  // scales of a chunk
    constexpr int WD = MB * R == 1 ? 4 : MB * R <= 4 ? 2 : 1, XD = MB == 1 ? 4 : MB == 2 ? 2 : 1;
    __shared__ float part[kWaves][MB * R][16][17];
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int r = lane & 15, h = lane >> 4;
    const int n0 = blockIdx.x * 16 * R, m0 = blockIdx.y * 16 * MB;
    // Rows past the end repeat the last one: what they give is not stored.
    const unsigned char* q[R];
    const E *sp[R], *zp[R], *xp[MB];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int64_t n = min(n0 + 16 * i + r, N - 1);
        q[i] = Q + n * ldq + 16 * h;
        sp[i] = scale + n * groups;
        zp[i] = ZERO ? zero + n * groups : nullptr;
    }
#pragma unroll
    for (int b = 0; b < MB; ++b) xp[b] = X + (int64_t)min(m0 + 16 * b + r, M - 1) * ldx + 8 * h;

    f32x4 total[R][MB], acc[R][MB], sum[MB];
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int b = 0; b < MB; ++b) total[i][b] = f32x4{0, 0, 0, 0};

    const int chunks = (K + kChunk - 1) / kChunk, each = (chunks + kWaves - 1) / kWaves;
    const int first = wave * each, last = min(first + each, chunks), runs = min(last * 4, K / 32);
    struct Chunk {
        u32x4 w[R];
        Few<SC> s[R], z[R];
    } c[WD];
    u32x4 x[XD][MB];
    auto fetch = [&](Chunk& c, int at) __attribute__((always_inline)) {
        const int k0 = at * kChunk;
        const bool whole = k0 + kChunk <= K;  // (the same for all lanes)
#pragma unroll
        for (int i = 0; i < R; ++i) {
            if (whole || k0 + 32 * h < K)
                c.w[i] = *(const u32x4*)(q[i] + k0 / 2);
            else
                c.w[i] = u32x4{0, 0, 0, 0};
            // the chunk's scales lie side by side where a group is shorter than it
            const int group = k0 >> shift, n = whole ? SC : min(SC, groups - group);
            load_few<E, SC>(c.s[i], sp[i] + group, n);
            if constexpr (ZERO) load_few<E, SC>(c.z[i], zp[i] + group, n);
        }
    };
    // (x of runs that the wave does not have is zero: the last chunk may hold
    // fewer than four)
    auto fetch_x = [&](u32x4 (&v)[MB], int run) __attribute__((always_inline)) {
        if (run < runs)
#pragma unroll
            for (int b = 0; b < MB; ++b) __builtin_memcpy(&v[b], xp[b] + run * 32, 16);  // (any 2-byte boundary)
        else
#pragma unroll
            for (int b = 0; b < MB; ++b) v[b] = u32x4{0, 0, 0, 0};
    };
    const u32x4 ones_bits = {Code<E>::ones, Code<E>::ones, Code<E>::ones, Code<E>::ones};
    const x8 ones = __builtin_bit_cast(x8, ones_bits);

    auto add = [&](Chunk& c, int at) __attribute__((always_inline)) {
        // 4 x 4 words across the lanes h: word j of lane h <- word h of lane j
#pragma unroll
        for (int i = 0; i < R; ++i) {
            u32x4& w = c.w[i];
            auto a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
            auto b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
            auto lo = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
            auto hi = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
            w = u32x4{lo[0], lo[1], hi[0], hi[1]};
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            // (one run after another where their sums would not fit together)
            if constexpr (MB * R >= 8) __builtin_amdgcn_sched_barrier(0);
            if (j % FLUSH == 0)
#pragma unroll
                for (int b = 0; b < MB; ++b) {
                    sum[b] = f32x4{0, 0, 0, 0};
#pragma unroll
                    for (int i = 0; i < R; ++i) acc[i][b] = f32x4{0, 0, 0, 0};
                }
            x8 xv[MB];
#pragma unroll
            for (int b = 0; b < MB; ++b) {
                xv[b] = __builtin_bit_cast(x8, pair_order(x[j % XD][b]));
                if constexpr (SUM) sum[b] = Elem<E>::mfma(xv[b], ones, sum[b]);
            }
            fetch_x(x[j % XD], at * 4 + j + XD);
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const x8 wv = codes<E>(c.w[i][j]);
#pragma unroll
                for (int b = 0; b < MB; ++b) acc[i][b] = Elem<E>::mfma(xv[b], wv, acc[i][b]);
            }
            if (j % FLUSH == FLUSH - 1)
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    const float s = few<E, SC>(c.s[i], j / FLUSH);
                    const float z = (ZERO ? few<E, SC>(c.z[i], j / FLUSH) : 8.0f) - Code<E>::bias;
#pragma unroll
                    for (int b = 0; b < MB; ++b)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            float v = acc[i][b][e];
                            if constexpr (SUM) v = __builtin_fmaf(-z, sum[b][e], v);
                            total[i][b][e] = __builtin_fmaf(s, v, total[i][b][e]);
                        }
                }
        }
    };

#pragma unroll
    for (int d = 0; d < WD; ++d)
        if (first + d < last) fetch(c[d], first + d);
#pragma unroll
    for (int d = 0; d < XD; ++d) fetch_x(x[d], first * 4 + d);
    for (int at = first; at < last; at += WD)
#pragma unroll
        for (int d = 0; d < WD; ++d)
            if (at + d < last) {
                add(c[d], at + d);
                if (at + d + WD < last) fetch(c[d], at + d + WD);
            }

#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int b = 0; b < MB; ++b)
#pragma unroll
            for (int e = 0; e < 4; ++e) part[wave][i * MB + b][4 * h + e][r] = total[i][b][e];
    __syncthreads();
    for (int at = threadIdx.x; at < R * MB * 256; at += kThreads) {
        const int p = at >> 8, m = m0 + p % MB * 16 + ((at >> 4) & 15), n = n0 + p / MB * 16 + (at & 15);
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) v += part[w][p][(at >> 4) & 15][at & 15];
        if (m < M && n < N) Y[(int64_t)m * ldy + n] = (E)v;
    }
}

struct Args {
    const void *X, *Q, *scale, *zero;
    void* Y;
    int64_t M, N, K;
    int shift;
    int64_t groups, ldx, ldq, ldy;
    hipStream_t stream;
};

template <class E, int MB, int R, int FLUSH, bool ZERO>
int launch(const Args& a)
{
    // grid.y holds 65535 at most: more rows go in further launches
    constexpr int64_t most = (int64_t)65535 * 16 * MB;
    for (int64_t m = 0; m < a.M; m += most) {
        const int64_t rows = std::min(most, a.M - m);
        hipLaunchKernelGGL((gemv_w4_kernel<E, MB, R, FLUSH, ZERO>),
                           dim3((unsigned)((a.N + 16 * R - 1) / (16 * R)), (unsigned)((rows + 16 * MB - 1) / (16 * MB))),
                           dim3(kThreads), 0, a.stream, (const E*)a.X + m * a.ldx, (const unsigned char*)a.Q,
                           (const E*)a.scale, (const E*)a.zero, (E*)a.Y + m * a.ldy, (int)rows, (int)a.N, (int)a.K,
                           a.shift, (int)a.groups, a.ldx, a.ldq, a.ldy);
        const int rc = (int)hipGetLastError();
        if (rc) return rc;
    }
    return hipSuccess;
}

template <class E, int MB, int R, int FLUSH>
int by_zero(const Args& a)
{
    return a.zero ? launch<E, MB, R, FLUSH, true>(a) : launch<E, MB, R, FLUSH, false>(a);
}

template <class E>
int run(const Args& a)
{
    // as many rows of W to a workgroup as leave one for every CU; with 64 rows
    // of X, groups of 32 need the registers that more rows of W would
    const int64_t mb = a.M <= 16 ? 1 : a.M <= 32 ? 2 : 4;
    const int64_t blocks = (a.N + 15) / 16 * ((a.M + 16 * mb - 1) / (16 * mb));
    const bool two = blocks >= 2 * 256;
#define BY_GROUP(MB, R)                             \
    (a.shift >= 7   ? by_zero<E, MB, R, 4>(a)       \
     : a.shift == 6 ? by_zero<E, MB, R, 2>(a)       \
                    : by_zero<E, MB, R, 1>(a))
    if (mb == 1) return two ? BY_GROUP(1, 2) : BY_GROUP(1, 1);
    if (mb == 2) return two ? BY_GROUP(2, 2) : BY_GROUP(2, 1);
    if (two && a.shift >= 6) return a.shift >= 7 ? by_zero<E, 4, 2, 4>(a) : by_zero<E, 4, 2, 2>(a);
    return BY_GROUP(4, 1);
#undef BY_GROUP
}

}  // namespace

extern "C" {

int gemv_w4_version(void) { return GEMV_W4_VERSION; }

int gemv_w4(const void* X, const void* Q, const void* scale, const void* zero, void* Y, int64_t M, int64_t N, int64_t K,
            int64_t group, int64_t ldx, int64_t ldq, int64_t ldy, int32_t type, hipStream_t stream)
{
    using namespace abi;
    if (!good_dim(M) || !good_dim(N) || N > kMaxDim - 16 || K < 0 || K > kMaxPitch) return hipErrorInvalidValue;
    if (K % 32 || ldx < K || ldx > kMaxDim || ldq < K / 2 || ldq % 16 || ldq > kMaxDim || ldy < N || ldy > kMaxDim)
        return hipErrorInvalidValue;
    if (K > 0 && (group < 1 || K % group || ((group < 32 || (group & (group - 1))) && group != K)))
        return hipErrorInvalidValue;
    if (type != GEMV_W4_F16 && type != GEMV_W4_BF16) return hipErrorInvalidValue;
    if (M == 0 || N == 0) return hipSuccess;
    const int64_t groups = K ? K / group : 0;
    if (!good_pointer(X, M, K, 2) || !good_pointer(Q, N, K, 16) || !good_pointer(scale, N, groups, 2) ||
        (uintptr_t)zero % 2 || !good_pointer(Y, M, N, 2))
        return hipErrorInvalidValue;
    const Range y(Y, M, N, ldy, 2);
    const Range in[] = {Range(X, M, K, ldx, 2), Range(Q, N, K / 2, ldq, 1), Range(scale, N, groups, groups, 2),
                        Range(zero, zero ? N : 0, groups, groups, 2)};
    for (const Range& i : in)
        if (y.meets(i)) return hipErrorInvalidValue;
    int shift = 30;  // one group: every k belongs to it
    if (group != K)
        for (shift = 5; ((int64_t)1 << shift) < group; ++shift) {}
    const Args a{X, Q, scale, zero, Y, M, N, K, shift, groups, ldx, ldq, ldy, stream};
    return type == GEMV_W4_F16 ? run<_Float16>(a) : run<__bf16>(a);
}

}  // extern "C"
