// Products of a few rows with 4-bit weights for gfx950: include/gemv_w4.h.
//
// A workgroup of eight waves takes 16 rows of W and 16 * MB rows of X; the
// waves share K in chunks of 128, each adds up its own in registers, and the
// eight partial sums meet in LDS.  Per chunk a lane reads 16 bytes (32 codes)
// of one row of W, so a wave reads 64 adjacent bytes of each of its 16 rows.
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

// FLUSH: runs of 32 k per group sum (4: the group holds whole chunks).
template <class E, int MB, int FLUSH, bool ZERO>
__global__ void __launch_bounds__(kThreads)
gemv_w4_kernel(const E* __restrict__ X, const unsigned char* __restrict__ Q, const E* __restrict__ scale,
               const E* __restrict__ zero, E* __restrict__ Y, int M, int N, int K, int shift, int groups, int64_t ldx,
               int64_t ldq, int64_t ldy, int x_vec)
{
    constexpr bool SUM = ZERO || !Code<E>::exact;  // the group's sum of x is needed
    __shared__ float part[kWaves][MB][16][17];
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int r = lane & 15, h = lane >> 4;
    const int n0 = blockIdx.x * 16, m0 = blockIdx.y * 16 * MB;
    const int n = min(n0 + r, N - 1);  // rows past N repeat the last one and are not stored
    const unsigned char* q = Q + n * ldq;
    const E* srow = scale + (int64_t)n * groups;
    const E* zrow = ZERO ? zero + (int64_t)n * groups : nullptr;

    f32x4 total[MB];
#pragma unroll
    for (int b = 0; b < MB; ++b) total[b] = f32x4{0, 0, 0, 0};

    auto load_x = [&](int b, int k) __attribute__((always_inline)) {
        const int m = m0 + b * 16 + r;
        u32x4 v = {0, 0, 0, 0};
        if (m < M && k < K) {
            const E* p = X + m * ldx + k;
            if (x_vec) {
                v = *(const u32x4*)p;
            } else {
                typename Elem<E>::x8 e;
#pragma unroll
                for (int i = 0; i < 8; ++i) e[i] = p[i];
                v = __builtin_bit_cast(u32x4, e);
            }
        }
        return v;
    };

    const int chunks = (K + kChunk - 1) / kChunk;
    for (int c = wave; c < chunks; c += kWaves) {
        const int k0 = c * kChunk;
        u32x4 w = {0, 0, 0, 0};
        if (k0 + 32 * h < K) w = *(const u32x4*)(q + k0 / 2 + 16 * h);
        float s[4 / FLUSH], z[4 / FLUSH];
#pragma unroll
        for (int g = 0; g < 4 / FLUSH; ++g) {
            const int at = min((k0 + 32 * FLUSH * g) >> shift, groups - 1);
            s[g] = (float)srow[at];
            z[g] = (ZERO ? (float)zrow[at] : 8.0f) - Code<E>::bias;
        }
        u32x4 x[4][MB];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int b = 0; b < MB; ++b) x[j][b] = load_x(b, k0 + 32 * j + 8 * h);
        // 4 x 4 words across the lanes h: word j of lane h <- word h of lane j
        {
            auto a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
            auto b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
            auto lo = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
            auto hi = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
            w[0] = lo[0];
            w[1] = lo[1];
            w[2] = hi[0];
            w[3] = hi[1];
        }
        f32x4 acc[MB], sum[MB];
        const u32x4 ones_bits = {Code<E>::ones, Code<E>::ones, Code<E>::ones, Code<E>::ones};
        const typename Elem<E>::x8 ones = __builtin_bit_cast(typename Elem<E>::x8, ones_bits);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (j % FLUSH == 0)
#pragma unroll
                for (int b = 0; b < MB; ++b) acc[b] = sum[b] = f32x4{0, 0, 0, 0};
            const typename Elem<E>::x8 wv = codes<E>(w[j]);
#pragma unroll
            for (int b = 0; b < MB; ++b) {
                const typename Elem<E>::x8 xv = __builtin_bit_cast(typename Elem<E>::x8, pair_order(x[j][b]));
                acc[b] = Elem<E>::mfma(xv, wv, acc[b]);
                if constexpr (SUM) sum[b] = Elem<E>::mfma(xv, ones, sum[b]);
            }
            if (j % FLUSH == FLUSH - 1)
#pragma unroll
                for (int b = 0; b < MB; ++b)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float v = acc[b][e];
                        if constexpr (SUM) v = __builtin_fmaf(-z[j / FLUSH], sum[b][e], v);
                        total[b][e] = __builtin_fmaf(s[j / FLUSH], v, total[b][e]);
                    }
        }
    }
#pragma unroll
    for (int b = 0; b < MB; ++b)
#pragma unroll
        for (int e = 0; e < 4; ++e) part[wave][b][4 * h + e][r] = total[b][e];
    __syncthreads();
    for (int i = threadIdx.x; i < MB * 256; i += kThreads) {
        const int b = i >> 8, m = (i >> 4) & 15, c = i & 15;
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) v += part[w][b][m][c];
        if (m0 + b * 16 + m < M && n0 + c < N) Y[(int64_t)(m0 + b * 16 + m) * ldy + n0 + c] = (E)v;
    }
}

template <class E, int MB, int FLUSH, bool ZERO>
int launch(const void* X, const void* Q, const void* scale, const void* zero, void* Y, int64_t M, int64_t N, int64_t K,
           int shift, int64_t groups, int64_t ldx, int64_t ldq, int64_t ldy, hipStream_t stream)
{
    const int x_vec = (uintptr_t)X % 16 == 0 && (M == 1 || ldx % 8 == 0);
    // grid.y holds 65535 at most: more rows go in further launches
    constexpr int64_t most = (int64_t)65535 * 16 * MB;
    for (int64_t m = 0; m < M; m += most) {
        const int64_t rows = std::min(most, M - m);
        hipLaunchKernelGGL((gemv_w4_kernel<E, MB, FLUSH, ZERO>),
                           dim3((unsigned)((N + 15) / 16), (unsigned)((rows + 16 * MB - 1) / (16 * MB))), dim3(kThreads),
                           0, stream, (const E*)X + m * ldx, (const unsigned char*)Q, (const E*)scale, (const E*)zero,
                           (E*)Y + m * ldy, (int)rows, (int)N, (int)K, shift, (int)groups, ldx, ldq, ldy, x_vec);
        const int rc = (int)hipGetLastError();
        if (rc) return rc;
    }
    return hipSuccess;
}

template <class E, int MB, bool ZERO>
int by_group(const void* X, const void* Q, const void* scale, const void* zero, void* Y, int64_t M, int64_t N, int64_t K,
             int shift, int64_t groups, int64_t ldx, int64_t ldq, int64_t ldy, hipStream_t stream)
{
    if (shift >= 7) return launch<E, MB, 4, ZERO>(X, Q, scale, zero, Y, M, N, K, shift, groups, ldx, ldq, ldy, stream);
    if (shift == 6) return launch<E, MB, 2, ZERO>(X, Q, scale, zero, Y, M, N, K, shift, groups, ldx, ldq, ldy, stream);
    return launch<E, MB, 1, ZERO>(X, Q, scale, zero, Y, M, N, K, shift, groups, ldx, ldq, ldy, stream);
}

template <class E>
int run(const void* X, const void* Q, const void* scale, const void* zero, void* Y, int64_t M, int64_t N, int64_t K,
        int shift, int64_t groups, int64_t ldx, int64_t ldq, int64_t ldy, hipStream_t stream)
{
#define ROWS(MB)                                                                                                 \
    (zero ? by_group<E, MB, true>(X, Q, scale, zero, Y, M, N, K, shift, groups, ldx, ldq, ldy, stream)           \
          : by_group<E, MB, false>(X, Q, scale, zero, Y, M, N, K, shift, groups, ldx, ldq, ldy, stream))
    if (M <= 16) return ROWS(1);
    if (M <= 32) return ROWS(2);
    return ROWS(4);
#undef ROWS
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
    return type == GEMV_W4_F16 ? run<_Float16>(X, Q, scale, zero, Y, M, N, K, shift, groups, ldx, ldq, ldy, stream)
                               : run<__bf16>(X, Q, scale, zero, Y, M, N, K, shift, groups, ldx, ldq, ldy, stream);
}

}  // extern "C"
