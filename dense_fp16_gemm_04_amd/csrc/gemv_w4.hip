// Products of a few rows with 4-bit weights for gfx950: include/gemv_w4.h.
//
// A workgroup of eight waves takes 16 R rows of W and 16 MB rows of X; the
// waves share K in ranges of whole blocks of 256, each adds up its own in
// registers, and the eight partial sums meet in LDS.  W is read once per 16 MB
// rows of X and x, from L2, once per 16 R rows of W.
//
// Reads.  A vector load is served 16 lanes at a time, one cache line each
// cycle: with a row to every lane (the matrix cores' layout) a load takes 64
// cycles, and the kernel was bound by that (3 TB/s however the data were
// placed).  So eight adjacent lanes read a whole 128-byte line of a row of W,
// and the wave turns the block round in LDS of its own; scales and zero points
// likewise.  Codes are loaded WD blocks ahead, x XD runs of 32 k ahead.
//
// From LDS, lane l = 16 h + r takes codes 32 h .. + 31 of 128 of row r as four
// words.  The matrix cores sum over the lanes h, so a sum that one scale can
// be applied to needs words of one group in one register: the 4 x 4 words of
// lanes r, r + 16, r + 32, r + 48 are transposed (two permlane32_swap, two
// permlane16_swap), after which word j of lane h holds k = 32 j + 8 h .. + 7
// and register j is one run of 32 k.
//
// Codes become numbers by placing them in the mantissa of 2^p: 1024 + q (or,
// four bits further up, 1024 + 16 q) in binary16, made q - 8 exactly by one
// packed addition or fused multiply; 128 + q in bfloat16, whose 136 goes out
// with the zero point.  One mask gives codes i and i + 4 of a word as a pair,
// so x's pairs are put in that order too.
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
constexpr int kBlock = 256;  // codes: 128 bytes of a row
// 64 rows of x or of codes span at most 2^30 bytes
constexpr int64_t kMaxLd = (int64_t)1 << 23;

template <class E>
struct Code;
template <>
struct Code<_Float16> {
    static constexpr float bias = 8.0f;  // the codes arrive less 8
    static constexpr bool exact = true;
    static constexpr uint32_t ones = 0x3c003c00u;
};
template <>
struct Code<__bf16> {
    static constexpr float bias = -128.0f;  // the codes arrive plus 128
    static constexpr bool exact = false;
    static constexpr uint32_t ones = 0x3f803f80u;
};

typedef _Float16 half2_t __attribute__((ext_vector_type(2)));

// (word & mask) | magic in one instruction, which takes one scalar register:
// the mask is held in one, the magic number in a vector register.
__device__ __forceinline__ uint32_t masked(uint32_t word, uint32_t mask, uint32_t magic) { return (word & mask) | magic; }

// The eight codes of a word as numbers (q + offset of the type), pairs (i, i + 4).
__device__ __forceinline__ Elem<_Float16>::x8 codes(uint32_t w, uint32_t magic, uint32_t low, uint32_t high, _Float16)
{
    const uint32_t v = w >> 8;
    const half2_t p0 = __builtin_bit_cast(half2_t, masked(w, low, magic)), p1 = __builtin_bit_cast(half2_t, masked(w, high, magic));
    const half2_t p2 = __builtin_bit_cast(half2_t, masked(v, low, magic)), p3 = __builtin_bit_cast(half2_t, masked(v, high, magic));
    const half2_t off = {(_Float16)-1032.0f, (_Float16)-1032.0f}, off16 = {(_Float16)-72.0f, (_Float16)-72.0f};
    const half2_t by16 = {(_Float16)0.0625f, (_Float16)0.0625f};
    const half2_t r0 = p0 + off, r1 = __builtin_elementwise_fma(p1, by16, off16);
    const half2_t r2 = p2 + off, r3 = __builtin_elementwise_fma(p3, by16, off16);
    return Elem<_Float16>::x8{r0[0], r0[1], r1[0], r1[1], r2[0], r2[1], r3[0], r3[1]};
}
__device__ __forceinline__ Elem<__bf16>::x8 codes(uint32_t w, uint32_t magic, uint32_t low, uint32_t, __bf16)
{
    const u32x4 v = {masked(w, low, magic), masked(w >> 4, low, magic), masked(w >> 8, low, magic),
                     masked(w >> 12, low, magic)};
    return __builtin_bit_cast(Elem<__bf16>::x8, v);
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

// 4 x 4 words across the lanes h: word j of lane h <- word h of lane j.
__device__ __forceinline__ u32x4 across(const u32x4& w)
{
    auto a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
    auto b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
    auto lo = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    auto hi = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    return u32x4{lo[0], lo[1], hi[0], hi[1]};
}

// N adjacent 16-bit values from LDS, two to a register.
template <int N>
struct Few {
    uint32_t v[(N + 1) / 2];
    template <class E>
    __device__ __forceinline__ float get(int i) const
    {
        const uint32_t word = v[i / 2];
        const uint16_t bits = (uint16_t)(i % 2 ? word >> 16 : word);
        return (float)__builtin_bit_cast(E, bits);
    }
};

// FLUSH: runs of 32 k per group sum (4: the group holds whole chunks of 128).
// EIGHTS: x's rows start on 16 bytes; otherwise its elements come one by one.
//
// Every load is a buffer load that the code always reaches: what does not
// exist (rows, k, blocks past the wave's) has an offset out of range and
// reads as zero, which adds nothing.  (With branches around loads the
// compiler cannot count those in flight and waits for all of them.)
template <class E, int MB, int R, int FLUSH, bool ZERO, bool EIGHTS>
__global__ void __launch_bounds__(kThreads)
gemv_w4_kernel(const E* __restrict__ X, const unsigned char* __restrict__ Q, const E* __restrict__ scale,
               const E* __restrict__ zero, E* __restrict__ Y, int M, int N, int K, int shift, int groups, int64_t ldx,
               int64_t ldq, int64_t ldy)
{
    using x8 = typename Elem<E>::x8;
    constexpr bool SUM = ZERO || !Code<E>::exact;  // the group's sum of x is needed
    constexpr int WD = MB * R <= 2 ? 2 : 1, XD = MB == 1 ? 4 : MB == 2 ? 2 : 1;
    constexpr int NS = 8 / FLUSH;                  // scales of a block's row
    constexpr int NL = (16 * R * NS + 63) / 64;    // loads for a block's scales
    constexpr int W_BYTES = R * 16 * 128, S_BYTES = R * 16 * 16, PART = MB * R * 16 * 17 * 4;
    constexpr int REGION = W_BYTES + 2 * S_BYTES > PART ? W_BYTES + 2 * S_BYTES : PART;
    __shared__ __attribute__((aligned(128))) unsigned char smem[kWaves * REGION];
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    unsigned char* mine = smem + wave * REGION;  // no other wave's until the partial sums meet
    const int r = lane & 15, h = lane >> 4;
    const int n0 = blockIdx.x * 16 * R, m0 = blockIdx.y * 16 * MB;
    const uint32_t rows_w = (uint32_t)min(16 * R, N - n0), rows_x = (uint32_t)min(16 * MB, M - m0);
    const __amdgpu_buffer_rsrc_t bq = make_rsrc(Q + n0 * ldq, rows_w * (uint32_t)ldq);
    const __amdgpu_buffer_rsrc_t bs = make_rsrc(scale + (int64_t)n0 * groups, rows_w * (uint32_t)groups * 2u);
    const __amdgpu_buffer_rsrc_t bz = make_rsrc(ZERO ? zero + (int64_t)n0 * groups : scale,
                                                ZERO ? rows_w * (uint32_t)groups * 2u : 0u);
    const __amdgpu_buffer_rsrc_t bx = make_rsrc(X + m0 * ldx, rows_x * (uint32_t)ldx * 2u);

    f32x4 total[R][MB], acc[R][MB], sum[MB];
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int b = 0; b < MB; ++b) total[i][b] = f32x4{0, 0, 0, 0};

    const int blocks = (K + kBlock - 1) / kBlock, each = (blocks + kWaves - 1) / kWaves;
    const int first = wave * each, last = min(first + each, blocks), k_end = min(last * kBlock, K);
    struct Block {
        u32x4 w[2 * R];  // eight rows each: row lane / 8, bytes 16 (lane % 8) .. + 15
        uint16_t s[NL], z[NL];
    } c[WD];
    u32x4 x[XD][MB];
    auto fetch = [&](Block& c, int at) __attribute__((always_inline)) {
        const int k0 = at * kBlock, k = k0 + 32 * (lane & 7);
#pragma unroll
        for (int i = 0; i < 2 * R; ++i) {
            const uint32_t row = 8 * i + (lane >> 3);
            c.w[i] = __builtin_amdgcn_raw_buffer_load_b128(bq, k < k_end ? row * (uint32_t)ldq + (uint32_t)(k / 2) : kOob,
                                                           0, 0);
        }
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            const uint32_t row = (i * 64 + lane) / NS;
            const int ks = k0 + 32 * FLUSH * (lane % NS);
            const uint32_t so =
                ks < k_end && row < 16 * R ? (row * (uint32_t)groups + (uint32_t)(ks >> shift)) * 2u : kOob;
            c.s[i] = __builtin_amdgcn_raw_buffer_load_b16(bs, so, 0, 0);
            if constexpr (ZERO) c.z[i] = __builtin_amdgcn_raw_buffer_load_b16(bz, so, 0, 0);
        }
    };
    uint32_t xo[MB];
#pragma unroll
    for (int b = 0; b < MB; ++b) xo[b] = ((16u * b + r) * (uint32_t)ldx + 8u * h) * 2u;
    auto fetch_x = [&](u32x4 (&v)[MB], int run) __attribute__((always_inline)) {
        // (xo is below 2^30: the sum with the mark is out of range too)
        const uint32_t ko = run * 32 < k_end ? (uint32_t)run * 64u : kOob;
#pragma unroll
        for (int b = 0; b < MB; ++b) {
            const uint32_t at = xo[b] + ko;
            if constexpr (EIGHTS) {
                v[b] = __builtin_amdgcn_raw_buffer_load_b128(bx, at, 0, 0);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t lo = __builtin_amdgcn_raw_buffer_load_b16(bx, at, 4 * e, 0);
                    const uint32_t hi = __builtin_amdgcn_raw_buffer_load_b16(bx, at, 4 * e + 2, 0);
                    v[b][e] = lo | hi << 16;
                }
            }
        }
    };
    const u32x4 ones_bits = {Code<E>::ones, Code<E>::ones, Code<E>::ones, Code<E>::ones};
    const x8 ones = __builtin_bit_cast(x8, ones_bits);
    uint32_t magic = Code<E>::exact ? 0x64006400u : 0x43004300u, low = 0x000f000fu, high = 0x00f000f0u;
    asm volatile("" : "+v"(magic), "+s"(low), "+s"(high));
    // what other lanes wrote is read after this (a wave's LDS accesses are in order)
    auto turn = [&]() __attribute__((always_inline)) {
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    };
    auto add = [&](Block& c, int at) __attribute__((always_inline)) {
        turn();  // (the last block's reads)
#pragma unroll
        for (int i = 0; i < 2 * R; ++i) {
            const int row = 8 * i + (lane >> 3);
            *(u32x4*)(mine + row * 128 + swizzle(row, lane & 7) * 16) = c.w[i];
        }
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            const int row = (i * 64 + lane) / NS, to = W_BYTES + row * 16 + (lane % NS) * 2;
            if (16 * R * NS % 64 == 0 || row < 16 * R) {
                *(uint16_t*)(mine + to) = c.s[i];
                if constexpr (ZERO) *(uint16_t*)(mine + S_BYTES + to) = c.z[i];
            }
        }
        turn();
        Few<NS> s[R], z[R];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const unsigned char* from = mine + W_BYTES + (16 * i + r) * 16;
            __builtin_memcpy(s[i].v, __builtin_assume_aligned(from, 16), 2 * NS);
            if constexpr (ZERO) __builtin_memcpy(z[i].v, __builtin_assume_aligned(from + S_BYTES, 16), 2 * NS);
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            u32x4 w[R];
#pragma unroll
            for (int i = 0; i < R; ++i)
                w[i] = across(*(const u32x4*)(mine + (16 * i + r) * 128 + swizzle(r, 4 * half + h) * 16));
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
                fetch_x(x[j % XD], at * 8 + 4 * half + j + XD);
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    const x8 wv = codes(w[i][j], magic, low, high, E{});
#pragma unroll
                    for (int b = 0; b < MB; ++b) acc[i][b] = Elem<E>::mfma(xv[b], wv, acc[i][b]);
                }
                if (j % FLUSH == FLUSH - 1)
#pragma unroll
                    for (int i = 0; i < R; ++i) {
                        const int g = (4 * half + j) / FLUSH;
                        const float sf = s[i].template get<E>(g);
                        const float zf = (ZERO ? z[i].template get<E>(g) : 8.0f) - Code<E>::bias;
#pragma unroll
                        for (int b = 0; b < MB; ++b)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                float v = acc[i][b][e];
                                if constexpr (SUM) v = __builtin_fmaf(-zf, sum[b][e], v);
                                total[i][b][e] = __builtin_fmaf(sf, v, total[i][b][e]);
                            }
                    }
            }
        }
    };

#pragma unroll
    for (int d = 0; d < WD; ++d) fetch(c[d], first + d);
#pragma unroll
    for (int d = 0; d < XD; ++d) fetch_x(x[d], first * 8 + d);
    for (int at = first; at < last; at += WD)
#pragma unroll
        for (int d = 0; d < WD; ++d) {
            add(c[d], at + d);
            fetch(c[d], at + d + WD);
        }

    turn();
    typedef float Part[MB * R][16][17];
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int b = 0; b < MB; ++b)
#pragma unroll
            for (int e = 0; e < 4; ++e) (*(Part*)mine)[i * MB + b][4 * h + e][r] = total[i][b][e];
    __syncthreads();
    for (int at = threadIdx.x; at < R * MB * 256; at += kThreads) {
        const int p = at >> 8, m = m0 + p % MB * 16 + ((at >> 4) & 15), n = n0 + p / MB * 16 + (at & 15);
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) v += (*(const Part*)(smem + w * REGION))[p][(at >> 4) & 15][at & 15];
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

template <class E, int MB, int R, int FLUSH, bool ZERO, bool EIGHTS>
int launch(const Args& a)
{
    // grid.y holds 65535 at most: more rows go in further launches
    constexpr int64_t most = (int64_t)65535 * 16 * MB;
    for (int64_t m = 0; m < a.M; m += most) {
        const int64_t rows = std::min(most, a.M - m);
        hipLaunchKernelGGL((gemv_w4_kernel<E, MB, R, FLUSH, ZERO, EIGHTS>),
                           dim3((unsigned)((a.N + 16 * R - 1) / (16 * R)), (unsigned)((rows + 16 * MB - 1) / (16 * MB))),
                           dim3(kThreads), 0, a.stream, (const E*)a.X + m * a.ldx, (const unsigned char*)a.Q,
                           (const E*)a.scale, (const E*)a.zero, (E*)a.Y + m * a.ldy, (int)rows, (int)a.N, (int)a.K,
                           a.shift, (int)a.groups, a.ldx, a.ldq, a.ldy);
        const int rc = (int)hipGetLastError();
        if (rc) return rc;
    }
    return hipSuccess;
}

template <class E, int MB, int R, int FLUSH, bool EIGHTS>
int by_zero(const Args& a)
{
    return a.zero ? launch<E, MB, R, FLUSH, true, EIGHTS>(a) : launch<E, MB, R, FLUSH, false, EIGHTS>(a);
}

template <class E, int MB, int R, bool EIGHTS = true>
int by_group(const Args& a)
{
    if (a.shift >= 7) return by_zero<E, MB, R, 4, EIGHTS>(a);
    if (a.shift == 6) return by_zero<E, MB, R, 2, EIGHTS>(a);
    return by_zero<E, MB, R, 1, EIGHTS>(a);
}

template <class E>
int run(const Args& a)
{
    if ((uintptr_t)a.X % 16 || (a.M > 1 && a.ldx % 8)) return by_group<E, 1, 1, false>(a);
    // as many rows of W to a workgroup as leave one for every CU
    const int64_t mb = a.M <= 16 ? 1 : a.M <= 32 ? 2 : 4;
    const int64_t blocks = (a.N + 15) / 16 * ((a.M + 16 * mb - 1) / (16 * mb));
    const bool two = blocks >= 2 * 256;
    if (mb == 1) return two ? by_group<E, 1, 2>(a) : by_group<E, 1, 1>(a);
    if (mb == 2) return two ? by_group<E, 2, 2>(a) : by_group<E, 2, 1>(a);
    return two ? by_group<E, 4, 2>(a) : by_group<E, 4, 1>(a);
}

}  // namespace

extern "C" {

int gemv_w4_version(void) { return GEMV_W4_VERSION; }

int gemv_w4(const void* X, const void* Q, const void* scale, const void* zero, void* Y, int64_t M, int64_t N, int64_t K,
            int64_t group, int64_t ldx, int64_t ldq, int64_t ldy, int32_t type, hipStream_t stream)
{
    using namespace abi;
    if (!good_dim(M) || !good_dim(N) || N > kMaxDim - 16 || K < 0 || K > kMaxPitch) return hipErrorInvalidValue;
    if (K % 32 || ldx < K || ldx > kMaxLd || ldq < K / 2 || ldq % 16 || ldq > kMaxLd || ldy < N || ldy > kMaxDim)
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
