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
// One row by 16384 x 16384: 34 us, 3.9 TB/s of codes (39 with zero points, 36
// in bfloat16); by 8192 x 4096 7.3 us, less than the call takes on the host.
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

// A sum that is not finite, from the definition term by term.  The kernels add
// up (q + offset) x and take offset + zero times the sum of x out again: an
// infinite x then gives inf - inf in place of the infinity that (q - zero) x
// is, and bfloat16 x past 2^128 / 143 overflow where q - zero alone would not.
// Whatever goes wrong so leaves an infinity or a NaN, so those results, and
// only those, are computed once more, in 64 bits, which no x, zero and scale
// overflow.  A wave takes one result, its lanes eight k each in turn (one row
// with an infinity by 8192 x 4096: 57 us instead of 9; a result to a lane
// took 305).  Rows that begin with a NaN, as those of unused memory and of
// masked tokens do, stay as they are: their results are NaN.
__device__ __forceinline__ bool is_finite(float v)
{
    return (__builtin_bit_cast(uint32_t, v) & 0x7f800000u) != 0x7f800000u;
}
__device__ __forceinline__ bool is_nan(float v) { return v != v; }
template <class E>
__device__ __forceinline__ float by_terms(const E* __restrict__ x, const unsigned char* __restrict__ q,
                                          const E* __restrict__ scale, const E* __restrict__ zero, int K, int shift, int lane)
{
    double sum = 0;
#pragma unroll 1
    for (int k = lane * 8; k < K; k += kWave * 8) {  // (a group holds whole eights)
        const uint32_t w = *(const uint32_t*)(q + k / 2);
        const double s = (double)(float)scale[k >> shift], z = zero ? (double)(float)zero[k >> shift] : 8.0;
#pragma unroll
        for (int e = 0; e < 8; ++e) sum += (double)(float)x[k + e] * (((double)(w >> 4 * e & 15) - z) * s);
    }
    for (int d = kWave / 2; d > 0; d >>= 1) sum += __shfl_xor(sum, d);
    return (float)sum;
}

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
        const bool there = m < M && n < N;
        // (a wave's lanes are all in the loop or none)
        uint64_t doubts = __ballot(there && !is_finite(v) && !is_nan((float)X[m * ldx]));
        while (doubts) {
            const int of = __builtin_ctzll(doubts);
            doubts &= doubts - 1;
            const int md = __builtin_amdgcn_readlane(m, of), nd = __builtin_amdgcn_readlane(n, of);
            const float sum64 = by_terms(X + md * ldx, Q + nd * ldq, scale + (int64_t)nd * groups,
                                         ZERO ? zero + (int64_t)nd * groups : nullptr, K, shift, lane);
            v = lane == of ? sum64 : v;
        }
        if (there) Y[(int64_t)m * ldy + n] = (E)v;
    }
}

// ---------------------------------------------------------- many rows of X --
//
// 64 rows of X by 64 FN rows of W per workgroup of sixteen waves, K in blocks
// of 256: x (four tiles of 64 rows by 64 k, 32 KiB) and codes (FN x 8 KiB) in
// LDS rings of three blocks, filled by direct global->LDS loads two blocks
// ahead.  Waves 4 q .. 4 q + 3 take x's tile q of every block; each of the
// four takes all rows of x and 16 FN rows of W, so each code becomes a number
// once per 64 rows of x and the numbers never reach LDS.  The four partial
// sums meet in LDS at the end.  (With four waves walking all of K, one to a
// SIMD, the chain from a barrier through LDS, the unpacking and the matrix
// cores to the next stood in full view: 28 us instead of 22 at 256 rows, 4096
// x 4096, binary16.)
//
// Bound by a block's chain and the vector instructions that unpack codes and
// apply scales: 256 rows by 4096 x 4096 take 21 us (24 in bfloat16, whose
// offset needs the sums of x), 128 rows, half as many workgroups, 21; the
// matrix cores are busy 31% of that.  512 rows by 8192 x 8192: 105 us, 655
// TFLOP/s, as FN is 2; 174 in bfloat16.
//
// The codes are the first operand here: lane l's four results belong to row
// l % 16 of x and rows 4 h .. 4 h + 3 of W, eight adjacent bytes of Y.
// Scales therefore come by fours; a block's are kept in LDS by group, read
// from memory a block ahead.  Codes are unpacked in their own order (a byte
// permute, a mask, a packed fused multiply or shift), since x is used by
// one wave's 16 FN rows only and would be permuted more often than they.

template <class E>
struct Unpack;
template <>
struct Unpack<_Float16> {
    // pair (q, q') of a byte: 1024 + q and 1024 + 16 q', made q - 8 and q' - 8
    static constexpr uint32_t magic = 0x64006400u, mask = 0x00f0000fu;
    static __device__ __forceinline__ uint32_t pair(uint32_t b, uint32_t magic, uint32_t mask)
    {
        const half2_t p = __builtin_bit_cast(half2_t, masked(b, mask, magic));
        const half2_t by = {(_Float16)1.0f, (_Float16)0.0625f}, off = {(_Float16)-1032.0f, (_Float16)-72.0f};
        const half2_t v = __builtin_elementwise_fma(p, by, off);
        return __builtin_bit_cast(uint32_t, v);
    }
};
template <>
struct Unpack<__bf16> {
    // 128 + q and 128 + q'
    static constexpr uint32_t magic = 0x43004300u, mask = 0x000f000fu;
    static __device__ __forceinline__ uint32_t pair(uint32_t b, uint32_t magic, uint32_t mask)
    {
        typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
        const u16x2 shift = {0, 4};
        const u16x2 v = __builtin_bit_cast(u16x2, b) >> shift;
        return masked(__builtin_bit_cast(uint32_t, v), mask, magic);
    }
};

// FLUSH: runs of 32 k per sum that a scale is applied to; a wave has two of a
// group at most.
template <class E, int FN, int FLUSH, bool ZERO>
__global__ void __launch_bounds__(1024, 1)
gemm_w4_kernel(const E* __restrict__ X, const unsigned char* __restrict__ Q, const E* __restrict__ scale,
               const E* __restrict__ zero, E* __restrict__ Y, int M, int N, int K, int shift, int groups, int64_t ldx,
               int64_t ldq, int64_t ldy, int tiles_m, int tiles_n, int whole)
{
    using x8 = typename Elem<E>::x8;
    using x4 = typename Elem<E>::x4;
    static_assert(FLUSH <= 2, "a wave's part of a block is two runs");
    constexpr bool SUM = ZERO || !Code<E>::exact;
    constexpr int BM = 64, BN = 64 * FN, NS = 8 / FLUSH;  // scales of a block's row
    constexpr int X_BYTES = 4 * BM * 128, W_BYTES = BN * 128, S_BYTES = NS * BN * 2;
    __shared__ __attribute__((aligned(1024))) unsigned char smem[3 * X_BYTES + 3 * W_BYTES + 4 * S_BYTES];
    static_assert(sizeof(smem) <= 160 * 1024 && 12 * 4096 * FN <= 3 * X_BYTES, "gfx950 has 160 KiB of LDS");
    unsigned char* const xs = smem;
    unsigned char* const ws = smem + 3 * X_BYTES;
    unsigned char* const ss = ws + 3 * W_BYTES;  // two blocks' scales, then two blocks' zero points
    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int q = wave >> 2, part = wave & 3;  // x's tile, and which 16 FN rows of W
    const int r = lane & 15, h = lane >> 4;
    int tm, tn;
    grid_tile(xcd_order(blockIdx.x, tiles_m * tiles_n), tiles_m, tiles_n, tm, tn);
    const int m0 = tm * BM, n0 = tn * BN;
    const uint32_t pitch_x = (uint32_t)ldx * 2u, pitch_q = (uint32_t)ldq;
    const __amdgpu_buffer_rsrc_t bx = make_rsrc(X + (int64_t)m0 * ldx, (uint32_t)min(BM, M - m0) * pitch_x);
    const __amdgpu_buffer_rsrc_t bq = make_rsrc(Q + (int64_t)n0 * ldq, (uint32_t)min(BN, N - n0) * pitch_q);
    const uint32_t s_bytes = (uint32_t)min(BN, N - n0) * (uint32_t)groups * 2u;
    const __amdgpu_buffer_rsrc_t bs = make_rsrc(scale + (int64_t)n0 * groups, s_bytes);
    const __amdgpu_buffer_rsrc_t bz = make_rsrc(ZERO ? zero + (int64_t)n0 * groups : scale, ZERO ? s_bytes : 0u);

    // A load fills eight rows of a tile: row lane / 8, position lane % 8,
    // which the swizzle gives chunk pos ^ ((row / 2) % 8).  Wave 4 q + p loads
    // rows 16 p .. + 15 of x's tile q, and wave w rows 8 w .. + 7 of the codes.
    const int lr = lane >> 3, lp = lane & 7;
    const int c01[2] = {swizzle(lr, lp), swizzle(8 + lr, lp)};
    auto load = [&](int stage, int block) __attribute__((always_inline)) {
        if (wave < 8 * FN) {
            const int c = c01[wave & 1], k = block * kBlock + c * 32;
            const uint32_t off = k < K ? (uint32_t)(wave * 8 + lr) * pitch_q + (uint32_t)(k / 2) : kOob;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(bq, (lds_void*)(ws + stage * W_BYTES + wave * 1024), 16, off, 0, 0,
                                                     0);
        }
#pragma unroll
        for (int l = 0; l < 2; ++l) {
            const int c = c01[l], k = block * kBlock + q * 64 + c * 8;
            const uint32_t off = k < K ? (uint32_t)(part * 16 + l * 8 + lr) * pitch_x + (uint32_t)k * 2u : kOob;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(bx, (lds_void*)(xs + stage * X_BYTES + (wave * 2 + l) * 1024), 16,
                                                     off, 0, 0, 0);
        }
    };
    uint16_t sv = 0, zv = 0;
    const bool has_scale = tid < BN * NS;
    auto load_s = [&](int block) __attribute__((always_inline)) {
        const int k = block * kBlock + 32 * FLUSH * (tid % NS);
        const uint32_t off = k < K && has_scale
                                 ? ((uint32_t)(tid / NS) * (uint32_t)groups + (uint32_t)(k >> shift)) * 2u
                                 : kOob;
        sv = __builtin_amdgcn_raw_buffer_load_b16(bs, off, 0, 0);
        if constexpr (ZERO) zv = __builtin_amdgcn_raw_buffer_load_b16(bz, off, 0, 0);
    };
    auto keep_s = [&](int block) __attribute__((always_inline)) {
        if (has_scale) {
            unsigned char* to = ss + (block & 1) * S_BYTES + (tid % NS * BN + tid / NS) * 2;
            *(uint16_t*)to = sv;
            if constexpr (ZERO) *(uint16_t*)(to + 2 * S_BYTES) = zv;
        }
    };

    f32x4 total[4][FN], acc[4][FN], sum[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) total[i][j] = f32x4{0, 0, 0, 0};
    const u32x4 ones_bits = {Code<E>::ones, Code<E>::ones, Code<E>::ones, Code<E>::ones};
    const x8 ones = __builtin_bit_cast(x8, ones_bits);
    uint32_t magic = Unpack<E>::magic, mask = Unpack<E>::mask;
    asm volatile("" : "+v"(magic), "+s"(mask));

    // This wave's part of block b.
    auto compute = [&](int b, const unsigned char* xt, const unsigned char* wt) __attribute__((always_inline)) {
        // words 0, 1 of lanes h: the codes of the 64 k's runs, from the half of
        // 128 that holds them
        uint32_t w[FN][2];
#pragma unroll
        for (int j = 0; j < FN; ++j) {
            const u32x4 v = across(
                *(const u32x4*)(wt + (part * 16 * FN + 16 * j + r) * 128 + swizzle(r, 4 * (q >> 1) + h) * 16));
            w[j][0] = q & 1 ? v[2] : v[0];
            w[j][1] = q & 1 ? v[3] : v[1];
        }
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            x8 xv[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) xv[i] = *(const x8*)(xt + (16 * i + r) * 128 + swizzle(r, 4 * kk + h) * 16);
            if (kk % FLUSH == 0)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    sum[i] = f32x4{0, 0, 0, 0};
#pragma unroll
                    for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
                }
#pragma unroll
            for (int j = 0; j < FN; ++j) {
                const uint32_t word = w[j][kk];
                const u32x4 bits = {Unpack<E>::pair(__builtin_amdgcn_perm(0, word, 0x0c000c00u), magic, mask),
                                    Unpack<E>::pair(__builtin_amdgcn_perm(0, word, 0x0c010c01u), magic, mask),
                                    Unpack<E>::pair(__builtin_amdgcn_perm(0, word, 0x0c020c02u), magic, mask),
                                    Unpack<E>::pair(__builtin_amdgcn_perm(0, word, 0x0c030c03u), magic, mask)};
                const x8 wv = __builtin_bit_cast(x8, bits);
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[i][j] = Elem<E>::mfma(wv, xv[i], acc[i][j]);
            }
            if constexpr (SUM)
#pragma unroll
                for (int i = 0; i < 4; ++i) sum[i] = Elem<E>::mfma(ones, xv[i], sum[i]);
            if (kk % FLUSH == FLUSH - 1)
#pragma unroll
                for (int j = 0; j < FN; ++j) {
                    const int g = (2 * q + kk) / FLUSH;
                    const unsigned char* at =
                        ss + (b & 1) * S_BYTES + (g * BN + part * 16 * FN + 16 * j + 4 * h) * 2;
                    const x4 s4 = *(const x4*)at;
                    f32x4 z4 = f32x4{8.0f, 8.0f, 8.0f, 8.0f};
                    if constexpr (ZERO) {
                        const x4 v = *(const x4*)(at + 2 * S_BYTES);
                        z4 = f32x4{(float)v[0], (float)v[1], (float)v[2], (float)v[3]};
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            float v = acc[i][j][e];
                            if constexpr (SUM) v = __builtin_fmaf(Code<E>::bias - z4[e], sum[i][e], v);
                            total[i][j][e] = __builtin_fmaf((float)s4[e], v, total[i][j][e]);
                        }
                }
        }
    };

    // At a block's barrier only the next block's two loads of x may be in
    // flight (its codes were issued before them).  The scales' loads go first,
    // so that waiting for them does not mean waiting for the loads behind.
    const int blocks = (K + kBlock - 1) / kBlock;
    load_s(0);
    load(0, 0);
    load(1, 1);
    keep_s(0);
    int st = 0;
    for (int b = 0; b < blocks; ++b) {
        lds_barrier<2>();
        load_s(b + 1);
        load(st == 0 ? 2 : st - 1, b + 2);  // (past the end of K: zeros, never read)
        compute(b, xs + st * X_BYTES + q * (BM * 128), ws + st * W_BYTES);
        keep_s(b + 1);
        st = st == 2 ? 0 : st + 1;
    }
    lds_barrier<0>();  // no load may still be writing LDS when it is used again

    // Partial sums of waves 4 .. 15 through LDS to waves 0 .. 3.
    if (q > 0)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j)
                *(f32x4*)(smem + ((((wave - 4) * 4 + i) * FN + j) * 64 + lane) * 16) = total[i][j];
    __syncthreads();
    if (q > 0) return;
    uint32_t doubts = 0;  // bit (i FN + j) 4 + e: of the lane's results
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int m = m0 + 16 * i + r;
#pragma unroll
        for (int j = 0; j < FN; ++j) {
            f32x4 sum4 = total[i][j];
#pragma unroll
            for (int o = 0; o < 3; ++o)
                sum4 += *(const f32x4*)(smem + ((((o * 4 + part) * 4 + i) * FN + j) * 64 + lane) * 16);
            const int n = n0 + part * 16 * FN + 16 * j + 4 * h;
            if (m >= M) continue;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                doubts |= is_finite(sum4[e]) || n + e >= N ? 0u : 1u << ((i * FN + j) * 4 + e);
            const x4 v = round4<E>(sum4);
            E* y = Y + (int64_t)m * ldy + n;
            if (whole && n + 3 < N) {
                *(x4*)y = v;
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (n + e < N) y[e] = v[e];
            }
        }
    }
    for (int i = 0; i < 4; ++i) {
        const uint32_t row = ((1u << (4 * FN)) - 1) << (i * 4 * FN);
        if ((doubts & row) && is_nan((float)X[(m0 + 16 * i + r) * ldx])) doubts &= ~row;
    }
    while (const uint64_t lanes = __ballot(doubts != 0)) {
        const int of = __builtin_ctzll(lanes);
        const int bit = __builtin_ctz((uint32_t)__builtin_amdgcn_readlane((int)doubts, of)), block = bit >> 2;
        const int m = m0 + 16 * (block / FN) + (of & 15);
        const int n = n0 + part * 16 * FN + 16 * (block % FN) + 4 * (of >> 4) + (bit & 3);
        const float sum64 = by_terms(X + m * ldx, Q + n * ldq, scale + (int64_t)n * groups,
                                     ZERO ? zero + (int64_t)n * groups : nullptr, K, shift, lane);
        if (lane == of) {
            Y[(int64_t)m * ldy + n] = (E)sum64;
            doubts &= doubts - 1;
        }
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
    if (!abi::good_grid((a.N + 16 * R - 1) / (16 * R), kThreads)) return hipErrorInvalidValue;
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

template <class E, int FN, int FLUSH, bool ZERO>
int launch_gemm(const Args& a)
{
    const int64_t tm = (a.M + 63) / 64, tn = (a.N + 64 * FN - 1) / (64 * FN);
    if (!abi::good_grid(tm * tn, 1024)) return hipErrorInvalidValue;
    const int whole = (uintptr_t)a.Y % 8 == 0 && a.ldy % 4 == 0;
    hipLaunchKernelGGL((gemm_w4_kernel<E, FN, FLUSH, ZERO>), dim3((unsigned)(tm * tn)), dim3(1024), 0, a.stream,
                       (const E*)a.X, (const unsigned char*)a.Q, (const E*)a.scale, (const E*)a.zero, (E*)a.Y, (int)a.M,
                       (int)a.N, (int)a.K, a.shift, (int)a.groups, a.ldx, a.ldq, a.ldy, (int)tm, (int)tn, whole);
    return (int)hipGetLastError();
}

// KIND(FLUSH, ZERO) by the group's size and the zero points.
#define BY_GROUP(a, KIND)                                        \
    ((a).shift >= 7   ? ((a).zero ? KIND(4, true) : KIND(4, false)) \
     : (a).shift == 6 ? ((a).zero ? KIND(2, true) : KIND(2, false)) \
                      : ((a).zero ? KIND(1, true) : KIND(1, false)))

template <class E, int MB, int R, bool EIGHTS = true>
int few_rows(const Args& a)
{
#define KIND(FLUSH, ZERO) launch<E, MB, R, FLUSH, ZERO, EIGHTS>(a)
    return BY_GROUP(a, KIND);
#undef KIND
}

template <class E>
int many_rows(const Args& a)
{
    // Twice the rows of W for each read of x where both are enough for all
    // CUs; with the sums of x that zero points (and bfloat16) need, twice the
    // totals do not fit in 128 registers.
    if constexpr (Code<E>::exact)
        if (!a.zero && (a.N + 127) / 128 * ((a.M + 63) / 64) >= 256)
            return a.shift >= 6 ? launch_gemm<E, 2, 2, false>(a) : launch_gemm<E, 2, 1, false>(a);
    if (a.shift >= 6) return a.zero ? launch_gemm<E, 1, 2, true>(a) : launch_gemm<E, 1, 2, false>(a);
    return a.zero ? launch_gemm<E, 1, 1, true>(a) : launch_gemm<E, 1, 1, false>(a);
}

template <class E>
int run(const Args& a)
{
    if ((uintptr_t)a.X % 16 || (a.M > 1 && a.ldx % 8)) return few_rows<E, 1, 1, false>(a);
    // As many rows of W to a workgroup as leave one for every CU.  Up to two
    // workgroups of 32 x 32 a CU that kernel is the faster one (48 rows of X,
    // 4096 x 4096: 11 us against 21; 64 rows, 8192 x 4096: 19 and 19; 256
    // rows, 4096 x 4096: 36 against 22).
    if (a.M <= 16) return (a.N + 15) / 16 >= 2 * 256 ? few_rows<E, 1, 2>(a) : few_rows<E, 1, 1>(a);
    if (a.M <= 32 && (a.N + 15) / 16 < 2 * 256) return few_rows<E, 2, 1>(a);
    if (a.M <= 32 || (a.M + 31) / 32 * ((a.N + 31) / 32) < 2 * 256) return few_rows<E, 2, 2>(a);
    return many_rows<E>(a);
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
