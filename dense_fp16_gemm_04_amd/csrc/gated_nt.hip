// The gated linear layer H = act(X Wg^T) * (X Wu^T) and its backward pass for
// gfx950: include/gated_nt.h.
//
// Forward: one NT product whose B tile is half rows of Wg and half rows of
// Wu, arranged so that each wave's sub-tile holds, for the same columns of H,
// g in its first half and u in its second; the epilogue then combines them
// lane by lane and g and u never leave the registers.
//
// Backward: dG = dH * P and dU = dH * Q element by element from the saved P =
// u act'(g) and Q = act(g), written row-major ([dG dU], T x 2F) and
// transposed (2F x T); then dX = [dG dU] [Wg; Wu] is one product with 2F
// terms to a sum, and dWg, dWu are two of one shape over T, all in NT form on
// transposed copies of X and of the weights.
//
// Measured: binary16 forward 4096 x 4096 x 8192, 371 to 401 us on four MI355X (1480
// to 1370 TFLOP/s, the matrix cores busy 87% of the cycles).  bfloat16 step 8192 x
// 4096 x 8192, 2473 to 2586 us on as many; 2584 of one trace are the forward pass
// 798, the gradients' operands 344 at 4.7 TB/s, and the two products 721 each.
#include "gated_nt.h"

#include <algorithm>

#include "abi.h"
#include "nt_launch.h"
#include "relayout.h"

namespace {

using namespace nt;

// act(g) = g * sigmoid(g * (c0 + c1 * g^2)): silu has c0 = 1, c1 = 0; the
// tanh form of gelu has 0.5 g (1 + tanh y) = g sigmoid(2 y).
struct Activation {
    float c0, c1;
};

// One activation's value and derivative.  exp2 and rcp are the hardware's
// (1 ulp): 2^-22 relative beside the 2^-12 of the narrowest result.  Where
// exp2 overflows, rcp gives the limit 0.  The sigmoid's argument is taken of
// g held within +-2^13, where it is 0 or 1 long since: an infinite g would
// make 0 * inf of a zero c1, a large one overflow its square.
__device__ __forceinline__ float bounded(float g) { return __builtin_amdgcn_fmed3f(g, -8192.0f, 8192.0f); }
__device__ __forceinline__ float act_value(const Activation& c, float g, float& s)
{
    const float x = bounded(g);
    const float z = x * __builtin_fmaf(c.c1 * x, x, c.c0);
    s = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504f * z));
    return g * s;
}
__device__ __forceinline__ float act_slope(const Activation& c, float g, float s)
{
    const float x = bounded(g);
    const float dz = __builtin_fmaf(3.0f * c.c1 * x, x, c.c0);
    return __builtin_fmaf(g * s * (1.0f - s), dz, s);
}

// `saved` in blocks of 16 x 16, row of blocks by row: P of a block, then Q,
// each as 64 times four values in the order in which a wave's lanes hold
// them (lane l: row l % 16, columns 4 (l / 16) .. + 3), so that a wave stores
// and loads 1 KiB at once.
__host__ __device__ __forceinline__ int64_t blocks_of(int64_t n) { return (n + 15) / 16; }
constexpr int kBlockFloats = 512;

template <class E, bool SAVE, bool EIGHTS>
struct GatedOp {
    static constexpr bool kPersist = true, kSplit = false;
    const E *X, *Wg, *Wu;
    E* H;
    float* saved;
    int M, F, K, lda, ldg, ldu, ldh, tiles, tiles_m, tiles_n;
    Activation act;

    template <int BM, int BN>
    __device__ __forceinline__ void tile(int id, Tile& t) const
    {
        int tm, tn;
        grid_tile(xcd_order(id, tiles), tiles_m, tiles_n, tm, tn);
        t.m0 = tm * BM;
        t.n0 = tn * (BN / 2);
        t.batch = 0;
    }
    __device__ __forceinline__ const E* a_rows(const Tile& t, int row, int& n) const
    {
        return rows_from(X, t.m0 + row, M, lda, n);
    }
    // A wave's WTN rows of the B tile are WTN / 2 of Wg, then the same of Wu.
    template <int WTN>
    __device__ __forceinline__ const E* b_rows(const Tile& t, int row, int& n) const
    {
        const bool up = row % WTN >= WTN / 2;
        return rows_from(up ? Wu : Wg, t.n0 + row / WTN * (WTN / 2) + row % (WTN / 2), F, up ? ldu : ldg, n);
    }
    template <int WTN>
    __device__ __forceinline__ int b_pitch(int row) const
    {
        return row % WTN >= WTN / 2 ? ldu : ldg;
    }
    template <class T>
    __device__ __forceinline__ void epilogue(const Tile& t, const f32x4 (&acc)[T::FM][T::FN], int lane, int wave,
                                             unsigned char* s0, unsigned char* s1) const
    {
        constexpr int HF = T::FN / 2;
        // the tile's rows of blocks of `saved` (below 2^31 bytes)
        const int bf = (int)blocks_of(F);
        const uint32_t pitch_s = (uint32_t)bf * (kBlockFloats * 4u);
        __amdgpu_buffer_rsrc_t rs;
        if constexpr (SAVE)
            rs = make_rsrc((unsigned char*)saved + (int64_t)(t.m0 / 16) * pitch_s,
                           (uint32_t)min(T::BM / 16, (int)blocks_of(M) - t.m0 / 16) * pitch_s);
        auto value = [&](int i, int j) __attribute__((always_inline)) {
            const f32x4 g4 = acc[i][j], u4 = acc[i][j + HF];
            f32x4 h, p, q;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float g = g4[e], u = u4[e];
                float s;
                q[e] = act_value(act, g, s);
                h[e] = q[e] * u;
                if constexpr (SAVE) p[e] = u * act_slope(act, g, s);
            }
            if constexpr (SAVE) {
                __builtin_amdgcn_sched_barrier(0);  // (block by block, for the registers' sake)
                const int b = (t.n0 + wave % T::WAVES_N * (T::WTN / 2)) / 16 + j;
                const uint32_t row = as_vector(pitch_s) * (uint32_t)(wave / T::WAVES_N * T::FM + i);
                const uint32_t at = (b < bf ? row + (uint32_t)b * (kBlockFloats * 4u) : kOob) + pinned(lane) * 16u;
                __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, p), rs, at, 0, 0);
                // (the distance is part of the vector offset, which makes it an
                // immediate.  Given as the scalar offset it takes a register,
                // after which the compiler lets the next instruction write the
                // store's data registers: the first of them then came out
                // wrong now and then in the last lanes of each sixteen.)
                __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, q), rs, at + kBlockFloats * 2u, 0, 0);
            }
            return round4<E>(h);
        };
        write_rows<T, HF, EIGHTS>(value, rows_at(H, t.m0, M, T::BM, ldh, t.n0, F), lane, wave, s0, s1);
    }
};

// The forward pass of up to 16 MB rows of X, where reading the weights is all the
// work: a workgroup of eight waves takes G rows of each weight, and the waves
// take K's steps of 64 in turn.  Each has an LDS ring of its own, filled by
// direct loads (whole 128-byte lines to eight adjacent lanes) and waited for
// without barriers; the eight partial sums meet in LDS.  Bound by the weights'
// bytes: one row by 8192 x 4096 twice 27.7 us, 4.85 TB/s.
constexpr int kFewWaves = 8;

template <class E, int MB, int G, bool SAVE>
__global__ void __launch_bounds__(kFewWaves * kWave, 2) gated_few(const GatedOp<E, SAVE, true> op)
{
    using x8 = typename Elem<E>::x8;
    constexpr int NB = 2 * G / 16;                               // blocks of 16 weight rows
    constexpr int X_LOADS = 2 * MB, LOADS = X_LOADS + 2 * G / 8;  // eight rows each
    constexpr int STAGE = LOADS * 1024, S = LOADS == 4 ? 4 : 3, PITCH = 20;
    static_assert(MB * NB * 16 * PITCH * 4 <= S * STAGE, "the partial sums fit");
    __shared__ __attribute__((aligned(1024))) unsigned char smem[kFewWaves * S * STAGE];
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    unsigned char* const mine = smem + wave * (S * STAGE);
    const int r = lane & 15, h = lane >> 4;
    const int n0 = blockIdx.x * G, K = op.K;
    const uint32_t rows = (uint32_t)min(G, op.F - n0);
    const uint32_t pitch_g = (uint32_t)op.ldg * 2u, pitch_u = (uint32_t)op.ldu * 2u, pitch_x = (uint32_t)op.lda * 2u;
    const __amdgpu_buffer_rsrc_t bg = make_rsrc(op.Wg + (int64_t)n0 * op.ldg, rows * pitch_g);
    const __amdgpu_buffer_rsrc_t bu = make_rsrc(op.Wu + (int64_t)n0 * op.ldu, rows * pitch_u);
    const __amdgpu_buffer_rsrc_t bx = make_rsrc(op.X, (uint32_t)op.M * pitch_x);
    const int lr = lane >> 3, lp = lane & 7;
    const int c01[2] = {swizzle(lr, lp), swizzle(8 + lr, lp)};
    // rows of the stage: x's, then G of Wg, then G of Wu
    auto issue = [&](int slot, int ks) __attribute__((always_inline)) {
#pragma unroll
        for (int l = 0; l < LOADS; ++l) {
            const int c = c01[l & 1], w = l - X_LOADS;
            const bool up = w >= G / 8;
            const uint32_t row = (uint32_t)((l < X_LOADS ? l : up ? w - G / 8 : w) * 8 + lr);
            const uint32_t at = row * (l < X_LOADS ? pitch_x : up ? pitch_u : pitch_g) + (uint32_t)(ks * 128 + c * 16);
            const uint32_t off = c * 8 < K - ks * 64 ? at : kOob;
            lds_void* to = (lds_void*)(mine + slot * STAGE + l * 1024);
            if (l < X_LOADS)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(bx, to, 16, off, 0, 0, 0);
            else if (!up)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(bg, to, 16, off, 0, 0, 0);
            else
                __builtin_amdgcn_raw_ptr_buffer_load_lds(bu, to, 16, off, 0, 0, 0);
        }
    };
    f32x4 acc[MB][NB];
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
    const int nk = (K + 63) / 64;
#pragma unroll
    for (int s = 0; s < S - 1; ++s) issue(s, wave + s * kFewWaves);
    int cur = 0, fill = S - 1;
    for (int ks = wave; ks < nk; ks += kFewWaves) {
        // the step's loads have landed, and the last step's reads are back:
        // its slot may be filled (past the end: with zeros, never read)
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"i"((S - 2) * LOADS) : "memory");
        issue(fill, ks + (S - 1) * kFewWaves);
        const unsigned char* base = mine + cur * STAGE + r * 128;
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            const int pos = swizzle(r, 4 * kk + h) * 16;
            x8 fx[MB];
#pragma unroll
            for (int i = 0; i < MB; ++i) fx[i] = *(const x8*)(base + i * 2048 + pos);
#pragma unroll
            for (int j = 0; j < NB; ++j) {
                const x8 fw = *(const x8*)(base + (MB + j) * 2048 + pos);
#pragma unroll
                for (int i = 0; i < MB; ++i) acc[i][j] = Elem<E>::mfma(fw, fx[i], acc[i][j]);
            }
        }
        cur = cur + 1 == S ? 0 : cur + 1;
        fill = fill + 1 == S ? 0 : fill + 1;
    }
    lds_barrier<0>();  // no load may still be writing LDS when it is used again
    // the lane has row 16 i + r of x, weight rows 4 h .. + 3 of block j
    float* part = (float*)smem;
    constexpr int WAVE = NB * 16 * MB * PITCH;
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j)
            *(f32x4*)(part + wave * WAVE + ((j * MB + i) * 16 + r) * PITCH + 4 * h) = acc[i][j];
    __syncthreads();
    const int t = threadIdx.x / G, c = threadIdx.x % G, f = n0 + c;
    if (t >= op.M || f >= op.F) return;  // (which t below 16 MB is)
    float g = 0.0f, u = 0.0f;
#pragma unroll
    for (int w = 0; w < kFewWaves; ++w) {
        const float* at = part + w * WAVE + t * PITCH + c;
        g += at[0];
        u += at[NB == 2 ? 16 * MB * PITCH : G];
    }
    float s;
    const float q = act_value(op.act, g, s);
    op.H[(int64_t)t * op.ldh + f] = (E)(q * u);
    if constexpr (SAVE) {
        float* at = op.saved + ((int64_t)(t / 16) * blocks_of(op.F) + f / 16) * kBlockFloats +
                    (t % 16 + 16 * (f % 16 / 4)) * 4 + f % 4;
        at[0] = u * act_slope(op.act, g, s);
        at[kBlockFloats / 2] = q;
    }
}

// binary16 ends at 2^-24, and gradients often lie near it: dG and dU are
// therefore held times a power of two that brings dH's largest finite entry to
// 2^-4 .. 2^-3, which leaves them 2^19 upwards (P and Q are about 1) and, below,
// full precision to 2^-10 of that entry; the products' epilogues take it out.
// (dW's error for dH of 1e-5 and 1e-6, 512 rows: 2.8e-3 and 2.7e-2 without;
// 3.0e-4 and 1.2e-3 with, of which its own rounding 2.2e-4 and 1.2e-3.)
// bfloat16 has the range of 32 bits and needs none.
template <class E>
constexpr bool kScaled = false;
template <>
constexpr bool kScaled<_Float16> = true;
constexpr int kMostBlocks = 1024;  // (8 MB of loads in flight)

// Largest finite magnitudes of dH, one to a workgroup, as bits; and the factor
// of products of nothing.
struct Most {
    const _Float16* dH;
    int64_t lddh;
    int T, F, vec;
    uint32_t* most;
    float* factor;

    __device__ __forceinline__ void run(int id) const
    {
        if (T == 0 || F == 0) {
            if (id == 0 && threadIdx.x == 0) *factor = 1.0f;
            return;
        }
        uint32_t m = 0;
        relayout::each_four(dH, lddh, T, F, vec, id, kMostBlocks, [&](const relayout::Four<_Float16>& v) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t bits = __builtin_bit_cast(uint16_t, v[e]) & 0x7fffu;
                m = max(m, bits < 0x7c00u ? bits : 0u);
            }
        });
        for (int d = 32; d > 0; d >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d));
        __shared__ uint32_t part[4];
        if (threadIdx.x % 64 == 0) part[threadIdx.x / 64] = m;
        __syncthreads();
        if (threadIdx.x == 0) most[id] = max(max(part[0], part[1]), max(part[2], part[3]));
    }
};

// The power of two, the same in every workgroup of 256 threads.
__device__ __forceinline__ int scale_of(const uint32_t* most, uint32_t (&part)[4])
{
    static_assert(kMostBlocks == 4 * relayout::kThreads, "four to a thread");
    const u32x4 four = ((const u32x4*)most)[threadIdx.x];
    uint32_t m = max(max(four[0], four[1]), max(four[2], four[3]));
    for (int d = 32; d > 0; d >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d));
    if (threadIdx.x % 64 == 0) part[threadIdx.x / 64] = m;
    __syncthreads();
    m = max(max(part[0], part[1]), max(part[2], part[3]));
    const float f = (float)__builtin_bit_cast(_Float16, (uint16_t)m);
    return m ? -4 - ilogbf(f) : 0;
}

// dG = dH * P, dU = dH * Q for a 64 x 64 tile: row-major into rows of dGU
// (dG at column 0, dU at column Fp), transposed into dGT and dUT (pitch Tp).
// Rows and columns past the end, up to Tp and Fp, become zeros.
// dH comes in by rows and turns in LDS to the blocks that `saved` holds.
// Bound by its bytes: 2 + 8 read, 8 written per element.
template <class E>
struct Slopes {
    const E* dH;
    const float* saved;
    E *dGU, *dGT, *dUT;
    int T, F, Fp, Tp, vec;
    int64_t lddh;
    const uint32_t* most;  // (kScaled) of dH
    float* factor;         // what takes the power of two out of the products

    __host__ __device__ int64_t tiles() const
    {
        return (int64_t)((Tp + relayout::kTile - 1) / relayout::kTile) * ((Fp + relayout::kTile - 1) / relayout::kTile);
    }
    __device__ __forceinline__ void run(int id, E* tg, E* tu) const;
};

template <class E>
__device__ __forceinline__ void Slopes<E>::run(int id, E* tg, E* tu) const
{
    using x4 = typename Elem<E>::x4;
    using namespace relayout;
    const int tiles_f = (Fp + kTile - 1) / kTile;
    const int t0 = id / tiles_f * kTile, f0 = id % tiles_f * kTile;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int x = threadIdx.x & 15, y = threadIdx.x >> 4;
    // wave w takes the blocks of rows 16 w .. + 15; their P and Q first
    const int64_t bt = t0 / 16 + wave, bf0 = f0 / 16, bf = blocks_of(F);
    f32x4 p[4], q[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        p[j] = q[j] = f32x4{0, 0, 0, 0};
        if (bt * 16 < T && bf0 + j < bf) {
            const float* at = saved + (bt * bf + bf0 + j) * kBlockFloats + lane * 4;
            p[j] = *(const f32x4*)at;
            q[j] = *(const f32x4*)(at + kBlockFloats / 2);
        }
    }
#pragma unroll
    for (int it = 0; it < 4; ++it) {
        const int r = it * 16 + y;
        x4 d = {};
        if (t0 + r < T) d = load4(dH + (int64_t)(t0 + r) * lddh, f0 + x * 4, F, vec);
        *(x4*)(tg + r * kPitch + x * 4) = d;
    }
    float scale = 1.0f;
    if constexpr (kScaled<E>) {
        __shared__ uint32_t part[4];
        const int k = scale_of(most, part);  // (meets the other waves)
        scale = ldexpf(1.0f, k);
        if (id == 0 && threadIdx.x == 0) *factor = ldexpf(1.0f, -k);
    } else {
        __syncthreads();
    }
    const int row = wave * 16 + (lane & 15);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int at = row * kPitch + j * 16 + 4 * (lane >> 4);
        const x4 d = *(const x4*)(tg + at);
        x4 vg, vu;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            // (of a row or column that is not there P and Q may be anything:
            // an infinite weight times the zeros past the end is NaN)
            const bool there = t0 + row < T && f0 + j * 16 + 4 * (lane >> 4) + e < F;
            vg[e] = (E)(there ? (float)d[e] * scale * p[j][e] : 0.0f);
            vu[e] = (E)(there ? (float)d[e] * scale * q[j][e] : 0.0f);
        }
        *(x4*)(tg + at) = vg;  // (each element of dH is read by one lane, this one)
        *(x4*)(tu + at) = vu;
    }
    __syncthreads();
    const int f = f0 + x * 4;
#pragma unroll
    for (int it = 0; it < 4; ++it) {
        const int r = it * 16 + y;
        if (t0 + r < T && f < Fp) {
            E* to = dGU + (int64_t)(t0 + r) * 2 * Fp;
            *(x4*)(to + f) = *(const x4*)(tg + r * kPitch + x * 4);
            *(x4*)(to + Fp + f) = *(const x4*)(tu + r * kPitch + x * 4);
        }
    }
    store_transposed(tg, dGT, Tp, t0, f0, Tp, F);
    store_transposed(tu, dUT, Tp, t0, f0, Tp, F);
}

// All that the backward pass's products read: the slopes and up to three
// transposes, a 64 x 64 tile to a workgroup, in one launch.  In binary16 the
// slopes wait for dH's largest entry, which a launch before theirs finds beside
// the transposes (1000 x 1032 x 2730: 73 us for the whole pass, 76 in a launch of
// its own and the rest in one, 66 in bfloat16).
template <class E>
struct Prepare {
    Most most;
    Slopes<E> slopes;
    relayout::Transpose<E> turn[3];
    int first[3];  // the transposes' first workgroups
};

template <class E, bool SLOPES>
__global__ void __launch_bounds__(relayout::kThreads) gated_prepare(const Prepare<E> p)
{
    __shared__ E tiles[2][relayout::kTile * relayout::kPitch];
    const int id = blockIdx.x;
    if (id < p.first[0]) {
        if constexpr (SLOPES)
            p.slopes.run(id, tiles[0], tiles[1]);
        else
            p.most.run(id);
    } else if (id < p.first[1]) {
        p.turn[0].run(id - p.first[0], tiles[0]);
    } else if (id < p.first[2]) {
        p.turn[1].run(id - p.first[1], tiles[0]);
    } else {
        p.turn[2].run(id - p.first[2], tiles[0]);
    }
}

template <class E>
__global__ void __launch_bounds__(relayout::kThreads) gated_slopes(const Slopes<E> slopes)
{
    __shared__ E tiles[2][relayout::kTile * relayout::kPitch];
    slopes.run(blockIdx.x, tiles[0], tiles[1]);
}

// ------------------------------------------------------------------ host --

bool vec4(const void* p, int64_t ld) { return (uintptr_t)p % 8 == 0 && ld % 4 == 0; }
bool vec8(const void* p, int64_t ld) { return (uintptr_t)p % 16 == 0 && ld % 8 == 0; }
// a result's rows take eight columns at a time
bool eights(const void* p, int64_t cols, int64_t ld) { return vec8(p, ld) && cols % 8 == 0; }

// C [M, N] = A B^T (kScaled: times *factor), all operands with K
// elements to a row; with a second A and C, two products with the same B at once.
template <class E>
int product(const E* A0, const E* A1, const E* B, E* C0, E* C1, int64_t M, int64_t N, int64_t K, int64_t ldc0, int64_t ldc1,
            const float* factor, float* partial, hipStream_t stream)
{
    auto with = [&](auto op) {
        op.factor = factor;
        op.A[0] = A0;
        op.A[1] = A1;
        op.B = B;
        op.C[0] = C0;
        op.C[1] = C1;
        op.M = (int)M;
        op.N = (int)N;
        op.K = op.lda = op.ldb = (int)K;
        op.ldc[0] = (int)ldc0;
        op.ldc[1] = (int)ldc1;
        return launch_grid<E>(op, M, N, 1, A1 ? 2 : 1, K, partial, stream);
    };
    return eights(C0, N, ldc0) && (!A1 || eights(C1, N, ldc1)) ? with(StoreOp<E, true, kScaled<E>>{})
                                                               : with(StoreOp<E, false, kScaled<E>>{});
}

// Rows of what is copied, transposed or computed for the products start on 128
// bytes: the 64 x 64 tiles that write them then write whole cache lines (by 16 bytes, lines are shared by
// workgroups of different XCDs, whose L2s write parts of them: 2595 x 264 x
// 13232 backward 320 us, and 250 by lines; 6872 x 1551 x 2957 425 and 360).
constexpr int64_t kLine = 64;

// Copies of the operands that the kernels cannot read in place.
template <class E>
struct ForwardSpace {
    E *x, *g, *u;  // null: read in place
    int64_t bytes;
    bool copy_x, copy_g, copy_u;
    ForwardSpace(void* base, const void* X, const void* Wg, const void* Wu, int64_t T, int64_t D, int64_t F, int64_t ldx,
                 int64_t ldg, int64_t ldu)
    {
        abi::Carve c(base);
        // a row's last chunk is read whole: K % 8 == 0 as well
        copy_x = D % 8 || !vec8(X, ldx);
        copy_g = D % 8 || !vec8(Wg, ldg);
        copy_u = D % 8 || !vec8(Wu, ldu);
        const int64_t ld = abi::up(D, kLine);
        x = copy_x ? c.take<E>(T * ld) : nullptr;
        g = copy_g ? c.take<E>(F * ld) : nullptr;
        u = copy_u ? c.take<E>(F * ld) : nullptr;
        bytes = c.used();
    }
};

template <class E>
struct BackwardSpace {
    E *wt, *xt, *dgu, *dgt, *dut;
    float *partial, *factor;
    uint32_t* most;
    int64_t Tp, Fp, bytes;
    BackwardSpace(void* base, int64_t T, int64_t D, int64_t F)
    {
        abi::Carve c(base);
        Tp = abi::up(T, kLine);
        Fp = abi::up(F, kLine);
        wt = c.take<E>(D * 2 * Fp);
        xt = c.take<E>(D * Tp);
        dgu = c.take<E>(T * 2 * Fp);
        dgt = c.take<E>(F * Tp);
        dut = c.take<E>(F * Tp);
        partial = std::max(2 * Fp, Tp) >= kSplitK ? c.take<float>(kSplitFloats) : nullptr;
        factor = c.take<float>(1);
        most = c.take<uint32_t>(kMostBlocks);
        bytes = c.used();
    }
};

Activation activation_of(int32_t a)
{
    if (a == GATED_NT_SILU) return {1.0f, 0.0f};
    return {1.59576912f, 0.0713548163f};  // 2 sqrt(2 / pi), 0.044715 times that
}

bool good_sizes(int64_t T, int64_t D, int64_t F)
{
    // a row of [dG dU] has 2F elements (and padding)
    return abi::good_dim(T) && D >= 0 && D <= abi::kMaxPitch - 63 && F >= 0 && 2 * F <= abi::kMaxPitch - 127 &&
           T <= abi::kMaxDim - 256;
}

template <class E, bool SAVE, bool EIGHTS>
int forward(const E* X, const E* Wg, const E* Wu, E* H, float* saved, int64_t T, int64_t D, int64_t F, int64_t ldx,
            int64_t ldg, int64_t ldu, int64_t ldh, int32_t activation, void* workspace, hipStream_t stream)
{
    const ForwardSpace<E> w(workspace, X, Wg, Wu, T, D, F, ldx, ldg, ldu);
    const int64_t Dp = abi::up(D, 8), copied_ld = abi::up(D, kLine);
    GatedOp<E, SAVE, EIGHTS> op = {};
    op.X = X;
    op.Wg = Wg;
    op.Wu = Wu;
    op.lda = (int)ldx;
    op.ldg = (int)ldg;
    op.ldu = (int)ldu;
    op.K = (int)Dp;
    relayout::Copies<E> copies = {};
    auto copied = [&](bool copy, const E*& src, int& ld, E* dst, int64_t rows) {
        if (!copy) return;
        copies.job[copies.jobs++] = {src, dst, ld, rows};
        src = dst;
        ld = (int)copied_ld;
    };
    copied(w.copy_x, op.X, op.lda, w.x, T);
    copied(w.copy_g, op.Wg, op.ldg, w.g, F);
    copied(w.copy_u, op.Wu, op.ldu, w.u, F);
    if (copies.jobs && Dp) {
        const int64_t work = std::max(T, F) * (copied_ld / 4);
        hipLaunchKernelGGL(relayout::copy_rows<E>, dim3((unsigned)std::min<int64_t>((work + 255) / 256, 16384), copies.jobs),
                           dim3(relayout::kThreads), 0, stream, copies, (int)D, (int)copied_ld);
        const int rc = (int)hipGetLastError();
        if (rc) return rc;
    }
    op.H = H;
    op.saved = saved;
    op.M = (int)T;
    op.F = (int)F;
    op.ldh = (int)ldh;
    op.act = activation_of(activation);
    // Few rows and too few columns of H for a tile on every CU.  (One row by
    // 8192 x 1024 twice 11 us, as tiles 33; 8192 x 2560 18 and 34; 8192 x 4096
    // 28 and 37; 8192 x 5120 38 and 38, 2048 x 5120 12.8 and 11.8.  32 rows:
    // 8192 x 1024 16 and 34, 8192 x 4096 36 and 39, 4096 x 8000 37 and 26.)
    if (T <= 32 && F <= 16 * num_cus()) {
        auto few = __builtin_bit_cast(GatedOp<E, SAVE, true>, op);
        auto with = [&](auto kernel, int columns) {
            hipLaunchKernelGGL(kernel, dim3((unsigned)((F + columns - 1) / columns)), dim3(kFewWaves * kWave), 0, stream, few);
            return (int)hipGetLastError();
        };
        if (T > 16) return with(gated_few<E, 2, 8, SAVE>, 8);
        // (8192 x 1792: 12 us by 8 columns, 15 by 16; 8192 x 2304: 21 and 18)
        return F <= 8 * num_cus() ? with(gated_few<E, 1, 8, SAVE>, 8) : with(gated_few<E, 1, 16, SAVE>, 16);
    }
    return launch_grid<E>(op, T, F, 2, 1, Dp, nullptr, stream);
}

template <class E>
int backward(const E* dH, const E* X, const E* Wg, const E* Wu, const float* saved, E* dX, E* dWg, E* dWu, int64_t T,
             int64_t D, int64_t F, int64_t lddh, int64_t ldx, int64_t ldg, int64_t ldu, int64_t lddx, int64_t lddg,
             int64_t lddu, void* workspace, hipStream_t stream)
{
    const BackwardSpace<E> w(workspace, T, D, F);
    int rc;
    Prepare<E> p = {};
    p.slopes = {dH, saved, w.dgu, w.dgt, w.dut, (int)T, (int)F, (int)w.Fp, (int)w.Tp, (int)vec4(dH, lddh), lddh,
                w.most, w.factor};
    if (T > 0) {
        // [Wg; Wu]^T, D x 2 Fp, zeros between the two
        p.turn[0] = {Wg, w.wt, ldg, 2 * w.Fp, (int)F, (int)D, (int)w.Fp, (int)vec4(Wg, ldg)};
        p.turn[1] = {Wu, w.wt + w.Fp, ldu, 2 * w.Fp, (int)F, (int)D, (int)w.Fp, (int)vec4(Wu, ldu)};
    }
    if (F > 0) p.turn[2] = {X, w.xt, ldx, w.Tp, (int)T, (int)D, (int)w.Tp, (int)vec4(X, ldx)};
    const int64_t slopes = p.slopes.tiles();
    int64_t n = kScaled<E> ? kMostBlocks : slopes;
    for (int i = 0; i < 3; ++i) {
        p.first[i] = (int)n;
        n += p.turn[i].tiles();
    }
    // (nothing is enqueued yet)
    if (!abi::good_grid(std::max(n, slopes), relayout::kThreads)) return hipErrorInvalidValue;
    if constexpr (kScaled<E>) p.most = {dH, lddh, (int)T, (int)F, p.slopes.vec, w.most, w.factor};
    if (n > 0) {
        hipLaunchKernelGGL((gated_prepare<E, !kScaled<E>>), dim3((unsigned)n), dim3(relayout::kThreads), 0, stream, p);
        if ((rc = (int)hipGetLastError())) return rc;
    }
    if constexpr (kScaled<E>)
        if (slopes > 0) {
            hipLaunchKernelGGL(gated_slopes<E>, dim3((unsigned)slopes), dim3(relayout::kThreads), 0, stream, p.slopes);
            if ((rc = (int)hipGetLastError())) return rc;
        }
    if (T > 0 && D > 0) {
        rc = product<E>(w.dgu, nullptr, w.wt, dX, nullptr, T, D, 2 * w.Fp, lddx, 0, w.factor, w.partial, stream);
        if (rc) return rc;
    }
    if (F > 0 && D > 0) {
        rc = product<E>(w.dgt, w.dut, w.xt, dWg, dWu, F, D, w.Tp, lddg, lddu, w.factor, w.partial, stream);
        if (rc) return rc;
    }
    return hipSuccess;
}

}  // namespace

extern "C" {

int gated_nt_version(void) { return GATED_NT_VERSION; }

int64_t gated_nt_saved_bytes(int64_t T, int64_t F)
{
    if (!good_sizes(T, 0, F)) return -1;
    return blocks_of(T) * blocks_of(F) * kBlockFloats * 4;
}

int64_t gated_nt_workspace(const void* X, const void* Wg, const void* Wu, int64_t T, int64_t D, int64_t F, int64_t ldx,
                           int64_t ldg, int64_t ldu)
{
    if (!good_sizes(T, D, F)) return -1;
    return ForwardSpace<_Float16>(nullptr, X, Wg, Wu, T, D, F, ldx, ldg, ldu).bytes;
}

int64_t gated_nt_backward_workspace(int64_t T, int64_t D, int64_t F)
{
    if (!good_sizes(T, D, F)) return -1;
    return BackwardSpace<_Float16>(nullptr, T, D, F).bytes;
}

int gated_nt(const void* X, const void* Wg, const void* Wu, void* H, void* saved, int64_t T, int64_t D, int64_t F,
             int64_t ldx, int64_t ldg, int64_t ldu, int64_t ldh, int32_t type, int32_t activation, void* workspace,
             int64_t workspace_bytes, hipStream_t stream)
{
    using namespace abi;
    if (!good_sizes(T, D, F)) return hipErrorInvalidValue;
    if (!good_pitch(ldx, D) || !good_pitch(ldg, D) || !good_pitch(ldu, D) || !good_pitch(ldh, F))
        return hipErrorInvalidValue;
    if (type != GATED_NT_F16 && type != GATED_NT_BF16) return hipErrorInvalidValue;
    if (activation != GATED_NT_SILU && activation != GATED_NT_GELU_TANH) return hipErrorInvalidValue;
    if (T == 0 || F == 0) return hipSuccess;
    if (!nt::fits(T, 2 * F, 1)) return hipErrorInvalidValue;
    if (!good_pointer(X, T, D, 2) || !good_pointer(Wg, F, D, 2) || !good_pointer(Wu, F, D, 2) ||
        !good_pointer(H, T, F, 2) || (uintptr_t)saved % 16 || (uintptr_t)workspace % 16)
        return hipErrorInvalidValue;
    const int64_t need = gated_nt_workspace(X, Wg, Wu, T, D, F, ldx, ldg, ldu);
    if (need > 0 && (!workspace || workspace_bytes < need)) return hipErrorInvalidValue;
    const Range h(H, T, F, ldh, 2), s(saved, 1, saved ? gated_nt_saved_bytes(T, F) : 0, 0, 1);
    const Range w(workspace, 1, need, 0, 1);
    const Range in[] = {Range(X, T, D, ldx, 2), Range(Wg, F, D, ldg, 2), Range(Wu, F, D, ldu, 2)};
    for (const Range& r : in)
        if (h.meets(r) || s.meets(r) || w.meets(r)) return hipErrorInvalidValue;
    if (h.meets(s) || h.meets(w) || s.meets(w)) return hipErrorInvalidValue;
#define FORWARD(E, SAVE, EIGHTS)                                                                                 \
    forward<E, SAVE, EIGHTS>((const E*)X, (const E*)Wg, (const E*)Wu, (E*)H, (float*)saved, T, D, F, ldx, ldg, ldu, \
                            ldh, activation, workspace, stream)
#define FORWARD_OF(E)                                                                  \
    (eights(H, F, ldh) ? (saved ? FORWARD(E, true, true) : FORWARD(E, false, true)) \
                           : (saved ? FORWARD(E, true, false) : FORWARD(E, false, false)))
    return type == GATED_NT_F16 ? FORWARD_OF(_Float16) : FORWARD_OF(__bf16);
#undef FORWARD_OF
#undef FORWARD
}

int gated_nt_backward(const void* dH, const void* X, const void* Wg, const void* Wu, const void* saved, void* dX,
                      void* dWg, void* dWu, int64_t T, int64_t D, int64_t F, int64_t lddh, int64_t ldx, int64_t ldg,
                      int64_t ldu, int64_t lddx, int64_t lddg, int64_t lddu, int32_t type, void* workspace,
                      int64_t workspace_bytes, hipStream_t stream)
{
    using namespace abi;
    if (!good_sizes(T, D, F)) return hipErrorInvalidValue;
    if (!good_pitch(lddh, F) || !good_pitch(ldx, D) || !good_pitch(ldg, D) || !good_pitch(ldu, D) ||
        !good_pitch(lddx, D) || !good_pitch(lddg, D) || !good_pitch(lddu, D))
        return hipErrorInvalidValue;
    if (up(T, kLine) > kMaxPitch) return hipErrorInvalidValue;  // rows of the transposed operands
    if (!nt::fits(T, D, 1) || !nt::fits(F, D, 2)) return hipErrorInvalidValue;
    if (type != GATED_NT_F16 && type != GATED_NT_BF16) return hipErrorInvalidValue;
    if (!good_pointer(dH, T, F, 2) || !good_pointer(X, T, D, 2) || !good_pointer(Wg, F, D, 2) ||
        !good_pointer(Wu, F, D, 2) || !good_pointer(saved, T, F, 16) || !good_pointer(dX, T, D, 2) ||
        !good_pointer(dWg, F, D, 2) || !good_pointer(dWu, F, D, 2) || (uintptr_t)workspace % 16)
        return hipErrorInvalidValue;
    const int64_t need = gated_nt_backward_workspace(T, D, F);
    if (need > 0 && (!workspace || workspace_bytes < need)) return hipErrorInvalidValue;
    const Range in[] = {Range(dH, T, F, lddh, 2), Range(X, T, D, ldx, 2), Range(Wg, F, D, ldg, 2),
                        Range(Wu, F, D, ldu, 2), Range(saved, 1, gated_nt_saved_bytes(T, F), 0, 1)};
    const Range out[] = {Range(dX, T, D, lddx, 2), Range(dWg, F, D, lddg, 2), Range(dWu, F, D, lddu, 2),
                         Range(workspace, 1, need, 0, 1)};
    for (int i = 0; i < 4; ++i) {
        for (const Range& r : in)
            if (out[i].meets(r)) return hipErrorInvalidValue;
        for (int k = 0; k < i; ++k)
            if (out[i].meets(out[k])) return hipErrorInvalidValue;
    }
#define BACKWARD(E)                                                                                                    \
    backward<E>((const E*)dH, (const E*)X, (const E*)Wg, (const E*)Wu, (const float*)saved, (E*)dX, (E*)dWg, (E*)dWu, T, \
                D, F, lddh, ldx, ldg, ldu, lddx, lddg, lddu, workspace, stream)
    return type == GATED_NT_F16 ? BACKWARD(_Float16) : BACKWARD(__bf16);
#undef BACKWARD
}

}  // extern "C"
