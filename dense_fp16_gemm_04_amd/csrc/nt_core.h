// Tiled NT products (both operands row-major, k contiguous) on gfx950, with
// the operands' rows and the epilogue supplied by an operation OP.
//
// Three kernels share one scheme: a BM x BN tile of the accumulator per
// workgroup, K in steps of 64, operand tiles in an LDS ring filled by direct
// global->LDS loads, and v_mfma_f32_16x16x32 with 32-bit accumulators.
//   nt_persist  256 x 256, four waves, one workgroup per CU walking its tiles
//   nt_ordered  256 x 128 and 128 x 128, eight waves, four of which load
//   nt_tile     64 x 64, four waves, scheduled by the compiler
// A wave holds a WTM x WTN sub-tile as FM x FN blocks of 16 x 16: lane l has,
// of block (i, j), row l % 16 and columns 4 * (l / 16) .. + 3 (the B fragment
// is the MFMA's first operand, which gives the block transposed: four
// consecutive columns per lane).
//
// OP has, as device functions,
//   tile<BM, BN>(id, Tile&)        what tile number `id` is (row and column
//                                  of its first element, batch);
//   const E* a_rows(t, row, &n)    A's row `row` of the tile's BM and how
//                                  many rows exist from there (rows_from);
//   const E* b_rows<WTN>(t, row, &n)  the same for B, and
//   int b_pitch<WTN>(row)             the pitch of that row's operand: BN / 8
//                                     rows from a multiple of BN / 8 on are
//                                     evenly spaced
//   epilogue<T>(t, acc, lane, wave, s0, s1)
//                                  writes the sub-tiles out, through
//                                  T::STAGE_MAX bytes of LDS: 32 KiB at s0 and
//                                  the rest at s1; a barrier has passed that
//                                  makes them free, and another follows
//   bool outside(t)                (kSplit) nothing of the result is in a
//                                  sub-tile that starts there
//   const E* b_turned(t, &steps, &cols)  (kTurned, nt_ordered alone) B lies the
//                                  other way, k by k, in rows ldb apart: its
//                                  first row from the tile's first column on,
//                                  how many rows exist and how many columns
//                                  (a multiple of 8) from there
// and the fields K (elements, a multiple of 8), lda (A's row pitch in
// elements; pitches are multiples of 8 and below 2^21), tiles.  Every row
// starts on 16 bytes.
#ifndef DENSE_FP16_GEMM_NT_CORE_H
#define DENSE_FP16_GEMM_NT_CORE_H

#include <type_traits>

#include "cdna4.h"

namespace nt {

using namespace cdna4;

struct Tile {
    int m0, n0, batch;
    bool mirror;  // (symmetric results) the tile's transpose is written too
};

// Row `row` of an operand of `rows` rows and the number of rows from there
// on.  Past the end it is row 0 and one row: what is loaded then only reaches
// results that are not stored, and a buffer of no bytes is never made (the
// range check subtracts the scalar offset from the size).
template <class E>
__device__ __forceinline__ const E* rows_from(const E* base, int row, int rows, int ld, int& n)
{
    n = row < rows ? rows - row : 1;
    return base + (row < rows ? (int64_t)row * ld : 0);
}

// WM x WN waves; RS, LS: MFMAs per fragment read and per load (nt_ordered).
template <class E_, int BM_, int BN_, int WM, int WN, int STAGES_, int OCC_, int LOADERS_, int RS_ = 1, int LS_ = 1>
struct Shape {
    using E = E_;
    using x8 = typename Elem<E>::x8;
    static constexpr int BM = BM_, BN = BN_, BK = 64, STAGES = STAGES_, OCC = OCC_;
    static constexpr int WAVES_M = WM, WAVES_N = WN, WAVES = WM * WN, THREADS = WAVES * kWave;
    static constexpr int WTM = BM / WM, WTN = BN / WN;  // a wave's sub-tile
    static constexpr int FM = WTM / 16, FN = WTN / 16;
    static constexpr int ROW_BYTES = 128;
    static constexpr int A_BYTES = BM * ROW_BYTES, B_BYTES = BN * ROW_BYTES;
    static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
    static constexpr int LDS_BYTES = STAGES * STAGE_BYTES, STAGE_MAX = LDS_BYTES;
    static constexpr int LOADERS = LOADERS_;             // waves 0 .. LOADERS - 1 load
    static constexpr int A_LOADS = BM / 8 / LOADERS, B_LOADS = BN / 8 / LOADERS;  // 8 rows each, per wave
    static constexpr int LOADS = A_LOADS + B_LOADS;
    static constexpr int RS = RS_, LS = LS_;
    static_assert(LOADERS == 4 && BM % 64 == 0 && BN % 64 == 0, "a wave loads whole 16-row groups");
    static_assert(LDS_BYTES <= 160 * 1024, "gfx950 has 160 KiB of LDS per workgroup");
    static_assert(STAGES >= 2 && LOADS * (STAGES - 1) <= 63, "vmcnt holds at most 63");
};

template <bool B>
struct Flag {
    static constexpr bool value = B;
};
template <int V>
struct Int {
    static constexpr int value = V;
};

// Whether OP has B k by k.
template <class OP, class = void>
struct Turned : std::false_type {};
template <class OP>
struct Turned<OP, std::enable_if_t<OP::kTurned>> : std::true_type {};

// LDS of such a B: a step's 64 rows of 128 columns, 16 chunks of 16 bytes.  A
// turning read takes 32 bytes of four rows in each 16 lanes, whose places differ
// in four rows' chunks and every other eight rows': 256 bytes apart, on all banks.
__device__ __forceinline__ int turned_swizzle(int k, int chunk) { return chunk ^ ((k & 3) << 1) ^ (((k >> 3) & 1) << 3); }

// The loads of one wave: load l of an operand fills rows 8 l .. 8 l + 7 of
// the wave's quarter of its tile; lane -> row lane / 8, position lane % 8,
// which the swizzle fills with chunk pos ^ ((row / 2) % 8).  (A quarter starts
// at a multiple of 16 rows, so the row's place within it decides.)  B's
// quarter is two operands of BN / 8 rows, which the gated layer needs.
template <class T, bool TURNED = false>
struct Loader {
    __amdgpu_buffer_rsrc_t ra, rb0, rb1;
    uint32_t va[T::A_LOADS], vb[T::B_LOADS];
    int c01[2], wave;
    template <class OP>
    __device__ __forceinline__ Loader(const OP& op, const Tile& t, int lane, int w) : wave(w)
    {
        constexpr int BR = T::BN / 8;
        const int row_b = w * (T::BN / 4);
        const uint32_t pitch_a = (uint32_t)op.lda * 2u;
        const uint32_t pitch_0 = (uint32_t)op.template b_pitch<T::WTN>(row_b) * 2u;
        const uint32_t pitch_1 = (uint32_t)op.template b_pitch<T::WTN>(row_b + BR) * 2u;
        int na = 0, n0 = 0, n1 = 0;
        const void* pa = op.a_rows(t, w * (T::BM / 4), na);
        const void* p0 = op.template b_rows<T::WTN>(t, row_b, n0);
        const void* p1 = op.template b_rows<T::WTN>(t, row_b + BR, n1);
        ra = make_rsrc(pa, (uint32_t)min(na, T::BM / 4) * pitch_a);
        rb0 = make_rsrc(p0, (uint32_t)min(n0, BR) * pitch_0);
        rb1 = make_rsrc(p1, (uint32_t)min(n1, BR) * pitch_1);
        const int lr = lane >> 3, lp = lane & 7;
        c01[0] = swizzle(lr, lp);
        c01[1] = swizzle(8 + lr, lp);
#pragma unroll
        for (int l = 0; l < T::A_LOADS; ++l) va[l] = (uint32_t)(l * 8 + lr) * pitch_a + (uint32_t)c01[l & 1] * 16u;
#pragma unroll
        for (int l = 0; l < T::B_LOADS; ++l) {
            const bool second = l >= T::B_LOADS / 2;
            vb[l] = (uint32_t)((second ? l - T::B_LOADS / 2 : l) * 8 + lr) * (second ? pitch_1 : pitch_0) +
                    (uint32_t)c01[l & 1] * 16u;
        }
    }
    // Load l (A's first) of K step ks into the stage at `base`.  MASKED: the
    // step may reach past K, where chunks read as zero; the K position is then
    // part of the vector offset, since it may exceed the buffer.
    template <class Masked>
    __device__ __forceinline__ void load(unsigned char* base, int l, int ks, int K, Masked) const
    {
        const int lb = l - T::A_LOADS;
        const bool is_a = l < T::A_LOADS;
        uint32_t off = is_a ? va[is_a ? l : 0] : vb[is_a ? 0 : lb], soff = (uint32_t)ks * (T::BK * 2);
        if constexpr (Masked::value) {
            off = c01[l & 1] * 8 < K - ks * T::BK ? off + soff : kOob;
            soff = 0;
        }
        // (a buffer resource cannot be the result of ?:)
        if (is_a)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void*)(base + (wave * T::A_LOADS + l) * 1024), 16, off,
                                                     soff, 0, 0);
        else if (lb < T::B_LOADS / 2)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                rb0, (lds_void*)(base + T::A_BYTES + (wave * T::B_LOADS + lb) * 1024), 16, off, soff, 0, 0);
        else
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                rb1, (lds_void*)(base + T::A_BYTES + (wave * T::B_LOADS + lb) * 1024), 16, off, soff, 0, 0);
    }
};

template <class T, class OP>
__global__ void __launch_bounds__(T::THREADS, T::OCC) nt_tile(const OP op)
{
    using x8 = typename T::x8;
    static_assert(T::WAVES == 4, "every wave loads");
    __shared__ __attribute__((aligned(1024))) unsigned char smem[T::LDS_BYTES];
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int wm = wave / T::WAVES_N, wn = wave % T::WAVES_N;

    Tile t;
    op.template tile<T::BM, T::BN>(blockIdx.x, t);
    const Loader<T> loader(op, t, lane, wave);
    const int K = op.K;
    auto issue = [&](int stage, int ks) __attribute__((always_inline)) {
#pragma unroll
        for (int l = 0; l < T::LOADS; ++l) loader.load(smem + stage * T::STAGE_BYTES, l, ks, K, Flag<true>{});
    };

    const int fr = lane & 15, fh = lane >> 4;
    const int pos0 = swizzle(fr, fh) * 16, pos1 = swizzle(fr, 4 + fh) * 16;
    const int arow = (wm * T::WTM + fr) * T::ROW_BYTES;
    const int brow = T::A_BYTES + (wn * T::WTN + fr) * T::ROW_BYTES;

    f32x4 acc[T::FM][T::FN];
#pragma unroll
    for (int i = 0; i < T::FM; ++i)
#pragma unroll
        for (int j = 0; j < T::FN; ++j) acc[i][j] = f32x4{0, 0, 0, 0};

    // Step ks lives in stage ks % S.  Its loads are issued S - 1 steps ahead,
    // after the barrier that shows every wave is done with the stage's old
    // content (step ks - 1's reads ended before that wave's barrier).  Steps
    // past the end load zeros into stages that nobody reads.
    const int nk = (K + T::BK - 1) / T::BK;
#pragma unroll
    for (int s = 0; s < T::STAGES - 1; ++s) issue(s, s);
    int cur = 0, fill = T::STAGES - 1;
    for (int ks = 0; ks < nk; ++ks) {
        lds_barrier<T::LOADS * (T::STAGES - 2)>();
        issue(fill, ks + T::STAGES - 1);
        const unsigned char* base = smem + cur * T::STAGE_BYTES;
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            const int pos = kk ? pos1 : pos0;
            x8 fa[T::FM], fb[T::FN];
#pragma unroll
            for (int i = 0; i < T::FM; ++i) fa[i] = *(const x8*)(base + arow + i * 16 * T::ROW_BYTES + pos);
#pragma unroll
            for (int j = 0; j < T::FN; ++j) fb[j] = *(const x8*)(base + brow + j * 16 * T::ROW_BYTES + pos);
#pragma unroll
            for (int i = 0; i < T::FM; ++i)
#pragma unroll
                for (int j = 0; j < T::FN; ++j) acc[i][j] = Elem<typename T::E>::mfma(fb[j], fa[i], acc[i][j]);
        }
        cur = cur + 1 == T::STAGES ? 0 : cur + 1;
        fill = fill + 1 == T::STAGES ? 0 : fill + 1;
    }
    // no load may still be writing LDS when the ring is used again or the
    // workgroup ends
    lds_barrier<0>();
    op.template epilogue<T>(t, acc, lane, wave, smem, smem + 32768);
}

// The same with B k by k: a wave's quarter of B is 16 rows, four to a load, lane ->
// row lane / 16, position lane % 16.  A step's rows are a buffer of their own, as
// all of them may span more than its 32 bits.
template <class T>
struct Loader<T, true> {
    __amdgpu_buffer_rsrc_t ra;
    const typename T::E* b;
    uint32_t va[T::A_LOADS], vb[T::B_LOADS], pitch_b;
    int c01[2], wave, steps, cols;
    // B's rows of step ks
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t rows(int ks) const
    {
        const int left = min(steps - ks * T::BK, T::BK);
        return make_rsrc((const unsigned char*)b + (int64_t)ks * T::BK * pitch_b,
                         left > 0 ? (uint32_t)(left - 1) * pitch_b + (uint32_t)cols * 2u : 0u);
    }
    template <class OP>
    __device__ __forceinline__ Loader(const OP& op, const Tile& t, int lane, int w) : wave(w)
    {
        static_assert(T::BN == 128 && T::B_LOADS == 4, "four rows of B to a load");
        const uint32_t pitch_a = (uint32_t)op.lda * 2u;
        int na = 0;
        const void* pa = op.a_rows(t, w * (T::BM / 4), na);
        ra = make_rsrc(pa, (uint32_t)min(na, T::BM / 4) * pitch_a);
        b = op.b_turned(t, steps, cols);
        pitch_b = (uint32_t)op.ldb * 2u;
        const int lr = lane >> 3, lp = lane & 7;
        c01[0] = swizzle(lr, lp);
        c01[1] = swizzle(8 + lr, lp);
#pragma unroll
        for (int l = 0; l < T::A_LOADS; ++l) va[l] = (uint32_t)(l * 8 + lr) * pitch_a + (uint32_t)c01[l & 1] * 16u;
#pragma unroll
        for (int l = 0; l < T::B_LOADS; ++l) {
            const int k = w * 16 + l * 4 + (lane >> 4);
            vb[l] = (uint32_t)k * pitch_b + (uint32_t)turned_swizzle(k, lane & 15) * 16u;
        }
    }
    template <class Masked>
    __device__ __forceinline__ void load(unsigned char* base, int l, int ks, int K, Masked) const
    {
        if (l < T::A_LOADS) {
            uint32_t off = va[l < T::A_LOADS ? l : 0], soff = (uint32_t)ks * (T::BK * 2);
            if constexpr (Masked::value) {
                off = c01[l & 1] * 8 < K - ks * T::BK ? off + soff : kOob;
                soff = 0;
            }
            load_lds(ra, (lds_void*)(base + (wave * T::A_LOADS + l) * 1024), off, soff);
        } else {
            const int lb = l < T::A_LOADS ? 0 : l - T::A_LOADS;
            load_lds(rows(ks), (lds_void*)(base + T::A_BYTES + (wave * T::B_LOADS + lb) * 1024), vb[lb], 0);
        }
    }
};

// acc += b * a with the accumulator in AGPRs; the memory clobber keeps every
// LDS and global access on its side, so the source order of a loop built from
// these is its issue order.
__device__ __forceinline__ void mfma_agpr(f32x4& acc, const Elem<_Float16>::x8& b, const Elem<_Float16>::x8& a)
{
    asm volatile("v_mfma_f32_16x16x32_f16 %0, %1, %2, %0" : "+a"(acc) : "v"(b), "v"(a) : "memory");
}
__device__ __forceinline__ void mfma_agpr(f32x4& acc, const Elem<__bf16>::x8& b, const Elem<__bf16>::x8& a)
{
    asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(acc) : "v"(b), "v"(a) : "memory");
}

// One tile per workgroup, eight waves (two per SIMD), every instruction of
// the K loop in a fixed order.  Waves 0 .. 3 (one per SIMD) issue the loads,
// so that each SIMD has a wave that never waits on the vector memory queue.
// A step is two sub-steps of 32 k:
//   sub-step 0: its MFMAs, with the fragment reads of sub-step 1 between them;
//   barrier:    the wave's loads of the next step have landed, its reads are
//               back, so every wave is done with this step's operand tiles;
//   sub-step 1: its MFMAs, with the next step's first fragment reads and the
//               loads of step ks + S, into the stage this step leaves.
//
// Split: tiles `full` and on are summed by `parts` workgroups each, over
// equal shares of K's steps; each leaves its accumulators, in the lanes'
// order, in `partial`, and nt_join adds them (in a fixed order) and writes
// the tile out.  This fills the CUs that a last wave of few tiles would
// leave idle.  Units run part by part, an XCD's one after another: its tiles
// then read the same share of K, which its L2 holds once.  (1000 x 1032 over
// 32008, 36 tiles in 7 parts: 94 us with a tile's parts one after another, and 81.)
struct Split {
    int full, parts;
    float* partial;
};

template <class T, class OP>
__global__ void __launch_bounds__(T::THREADS, 1) nt_ordered(const OP op, const Split split)
{
    using x8 = typename T::x8;
    constexpr bool TURNED = Turned<OP>::value;
    constexpr int S = T::STAGES, G = T::FM * T::FN, BR = TURNED ? 2 * T::FN : T::FN, R = T::FM + BR;
    static_assert(T::WAVES == 8, "two waves per SIMD, one of which loads");
    static_assert(T::RS * (R - 1) < G && T::LS * (T::LOADS - 1) + T::LS / 2 < G, "reads and loads fit in a sub-step");
    __shared__ __attribute__((aligned(1024))) unsigned char smem[T::LDS_BYTES];
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int wm = wave / T::WAVES_N, wn = wave % T::WAVES_N;

    const int K = op.K;
    const int nk = (K + T::BK - 1) / T::BK, nfull = K / T::BK;
    int id = blockIdx.x, part = -1, begin = 0, end = nk;  // the steps to add up
    if (id >= split.full) {
        const int units = (int)gridDim.x - split.full, rest = units / split.parts, n = xcd_order(id - split.full, units);
        id = split.full + n % rest;
        part = n / rest;
        begin = (int)((int64_t)nk * part / split.parts);
        end = (int)((int64_t)nk * (part + 1) / split.parts);
    }
    Tile t;
    op.template tile<T::BM, T::BN>(id, t);
    const Loader<T, TURNED> loader(op, t, lane, wave & 3);

    const int fr = lane & 15, fh = lane >> 4;
    const int pos[2] = {swizzle(fr, fh) * 16, swizzle(fr, 4 + fh) * 16};
    const int arow = (wm * T::WTM + fr) * T::ROW_BYTES;
    const int brow = T::A_BYTES + (wn * T::WTN + fr) * T::ROW_BYTES;
    // (turned: the lane reads columns 4 (l % 4) .. + 3 of row l / 4 of four, l of 16
    // lanes, and gets column l of all four)
    int bturn[T::FN];
    if constexpr (TURNED)
#pragma unroll
        for (int j = 0; j < T::FN; ++j) {
            const int k = fh * 8 + (fr >> 2), chunk = (wn * T::WTN + j * 16) / 8 + ((fr & 3) >> 1);
            bturn[j] = T::A_BYTES + k * (T::BN * 2) + turned_swizzle(k, chunk) * 16 + (fr & 1) * 8;
        }

    x8 fa[2][T::FM], fb[2][T::FN];
    f32x4 acc[T::FM][T::FN];
#pragma unroll
    for (int i = 0; i < T::FM; ++i)
#pragma unroll
        for (int j = 0; j < T::FN; ++j) acc[i][j] = f32x4{0, 0, 0, 0};

    typename Elem<typename T::E>::x4 half[2][TURNED ? T::FN : 1][2];
    // fragment read idx of set `set`, in the order the MFMAs need them
    auto read_one = [&](int set, const unsigned char* base, int idx) __attribute__((always_inline)) {
        if (idx == 0)
            fa[set][0] = *(const x8*)(base + arow + pos[set]);
        else if (TURNED && idx <= BR)
            half[set][(idx - 1) / 2][(idx - 1) % 2] =
                read_turned<typename T::E>(base + bturn[(idx - 1) / 2] + (set * 32 + (idx - 1) % 2 * 4) * (T::BN * 2));
        else if (idx <= BR)
            fb[set][idx - 1] = *(const x8*)(base + brow + pos[set] + (idx - 1) * 16 * T::ROW_BYTES);
        else
            fa[set][idx - BR] = *(const x8*)(base + arow + pos[set] + (idx - BR) * 16 * T::ROW_BYTES);
    };
    auto fragment = [&](int set, int j) __attribute__((always_inline)) {
        if constexpr (TURNED)
            return (x8)__builtin_shufflevector(half[set][j][0], half[set][j][1], 0, 1, 2, 3, 4, 5, 6, 7);
        else
            return fb[set][j];
    };
    // MFMAs along the rows of blocks and back, so that neighbours share a fragment
    auto substep = [&](int set, const unsigned char* reads, auto ld, unsigned char* into, int lstep, auto masked)
                       __attribute__((always_inline)) {
#pragma unroll
        for (int n = 0; n < G; ++n) {
            const int i = n / T::FN, j = (i & 1) ? T::FN - 1 - n % T::FN : n % T::FN;
            mfma_agpr(acc[i][j], fragment(set, j), fa[set][i]);
            if (n % T::RS == 0 && n / T::RS < R) read_one(1 - set, reads, n / T::RS);
            if constexpr (decltype(ld)::value)
                if (n % T::LS == T::LS / 2 && n / T::LS < T::LOADS) loader.load(into, n / T::LS, lstep, K, masked);
        }
    };

    auto run = [&](auto ldtag) __attribute__((always_inline)) {
        constexpr bool LD = decltype(ldtag)::value;
        // every stage is free at the start: fill them all, then wait for step 0
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
            for (int l = 0; l < T::LOADS; ++l)
                if constexpr (LD) loader.load(smem + s * T::STAGE_BYTES, l, begin + s, K, Flag<true>{});
        lds_barrier<T::LOADS * (S - 1)>();
#pragma unroll
        for (int idx = 0; idx < R; ++idx) read_one(0, smem, idx);
        int cur = 0;
        auto step = [&](int ks, auto masked) __attribute__((always_inline)) {
            const int nxt = cur + 1 == S ? 0 : cur + 1;
            unsigned char* base = smem + cur * T::STAGE_BYTES;
            unsigned char* next = smem + nxt * T::STAGE_BYTES;
            substep(0, base, Flag<false>{}, base, 0, masked);
            lds_barrier<T::LOADS * (S - 2)>();
            // (what steps past the last load, zeros past the end of K, is
            // never read)
            substep(1, next, Flag<LD>{}, base, ks + S, masked);
            cur = nxt;
        };
        int ks = begin;
        for (; ks < end && ks + S < nfull; ++ks) step(ks, Flag<false>{});
        for (; ks < end; ++ks) step(ks, Flag<true>{});
    };
    if (end > begin) {
        if (wave < T::LOADERS)
            run(Flag<true>{});
        else
            run(Flag<false>{});
        // the last MFMAs write their accumulators before they are read: asm
        // hides them from the compiler's hazard checks
        asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7" ::: "memory");
    }
    // no load may still be writing LDS when the ring is used again or the
    // workgroup ends
    lds_barrier<0>();
    if (part < 0) {
        op.template epilogue<T>(t, acc, lane, wave, smem, smem + 32768);
        return;
    }
    float* to = split.partial + ((int64_t)((id - split.full) * split.parts + part) * T::WAVES + wave) * (G * 256) + lane * 4;
#pragma unroll
    for (int i = 0; i < T::FM; ++i)
#pragma unroll
        for (int j = 0; j < T::FN; ++j) *(f32x4*)(to + (i * T::FN + j) * 256) = acc[i][j];
}

// Adds up the parts of the tiles that nt_ordered split and writes them out: a
// workgroup for the sub-tile of each wave of a tile, so that few tiles still
// read with many CUs, of four waves that take every fourth part (one wave
// walking all parts took 24 us for sixteen, one workgroup for a whole tile 15).
template <class T>
struct WaveShape {
    using E = typename T::E;
    static constexpr int BM = T::WTM, BN = T::WTN, WAVES_M = 1, WAVES_N = 1, WAVES = 1;
    static constexpr int WTM = T::WTM, WTN = T::WTN, FM = T::FM, FN = T::FN, STAGE_MAX = BM * BN * 2;
};
constexpr int kJoinWaves = 4;

template <class T, class OP>
__global__ void __launch_bounds__(kJoinWaves * kWave) nt_join(const OP op, const Split split)
{
    using W = WaveShape<T>;
    constexpr int G = T::FM * T::FN;
    __shared__ __attribute__((aligned(1024))) unsigned char smem[(kJoinWaves - 1) * G * 1024];
    static_assert(sizeof(smem) >= W::STAGE_MAX, "the image fits");
    const int lane = threadIdx.x & (kWave - 1), share = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int n = blockIdx.x / T::WAVES, wave = blockIdx.x % T::WAVES;
    Tile t;
    op.template tile<T::BM, T::BN>(split.full + n, t);
    t.m0 += wave / T::WAVES_N * T::WTM;
    t.n0 += wave % T::WAVES_N * T::WTN;
    if (op.outside(t)) return;
    f32x4 acc[T::FM][T::FN];
#pragma unroll
    for (int i = 0; i < T::FM; ++i)
#pragma unroll
        for (int j = 0; j < T::FN; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
    const float* from = split.partial + ((int64_t)n * split.parts * T::WAVES + wave) * (G * 256) + lane * 4;
    constexpr int AHEAD = 32 / G;  // parts whose loads are in flight together
#pragma unroll AHEAD
    for (int p = share; p < split.parts; p += kJoinWaves) {
        const float* at = from + (int64_t)p * (T::WAVES * G * 256);
#pragma unroll
        for (int i = 0; i < T::FM; ++i)
#pragma unroll
            for (int j = 0; j < T::FN; ++j) acc[i][j] += *(const f32x4*)(at + (i * T::FN + j) * 256);
    }
    f32x4* sums = (f32x4*)smem + lane;
    if (share > 0)
#pragma unroll
        for (int i = 0; i < T::FM; ++i)
#pragma unroll
            for (int j = 0; j < T::FN; ++j) sums[((share - 1) * G + i * T::FN + j) * 64] = acc[i][j];
    __syncthreads();
    if (share > 0) return;
#pragma unroll
    for (int s = 0; s < kJoinWaves - 1; ++s)
#pragma unroll
        for (int i = 0; i < T::FM; ++i)
#pragma unroll
            for (int j = 0; j < T::FN; ++j) acc[i][j] += sums[(s * G + i * T::FN + j) * 64];
    lds_barrier<0>();
    op.template epilogue<W>(t, acc, lane, 0, smem, smem);
}

// One 256 x 256 tile after another per workgroup, one workgroup per CU, four
// waves, one per SIMD, each holding a 128 x 128 quarter of the tile in its
// 256 AGPRs.  LDS is a ring of five 32 KiB slots of one operand tile each
// (A of step j in slot 2j mod 5, B in slot 2j + 1 mod 5), and the load
// stream runs on across tiles: a tile's last two steps load the first two of
// the next.  Every MFMA is an asm statement, so the source order is the issue
// order: a fragment read of the next sub-step after every third MFMA, a
// global->LDS load after every eighth, one barrier a step.
//
// With one wave per SIMD nothing hides scalar or vector arithmetic between
// two MFMAs.  The steps that load whole K ranges therefore run as a cycle of
// five, one per position of the ring, in which every slot is a constant of
// the code, every LDS address a register and an immediate, and the K
// position one scalar register; the others (K's tail, the two that start the
// next tile, up to four before and after the cycles) keep the ring position
// in a register.
//
// The epilogue has the two slots that no load is writing.  Nothing clears the
// accumulators: a tile's first MFMAs add to an inline zero.
//
// Needs three steps at least: K > 128.
template <class E_>
struct Shape256 {
    using E = E_;
    using x8 = typename Elem<E>::x8;
    static constexpr int BM = 256, BN = 256, BK = 64, THREADS = 256;
    static constexpr int WAVES_M = 2, WAVES_N = 2, WAVES = 4;
    static constexpr int WTM = 128, WTN = 128, FM = 8, FN = 8;
    static constexpr int ROW_BYTES = 128;
    static constexpr int SLOT = 32768, STAGE_MAX = 2 * SLOT;
    static constexpr int RS = 3, LS = 8;  // MFMAs per fragment read, per load
};

// The same with nothing to add to.  (The old value is an operand only to keep
// the accumulator in its registers: as a plain output it made the register
// allocator spill.)
__device__ __forceinline__ void mfma_agpr_first(f32x4& acc, const Elem<_Float16>::x8& b, const Elem<_Float16>::x8& a)
{
    asm volatile("v_mfma_f32_16x16x32_f16 %0, %1, %2, 0" : "+a"(acc) : "v"(b), "v"(a) : "memory");
}
__device__ __forceinline__ void mfma_agpr_first(f32x4& acc, const Elem<__bf16>::x8& b, const Elem<__bf16>::x8& a)
{
    asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, 0" : "+a"(acc) : "v"(b), "v"(a) : "memory");
}

// The kernel's argument, read again: what only the epilogue uses then needs
// no scalar register through the K loop (kept, some would spill).
template <class OP>
__device__ __forceinline__ OP argument_again()
{
    typedef const __attribute__((address_space(4))) uint32_t word;
    word* p = (word*)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(p));
    struct Words {
        uint32_t w[sizeof(OP) / 4];
    } a;
    static_assert(sizeof(Words) == sizeof(OP), "whole words");
#pragma unroll
    for (unsigned i = 0; i < sizeof(OP) / 4; ++i) a.w[i] = p[i];
    return __builtin_bit_cast(OP, a);
}

template <class T, class OP>
__global__ void __launch_bounds__(T::THREADS, 1) nt_persist(const OP op)
{
    using x8 = typename T::x8;
    constexpr int SLOT = T::SLOT, G = 64, R = 16;  // MFMAs and fragment reads per sub-step
    __shared__ __attribute__((aligned(1024))) unsigned char smem[5 * SLOT];

    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int wm = wave >> 1, wn = wave & 1;
    const int K = op.K;
    const int nk = (K + T::BK - 1) / T::BK;
    const int nfull = K / T::BK;  // steps wholly inside K
    const uint32_t pitch_a = (uint32_t)op.lda * 2u, pitch_b = (uint32_t)op.template b_pitch<T::WTN>(wave * 64) * 2u;

    // Load l of a wave fills rows 8 l .. + 7 of its quarter of an operand's
    // tile, KiB wave * 8 + l of the slot.  Loads of a group of four share the
    // LDS base (M0); the instruction offset (l & 3) KiB places them, and as
    // the hardware adds it to the global offset too, the VGPR offset gives it
    // back (no wrap: row 8 l starts at 8 l * pitch >= l KiB, the pitch being
    // at least 128 bytes).
    const int lr = lane >> 3, lp = lane & 7;
    const int c01[2] = {swizzle(lr, lp), swizzle(8 + lr, lp)};
    uint32_t va[8], vb[8];
#pragma unroll
    for (int l = 0; l < 8; ++l) {
        const uint32_t c = (uint32_t)c01[l & 1] * 16u - (uint32_t)(l & 3) * 1024u;
        va[l] = (uint32_t)(l * 8 + lr) * pitch_a + c;
        vb[l] = (uint32_t)(l * 8 + lr) * pitch_b + c;
        asm volatile("" : "+v"(va[l]), "+v"(vb[l]));
    }
    int wave_bytes = __builtin_amdgcn_readfirstlane(wave * 8192);

    // The tile being loaded runs up to one ahead of the one being computed.
    int id = blockIdx.x;
    const int tiles = op.tiles;
    if (id >= tiles) return;
    Tile t;
    __amdgpu_buffer_rsrc_t la, lb;
    auto start = [&](const OP& o, int n) __attribute__((always_inline)) {
        o.template tile<T::BM, T::BN>(n, t);
        int na = 0, nb = 0;
        const void* pa = o.a_rows(t, wave * 64, na);
        const void* pb = o.template b_rows<T::WTN>(t, wave * 64, nb);
        la = make_rsrc(pa, (uint32_t)min(na, 64) * (uint32_t)o.lda * 2u);
        lb = make_rsrc(pb, (uint32_t)min(nb, 64) * (uint32_t)o.template b_pitch<T::WTN>(wave * 64) * 2u);
    };
    start(op, id);

    auto load = [&](unsigned char* dst, int l, uint32_t off, uint32_t soff) __attribute__((always_inline)) {
        lds_void* d = (lds_void*)(dst + (l & 4) * 1024);
        // (the instruction offset must be a constant, and a buffer resource
        // cannot be the result of ?:)
#define NT_LOAD(RS)                                                                                  \
    switch (l & 3) {                                                                                 \
        case 0: __builtin_amdgcn_raw_ptr_buffer_load_lds(RS, d, 16, off, soff, 0, 0); break;         \
        case 1: __builtin_amdgcn_raw_ptr_buffer_load_lds(RS, d, 16, off, soff, 1024, 0); break;      \
        case 2: __builtin_amdgcn_raw_ptr_buffer_load_lds(RS, d, 16, off, soff, 2048, 0); break;      \
        default: __builtin_amdgcn_raw_ptr_buffer_load_lds(RS, d, 16, off, soff, 1024 * 3, 0); break; \
    }
        if (l < 8) {
            NT_LOAD(la)
        } else {
            NT_LOAD(lb)
        }
#undef NT_LOAD
    };
    // Load l (0 .. 7 of A, 8 .. 15 of B) of step ks of the loading tile into
    // slot `where`; chunks at or past K read as zero.  The K position is part
    // of the vector offset: past the end it may exceed the buffer.
    auto load_any = [&](int where, int ks, int l) __attribute__((always_inline)) {
        const uint32_t v = l < 8 ? va[l & 7] : vb[l & 7];
        const uint32_t koff = (uint32_t)ks * (T::BK * 2);
        // (the mark less the instruction offset, so that the sum stays out of range)
        const uint32_t off = c01[l & 1] * 8 < K - ks * T::BK ? v + koff : kOob;
        load(smem + where * SLOT + wave_bytes, l, off, 0);
    };

    const int fr = lane & 15, fh = lane >> 4;
    const int pos[2] = {swizzle(fr, fh) * 16, swizzle(fr, 4 + fh) * 16};
    const int arow = (wm * T::WTM + fr) * T::ROW_BYTES, brow = (wn * T::WTN + fr) * T::ROW_BYTES;
    // LDS address of operand x's fragment rows at k-half kk, plus c * 64 KiB:
    // slots 2c and 2c + 1 lie within an immediate's reach of it.
    uint32_t rdb[3][2][2];
#pragma unroll
    for (int c = 0; c < 3; ++c)
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            rdb[c][0][kk] = (uint32_t)(c * 65536 + arow + pos[kk]);
            rdb[c][1][kk] = (uint32_t)(c * 65536 + brow + pos[kk]);
        }

    x8 fa[2][T::FM], fb[2][T::FN];
    f32x4 acc[T::FM][T::FN];

    // Fragment read idx of set `set`: B's blocks, then A's from the last to
    // the first, the order in which the other set's MFMAs last used them.
    auto read_any = [&](int set, const unsigned char* abase, const unsigned char* bbase, int idx)
                        __attribute__((always_inline)) {
        if (idx < 8)
            fb[set][idx] = *(const x8*)(bbase + brow + pos[set] + idx * 16 * T::ROW_BYTES);
        else
            fa[set][15 - idx] = *(const x8*)(abase + arow + pos[set] + (15 - idx) * 16 * T::ROW_BYTES);
    };
    auto read_fast = [&](auto sa_c, auto sb_c, int set, int idx) __attribute__((always_inline)) {
        constexpr int SA = decltype(sa_c)::value, SB = decltype(sb_c)::value;
        if (idx < 8)
            fb[set][idx] = *(const x8*)(smem + rdb[SB / 2][1][set] + (SB % 2) * SLOT + idx * 16 * T::ROW_BYTES);
        else
            fa[set][15 - idx] =
                *(const x8*)(smem + rdb[SA / 2][0][set] + (SA % 2) * SLOT + (15 - idx) * 16 * T::ROW_BYTES);
    };
    // MFMA number n of a sub-step: down the columns of blocks and back up
    // every second one, so that neighbours share a fragment.
    auto mma = [&](int set, int n, auto first) __attribute__((always_inline)) {
        const int j = n / 8, i = (j & 1) ? 7 - n % 8 : n % 8;
        if constexpr (decltype(first)::value)
            mfma_agpr_first(acc[i][j], fb[set][j], fa[set][i]);
        else
            mfma_agpr(acc[i][j], fb[set][j], fa[set][i]);
    };
    auto substep = [&](int set, const unsigned char* abase, const unsigned char* bbase, auto ld, auto rd, int where,
                       int lstep, int l0, auto first) __attribute__((always_inline)) {
#pragma unroll
        for (int n = 0; n < G; ++n) {
            mma(set, n, first);
            if constexpr (decltype(rd)::value)
                if (n % T::RS == 0 && n / T::RS < R) read_any(1 - set, abase, bbase, n / T::RS);
            if constexpr (decltype(ld)::value)
                if (n % T::LS == T::LS / 2) load_any(where, lstep, l0 + n / T::LS);
        }
    };
    auto substep_fast = [&](int set, auto ra, auto rb, auto where_c, int l0, uint32_t soff)
                            __attribute__((always_inline)) {
        constexpr int WHERE = decltype(where_c)::value;
#pragma unroll
        for (int n = 0; n < G; ++n) {
            mma(set, n, Flag<false>{});
            if (n % T::RS == 0 && n / T::RS < R) read_fast(ra, rb, 1 - set, n / T::RS);
            if (n % T::LS == T::LS / 2) {
                const int l = l0 + n / T::LS;
                load(smem + WHERE * SLOT + wave_bytes, l, l < 8 ? va[l & 7] : vb[l & 7], soff);
            }
        }
    };
    // A step with its A tile in slot S that loads K bytes soff .. + 127.  The
    // base registers are redefined in place, by no instruction, so that base
    // plus offset is not hoisted into registers of its own.
    auto step_fast = [&](auto s_c, uint32_t soff) __attribute__((always_inline)) {
        constexpr int S = decltype(s_c)::value;
#pragma unroll
        for (int c = 0; c < 3; ++c)
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) asm volatile("" : "+v"(rdb[c][0][kk]), "+v"(rdb[c][1][kk]));
        asm volatile("" : "+s"(wave_bytes));
        substep_fast(0, Int<S>{}, Int<(S + 1) % 5>{}, Int<(S + 4) % 5>{}, 0, soff);
        lds_barrier<8>();
        substep_fast(1, Int<(S + 2) % 5>{}, Int<(S + 3) % 5>{}, Int<S>{}, 8, soff);
    };

#pragma unroll
    for (int i = 0; i < T::FM; ++i)
#pragma unroll
        for (int j = 0; j < T::FN; ++j) asm volatile("" : "=a"(acc[i][j]));  // (any value)
    // steps 0 and 1 of the first tile into slots 0 .. 3, then wait for step 0
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int l = 0; l < 16; ++l) load_any(l < 8 ? 2 * s : 2 * s + 1, s, l);
    lds_barrier<16>();
#pragma unroll
    for (int idx = 0; idx < R; ++idx) read_any(0, smem, smem + SLOT, idx);
    int sa = 0;  // slot of the computed step's A tile; its B, then A, B, A of the next two follow
    auto slot = [&](int i) __attribute__((always_inline)) { return smem + (sa + i >= 5 ? sa + i - 5 : sa + i) * SLOT; };
    // Sub-step 0 loads A of step lstep into the slot after the next step's;
    // sub-step 1 reads the next step's first fragments and loads its B into
    // the slot this step's A leaves, unless LAST (the last of a tile, whose
    // epilogue may use both slots first).
    auto step = [&](int lstep, auto last, auto first) __attribute__((always_inline)) {
        constexpr bool LAST = decltype(last)::value;
        const int a2 = sa + 4 >= 5 ? sa - 1 : sa + 4;
        substep(0, slot(0), slot(1), Flag<true>{}, Flag<true>{}, a2, lstep, 0, first);
        lds_barrier<8>();  // all but the A tile just loaded have landed
        substep(1, slot(2), slot(3), Flag<!LAST>{}, Flag<!LAST>{}, sa, lstep, 8, Flag<false>{});
    };
    auto advance = [&]() __attribute__((always_inline)) { sa = sa + 2 >= 5 ? sa - 3 : sa + 2; };
    for (;;) {
        step(2, Flag<false>{}, Flag<true>{});
        advance();
        int ks = 1;
        // general steps until the ring is back at slot 0, then whole cycles
        for (; ks + 2 < nfull && sa != 0; ++ks) {
            step(ks + 2, Flag<false>{}, Flag<false>{});
            advance();
        }
        uint32_t soff = (uint32_t)(ks + 2) * T::ROW_BYTES;
        for (; ks + 2 + 5 <= nfull; ks += 5) {
            step_fast(Int<0>{}, soff);
            step_fast(Int<2>{}, soff + T::ROW_BYTES);
            step_fast(Int<4>{}, soff + 2 * T::ROW_BYTES);
            step_fast(Int<1>{}, soff + 3 * T::ROW_BYTES);
            step_fast(Int<3>{}, soff + 4 * T::ROW_BYTES);
            soff += 5 * T::ROW_BYTES;
        }
        for (; ks + 2 < nk; ++ks) {
            step(ks + 2, Flag<false>{}, Flag<false>{});
            advance();
        }
        // The last two steps load steps 0 and 1 of the next tile (after the
        // last one: zeros from past the end of K, into slots never read).
        const Tile done = t;
        const int next = id + (int)gridDim.x;
        int lbase = nk;
        if (next < tiles) {
            start(argument_again<OP>(), next);
            lbase = 0;
        }
        step(lbase, Flag<false>{}, Flag<false>{});
        advance();
        step(lbase + 1, Flag<true>{}, Flag<false>{});
        // the last MFMAs write their accumulators before they are read: asm
        // hides them from the compiler's hazard checks
        asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
        const OP again = argument_again<OP>();
        again.template epilogue<T>(done, acc, lane, wave, slot(0), slot(1));
        if (next >= tiles) break;
        // every wave is done with this step's slots
        lds_barrier<63>();
        // B of the next tile's step 1 where the last step's A was
#pragma unroll
        for (int l = 8; l < 16; ++l) load_any(sa, lbase + 1, l);
        advance();
#pragma unroll
        for (int idx = 0; idx < R; ++idx) read_any(0, slot(0), slot(1), idx);
        id = next;
    }
    // no load may still be writing LDS when the workgroup ends
    lds_barrier<0>();
}

// The lane, as if newly read: addresses derived from it are computed where
// they are used, not early and kept (or spilled) through the K loop.
__device__ __forceinline__ int pinned(int lane)
{
    asm volatile("" : "+v"(lane)::"memory");
    return lane;
}

// The same of a value that all lanes share, as a vector: offsets made of it
// then need no scalar register each.
__device__ __forceinline__ uint32_t as_vector(uint32_t v)
{
    asm volatile("" : "+v"(v));
    return v;
}

// LDS image of part of a tile: rows of COLS 16-bit values, 16-byte chunk c of
// row x at c ^ (x % 16) (or % COLS / 8): the eight-byte pieces that the lanes
// of a wave put fall on the banks evenly, and whole rows are read back without
// conflicts.  The first 32 KiB lie at s0, the rest at s1.
template <int COLS>
struct Image {
    static constexpr int PITCH = COLS * 2, CH = COLS / 8, KEY = (CH < 16 ? CH : 16) - 1;
    unsigned char *s0, *s1;
    __device__ __forceinline__ unsigned char* row(int x) const
    {
        const int off = x * PITCH;
        return off < 32768 ? s0 + off : s1 + (off - 32768);
    }
    // where four values at row x, column c (a multiple of four) lie
    template <class V>
    __device__ __forceinline__ V* at(int x, int c) const
    {
        static_assert(sizeof(V) == 8, "four 16-bit values");
        return (V*)(row(x) + (((c >> 3) ^ (x & KEY)) << 4) + (c & 4) * 2);
    }
    template <class V>
    __device__ __forceinline__ void put(int x, int c, const V& v) const
    {
        *at<V>(x, c) = v;
    }
    // one value, after what the wave has put there before
    template <class E>
    __device__ __forceinline__ void set(int x, int c, E v) const
    {
        static_assert(sizeof(E) == 2, "one 16-bit value");
        asm volatile("" ::: "memory");
        *(E*)(row(x) + (((c >> 3) ^ (x & KEY)) << 4) + (c & 7) * 2) = v;
    }
    __device__ __forceinline__ u32x4 get(int x, int chunk) const
    {
        return *(const u32x4*)(row(x) + ((chunk ^ (x & KEY)) << 4));
    }
};

// Where a tile's rows go: a buffer from the tile's first row on, `pitch`
// bytes to a row, columns first .. cols - 1.
struct Rows {
    __amdgpu_buffer_rsrc_t rs;
    uint32_t pitch;
    int first, cols;
};
template <class E>
__device__ __forceinline__ Rows rows_at(E* base, int row, int rows, int most, int ld, int first, int cols)
{
    Rows r;
    r.pitch = (uint32_t)ld * 2u;
    r.rs = make_rsrc(base + (int64_t)row * ld, (uint32_t)min(most, rows - row) * r.pitch);
    r.first = first;
    r.cols = cols;
    return r;
}

// Writes ROWS rows of an image out, whole rows by adjacent lanes, 16 bytes
// each; `to(x)` is the row of `out` that image row x belongs to.  A store is
// served 16 lanes at a time, a cache line each cycle: stored from the
// accumulators' layout, where 16 adjacent lanes hold 16 rows, each would take
// 64 cycles.  EIGHTS: out's rows take 16-byte pieces and hold a multiple of
// eight columns; otherwise each element goes out alone.  (Templates, not
// conditions: with two ways through an epilogue that holds 256 accumulators
// the register allocator spills.)
template <class T, int COLS, int ROWS, bool EIGHTS, class To>
__device__ __forceinline__ void drain(const Image<COLS>& image, const Rows& out, To to, int lane, int wave)
{
    constexpr int CH = COLS / 8, RPI = 64 / CH, ITERS = ROWS / RPI / T::WAVES;
    static_assert(ITERS * RPI * T::WAVES == ROWS, "rows split evenly over the waves");
    const int ln = pinned(lane);
    const int ch = ln % CH, n = out.first + ch * 8;
    const int x0 = (int)as_vector((uint32_t)wave * (ITERS * RPI)) + ln / CH;
#pragma unroll
    for (int it = 0; it < ITERS; ++it) {
        const int x = x0 + it * RPI;
        if constexpr (EIGHTS) {
            const u32x4 v = image.get(x, ch);
            const uint32_t at = (uint32_t)to(x) * out.pitch + (uint32_t)n * 2u;
            __builtin_amdgcn_raw_buffer_store_b128(v, out.rs, n < out.cols ? at : kOob, 0, 0);
        } else {
            // 64 adjacent elements at a time, which 16 lanes find in one line
            // or two; with eight to a lane they span three (1000 x 1032 x
            // 2730: 19.1 us, and 22.2)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                // (one after another: the comparisons' results are scalar registers)
                __builtin_amdgcn_sched_barrier(0);
                const int q = e * 64 + ln, xe = (int)as_vector((uint32_t)wave * (ITERS * RPI)) + it * RPI + q / COLS;
                const int c = q % COLS;
                const uint16_t v = *(const uint16_t*)(image.row(xe) + (((c >> 3) ^ (xe & Image<COLS>::KEY)) << 4) + (c & 7) * 2);
                const int ne = out.first + c;
                __builtin_amdgcn_raw_buffer_store_b16(
                    v, out.rs, ne < out.cols ? (uint32_t)to(xe) * out.pitch + (uint32_t)ne * 2u : kOob, 0, 0);
            }
        }
    }
}

// The other way: fills ROWS rows of an image from `in`, zeros where there is
// nothing; rows take 16-byte pieces.
template <class T, int COLS, int ROWS, class To>
__device__ __forceinline__ void fill(const Image<COLS>& image, const Rows& in, To to, int lane, int wave)
{
    constexpr int CH = COLS / 8, RPI = 64 / CH, ITERS = ROWS / RPI / T::WAVES;
    const int ln = pinned(lane);
    const int x0 = (int)as_vector((uint32_t)wave * (ITERS * RPI)) + ln / CH;
#pragma unroll
    for (int it = 0; it < ITERS; ++it) {
        const int x = x0 + it * RPI, n = in.first + ((ln % CH) ^ (x & Image<COLS>::KEY)) * 8;
        const uint32_t at = (uint32_t)to(x) * in.pitch + (uint32_t)n * 2u;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(in.rs, (lds_void*)image.row((wave * ITERS + it) * RPI), 16,
                                                 n < in.cols ? at : kOob, 0, 0, 0);
    }
}

// The tile row by row: value(i, j) is the four columns that this lane holds
// of block (i, j) of FN in a wave row.
template <class T, int FN, bool EIGHTS, class Value>
__device__ __forceinline__ void write_rows(Value value, const Rows& out, int lane, int wave, unsigned char* s0,
                                           unsigned char* s1)
{
    constexpr int WCOLS = FN * 16, COLS = WCOLS * T::WAVES_N, ROUNDS = T::BM * COLS * 2 > T::STAGE_MAX ? 2 : 1;
    constexpr int RW = T::WTM / ROUNDS;  // staged rows of a wave row
    static_assert(T::BM * COLS * 2 <= ROUNDS * T::STAGE_MAX, "a round fits");
    const Image<COLS> image{s0, s1};
    const int wm = wave / T::WAVES_N, wn = wave % T::WAVES_N;
#pragma unroll
    for (int h = 0; h < ROUNDS; ++h) {
        const int ln = pinned(lane);
#pragma unroll
        for (int i = 0; i < T::FM / ROUNDS; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j)
                image.put(wm * RW + i * 16 + (ln & 15), wn * WCOLS + j * 16 + 4 * (ln >> 4),
                          value(h * (T::FM / ROUNDS) + i, j));
        lds_barrier<63>();
        drain<T, COLS, T::WAVES_M * RW, EIGHTS>(
            image, out, [&](int x) { return x / RW * T::WTM + h * RW + x % RW; }, lane, wave);
        lds_barrier<63>();
    }
}

// Lanes 4 q .. 4 q + 3 hold values a, b, c, d of rows 4 q .. 4 q + 3; after
// this they hold the four rows' a, the four rows' b, and so on.
template <class X4>
__device__ __forceinline__ X4 quad_transposed(const X4& v, int lane)
{
    const u32x2 d = __builtin_bit_cast(u32x2, v);
    // with the neighbour: the even lane gets the pair's a and c, the odd one b and d
    const bool odd = lane & 1, far = lane & 2;
    const uint32_t n0 = __builtin_amdgcn_mov_dpp(d[0], 0xb1, 0xf, 0xf, true);  // quad_perm 1, 0, 3, 2
    const uint32_t n1 = __builtin_amdgcn_mov_dpp(d[1], 0xb1, 0xf, 0xf, true);
    const uint32_t sel = odd ? 0x03020706u : 0x05040100u;  // (own bytes 0 .. 3, the neighbour's 4 .. 7)
    const uint32_t p0 = __builtin_amdgcn_perm(n0, d[0], sel), p1 = __builtin_amdgcn_perm(n1, d[1], sel);
    // with the pair two lanes on: lanes 0, 1 give c, d (p1) and get a, b
    const uint32_t give = far ? p0 : p1;
    const uint32_t got = __builtin_amdgcn_mov_dpp(give, 0x4e, 0xf, 0xf, true);  // quad_perm 2, 3, 0, 1
    const u32x2 r = {far ? got : p0, far ? p1 : got};
    return __builtin_bit_cast(X4, r);
}

// The tile's transpose, row by row (rows n of BM columns m).  A lane's four
// values belong to four rows of it, so four lanes exchange theirs first.
template <class T, bool EIGHTS, class Value>
__device__ __forceinline__ void write_turned(Value value, const Rows& out, int lane, int wave, unsigned char* s0,
                                             unsigned char* s1)
{
    constexpr int ROUNDS = T::BM * T::BN * 2 > T::STAGE_MAX ? 2 : 1;
    constexpr int RW = T::WTN / ROUNDS;  // staged rows of a wave column
    const Image<T::BM> image{s0, s1};
    const int wm = wave / T::WAVES_N, wn = wave % T::WAVES_N;
#pragma unroll
    for (int h = 0; h < ROUNDS; ++h) {
        const int ln = pinned(lane);
#pragma unroll
        for (int i = 0; i < T::FM; ++i)
#pragma unroll
            for (int j = 0; j < T::FN / ROUNDS; ++j)
                image.put(wn * RW + j * 16 + 4 * (ln >> 4) + (ln & 3), wm * T::WTM + i * 16 + (ln & 12),
                          quad_transposed(value(i, h * (T::FN / ROUNDS) + j), ln));
        lds_barrier<63>();
        drain<T, T::BM, T::WAVES_N * RW, EIGHTS>(
            image, out, [&](int x) { return x / RW * T::WTN + h * RW + x % RW; }, lane, wave);
        lds_barrier<63>();
    }
}

// C = A B^T; SCALED: times *factor.
template <class E, bool EIGHTS, bool SCALED>
struct StoreOp {
    static constexpr bool kPersist = true, kSplit = true;
    const E *A[2], *B;  // one product, or two with the same B
    E* C[2];
    const float* factor;
    int M, N, K, lda, ldb, ldc[2], tiles, tiles_m, tiles_n;

    template <int BM, int BN>
    __device__ __forceinline__ void tile(int id, Tile& t) const
    {
        int tm, tn;
        id = xcd_order(id, tiles);
        t.batch = id >= tiles_m * tiles_n;
        grid_tile(t.batch ? id - tiles_m * tiles_n : id, tiles_m, tiles_n, tm, tn);
        t.m0 = tm * BM;
        t.n0 = tn * BN;
    }
    __device__ __forceinline__ bool outside(const Tile& t) const { return t.m0 >= M || t.n0 >= N; }
    __device__ __forceinline__ const E* a_rows(const Tile& t, int row, int& n) const
    {
        return rows_from(t.batch ? A[1] : A[0], t.m0 + row, M, lda, n);
    }
    template <int WTN>
    __device__ __forceinline__ const E* b_rows(const Tile& t, int row, int& n) const
    {
        return rows_from(B, t.n0 + row, N, ldb, n);
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
        // (from constant memory: a scalar register, of which 256 x 256 has some left)
        float f = 1.0f;
        if constexpr (SCALED) f = *(const __attribute__((address_space(4))) float*)factor;
        write_rows<T, T::FN, EIGHTS>([&](int i, int j) { return round4<E>(SCALED ? acc[i][j] * f : acc[i][j]); },
                                     rows_at(t.batch ? C[1] : C[0], t.m0, M, T::BM, t.batch ? ldc[1] : ldc[0], t.n0, N), lane, wave, s0, s1);
    }
};

}  // namespace nt

#endif
