// Tiled NT products (both operands row-major, k contiguous) on gfx950, with
// the operands' rows and the epilogue supplied by an operation OP.
//
// nt_tile: one BM x BN tile of the accumulator per workgroup, four waves
// (2 x 2), a ring of S stages in LDS filled by direct global->LDS loads, and
// v_mfma_f32_16x16x32 with 32-bit accumulators.  In a wave's sub-tile lane l
// holds, of the 16 x 16 block (i, j), row l % 16 and columns 4 * (l / 16) ..
// + 3 (the B fragment is the MFMA's first operand, which gives the block
// transposed: four consecutive columns per lane).
//
// OP has, as device functions,
//   bool tile<BM, BN>(id, Tile&)   what tile number `id` is (row and column
//                                  of its first element, batch);
//   const E* a_rows(t, row, &n)    A's row `row` of the tile's BM and how
//                                  many rows exist from there (rows_from);
//   const E* b_rows<BN>(t, row, &n)  the same for B;
//   epilogue<T>(t, acc, lane, wm, wn, smem)
//   int b_pitch(q)                 the pitch of B's rows in quarter q
// and the fields K (elements, a multiple of 8) and lda (A's row pitch in
// elements; pitches are multiples of 8 and below 2^21).  Every row starts on
// 16 bytes.  Each of the four waves loads a quarter of each
// operand's tile, so the rows of one quarter are evenly spaced.
#ifndef DENSE_FP16_GEMM_NT_CORE_H
#define DENSE_FP16_GEMM_NT_CORE_H

#include "cdna4.h"

namespace nt {

using namespace cdna4;

struct Tile {
    int m0, n0, batch;
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

template <class E_, int BM_, int BN_, int STAGES_, int OCC_>
struct Shape {
    using E = E_;
    using x8 = typename Elem<E>::x8;
    static constexpr int BM = BM_, BN = BN_, BK = 64, STAGES = STAGES_, OCC = OCC_;
    static constexpr int WAVES = 4, THREADS = 256;
    static constexpr int WTM = BM / 2, WTN = BN / 2;   // a wave's sub-tile
    static constexpr int FM = WTM / 16, FN = WTN / 16;
    static constexpr int ROW_BYTES = 128;
    static constexpr int A_BYTES = BM * ROW_BYTES, B_BYTES = BN * ROW_BYTES;
    static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
    static constexpr int LDS_BYTES = STAGES * STAGE_BYTES;
    static constexpr int A_LOADS = BM / 32, B_LOADS = BN / 32;  // 8 rows each, per wave
    static constexpr int LOADS = A_LOADS + B_LOADS;
    static_assert(LDS_BYTES <= 160 * 1024, "gfx950 has 160 KiB of LDS per workgroup");
    static_assert(STAGES >= 2 && LOADS * (STAGES - 2) <= 63, "vmcnt holds at most 63");
};

template <class T>
using Acc = f32x4[T::FM][T::FN];

template <class T, class OP>
__global__ void __launch_bounds__(T::THREADS, T::OCC) nt_tile(const OP op)
{
    using x8 = typename T::x8;
    __shared__ __attribute__((aligned(1024))) unsigned char smem[T::LDS_BYTES];
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int wm = wave / 2, wn = wave % 2;

    Tile t;
    if (!op.template tile<T::BM, T::BN>(blockIdx.x, t)) return;

    // Loads: load l of a wave fills rows 8 l .. 8 l + 7 of the wave's quarter
    // of the operand's tile; lane -> row lane / 8, position lane % 8, which
    // the swizzle fills with chunk pos ^ ((row / 2) % 8).  (A quarter starts
    // at a multiple of 16 rows, so the row's place within it decides.)
    const uint32_t pitch_a = (uint32_t)op.lda * 2u, pitch_b = (uint32_t)op.b_pitch(wave) * 2u;
    int na = 0, nb = 0;
    const void* pa = op.a_rows(t, wave * (T::BM / 4), na);
    const void* pb = op.template b_rows<T::BN>(t, wave * (T::BN / 4), nb);
    const __amdgpu_buffer_rsrc_t ra = make_rsrc(pa, (uint32_t)min(na, T::BM / 4) * pitch_a);
    const __amdgpu_buffer_rsrc_t rb = make_rsrc(pb, (uint32_t)min(nb, T::BN / 4) * pitch_b);
    const int lr = lane >> 3, lp = lane & 7;
    const int c0 = swizzle(lr, lp), c1 = swizzle(8 + lr, lp);
    const int K = op.K;
    auto issue = [&](int stage, int ks) __attribute__((always_inline)) {
        const int krem = K - ks * T::BK;
        const uint32_t koff = (uint32_t)ks * (T::BK * 2);
        unsigned char* base = smem + stage * T::STAGE_BYTES;
#pragma unroll
        for (int l = 0; l < T::A_LOADS; ++l) {
            const int c = l & 1 ? c1 : c0;
            const uint32_t off = c * 8 < krem ? koff + (uint32_t)(l * 8 + lr) * pitch_a + (uint32_t)c * 16u : kOob;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void*)(base + (wave * T::A_LOADS + l) * 1024), 16, off, 0,
                                                     0, 0);
        }
#pragma unroll
        for (int l = 0; l < T::B_LOADS; ++l) {
            const int c = l & 1 ? c1 : c0;
            const uint32_t off = c * 8 < krem ? koff + (uint32_t)(l * 8 + lr) * pitch_b + (uint32_t)c * 16u : kOob;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                rb, (lds_void*)(base + T::A_BYTES + (wave * T::B_LOADS + l) * 1024), 16, off, 0, 0, 0);
        }
    };

    const int fr = lane & 15, fh = lane >> 4;
    const int pos0 = swizzle(fr, fh) * 16, pos1 = swizzle(fr, 4 + fh) * 16;
    const int arow = (wm * T::WTM + fr) * T::ROW_BYTES;
    const int brow = T::A_BYTES + (wn * T::WTN + fr) * T::ROW_BYTES;

    Acc<T> acc;
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
    op.template epilogue<T>(t, acc, lane, wm, wn, smem);
}

// Stores four consecutive columns of one row: n .. n + 3 of N, as one 8-byte
// piece where `vec` says that rows take it.
template <class E>
__device__ __forceinline__ void store4(E* row, int n, int N, const f32x4& v, bool vec)
{
    const typename Elem<E>::x4 h = round4<E>(v);
    if (vec && n + 3 < N) {
        *(typename Elem<E>::x4*)(row + n) = h;
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (n + e < N) row[n + e] = h[e];
    }
}

// C = A B^T, `batch` products of one shape.
template <class E>
struct StoreOp {
    const E *A, *B;
    E* C[2];  // batch 0 and 1
    int M, N, K, lda, ldb, ldc, tiles_m, tiles_n, group_m, vec;
    int64_t stride_a;  // A of batch 1 (B is shared)

    template <int BM, int BN>
    __device__ __forceinline__ bool tile(int id, Tile& t) const
    {
        const int per = tiles_m * tiles_n;
        t.batch = id / per;
        int tm, tn;
        tile_of(id - t.batch * per, tiles_m, tiles_n, group_m, tm, tn);
        t.m0 = tm * BM;
        t.n0 = tn * BN;
        return true;
    }
    __device__ __forceinline__ const E* a_rows(const Tile& t, int row, int& n) const
    {
        return rows_from(A + t.batch * stride_a, t.m0 + row, M, lda, n);
    }
    template <int BN>
    __device__ __forceinline__ const E* b_rows(const Tile& t, int row, int& n) const
    {
        return rows_from(B, t.n0 + row, N, ldb, n);
    }
    __device__ __forceinline__ int b_pitch(int) const { return ldb; }
    template <class T>
    __device__ __forceinline__ void epilogue(const Tile& t, const Acc<T>& acc, int lane, int wm, int wn,
                                             unsigned char*) const
    {
        E* out = t.batch ? C[1] : C[0];
#pragma unroll
        for (int i = 0; i < T::FM; ++i) {
            const int m = t.m0 + wm * T::WTM + i * 16 + (lane & 15);
            if (m >= M) continue;
#pragma unroll
            for (int j = 0; j < T::FN; ++j)
                store4<E>(out + (int64_t)m * ldc, t.n0 + wn * T::WTN + j * 16 + 4 * (lane >> 4), N, acc[i][j], vec);
        }
    }
};

}  // namespace nt

#endif
