// Device building blocks of the operators beside the fp16 product: element
// types, buffer resources, global->LDS loads, waits, the LDS swizzle and the
// XCD-aware tile order.
#ifndef DENSE_FP16_GEMM_CDNA4_H
#define DENSE_FP16_GEMM_CDNA4_H

#include <hip/hip_runtime.h>

#include <stdint.h>

namespace cdna4 {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) void lds_void;

constexpr int kWave = 64;
constexpr int kXcds = 8;                // MI355X: 8 dies, workgroups dealt to them in turn
constexpr uint32_t kOob = 0x80000000u;  // a buffer offset past every tile: loads 0, stores nothing
constexpr int kRsrcWord3 = 0x00020000;  // buffer resource word 3: 32-bit data, no swizzle

// A 16-bit element type: its vectors, the MFMA that multiplies it, and its
// rounding (to nearest, ties to even, both by one conversion instruction).
template <class E>
struct Elem;

template <>
struct Elem<_Float16> {
    typedef _Float16 x4 __attribute__((ext_vector_type(4)));
    typedef _Float16 x8 __attribute__((ext_vector_type(8)));
    static __device__ __forceinline__ f32x4 mfma(const x8& a, const x8& b, const f32x4& c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
};

template <>
struct Elem<__bf16> {
    typedef __bf16 x4 __attribute__((ext_vector_type(4)));
    typedef __bf16 x8 __attribute__((ext_vector_type(8)));
    static __device__ __forceinline__ f32x4 mfma(const x8& a, const x8& b, const f32x4& c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
};

template <class E>
__device__ __forceinline__ typename Elem<E>::x4 round4(const f32x4& v)
{
    typename Elem<E>::x4 r;
    r[0] = (E)v[0];
    r[1] = (E)v[1];
    r[2] = (E)v[2];
    r[3] = (E)v[3];
    return r;
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* base, uint32_t bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, kRsrcWord3);
}

// 16 bytes to each lane's place in LDS, `to` plus 16 times the lane.
__device__ __forceinline__ void load_lds(__amdgpu_buffer_rsrc_t from, lds_void* __restrict to, uint32_t off, uint32_t soff)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(from, to, 16, off, soff, 0, 0);
}

// Wait until at most VM of this wave's vector memory accesses are in flight
// and its LDS accesses are done, then meet the workgroup's other waves.  One
// asm statement, so that no access moves across it; __syncthreads() would
// wait for every load in flight.
template <int VM>
__device__ __forceinline__ void lds_barrier()
{
    static_assert(VM >= 0 && VM <= 63, "vmcnt holds 0 .. 63");
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"i"(VM) : "memory");
}

// Four 16-bit values of each lane's from LDS, turned among 16 lanes: lane l gets
// value l % 4 of lanes 4 e + l / 4, e = 0 .. 3.  (Lanes 4 e .. 4 e + 3 read 16
// columns of row e, and lane l gets column l of four rows.)  `__restrict`, here and in
// load_lds: else the compiler waits before each such read for all loads into LDS that
// are in flight, where the barriers have waited for those that matter.
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
__device__ __forceinline__ s16x4 read_turned(lds_s16x4* __restrict p) { return __builtin_amdgcn_ds_read_tr16_b64_v4i16(p); }
template <class E>
__device__ __forceinline__ typename Elem<E>::x4 read_turned(const unsigned char* p)
{
    return __builtin_bit_cast(typename Elem<E>::x4, read_turned((lds_s16x4*)p));
}

// LDS tiles hold 128-byte rows (64 elements) as eight 16-byte chunks; chunk
// c of row r sits at c ^ ((r / 2) % 8), so the 16 lanes that one pass of a
// 16-byte read serves fall on 16 different bank groups.
__device__ __forceinline__ int swizzle(int row, int chunk) { return chunk ^ ((row >> 1) & 7); }

// Workgroup (or persistent tile) number -> place in the linear order of all
// tiles.  Workgroups are dealt to the XCDs in turn, so numbers are renamed to
// give each XCD, with its own L2, one contiguous range.
__device__ __forceinline__ int xcd_order(int id, int total)
{
    const int per = total / kXcds, extra = total % kXcds;
    const int x = id % kXcds;
    return x * per + (x < extra ? x : extra) + id / kXcds;
}

// Place in the linear order of one matrix -> tile.  Groups of eight tile rows
// are swept column by column, so tiles that run together share rows of both
// operands.
__device__ __forceinline__ void grid_tile(int lin, int tiles_m, int tiles_n, int& tm, int& tn)
{
    constexpr int group_m = 8;
    const int width = group_m * tiles_n;
    const int g = lin / width;
    const int first = g * group_m;
    const int rows = min(tiles_m - first, group_m);
    const int r = lin - g * width;
    tm = first + r % rows;
    tn = r / rows;
}

// The same for the tiles that reach the diagonal of a square matrix of
// `tiles` tile rows or lie below it, q tiles wide to each tile row's height:
// of a group's rows first the columns before the group's own, then the rest
// row by row.
__device__ __forceinline__ void triangle_tile(int lin, int tiles, int q, int& tm, int& tn)
{
    constexpr int group_m = 8;
    auto before = [=](int row) { return q * (row * (row + 1) / 2); };
    int row = (int)((__builtin_sqrtf(8.0f * (float)(lin / q) + 1.0f) - 1.0f) * 0.5f);  // off by one at most
    while (before(row) > lin) --row;
    while (before(row + 1) <= lin) ++row;
    const int first = row / group_m * group_m, rows = min(tiles - first, group_m);
    int r = lin - before(first);
    if (r < rows * q * first) {
        tm = first + r % rows;
        tn = r / rows;
        return;
    }
    r -= rows * q * first;
    int i = 0;
    while (before(i + 1) <= r) ++i;
    tm = first + i;
    tn = q * first + r - before(i);
}

}  // namespace cdna4

#endif
