// Host-side argument checks and workspace layout shared by the C entry points.
#ifndef DENSE_FP16_GEMM_ABI_H
#define DENSE_FP16_GEMM_ABI_H

#include <hip/hip_runtime.h>

#include <stdint.h>

namespace abi {

constexpr int64_t kMaxDim = ((int64_t)1 << 31) - 1;
// 256 rows of an operand span less than 2^30 bytes: the reach of the
// kernels' 32-bit buffer offsets, with the mark for "nothing" beyond it.
constexpr int64_t kMaxPitch = ((int64_t)1 << 21) - 1;

inline int64_t up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

// Bytes [first, last) of a rows x cols matrix with rows `ld` elements apart.
struct Range {
    uintptr_t first = 0, last = 0;
    Range() = default;
    Range(const void* p, int64_t rows, int64_t cols, int64_t ld, int64_t elem)
    {
        if (rows > 0 && cols > 0) {
            first = (uintptr_t)p;
            last = first + (uintptr_t)(((rows - 1) * ld + cols) * elem);
        }
    }
    bool meets(const Range& o) const { return first < o.last && o.first < last; }
};

// A pointer is given and aligned, or there is nothing behind it.
inline bool good_pointer(const void* p, int64_t rows, int64_t cols, uintptr_t align)
{
    return rows == 0 || cols == 0 || (p && (uintptr_t)p % align == 0);
}

inline bool good_dim(int64_t n) { return n >= 0 && n <= kMaxDim; }
// What one launch may hold: 2^32 - 1 threads in a dimension.
inline bool good_grid(int64_t workgroups, int64_t threads) { return workgroups <= (((int64_t)1 << 32) - 1) / threads; }
inline bool good_pitch(int64_t ld, int64_t cols) { return ld >= cols && ld <= kMaxPitch; }

// Hands out 16-byte aligned pieces of a workspace; with no base it only adds
// up the sizes.
class Carve {
  public:
    explicit Carve(void* base) : base_((unsigned char*)base) {}
    template <class T>
    T* take(int64_t elements)
    {
        T* p = base_ ? (T*)(base_ + used_) : nullptr;
        used_ += up(elements * (int64_t)sizeof(T), 256);
        return p;
    }
    int64_t used() const { return used_; }

  private:
    unsigned char* base_;
    int64_t used_ = 0;
};

}  // namespace abi

#endif
