// How many CUs the current device has, and an MI355X (for what sizes a workspace or
// orders a sum, and so may not depend on the device that is current).
#ifndef DENSE_FP16_GEMM_CUS_H
#define DENSE_FP16_GEMM_CUS_H

#include <hip/hip_runtime.h>

namespace cus {

constexpr int kCus = 256;

inline int num_cus()
{
    static int cache[64];
    int device = 0;
    if (hipGetDevice(&device) != hipSuccess || device < 0 || device >= 64) return 256;
    int n = __atomic_load_n(&cache[device], __ATOMIC_RELAXED);
    if (n == 0) {
        if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, device) != hipSuccess || n <= 0) n = 256;
        __atomic_store_n(&cache[device], n, __ATOMIC_RELAXED);
    }
    return n;
}

}  // namespace cus

#endif
