// Host side of the tiled products: which tile runs a shape, and its launch.
#ifndef DENSE_FP16_GEMM_NT_LAUNCH_H
#define DENSE_FP16_GEMM_NT_LAUNCH_H

#include <algorithm>

#include "abi.h"
#include "nt_core.h"

namespace nt {

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

// The kernels, by their tiles, with the rate that each sustains on a full
// chip and the fixed cost of a wave of tiles (pipeline fill and epilogue).
struct Kind {
    int bm, bn;
    double tflops;  // on 256 CUs
    double wave_us;
};
constexpr Kind kKinds[] = {{256, 256, 1450.0, 4.0}, {256, 128, 1250.0, 3.0}, {128, 128, 1050.0, 3.0}, {64, 64, 480.0, 3.0}};
constexpr int kNumKinds = 4;

// Time of `tiles` tiles of sums over K: whole waves of tiles over the CUs at
// the kernel's rate plus the fixed cost of each; a wave that leaves CUs idle
// runs the others up to 1.25 times faster (clock and L2 headroom).
inline double model_us(const Kind& k, int64_t tiles, int64_t K, int cus)
{
    const int64_t full = tiles / cus, rest = tiles % cus;
    const double us = 2.0 * k.bm * k.bn * (double)K / (k.tflops * 1e12 / 256) * 1e6;
    double sum = (double)full * (us + k.wave_us);
    if (rest) sum += us / (1.0 + 0.25 * (1.0 - (double)rest / cus)) + k.wave_us;
    return sum;
}

// Runs OP over `count(kind)` tiles with the kernel that the model finds
// fastest (a count of -1: not with this kind).  256 x 256 tiles need three K
// steps and an OP that offers them (kPersist).
template <class E, class OP, class Count, class Prepare>
int launch(OP op, int64_t K, Count count, Prepare prepare, hipStream_t stream)
{
    const int cus = num_cus();
    int best = -1;
    int64_t tiles = 0;
    double best_us = 0;
    for (int i = 0; i < kNumKinds; ++i) {
        if (i == 0 && (!OP::kPersist || K <= 128)) continue;
        const int64_t n = count(kKinds[i]);
        if (n < 0) continue;
        const double us = model_us(kKinds[i], n, K, cus);
        if (best < 0 || us < best_us) {
            best = i;
            best_us = us;
            tiles = n;
        }
    }
    if (tiles > abi::kMaxDim) return hipErrorInvalidValue;
    if (tiles == 0) return hipSuccess;
    op.tiles = (int)tiles;
    prepare(op, kKinds[best]);
    const dim3 grid((unsigned)tiles);
    if constexpr (OP::kPersist)
        if (best == 0)
            hipLaunchKernelGGL((nt_persist<Shape256<E>, OP>), dim3((unsigned)std::min<int64_t>(tiles, cus)), dim3(256),
                               0, stream, op);
    if constexpr (OP::kOblong)
        if (best == 1)
            hipLaunchKernelGGL((nt_ordered<Shape<E, 256, 128, 4, 2, 3, 1, 4>, OP>), grid, dim3(512), 0, stream, op);
    if (best == 2)
        hipLaunchKernelGGL((nt_ordered<Shape<E, 128, 128, 2, 4, 3, 1, 4>, OP>), grid, dim3(512), 0, stream, op);
    if (best == 3) hipLaunchKernelGGL((nt_tile<Shape<E, 64, 64, 2, 2, 3, 2, 4>, OP>), grid, dim3(256), 0, stream, op);
    return (int)hipGetLastError();
}

// A rows x cols grid of tiles, `batch` times; `split` columns of the product
// make one column of the result (2 for the gated layer).
template <class E, class OP>
int launch_grid(const OP& op, int64_t rows, int64_t cols, int split, int64_t batch, int64_t K, hipStream_t stream)
{
    auto tm = [=](const Kind& k) { return (rows + k.bm - 1) / k.bm; };
    auto tn = [=](const Kind& k) { return (cols * split + k.bn - 1) / k.bn; };
    return launch<E>(
        op, K, [=](const Kind& k) { return tm(k) * tn(k) * batch; },
        [=](OP& o, const Kind& k) {
            o.tiles_m = (int)tm(k);
            o.tiles_n = (int)tn(k);
        },
        stream);
}

}  // namespace nt

#endif
