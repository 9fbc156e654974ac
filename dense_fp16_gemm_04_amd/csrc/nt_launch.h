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

// Time of `tiles` tiles of edge x edge sums over K: whole waves of tiles over
// the CUs at the rate that the kernel sustains on a full chip, plus a fixed
// cost per wave; a wave that leaves CUs idle runs the others up to 1.25 times
// faster (clock and L2 headroom).
struct Kind {
    int edge;
    double tflops;   // on a full chip of 256 CUs
    double wave_us;  // pipeline fill and epilogue
};
constexpr Kind kKinds[] = {{256, 1450.0, 4.0}, {128, 760.0, 3.0}, {64, 480.0, 3.0}};

inline double model_us(const Kind& k, int64_t tiles, int64_t K, int cus)
{
    const int64_t full = tiles / cus, rest = tiles % cus;
    const double us = 2.0 * k.edge * k.edge * (double)K / (k.tflops * 1e12 / 256) * 1e6;
    double sum = (double)full * (us + k.wave_us);
    if (rest) sum += us / (1.0 + 0.25 * (1.0 - (double)rest / cus)) + k.wave_us;
    return sum;
}

// Runs OP over `count(edge)` tiles with the kernel that the model finds
// fastest.  256 x 256 tiles need three K steps and
// an OP that offers them (kPersist).
template <class E, class OP, class Count, class Prepare>
int launch(OP op, int64_t K, Count count, Prepare prepare, hipStream_t stream)
{
    const int cus = num_cus();
    int best = -1;
    double best_us = 0;
    for (int i = 0; i < 3; ++i) {
        if (kKinds[i].edge == 256 && (!OP::kPersist || K <= 128)) continue;
        const double us = model_us(kKinds[i], count(kKinds[i].edge), K, cus);
        if (best < 0 || us < best_us) {
            best = i;
            best_us = us;
        }
    }
    const int64_t tiles = count(kKinds[best].edge);
    if (tiles > abi::kMaxDim) return hipErrorInvalidValue;
    if (tiles == 0) return hipSuccess;
    op.tiles = (int)tiles;
    prepare(op, kKinds[best].edge);
    if constexpr (OP::kPersist) {
        if (best == 0) {
            hipLaunchKernelGGL((nt_persist<Shape256<E>, OP>), dim3((unsigned)std::min<int64_t>(tiles, cus)), dim3(256),
                               0, stream, op);
            return (int)hipGetLastError();
        }
    }
    if (best == 1)
        hipLaunchKernelGGL((nt_tile<Shape<E, 128, 128, 3, 1>, OP>), dim3((unsigned)tiles), dim3(256), 0, stream, op);
    else
        hipLaunchKernelGGL((nt_tile<Shape<E, 64, 64, 3, 2>, OP>), dim3((unsigned)tiles), dim3(256), 0, stream, op);
    return (int)hipGetLastError();
}

// A rows x cols grid of tiles, `batch` times; `split` columns of the product
// make one column of the result (2 for the gated layer).
template <class E, class OP>
int launch_grid(const OP& op, int64_t rows, int64_t cols, int split, int64_t batch, int64_t K, hipStream_t stream)
{
    auto tm = [=](int64_t edge) { return (rows + edge - 1) / edge; };
    auto tn = [=](int64_t edge) { return (cols * split + edge - 1) / edge; };
    return launch<E>(
        op, K, [=](int64_t edge) { return tm(edge) * tn(edge) * batch; },
        [=](OP& o, int edge) {
            o.tiles_m = (int)tm(edge);
            o.tiles_n = (int)tn(edge);
        },
        stream);
}

}  // namespace nt

#endif
