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
constexpr Kind kKinds[] = {{256, 256, 1450.0, 6.0}, {256, 128, 1280.0, 5.0}, {128, 128, 1060.0, 3.5}, {64, 64, 600.0, 3.0}};
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

// The split of a last wave of 128-wide tiles over all CUs (Split), and the
// time of the whole: the last wave's tiles take 1 / parts of their time, and
// joining them costs a launch and the partial sums' way out and back.
constexpr int kMaxParts = 256;  // of all tiles together: a workgroup for every CU of an MI355X
constexpr int64_t kSplitFloats = kMaxParts * (256 * 128);
constexpr int64_t kSplitK = 512;  // the shortest sum that is split

inline double split_us(const Kind& k, int64_t tiles, int64_t K, int cus, int& parts)
{
    const int64_t full = tiles / cus, rest = tiles % cus;
    const double us = 2.0 * k.bm * k.bn * (double)K / (k.tflops * 1e12 / 256) * 1e6;
    double best = -1;
    const int most = rest ? (int)std::min<int64_t>(std::min<int64_t>(std::min(cus, kMaxParts) / rest, 16), K / (kSplitK / 2)) : 1;
    for (int p = 2; p <= most; ++p) {
        // (measured: 1000 x 1032 x 5472 as 72 tiles in 3 parts 23 + 5 us,
        // as 36 of 256 x 128 in 7 parts 23 + 9)
        const double sum = (double)full * (us + k.wave_us) + us / p + k.wave_us + 8.0 + 0.4 * p * (k.bm / 128);
        if (best < 0 || sum < best) {
            best = sum;
            parts = p;
        }
    }
    return best;
}

// The last `rest` of the tiles in `parts` parts each, if that is more than one.
template <class T, class OP>
int launch_ordered(const OP& op, int tiles, int rest, int parts, float* partial, hipStream_t stream)
{
    const Split split{parts > 1 ? tiles - rest : tiles, parts, partial};
    const int units = split.full + (parts > 1 ? rest * parts : 0);
    hipLaunchKernelGGL((nt_ordered<T, OP>), dim3((unsigned)units), dim3(T::THREADS), 0, stream, op, split);
    int rc = (int)hipGetLastError();
    if constexpr (OP::kSplit)
        if (rc == hipSuccess && parts > 1) {
            hipLaunchKernelGGL((nt_join<T, OP>), dim3((unsigned)(rest * T::WAVES)), dim3(kJoinWaves * kWave), 0, stream, op, split);
            rc = (int)hipGetLastError();
        }
    return rc;
}

// Runs OP over `count(kind)` tiles with the kernel that the model finds
// fastest.  256 x 256 tiles need three K steps and an OP that offers them
// (kPersist); a split needs `partial` (kSplitFloats floats) and one that offers
// it (kSplit).
template <class E, class OP, class Count, class Prepare>
int launch(OP op, int64_t K, float* partial, Count count, Prepare prepare, hipStream_t stream)
{
    const int cus = num_cus();
    int best = -1, parts = 1;
    int64_t tiles = 0;
    double best_us = 0;
    for (int i = 0; i < kNumKinds; ++i) {
        if (i == 0 && (!OP::kPersist || K <= 128)) continue;
        const int64_t n = count(kKinds[i]);
        if (!abi::good_grid(n, i == 1 || i == 2 ? 512 : 256)) continue;
        const double us = model_us(kKinds[i], n, K, cus);
        if (best < 0 || us < best_us) {
            best = i;
            best_us = us;
            tiles = n;
            parts = 1;
        }
        int p = 1;
        const double split = (i == 1 || i == 2) && partial ? split_us(kKinds[i], n, K, cus, p) : -1;
        if (split > 0 && split < best_us) {
            best = i;
            best_us = split;
            tiles = n;
            parts = p;
        }
    }
    if (best < 0) return hipErrorInvalidValue;
    if (tiles == 0) return hipSuccess;
    op.tiles = (int)tiles;
    prepare(op, kKinds[best]);
    if constexpr (OP::kPersist)
        if (best == 0)
            hipLaunchKernelGGL((nt_persist<Shape256<E>, OP>), dim3((unsigned)std::min<int64_t>(tiles, cus)), dim3(256),
                               0, stream, op);
    if (best == 1)
        return launch_ordered<Shape<E, 256, 128, 4, 2, 3, 1, 4>>(op, (int)tiles, (int)(tiles % cus), parts, partial,
                                                                 stream);
    if (best == 2)
        return launch_ordered<Shape<E, 128, 128, 2, 4, 3, 1, 4>>(op, (int)tiles, (int)(tiles % cus), parts, partial,
                                                                 stream);
    // (four stages, two workgroups to a CU: 30.8 us with three for one row and
    // 4096 x 8192 twice, 29.7 with four, 29.5 with five, which take all of LDS)
    if (best == 3)
        hipLaunchKernelGGL((nt_tile<Shape<E, 64, 64, 2, 2, 4, 2, 4>, OP>), dim3((unsigned)tiles), dim3(256), 0, stream, op);
    return (int)hipGetLastError();
}

// The largest of the kinds that every OP has, 256 x 128, can hold the result.
inline bool fits(int64_t rows, int64_t cols, int64_t batch)
{
    return abi::good_grid((rows + 255) / 256 * ((cols + 127) / 128) * batch, 512);
}

// A rows x cols grid of tiles, `batch` times; `split` columns of the product
// make one column of the result (2 for the gated layer).
template <class E, class OP>
int launch_grid(const OP& op, int64_t rows, int64_t cols, int split, int64_t batch, int64_t K, float* partial,
                hipStream_t stream)
{
    auto tm = [=](const Kind& k) { return (rows + k.bm - 1) / k.bm; };
    auto tn = [=](const Kind& k) { return (cols * split + k.bn - 1) / k.bn; };
    return launch<E>(
        op, K, partial, [=](const Kind& k) { return tm(k) * tn(k) * batch; },
        [=](OP& o, const Kind& k) {
            o.tiles_m = (int)tm(k);
            o.tiles_n = (int)tn(k);
        },
        stream);
}

}  // namespace nt

#endif
