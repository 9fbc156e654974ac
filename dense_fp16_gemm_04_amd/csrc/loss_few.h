// The loss over a vocabulary for up to 16 tokens, where reading W is most of the
// work (included by linear_cross_entropy.hip).
//
// W is read where it lies, at any alignment, 16 bytes to a lane: no copies, no
// transposes.  Outputs are products by the matrix cores of blocks of 16 rows of W
// with all tokens.  dl is 32 bits, never rounded, and both gradients are sums by
// the vector units in one pass over W: dX += dl W[v] and dW[v] = sum dl X of a row v.
// (8 x 2048 x 32000, bound by W's 131 MB: the loss 28.5 us, 4.6 TB/s, dl 21.5, the
// gradients, which write as much, 63.)
#ifndef DENSE_FP16_GEMM_LOSS_FEW_H
#define DENSE_FP16_GEMM_LOSS_FEW_H

#include "cus.h"
#include "rows.h"

namespace few {

using namespace cdna4;

constexpr int kTokens = 16;   // the most
constexpr int kWaves = 4;     // of a workgroup, which take K's steps of 32 in turn
constexpr int kRows = 32;     // of W to a part at least

// B blocks of 16 rows of W to a workgroup at a time: four, with half the loads of X,
// where they are enough for the chip (8 tokens by 32000 x 2048, a graph's replay: 34.0 us with
// two, 30.3 with four; 3 by 13991 x 640 15.0 and 15.9).
inline int blocks_of(int64_t V) { return V >= 96 * cus::kCus ? 4 : 2; }

// The outputs of 16 B rows of W from `first` on: wave b has block b, lane l token l % 16
// and rows 4 (l / 16) .. + 3 of it, once all waves' shares have met in `part`.
template <class E, int B>
__device__ __forceinline__ f32x4 outputs(const E* X, const E* W, int64_t ldx, int64_t ldw, int T, int D, int V, int64_t first,
                                         f32x4 (&part)[kWaves][B][kWave])
{
    using x8 = typename Elem<E>::x8;
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave, r = lane & 15, q = lane >> 4;
    const E* const x = X + min(r, T - 1) * ldx;
    const E* w[B];
    f32x4 acc[B];
#pragma unroll
    for (int b = 0; b < B; ++b) {
        w[b] = W + min(first + b * 16 + r, (int64_t)V - 1) * ldw;
        acc[b] = f32x4{0, 0, 0, 0};
    }
    // eight steps' loads in flight; in the last round, of steps that may reach past
    // K or not be there (zeros)
    constexpr int AHEAD = 8;
    // The last eight of a K that is no multiple end with it.  What the eight before
    // hold too is then zeros in both operands: zero times an infinity is NaN.
    const int twice = D < 8 ? 0 : -D & 7, last = twice ? D & ~7 : -1;
    u32x4 keep;
#pragma unroll
    for (int i = 0; i < 4; ++i) keep[i] = twice <= 2 * i ? ~0u : twice == 2 * i + 1 ? 0xffff0000u : 0u;
    auto round = [&](int s, auto all) __attribute__((always_inline)) {
        constexpr bool ALL = decltype(all)::value;
        auto load8 = [&](const E* p, int k) __attribute__((always_inline)) {
            rows::Vec<E, 8> v = {};
            if (ALL || k < D) v = rows::load<E, 8>(p + (ALL || D < 8 ? k : min(k, D - 8)), ALL || D >= 8 ? 8 : D - k);
            u32x4 words = __builtin_bit_cast(u32x4, v);
            if constexpr (!ALL)
#pragma unroll
                for (int i = 0; i < 4; ++i) words[i] &= k == last ? keep[i] : ~0u;
            return __builtin_bit_cast(x8, words);
        };
        x8 fx[AHEAD], fw[AHEAD][B];
#pragma unroll
        for (int a = 0; a < AHEAD; ++a) {
            const int k = (s + a * kWaves) * 32 + q * 8;
            fx[a] = load8(x, k);
#pragma unroll
            for (int b = 0; b < B; ++b) fw[a][b] = load8(w[b], k);
        }
#pragma unroll
        for (int a = 0; a < AHEAD; ++a)
#pragma unroll
            for (int b = 0; b < B; ++b) acc[b] = Elem<E>::mfma(fw[a][b], fx[a], acc[b]);
    };
    int s = wave;
    for (; s + (AHEAD - 1) * kWaves < D / 32; s += AHEAD * kWaves) round(s, nt::Flag<true>{});
    if (s * 32 < D) round(s, nt::Flag<false>{});
#pragma unroll
    for (int b = 0; b < B; ++b) part[wave][b][lane] = acc[b];
    __syncthreads();
    f32x4 l = {0, 0, 0, 0};
    if (wave < B) {
#pragma unroll
        for (int v = 0; v < kWaves; ++v) l += part[v][wave][lane];
    }
    __syncthreads();
    return l;
}

template <class E>
struct Lse {
    const E *X, *W;
    const int64_t* target;
    float* tl;
    f32x2* parts;  // [workgroups' blocks][kTokens]
    int64_t target_stride, ldx, ldw;
    int T, D, V;
};

template <class E, int B>
__global__ void __launch_bounds__(kWaves* kWave) few_lse(const Lse<E> f)
{
    __shared__ f32x4 part[kWaves][B][kWave];
    __shared__ f32x2 meet[kWaves][kTokens];
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave, t = lane & 15;
    const int64_t blocks = ((int64_t)f.V + 16 * B - 1) / (16 * B);
    for (int64_t block = blockIdx.x; block < blocks; block += gridDim.x) {
        f32x4 l = outputs<E, B>(f.X, f.W, f.ldx, f.ldw, f.T, f.D, f.V, block * (16 * B), part);
        const int64_t v0 = block * (16 * B) + wave * 16 + 4 * (lane >> 4);
        f32x2 p = {-INFINITY, 0.0f};
        if (wave < B) {
            const int64_t at = t < f.T ? f.target[t * f.target_stride] - v0 : -1;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (v0 + e >= f.V)
                    l[e] = -INFINITY;
                else if (at == e)
                    f.tl[t] = l[e];
            }
            p[0] = max_over_groups(fmaxf(fmaxf(l[0], l[1]), fmaxf(l[2], l[3])));
            float sum = 0.0f;
#pragma unroll
            for (int e = 0; e < 4; ++e) sum += __builtin_amdgcn_exp2f((l[e] - about(p[0])) * kLog2e);
            p[1] = sum_over_groups(sum);
        }
        if (lane < kTokens) meet[wave][lane] = p;
        __syncthreads();
        if (wave == 0 && lane < kTokens) {
            p = joined(p, meet[1][lane]);
            if constexpr (B == 4) p = joined(p, joined(meet[2][lane], meet[3][lane]));
            f.parts[block * kTokens + lane] = p;
        }
    }
}

// dl[v][16 tokens], 32 bits: zeros for tokens that are ignored or not there.
template <class E>
struct Dl {
    const E *X, *W;
    const int64_t* target;
    const float *dloss, *saved;
    float* dl;
    int64_t target_stride, dloss_stride, ignore, ldx, ldw;
    int T, D, V;
};

template <class E, int B>
__global__ void __launch_bounds__(kWaves* kWave) few_dl(const Dl<E> f)
{
    __shared__ f32x4 part[kWaves][B][kWave];
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave, t = lane & 15;
    float top = 0.0f, bias = -INFINITY, g = 0.0f, hit = 0.0f;
    int64_t c = -1;
    if (t < f.T && f.target[t * f.target_stride] != f.ignore) {
        c = f.target[t * f.target_stride];
        const float sum = f.saved[3 * t + 1], tl = f.saved[3 * t + 2];
        top = f.saved[3 * t];
        bias = c >= 0 && c < f.V ? -log2f(sum) : NAN;
        g = f.dloss[t * f.dloss_stride];
        hit = (expf(tl - top) - sum) / sum;
    }
    const int64_t blocks = ((int64_t)f.V + 16 * B - 1) / (16 * B);
    for (int64_t block = blockIdx.x; block < blocks; block += gridDim.x) {
        const f32x4 l = outputs<E, B>(f.X, f.W, f.ldx, f.ldw, f.T, f.D, f.V, block * (16 * B), part);
        const int64_t v0 = block * (16 * B) + wave * 16 + 4 * (lane >> 4);
        if (wave < B)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                // (the minimum as in RowInfo)
                const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(fminf(l[e] - top, 0.0f), kLog2e, bias));
                if (v0 + e < f.V) f.dl[(v0 + e) * kTokens + t] = g * (v0 + e == c ? hit : p);
            }
    }
}

// Both gradients of a share of W's rows, NC columns to a thread: dW's rows, and the
// share's sums for dX.  TT: tokens that the registers have room for.
template <class E>
struct Grads {
    const E *X, *W;
    const int64_t* target;
    const float* dl;
    E* dW;
    float* partial;  // [shares][T][D]
    int64_t target_stride, ignore, ldx, ldw, lddw;
    int T, D, V, per;  // rows to a share
};
constexpr int kGradThreads = 256;

template <class E, int TT, int NC>
__global__ void __launch_bounds__(kGradThreads) few_grads(const Grads<E> f)
{
    typedef rows::Vec<E, NC> V;
    int64_t c = ((int64_t)blockIdx.y * kGradThreads + threadIdx.x) * NC;
    if (c >= f.D) return;
    // (the last columns of a D that is no multiple end with it: some are then made
    // twice, alike: steps of 8 x 333 x 30001
    // 108 us with single elements, and 75)
    if (f.D >= NC) c = min(c, (int64_t)f.D - NC);
    const int left = (int)std::min<int64_t>(f.D - c, NC);
    float x[TT][NC], sum[TT][NC];
    V v[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) v[t] = rows::load<E, NC>(f.X + min(t, f.T - 1) * f.ldx + c, left);
#pragma unroll
    for (int t = 0; t < TT; ++t) {
        // (of a token that is ignored nothing counts: 0 times what it holds may be NaN)
        const bool counts = t < f.T && f.target[min(t, f.T - 1) * f.target_stride] != f.ignore;
#pragma unroll
        for (int k = 0; k < NC; ++k) {
            x[t][k] = counts ? (float)v[t][k] : 0.0f;
            sum[t][k] = 0.0f;
        }
    }
    const int64_t begin = (int64_t)blockIdx.x * f.per, end = std::min<int64_t>(begin + f.per, f.V);
    const E* w = f.W + begin * f.ldw + c;
    E* to = f.dW + begin * f.lddw + c;
    const float* dl = f.dl + begin * kTokens;
    auto row = [&](const V& v, const float* d, E* out) __attribute__((always_inline)) {
        float o[NC];
#pragma unroll
        for (int k = 0; k < NC; ++k) o[k] = 0.0f;
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            const float g = d[t];
#pragma unroll
            for (int k = 0; k < NC; ++k) {
                o[k] = __builtin_fmaf(g, x[t][k], o[k]);
                sum[t][k] = __builtin_fmaf(g, (float)v[k], sum[t][k]);
            }
        }
        V r;
#pragma unroll
        for (int k = 0; k < NC; ++k) r[k] = (E)o[k];
        rows::store<E, NC>(out, left, r);
    };
    constexpr int AHEAD = 4;
    int64_t n = begin;
    for (; n + AHEAD <= end; n += AHEAD) {
        V v[AHEAD];
#pragma unroll
        for (int a = 0; a < AHEAD; ++a) v[a] = rows::load<E, NC>(w + a * f.ldw, left);
#pragma unroll
        for (int a = 0; a < AHEAD; ++a) row(v[a], dl + a * kTokens, to + a * f.lddw);
        w += AHEAD * f.ldw;
        to += AHEAD * f.lddw;
        dl += AHEAD * kTokens;
    }
    for (; n < end; ++n) {
        row(rows::load<E, NC>(w, left), dl, to);
        w += f.ldw;
        to += f.lddw;
        dl += kTokens;
    }
#pragma unroll
    for (int t = 0; t < TT; ++t)
        if (t < f.T) {
            float* const at = f.partial + ((int64_t)blockIdx.x * f.T + t) * f.D + c;
            rows::Vec<float, NC> s;
#pragma unroll
            for (int k = 0; k < NC; ++k) s[k] = sum[t][k];
            rows::store<float, NC>(at, left, s);
        }
}

// dX of the shares' sums.
template <class E>
struct Sum {
    const float* partial;
    const int64_t* target;
    E* dX;
    int64_t target_stride, ignore, ldx;
    int T, D, shares;
};

template <class E, int C>
__global__ void __launch_bounds__(rows::kSumThreads) few_sum(const Sum<E> f)
{
    const int t = blockIdx.y;
    const int64_t c = (int64_t)blockIdx.x * C + threadIdx.x % C;
    const float sum = rows::columns_sum<C>(c < f.D ? f.partial + (int64_t)t * f.D + c : nullptr, (int64_t)f.T * f.D, f.shares);
    if (threadIdx.x < C && c < f.D) f.dX[t * f.ldx + c] = f.target[t * f.target_stride] == f.ignore ? (E)0.0f : (E)sum;
}

}  // namespace few

#endif
