// na_glu.h -- the gated feed-forward product's parameters and activations, shared by its host code (na_glu.cu), its CUDA-core kernels
// (na_glu_fma.cuh) and its tensor-core kernels (na_glu_tc.cuh).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/na.h"
#include "na_device.cuh"
#include "na_glu_plan.h"

namespace na {
namespace glu {

struct GluParams {
    const void* x;        // [T, D]
    const void* wg;       // [F, D]
    const void* wu;
    const void* bg;       // [F], null: zeros
    const void* bu;
    const void* dh;       // [T, F]
    void* h;              // [T, F]
    void* dg;             // [T, pitch], workspace
    void* du;
    void* dx;             // [T, D]
    void* dwg;            // [F, D]
    void* dwu;
    float* partial;       // sums of several splits: [split][2][F][D] of kWeights, [split][T][D] of kTokens
    float* sums;          // kSlopes: sums of dg and du over the rows of a tile, [tile][2][sum_pitch]; null: not wanted
    int sum_pitch;
    long long T, pitch;   // pitch: F rounded up to whole 16-byte chunks
    int D, F;
    int act;              // na_glu_act
    int splits;           // CUDA cores: as FmaTile
    long long run;
};

// The tiles of kTokens or kWeights: rows (kWeights: of dWg and dWu together) x cols.  Each is the sum of `splits` parts of the
// `steps` steps of 64 along the summed axis: part w + ways t takes the steps w + ways (t run + j), j < run; none is empty.
struct GluJob {
    unsigned rows, cols, splits, ways, run, steps;
};

// Parameters of the tensor-core kernels.
struct GluTcParams {
    CUtensorMap a[2];     // rows' operand: x; dg, du
    CUtensorMap b[4];     // columns' operand: Wg, Wu and (forward, slopes) again in boxes for a row's last tile; [2]: x (weights)
    CUtensorMap in;       // slopes: dh (where its rows are not whole chunks a copy in dg's place: a warp's box of it is read before dg is written)
    CUtensorMap out[2];   // forward: h; slopes: dg, du
    const void* bg;
    const void* bu;
    const void* dh;
    void* h;
    void* dg;
    void* du;
    void* dx;
    void* dwg;
    void* dwu;
    float* partial;
    float* sums;          // slopes: as in GluParams, of 32 tokens, or of all few ones; null: not wanted
    long long pitch;      // of dg and du
    int T, D, F, act, sum_pitch;
    uint32_t wide;        // rows of h are whole 16-byte chunks
    GluJob job[2];        // tokens, weights
    unsigned token_workers;   // both: pairs of blocks that make dx
    unsigned rows, cols;  // forward, slopes: tiles
    unsigned last_nf;     // forward, slopes: columns of g (and of u) of a row's last tile
    unsigned span, groups;   // forward, slopes: columns of tiles that a block takes in a row, and such runs of a row
    unsigned splits;      // few tokens: blocks to a tile's sum
    unsigned steps, run;  // forward, slopes: steps of 64 along the summed axis; few tokens: of one block
    unsigned* err;
    unsigned long long wait_ns;
    uint32_t withhold;
};

// act(v) and its derivative.  FAST: exponentials and reciprocals of the hardware's approximations (results below 2^-126 are
// zeros).  An exponential's error grows with its argument: act(v) is off by less than 2^-17 of its value down to values of 2^-46, by
// less than 2^-15.5 below (GELU's tanh form, whose argument is a cubic; the others 2^-16.9).  Else the full ones of fp32, zeros where
// the exponential's inverse leaves fp32 (below 2^-121).
template <int ACT>   // an activation as a type
struct ActTag {
    static constexpr int value = ACT;
};

template <bool FAST>
__device__ __forceinline__ float exp_of(float v) {
    if constexpr (FAST) return dev::fast_exp2(v * 1.4426950408889634f);
    else return expf(v);
}
template <bool FAST>
__device__ __forceinline__ float inverse(float v) {
    if constexpr (FAST) {
        float y;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(v));
        return y;
    } else {
        return 1.f / v;
    }
}

template <int ACT, bool FAST>
__device__ __forceinline__ void activate(float v, float& a, float& slope) {
    if constexpr (ACT == NA_ACT_RELU) {
        a = v < 0.f ? 0.f : v;   // a NaN stays one
        slope = v > 0.f ? 1.f : 0.f;
    } else if constexpr (ACT == NA_ACT_GELU) {
        // v Phi(v), and Phi(v) + v phi(v); the complementary error function keeps Phi's digits far below zero
        const float cdf = 0.5f * erfcf(v * -0.70710678118654752f);
        a = v * cdf;
        slope = fmaf(v * 0.39894228040143268f, exp_of<FAST>(-0.5f * v * v), cdf);
    } else if constexpr (ACT == NA_ACT_GELU_TANH) {
        // (1 + tanh t) / 2 = 1 / (1 + exp(-2 t)), t = sqrt(2 / pi) (v + 0.044715 v^3); beyond |v| = 100 it is 0 or 1
        const float v2 = fminf(v * v, 10000.f), t2 = v * fmaf(v2, 2.f * 0.79788456080286536f * 0.044715f, 2.f * 0.79788456080286536f);
        const float y = inverse<FAST>(1.f + exp_of<FAST>(-t2));
        const float rise = fmaf(v2, 6.f * 0.79788456080286536f * 0.044715f, 2.f * 0.79788456080286536f);
        a = v * y;
        slope = fmaf(a * (1.f - y), rise, y);
    } else {
        const float e = exp_of<FAST>(-v), y = inverse<FAST>(1.f + e);
        if constexpr (ACT == NA_ACT_SIGMOID) {
            a = y;
            slope = y * (v > 0.f ? e * y : 1.f - y);   // 1 - y without cancellation on either side
        } else {
            a = v * y;
            slope = fmaf(a, 1.f - y, y);
        }
    }
}

// act and its derivative of eight values, with the approximations, in pairs of fp32 operations.  Each value has a reciprocal of
// its own: one for two, 1 / p = q / (p q), is no faster here (its exponentials and products are not what bounds the kernels), and
// a value's bits would depend on its neighbour's.
template <int ACT>
__device__ __forceinline__ void activate8(const float (&v)[8], float (&a)[8], float (&slope)[8]) {
    using namespace dev;
    constexpr float L = 1.4426950408889634f, K = 2.f * 0.79788456080286536f;
    const uint64_t one = pack2(1.f, 1.f);
    if constexpr (ACT == NA_ACT_RELU) {
#pragma unroll
        for (int k = 0; k < 8; ++k) activate<ACT, true>(v[k], a[k], slope[k]);
    } else if constexpr (ACT == NA_ACT_GELU) {
        // Phi(-|v|) = exp(-v^2 / 2) t Q(t) / 2, t = 1 / (1 + p |v| / sqrt 2): the form of Abramowitz and Stegun 7.1.26, with
        // p = 0.52 and a Q of degree 6 fitted to the relative error of erfc over [0, 14] (2^-19.6; with the roundings as above).
#pragma unroll
        for (int k = 0; k < 8; k += 2) {
            const uint64_t x = pack2(v[k], v[k + 1]);
            float q0, q1, z0, z1, phi0, phi1;
            split2(mul2(mul2(x, x), pack2(-0.5f * L, -0.5f * L)), q0, q1);   // log2 of exp(-v^2 / 2)
            split2(fma2(pack2(fminf(fabsf(v[k]), 100.f), fminf(fabsf(v[k + 1]), 100.f)), pack2(0.36769554f, 0.36769554f), one), z0, z1);
            const uint64_t t = pack2(inverse<true>(z0), inverse<true>(z1)), e = pack2(fast_exp2(q0), fast_exp2(q1));
            auto coefficient = [](float c) { return pack2(0.5f * c, 0.5f * c); };
            uint64_t q = fma2(t, coefficient(0.09600309f), coefficient(-0.3451418f));
            q = fma2(t, q, coefficient(0.3083583f));
            q = fma2(t, q, coefficient(0.08299062f));
            q = fma2(t, q, coefficient(0.273033f));
            q = fma2(t, q, coefficient(0.29128924f));
            q = fma2(t, q, coefficient(0.29346788f));
            split2(mul2(mul2(e, t), q), phi0, phi1);
            const uint64_t phi = pack2(v[k] < 0.f ? phi0 : 1.f - phi0, v[k + 1] < 0.f ? phi1 : 1.f - phi1);
            split2(mul2(x, phi), a[k], a[k + 1]);
            split2(fma2(mul2(x, e), pack2(0.39894228f, 0.39894228f), phi), slope[k], slope[k + 1]);
        }
    } else {
#pragma unroll
        for (int k = 0; k < 8; k += 2) {
            const uint64_t x = pack2(v[k], v[k + 1]);
            uint64_t q = 0, t;   // v^2; the exponent of exp(-..) of the sigmoid's argument
            if constexpr (ACT == NA_ACT_GELU_TANH) {
                float q0, q1;
                split2(mul2(x, x), q0, q1);
                q = pack2(fminf(q0, 10000.f), fminf(q1, 10000.f));   // beyond |v| = 100 the sigmoid is 0 or 1
                t = mul2(x, fma2(q, pack2(-L * K * 0.044715f, -L * K * 0.044715f), pack2(-L * K, -L * K)));
            } else {
                t = mul2(x, pack2(-L, -L));
            }
            float t0, t1, p0, p1;
            split2(t, t0, t1);
            const float e0 = fast_exp2(t0), e1 = fast_exp2(t1);
            split2(add2(pack2(e0, e1), one), p0, p1);
            const float y0 = inverse<true>(p0), y1 = inverse<true>(p1);
            const uint64_t y = pack2(y0, y1), rest = fma2(y, pack2(-1.f, -1.f), one);
            if constexpr (ACT == NA_ACT_SIGMOID) {
                a[k] = y0;
                a[k + 1] = y1;
                float r0, r1;   // 1 - y without cancellation on either side
                split2(rest, r0, r1);
                slope[k] = y0 * (v[k] > 0.f ? e0 * y0 : r0);
                slope[k + 1] = y1 * (v[k + 1] > 0.f ? e1 * y1 : r1);
            } else {
                const uint64_t s = mul2(x, y);
                split2(s, a[k], a[k + 1]);
                if constexpr (ACT == NA_ACT_GELU_TANH) {
                    const uint64_t rise = fma2(q, pack2(3.f * K * 0.044715f, 3.f * K * 0.044715f), pack2(K, K));
                    split2(fma2(mul2(s, rest), rise, y), slope[k], slope[k + 1]);
                } else {
                    split2(fma2(s, rest, y), slope[k], slope[k + 1]);
                }
            }
        }
    }
}

// Calls f<ACT>() for a run-time activation.
template <typename Call>
__device__ __forceinline__ void with_act(int act, Call&& call) {
    switch (act) {
        case NA_ACT_RELU: call(ActTag<NA_ACT_RELU>{}); break;
        case NA_ACT_GELU: call(ActTag<NA_ACT_GELU>{}); break;
        case NA_ACT_GELU_TANH: call(ActTag<NA_ACT_GELU_TANH>{}); break;
        case NA_ACT_SIGMOID: call(ActTag<NA_ACT_SIGMOID>{}); break;
        default: call(ActTag<NA_ACT_SILU>{}); break;
    }
}

// Up to three matrices of 2-byte elements, rows of D elements in one place and of W >= D, whole chunks, in the other.
struct GluCopies {
    const void* from[3];
    void* to[3];
    long long rows[3];   // 0: none
    int D, W;
};
// Launchers of the CUDA-core kernels, of the sums over runs (out0 the first `cut` of n elements, out1 the others; either may be
// null) (na_glu_fma.cuh).
template <typename T>
na_status launch_fma(const GluParams& p, Product which, const FmaTile& tile, cudaStream_t s);
template <typename T>
na_status launch_sum(const float* partial, int runs, long long n, long long cut, void* out0, void* out1, cudaStream_t s);

// Launchers of the tensor-core kernels (na_glu_tc.cuh).  blocks: of a tile, 2 (256 x 256) or 1 (128 x 128); tokens: 16, 64 or
// 128, the most that a product of few tokens holds.
template <int WHICH, typename T>
na_status launch_tiles(const GluTcParams& p, int blocks, cudaStream_t s);
template <int WHICH, typename T>
na_status launch_few(const GluTcParams& p, int tokens, cudaStream_t s);

}  // namespace glu
}  // namespace na
