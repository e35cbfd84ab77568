// na_glu_fma.cuh -- the gated feed-forward product on CUDA cores, and the sums that follow the products (see na_glu.cu).
//
// What bounds it: products.  fp32 runs on FMA units, in pairs (fma.rn.f32x2), no TF32; operands are widened and laid out
// [k][row] in shared memory, two stages of 16 steps of k.  Tiles of 128 x 128, 8 x 8 per thread, run at 45 TFLOP/s (20000 x 512
// x 1376, forward: 1.24 ms); 32 in place of 128 on either side where a problem has few tiles or short sides.  Those are bound
// by the latency of a step's loads, so that they keep two or four pieces on their way in registers (32 x 512 x 512: 32 -> 14 us).
#pragma once

#include <algorithm>

#include "na_block.cuh"
#include "na_device.cuh"
#include "na_glu.h"

namespace na {
namespace glu {

using namespace dev;

constexpr int kDepth = 16, kGluThreads = 256;

// One operand of a product: rows (of the result's rows or columns) by k.  Element (r, k) is at base[r * ld + k], or with
// ALONG_ROWS at base[k * ld + r].
template <typename T>
struct Operand {
    const T* base;
    long long ld;
    long long rows, depth;   // zeros past them
    bool wide;               // rows of memory start at 16 bytes
};

// A thread's N elements of a piece: from row r, steps k .. k + N - 1, or with ALONG_ROWS from step k, rows r .. r + N - 1.  They are
// widened when they are placed: until then nothing waits for them.
template <typename T, bool ALONG_ROWS, int N>
__device__ __forceinline__ void fetch(const Operand<T>& o, long long r, long long k, T (&f)[N]) {
    const bool in = r < o.rows && k < o.depth;
    const long long left = ALONG_ROWS ? o.rows - r : o.depth - k;   // elements there along memory
    const T* at = o.base + (ALONG_ROWS ? k * o.ld + r : r * o.ld + k);
    constexpr int RUN = N * sizeof(T) < 16 ? N : 16 / sizeof(T);   // elements of one load
    if (in && o.wide && left >= N) {
        struct alignas(RUN * sizeof(T)) Run { T v[RUN]; };
#pragma unroll
        for (int c = 0; c < N / RUN; ++c) {
            Run run;
            if constexpr (sizeof run == 16) *reinterpret_cast<uint4*>(&run) = __ldg(reinterpret_cast<const uint4*>(at) + c);
            else run = reinterpret_cast<const Run*>(at)[c];
#pragma unroll
            for (int e = 0; e < RUN; ++e) f[c * RUN + e] = run.v[e];
        }
        return;
    }
#pragma unroll
    for (int e = 0; e < N; ++e) f[e] = in && e < left ? at[e] : Elem<T>::put(0.f);
}

// Where thread t fetches in a piece of TS rows by kDepth steps: N = TS / 16 elements along memory.  128 rows: eight steps are a
// sector of a row of theirs; 32: eight threads take the 16 steps of a row.
template <bool ALONG_ROWS, int TS>
__device__ __forceinline__ int row_of(int t) { return ALONG_ROWS ? (t & 15) * (TS / 16) : (TS == 128 ? t % TS : t >> 3); }
template <bool ALONG_ROWS, int TS>
__device__ __forceinline__ int step_of(int t) { return ALONG_ROWS ? t >> 4 : (TS == 128 ? t / TS * 8 : (t & 7) * 2); }

// A piece in shared memory: [step][row], of 32 rows those 16 apart, a thread's two, side by side.
template <bool ALONG_ROWS, int TS, int N, typename T>
__device__ __forceinline__ void place(float (*sm)[TS + 4], int t, const T (&raw)[N]) {
    float f[N];
#pragma unroll
    for (int e = 0; e < N; ++e) f[e] = Elem<T>::get(raw[e]);
    const int r = row_of<ALONG_ROWS, TS>(t), k = step_of<ALONG_ROWS, TS>(t);
    if constexpr (TS == 32) {
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const int row = ALONG_ROWS ? r + e : r;
            sm[ALONG_ROWS ? k : k + e][(row & 15) * 2 + (row >> 4)] = f[e];
        }
    } else if constexpr (!ALONG_ROWS) {
#pragma unroll
        for (int e = 0; e < N; ++e) sm[k + e][r] = f[e];
    } else {
        float* to = &sm[k][r];
        *reinterpret_cast<float4*>(to) = make_float4(f[0], f[1], f[2], f[3]);
        *reinterpret_cast<float4*>(to + 4) = make_float4(f[4], f[5], f[6], f[7]);
    }
}

// Products on CUDA cores.  A block makes TR x TC elements (kForward, kSlopes: TR rows x TC / 2 columns of g and the same of u);
// rows along blockIdx.x, columns along blockIdx.y; along blockIdx.z the splits of the summed axis, kWeights: of dWg and dWu each
// (fma_grid).  LONG (kForward, kSlopes): sums over more than kMostProducts channels, which are added up in runs of that many.
// A thread's elements are two runs of GR rows by two of GC columns, half a tile apart, so that g and u of an element are its own.
template <typename T, int WHICH, int TR, int TC, bool LONG>
__global__ void __launch_bounds__(kGluThreads, TR + TC == 256 ? 2 : 4) glu_fma_kernel(const GluParams p) {
    constexpr bool PAIR = WHICH == kForward || WHICH == kSlopes;
    constexpr bool A_ROWS = WHICH == kWeights, B_ROWS = !PAIR;
    constexpr int GR = TR / 32, GC = TC / 32, R = 2 * GR, NA = TR / 16, NB = TC / 16;
    __shared__ __align__(16) float sa[2][kDepth][TR + 4], sb[2][kDepth][TC + 4];
    const int t = threadIdx.x, tx = t & 15, ty = t >> 4;
    int half = 0, split = blockIdx.z, row_tile = blockIdx.x;
    if constexpr (WHICH == kWeights) {
        const int tiles = (p.F + TR - 1) / TR, turn = row_tile / tiles;
        half = blockIdx.z & 1;
        split = turn * static_cast<int>(gridDim.z >> 1) + static_cast<int>(blockIdx.z >> 1);
        row_tile -= turn * tiles;
        if (split >= p.splits) return;
    }
    const long long m0 = static_cast<long long>(row_tile) * TR, n0 = static_cast<long long>(blockIdx.y) * (PAIR ? TC / 2 : TC);
    const T *x = static_cast<const T*>(p.x), *wg = static_cast<const T*>(p.wg), *wu = static_cast<const T*>(p.wu);
    const T *dg = static_cast<const T*>(p.dg), *du = static_cast<const T*>(p.du);
    const bool wide = p.D % Elem<T>::EPC == 0;
    // pieces of 16 steps of k: of kWeights a run of tokens; kTokens has two runs of columns of them, dg Wg and du Wu, cut together
    const long long k0 = WHICH == kWeights ? split * p.run : 0;
    const long long depth = PAIR ? p.D : (WHICH == kTokens ? p.F : min(p.run, p.T - k0));
    const long long pieces = (depth + kDepth - 1) / kDepth;
    const long long first = WHICH == kTokens ? split * p.run : 0, last = WHICH == kTokens ? min(2 * pieces, first + p.run) : pieces;
    // where this thread fetches within a piece
    const int ra = row_of<A_ROWS, TR>(t), ka = step_of<A_ROWS, TR>(t), rb = row_of<B_ROWS, TC>(t), kb = step_of<B_ROWS, TC>(t);
    // pieces on their way in registers; small tiles take less time than a load, and have the registers for more of them
    constexpr int AHEAD = TR + TC == 256 ? 1 : (TR + TC == 64 ? 4 : 2);
    T pa[AHEAD][NA], pb[AHEAD][NB];
    auto load = [&](long long i, T (&fa)[NA], T (&fb)[NB]) {
        const bool second = WHICH == kTokens && i >= pieces;
        const long long k = (second ? i - pieces : i) * kDepth;
        Operand<T> a, b;
        if (PAIR) {
            a = {x, p.D, p.T, p.D, wide};
            b = {rb < TC / 2 ? wg : wu, p.D, p.F, p.D, wide};
            fetch<T, false>(a, m0 + ra, k + ka, fa);
            fetch<T, false>(b, n0 + (rb & (TC / 2 - 1)), k + kb, fb);
        } else if (WHICH == kTokens) {
            a = {second ? du : dg, p.pitch, p.T, p.F, true};
            b = {second ? wu : wg, p.D, p.D, p.F, wide};
            fetch<T, false>(a, m0 + ra, k + ka, fa);
            fetch<T, true>(b, n0 + rb, k + kb, fb);
        } else {
            a = {half ? du : dg, p.pitch, p.F, k0 + depth, true};
            b = {x, p.D, p.D, k0 + depth, wide};
            fetch<T, true>(a, m0 + ra, k0 + k + ka, fa);
            fetch<T, true>(b, n0 + rb, k0 + k + kb, fb);
        }
    };
    uint64_t acc[R][GC], total[LONG ? R : 1][LONG ? GC : 1];   // pairs of columns
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < GC; ++j) {
            acc[i][j] = 0;
            if constexpr (LONG) total[i][j] = 0;
        }
    auto add_up = [&]() {
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int j = 0; j < GC; ++j) {
                total[i][j] = add2(total[i][j], acc[i][j]);
                acc[i][j] = 0;
            }
    };
#pragma unroll
    for (int q = 0; q < AHEAD; ++q)
        if (first + q < last) load(first + q, pa[q], pb[q]);
    int st = 0;
    auto piece = [&](long long i, T (&fa)[NA], T (&fb)[NB]) {
        place<A_ROWS, TR>(sa[st], t, fa);
        place<B_ROWS, TC>(sb[st], t, fb);
        __syncthreads();   // also: the stage filled next was last read before this barrier
        if (i + AHEAD < last) load(i + AHEAD, fa, fb);
#pragma unroll
        for (int k = 0; k < kDepth; ++k) {
            float a[R];
            uint64_t b[GC];
            if constexpr (GR == 4) {
                const float4 a0 = *reinterpret_cast<const float4*>(&sa[st][k][ty * 4]), a1 = *reinterpret_cast<const float4*>(&sa[st][k][64 + ty * 4]);
                a[0] = a0.x, a[1] = a0.y, a[2] = a0.z, a[3] = a0.w, a[4] = a1.x, a[5] = a1.y, a[6] = a1.z, a[7] = a1.w;
            } else {
                const float2 a0 = *reinterpret_cast<const float2*>(&sa[st][k][ty * 2]);
                a[0] = a0.x, a[1] = a0.y;
            }
            if constexpr (GC == 4) {
                const ulonglong2 b0 = *reinterpret_cast<const ulonglong2*>(&sb[st][k][tx * 4]), b1 = *reinterpret_cast<const ulonglong2*>(&sb[st][k][64 + tx * 4]);
                b[0] = b0.x, b[1] = b0.y, b[2] = b1.x, b[3] = b1.y;
            } else {
                b[0] = *reinterpret_cast<const uint64_t*>(&sb[st][k][tx * 2]);
            }
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const uint64_t aa = pack2(a[r], a[r]);
#pragma unroll
                for (int c = 0; c < GC; ++c) acc[r][c] = fma2(aa, b[c], acc[r][c]);
            }
        }
        st ^= 1;
    };
    static_assert(kMostProducts % (kDepth * AHEAD) == 0, "a run ends between turns of the loop");
    for (long long i = first; i < last; i += AHEAD) {
#pragma unroll
        for (int q = 0; q < AHEAD; ++q)
            if (i + q < last) piece(i + q, pa[q], pb[q]);
        if constexpr (LONG)
            if ((i + AHEAD) % (kMostProducts / kDepth) == 0) add_up();
    }
    if constexpr (LONG) {
        add_up();
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int c = 0; c < GC; ++c) acc[r][c] = total[r][c];
    }
    float sum_g[WHICH == kSlopes ? GC : 1] = {}, sum_u[WHICH == kSlopes ? GC : 1] = {};   // of dg and du over this thread's rows
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const long long row = m0 + (r < GR ? ty * GR + r : TR / 2 + ty * GR + r - GR);
        float v[2 * GC];   // the first run of columns, then the second
#pragma unroll
        for (int c = 0; c < GC; ++c) split2(acc[r][c], v[2 * c], v[2 * c + 1]);
        if constexpr (PAIR) {
            if (row >= p.T) continue;
            with_act(p.act, [&](auto tag) {
                constexpr int ACT = decltype(tag)::value;
#pragma unroll
                for (int c = 0; c < GC; ++c) {
                    const long long f = n0 + tx * GC + c;
                    if (f >= p.F) break;
                    const float g = v[c] + (p.bg ? Elem<T>::get(static_cast<const T*>(p.bg)[f]) : 0.f);
                    const float u = v[GC + c] + (p.bu ? Elem<T>::get(static_cast<const T*>(p.bu)[f]) : 0.f);
                    float a, slope;
                    activate<ACT, false>(g, a, slope);
                    if constexpr (WHICH == kForward) {
                        static_cast<T*>(p.h)[row * p.F + f] = Elem<T>::put(a * u);
                    } else {
                        const float dh = Elem<T>::get(static_cast<const T*>(p.dh)[row * p.F + f]);
                        const float dg = dh * u * slope, du = dh * a;
                        static_cast<T*>(p.dg)[row * p.pitch + f] = Elem<T>::put(dg);
                        static_cast<T*>(p.du)[row * p.pitch + f] = Elem<T>::put(du);
                        sum_g[c] += dg;
                        sum_u[c] += du;
                    }
                }
            });
        } else {
            const long long rows = WHICH == kTokens ? p.T : p.F;
            if (row >= rows) continue;
            float* sums = p.partial + (WHICH == kTokens ? static_cast<long long>(split) : 2LL * split + half) * rows * p.D;
            T* out = static_cast<T*>(WHICH == kTokens ? p.dx : half ? p.dwu : p.dwg);
#pragma unroll
            for (int c = 0; c < 2 * GC; ++c) {
                const long long col = n0 + (c < GC ? tx * GC + c : TC / 2 + tx * GC + c - GC);
                if (col >= p.D) continue;
                const long long at = row * p.D + col;
                if (p.splits > 1) sums[at] = v[c];
                else out[at] = Elem<T>::put(v[c]);
            }
        }
    }
    if constexpr (WHICH == kSlopes) {
        if (!p.sums) return;
        // over the block's rows: the two of a warp, then the warps through shared memory
        float (*part)[2][TC / 2] = reinterpret_cast<float (*)[2][TC / 2]>(&sa[0][0][0]);
        static_assert(sizeof(float) * 8 * TC <= sizeof(sa), "the warps' sums take the rows' operand's place");
        __syncthreads();   // which has been read
#pragma unroll
        for (int c = 0; c < GC; ++c) {
            sum_g[c] += __shfl_xor_sync(0xffffffffu, sum_g[c], 16);
            sum_u[c] += __shfl_xor_sync(0xffffffffu, sum_u[c], 16);
            if ((t & 16) == 0) {
                part[t >> 5][0][tx * GC + c] = sum_g[c];
                part[t >> 5][1][tx * GC + c] = sum_u[c];
            }
        }
        __syncthreads();
        const int which = t / (TC / 2), col = t % (TC / 2);
        if (which < 2 && n0 + col < p.F) {
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < kGluThreads / 32; ++w) s += part[w][which][col];
            p.sums[(static_cast<long long>(row_tile) * 2 + which) * p.sum_pitch + n0 + col] = s;
        }
    }
}

// out[i] = sums over the runs of partial[run][n], in order: the first `cut` elements to out0, the others to out1; either may
// be null.  V elements at a time (n and cut are multiples of V).
template <typename T, int V>
__global__ void __launch_bounds__(256) glu_sum_kernel(const float* partial, int runs, long long n, long long cut, T* out0, T* out1) {
    after_previous();
    next_may_start();
    for (long long i = (blockIdx.x * 256LL + threadIdx.x) * V; i < n; i += gridDim.x * 256LL * V) {
        T* out = i < cut ? (out0 ? out0 + i : nullptr) : (out1 ? out1 + (i - cut) : nullptr);
        if (!out) continue;
        float s[V] = {};
#pragma unroll 4
        for (int r = 0; r < runs; ++r) {
            if constexpr (V == 4) {
                const float4 t = *reinterpret_cast<const float4*>(partial + r * n + i);
                s[0] += t.x, s[1] += t.y, s[2] += t.z, s[3] += t.w;
            } else {
                s[0] += partial[r * n + i];
            }
        }
        if constexpr (V == 4 && sizeof(T) == 2) *reinterpret_cast<uint2*>(out) = make_uint2(Elem<T>::pair(s[0], s[1]), Elem<T>::pair(s[2], s[3]));
        else
#pragma unroll
            for (int e = 0; e < V; ++e) out[e] = Elem<T>::put(s[e]);
    }
}

// The same of many runs of few elements: a block takes 32 elements, a warp every eighth run (102 runs of 1376: 39 -> 5 us).
template <typename T>
__global__ void __launch_bounds__(256) glu_sum_runs_kernel(const float* partial, int runs, long long n, long long cut, T* out0, T* out1) {
    after_previous();
    next_may_start();
    __shared__ float sums[8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long i = blockIdx.x * 32LL + lane;
    float s = 0.f;
    if (i < n)
#pragma unroll 8
        for (int r = warp; r < runs; r += 8) s += partial[r * n + i];
    sums[warp][lane] = s;
    __syncthreads();
    T* out = i < cut ? out0 : out1;
    if (warp > 0 || i >= n || !out) return;
    float t = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) t += sums[w][lane];
    out[i < cut ? i : i - cut] = Elem<T>::put(t);
}

template <typename T, int TR, int TC>
na_status launch_fma(const GluParams& p, Product which, dim3 grid, cudaStream_t s) {
    if constexpr (TR == TC)   // as plan_fma
        if (p.D > kMostProducts && (which == kForward || which == kSlopes)) {
            if (which == kForward) glu_fma_kernel<T, kForward, TR, TC, true><<<grid, kGluThreads, 0, s>>>(p);
            else glu_fma_kernel<T, kSlopes, TR, TC, true><<<grid, kGluThreads, 0, s>>>(p);
            return launch_result();
        }
    switch (which) {
        case kForward: glu_fma_kernel<T, kForward, TR, TC, false><<<grid, kGluThreads, 0, s>>>(p); break;
        case kSlopes: glu_fma_kernel<T, kSlopes, TR, TC, false><<<grid, kGluThreads, 0, s>>>(p); break;
        case kTokens: glu_fma_kernel<T, kTokens, TR, TC, false><<<grid, kGluThreads, 0, s>>>(p); break;
        default: glu_fma_kernel<T, kWeights, TR, TC, false><<<grid, kGluThreads, 0, s>>>(p); break;
    }
    return launch_result();
}

template <typename T>
na_status launch_fma(const GluParams& p, Product which, const FmaTile& tile, cudaStream_t s) {
    const FmaGrid n = fma_grid(which, p.T, p.D, p.F, tile);
    const dim3 grid(n.x, n.y, n.z);
    if (tile.rows == 128) return tile.cols == 128 ? launch_fma<T, 128, 128>(p, which, grid, s) : launch_fma<T, 128, 32>(p, which, grid, s);
    return tile.cols == 128 ? launch_fma<T, 32, 128>(p, which, grid, s) : launch_fma<T, 32, 32>(p, which, grid, s);
}

template <typename T>
na_status launch_sum(const float* partial, int runs, long long n, long long cut, void* out0, void* out1, cudaStream_t s) {
    const bool wide = n % 4 == 0 && cut % 4 == 0;
    const unsigned blocks = static_cast<unsigned>(std::min((n / (wide ? 4 : 1) + 255) / 256, 8LL * kSms));
    if (blocks < kSms / 2 && runs >= 8)
        return launch_after(glu_sum_runs_kernel<T>, dim3(static_cast<unsigned>((n + 31) / 32)), 256, s, partial, runs, n, cut, static_cast<T*>(out0), static_cast<T*>(out1));
    return launch_after(wide ? glu_sum_kernel<T, 4> : glu_sum_kernel<T, 1>, dim3(blocks), 256, s, partial, runs, n, cut, static_cast<T*>(out0), static_cast<T*>(out1));
}

}  // namespace glu
}  // namespace na
