// na_glu_fma.cuh -- the gated feed-forward product on CUDA cores, and the sums that follow the products (see na_glu.cu).
//
// What bounds it: products.  fp32 runs on FMA units, in pairs (fma.rn.f32x2), no TF32: tiles of 128 x 128, 8 x 8 per
// thread, operands widened and laid out [k][row] in shared memory, two stages of 16 steps of k.
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

// A thread's N elements of a piece: from row r, steps k .. k + N - 1, or with ALONG_ROWS from step k, rows r .. r + N - 1.
template <typename T, bool ALONG_ROWS, int N>
__device__ __forceinline__ void fetch(const Operand<T>& o, long long r, long long k, float (&f)[N]) {
    constexpr int EPC = Elem<T>::EPC;
    const bool in = r < o.rows && k < o.depth;
    const long long left = ALONG_ROWS ? o.rows - r : o.depth - k;   // elements there along memory
    const T* at = o.base + (ALONG_ROWS ? k * o.ld + r : r * o.ld + k);
    if constexpr (N == 8) {
        if (in && o.wide && left >= 8) {
#pragma unroll
            for (int c = 0; c < 8 / EPC; ++c) {
                const uint4 raw = __ldg(reinterpret_cast<const uint4*>(at) + c);
                float g[EPC];
                Elem<T>::unpack(raw, g);
#pragma unroll
                for (int e = 0; e < EPC; ++e) f[c * EPC + e] = g[e];
            }
            return;
        }
    }
#pragma unroll
    for (int e = 0; e < N; ++e) f[e] = in && e < left ? Elem<T>::get(at[e]) : 0.f;
}

template <bool ALONG_ROWS, int TS, int N>
__device__ __forceinline__ void place(float (*sm)[TS + 4], int t, const float (&f)[N]) {
    if constexpr (!ALONG_ROWS) {
#pragma unroll
        for (int e = 0; e < N; ++e) sm[t / TS * N + e][t % TS] = f[e];
    } else {
        float* to = &sm[t >> 4][(t & 15) * N];
        if constexpr (N == 8) {
            *reinterpret_cast<float4*>(to) = make_float4(f[0], f[1], f[2], f[3]);
            *reinterpret_cast<float4*>(to + 4) = make_float4(f[4], f[5], f[6], f[7]);
        } else {
#pragma unroll
            for (int e = 0; e < N; ++e) to[e] = f[e];
        }
    }
}

// Products on CUDA cores.  A block makes TR x TC elements (kForward, kSlopes: TR rows x TC / 2 columns of g and the same of u);
// rows along blockIdx.x, columns along blockIdx.y; along blockIdx.z the splits of the summed axis, kWeights: of dWg and dWu each.
// A thread's elements are two runs of GR rows by two of GC columns, half a tile apart, so that g and u of an element are its own.
template <typename T, int WHICH, int TR, int TC>
__global__ void __launch_bounds__(kGluThreads, TR + TC == 256 ? 2 : 4) glu_fma_kernel(const GluParams p) {
    constexpr bool PAIR = WHICH == kForward || WHICH == kSlopes;
    constexpr bool A_ROWS = WHICH == kWeights, B_ROWS = !PAIR;
    constexpr int GR = TR / 32, GC = TC / 32, R = 2 * GR, NA = TR / 16, NB = TC / 16;
    __shared__ __align__(16) float sa[2][kDepth][TR + 4], sb[2][kDepth][TC + 4];
    const int t = threadIdx.x, tx = t & 15, ty = t >> 4;
    const long long m0 = static_cast<long long>(blockIdx.x) * TR, n0 = static_cast<long long>(blockIdx.y) * (PAIR ? TC / 2 : TC);
    const int half = WHICH == kWeights ? blockIdx.z & 1 : 0, split = WHICH == kWeights ? blockIdx.z >> 1 : blockIdx.z;
    const T *x = static_cast<const T*>(p.x), *wg = static_cast<const T*>(p.wg), *wu = static_cast<const T*>(p.wu);
    const T *dg = static_cast<const T*>(p.dg), *du = static_cast<const T*>(p.du);
    const bool wide = p.D % Elem<T>::EPC == 0;
    // pieces of 16 steps of k: of kWeights a run of tokens; kTokens has two runs of columns of them, dg Wg and du Wu, cut together
    const long long k0 = WHICH == kWeights ? split * p.run : 0;
    const long long depth = PAIR ? p.D : (WHICH == kTokens ? p.F : min(p.run, p.T - k0));
    const long long pieces = (depth + kDepth - 1) / kDepth;
    const long long first = WHICH == kTokens ? split * p.run : 0, last = WHICH == kTokens ? min(2 * pieces, first + p.run) : pieces;
    // where this thread fetches within a piece
    const int ra = A_ROWS ? (t & 15) * NA : t % TR, ka = A_ROWS ? t >> 4 : t / TR * NA;
    const int rb = B_ROWS ? (t & 15) * NB : t % TC, kb = B_ROWS ? t >> 4 : t / TC * NB;
    float fa[NA], fb[NB];
    auto load = [&](long long i) {
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
    uint64_t acc[R][GC];   // pairs of columns
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < GC; ++j) acc[i][j] = 0;
    load(first);
    for (long long i = first; i < last; ++i) {
        const int st = static_cast<int>(i & 1);
        place<A_ROWS, TR>(sa[st], t, fa);
        place<B_ROWS, TC>(sb[st], t, fb);
        __syncthreads();   // also: the stage filled next was last read before this barrier
        if (i + 1 < last) load(i + 1);
#pragma unroll
        for (int k = 0; k < kDepth; ++k) {
            float a[R];
            uint64_t b[GC];
            if constexpr (GR == 4) {
                const float4 a0 = *reinterpret_cast<const float4*>(&sa[st][k][ty * 4]), a1 = *reinterpret_cast<const float4*>(&sa[st][k][64 + ty * 4]);
                a[0] = a0.x, a[1] = a0.y, a[2] = a0.z, a[3] = a0.w, a[4] = a1.x, a[5] = a1.y, a[6] = a1.z, a[7] = a1.w;
            } else {
                a[0] = sa[st][k][ty], a[1] = sa[st][k][16 + ty];
            }
            if constexpr (GC == 4) {
                const ulonglong2 b0 = *reinterpret_cast<const ulonglong2*>(&sb[st][k][tx * 4]), b1 = *reinterpret_cast<const ulonglong2*>(&sb[st][k][64 + tx * 4]);
                b[0] = b0.x, b[1] = b0.y, b[2] = b1.x, b[3] = b1.y;
            } else {
                b[0] = pack2(sb[st][k][tx], sb[st][k][16 + tx]);
            }
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const uint64_t aa = pack2(a[r], a[r]);
#pragma unroll
                for (int c = 0; c < GC; ++c) acc[r][c] = fma2(aa, b[c], acc[r][c]);
            }
        }
    }
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
                        static_cast<T*>(p.dg)[row * p.pitch + f] = Elem<T>::put(dh * u * slope);
                        static_cast<T*>(p.du)[row * p.pitch + f] = Elem<T>::put(dh * a);
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
}

// out[i] = sums over the runs of partial[run][n], in order: the first `cut` elements to out0, the others to out1; either may
// be null.  V elements at a time (n and cut are multiples of V).
template <typename T, int V>
__global__ void __launch_bounds__(256) glu_sum_kernel(const float* partial, int runs, long long n, long long cut, T* out0, T* out1) {
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

// Column sums of dg and du over runs of tokens: partial[run][2][F].  A lane takes a chunk of 16 bytes of every eighth row (rows
// are padded to whole chunks).
template <typename T>
__global__ void __launch_bounds__(256) glu_column_kernel(const T* dg, const T* du, long long T_, int F, long long pitch, long long run, float* partial) {
    constexpr int V = Elem<T>::EPC;
    __shared__ float sums[8][32 * V];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int first_col = blockIdx.x * 32 * V, c = first_col + lane * V;
    const T* from = blockIdx.z ? du : dg;
    const long long first = blockIdx.y * run, end = min(first + run, T_);
    float s[V] = {};
    if (c < pitch)
#pragma unroll 4
        for (long long r = first + warp; r < end; r += 8) {
            float f[V];
            Elem<T>::unpack(ld_stream(from + r * pitch + c), f);
#pragma unroll
            for (int e = 0; e < V; ++e) s[e] += f[e];
        }
#pragma unroll
    for (int e = 0; e < V; ++e) sums[warp][lane * V + e] = s[e];
    __syncthreads();
    for (int i = threadIdx.x; i < 32 * V && first_col + i < F; i += 256) {
        float t = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) t += sums[w][i];
        partial[(blockIdx.y * 2LL + blockIdx.z) * F + first_col + i] = t;
    }
}

template <typename T, int TR, int TC>
na_status launch_fma(const GluParams& p, Product which, cudaStream_t s) {
    const unsigned splits = p.splits;
    switch (which) {
        case kForward: glu_fma_kernel<T, kForward, TR, TC><<<dim3(up(p.T, TR), up(p.F, TC / 2)), kGluThreads, 0, s>>>(p); break;
        case kSlopes: glu_fma_kernel<T, kSlopes, TR, TC><<<dim3(up(p.T, TR), up(p.F, TC / 2)), kGluThreads, 0, s>>>(p); break;
        case kTokens: glu_fma_kernel<T, kTokens, TR, TC><<<dim3(up(p.T, TR), up(p.D, TC), splits), kGluThreads, 0, s>>>(p); break;
        default: glu_fma_kernel<T, kWeights, TR, TC><<<dim3(up(p.F, TR), up(p.D, TC), 2 * splits), kGluThreads, 0, s>>>(p); break;
    }
    return launch_result();
}

template <typename T>
na_status launch_fma(const GluParams& p, Product which, const FmaTile& tile, cudaStream_t s) {
    if (tile.rows == 128) return tile.cols == 128 ? launch_fma<T, 128, 128>(p, which, s) : launch_fma<T, 128, 32>(p, which, s);
    return tile.cols == 128 ? launch_fma<T, 32, 128>(p, which, s) : launch_fma<T, 32, 32>(p, which, s);
}

template <typename T>
na_status launch_sum(const float* partial, int runs, long long n, long long cut, void* out0, void* out1, cudaStream_t s) {
    const bool wide = n % 4 == 0 && cut % 4 == 0;
    const unsigned blocks = static_cast<unsigned>(std::min((n / (wide ? 4 : 1) + 255) / 256, 8LL * kSms));
    if (wide) glu_sum_kernel<T, 4><<<blocks, 256, 0, s>>>(partial, runs, n, cut, static_cast<T*>(out0), static_cast<T*>(out1));
    else glu_sum_kernel<T, 1><<<blocks, 256, 0, s>>>(partial, runs, n, cut, static_cast<T*>(out0), static_cast<T*>(out1));
    return launch_result();
}

template <typename T>
na_status launch_columns(const GluParams& p, int runs, long long run, float* partial, cudaStream_t s) {
    glu_column_kernel<T><<<dim3(up(p.F, 32 * Elem<T>::EPC), runs, 2), 256, 0, s>>>(static_cast<const T*>(p.dg), static_cast<const T*>(p.du), p.T, p.F,
                                                                         p.pitch, run, partial);
    return launch_result();
}

}  // namespace glu
}  // namespace na
