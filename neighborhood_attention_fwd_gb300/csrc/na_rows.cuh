// na_rows.cuh -- what the kernels over rows of channels (na_norm.cu, na_addnorm.cu) share: chunks of a row, sums over
// the team of threads that holds a row, and fp32 arithmetic on pairs of columns.
#pragma once

#include <type_traits>

#include "na_block.cuh"
#include "na_device.cuh"

namespace na {
namespace rows {

using namespace dev;

// A chunk: V elements, 16 bytes, or one element where a row is not whole chunks.  Loads are unconditional (places past
// the end are clamped to the last one and left out afterwards): a guarded load would be waited for before the next one.
template <typename T, int V>
struct Chunk {
    uint4 raw;
    __device__ __forceinline__ void load(const void* base, long long at) { raw = ld_stream(static_cast<const T*>(base) + at); }
    __device__ __forceinline__ void get(float (&f)[V]) const { Elem<T>::unpack(raw, f); }
};
template <typename T>
struct Chunk<T, 1> {
    T raw;
    __device__ __forceinline__ void load(const void* base, long long at) { raw = static_cast<const T*>(base)[at]; }
    __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = Elem<T>::get(raw); }
};

template <typename T, int V>
__device__ __forceinline__ void store_chunk(void* base, long long at, const float (&f)[V]) {
    if constexpr (V == 1) static_cast<T*>(base)[at] = Elem<T>::put(f[0]);
    else st_stream(static_cast<T*>(base) + at, Elem<T>::pack(f));
}

template <int V>
__device__ __forceinline__ void load_weights(const float* w, int c, float (&f)[V], float none) {
    if (!w) {
#pragma unroll
        for (int e = 0; e < V; ++e) f[e] = none;
    } else if constexpr (V == 1) {
        f[0] = __ldg(w + c);
    } else {
#pragma unroll
        for (int e = 0; e < V; e += 4) {
            const float4 t = __ldg(reinterpret_cast<const float4*>(w + c + e));
            f[e] = t.x;
            f[e + 1] = t.y;
            f[e + 2] = t.z;
            f[e + 3] = t.w;
        }
    }
}

// Sums N values over the row's team: lanes of a warp, or the whole block through shared memory (slot: one of
// two buffers taken in turn, so that one barrier per sum is enough).
template <int N, bool BLOCK>
__device__ __forceinline__ void team_sum(float (&v)[N], int team, float (*slot)[32]) {
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1)
        if (BLOCK || m < team) {
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], m);
        }
    if (BLOCK) {
        const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
        if (lane == 0) {
#pragma unroll
            for (int i = 0; i < N; ++i) slot[i][threadIdx.x >> 5] = v[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float s = lane < warps ? slot[i][lane] : 0.f;
#pragma unroll
            for (int m = 16; m >= 1; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
            v[i] = s;
        }
    }
}

// Chunk-wise arithmetic, H words of one or two columns each.
template <int V>
struct Cols {
    static constexpr int H = V == 1 ? 1 : V / 2;
    using W = typename std::conditional<V == 1, float, uint64_t>::type;
    static __device__ __forceinline__ W both(float a) {
        if constexpr (V == 1) return a;
        else return pack2(a, a);
    }
    static __device__ __forceinline__ W fma(W a, W b, W c) {
        if constexpr (V == 1) return fmaf(a, b, c);
        else return fma2(a, b, c);
    }
    static __device__ __forceinline__ W mul(W a, W b) {
        if constexpr (V == 1) return a * b;
        else return mul2(a, b);
    }
    static __device__ __forceinline__ W add(W a, W b) {
        if constexpr (V == 1) return a + b;
        else return add2(a, b);
    }
    static __device__ __forceinline__ float sum(W a) {
        if constexpr (V == 1) {
            return a;
        } else {
            float x, y;
            split2(a, x, y);
            return x + y;
        }
    }
    static __device__ __forceinline__ void from(const float (&f)[V], W (&w)[H]) {
#pragma unroll
        for (int e = 0; e < H; ++e) {
            if constexpr (V == 1) w[e] = f[e];
            else w[e] = pack2(f[2 * e], f[2 * e + 1]);
        }
    }
    static __device__ __forceinline__ void to(const W (&w)[H], float (&f)[V]) {
#pragma unroll
        for (int e = 0; e < H; ++e) {
            if constexpr (V == 1) f[e] = w[e];
            else split2(w[e], f[2 * e], f[2 * e + 1]);
        }
    }
};

}  // namespace rows
}  // namespace na
