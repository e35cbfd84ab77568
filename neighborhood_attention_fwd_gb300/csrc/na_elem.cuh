// na_elem.cuh -- element types of libna's CUDA-core kernels: 16-byte chunks widened to fp32 and back.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace na {

// 16-byte chunks: EPC elements widened to fp32 and back (round to nearest even).
template <typename T>
struct Elem;

template <>
struct Elem<float> {
    static constexpr int EPC = 4;
    __device__ static void unpack(const uint4& u, float (&f)[4]) {
        f[0] = __uint_as_float(u.x);
        f[1] = __uint_as_float(u.y);
        f[2] = __uint_as_float(u.z);
        f[3] = __uint_as_float(u.w);
    }
    __device__ static uint4 pack(const float (&f)[4]) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
    __device__ static float get(float v) { return v; }
    __device__ static float put(float v) { return v; }
};

template <>
struct Elem<__nv_bfloat16> {
    static constexpr int EPC = 8;
    // a bf16 is the upper half of the fp32 with the same bits
    __device__ static void two(uint32_t w, float& lo, float& hi) {
        lo = __uint_as_float(w << 16);
        hi = __uint_as_float(w & 0xffff0000u);
    }
    __device__ static void unpack(const uint4& u, float (&f)[8]) {
        two(u.x, f[0], f[1]);
        two(u.y, f[2], f[3]);
        two(u.z, f[4], f[5]);
        two(u.w, f[6], f[7]);
    }
    __device__ static uint32_t pair(float lo, float hi) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    __device__ static uint4 pack(const float (&f)[8]) {
        return make_uint4(pair(f[0], f[1]), pair(f[2], f[3]), pair(f[4], f[5]), pair(f[6], f[7]));
    }
    __device__ static float get(__nv_bfloat16 v) { return __bfloat162float(v); }
    __device__ static __nv_bfloat16 put(float v) { return __float2bfloat16_rn(v); }
};

template <>
struct Elem<__half> {
    static constexpr int EPC = 8;
    __device__ static void two(uint32_t w, float& lo, float& hi) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
        lo = f.x;
        hi = f.y;
    }
    __device__ static void unpack(const uint4& u, float (&f)[8]) {
        two(u.x, f[0], f[1]);
        two(u.y, f[2], f[3]);
        two(u.z, f[4], f[5]);
        two(u.w, f[6], f[7]);
    }
    __device__ static uint32_t pair(float lo, float hi) {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    __device__ static uint4 pack(const float (&f)[8]) {
        return make_uint4(pair(f[0], f[1]), pair(f[2], f[3]), pair(f[4], f[5]), pair(f[6], f[7]));
    }
    __device__ static float get(__half v) { return __half2float(v); }
    __device__ static __half put(float v) { return __float2half_rn(v); }
};

}  // namespace na
