// na_block.cuh -- what the operators around the attention (na_rope.cu, na_norm.cu, na_winsoft.cu) share:
// argument checks on the host, cache-streaming 16-byte accesses and the dropout generator.
#pragma once

#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "../../include/na.h"
#include "na_elem.cuh"
#include "na_internal.h"

namespace na {

// Device status word of the current device, the time limit of one bounded wait, and the test hook that withholds a copy
// (na_api.cu).
na_status device_status_word(unsigned** out);
unsigned long long wait_limit_ns();
uint32_t wait_withhold();

// ---------------------------------------------------------------------------------------------
// Host: argument checks
// ---------------------------------------------------------------------------------------------

struct Span {
    const void* p;
    long long bytes;
};

inline bool spans_overlap(const Span& a, const Span& b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return a.p && b.p && x < y + static_cast<uintptr_t>(b.bytes) && y < x + static_cast<uintptr_t>(a.bytes);
}

// An output may be one of the tensors in `same` (the very same memory) and overlaps nothing else.
inline bool output_clear(const Span& out, std::initializer_list<Span> same, std::initializer_list<Span> apart) {
    for (const Span& s : same)
        if (spans_overlap(out, s) && (out.p != s.p || out.bytes != s.bytes)) return false;
    for (const Span& s : apart)
        if (spans_overlap(out, s)) return false;
    return true;
}

inline bool ptr_aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

inline bool known_dtype(na_dtype dt) { return dt == NA_BF16 || dt == NA_FP16 || dt == NA_FP32; }
inline int elem_bytes(na_dtype dt) { return dt == NA_FP32 ? 4 : 2; }

// Tokens (B times the grid) of a [B, L_1 .., heads, width] tensor, with the size limits of the attention
// entry points (2^31 grid positions, 2^40 elements); L receives the grid as 3 axes, outermost first.
inline na_status grid_tokens(int B, int ndim, const int* spatial, int heads, long long width, int (&L)[3], long long& tokens) {
    if (ndim < 1 || ndim > 3 || !spatial || B < 1 || heads < 1 || width < 1) return NA_ERR_INVALID_ARG;
    for (int a = 0; a < ndim; ++a)
        if (spatial[a] < 1) return NA_ERR_INVALID_ARG;
    for (int a = 0; a < 3; ++a) L[a] = 1;
    long long n = 1;
    for (int a = 0; a < ndim; ++a) {
        L[3 - ndim + a] = spatial[a];
        n *= spatial[a];
        if (n > (1LL << 31)) return NA_ERR_UNSUPPORTED;
    }
    tokens = n * B;
    if (tokens > (1LL << 40) / heads || tokens * heads > (1LL << 40) / width) return NA_ERR_UNSUPPORTED;
    return NA_OK;
}

constexpr int kSms = 152;   // multiprocessors of a GB300: grids are sized for them

inline na_status launch_result() { return cudaGetLastError() == cudaSuccess ? NA_OK : NA_ERR_CUDA; }

// ---------------------------------------------------------------------------------------------
// Device: 16-byte accesses.  The operators read and write every byte once, so they leave L1 alone.
// Not the read-only path: an output may be the input's tensor.
// ---------------------------------------------------------------------------------------------

__device__ __forceinline__ uint4 ld_stream(const void* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

__device__ __forceinline__ void st_stream(void* p, const uint4& v) {
    asm volatile("st.global.L1::no_allocate.v4.u32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                 : "memory");
}

// ---------------------------------------------------------------------------------------------
// Dropout: which elements are kept is a function of (seed, offset, element index) alone, so no mask is
// stored: the backward pass computes it again.  Generator: Philox4x32 (Salmon, Moraes, Dror and Shaw,
// "Parallel random numbers: as easy as 1, 2, 3", 2011) with seven rounds, the fewest that the paper
// reports as passing all of BigCrush; it costs 0.7 of the default ten.  One block of 128 bits serves
// eight elements of 16 bits each: block i / 8 of element i sits at counter (i / 8, offset) under key
// seed, and field i % 8 is compared with the number of steps kept.  Sixteen bits make the keep
// probability a multiple of 2^-16; the gain is the inverse of that multiple, so the mean is exact.
// ---------------------------------------------------------------------------------------------

struct Dropout {
    const unsigned long long* state;  // device: {seed, offset}; null: nothing is dropped
    uint32_t steps;                   // fields below it are kept, 0 .. 65535 with a state
    float gain;                       // 65536 / steps (0 when steps is 0)
};

// false for a probability outside [0, 1] or a missing generator state.
inline bool make_dropout(double p, const void* state, Dropout& d) {
    if (!(p >= 0.0 && p <= 1.0)) return false;
    d.steps = static_cast<uint32_t>(std::floor((1.0 - p) * 65536.0 + 0.5));
    d.gain = d.steps ? static_cast<float>(65536.0 / d.steps) : 0.f;
    d.state = d.steps == 65536u ? nullptr : static_cast<const unsigned long long*>(state);
    return d.steps == 65536u || state != nullptr;
}

struct RngState {
    uint32_t k0, k1, o0, o1;
};

__device__ __forceinline__ RngState rng_load(const unsigned long long* s) {
    const unsigned long long seed = s[0], off = s[1];
    return RngState{static_cast<uint32_t>(seed), static_cast<uint32_t>(seed >> 32), static_cast<uint32_t>(off),
                    static_cast<uint32_t>(off >> 32)};
}

// The 128 random bits of a block.
__device__ __forceinline__ uint4 rng_block(const RngState& s, unsigned long long block) {
    uint32_t c0 = static_cast<uint32_t>(block), c1 = static_cast<uint32_t>(block >> 32), c2 = s.o0, c3 = s.o1;
    uint32_t k0 = s.k0, k1 = s.k1;
#pragma unroll
    for (int r = 0; r < 7; ++r) {
        const unsigned long long a = static_cast<unsigned long long>(c0) * 0xD2511F53u;
        const unsigned long long b = static_cast<unsigned long long>(c2) * 0xCD9E8D57u;
        c0 = static_cast<uint32_t>(b >> 32) ^ c1 ^ k0;
        c1 = static_cast<uint32_t>(b);
        c2 = static_cast<uint32_t>(a >> 32) ^ c3 ^ k1;
        c3 = static_cast<uint32_t>(a);
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return make_uint4(c0, c1, c2, c3);
}

// The same bits for the blocks below 2^32, whose upper counter word is zero: then all of the first round's second product and
// the second round's first one are the same for every block.  A plan holds them folded into the constants that the
// rounds xor in (12 products and 13 xors a block instead of 14 and 14 with 12 additions for the keys).
struct RngPlan {
    uint32_t c[4];               // o1 ^ k1[0], low(o0 M1) ^ k0[1], high(P M0) ^ k1[1], low(P M0) ^ k1[2]; P = high(o0 M1) ^ k0[0]
    uint32_t k0[5], k1[4];       // k0[2..6], k1[3..6]
    uint32_t pad[3];
};

__device__ __forceinline__ RngPlan rng_plan(const RngState& s) {
    RngPlan p;
    const unsigned long long b = static_cast<unsigned long long>(s.o0) * 0xCD9E8D57u;
    const unsigned long long a = static_cast<unsigned long long>(static_cast<uint32_t>(b >> 32) ^ s.k0) * 0xD2511F53u;
    auto k0 = [&](uint32_t r) { return s.k0 + r * 0x9E3779B9u; };
    auto k1 = [&](uint32_t r) { return s.k1 + r * 0xBB67AE85u; };
    p.c[0] = s.o1 ^ k1(0);
    p.c[1] = static_cast<uint32_t>(b) ^ k0(1);
    p.c[2] = static_cast<uint32_t>(a >> 32) ^ k1(1);
    p.c[3] = static_cast<uint32_t>(a) ^ k1(2);
#pragma unroll
    for (uint32_t r = 0; r < 5; ++r) p.k0[r] = k0(2 + r);
#pragma unroll
    for (uint32_t r = 0; r < 4; ++r) p.k1[r] = k1(3 + r);
    p.pad[0] = p.pad[1] = p.pad[2] = 0;
    return p;
}

__device__ __forceinline__ uint4 rng_block(const RngPlan& p, uint32_t block) {
    auto mul = [](uint32_t x, uint32_t m) { return static_cast<unsigned long long>(x) * m; };
    unsigned long long a = mul(block, 0xD2511F53u);
    unsigned long long b = mul(static_cast<uint32_t>(a >> 32) ^ p.c[0], 0xCD9E8D57u);
    const uint32_t x2 = static_cast<uint32_t>(a) ^ p.c[2], x1 = static_cast<uint32_t>(b);
    a = mul(static_cast<uint32_t>(b >> 32) ^ p.c[1], 0xD2511F53u);
    b = mul(x2, 0xCD9E8D57u);
    uint32_t c0 = static_cast<uint32_t>(b >> 32) ^ x1 ^ p.k0[0], c1 = static_cast<uint32_t>(b);
    uint32_t c2 = static_cast<uint32_t>(a >> 32) ^ p.c[3], c3 = static_cast<uint32_t>(a);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        a = mul(c0, 0xD2511F53u);
        b = mul(c2, 0xCD9E8D57u);
        c0 = static_cast<uint32_t>(b >> 32) ^ c1 ^ p.k0[1 + r];
        c1 = static_cast<uint32_t>(b);
        c2 = static_cast<uint32_t>(a >> 32) ^ c3 ^ p.k1[r];
        c3 = static_cast<uint32_t>(a);
    }
    return make_uint4(c0, c1, c2, c3);
}

// Whole words below steps << 16 are those whose high field is below steps (steps < 65536).
__device__ __forceinline__ bool keep_high(uint32_t w, uint32_t steps) { return w < (steps << 16); }
__device__ __forceinline__ bool keep_low(uint32_t w, uint32_t steps) { return (w << 16) < (steps << 16); }

// Whether masks of eight 16-bit elements (all bits of a kept one) keep element i.
__device__ __forceinline__ bool keep_of(const uint4& m, int i) {
    const uint32_t w = i < 2 ? m.x : (i < 4 ? m.y : (i < 6 ? m.z : m.w));
    return ((w >> (16 * (i & 1))) & 1u) != 0u;
}

// Zeros the dropped elements of an octet, given its block's bits: eight 16-bit elements, or eight 32-bit ones in
// two chunks.
__device__ __forceinline__ void drop_words(uint4& d, const uint4& bits, uint32_t steps) {
    auto drop = [steps](uint32_t& v, uint32_t r) {
        if (!keep_high(r, steps)) v &= 0x0000ffffu;
        if (!keep_low(r, steps)) v &= 0xffff0000u;
    };
    drop(d.x, bits.x);
    drop(d.y, bits.y);
    drop(d.z, bits.z);
    drop(d.w, bits.w);
}
__device__ __forceinline__ void drop_words(uint4& a, uint4& b, const uint4& bits, uint32_t steps) {
    auto drop = [steps](uint32_t& lo, uint32_t& hi, uint32_t r) {
        if (!keep_low(r, steps)) lo = 0u;
        if (!keep_high(r, steps)) hi = 0u;
    };
    drop(a.x, a.y, bits.x);
    drop(a.z, a.w, bits.y);
    drop(b.x, b.y, bits.z);
    drop(b.z, b.w, bits.w);
}

// Masks of an octet's eight elements, 16 bits each, all ones where the element is kept.
__device__ __forceinline__ uint4 keep_masks(const RngState& s, unsigned long long block, uint32_t steps) {
    uint4 m = make_uint4(~0u, ~0u, ~0u, ~0u);
    drop_words(m, rng_block(s, block), steps);
    return m;
}

}  // namespace na
