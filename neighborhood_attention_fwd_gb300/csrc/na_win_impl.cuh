// na_win_impl.cuh -- the window softmax in the forms that a transformer's training needs: with dropout on its
// weights, and as the difference of two softmax maps with learned weights, forward and backward.  Included by
// na_win_bf16.cu, na_win_f16.cu and na_win_f32.cu (one type's instances each).
//
//   s_m = softmax(x_m) over a row's K weights (a row of -inf alone has no weights: s_m = 0)
//   forward:  y = drop(s_1), or drop(s_1 - lam s_2);  drop(v) = gain v where the generator keeps the place, else 0
//   backward: g = drop(dy), r_m = sum s_m g, dx_1 = s_1 (g - r_1), dx_2 = -lam s_2 (g - r_2), dlam = -sum r_2
// The backward recomputes the maps from the logits and the mask from the generator: neither is stored.
//
// What bounds it.  Every tensor passes once: memory first, the issue slots next.  K is a product of odd sizes, so
// rows of 2-byte weights start at any even address.  Eight rows are a whole number of 16-byte chunks, so a tile is
// a multiple of eight rows: it moves as a whole between global and shared memory (cp.async.bulk), 1 to 32
// lanes work on each row in 4-byte words (two weights; the one word that a row shares with a neighbour is written by
// halves), and the result overwrites the logits in shared memory.  Persistent blocks keep a ring of tiles, so that the
// next tiles are on their way while one is worked on.  Dropout works on aligned octets of the tile, one
// generator block each, before (backward) or after (forward) the rows.  fp32 arithmetic runs on pairs (f32x2).
#pragma once

#include <cmath>
#include <type_traits>

#include "na_block.cuh"
#include "na_device.cuh"
#include "na_win.h"

namespace na {
using namespace dev;

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kMaxStages = 4;

// A row's words: 4 bytes, one or two weights.
template <typename T>
struct Words {
    static constexpr int N = 2;
    static constexpr uint32_t kNegInf = std::is_same<T, __half>::value ? 0xFC00FC00u : 0xFF80FF80u;
    static __device__ __forceinline__ void get(uint32_t w, float* f) { Elem<T>::two(w, f[0], f[1]); }
    static __device__ __forceinline__ uint32_t put(const float* f) { return Elem<T>::pair(f[0], f[1]); }
    using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
    // the larger of each half, numbers before NaN
    static __device__ __forceinline__ uint32_t max(uint32_t a, uint32_t b) {
        const T2 m = __hmax2(*reinterpret_cast<const T2*>(&a), *reinterpret_cast<const T2*>(&b));
        return *reinterpret_cast<const uint32_t*>(&m);
    }
    static __device__ __forceinline__ float top(uint32_t w) {
        float f[2];
        get(w, f);
        return fmaxf(f[0], f[1]);
    }
};
template <>
struct Words<float> {
    static constexpr int N = 1;
    static constexpr uint32_t kNegInf = 0xFF800000u;
    static __device__ __forceinline__ void get(uint32_t w, float* f) { f[0] = __uint_as_float(w); }
    static __device__ __forceinline__ uint32_t put(const float* f) { return __float_as_uint(f[0]); }
    static __device__ __forceinline__ uint32_t max(uint32_t a, uint32_t b) {
        return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
    }
    static __device__ __forceinline__ float top(uint32_t w) { return __uint_as_float(w); }
};

// Pairs of fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void split2(uint64_t v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// The place of a lane in its row.  Lane l holds words l, l + lanes, .., J of them; the row has (K + 1) / 2 words (K is
// odd) and fills all but the last of every lane's: only word 0 (`head`: its low half is the row before's) and the
// last words (`last` 0: past the row, 1: the low half alone, 2: whole) need care.
struct Place {
    uint32_t* s;     // the lane's first word of the first tensor's tile
    int lanes;
    bool head;
    int last;
};

template <typename T, int J>
__device__ __forceinline__ void row_load(uint32_t (&r)[J], const Place& a, uint32_t shift, uint32_t fill) {
    const uint32_t* s = a.s + shift;
#pragma unroll
    for (int j = 0; j < J - 1; ++j) r[j] = s[a.lanes * j];
    r[J - 1] = a.last ? s[a.lanes * (J - 1)] : fill;
    if (Words<T>::N == 2) {
        if (a.last == 1) r[J - 1] = (r[J - 1] & 0xffffu) | (fill & 0xffff0000u);
        if (a.head) r[0] = (r[0] & 0xffff0000u) | (fill & 0xffffu);
    }
}

template <typename T, int J>
__device__ __forceinline__ void row_store(const float (&v)[J * Words<T>::N], const Place& a, uint32_t shift) {
    constexpr int N = Words<T>::N;
    uint32_t* s = a.s + shift;
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const uint32_t u = Words<T>::put(v + j * N);
        uint32_t* to = s + a.lanes * j;
        if (N == 2 && j == 0 && a.head) {   // the low half is the row before's
            if (J > 1 || a.last == 2) reinterpret_cast<uint16_t*>(to)[1] = static_cast<uint16_t>(u >> 16);
        } else if (j < J - 1 || a.last == 2) {
            *to = u;
        } else if (N == 2 && a.last == 1) {
            reinterpret_cast<uint16_t*>(to)[0] = static_cast<uint16_t>(u);
        }
    }
}

__device__ __forceinline__ float lanes_max(float v, int lanes) {
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1)
        if (m < lanes) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, m));
    return v;
}

__device__ __forceinline__ float lanes_sum(float v, int lanes) {
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1)
        if (m < lanes) v += __shfl_xor_sync(0xffffffffu, v, m);
    return v;
}

// The reference point of a row's exponentials: its maximum, or 0 for a row of -inf alone.  A maximum near the
// type's limits (a mask of the lowest finite value) would overflow once multiplied by log2 e: `far` says that the
// row has to be shifted before, not after, that product.
__device__ __forceinline__ float row_top(float m, bool& far) {
    if (m == -INFINITY) m = 0.f;
    far = !(fabsf(m) < 1e37f);
    return m;
}

// v = exp(x - max) of a row, and its sum over the lanes (0 for an empty row).
template <typename T, int J>
__device__ __forceinline__ float row_exp(const uint32_t (&r)[J], float (&v)[J * Words<T>::N], int lanes) {
    constexpr int N = Words<T>::N, NV = J * N;
    uint32_t mw = r[0];
#pragma unroll
    for (int j = 1; j < J; ++j) mw = Words<T>::max(mw, r[j]);
    // a NaN in mw loses to any number, and is none where it is alone: its exponential is NaN all the same
    bool far;
    float m = row_top(lanes_max(fmaxf(Words<T>::top(mw), -INFINITY), lanes), far);
#pragma unroll
    for (int j = 0; j < J; ++j) Words<T>::get(r[j], v + j * N);
    if (far) {
#pragma unroll
        for (int i = 0; i < NV; ++i) v[i] -= m;
        m = 0.f;
    }
    const float ml2 = -m * kLog2e;
    const uint64_t c = pack2(kLog2e, kLog2e), d = pack2(ml2, ml2);
    uint64_t sum = 0;   // two zeros
#pragma unroll
    for (int i = 0; i + 1 < NV; i += 2) {
        float a, b;
        split2(fma2(pack2(v[i], v[i + 1]), c, d), a, b);
        v[i] = fast_exp2(a);
        v[i + 1] = fast_exp2(b);
        sum = add2(sum, pack2(v[i], v[i + 1]));
    }
    float a, b;
    split2(sum, a, b);
    a += b;
    if (NV % 2) {
        v[NV - 1] = fast_exp2(fmaf(v[NV - 1], kLog2e, ml2));
        a += v[NV - 1];
    }
    return lanes_sum(a, lanes);
}

// 1 / l of a row's sum: at least 1 (its largest term), 0 for an empty row, or NaN.
__device__ __forceinline__ float inverse_or_zero(float l) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(l));
    return l == 0.f ? 0.f : r;
}

// v = v a (+ u b), pairwise.
template <int NV>
__device__ __forceinline__ void row_scale(float (&v)[NV], float a) {
    const uint64_t aa = pack2(a, a);
#pragma unroll
    for (int i = 0; i + 1 < NV; i += 2) split2(mul2(pack2(v[i], v[i + 1]), aa), v[i], v[i + 1]);
    if (NV % 2) v[NV - 1] *= a;
}
template <int NV>
__device__ __forceinline__ void row_axpy(float (&v)[NV], const float (&u)[NV], float b) {
    const uint64_t bb = pack2(b, b);
#pragma unroll
    for (int i = 0; i + 1 < NV; i += 2) split2(fma2(pack2(u[i], u[i + 1]), bb, pack2(v[i], v[i + 1])), v[i], v[i + 1]);
    if (NV % 2) v[NV - 1] = fmaf(u[NV - 1], b, v[NV - 1]);
}

// sum v g over the lanes.
template <int NV>
__device__ __forceinline__ float row_dot(const float (&v)[NV], const float (&g)[NV], int lanes) {
    uint64_t t = 0;
#pragma unroll
    for (int i = 0; i + 1 < NV; i += 2) t = fma2(pack2(v[i], v[i + 1]), pack2(g[i], g[i + 1]), t);
    float a, b;
    split2(t, a, b);
    a += b;
    if (NV % 2) a = fmaf(v[NV - 1], g[NV - 1], a);
    return lanes_sum(a, lanes);
}

// v = v a (g - q), pairwise.
template <int NV>
__device__ __forceinline__ void row_grad(float (&v)[NV], const float (&g)[NV], float a, float q) {
    const uint64_t aa = pack2(a, a), qq = pack2(-q, -q);
#pragma unroll
    for (int i = 0; i + 1 < NV; i += 2)
        split2(mul2(mul2(pack2(v[i], v[i + 1]), aa), add2(pack2(g[i], g[i + 1]), qq)), v[i], v[i + 1]);
    if (NV % 2) v[NV - 1] = v[NV - 1] * a * (g[NV - 1] - q);
}

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

__device__ __forceinline__ void bulk_store(void* dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_u32(src)), "r"(bytes)
                 : "memory");
}

// Zeros the dropped places of a tile in shared memory: octet o of the tile is block block0 + o of the tensor.
template <typename T>
__device__ __forceinline__ void drop_tile(unsigned char* tile, uint32_t octets, unsigned long long block0, const RngState& rng,
                                          uint32_t steps) {
    for (uint32_t o = threadIdx.x; o < octets; o += kWinThreads) {
        if constexpr (sizeof(T) == 4) {
            uint4* at = reinterpret_cast<uint4*>(tile) + 2 * o;
            uint4 a = at[0], b = at[1];
            drop_octet(a, b, rng, block0 + o, steps);
            at[0] = a;
            at[1] = b;
        } else {
            uint4* at = reinterpret_cast<uint4*>(tile) + o;
            uint4 a = at[0];
            drop_octet(a, rng, block0 + o, steps);
            at[0] = a;
        }
    }
}

template <typename T, bool DIFF, bool BWD, int J>
__global__ void __launch_bounds__(kWinThreads) win_kernel(const __grid_constant__ WinParams p) {
    constexpr int N = Words<T>::N, NV = J * N, NB = (DIFF ? 2 : 1) + (BWD ? 1 : 0), NO = DIFF && BWD ? 2 : 1;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ uint64_t full[kMaxStages];
    const uint32_t buf = static_cast<uint32_t>(p.tile) * p.K * sizeof(T);   // a multiple of 16
    const uint32_t stage = NB * buf;
    const WaitGuard guard{p.err, p.wait_ns};
    // bytes of tile t
    auto tile_bytes = [&](long long t) {
        return static_cast<uint32_t>(min(static_cast<long long>(p.tile), p.rows - t * p.tile)) * p.K * static_cast<uint32_t>(sizeof(T));
    };
    auto load = [&](long long t, int s) {   // one thread
        const uint32_t bulk = tile_bytes(t) & ~15u;
        const long long off = t * static_cast<long long>(buf);
        unsigned char* to = smem + s * stage;
        mbar_arrive_expect_tx(&full[s], NB * bulk);
        if (bulk != 0) {
            bulk_load(to, static_cast<const char*>(p.x1) + off, bulk, &full[s]);
            if (DIFF) bulk_load(to + buf, static_cast<const char*>(p.x2) + off, bulk, &full[s]);
            if (BWD) bulk_load(to + (NB - 1) * buf, static_cast<const char*>(p.dy) + off, bulk, &full[s]);
        }
    };
    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) mbar_init(&full[s], 1);
        fence_barrier_init();
        long long t = blockIdx.x;
        for (int s = 0; s < p.stages - 1 && t < p.tiles; ++s, t += gridDim.x) load(t, s);
    }
    RngState rng{};
    const bool dropping = p.drop.state != nullptr;
    if (dropping) rng = rng_load(p.drop.state);
    const int l = threadIdx.x & (p.lanes - 1), rpp = kWinThreads >> p.log_lanes, r_first = threadIdx.x >> p.log_lanes;
    const int words = N == 2 ? (p.K + 1) / 2 : p.K;
    const int last_word = l + p.lanes * (J - 1);
    __syncthreads();
    int s = 0;
    uint32_t parity = 0;
    for (long long t = blockIdx.x; t < p.tiles; t += gridDim.x) {
        const long long row0 = t * p.tile;
        unsigned char* tile = smem + s * stage;
        const uint32_t bytes = tile_bytes(t), bulk = bytes & ~15u;
        const long long off = t * static_cast<long long>(buf);
        if (!mbar_wait(&full[s], parity, guard, kSiteWin)) break;
        // the tensor may end inside a chunk: its last elements one by one
        const uint32_t tail = (bytes - bulk) / static_cast<uint32_t>(sizeof(T));
        if (tail != 0) {
            if (threadIdx.x < tail) {
                auto copy = [&](int i, const void* src) {
                    reinterpret_cast<T*>(tile + i * buf + bulk)[threadIdx.x] =
                        reinterpret_cast<const T*>(static_cast<const char*>(src) + off + bulk)[threadIdx.x];
                };
                copy(0, p.x1);
                if (DIFF) copy(1, p.x2);
                if (BWD) copy(NB - 1, p.dy);
            }
            __syncthreads();
        }
        const unsigned long long block0 = static_cast<unsigned long long>(row0) * p.K / 8;   // row0 is a multiple of 8
        const uint32_t octets = (bytes / static_cast<uint32_t>(sizeof(T)) + 7) / 8;
        if (BWD && dropping) {
            drop_tile<T>(tile + (NB - 1) * buf, octets, block0, rng, p.drop.steps);
            __syncthreads();
        }
        uint32_t head0 = 0;
        if (DIFF && !p.lam_rows)
            head0 = p.rows32 ? static_cast<uint32_t>(row0) - fdiv(static_cast<uint32_t>(row0), p.fd_heads) * p.heads
                             : static_cast<uint32_t>(row0 % p.heads);
        const int nrows = static_cast<int>(min(static_cast<long long>(p.tile), p.rows - row0));
        for (int r = r_first; r - r_first < nrows; r += rpp) {   // rows past the end work on what the buffer holds, for nothing
            const uint32_t e0 = static_cast<uint32_t>(r) * p.K;
            Place a;
            a.s = reinterpret_cast<uint32_t*>(tile) + e0 / N + l;
            a.lanes = p.lanes;
            a.head = N == 2 && (e0 & 1u) && l == 0;
            a.last = last_word < words - 1 ? 2 : (last_word == words - 1 ? (N == 2 && !(e0 & 1u) ? 1 : 2) : 0);
            float lam = 0.f;
            if (DIFF && r < nrows) {
                if (p.lam_rows) {
                    lam = __ldg(p.lam + row0 + r);
                } else {
                    const uint32_t h = head0 + r;
                    lam = __ldg(p.lam + (h - fdiv(h, p.fd_heads) * p.heads));
                }
            }
            uint32_t w[J];
            float v[NV];
            row_load<T, J>(w, a, 0, Words<T>::kNegInf);
            if (!BWD) {
                row_scale(v, inverse_or_zero(row_exp<T, J>(w, v, p.lanes)) * p.drop.gain);
                if (DIFF) {
                    float u[NV];
                    row_load<T, J>(w, a, buf / 4, Words<T>::kNegInf);
                    const float b = inverse_or_zero(row_exp<T, J>(w, u, p.lanes)) * p.drop.gain;
                    row_axpy(v, u, -(b * lam));
                }
                row_store<T, J>(v, a, 0);
            } else {
                float g[NV];
                {
                    uint32_t gw[J];
                    row_load<T, J>(gw, a, (NB - 1) * (buf / 4), 0u);
#pragma unroll
                    for (int j = 0; j < J; ++j) Words<T>::get(gw[j], g + j * N);
                }
#pragma unroll
                for (int m = 0; m < NO; ++m) {
                    if (m == 1) row_load<T, J>(w, a, buf / 4, Words<T>::kNegInf);
                    const float inv = inverse_or_zero(row_exp<T, J>(w, v, p.lanes));
                    const float k = inv * p.drop.gain * (m == 1 ? -lam : 1.f);
                    float q = row_dot(v, g, p.lanes) * inv;
                    if (fabsf(q) < INFINITY) {
                        row_grad(v, g, k, q);
                    }
                    // a place of weight zero (a masked one) takes no part, whatever dy holds there: where the sum is not
                    // finite it is taken again without those places.  Whole warps decide together, for the shuffles.
                    if (__any_sync(0xffffffffu, !(fabsf(q) < INFINITY))) {
                        const bool again = !(fabsf(q) < INFINITY);
                        float sum = 0.f;
#pragma unroll
                        for (int i = 0; i < NV; ++i) sum += v[i] == 0.f ? 0.f : v[i] * g[i];
                        sum = lanes_sum(sum, p.lanes);
                        if (again) {
                            q = sum * inv;
#pragma unroll
                            for (int i = 0; i < NV; ++i) v[i] = v[i] == 0.f ? 0.f : v[i] * k * (g[i] - q);
                        }
                    }
                    row_store<T, J>(v, a, m == 0 ? 0 : buf / 4);
                    if (m == 1 && r < nrows && l == 0) p.dlam[row0 + r] = -p.drop.gain * q;
                }
            }
        }
        if (!BWD && dropping) {
            __syncthreads();
            drop_tile<T>(tile, octets, block0, rng, p.drop.steps);
        }
        fence_proxy_async_smem();
        __syncthreads();
        char* out[2] = {static_cast<char*>(p.out1) + off, static_cast<char*>(NO == 2 ? p.out2 : p.out1) + off};
        if (threadIdx.x < tail) {
#pragma unroll
            for (int i = 0; i < NO; ++i)
                reinterpret_cast<T*>(out[i] + bulk)[threadIdx.x] = reinterpret_cast<const T*>(tile + i * buf + bulk)[threadIdx.x];
        }
        if (threadIdx.x == 0) {
            if (bulk != 0) {
#pragma unroll
                for (int i = 0; i < NO; ++i) bulk_store(out[i], tile + i * buf, bulk);
            }
            tma_store_commit();
            // the tile before this one has left its buffer: the tile stages - 1 on from here takes it
            asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
            const long long next = t + static_cast<long long>(gridDim.x) * (p.stages - 1);
            if (next < p.tiles) load(next, s == 0 ? p.stages - 1 : s - 1);
        }
        if (++s == p.stages) {
            s = 0;
            parity ^= 1u;
        }
    }
    if (threadIdx.x == 0) tma_store_wait_read();
}

// Rows that no tile holds (longer than 32 lanes of kMaxWords words): a block per row, read again for
// each pass (a row is a few tens of KB at most for any sensible window, and stays in L1 or L2).
template <int N>
__device__ __forceinline__ void block_reduce(float (&v)[N], bool maximum, float (*slot)[8]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        v[i] = maximum ? lanes_max(v[i], 32) : lanes_sum(v[i], 32);
        if (lane == 0) slot[i][warp] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float t = lane < kWinThreads / 32 ? slot[i][lane] : (maximum ? -INFINITY : 0.f);
        v[i] = maximum ? lanes_max(t, 32) : lanes_sum(t, 32);
    }
    __syncthreads();
}

template <typename T, bool DIFF, bool BWD>
__global__ void __launch_bounds__(kWinThreads) win_long_kernel(const __grid_constant__ WinParams p) {
    constexpr int M = DIFF ? 2 : 1;
    __shared__ float slot[2][8];
    const long long row = blockIdx.x;
    const long long first = row * p.K;
    const T* x[2] = {static_cast<const T*>(p.x1) + first, static_cast<const T*>(DIFF ? p.x2 : p.x1) + first};
    const T* dy = static_cast<const T*>(p.dy) + (BWD ? first : 0);
    T* out[2] = {static_cast<T*>(p.out1) + first, static_cast<T*>(DIFF && BWD ? p.out2 : p.out1) + first};
    float lam = 0.f;
    if (DIFF) lam = __ldg(p.lam + (p.lam_rows ? row : row % p.heads));
    RngState rng{};
    const bool dropping = p.drop.state != nullptr;
    if (dropping) rng = rng_load(p.drop.state);
    float m[M], l[M], ml2[M];
    bool far[M];
#pragma unroll
    for (int i = 0; i < M; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
    }
    for (int t = threadIdx.x; t < p.K; t += kWinThreads)
#pragma unroll
        for (int i = 0; i < M; ++i) m[i] = fmaxf(m[i], Elem<T>::get(x[i][t]));
    block_reduce<M>(m, true, slot);
#pragma unroll
    for (int i = 0; i < M; ++i) {
        m[i] = row_top(m[i], far[i]);
        ml2[i] = far[i] ? 0.f : m[i] * kLog2e;
    }
    auto weight = [&](int i, int t) {
        const float v = Elem<T>::get(x[i][t]);
        return fast_exp2(fmaf(far[i] ? v - m[i] : v, kLog2e, -ml2[i]));
    };
    for (int t = threadIdx.x; t < p.K; t += kWinThreads)
#pragma unroll
        for (int i = 0; i < M; ++i) l[i] += weight(i, t);
    block_reduce<M>(l, false, slot);
#pragma unroll
    for (int i = 0; i < M; ++i) l[i] = inverse_or_zero(l[i]);
    // octets of the tensor that hold this row's weights; an octet shared with a neighbour is taken in part
    const long long o0 = first >> 3, o1 = (first + p.K + 7) >> 3;
    float q[M];
    if (BWD) {
#pragma unroll
        for (int i = 0; i < M; ++i) q[i] = 0.f;
        for (long long o = o0 + threadIdx.x; o < o1; o += kWinThreads) {
            const uint4 keep = dropping ? keep_masks(rng, static_cast<unsigned long long>(o), p.drop.steps) : uint4{};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const long long t = o * 8 + e - first;
                if (t < 0 || t >= p.K || (dropping && !keep_of(keep, e))) continue;
                const float g = Elem<T>::get(dy[t]);
#pragma unroll
                for (int i = 0; i < M; ++i) {
                    const float w = weight(i, static_cast<int>(t));
                    q[i] += w == 0.f ? 0.f : w * g;
                }
            }
        }
        block_reduce<M>(q, false, slot);
#pragma unroll
        for (int i = 0; i < M; ++i) q[i] *= l[i];
        if (DIFF && threadIdx.x == 0) p.dlam[row] = -p.drop.gain * q[M - 1];
    }
    for (long long o = o0 + threadIdx.x; o < o1; o += kWinThreads) {
        const uint4 keep = dropping ? keep_masks(rng, static_cast<unsigned long long>(o), p.drop.steps) : uint4{};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const long long t = o * 8 + e - first;
            if (t < 0 || t >= p.K) continue;
            const bool kept = !dropping || keep_of(keep, e);
            float w[M];
#pragma unroll
            for (int i = 0; i < M; ++i) w[i] = weight(i, static_cast<int>(t));
            if (BWD) {
                const float g = kept ? Elem<T>::get(dy[t]) : 0.f;
#pragma unroll
                for (int i = 0; i < M; ++i)
                    out[i][t] = Elem<T>::put(w[i] == 0.f ? 0.f : w[i] * (l[i] * p.drop.gain * (i == 1 ? -lam : 1.f)) * (g - q[i]));
            } else {
                float y = w[0] * (l[0] * p.drop.gain);
                if (DIFF) y -= w[M - 1] * (l[M - 1] * p.drop.gain * lam);
                out[0][t] = Elem<T>::put(kept ? y : 0.f);
            }
        }
    }
}

// ---------------------------------------------------------------------------------------------
// Launch
// ---------------------------------------------------------------------------------------------

constexpr int kMaxWords = 12;             // words per lane, at most
constexpr uint32_t kWinSmem = 200 * 1024; // shared memory of a multiprocessor that the blocks' rings share

// Lanes per row and words per lane: the least work, a lane's words and what a row costs each of its lanes besides.
inline bool plan_row(int words, int& lanes, int& log_lanes, int& per_lane) {
    int best = 0;
    for (int g = 1, lg = 0; g <= 32; g *= 2, ++lg) {
        const int j = (words + g - 1) / g;
        if (j > kMaxWords) continue;
        const int cost = g * (12 * j + 8 * lg + 30);
        if (best == 0 || cost < best) {
            best = cost;
            lanes = g;
            log_lanes = lg;
            per_lane = j;
        }
    }
    return best != 0;
}

template <typename T, bool DIFF, bool BWD, int J>
na_status run_win(WinParams& p, cudaStream_t s) {
    if constexpr (J > kMaxWords) {
        return NA_ERR_UNSUPPORTED;
    } else {
        constexpr uint32_t NB = (DIFF ? 2 : 1) + (BWD ? 1 : 0);
        // a tile is whole passes of the threads, about 8 KB per tensor; fewer passes where the grid is small
        const int rpp = kWinThreads / p.lanes, row = p.K * static_cast<int>(sizeof(T));
        int passes = 8192 / (rpp * row);
        passes = passes < 1 ? 1 : passes;
        while (passes > 1 && p.rows / (static_cast<long long>(rpp) * passes) < 4 * kSms) --passes;
        p.tile = rpp * passes;
        p.tiles = (p.rows + p.tile - 1) / p.tile;
        const uint32_t stage = NB * static_cast<uint32_t>(p.tile) * row;
        p.stages = 3;
        const size_t smem = static_cast<size_t>(p.stages) * stage;
        const auto kernel = win_kernel<T, DIFF, BWD, J>;
        if (smem > 48 * 1024 &&
            cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) != cudaSuccess)
            return NA_ERR_CUDA;
        int per_sm = static_cast<int>(kWinSmem / smem);
        per_sm = per_sm < 1 ? 1 : (per_sm > 4 ? 4 : per_sm);
        const long long most = static_cast<long long>(per_sm) * kSms;
        kernel<<<static_cast<unsigned>(p.tiles < most ? p.tiles : most), kWinThreads, smem, s>>>(p);
        return launch_result();
    }
}

template <typename T, bool DIFF, bool BWD>
na_status launch_win_rows(WinParams& p, cudaStream_t s) {
    int words = 0;
    if (!plan_row(sizeof(T) == 4 ? p.K : (p.K + 1) / 2, p.lanes, p.log_lanes, words)) {
        if (p.rows > 0x7fffffffLL) return NA_ERR_UNSUPPORTED;
        win_long_kernel<T, DIFF, BWD><<<static_cast<unsigned>(p.rows), kWinThreads, 0, s>>>(p);
        return launch_result();
    }
    switch (words) {
        case 1: return run_win<T, DIFF, BWD, 1>(p, s);
        case 2: return run_win<T, DIFF, BWD, 2>(p, s);
        case 3: return run_win<T, DIFF, BWD, 3>(p, s);
        case 4: return run_win<T, DIFF, BWD, 4>(p, s);
        case 5: return run_win<T, DIFF, BWD, 5>(p, s);
        case 6: return run_win<T, DIFF, BWD, 6>(p, s);
        case 7: return run_win<T, DIFF, BWD, 7>(p, s);
        case 8: return run_win<T, DIFF, BWD, 8>(p, s);
        case 9: return run_win<T, DIFF, BWD, 9>(p, s);
        case 10: return run_win<T, DIFF, BWD, 10>(p, s);
        case 11: return run_win<T, DIFF, BWD, 11>(p, s);
        default: return run_win<T, DIFF, BWD, kMaxWords>(p, s);
    }
}

template <typename T>
na_status launch_win_type(WinParams& p, bool diff, bool bwd, cudaStream_t s) {
    if (diff) return bwd ? launch_win_rows<T, true, true>(p, s) : launch_win_rows<T, true, false>(p, s);
    return bwd ? launch_win_rows<T, false, true>(p, s) : launch_win_rows<T, false, false>(p, s);
}

}  // namespace
}  // namespace na
