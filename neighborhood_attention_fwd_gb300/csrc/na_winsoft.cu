// na_winsoft.cu -- the window softmax in the forms that a transformer's training needs: with dropout on its
// weights, and as the difference of two softmax maps with learned weights, forward and backward; and
// dropout of a whole tensor.
//
//   s_m = softmax(x_m) over a row's K weights (a row of -inf alone has no weights: s_m = 0)
//   forward:  y = drop(s_1), or drop(s_1 - lam s_2);  drop(v) = gain v where the generator keeps the place, else 0
//   backward: g = drop(dy), r_m = sum s_m g, dx_1 = s_1 (g - r_1), dx_2 = -lam s_2 (g - r_2), dlam = -sum r_2
// The backward recomputes the maps from the logits and the mask from the generator: neither is stored.
//
// What bounds it.  Every tensor passes once: memory, then (with dropout) the issue slots that the generator takes.
// K is odd, so a row of 2-byte weights starts at any even address.  Eight rows are a whole number of 16-byte
// chunks, so a block takes a multiple of eight rows, copies them whole into shared memory (cp.async.bulk), lets 1
// to 32 lanes work on each row in 4-byte words (two weights, a row's first and last word shared with its
// neighbours), writes the result over the logits in shared memory and copies it out whole.  Dropout works on
// aligned octets of the block's rows, one generator block each, before (backward) or after (forward) the rows.
#include <cmath>
#include <type_traits>

#include "na_block.cuh"
#include "na_device.cuh"

namespace na {
using namespace dev;

namespace {

constexpr int kWinThreads = 256;
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kMaxWords = 12;   // words of one row per lane, at most

struct WinParams {
    const void* x1;
    const void* x2;
    const void* dy;
    const float* lam;      // [heads], or [rows] with lam_rows
    void* out1;            // y; dx1
    void* out2;            // dx2
    float* dlam;           // backward: -r_2 of every row
    long long rows;
    int K, heads;
    int lanes;             // lanes per row (power of two)
    int tile;              // rows per block (a multiple of 8)
    uint32_t lam_rows, rows32;
    FastDiv fd_heads;
    Dropout drop;
    unsigned* err;
    unsigned long long wait_ns;
};

template <typename T>
struct Words {   // 4-byte words of a row: one or two weights
    static constexpr int N = 2;
    static __device__ __forceinline__ void get(uint32_t w, float* f) { Elem<T>::two(w, f[0], f[1]); }
    static __device__ __forceinline__ uint32_t put(const float* f) { return Elem<T>::pair(f[0], f[1]); }
};
template <>
struct Words<float> {
    static constexpr int N = 1;
    static __device__ __forceinline__ void get(uint32_t w, float* f) { f[0] = __uint_as_float(w); }
    static __device__ __forceinline__ uint32_t put(const float* f) { return __float_as_uint(f[0]); }
};

// A row in the lanes' registers: lane l holds words l, l + lanes, ..; `odd`: the first word's low half belongs
// to the row before; `end`: K + odd, the end in weights from the first word's start (0: no row).
template <typename T, int J>
__device__ __forceinline__ void row_load(float (&v)[J * Words<T>::N], const uint32_t* s, int l, int lanes, int odd, int end,
                                         float fill) {
    constexpr int N = Words<T>::N;
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const int w = l + lanes * j;
        float* f = v + j * N;
        if (w * N < end) {
            Words<T>::get(s[w], f);
            if (N == 2 && w * 2 + 1 >= end) f[N - 1] = fill;
        } else {
#pragma unroll
            for (int e = 0; e < N; ++e) f[e] = fill;
        }
    }
    if (N == 2 && odd && l == 0) v[0] = fill;
}

template <typename T, int J>
__device__ __forceinline__ void row_store(const float (&v)[J * Words<T>::N], uint32_t* s, int l, int lanes, int odd, int end) {
    constexpr int N = Words<T>::N;
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const int w = l + lanes * j;
        if (w * N < end) {
            const uint32_t u = Words<T>::put(v + j * N);
            const bool lo = !(N == 2 && j == 0 && odd && l == 0), hi = N == 1 || w * 2 + 1 < end;
            if (lo && hi) {
                s[w] = u;
            } else {   // the other half is a neighbour's
                uint16_t* h = reinterpret_cast<uint16_t*>(s + w);
                if (lo) h[0] = static_cast<uint16_t>(u);
                if (hi) h[1] = static_cast<uint16_t>(u >> 16);
            }
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

// exp(v - max) of a row in place, and its sum over the lanes (0 for an empty row).
template <int NV>
__device__ __forceinline__ float row_exp(float (&v)[NV], int lanes) {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < NV; ++i) m = fmaxf(m, v[i]);
    bool far;
    m = row_top(lanes_max(m, lanes), far);
    if (far) {
#pragma unroll
        for (int i = 0; i < NV; ++i) v[i] -= m;
        m = 0.f;
    }
    const float ml2 = m * kLog2e;
    float l = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        v[i] = fast_exp2(fmaf(v[i], kLog2e, -ml2));
        l += v[i];
    }
    return lanes_sum(l, lanes);
}

__device__ __forceinline__ float inverse_or_zero(float l) { return l == 0.f ? 0.f : 1.f / l; }

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

__device__ __forceinline__ void bulk_store(void* dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_u32(src)), "r"(bytes)
                 : "memory");
}

// Applies the generator's masks to octets of a tile in shared memory; o: octet of the tile, block: of the tensor.
template <typename T>
__device__ __forceinline__ uint4 mask_octet(uint4* tile, uint32_t o, const RngState& rng, unsigned long long block,
                                            uint32_t steps, uint4& second) {
    const uint4 m = keep_masks(rng, block, steps);
    if constexpr (sizeof(T) == 4) {
        uint4 a, b;
        widen_masks(m, a, b);
        second = and4(tile[2 * o + 1], b);
        return and4(tile[2 * o], a);
    } else {
        return and4(tile[o], m);
    }
}

__device__ __forceinline__ uint32_t head_of(const WinParams& p, uint32_t base, uint32_t r) {
    const uint32_t x = base + r;
    return x - fdiv(x, p.fd_heads) * static_cast<uint32_t>(p.heads);
}

template <typename T, bool DIFF, bool BWD, int J>
__global__ void __launch_bounds__(kWinThreads) win_kernel(const __grid_constant__ WinParams p) {
    constexpr int N = Words<T>::N, NV = J * N, NB = (DIFF ? 2 : 1) + (BWD ? 1 : 0);
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ uint64_t bar;
    const long long row0 = static_cast<long long>(blockIdx.x) * p.tile;
    const int nrows = static_cast<int>(min(static_cast<long long>(p.tile), p.rows - row0));
    const uint32_t buf = static_cast<uint32_t>(p.tile) * p.K * sizeof(T);   // a multiple of 16
    const uint32_t bytes = static_cast<uint32_t>(nrows) * p.K * sizeof(T), bulk = bytes & ~15u;
    const long long off = row0 * p.K * static_cast<long long>(sizeof(T));   // of the tile, in bytes
    const void* src[3] = {p.x1, DIFF ? p.x2 : p.dy, p.dy};
    if (threadIdx.x == 0) {
        mbar_init(&bar, 1);
        fence_barrier_init();
        mbar_arrive_expect_tx(&bar, NB * bulk);
        if (bulk != 0) {
#pragma unroll
            for (int i = 0; i < NB; ++i) bulk_load(smem + i * buf, static_cast<const char*>(src[i]) + off, bulk, &bar);
        }
    }
    // the last tile may end inside a chunk: its last elements one by one
    const uint32_t tail = (bytes - bulk) / static_cast<uint32_t>(sizeof(T));
    if (threadIdx.x < tail) {
#pragma unroll
        for (int i = 0; i < NB; ++i)
            reinterpret_cast<T*>(smem + i * buf + bulk)[threadIdx.x] =
                reinterpret_cast<const T*>(static_cast<const char*>(src[i]) + off + bulk)[threadIdx.x];
    }
    RngState rng{};
    const bool dropping = p.drop.state != nullptr;
    if (dropping) rng = rng_load(p.drop.state);
    const unsigned long long block0 = static_cast<unsigned long long>(row0) * p.K / 8;   // row0 is a multiple of 8
    const uint32_t octets = (static_cast<uint32_t>(nrows) * p.K + 7) / 8;
    uint32_t head0 = 0;
    if (DIFF && !p.lam_rows) {
        head0 = p.rows32 ? static_cast<uint32_t>(row0) - fdiv(static_cast<uint32_t>(row0), p.fd_heads) * p.heads
                         : static_cast<uint32_t>(row0 % p.heads);
    }
    __syncthreads();
    const WaitGuard guard{p.err, p.wait_ns};
    if (!__syncthreads_and(mbar_wait(&bar, 0, guard, kSiteWin))) {
        mbar_drain(&bar, 0, p.wait_ns);
        return;
    }
    unsigned char* sdy = smem + (NB - 1) * buf;
    if (BWD && dropping) {
        for (uint32_t o = threadIdx.x; o < octets; o += kWinThreads) {
            uint4 second, first = mask_octet<T>(reinterpret_cast<uint4*>(sdy), o, rng, block0 + o, p.drop.steps, second);
            if constexpr (sizeof(T) == 4) {
                reinterpret_cast<uint4*>(sdy)[2 * o] = first;
                reinterpret_cast<uint4*>(sdy)[2 * o + 1] = second;
            } else {
                reinterpret_cast<uint4*>(sdy)[o] = first;
            }
        }
        __syncthreads();
    }
    const int l = threadIdx.x & (p.lanes - 1), rpp = kWinThreads / p.lanes;
    for (int rb = 0; rb < nrows; rb += rpp) {   // whole warps stay together: rows past the end are empty
        const int r = rb + threadIdx.x / p.lanes;
        const bool live = r < nrows;
        const int e0 = r * p.K, odd = N == 2 ? e0 & 1 : 0, end = live ? p.K + odd : 0;
        const uint32_t w0 = static_cast<uint32_t>(e0) / N;
        uint32_t* s1 = reinterpret_cast<uint32_t*>(smem) + w0;
        uint32_t* s2 = reinterpret_cast<uint32_t*>(smem + buf) + w0;
        float lam = 0.f;
        if (DIFF && live) lam = __ldg(p.lam + (p.lam_rows ? row0 + r : static_cast<long long>(head_of(p, head0, r))));
        float v[NV];
        row_load<T, J>(v, s1, l, p.lanes, odd, end, -INFINITY);
        if (!BWD) {
            const float a = inverse_or_zero(row_exp(v, p.lanes)) * p.drop.gain;
            if (DIFF) {
                float u[NV];
                row_load<T, J>(u, s2, l, p.lanes, odd, end, -INFINITY);
                const float b = inverse_or_zero(row_exp(u, p.lanes)) * p.drop.gain * lam;
#pragma unroll
                for (int i = 0; i < NV; ++i) v[i] = v[i] * a - u[i] * b;
            } else {
#pragma unroll
                for (int i = 0; i < NV; ++i) v[i] *= a;
            }
            row_store<T, J>(v, s1, l, p.lanes, odd, end);
        } else {
            float g[NV];
            row_load<T, J>(g, reinterpret_cast<const uint32_t*>(sdy) + w0, l, p.lanes, odd, end, 0.f);
#pragma unroll
            for (int m = 0; m < (DIFF ? 2 : 1); ++m) {
                if (m == 1) row_load<T, J>(v, s2, l, p.lanes, odd, end, -INFINITY);
                const float inv = inverse_or_zero(row_exp(v, p.lanes));
                // a weight of exactly zero (a masked place) takes no part, whatever dy holds there
                float t = 0.f;
#pragma unroll
                for (int i = 0; i < NV; ++i) t += v[i] == 0.f ? 0.f : v[i] * g[i];
                const float q = lanes_sum(t, p.lanes) * inv;
                const float a = inv * p.drop.gain * (m == 1 ? -lam : 1.f);
#pragma unroll
                for (int i = 0; i < NV; ++i) v[i] = v[i] == 0.f ? 0.f : v[i] * a * (g[i] - q);
                row_store<T, J>(v, m == 0 ? s1 : s2, l, p.lanes, odd, end);
                if (m == 1 && live && l == 0) p.dlam[row0 + r] = -p.drop.gain * q;
            }
        }
    }
    char* out[2] = {static_cast<char*>(p.out1) + off, static_cast<char*>(p.out2) + off};
    if (!BWD && dropping) {
        __syncthreads();
        for (uint32_t o = threadIdx.x; o < octets; o += kWinThreads) {
            uint4 second{}, first = mask_octet<T>(reinterpret_cast<uint4*>(smem), o, rng, block0 + o, p.drop.steps, second);
            constexpr uint32_t kOctet = 8 * sizeof(T);
            char* to = out[0] + static_cast<size_t>(o) * kOctet;
            if ((o + 1) * kOctet <= bytes) {
                st_stream(to, first);
                if constexpr (sizeof(T) == 4) st_stream(to + 16, second);
            } else {   // the tensor ends inside this octet
                const uint32_t left = (bytes - o * kOctet) / static_cast<uint32_t>(sizeof(T));
                const T* a = reinterpret_cast<const T*>(&first);
                const T* b = reinterpret_cast<const T*>(&second);
                for (uint32_t i = 0; i < left; ++i) reinterpret_cast<T*>(to)[i] = i < 16 / sizeof(T) ? a[i] : b[i - 16 / sizeof(T)];
            }
        }
        return;
    }
    fence_proxy_async_smem();
    __syncthreads();
    constexpr int NO = DIFF && BWD ? 2 : 1;
    if (threadIdx.x < tail) {
#pragma unroll
        for (int i = 0; i < NO; ++i)
            reinterpret_cast<T*>(out[i] + bulk)[threadIdx.x] = reinterpret_cast<const T*>(smem + i * buf + bulk)[threadIdx.x];
    }
    if (threadIdx.x == 0 && bulk != 0) {
#pragma unroll
        for (int i = 0; i < NO; ++i) bulk_store(out[i], smem + i * buf, bulk);
        tma_store_commit();
        tma_store_wait_read();
    }
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

// Sums of a [n, heads] matrix over n, per_block rows of it to each block: out[block][heads].
__global__ void __launch_bounds__(kWinThreads) head_sum_kernel(const float* in, long long n, int heads, long long per_block,
                                                              float* out) {
    __shared__ float part[kWinThreads];
    const long long r0 = blockIdx.x * per_block, r1 = min(r0 + per_block, n);
    float* to = out + static_cast<long long>(blockIdx.x) * heads;
    if (heads > kWinThreads) {
        for (int h = threadIdx.x; h < heads; h += kWinThreads) {
            float s = 0.f;
            for (long long r = r0; r < r1; ++r) s += in[r * heads + h];
            to[h] = s;
        }
        return;
    }
    const int lanes = kWinThreads / heads, use = lanes * heads;
    float s = 0.f;
    if (threadIdx.x < use) {
        const long long end = r1 * heads;
        float a[4] = {0.f, 0.f, 0.f, 0.f};
        long long i = r0 * heads + threadIdx.x;
        for (; i + 3LL * use < end; i += 4LL * use)
#pragma unroll
            for (int k = 0; k < 4; ++k) a[k] += in[i + static_cast<long long>(k) * use];
        for (; i < end; i += use) a[0] += in[i];
        s = (a[0] + a[1]) + (a[2] + a[3]);
    }
    part[threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.x < heads) {
        float t = 0.f;
        for (int k = 0; k < lanes; ++k) t += part[k * heads + threadIdx.x];
        to[threadIdx.x] = t;
    }
}

// Dropout of a tensor: y = gain x where the generator keeps the element, else 0 (y may be x).  A thread takes
// kOct octets of a block's run, loads them all, then draws.
template <typename T>
__global__ void __launch_bounds__(kWinThreads) dropout_kernel(const T* x, T* y, long long n, Dropout d) {
    using E = Elem<T>;
    constexpr int C = sizeof(T) == 4 ? 2 : 1, V = E::EPC, kOct = 4 / C;
    const unsigned long long o0 = static_cast<unsigned long long>(blockIdx.x) * (kWinThreads * kOct) + threadIdx.x;
    RngState rng{};
    if (d.state) rng = rng_load(d.state);
    uint4 r[kOct][C];
#pragma unroll
    for (int j = 0; j < kOct; ++j) {
        const unsigned long long o = o0 + static_cast<unsigned>(j) * kWinThreads;
        if (static_cast<long long>(o * 8 + 8) <= n)
#pragma unroll
            for (int c = 0; c < C; ++c) r[j][c] = ld_stream(x + o * 8 + c * V);
    }
#pragma unroll
    for (int j = 0; j < kOct; ++j) {
        const unsigned long long o = o0 + static_cast<unsigned>(j) * kWinThreads;
        if (static_cast<long long>(o * 8) >= n) continue;
        uint4 m = make_uint4(~0u, ~0u, ~0u, ~0u), w[2] = {m, m};
        if (d.state) m = keep_masks(rng, o, d.steps);
        if (static_cast<long long>(o * 8 + 8) <= n) {
            if (C == 2) widen_masks(m, w[0], w[1]);
            else w[0] = m;
#pragma unroll
            for (int c = 0; c < C; ++c) {
                float f[V];
                E::unpack(r[j][c], f);
#pragma unroll
                for (int e = 0; e < V; ++e) f[e] *= d.gain;
                st_stream(y + o * 8 + c * V, and4(E::pack(f), w[c]));
            }
        } else {
            for (int e = 0; o * 8 + e < static_cast<unsigned long long>(n); ++e) {
                const float v = E::get(x[o * 8 + e]) * d.gain;
                y[o * 8 + e] = E::put(keep_of(m, e) ? v : 0.f);
            }
        }
    }
}

// ---------------------------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------------------------

// Lanes per row and words per lane: the fewest lane slots, counting a row's reductions (two steps and
// a few fixed instructions per doubling) beside its words.
constexpr int kWordCounts[] = {2, 3, 4, 6, 8, 10, 11, 12};

bool plan_row(int K, int es, int& lanes, int& words) {
    const int need = es == 4 ? K : K / 2 + 1;   // an odd row may share both its end words
    long long best = -1;
    for (int g = 1; g <= 32; g *= 2)
        for (int j : kWordCounts) {
            if (g * j < need) continue;
            int steps = 0;
            while ((1 << steps) < g) ++steps;
            const long long cost = static_cast<long long>(g) * (j * (es == 4 ? 10 : 18) + 10 * steps + 30);
            if (best < 0 || cost < best) {
                best = cost;
                lanes = g;
                words = j;
            }
            break;
        }
    return best >= 0;
}

template <typename T, bool DIFF, bool BWD>
na_status launch_win(WinParams& p, cudaStream_t s) {
    int words = 0;
    if (!plan_row(p.K, sizeof(T), p.lanes, words)) {
        if (p.rows > 0x7fffffffLL) return NA_ERR_UNSUPPORTED;
        win_long_kernel<T, DIFF, BWD><<<static_cast<unsigned>(p.rows), kWinThreads, 0, s>>>(p);
        return launch_result();
    }
    // rows of a block: whole passes of the threads, about 12 KB per tensor; fewer where the grid is small
    const int rpp = kWinThreads / p.lanes, row = p.K * static_cast<int>(sizeof(T));
    int passes = 12288 / (rpp * row);
    passes = passes < 1 ? 1 : passes;
    while (passes > 1 && p.rows / (static_cast<long long>(rpp) * passes) < 4 * kSms) --passes;
    p.tile = rpp * passes;
    const long long blocks = (p.rows + p.tile - 1) / p.tile;
    if (blocks > 0x7fffffffLL) return NA_ERR_UNSUPPORTED;
    const size_t smem = static_cast<size_t>((DIFF ? 2 : 1) + (BWD ? 1 : 0)) * p.tile * row;
    const unsigned nb = static_cast<unsigned>(blocks);
    switch (words) {
        case 2: win_kernel<T, DIFF, BWD, 2><<<nb, kWinThreads, smem, s>>>(p); break;
        case 3: win_kernel<T, DIFF, BWD, 3><<<nb, kWinThreads, smem, s>>>(p); break;
        case 4: win_kernel<T, DIFF, BWD, 4><<<nb, kWinThreads, smem, s>>>(p); break;
        case 6: win_kernel<T, DIFF, BWD, 6><<<nb, kWinThreads, smem, s>>>(p); break;
        case 8: win_kernel<T, DIFF, BWD, 8><<<nb, kWinThreads, smem, s>>>(p); break;
        case 10: win_kernel<T, DIFF, BWD, 10><<<nb, kWinThreads, smem, s>>>(p); break;
        case 11: win_kernel<T, DIFF, BWD, 11><<<nb, kWinThreads, smem, s>>>(p); break;
        default: win_kernel<T, DIFF, BWD, kMaxWords><<<nb, kWinThreads, smem, s>>>(p); break;
    }
    return launch_result();
}

template <bool DIFF, bool BWD>
na_status dispatch_win(WinParams& p, na_dtype dtype, cudaStream_t s) {
    if (dtype == NA_BF16) return launch_win<__nv_bfloat16, DIFF, BWD>(p, s);
    if (dtype == NA_FP16) return launch_win<__half, DIFF, BWD>(p, s);
    return launch_win<float, DIFF, BWD>(p, s);
}

// Sizes, types and the generator of a window-weights call; rows, K and the status word into p.
na_status win_common(int B, int ndim, const int* spatial, int heads, const int* kernel, double p_drop, const void* rng,
                     na_dtype dtype, WinParams& p) {
    if (!kernel || !known_dtype(dtype)) return NA_ERR_INVALID_ARG;
    int L[3];
    long long tokens = 0, K = 1;
    na_status st = grid_tokens(B, ndim, spatial, heads, 1, L, tokens);
    if (st != NA_OK) return st;
    for (int a = 0; a < ndim; ++a) {
        if (kernel[a] < 1 || kernel[a] % 2 == 0 || kernel[a] > spatial[a]) return NA_ERR_INVALID_ARG;
        K *= kernel[a];
        if (K > (1LL << 30)) return NA_ERR_UNSUPPORTED;
    }
    if ((st = grid_tokens(B, ndim, spatial, heads, K, L, tokens)) != NA_OK) return st;
    if (!make_dropout(p_drop, rng, p.drop)) return NA_ERR_INVALID_ARG;
    if (!ptr_aligned(rng, 8)) return NA_ERR_ALIGNMENT;
    p.rows = tokens * heads;
    p.K = static_cast<int>(K);
    p.heads = heads;
    p.rows32 = p.rows < (1LL << 31) ? 1u : 0u;
    p.fd_heads = make_fastdiv(static_cast<uint32_t>(heads));
    p.wait_ns = wait_limit_ns();
    return NA_OK;
}

Span weights_span(const void* t, const WinParams& p, na_dtype dtype) { return Span{t, p.rows * p.K * elem_bytes(dtype)}; }

na_status all_aligned(std::initializer_list<const void*> ps) {
    for (const void* q : ps)
        if (!q) return NA_ERR_INVALID_ARG;
    for (const void* q : ps)
        if (!ptr_aligned(q, 16)) return NA_ERR_ALIGNMENT;
    return NA_OK;
}

// Workspace of the weights' gradient per head: a value per row, and a partial sum per block and head.
constexpr int kSumBlocks = 2 * kSms;
long long sum_tokens(long long tokens) { return (tokens + kSumBlocks - 1) / kSumBlocks; }

size_t diff_workspace(const WinParams& p) {
    const size_t rows = (static_cast<size_t>(p.rows) * 4 + 255) / 256 * 256;
    return rows + (static_cast<size_t>(kSumBlocks) * p.heads * 4 + 255) / 256 * 256;
}

}  // namespace
}  // namespace na

extern "C" {

na_status na_dropout(const void* x, void* y, int64_t n, double p, const void* rng, na_dtype dtype, void* stream) {
    using namespace na;
    if (n < 1 || !known_dtype(dtype) || !x || !y) return NA_ERR_INVALID_ARG;
    if (n > (1LL << 40)) return NA_ERR_UNSUPPORTED;
    Dropout d{};
    if (!make_dropout(p, rng, d)) return NA_ERR_INVALID_ARG;
    if (!ptr_aligned(x, 16) || !ptr_aligned(y, 16) || !ptr_aligned(rng, 8)) return NA_ERR_ALIGNMENT;
    const Span sx{x, n * elem_bytes(dtype)}, sy{y, sx.bytes}, sr{rng, 16};
    if (!output_clear(sy, {sx}, {sr})) return NA_ERR_INVALID_ARG;
    const long long per = 8LL * kWinThreads * (dtype == NA_FP32 ? 2 : 4), blocks = (n + per - 1) / per;
    if (blocks > 0x7fffffffLL) return NA_ERR_UNSUPPORTED;
    const unsigned nb = static_cast<unsigned>(blocks);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == NA_BF16)
        dropout_kernel<<<nb, kWinThreads, 0, s>>>(static_cast<const __nv_bfloat16*>(x), static_cast<__nv_bfloat16*>(y), n, d);
    else if (dtype == NA_FP16)
        dropout_kernel<<<nb, kWinThreads, 0, s>>>(static_cast<const __half*>(x), static_cast<__half*>(y), n, d);
    else
        dropout_kernel<<<nb, kWinThreads, 0, s>>>(static_cast<const float*>(x), static_cast<float*>(y), n, d);
    return launch_result();
}

na_status na_softmax_dropout(const void* x, void* y, int B, int ndim, const int* spatial, int heads, const int* kernel,
                             double p, const void* rng, na_dtype dtype, void* stream) {
    using namespace na;
    WinParams w{};
    na_status st = win_common(B, ndim, spatial, heads, kernel, p, rng, dtype, w);
    if (st != NA_OK) return st;
    if ((st = all_aligned({x, y})) != NA_OK) return st;
    if (!output_clear(weights_span(y, w, dtype), {weights_span(x, w, dtype)}, {Span{rng, 16}})) return NA_ERR_INVALID_ARG;
    if ((st = device_status_word(&w.err)) != NA_OK) return st;
    w.x1 = x;
    w.out1 = y;
    return dispatch_win<false, false>(w, dtype, static_cast<cudaStream_t>(stream));
}

na_status na_softmax_dropout_bwd(const void* x, const void* dy, void* dx, int B, int ndim, const int* spatial, int heads,
                                 const int* kernel, double p, const void* rng, na_dtype dtype, void* stream) {
    using namespace na;
    WinParams w{};
    na_status st = win_common(B, ndim, spatial, heads, kernel, p, rng, dtype, w);
    if (st != NA_OK) return st;
    if ((st = all_aligned({x, dy, dx})) != NA_OK) return st;
    if (!output_clear(weights_span(dx, w, dtype), {weights_span(x, w, dtype), weights_span(dy, w, dtype)}, {Span{rng, 16}}))
        return NA_ERR_INVALID_ARG;
    if ((st = device_status_word(&w.err)) != NA_OK) return st;
    w.x1 = x;
    w.dy = dy;
    w.out1 = dx;
    return dispatch_win<false, true>(w, dtype, static_cast<cudaStream_t>(stream));
}

na_status na_diff_softmax(const void* x1, const void* x2, const float* lam, int lam_per_row, void* y, int B, int ndim,
                          const int* spatial, int heads, const int* kernel, double p, const void* rng, na_dtype dtype,
                          void* stream) {
    using namespace na;
    WinParams w{};
    na_status st = win_common(B, ndim, spatial, heads, kernel, p, rng, dtype, w);
    if (st != NA_OK) return st;
    if (!lam || (lam_per_row != 0 && lam_per_row != 1)) return NA_ERR_INVALID_ARG;
    if ((st = all_aligned({x1, x2, y})) != NA_OK) return st;
    if (!ptr_aligned(lam, 4)) return NA_ERR_ALIGNMENT;
    if (!output_clear(weights_span(y, w, dtype), {weights_span(x1, w, dtype), weights_span(x2, w, dtype)},
                      {Span{rng, 16}, Span{lam, 4 * (lam_per_row ? w.rows : heads)}}))
        return NA_ERR_INVALID_ARG;
    if ((st = device_status_word(&w.err)) != NA_OK) return st;
    w.x1 = x1;
    w.x2 = x2;
    w.lam = lam;
    w.lam_rows = static_cast<uint32_t>(lam_per_row);
    w.out1 = y;
    return dispatch_win<true, false>(w, dtype, static_cast<cudaStream_t>(stream));
}

size_t na_diff_softmax_bwd_workspace_size(int B, int ndim, const int* spatial, int heads, const int* kernel) {
    using namespace na;
    WinParams w{};
    return win_common(B, ndim, spatial, heads, kernel, 0.0, nullptr, NA_FP32, w) == NA_OK ? diff_workspace(w) : 0;
}

na_status na_diff_softmax_bwd(const void* x1, const void* x2, const float* lam, int lam_per_row, const void* dy, void* dx1,
                              void* dx2, float* dlam, int B, int ndim, const int* spatial, int heads, const int* kernel,
                              double p, const void* rng, na_dtype dtype, void* workspace, size_t workspace_bytes,
                              void* stream) {
    using namespace na;
    WinParams w{};
    na_status st = win_common(B, ndim, spatial, heads, kernel, p, rng, dtype, w);
    if (st != NA_OK) return st;
    if (!lam || !dlam || (lam_per_row != 0 && lam_per_row != 1)) return NA_ERR_INVALID_ARG;
    if ((st = all_aligned({x1, x2, dy, dx1, dx2})) != NA_OK) return st;
    if (!ptr_aligned(lam, 4) || !ptr_aligned(dlam, 4)) return NA_ERR_ALIGNMENT;
    const Span s1 = weights_span(x1, w, dtype), s2 = weights_span(x2, w, dtype), sd = weights_span(dy, w, dtype),
               o1 = weights_span(dx1, w, dtype), o2 = weights_span(dx2, w, dtype), sr{rng, 16},
               sl{lam, 4 * (lam_per_row ? w.rows : heads)}, ol{dlam, sl.bytes};
    if (!output_clear(o1, {s1, s2, sd}, {sr, sl, o2, ol}) || !output_clear(o2, {s1, s2, sd}, {sr, sl, ol}) ||
        !output_clear(ol, {}, {s1, s2, sd, sr, sl}))
        return NA_ERR_INVALID_ARG;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    void* ws = nullptr;
    bool owned = false;
    if (!lam_per_row) {
        const size_t need = diff_workspace(w);
        if (workspace) {
            if (workspace_bytes < need) return NA_ERR_WORKSPACE;
            if (!ptr_aligned(workspace, 16)) return NA_ERR_ALIGNMENT;
            if (!output_clear(Span{workspace, static_cast<long long>(need)}, {}, {s1, s2, sd, o1, o2, sr, sl, ol}))
                return NA_ERR_INVALID_ARG;
            ws = workspace;
        }
    }
    if ((st = device_status_word(&w.err)) != NA_OK) return st;
    if (!lam_per_row && !ws) {
        if (cudaMallocAsync(&ws, diff_workspace(w), s) != cudaSuccess) return NA_ERR_WORKSPACE;
        owned = true;
    }
    w.x1 = x1;
    w.x2 = x2;
    w.dy = dy;
    w.lam = lam;
    w.lam_rows = static_cast<uint32_t>(lam_per_row);
    w.out1 = dx1;
    w.out2 = dx2;
    w.dlam = lam_per_row ? dlam : static_cast<float*>(ws);
    st = dispatch_win<true, true>(w, dtype, s);
    if (st == NA_OK && !lam_per_row) {
        // the rows' values [tokens, heads] summed over the tokens, in two steps of a fixed order
        const long long tokens = w.rows / heads, per = sum_tokens(tokens);
        const int blocks = static_cast<int>((tokens + per - 1) / per);
        float* partial = w.dlam + (w.rows + 63) / 64 * 64;
        head_sum_kernel<<<blocks, kWinThreads, 0, s>>>(w.dlam, tokens, heads, per, blocks == 1 ? dlam : partial);
        if (blocks > 1) head_sum_kernel<<<1, kWinThreads, 0, s>>>(partial, blocks, heads, blocks, dlam);
        st = launch_result();
    }
    if (owned && cudaFreeAsync(ws, s) != cudaSuccess && st == NA_OK) st = NA_ERR_CUDA;
    return st;
}

}  // extern "C"
