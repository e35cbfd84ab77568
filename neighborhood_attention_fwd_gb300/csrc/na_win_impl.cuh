// na_win_impl.cuh -- the window softmax in the forms that a transformer's training needs: with dropout on its
// weights, and as the difference of two softmax maps with learned weights, forward and backward.  Included by
// na_win_soft_*.cu and na_win_diff_*.cu (the instances of one form, direction and type each).
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
//
// Measured (bf16; share of the copy rate): softmax with dropout over 9x9 windows at 1024x1024 x 8 heads 472 us, 5.8 TB/s (85%;
// without dropout 454 us); its gradient over (3,5,5) at 4x256x256 x 8 heads, fp16, 167 us (83%); differential softmax with
// dropout at 512x512 184 us (82%); its gradients without dropout over (5,7,7) at 2x8x128x128 847 us, 6.1 TB/s (89%).
// A ring per warp instead of per block took 528 us and more where this took 505, hand-over by a counter instead of
// barriers 550.
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
constexpr int kMaxStages = 3;
// A tile of every input, about; with dropout.  Without: 8 to 24 KB run alike, 12 best.  With (two stages): softmax forward at
// 1024x1024 464 us at 16 KB, 468 at 21, 512 at 32; its gradient at 4x256x256 199, 181, 210.
constexpr int kStageBytes[2] = {12 * 1024, 21 * 1024};
constexpr int kLongThreads = 128;   // block of a row that no tile holds

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

// The place of a lane in its row.  Lane l of L holds words l, l + L, .., J of them; the row has (K + 1) / 2 words (K is
// odd) and fills all but the last of every lane's: only word 0 (`head`: its low half is the row before's) and the
// last words (`last` 0: past the row, 1: the low half alone, 2: whole) need care.
struct Place {
    uint32_t at;     // the lane's first word, in words from the tile's start
    bool head;
    int last;
};

template <typename T, int L, int J>
__device__ __forceinline__ void row_load(uint32_t (&r)[J], const uint32_t* s, const Place& a, uint32_t fill) {
#pragma unroll
    for (int j = 0; j < J - 1; ++j) r[j] = s[L * j];
    r[J - 1] = a.last ? s[L * (J - 1)] : fill;
    if (Words<T>::N == 2) {
        if (a.last == 1) r[J - 1] = (r[J - 1] & 0xffffu) | (fill & 0xffff0000u);
        if (a.head) r[0] = (r[0] & 0xffff0000u) | (fill & 0xffffu);
    }
}

template <typename T, int L, int J>
__device__ __forceinline__ void row_store(const float (&v)[J * Words<T>::N], uint32_t* s, const Place& a) {
    constexpr int N = Words<T>::N;
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const uint32_t u = Words<T>::put(v + j * N);
        uint32_t* to = s + L * j;
        if (N == 2 && j == 0 && a.head) {   // the low half is the row before's
            if (J > 1 || a.last == 2) reinterpret_cast<uint16_t*>(to)[1] = static_cast<uint16_t>(u >> 16);
        } else if (j < J - 1 || a.last == 2) {
            *to = u;
        } else if (N == 2 && a.last == 1) {
            reinterpret_cast<uint16_t*>(to)[0] = static_cast<uint16_t>(u);
        }
    }
}

template <int L>
__device__ __forceinline__ float lanes_max(float v) {
#pragma unroll
    for (int m = L / 2; m >= 1; m >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, m));
    return v;
}

template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int m = L / 2; m >= 1; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
    return v;
}

// The reference point of a row's exponentials: its maximum, or 0 for a row of -inf alone.  `far`: the row has to be shifted
// before the product with log2 e.
__device__ __forceinline__ float row_top(float m, bool& far) {
    if (m == -INFINITY) m = 0.f;
    far = !(fabsf(m) < kFarLogit);
    return m;
}

// v = exp(x - max) of a row, and its sum over the lanes (0 for an empty row).
template <typename T, int L, int J>
__device__ __forceinline__ float row_exp(const uint32_t (&r)[J], float (&v)[J * Words<T>::N]) {
    constexpr int N = Words<T>::N, NV = J * N;
    uint32_t mw = r[0];
#pragma unroll
    for (int j = 1; j < J; ++j) mw = Words<T>::max(mw, r[j]);
    // a NaN in mw loses to any number, and is none where it is alone: its exponential is NaN all the same
    bool far;
    float m = row_top(lanes_max<L>(fmaxf(Words<T>::top(mw), -INFINITY)), far);
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
    return lanes_sum<L>(a);
}

// 1 / l of a row's sum, whose largest term is 1 to within 2^(1/16): 0 for an empty row, or NaN.
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
template <int L, int NV>
__device__ __forceinline__ float row_dot(const float (&v)[NV], const float (&g)[NV]) {
    uint64_t t = 0;
#pragma unroll
    for (int i = 0; i + 1 < NV; i += 2) t = fma2(pack2(v[i], v[i + 1]), pack2(g[i], g[i + 1]), t);
    float a, b;
    split2(t, a, b);
    a += b;
    if (NV % 2) a = fmaf(v[NV - 1], g[NV - 1], a);
    return lanes_sum<L>(a);
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

// Zeros the dropped places of a tile in shared memory: octet o of the tile is block block0 + o of the tensor.
template <typename T, typename Bits>
__device__ __forceinline__ void drop_octets(unsigned char* tile, uint32_t octets, uint32_t steps, Bits bits) {
    constexpr int C = sizeof(T) == 4 ? 2 : 1;
    for (uint32_t o = threadIdx.x; o < octets; o += kWinThreads) {
        uint4* at = reinterpret_cast<uint4*>(tile) + C * o;
        uint4 d[C];
#pragma unroll
        for (int c = 0; c < C; ++c) d[c] = at[c];
        if constexpr (C == 2) drop_words(d[0], d[1], bits(o), steps);
        else drop_words(d[0], bits(o), steps);
#pragma unroll
        for (int c = 0; c < C; ++c) at[c] = d[c];
    }
}
template <typename T>
__device__ __forceinline__ void drop_tile(unsigned char* tile, uint32_t octets, unsigned long long block0, const RngPlan* plan,
                                          const unsigned long long* state, uint32_t steps) {
    if (block0 + octets <= (1ull << 32)) {
        const RngPlan p = *plan;
        const uint32_t first = static_cast<uint32_t>(block0);
        drop_octets<T>(tile, octets, steps, [&](uint32_t o) { return rng_block(p, first + o); });
    } else {
        const RngState rng = rng_load(state);
        drop_octets<T>(tile, octets, steps, [&](uint32_t o) { return rng_block(rng, block0 + o); });
    }
}

// Blocks per multiprocessor that the registers leave room for: the backward holds a row's weights and gradients.
template <bool DIFF, bool BWD>
constexpr int win_blocks() { return BWD && DIFF ? 6 : (BWD || DIFF ? 7 : 8); }

template <typename T, bool DIFF, bool BWD, int L, int J>
__global__ void __launch_bounds__(kWinThreads, win_blocks<DIFF, BWD>()) win_kernel(const __grid_constant__ WinParams p) {
    constexpr int N = Words<T>::N, NV = J * N, NB = (DIFF ? 2 : 1) + (BWD ? 1 : 0), NO = DIFF && BWD ? 2 : 1;
    constexpr int kRows = kWinThreads / L;   // rows of a pass: even, so a lane's place in its row is the same in every pass
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ uint64_t full[kMaxStages];
    __shared__ __align__(16) RngPlan plan;
    __shared__ int issued, lost;   // thread 0's: tiles loaded; the first one whose copy did not land in time (-1: none)
    const uint32_t buf = static_cast<uint32_t>(p.tile) * p.K * sizeof(T);   // a multiple of 16
    const uint32_t stage = NB * buf;
    const WaitGuard guard{p.err, p.wait_ns};
    const long long last_tile = p.tiles - 1;
    const int last_rows = static_cast<int>(p.rows - last_tile * p.tile);
    auto load = [&](long long t, int s) {   // thread 0
        ++issued;
        const uint32_t bulk = t == last_tile ? (static_cast<uint32_t>(last_rows) * p.K * sizeof(T)) & ~15u : buf;
        const long long off = t * static_cast<long long>(buf);
        unsigned char* to = smem + s * stage;
        mbar_arrive_expect_tx(&full[s], NB * bulk);
        if (bulk != 0 && !(p.withhold && blockIdx.x == 0 && issued == 1)) {   // test hook: the first copy never lands
            bulk_load(to, static_cast<const char*>(p.x1) + off, bulk, &full[s]);
            if (DIFF) bulk_load(to + buf, static_cast<const char*>(p.x2) + off, bulk, &full[s]);
            if (BWD) bulk_load(to + (NB - 1) * buf, static_cast<const char*>(p.dy) + off, bulk, &full[s]);
        }
    };
    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) mbar_init(&full[s], 1);
        fence_barrier_init();
        issued = 0;
        lost = -1;
        long long t = blockIdx.x;
        for (int s = 0; s < 2 && t < p.tiles; ++s, t += gridDim.x) load(t, s);
    }
    const bool dropping = p.drop.state != nullptr;
    if (dropping && threadIdx.x == 32) plan = rng_plan(rng_load(p.drop.state));
    const int l = threadIdx.x & (L - 1), r0 = threadIdx.x / L;
    const int words = N == 2 ? (p.K + 1) / 2 : p.K, last_word = l + L * (J - 1);
    const uint32_t e0 = static_cast<uint32_t>(r0) * p.K, pass_words = static_cast<uint32_t>(kRows) * p.K / N;
    Place a;
    a.at = e0 / N + l;
    a.head = N == 2 && (e0 & 1u) && l == 0;
    a.last = last_word < words - 1 ? 2 : (last_word == words - 1 ? (N == 2 && !(e0 & 1u) ? 1 : 2) : 0);
    // head of this lane's row in the first pass of a tile, and its steps from pass to pass and from tile to tile
    uint32_t head = 0, head_pass = 0, head_tile = 0;
    const uint32_t heads = static_cast<uint32_t>(p.heads);
    if (DIFF && !p.lam_rows) {
        head = static_cast<uint32_t>((static_cast<unsigned long long>(blockIdx.x) * p.tile + r0) % heads);
        head_pass = kRows % heads;
        head_tile = static_cast<uint32_t>(static_cast<unsigned long long>(gridDim.x) * p.tile % heads);
    }
    __syncthreads();
    int s = 0;
    uint32_t parity = 0;
    for (long long t = blockIdx.x; t < p.tiles; t += gridDim.x) {
        const long long row0 = t * p.tile;
        unsigned char* tile = smem + s * stage;
        const bool is_last = t == last_tile;
        const int nrows = is_last ? last_rows : p.tile;
        const uint32_t elems = static_cast<uint32_t>(nrows) * p.K, bytes = elems * sizeof(T), bulk = bytes & ~15u;
        const long long off = t * static_cast<long long>(buf);
        // A wait that runs out records itself; the block then goes on to its end without copies, so that its
        // threads keep meeting at the barriers (every later wait gives up at once).
        if (!mbar_wait(&full[s], parity, guard, kSiteWin) && threadIdx.x == 0 && lost < 0)
            lost = static_cast<int>((t - blockIdx.x) / gridDim.x);
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
        // With dropout there are two stages: the tile before this one leaves its buffer during the first of the tile's two
        // phases, and the next one arrives during the second.
        auto refill = [&] {
            if (threadIdx.x == 0 && lost < 0 && t >= gridDim.x) {
                tma_store_wait_read();
                const long long next = t + gridDim.x;
                if (next < p.tiles) load(next, s ^ 1);
            }
        };
        if (BWD && dropping) {
            drop_tile<T>(tile + (NB - 1) * buf, (elems + 7) / 8, block0, &plan, p.drop.state, p.drop.steps);
            refill();
            __syncthreads();
        }
        uint32_t* s1 = reinterpret_cast<uint32_t*>(tile) + a.at;
        uint32_t h = head;
        // rows past the end work on what the buffer holds, for nothing
        for (int r = r0; r - r0 < nrows; r += kRows, s1 += pass_words) {
            uint32_t* s2 = s1 + buf / 4;
            const uint32_t* sg = s1 + (NB - 1) * (buf / 4);
            float lam = 0.f;
            if (DIFF) {
                if (p.lam_rows) {
                    if (r < nrows) lam = __ldg(p.lam + row0 + r);
                } else {
                    lam = __ldg(p.lam + h);
                    h += head_pass;
                    if (h >= heads) h -= heads;
                }
            }
            uint32_t w[J];
            float v[NV];
            row_load<T, L, J>(w, s1, a, Words<T>::kNegInf);
            if (!BWD) {
                row_scale(v, inverse_or_zero(row_exp<T, L, J>(w, v)) * p.drop.gain);
                if (DIFF) {
                    float u[NV];
                    row_load<T, L, J>(w, s2, a, Words<T>::kNegInf);
                    const float b = inverse_or_zero(row_exp<T, L, J>(w, u)) * p.drop.gain;
                    row_axpy(v, u, -(b * lam));
                }
                row_store<T, L, J>(v, s1, a);
            } else {
                float g[NV];
                {
                    uint32_t gw[J];
                    row_load<T, L, J>(gw, sg, a, 0u);
#pragma unroll
                    for (int j = 0; j < J; ++j) Words<T>::get(gw[j], g + j * N);
                }
#pragma unroll
                for (int m = 0; m < NO; ++m) {
                    if (m == 1) row_load<T, L, J>(w, s2, a, Words<T>::kNegInf);
                    const float inv = inverse_or_zero(row_exp<T, L, J>(w, v));
                    const float k = inv * p.drop.gain * (m == 1 ? -lam : 1.f);
                    float q = row_dot<L>(v, g) * inv;
                    const bool fine = fabsf(q) < INFINITY;
                    if (__any_sync(0xffffffffu, !fine)) {
                        // a place of weight zero (a masked one) takes no part, whatever dy holds there: where the sum is
                        // not finite it is taken again without those places
                        float sum = 0.f;
#pragma unroll
                        for (int i = 0; i < NV; ++i) sum += v[i] == 0.f ? 0.f : v[i] * g[i];
                        sum = lanes_sum<L>(sum);
                        if (!fine) q = sum * inv;
                    }
                    // by the row's own sum: the rows that share the warp, or lie past the end, have no say in its bits
                    if (fine) {
                        row_grad(v, g, k, q);
                    } else {
#pragma unroll
                        for (int i = 0; i < NV; ++i) v[i] = v[i] == 0.f ? 0.f : v[i] * k * (g[i] - q);
                    }
                    row_store<T, L, J>(v, m == 0 ? s1 : s2, a);
                    if (m == 1 && r < nrows && l == 0) p.dlam[row0 + r] = -p.drop.gain * q;
                }
            }
        }
        if (DIFF) {
            head += head_tile;
            if (head >= heads) head -= heads;
        }
        if (!BWD && dropping) {
            refill();
            __syncthreads();
            drop_tile<T>(tile, (elems + 7) / 8, block0, &plan, p.drop.state, p.drop.steps);
        }
        fence_proxy_async_smem();
        __syncthreads();
        char* out[2] = {static_cast<char*>(p.out1) + off, static_cast<char*>(NO == 2 ? p.out2 : p.out1) + off};
        if (threadIdx.x < tail) {
#pragma unroll
            for (int i = 0; i < NO; ++i)
                reinterpret_cast<T*>(out[i] + bulk)[threadIdx.x] = reinterpret_cast<const T*>(tile + i * buf + bulk)[threadIdx.x];
        }
        if (threadIdx.x == 0 && lost < 0) {
            if (bulk != 0) {
#pragma unroll
                for (int i = 0; i < NO; ++i) bulk_store(out[i], tile + i * buf, bulk);
            }
            tma_store_commit();
            // without, three: the tile before this one has left its buffer, the second tile from here takes it
            if (!dropping) {
                asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
                const long long next = t + 2LL * gridDim.x;
                if (next < p.tiles) load(next, s == 0 ? 2 : s - 1);
            }
        }
        if (++s == p.stages) {
            s = 0;
            parity ^= 1u;
        }
    }
    if (threadIdx.x == 0) {
        tma_store_wait_read();
        if (lost >= 0)   // the copies in flight have to land before the shared memory is given back
            for (int i = lost; i < issued; ++i) mbar_drain(&full[i % p.stages], (i / p.stages) & 1, p.wait_ns);
    }
}

// Rows that no tile holds (over 767 weights): a block per row, in aligned octets of the tensor (the row's first and last may
// be shared with its neighbours), read again for each pass: a row is a few KB and stays in L1.  Bound by the latency of a
// block's passes: 11x11x11 at 16x32x32 x 8 heads runs at 24 to 34% of the copy rate in bf16, 53 to 68% in fp32.
template <int N>
__device__ __forceinline__ void block_reduce(float (&v)[N], bool maximum, float (*slot)[kLongThreads / 32]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        v[i] = maximum ? lanes_max<32>(v[i]) : lanes_sum<32>(v[i]);
        if (lane == 0) slot[i][warp] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float t = lane < kLongThreads / 32 ? slot[i][lane] : (maximum ? -INFINITY : 0.f);
        v[i] = maximum ? lanes_max<32>(t) : lanes_sum<32>(t);
    }
    __syncthreads();
}

// An octet of the tensor as fp32, with `fill` at the places outside [first, end).
template <typename T>
__device__ __forceinline__ void octet_load(const T* base, long long o, long long first, long long end, long long total, float fill,
                                           float (&f)[8]) {
    constexpr int V = Elem<T>::EPC;
    const long long e0 = o * 8;
    if (e0 + 8 <= total) {
#pragma unroll
        for (int c = 0; c < 8 / V; ++c) {
            float g[V];
            Elem<T>::unpack(*reinterpret_cast<const uint4*>(base + e0 + c * V), g);
#pragma unroll
            for (int e = 0; e < V; ++e) f[c * V + e] = g[e];
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = e0 + e < total ? Elem<T>::get(base[e0 + e]) : fill;
    }
    if (e0 < first || e0 + 8 > end) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e0 + e < first || e0 + e >= end) f[e] = fill;
    }
}

template <typename T>
__device__ __forceinline__ void octet_store(T* base, long long o, long long first, long long end, const float (&f)[8]) {
    constexpr int V = Elem<T>::EPC;
    const long long e0 = o * 8;
    if (e0 >= first && e0 + 8 <= end) {
#pragma unroll
        for (int c = 0; c < 8 / V; ++c) {
            float g[V];
#pragma unroll
            for (int e = 0; e < V; ++e) g[e] = f[c * V + e];
            *reinterpret_cast<uint4*>(base + e0 + c * V) = Elem<T>::pack(g);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e0 + e >= first && e0 + e < end) base[e0 + e] = Elem<T>::put(f[e]);
    }
}

template <typename T, bool DIFF, bool BWD>
__global__ void __launch_bounds__(kLongThreads) win_long_kernel(const __grid_constant__ WinParams p) {
    constexpr int M = DIFF ? 2 : 1;
    __shared__ float slot[M][kLongThreads / 32];
    const long long row = blockIdx.x, first = row * p.K, end = first + p.K, total = p.rows * p.K;
    const long long o0 = (first >> 3) + threadIdx.x, o1 = (end + 7) >> 3;
    const T* x[M];
    x[0] = static_cast<const T*>(p.x1);
    if (DIFF) x[M - 1] = static_cast<const T*>(p.x2);
    const T* dy = static_cast<const T*>(p.dy);
    float lam = 0.f;
    if (DIFF) lam = __ldg(p.lam + (p.lam_rows ? row : row % p.heads));
    RngState rng{};
    const bool dropping = p.drop.state != nullptr;
    if (dropping) rng = rng_load(p.drop.state);
    float m[M], l[M], ml2[M], q[M], f[8];
    bool far[M];
#pragma unroll
    for (int i = 0; i < M; ++i) m[i] = -INFINITY;
    for (long long o = o0; o < o1; o += kLongThreads)
#pragma unroll
        for (int i = 0; i < M; ++i) {
            octet_load(x[i], o, first, end, total, -INFINITY, f);
#pragma unroll
            for (int e = 0; e < 8; ++e) m[i] = fmaxf(m[i], f[e]);
        }
    block_reduce<M>(m, true, slot);
#pragma unroll
    for (int i = 0; i < M; ++i) {
        m[i] = row_top(m[i], far[i]);
        ml2[i] = far[i] ? 0.f : m[i] * kLog2e;
        l[i] = q[i] = 0.f;
    }
    auto weights = [&](int i, long long o, float (&w)[8]) {   // exp(x - max): 0 outside the row
        octet_load(x[i], o, first, end, total, -INFINITY, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = fast_exp2(fmaf(far[i] ? w[e] - m[i] : w[e], kLog2e, -ml2[i]));
    };
    auto gradient = [&](long long o, float (&g)[8]) {   // dy, 0 where it was dropped
        octet_load(dy, o, first, end, total, 0.f, g);
        if (dropping) {
            const uint4 keep = keep_masks(rng, static_cast<unsigned long long>(o), p.drop.steps);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (!keep_of(keep, e)) g[e] = 0.f;
        }
    };
    for (long long o = o0; o < o1; o += kLongThreads) {
        float g[8];
        if (BWD) gradient(o, g);
#pragma unroll
        for (int i = 0; i < M; ++i) {
            weights(i, o, f);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                l[i] += f[e];
                if (BWD) q[i] += f[e] == 0.f ? 0.f : f[e] * g[e];   // a place of weight zero takes no part
            }
        }
    }
    block_reduce<M>(l, false, slot);
    if (BWD) block_reduce<M>(q, false, slot);
#pragma unroll
    for (int i = 0; i < M; ++i) {
        l[i] = inverse_or_zero(l[i]);
        q[i] *= l[i];
        l[i] *= p.drop.gain;
    }
    if (DIFF && BWD && threadIdx.x == 0) p.dlam[row] = -p.drop.gain * q[M - 1];
    if (DIFF) l[M - 1] *= -lam;
    for (long long o = o0; o < o1; o += kLongThreads) {
        if (BWD) {
            float g[8];
            gradient(o, g);
            float w[M][8];
#pragma unroll
            for (int i = 0; i < M; ++i) weights(i, o, w[i]);   // before any store: an output may be an input's tensor
#pragma unroll
            for (int i = 0; i < M; ++i) {
#pragma unroll
                for (int e = 0; e < 8; ++e) w[i][e] = w[i][e] == 0.f ? 0.f : w[i][e] * l[i] * (g[e] - q[i]);
                octet_store(static_cast<T*>(i == 0 ? p.out1 : p.out2), o, first, end, w[i]);
            }
        } else {
            float y[8];
            weights(0, o, y);
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] *= l[0];
            if (DIFF) {
                weights(M - 1, o, f);
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = fmaf(f[e], l[M - 1], y[e]);
            }
            if (dropping) {
                const uint4 keep = keep_masks(rng, static_cast<unsigned long long>(o), p.drop.steps);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (!keep_of(keep, e)) y[e] = 0.f;
            }
            octet_store(static_cast<T*>(p.out1), o, first, end, y);
        }
    }
}

// ---------------------------------------------------------------------------------------------
// Launch
// ---------------------------------------------------------------------------------------------

constexpr int kMaxWords = 12;             // words per lane, at most
constexpr int kMaxWide = 24;              // of a warp's lanes on 4-byte weights (one to a word)
constexpr uint32_t kWinSmem = 220 * 1024; // shared memory of a multiprocessor that the blocks' rings share

template <typename T, bool DIFF, bool BWD, int L, int J>
na_status run_win(WinParams& p, cudaStream_t s) {
    constexpr uint32_t NB = (DIFF ? 2 : 1) + (BWD ? 1 : 0);
    // a tile is whole passes of the threads, about kStageBytes for all inputs; fewer passes where the grid is small
    constexpr int kRows = kWinThreads / L;
    const int row = p.K * static_cast<int>(sizeof(T));
    const bool dropping = p.drop.state != nullptr;
    int passes = kStageBytes[dropping] / static_cast<int>(NB * kRows * row);
    passes = passes < 1 ? 1 : passes;
    while (passes > 1 && p.rows / (static_cast<long long>(kRows) * passes) < 8 * kSms) --passes;
    p.tile = kRows * passes;
    if (p.tile % 8 != 0) p.tile = kRows * (passes += passes & 1);   // 32 lanes: four rows a pass
    p.tiles = (p.rows + p.tile - 1) / p.tile;
    const uint32_t stage = NB * static_cast<uint32_t>(p.tile) * row;
    p.stages = dropping ? 2 : 3;
    const size_t smem = static_cast<size_t>(p.stages) * stage;
    const auto kernel = win_kernel<T, DIFF, BWD, L, J>;
    // 48 KB without asking, static shared memory included
    if (smem > 40 * 1024 && !allow_shared(reinterpret_cast<const void*>(kernel))) return NA_ERR_CUDA;
    int per_sm = static_cast<int>(kWinSmem / (smem + 1024));
    constexpr int kMost = win_blocks<DIFF, BWD>();
    per_sm = per_sm < 1 ? 1 : (per_sm > kMost ? kMost : per_sm);
    const long long most = static_cast<long long>(per_sm) * kSms;
    kernel<<<static_cast<unsigned>(p.tiles < most ? p.tiles : most), kWinThreads, smem, s>>>(p);
    return launch_result();
}

// Words per lane: exactly as many as the row needs.  With two lanes or more they are at least seven (else half the
// lanes would do).
template <typename T, bool DIFF, bool BWD, int L>
na_status run_words(int j, WinParams& p, cudaStream_t s) {
    if constexpr (L == 1) {
        switch (j) {
            case 1: return run_win<T, DIFF, BWD, L, 1>(p, s);
            case 2: return run_win<T, DIFF, BWD, L, 2>(p, s);
            case 3: return run_win<T, DIFF, BWD, L, 3>(p, s);
            case 4: return run_win<T, DIFF, BWD, L, 4>(p, s);
            case 5: return run_win<T, DIFF, BWD, L, 5>(p, s);
            case 6: return run_win<T, DIFF, BWD, L, 6>(p, s);
        }
    }
    switch (j) {
        case 7: return run_win<T, DIFF, BWD, L, 7>(p, s);
        case 8: return run_win<T, DIFF, BWD, L, 8>(p, s);
        case 9: return run_win<T, DIFF, BWD, L, 9>(p, s);
        case 10: return run_win<T, DIFF, BWD, L, 10>(p, s);
        case 11: return run_win<T, DIFF, BWD, L, 11>(p, s);
        case 12: return run_win<T, DIFF, BWD, L, 12>(p, s);
    }
    if constexpr (L == 32 && sizeof(T) == 4) {
        switch (j) {
            case 13: return run_win<T, DIFF, BWD, L, 13>(p, s);
            case 14: return run_win<T, DIFF, BWD, L, 14>(p, s);
            case 15: return run_win<T, DIFF, BWD, L, 15>(p, s);
            case 16: return run_win<T, DIFF, BWD, L, 16>(p, s);
            case 17: return run_win<T, DIFF, BWD, L, 17>(p, s);
            case 18: return run_win<T, DIFF, BWD, L, 18>(p, s);
            case 19: return run_win<T, DIFF, BWD, L, 19>(p, s);
            case 20: return run_win<T, DIFF, BWD, L, 20>(p, s);
            case 21: return run_win<T, DIFF, BWD, L, 21>(p, s);
            case 22: return run_win<T, DIFF, BWD, L, 22>(p, s);
            case 23: return run_win<T, DIFF, BWD, L, 23>(p, s);
            case 24: return run_win<T, DIFF, BWD, L, 24>(p, s);
        }
    }
    return NA_ERR_UNSUPPORTED;
}

template <typename T, bool DIFF, bool BWD>
na_status launch_win_rows(WinParams& p, cudaStream_t s) {
    const int words = sizeof(T) == 4 ? p.K : (p.K + 1) / 2;
    int lanes = 1;   // the fewest: a row costs each of its lanes its reductions besides its words
    while (lanes < 32 && words > kMaxWords * lanes) lanes *= 2;
    const int j = (words + lanes - 1) / lanes;
    if (j > (sizeof(T) == 4 ? kMaxWide : kMaxWords)) {
        if (p.rows > 0x7fffffffLL) return NA_ERR_UNSUPPORTED;
        win_long_kernel<T, DIFF, BWD><<<static_cast<unsigned>(p.rows), kLongThreads, 0, s>>>(p);
        return launch_result();
    }
    switch (lanes) {
        case 1: return run_words<T, DIFF, BWD, 1>(j, p, s);
        case 2: return run_words<T, DIFF, BWD, 2>(j, p, s);
        case 4: return run_words<T, DIFF, BWD, 4>(j, p, s);
        case 8: return run_words<T, DIFF, BWD, 8>(j, p, s);
        case 16: return run_words<T, DIFF, BWD, 16>(j, p, s);
        default: return run_words<T, DIFF, BWD, 32>(j, p, s);
    }
}

}  // namespace
}  // namespace na
