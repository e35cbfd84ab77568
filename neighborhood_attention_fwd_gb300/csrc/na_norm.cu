// na_norm.cu -- layer norm over the last axis of a contiguous tensor, forward and backward: the norm of
// queries, keys and outputs per head (C = D channels) and of tokens (C = heads * D).
//
//   mean = sum x / C,  rstd = (sum (x - mean)^2 / C + eps)^-1/2,  h = (x - mean) rstd,  y = h w + b
//   g = dy w:  dx = rstd (g - sum g / C - h sum (g h) / C),  dw = sum over rows of dy h,  db = sum of dy
//
// What bounds it.  A row is read once and held in registers for its statistics and its result (the variance from the
// centred values, so a large mean costs no digits): memory.  A row belongs to a team of threads, each with J chunks of
// the row: lanes of a warp (rows of up to 32 chunks, of 4-byte elements 64), else a block.  The backward's teams walk many rows, so
// a thread's columns stay the same and the weight gradients accumulate in its registers; a block writes one
// partial row, and a second kernel adds the partial rows in a fixed order (no atomics: deterministic).  Few wide rows need
// neither: blocks of columns beside the rows' blocks read x and dy again.
//
// Measured (bf16; share of the copy rate): 2M rows of 32 channels forward 52 us, 5.5 TB/s (81%); 1M rows of 256 backward
// 286 us, 5.7 TB/s (83%); fp32, 333 rows of 2048 backward 9 to 12 us a call, 3.9 us on the GPU.
#include <algorithm>
#include <type_traits>

#include "na_block.cuh"
#include "na_device.cuh"

namespace na {
using namespace dev;

namespace {

constexpr int kNormThreads = 256;     // blocks of warp teams
constexpr int kNormBlock = 512;       // most threads of a row's block (128 registers each)
constexpr int kNormMaxC = 8192;

struct NormParams {
    const void* x;
    const void* dy;
    void* out;             // y, or dx
    const float* w;        // null: ones
    const float* b;        // null: zeros
    float* mean;           // forward: written (null: not wanted); backward: read
    float* rstd;
    float* partial;        // backward: [blocks][2][C], null: no weight gradients
    float* dw;             // few rows: written by the blocks of columns
    float* db;
    int cols, first;       // few rows: blocks of columns, and the first block of the launch (rows follow columns)
    long long rows;
    int C, team;           // threads per row
    float eps, inv_c;
    long long tiles;       // ring: tiles of `tile` rows
    int tile;
    unsigned* err;         // ring: device status word
    unsigned long long wait_ns;
    uint32_t withhold;     // ring: test hook, block 0 leaves out its first copy
};

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

// Chunk-wise fp32 arithmetic, in pairs where a chunk has them.
template <int V>
__device__ __forceinline__ float chunk_sum(const float (&x)[V]) {
    if constexpr (V == 1) {
        return x[0];
    } else {
        uint64_t t = pack2(x[0], x[1]);
#pragma unroll
        for (int e = 2; e < V; e += 2) t = add2(t, pack2(x[e], x[e + 1]));
        float a, b;
        split2(t, a, b);
        return a + b;
    }
}
template <int V>   // x -= m; returns the sum of squares
__device__ __forceinline__ float chunk_centre(float (&x)[V], float m) {
    if constexpr (V == 1) {
        x[0] -= m;
        return x[0] * x[0];
    } else {
        const uint64_t mm = pack2(-m, -m);
        uint64_t t = 0;
#pragma unroll
        for (int e = 0; e < V; e += 2) {
            const uint64_t d = add2(pack2(x[e], x[e + 1]), mm);
            t = fma2(d, d, t);
            split2(d, x[e], x[e + 1]);
        }
        float a, b;
        split2(t, a, b);
        return a + b;
    }
}
template <int V>   // y = x r w + b
__device__ __forceinline__ void chunk_affine(const float (&x)[V], float r, const float (&w)[V], const float (&b)[V], float (&y)[V]) {
    if constexpr (V == 1) {
        y[0] = fmaf(x[0] * r, w[0], b[0]);
    } else {
        const uint64_t rr = pack2(r, r);
#pragma unroll
        for (int e = 0; e < V; e += 2)
            split2(fma2(mul2(pack2(x[e], x[e + 1]), rr), pack2(w[e], w[e + 1]), pack2(b[e], b[e + 1])), y[e], y[e + 1]);
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

// Rows that a team of the forward works on at once: their loads are in flight together and their sums share the steps.
__host__ __device__ constexpr int norm_rows(int J) { return J == 1 ? 4 : (J <= 4 ? 2 : 1); }

template <typename T, int V, int J, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? kNormBlock : kNormThreads) norm_fwd_kernel(const NormParams p) {
    constexpr int R = norm_rows(J);
    __shared__ float slots[2][R][32];
    const int l = BLOCK ? threadIdx.x : (threadIdx.x & (p.team - 1));
    const int team_in_block = BLOCK ? 0 : threadIdx.x / p.team, teams = BLOCK ? 1 : kNormThreads / p.team;
    const long long step = static_cast<long long>(gridDim.x) * teams * R;   // a block's rows of one turn follow one another
    constexpr bool KEEP = J * V <= 16;   // weights stay in registers over the rows
    float w[KEEP ? J : 1][V], b[KEEP ? J : 1][V];
    if (KEEP) {
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int c = (l + p.team * j) * V;
            if (c < p.C) {
                load_weights<V>(p.w, c, w[KEEP ? j : 0], 1.f);
                load_weights<V>(p.b, c, b[KEEP ? j : 0], 0.f);
            }
        }
    }
    // Every thread of a warp takes part in the sums: rows past the end repeat the last one and are not stored.  The next
    // turn's loads are issued before this turn's sums where that pays for the registers: 2-byte rows of 2048 channels 67%
    // -> 86% of the copy rate, of 4096 61% -> 84%, fp32 rows of 8192 59% -> 89% (two rows at once: 94%), of 1001, element by
    // element, 52% -> 67% (73%); heads of 32 lose (84% -> 82%), and fp32 rows of 2048 (97% -> 89%).
    constexpr bool AHEAD = BLOCK && (V == 8 || J == 4);
    Chunk<T, V> raw[R][J];
    auto load = [&](long long r0) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const long long row = min(r0 + r * teams + team_in_block, p.rows - 1);
#pragma unroll
            for (int j = 0; j < J; ++j) raw[r][j].load(p.x, row * p.C + min((l + p.team * j) * V, p.C - V));
        }
    };
    if (AHEAD) load(static_cast<long long>(blockIdx.x) * teams * R);
    for (long long r0 = static_cast<long long>(blockIdx.x) * teams * R; r0 < p.rows; r0 += step) {
        if (!AHEAD) load(r0);
        float x[R][J][V], s[R], q[R], rstd[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            s[r] = 0.f;
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const bool in = (l + p.team * j) * V < p.C;
                raw[r][j].get(x[r][j]);
                const float t = chunk_sum<V>(x[r][j]);
                s[r] += in ? t : 0.f;
            }
        }
        if (AHEAD) load(r0 + step);
        team_sum<R, BLOCK>(s, p.team, slots[0]);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            s[r] *= p.inv_c;   // the mean
            q[r] = 0.f;
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const bool in = (l + p.team * j) * V < p.C;
                const float t = chunk_centre<V>(x[r][j], s[r]);
                q[r] += in ? t : 0.f;
            }
        }
        team_sum<R, BLOCK>(q, p.team, slots[1]);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const long long row = r0 + r * teams + team_in_block;
            rstd[r] = rsqrtf(fmaf(q[r], p.inv_c, p.eps));
            if (l == 0 && p.mean && row < p.rows) {
                p.mean[row] = s[r];
                p.rstd[row] = rstd[r];
            }
        }
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int c = (l + p.team * j) * V;
            if (c >= p.C) continue;
            if (!KEEP) {
                load_weights<V>(p.w, c, w[0], 1.f);
                load_weights<V>(p.b, c, b[0], 0.f);
            }
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const long long row = r0 + r * teams + team_in_block;
                if (row < p.rows) {
                    float y[V];
                    chunk_affine<V>(x[r][j], rstd[r], w[KEEP ? j : 0], b[KEEP ? j : 0], y);
                    store_chunk<T, V>(p.out, row * p.C + c, y);
                }
            }
        }
    }
}

// A block's partial row of the weight gradients.  Warp teams: the warp's teams by shuffles, then the warps through
// shared memory (cols: [warp][2][C]).
template <int V, int J, bool BLOCK>
__device__ __forceinline__ void store_partial(const NormParams& p, float (&dw)[J][V], float (&db)[J][V], int l, float* cols) {
    float* out = p.partial + static_cast<long long>(blockIdx.x) * 2 * p.C;
    if (BLOCK) {
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int c = (l + p.team * j) * V;
#pragma unroll
            for (int e = 0; e < V; ++e)
                if (c < p.C) {
                    out[c + e] = dw[j][e];
                    out[p.C + c + e] = db[j][e];
                }
        }
        return;
    }
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1)
        if (m >= p.team) {
#pragma unroll
            for (int j = 0; j < J; ++j)
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    dw[j][e] += __shfl_xor_sync(0xffffffffu, dw[j][e], m);
                    db[j][e] += __shfl_xor_sync(0xffffffffu, db[j][e], m);
                }
        }
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (lane < p.team) {
        float* mine = cols + static_cast<size_t>(warp) * 2 * p.C;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int c = (l + p.team * j) * V;
#pragma unroll
            for (int e = 0; e < V; ++e)
                if (c < p.C) {
                    mine[c + e] = dw[j][e];
                    mine[p.C + c + e] = db[j][e];
                }
        }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * p.C; c += kNormThreads) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < kNormThreads / 32; ++i) s += cols[static_cast<size_t>(i) * 2 * p.C + c];
        out[c] = s;
    }
}

// Chunk-wise arithmetic of the backward, H words of one or two columns each: with h = (x - mean) rstd and g = dy w the
// gradient of x is rstd g - rstd sum g / C - h rstd sum (g h) / C.  No square of rstd, which could leave fp32's range where
// every term is within it.
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

// The backward of rows a block wide, and of rows that are not whole chunks.  The next row's loads are issued before this
// one's sums where that pays for the registers: 2-byte rows of 1024 channels 66% -> 73% of the copy rate, of 4096 58% -> 69%,
// fp32 rows of 8192 78% -> 89%; fp32 rows of 2048 lose (91% -> 82%).
template <typename T, int V, int J, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? kNormBlock : kNormThreads) norm_bwd_kernel(const NormParams p) {
    using A = Cols<V>;
    using W = typename A::W;
    constexpr int H = A::H;
    __shared__ float slots[2][2][32];
    extern __shared__ float cols[];   // warp teams: [warp][2][C]
    const int l = BLOCK ? threadIdx.x : (threadIdx.x & (p.team - 1));
    const int team_in_block = BLOCK ? 0 : threadIdx.x / p.team, teams = BLOCK ? 1 : kNormThreads / p.team;
    const long long step = static_cast<long long>(gridDim.x) * teams;
    W w[J][H], dw[J][H], db[J][H];
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const int c = (l + p.team * j) * V;
        float f[V];
        load_weights<V>(c < p.C ? p.w : nullptr, c, f, 1.f);   // threads past the row multiply zeros: by ones
        A::from(f, w[j]);
#pragma unroll
        for (int e = 0; e < H; ++e) dw[j][e] = db[j][e] = 0;
    }
    constexpr bool AHEAD = V != 4 || J == 4;
    Chunk<T, V> rx[J], rg[J];
    float mean = 0.f, rstd = 0.f;
    auto load = [&](long long r0) {
        const long long row = min(r0 + team_in_block, p.rows - 1);
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const long long at = row * p.C + min((l + p.team * j) * V, p.C - V);
            rx[j].load(p.x, at);
            rg[j].load(p.dy, at);
        }
        mean = p.mean[row];
        rstd = p.rstd[row];
    };
    int turn = 0;
    if (AHEAD) load(static_cast<long long>(blockIdx.x) * teams);
    for (long long r0 = static_cast<long long>(blockIdx.x) * teams; r0 < p.rows; r0 += step, turn ^= 1) {
        if (!AHEAD) load(r0);
        const long long row = r0 + team_in_block;
        const bool live = row < p.rows;   // whole warps stay together, for the sums
        W h[J][H], g[J][H], s0 = 0, s1 = 0;
        // a team past the end adds zeros made of zeros: what it read of the last row need not be finite, and may be dx already
        const float rs = rstd;   // the next row's loads overwrite it
        const W mm = A::both(-mean), rr = A::both(rs);
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const bool in = live && (l + p.team * j) * V < p.C;
            float fx[V], fy[V];
            rx[j].get(fx);
            rg[j].get(fy);
            W y[H];
            A::from(fx, h[j]);
            A::from(fy, y);
#pragma unroll
            for (int e = 0; e < H; ++e) {
                if (!in) y[e] = 0;
                h[j][e] = A::mul(A::add(h[j][e], mm), rr);
                if (!BLOCK && !live) h[j][e] = 0;
                dw[j][e] = A::fma(y[e], h[j][e], dw[j][e]);
                db[j][e] = A::add(db[j][e], y[e]);
                g[j][e] = A::mul(y[e], w[j][e]);
                s0 = A::add(s0, g[j][e]);
                s1 = A::fma(g[j][e], h[j][e], s1);
            }
        }
        if (AHEAD && r0 + step < p.rows) load(r0 + step);
        float s[2] = {A::sum(s0), A::sum(s1)};
        team_sum<2, BLOCK>(s, p.team, slots[turn]);
        const W k1 = A::both(-rs * (s[0] * p.inv_c)), k2 = A::both(-rs * (s[1] * p.inv_c));
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int c = (l + p.team * j) * V;
            if (live && c < p.C) {
                W o[H];
#pragma unroll
                for (int e = 0; e < H; ++e) o[e] = A::fma(h[j][e], k2, A::fma(g[j][e], rr, k1));
                float f[V];
                A::to(o, f);
                store_chunk<T, V>(p.out, row * p.C + c, f);
            }
        }
    }
    if (!p.partial) return;
    float fw[J][V], fb[J][V];
#pragma unroll
    for (int j = 0; j < J; ++j) {
        A::to(dw[j], fw[j]);
        A::to(db[j], fb[j]);
    }
    store_partial<V, J, BLOCK>(p, fw, fb, l, cols);
}

// The backward of few wide rows in one launch without a workspace: dw and db need only the saved statistics, so blocks of
// columns take them from x and dy (a second read, out of L2) beside the blocks that each take a row for dx.  A block of
// columns has eight words of them (a sector of a row); its groups of eight lanes each take every 64th row, and the groups'
// sums are added in a fixed order.  Where dx overwrites x or dy the columns are a launch of their own before the rows.
constexpr int kFewThreads = 512, kFewWords = 8;
template <typename T, int J>
__global__ void __launch_bounds__(kFewThreads) norm_bwd_few_kernel(const NormParams p) {
    constexpr int V = Elem<T>::EPC, PER = 4 / static_cast<int>(sizeof(T)), GROUPS = kFewThreads / kFewWords;
    __shared__ float slots[2][32];
    __shared__ float sums[kFewThreads / 32][2][kFewWords * PER];
    const int block = blockIdx.x + p.first;
    if (block < p.cols) {
        const int word = threadIdx.x % kFewWords, c = (block * kFewWords + word) * PER;
        float dw[PER] = {}, db[PER] = {};
        if (c < p.C) {
            const char* x = static_cast<const char*>(p.x) + static_cast<long long>(c) * sizeof(T);
            const char* dy = static_cast<const char*>(p.dy) + static_cast<long long>(c) * sizeof(T);
            const long long pitch = static_cast<long long>(p.C) * sizeof(T);
            const int rows = static_cast<int>(p.rows);
#pragma unroll 4
            for (int r = threadIdx.x / kFewWords; r < rows; r += GROUPS) {
                float fx[PER], fy[PER];
                const uint32_t wx = *reinterpret_cast<const uint32_t*>(x + r * pitch), wy = *reinterpret_cast<const uint32_t*>(dy + r * pitch);
                if constexpr (PER == 1) {
                    fx[0] = __uint_as_float(wx);
                    fy[0] = __uint_as_float(wy);
                } else {
                    Elem<T>::two(wx, fx[0], fx[1]);
                    Elem<T>::two(wy, fy[0], fy[1]);
                }
                const float mean = p.mean[r], rstd = p.rstd[r];
#pragma unroll
                for (int e = 0; e < PER; ++e) {
                    dw[e] = fmaf(fy[e], (fx[e] - mean) * rstd, dw[e]);
                    db[e] += fy[e];
                }
            }
        }
#pragma unroll
        for (int m = 16; m >= kFewWords; m >>= 1)
#pragma unroll
            for (int e = 0; e < PER; ++e) {
                dw[e] += __shfl_xor_sync(0xffffffffu, dw[e], m);
                db[e] += __shfl_xor_sync(0xffffffffu, db[e], m);
            }
        if ((threadIdx.x & 31) < kFewWords) {
#pragma unroll
            for (int e = 0; e < PER; ++e) {
                sums[threadIdx.x >> 5][0][word * PER + e] = dw[e];
                sums[threadIdx.x >> 5][1][word * PER + e] = db[e];
            }
        }
        __syncthreads();
        const int which = threadIdx.x / (kFewWords * PER), k = threadIdx.x % (kFewWords * PER);
        if (which < 2 && block * kFewWords * PER + k < p.C) {
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < kFewThreads / 32; ++i) s += sums[i][which][k];
            (which ? p.db : p.dw)[block * kFewWords * PER + k] = s;
        }
        return;
    }
    const long long row = block - p.cols;
    Chunk<T, V> rx[J], rg[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const long long at = row * p.C + min((static_cast<int>(threadIdx.x) + kFewThreads * j) * V, p.C - V);
        rx[j].load(p.x, at);
        rg[j].load(p.dy, at);
    }
    const float mean = p.mean[row], rstd = p.rstd[row];
    using A = Cols<V>;
    using W = typename A::W;
    constexpr int H = A::H;
    W h[J][H], g[J][H], s0 = 0, s1 = 0;
    const W mm = A::both(-mean), rr = A::both(rstd);
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const int c = (threadIdx.x + kFewThreads * j) * V;
        if (c < p.C) {
            float fx[V], fy[V], fw[V];
            load_weights<V>(p.w, c, fw, 1.f);
            rx[j].get(fx);
            rg[j].get(fy);
            W y[H], w[H];
            A::from(fx, h[j]);
            A::from(fy, y);
            A::from(fw, w);
#pragma unroll
            for (int e = 0; e < H; ++e) {
                h[j][e] = A::mul(A::add(h[j][e], mm), rr);
                g[j][e] = A::mul(y[e], w[e]);
                s0 = A::add(s0, g[j][e]);
                s1 = A::fma(g[j][e], h[j][e], s1);
            }
        }
    }
    float s[2] = {A::sum(s0), A::sum(s1)};
    team_sum<2, true>(s, kFewThreads, slots);
    const W k1 = A::both(-rstd * (s[0] * p.inv_c)), k2 = A::both(-rstd * (s[1] * p.inv_c));
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const int c = (threadIdx.x + kFewThreads * j) * V;
        if (c < p.C) {
            W o[H];
#pragma unroll
            for (int e = 0; e < H; ++e) o[e] = A::fma(h[j][e], k2, A::fma(g[j][e], rr, k1));
            float f[V];
            A::to(o, f);
            store_chunk<T, V>(p.out, row * p.C + c, f);
        }
    }
}

// The backward of warp teams on whole chunks (one each, of 4-byte rows up to two).  A register or two of loads per thread do not keep the memory busy
// beside the accumulators, so x and dy come through a ring of tiles in shared memory (cp.async.bulk; rows are whole
// chunks, so a tile is one run of bytes): a tile's stage is filled again once every thread has read it.  The
// tile's statistics are read a tile ahead.
constexpr int kNormStages = 2, kNormTileBytes = 8 * 1024, kNormTileRows = kNormThreads;   // a thread reads a row's statistics
// Blocks per multiprocessor that the registers leave room for.
__host__ __device__ constexpr int norm_ring_blocks(int J) { return J == 1 ? 4 : 3; }

template <typename T, int J>
__global__ void __launch_bounds__(kNormThreads, norm_ring_blocks(J)) norm_bwd_ring_kernel(const NormParams p) {
    constexpr int V = Elem<T>::EPC;
    extern __shared__ __align__(128) unsigned char smem[];   // [stage][x, dy][tile]; then the columns of store_partial
    __shared__ uint64_t full[kNormStages];
    __shared__ float stats[2][2][kNormTileRows];
    __shared__ int issued, lost;   // thread 0's: tiles loaded; the first one whose copy did not land in time (-1: none)
    const int l = threadIdx.x & (p.team - 1), first = threadIdx.x / p.team, teams = kNormThreads / p.team;
    const uint32_t row_bytes = static_cast<uint32_t>(p.C) * sizeof(T), buf = row_bytes * p.tile;
    const WaitGuard guard{p.err, p.wait_ns};
    auto rows_of = [&](long long t) { return static_cast<int>(min(static_cast<long long>(p.tile), p.rows - t * p.tile)); };
    auto load = [&](long long t, int s) {   // thread 0
        ++issued;
        const uint32_t bytes = row_bytes * rows_of(t);
        const long long off = t * static_cast<long long>(buf);
        mbar_arrive_expect_tx(&full[s], 2 * bytes);
        if (p.withhold && blockIdx.x == 0 && issued == 1) return;   // test hook: the first copy never lands
        bulk_load(smem + (2 * s) * buf, static_cast<const char*>(p.x) + off, bytes, &full[s]);
        bulk_load(smem + (2 * s + 1) * buf, static_cast<const char*>(p.dy) + off, bytes, &full[s]);
    };
    auto read_stats = [&](long long t, int i) {
        if (t < p.tiles && static_cast<int>(threadIdx.x) < rows_of(t)) {
            stats[i][0][threadIdx.x] = p.mean[t * p.tile + threadIdx.x];
            stats[i][1][threadIdx.x] = p.rstd[t * p.tile + threadIdx.x];
        }
    };
    if (threadIdx.x == 0) {
        for (int s = 0; s < kNormStages; ++s) mbar_init(&full[s], 1);
        fence_barrier_init();
        issued = 0;
        lost = -1;
        long long t = blockIdx.x;
        for (int s = 0; s < kNormStages && t < p.tiles; ++s, t += gridDim.x) load(t, s);
    }
    // pairs of columns
    constexpr int H = V / 2;
    uint64_t w[J][H], dw[J][H], db[J][H];
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const int c = (l + p.team * j) * V;
        float f[V];
        load_weights<V>(c < p.C ? p.w : nullptr, c, f, 1.f);
#pragma unroll
        for (int e = 0; e < H; ++e) {
            w[j][e] = pack2(f[2 * e], f[2 * e + 1]);
            dw[j][e] = db[j][e] = 0;
        }
    }
    read_stats(blockIdx.x, 0);
    __syncthreads();
    int s = 0, turn = 0;
    uint32_t parity = 0;
    for (long long t = blockIdx.x; t < p.tiles; t += gridDim.x, turn ^= 1) {
        // a wait that runs out records itself; the block then goes on to its end without copies
        if (!mbar_wait(&full[s], parity, guard, kSiteNorm) && threadIdx.x == 0 && lost < 0)
            lost = static_cast<int>((t - blockIdx.x) / gridDim.x);
        const int n = rows_of(t);
        read_stats(t + gridDim.x, turn ^ 1);
        const unsigned char* at = smem + (2 * s) * buf + first * row_bytes + l * 16;
        T* to = static_cast<T*>(p.out) + (t * p.tile + first) * p.C + l * V;
        // whole warps stay together, for the sums
        for (int r = first; r - first < n; r += teams, at += teams * row_bytes, to += static_cast<long long>(teams) * p.C) {
            const bool live = r < n;
            const float mean = live ? stats[turn][0][r] : 0.f, rstd = live ? stats[turn][1][r] : 0.f;
            const uint64_t mm = pack2(-mean, -mean), rr = pack2(rstd, rstd);
            uint64_t h[J][H], g[J][H], s0 = 0, s1 = 0;
#pragma unroll
            for (int j = 0; j < J; ++j) {
                if (live && (l + p.team * j) * V < p.C) {
                    float fx[V], fy[V];
                    Elem<T>::unpack(*reinterpret_cast<const uint4*>(at + p.team * j * 16), fx);
                    Elem<T>::unpack(*reinterpret_cast<const uint4*>(at + p.team * j * 16 + buf), fy);
#pragma unroll
                    for (int e = 0; e < H; ++e) {
                        const uint64_t y = pack2(fy[2 * e], fy[2 * e + 1]);
                        h[j][e] = mul2(add2(pack2(fx[2 * e], fx[2 * e + 1]), mm), rr);
                        dw[j][e] = fma2(y, h[j][e], dw[j][e]);
                        db[j][e] = add2(db[j][e], y);
                        g[j][e] = mul2(y, w[j][e]);
                        s0 = add2(s0, g[j][e]);
                        s1 = fma2(g[j][e], h[j][e], s1);
                    }
                }
            }
            float sums[2], other[2];
            split2(s0, sums[0], other[0]);
            split2(s1, sums[1], other[1]);
            sums[0] += other[0];
            sums[1] += other[1];
            team_sum<2, false>(sums, p.team, nullptr);
            const float k1 = -rstd * (sums[0] * p.inv_c), k2 = -rstd * (sums[1] * p.inv_c);
            const uint64_t kk1 = pack2(k1, k1), kk2 = pack2(k2, k2);
#pragma unroll
            for (int j = 0; j < J; ++j) {
                if (live && (l + p.team * j) * V < p.C) {
                    float f[V];
#pragma unroll
                    for (int e = 0; e < H; ++e) split2(fma2(h[j][e], kk2, fma2(g[j][e], rr, kk1)), f[2 * e], f[2 * e + 1]);
                    store_chunk<T, V>(to, p.team * j * V, f);
                }
            }
        }
        __syncthreads();   // the tile has been read, the next statistics are in place
        if (threadIdx.x == 0 && lost < 0) {
            const long long next = t + static_cast<long long>(gridDim.x) * kNormStages;
            if (next < p.tiles) load(next, s);
        }
        if (++s == kNormStages) {
            s = 0;
            parity ^= 1u;
        }
    }
    if (threadIdx.x == 0 && lost >= 0)   // the copies in flight have to land before the shared memory is given back
        for (int i = lost; i < issued; ++i) mbar_drain(&full[i % kNormStages], (i / kNormStages) & 1, p.wait_ns);
    __syncthreads();
    if (!p.partial) return;
    float fw[J][V], fb[J][V];
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
        for (int e = 0; e < H; ++e) {
            split2(dw[j][e], fw[j][2 * e], fw[j][2 * e + 1]);
            split2(db[j][e], fb[j][2 * e], fb[j][2 * e + 1]);
        }
    store_partial<V, J, false>(p, fw, fb, l, reinterpret_cast<float*>(smem));
}

// dw, db = sums of the blocks' partial rows.  A block takes eight columns (a sector of each row), four rows a warp, so
// every thread has its few loads in flight at once.
constexpr int kSumThreads = 1024;
__global__ void __launch_bounds__(kSumThreads) norm_sum_kernel(const float* partial, int blocks, int C, float* dw, float* db) {
    __shared__ float part[kSumThreads / 32][8];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 8 + (lane & 7);
    float s = 0.f;
    if (c < 2 * C)
#pragma unroll 8
        for (int r = threadIdx.x >> 3; r < blocks; r += kSumThreads / 8) s += partial[static_cast<long long>(r) * 2 * C + c];
    s += __shfl_xor_sync(0xffffffffu, s, 8);
    s += __shfl_xor_sync(0xffffffffu, s, 16);
    if (lane < 8) part[warp][lane] = s;
    __syncthreads();
    if (warp < 8) {
        float t = part[lane][warp];
#pragma unroll
        for (int m = 16; m >= 1; m >>= 1) t += __shfl_xor_sync(0xffffffffu, t, m);
        const int cc = blockIdx.x * 8 + warp;
        if (lane == 0 && cc < 2 * C) {
            if (cc < C) dw[cc] = t;
            else db[cc - C] = t;
        }
    }
}

// Wide rows up to here take the one launch (in a graph, before -> after: 333 rows of 2048, fp32 8.5 -> 3.8 us, bf16 9.0 -> 3.7;
// 1500 rows of 2048, fp32 15.9 -> 10.3; 1000 rows of 8192, fp32 37.7 -> 33.9; beyond, 1500 rows of 8192, fp32 47.1 -> 50.7, 4000 of
// 520, bf16 11.2 -> 13.5).
constexpr int kFewRows = 1536;
constexpr long long kFewBytes = 32ll << 20;

// How a problem is laid out: chunk width, chunks per thread, threads per row, blocks.
struct NormPlan {
    bool vec, block, ring, few;
    int j, team, blocks, tile;
    long long tiles;
};

NormPlan plan_norm(long long rows, int C, int es, bool bwd) {
    constexpr int sms = kSms;
    NormPlan n{};
    const int V = C % (16 / es) == 0 ? 16 / es : 1;
    n.vec = V > 1;
    const int chunks = (C + V - 1) / V;
    // Chunks per thread of a warp team, at most; longer rows are a block's.  2-byte rows run faster as small blocks with
    // two chunks to a thread (forward, 1024 channels 75% -> 87% of the copy rate; backward, 512 channels 64% -> 80%).
    const int warp_j = V == 8 ? 1 : (V == 4 || bwd ? 2 : 4);
    n.block = chunks > 32 * warp_j;
    if (!n.block) {
        n.team = 1;
        while (n.team < chunks && n.team < 32) n.team *= 2;
        n.j = 1;
        while (n.j * n.team < chunks) n.j *= 2;
        if (!n.vec) n.j = bwd ? 2 : (n.j > 1 ? 4 : 1);
        const long long per = static_cast<long long>(kNormThreads / n.team) * (bwd ? 1 : norm_rows(n.j)), need = (rows + per - 1) / per;
        const long long most = static_cast<long long>(sms) * (bwd ? 3 : 16);
        n.blocks = static_cast<int>(need < most ? need : most);
        if (bwd && n.vec) {   // tiles of whole passes of the teams; fewer where the grid is small
            n.ring = true;
            const int teams = kNormThreads / n.team, per_sm = norm_ring_blocks(n.j);
            int passes = kNormTileBytes / (teams * C * es);
            if (passes * teams > kNormTileRows) passes = kNormTileRows / teams;   // at least 1
            passes = passes < 1 ? 1 : passes;
            while (passes > 1 && rows / (static_cast<long long>(teams) * passes) < 4 * per_sm * sms) --passes;
            n.tile = teams * passes;
            n.tiles = (rows + n.tile - 1) / n.tile;
            const long long grid = static_cast<long long>(per_sm) * sms;
            n.blocks = static_cast<int>(n.tiles < grid ? n.tiles : grid);
        }
    } else if (bwd && n.vec && rows <= kFewRows && rows * C * es <= kFewBytes) {
        n.few = true;
        n.j = (chunks + kFewThreads - 1) / kFewThreads;   // 1, 2, 4 (or 3)
        n.blocks = (chunks * 4 + kFewWords - 1) / kFewWords;
    } else {
        n.j = n.vec ? 2 : 4;   // chunks to a thread
        while (n.j * kNormBlock < chunks) n.j *= n.vec ? 2 : 4;
        const int t = (chunks + n.j - 1) / n.j;
        n.team = (t + 31) / 32 * 32;
        // As many blocks as run at once.  In the backward a block's partial row costs about as much as three rows of its own,
        // so a block gets a few (bf16, 2000 rows of 1024: 25 us with a block per row, 12 with four rows each, 10 with eight; fp32,
        // 2000 rows of 512: 10.6, 8.3 and 9.3).
        const int threads = bwd && n.j > 1 && V == 8 ? 512 : 1024, few = V == 8 ? 8 : 4;
        const long long per_sm = std::max(1, std::min(16, threads / n.team));
        const long long most = static_cast<long long>(sms) * (bwd ? per_sm : 2 * per_sm);
        const long long need = bwd ? std::max(std::min<long long>(rows, sms), rows / few) : rows;
        n.blocks = static_cast<int>(std::min(need, most));
    }
    return n;
}

template <typename T, int V, int J, bool BLOCK, bool BWD>
na_status run_norm(const NormParams& p, const NormPlan& n, cudaStream_t s) {
    const int threads = BLOCK ? n.team : kNormThreads;
    if constexpr (BWD && !BLOCK && V > 1) {
        const size_t ring = 2ull * kNormStages * n.tile * p.C * sizeof(T), sums = static_cast<size_t>(kNormThreads / 32) * 2 * p.C * sizeof(float);
        // at most 32 KB, which a launch has without asking: one pass of the teams is up to 8 KB of x, a tile of several no more
        norm_bwd_ring_kernel<T, J><<<n.blocks, threads, ring > sums ? ring : sums, s>>>(p);
    } else if constexpr (BWD) {
        const size_t smem = BLOCK || !p.partial ? 0 : static_cast<size_t>(kNormThreads / 32) * 2 * p.C * sizeof(float);
        norm_bwd_kernel<T, V, J, BLOCK><<<n.blocks, threads, smem, s>>>(p);
    } else {
        norm_fwd_kernel<T, V, J, BLOCK><<<n.blocks, threads, 0, s>>>(p);
    }
    return launch_result();
}

template <typename T, bool BWD>
na_status launch_norm(const NormParams& p, const NormPlan& n, cudaStream_t s) {
    constexpr int V = Elem<T>::EPC;
    if (n.vec && !n.block) {
        if (n.j == 1) return run_norm<T, V, 1, false, BWD>(p, n, s);
        if constexpr (V == 4)
            if (n.j == 2) return run_norm<T, V, 2, false, BWD>(p, n, s);
    } else if (n.vec) {
        if (n.j == 2) return run_norm<T, V, 2, true, BWD>(p, n, s);
        if constexpr (V == 4) return run_norm<T, V, 4, true, BWD>(p, n, s);   // over 4096 channels of 4 bytes
    } else if (!n.block) {
        if constexpr (BWD) return run_norm<T, 1, 2, false, BWD>(p, n, s);
        else return n.j == 1 ? run_norm<T, 1, 1, false, BWD>(p, n, s) : run_norm<T, 1, 4, false, BWD>(p, n, s);
    }
    return n.j == 4 ? run_norm<T, 1, 4, true, BWD>(p, n, s) : run_norm<T, 1, 16, true, BWD>(p, n, s);
}

// n.blocks: of columns
template <typename T>
na_status launch_few(NormParams p, const NormPlan& n, cudaStream_t s) {
    auto run = [&](int first, int blocks) {
        p.first = first;
        if (n.j == 1) norm_bwd_few_kernel<T, 1><<<blocks, kFewThreads, 0, s>>>(p);
        else if (n.j == 2) norm_bwd_few_kernel<T, 2><<<blocks, kFewThreads, 0, s>>>(p);
        else if constexpr (sizeof(T) == 4) norm_bwd_few_kernel<T, 4><<<blocks, kFewThreads, 0, s>>>(p);
        return launch_result();
    };
    const int rows = static_cast<int>(p.rows);
    p.cols = p.dw ? n.blocks : 0;
    const bool over = p.out == p.x || p.out == p.dy;
    if (!over || !p.cols) return run(0, p.cols + rows);
    const na_status st = run(0, p.cols);
    return st == NA_OK ? run(p.cols, rows) : st;
}

template <bool BWD>
na_status dispatch_norm(const NormParams& p, const NormPlan& n, na_dtype dtype, cudaStream_t s) {
    if (dtype == NA_BF16) return launch_norm<__nv_bfloat16, BWD>(p, n, s);
    if (dtype == NA_FP16) return launch_norm<__half, BWD>(p, n, s);
    return launch_norm<float, BWD>(p, n, s);
}

na_status norm_sizes(long long rows, int C, na_dtype dtype) {
    if (rows < 1 || C < 1 || !known_dtype(dtype)) return NA_ERR_INVALID_ARG;
    if (C > kNormMaxC || rows > (1LL << 40) / C) return NA_ERR_UNSUPPORTED;
    return NA_OK;
}

size_t norm_workspace(const NormPlan& n, int C) {
    if (n.few) return 0;
    return (static_cast<size_t>(n.blocks) * 2 * C * sizeof(float) + 255) / 256 * 256;
}

}  // namespace
}  // namespace na

extern "C" {

na_status na_layernorm(const void* x, const float* w, const float* b, void* y, float* mean, float* rstd, int64_t rows,
                       int C, float eps, na_dtype dtype, void* stream) {
    using namespace na;
    na_status st = norm_sizes(rows, C, dtype);
    if (st != NA_OK) return st;
    if (!x || !y || (mean == nullptr) != (rstd == nullptr) || !std::isfinite(eps) || eps < 0.f) return NA_ERR_INVALID_ARG;
    for (const void* q : {x, static_cast<const void*>(y), static_cast<const void*>(w), static_cast<const void*>(b)})
        if (!ptr_aligned(q, 16)) return NA_ERR_ALIGNMENT;
    if (!ptr_aligned(mean, 4) || !ptr_aligned(rstd, 4)) return NA_ERR_ALIGNMENT;
    const Span sx{x, rows * C * elem_bytes(dtype)}, sy{y, sx.bytes}, sw{w, 4LL * C}, sb{b, 4LL * C}, sm{mean, 4 * rows}, sr{rstd, 4 * rows};
    if (!output_clear(sy, {sx}, {sw, sb, sm, sr}) || !output_clear(sm, {}, {sx, sw, sb, sr}) ||
        !output_clear(sr, {}, {sx, sw, sb}))
        return NA_ERR_INVALID_ARG;
    NormParams p{};
    p.x = x;
    p.out = y;
    p.w = w;
    p.b = b;
    p.mean = mean;
    p.rstd = rstd;
    p.rows = rows;
    p.C = C;
    p.eps = eps;
    p.inv_c = 1.f / static_cast<float>(C);
    const NormPlan n = plan_norm(rows, C, elem_bytes(dtype), false);
    p.team = n.team;
    return dispatch_norm<false>(p, n, dtype, static_cast<cudaStream_t>(stream));
}

size_t na_layernorm_bwd_workspace_size(int64_t rows, int C, na_dtype dtype) {
    using namespace na;
    if (norm_sizes(rows, C, dtype) != NA_OK) return 0;
    return norm_workspace(plan_norm(rows, C, elem_bytes(dtype), true), C);
}

na_status na_layernorm_bwd(const void* dy, const void* x, const float* w, const float* mean, const float* rstd, void* dx,
                           float* dw, float* db, int64_t rows, int C, na_dtype dtype, void* workspace,
                           size_t workspace_bytes, void* stream) {
    using namespace na;
    na_status st = norm_sizes(rows, C, dtype);
    if (st != NA_OK) return st;
    if (!dy || !x || !mean || !rstd || !dx || (dw == nullptr) != (db == nullptr)) return NA_ERR_INVALID_ARG;
    for (const void* q : {dy, x, static_cast<const void*>(dx), static_cast<const void*>(w)})
        if (!ptr_aligned(q, 16)) return NA_ERR_ALIGNMENT;
    for (const float* q : {mean, rstd, static_cast<const float*>(dw), static_cast<const float*>(db)})
        if (!ptr_aligned(q, 4)) return NA_ERR_ALIGNMENT;
    const Span sx{x, rows * C * elem_bytes(dtype)}, sdy{dy, sx.bytes}, sdx{dx, sx.bytes}, sw{w, 4LL * C}, sm{mean, 4 * rows},
        sr{rstd, 4 * rows}, sdw{dw, 4LL * C}, sdb{db, 4LL * C};
    if (!output_clear(sdx, {sx, sdy}, {sw, sm, sr, sdw, sdb}) || !output_clear(sdw, {}, {sx, sdy, sw, sm, sr, sdb}) ||
        !output_clear(sdb, {}, {sx, sdy, sw, sm, sr}))
        return NA_ERR_INVALID_ARG;
    NormParams p{};
    p.x = x;
    p.dy = dy;
    p.out = dx;
    p.w = w;
    p.mean = const_cast<float*>(mean);
    p.rstd = const_cast<float*>(rstd);
    p.rows = rows;
    p.C = C;
    p.inv_c = 1.f / static_cast<float>(C);
    const NormPlan n = plan_norm(rows, C, elem_bytes(dtype), true);
    p.team = n.team;
    p.tile = n.tile;
    p.tiles = n.tiles;
    p.wait_ns = wait_limit_ns();
    p.withhold = wait_withhold();
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const size_t need = norm_workspace(n, C);
    void* ws = dw ? workspace : nullptr;
    bool owned = false;
    if (ws) {
        if (workspace_bytes < need) return NA_ERR_WORKSPACE;
        if (!ptr_aligned(ws, 16)) return NA_ERR_ALIGNMENT;
        const Span sws{ws, static_cast<long long>(need)};
        if (!output_clear(sws, {}, {sx, sdy, sdx, sw, sm, sr, sdw, sdb})) return NA_ERR_INVALID_ARG;
    }
    if (n.ring && (st = device_status_word(&p.err)) != NA_OK) return st;
    if (n.few) {
        p.dw = dw;
        p.db = db;
        if (dtype == NA_BF16) return launch_few<__nv_bfloat16>(p, n, s);
        return dtype == NA_FP16 ? launch_few<__half>(p, n, s) : launch_few<float>(p, n, s);
    }
    if (dw && !ws) {
        if (cudaMallocAsync(&ws, need, s) != cudaSuccess) return NA_ERR_WORKSPACE;
        owned = true;
    }
    p.partial = static_cast<float*>(ws);
    st = dispatch_norm<true>(p, n, dtype, s);
    if (st == NA_OK && dw) {
        norm_sum_kernel<<<(2 * C + 7) / 8, kSumThreads, 0, s>>>(p.partial, n.blocks, C, dw, db);
        st = launch_result();
    }
    if (owned && cudaFreeAsync(ws, s) != cudaSuccess && st == NA_OK) st = NA_ERR_CUDA;
    return st;
}

}  // extern "C"
