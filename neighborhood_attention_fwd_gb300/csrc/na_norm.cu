// na_norm.cu -- layer norm over the last axis of a contiguous tensor, forward and backward: the norm of
// queries, keys and outputs per head (C = D channels) and of tokens (C = heads * D).
//
//   mean = sum x / C,  rstd = (sum (x - mean)^2 / C + eps)^-1/2,  h = (x - mean) rstd,  y = h w + b
//   g = dy w:  dx = rstd (g - sum g / C - h sum (g h) / C),  dw = sum over rows of dy h,  db = sum of dy
//
// What bounds it.  A row is read once and held in registers for its statistics and its result (the variance from the
// centred values, so a large mean costs no digits): memory.  A row belongs to a team of threads, each with J chunks of
// the row: lanes of a warp (rows of up to 64 or 128 chunks), else a block.  The backward's teams walk many rows, so
// a thread's columns stay the same and the weight gradients accumulate in its registers; a block writes one
// partial row, and a second kernel adds the partial rows in a fixed order (no atomics: deterministic).
#include "na_block.cuh"

namespace na {
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
    long long rows;
    int C, team;           // threads per row
    float eps, inv_c;
};

// A chunk: V elements, 16 bytes, or one element where a row is not whole chunks.
template <typename T, int V>
__device__ __forceinline__ void load_chunk(const void* base, long long at, float (&f)[V]) {
    if constexpr (V == 1) f[0] = Elem<T>::get(static_cast<const T*>(base)[at]);
    else Elem<T>::unpack(ld_stream(static_cast<const T*>(base) + at), f);
}

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

template <typename T, int V, int J, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? kNormBlock : kNormThreads) norm_fwd_kernel(const NormParams p) {
    __shared__ float slots[2][1][32];
    const int l = BLOCK ? threadIdx.x : (threadIdx.x & (p.team - 1));
    const int team_in_block = BLOCK ? 0 : threadIdx.x / p.team, teams = BLOCK ? 1 : kNormThreads / p.team;
    const long long step = static_cast<long long>(gridDim.x) * teams;
    // every thread of a warp takes part in the sums: rows past the end are computed on zeros and not stored
    const long long first = static_cast<long long>(blockIdx.x) * teams;
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
    for (long long r0 = first; r0 < p.rows; r0 += step) {
        const long long row = r0 + team_in_block;
        const bool live = row < p.rows;
        float x[J][V];
        float s[1] = {0.f};
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int c = (l + p.team * j) * V;
            const bool in = live && c < p.C;
            if (in) load_chunk<T, V>(p.x, row * p.C + c, x[j]);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                if (!in) x[j][e] = 0.f;
                s[0] += x[j][e];
            }
        }
        team_sum<1, BLOCK>(s, p.team, slots[0]);
        const float mean = s[0] * p.inv_c;
        float q[1] = {0.f};
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const bool in = (l + p.team * j) * V < p.C;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                x[j][e] = in ? x[j][e] - mean : 0.f;
                q[0] = fmaf(x[j][e], x[j][e], q[0]);
            }
        }
        team_sum<1, BLOCK>(q, p.team, slots[1]);
        const float rstd = rsqrtf(fmaf(q[0], p.inv_c, p.eps));
        if (live && l == 0 && p.mean) {
            p.mean[row] = mean;
            p.rstd[row] = rstd;
        }
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int c = (l + p.team * j) * V;
            if (live && c < p.C) {
                if (!KEEP) {
                    load_weights<V>(p.w, c, w[0], 1.f);
                    load_weights<V>(p.b, c, b[0], 0.f);
                }
                float y[V];
#pragma unroll
                for (int e = 0; e < V; ++e) y[e] = fmaf(x[j][e] * rstd, w[KEEP ? j : 0][e], b[KEEP ? j : 0][e]);
                store_chunk<T, V>(p.out, row * p.C + c, y);
            }
        }
    }
}

template <typename T, int V, int J, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? kNormBlock : kNormThreads) norm_bwd_kernel(const NormParams p) {
    __shared__ float slots[2][2][32];
    extern __shared__ float cols[];   // warp teams: [warp][2][C]
    const int l = BLOCK ? threadIdx.x : (threadIdx.x & (p.team - 1));
    const int team_in_block = BLOCK ? 0 : threadIdx.x / p.team, teams = BLOCK ? 1 : kNormThreads / p.team;
    const long long step = static_cast<long long>(gridDim.x) * teams;
    float w[J][V], dw[J][V], db[J][V];
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const int c = (l + p.team * j) * V;
        if (c < p.C) load_weights<V>(p.w, c, w[j], 1.f);
#pragma unroll
        for (int e = 0; e < V; ++e) dw[j][e] = db[j][e] = 0.f;
    }
    int turn = 0;
    for (long long r0 = static_cast<long long>(blockIdx.x) * teams; r0 < p.rows; r0 += step, turn ^= 1) {
        const long long row = r0 + team_in_block;
        const bool live = row < p.rows;
        const float mean = live ? __ldg(p.mean + row) : 0.f, rstd = live ? __ldg(p.rstd + row) : 0.f;
        float h[J][V], g[J][V];
        float s[2] = {0.f, 0.f};
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int c = (l + p.team * j) * V;
            if (live && c < p.C) {
                load_chunk<T, V>(p.x, row * p.C + c, h[j]);
                load_chunk<T, V>(p.dy, row * p.C + c, g[j]);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    h[j][e] = (h[j][e] - mean) * rstd;
                    dw[j][e] = fmaf(g[j][e], h[j][e], dw[j][e]);
                    db[j][e] += g[j][e];
                    g[j][e] *= w[j][e];
                    s[0] += g[j][e];
                    s[1] = fmaf(g[j][e], h[j][e], s[1]);
                }
            }
        }
        team_sum<2, BLOCK>(s, p.team, slots[turn]);
        const float c1 = s[0] * p.inv_c, c2 = s[1] * p.inv_c;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int c = (l + p.team * j) * V;
            if (live && c < p.C) {
                float d[V];
#pragma unroll
                for (int e = 0; e < V; ++e) d[e] = (g[j][e] - c1 - h[j][e] * c2) * rstd;
                store_chunk<T, V>(p.out, row * p.C + c, d);
            }
        }
    }
    if (!p.partial) return;
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
    // the warp's teams by shuffles, then the block's warps
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

// dw, db = sums of the blocks' partial rows.  A block takes 32 columns, its 32 warps every 32nd row each.
__global__ void __launch_bounds__(1024) norm_sum_kernel(const float* partial, int blocks, int C, float* dw, float* db) {
    __shared__ float part[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float s = 0.f;
    if (c < 2 * C)
#pragma unroll 4
        for (int r = warp; r < blocks; r += 32) s += partial[static_cast<long long>(r) * 2 * C + c];
    part[warp][lane] = s;
    __syncthreads();
    float t = part[lane][warp];
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) t += __shfl_xor_sync(0xffffffffu, t, m);
    const int cc = blockIdx.x * 32 + warp;
    if (lane == 0 && cc < 2 * C) {
        if (cc < C) dw[cc] = t;
        else db[cc - C] = t;
    }
}

// How a problem is laid out: chunk width, chunks per thread, threads per row, blocks.
struct NormPlan {
    bool vec, block;
    int j, team, blocks;
};

NormPlan plan_norm(long long rows, int C, int es, bool bwd) {
    constexpr int sms = kSms;
    NormPlan n{};
    const int V = C % (16 / es) == 0 ? 16 / es : 1;
    n.vec = V > 1;
    const int chunks = (C + V - 1) / V;
    // chunks per thread of a warp team: the backward keeps weights and two accumulators per column besides
    const int warp_j = n.vec ? (bwd ? 2 : 4) : (bwd ? 2 : 4);
    n.block = chunks > 32 * warp_j;
    if (!n.block) {
        n.team = 1;
        while (n.team < chunks && n.team < 32) n.team *= 2;
        n.j = 1;
        while (n.j * n.team < chunks) n.j *= 2;
        if (!n.vec) n.j = bwd ? 2 : (n.j > 1 ? 4 : 1);
        const long long teams = kNormThreads / n.team, need = (rows + teams - 1) / teams;
        const long long most = static_cast<long long>(sms) * (bwd ? 4 : 16);
        n.blocks = static_cast<int>(need < most ? need : most);
    } else {
        // few rows: a thread for every chunk; else two chunks each
        n.j = n.vec ? (rows < 4LL * sms ? 1 : 2) : 4;
        while (n.j * kNormBlock < chunks) n.j *= n.vec ? 2 : 4;
        const int t = (chunks + n.j - 1) / n.j;
        n.team = (t + 31) / 32 * 32;
        const long long per_sm = 1024 / n.team > 0 ? (1024 / n.team < 16 ? 1024 / n.team : 16) : 1;
        const long long most = static_cast<long long>(sms) * (bwd ? per_sm : 2 * per_sm);
        n.blocks = static_cast<int>(rows < most ? rows : most);
    }
    return n;
}

template <typename T, int V, int J, bool BLOCK, bool BWD>
na_status run_norm(const NormParams& p, const NormPlan& n, cudaStream_t s) {
    const int threads = BLOCK ? n.team : kNormThreads;
    if constexpr (BWD) {
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
        if (n.j == 2) return run_norm<T, V, 2, false, BWD>(p, n, s);
        if constexpr (!BWD) return run_norm<T, V, 4, false, BWD>(p, n, s);
    } else if (n.vec) {
        if (n.j == 1) return run_norm<T, V, 1, true, BWD>(p, n, s);
        if (n.j == 2) return run_norm<T, V, 2, true, BWD>(p, n, s);
        return run_norm<T, V, 4, true, BWD>(p, n, s);
    } else if (!n.block) {
        if constexpr (BWD) return run_norm<T, 1, 2, false, BWD>(p, n, s);
        else return n.j == 1 ? run_norm<T, 1, 1, false, BWD>(p, n, s) : run_norm<T, 1, 4, false, BWD>(p, n, s);
    }
    return n.j == 4 ? run_norm<T, 1, 4, true, BWD>(p, n, s) : run_norm<T, 1, 16, true, BWD>(p, n, s);
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
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    void* ws = nullptr;
    bool owned = false;
    if (dw) {
        const size_t need = norm_workspace(n, C);
        if (workspace) {
            if (workspace_bytes < need) return NA_ERR_WORKSPACE;
            if (!ptr_aligned(workspace, 16)) return NA_ERR_ALIGNMENT;
            const Span sws{workspace, static_cast<long long>(need)};
            if (!output_clear(sws, {}, {sx, sdy, sdx, sw, sm, sr, sdw, sdb})) return NA_ERR_INVALID_ARG;
            ws = workspace;
        } else {
            if (cudaMallocAsync(&ws, need, s) != cudaSuccess) return NA_ERR_WORKSPACE;
            owned = true;
        }
    }
    p.partial = static_cast<float*>(ws);
    st = dispatch_norm<true>(p, n, dtype, s);
    if (st == NA_OK && dw) {
        norm_sum_kernel<<<(2 * C + 31) / 32, 1024, 0, s>>>(p.partial, n.blocks, C, dw, db);
        st = launch_result();
    }
    if (owned && cudaFreeAsync(ws, s) != cudaSuccess && st == NA_OK) st = NA_ERR_CUDA;
    return st;
}

}  // extern "C"
