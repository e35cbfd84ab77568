// na_addnorm.cu -- the end of a block and the start of the next: the block's output normalised, gated and added to the
// stream, and the norm of the stream that the next block reads; forward and backward.
//
//   z = post(y),  s = residual x + scale gate z,  h = norm(s);   post, norm: none, layer norm or root mean square norm
//   e = (s - mean) rstd,  g = dh w,  D = ds + rstd (g - sum g / C - e sum (g e) / C)     (no middle term for root mean square)
//   dx = residual D;  f = (y - post_mean) post_rstd (y without a norm),  q = D scale gate post_w,
//   dy = post_rstd (q - sum q / C - f sum (q f) / C)  (q without a norm);   dw = sum of dh e,  db = sum of dh,
//   dgate = scale (post_w sum D f + post_b sum D),  dpost_w = scale sum gate D f,  dpost_b = scale sum gate D.
//
// What bounds it: memory.  A row belongs to a team of threads, each with J chunks of it: lanes of a warp, else a block; it
// is read once and held for its sums.  Rows that share their vectors (a batch entry's, or all) are a group; a group is cut
// into parts, a block takes parts in turn, and the vectors and the column sums of a part stay in its registers.  A part's
// sums are one partial row (dh e, dh, D f, D; those wanted), and a second kernel adds the parts in a fixed order and
// makes the gradients of the vectors from them (no atomics: deterministic).
#include <algorithm>

#include "na_rows.cuh"

namespace na {
using namespace rows;

namespace {

constexpr int kAddThreads = 256;   // blocks of warp teams
constexpr int kAddBlock = 512;     // most threads of a row's block (128 registers each)
constexpr int kAddMaxC = 8192;
constexpr long long kAddMaxGroups = 32768;   // a group is a row of blocks of the second kernel

struct AddParams {
    const void* x;            // forward
    const void* y;
    const void* s_in;         // backward: the stream that the forward wrote
    const void* dh;           // null: zeros
    const void* ds;           // null: zeros
    void* s;                  // forward: null: not wanted
    void* h;                  // null without a norm
    void* dx;
    void* dy;
    const float* w;           // null: ones; vectors of group i at i * w_step (0: one for all)
    const float* b;           // null: zeros; as w
    const float* gate;        // null: ones; at i * gate_step
    const float* post_w;      // null: ones
    const float* post_b;      // null: zeros
    long long w_step, gate_step;
    float* mean;              // forward: written (null: not wanted); backward: read
    float* rstd;
    float* post_mean;
    float* post_rstd;
    float* partial;           // backward: [parts][sums][C], null: no gradients of vectors
    int slot[4];              // place of dh e, dh, D f, D among a part's sums, -1: not wanted
    int sums;
    int norm, post;           // na_norm_kind
    float scale, residual, eps, inv_c;
    int C, team;              // threads per row
    long long rows, group_rows;
    int groups, per_group;    // parts of a group
};

// The coefficients of the unit rows in z scaled and gated: z = f a + c.  Threads past the row multiply zeros: by ones.
template <int V>
__device__ __forceinline__ void gate_weights(const AddParams& p, const float* gate, int at, float (&a)[V], float (&c)[V]) {
    float g[V], w[V], b[V];
    const bool in = at < p.C;
    load_weights<V>(in ? gate : nullptr, at, g, 1.f);
    load_weights<V>(in ? p.post_w : nullptr, at, w, 1.f);
    load_weights<V>(in ? p.post_b : nullptr, at, b, 0.f);
#pragma unroll
    for (int e = 0; e < V; ++e) {
        a[e] = p.scale * g[e] * w[e];
        c[e] = p.scale * g[e] * b[e];
    }
}

// Rows of a part: a group's tiles of `teams` rows, every per_group-th one.
struct Part {
    long long first, end;     // first row of the part's first tile, end of the group
    const float *w, *b, *gate;
};
__device__ __forceinline__ Part part_of(const AddParams& p, int part, int tile) {
    const int group = part / p.per_group, slice = part - group * p.per_group;
    Part r;
    r.first = group * p.group_rows + static_cast<long long>(slice) * tile;
    r.end = (group + 1) * p.group_rows;
    r.w = p.w ? p.w + group * p.w_step : nullptr;
    r.b = p.b ? p.b + group * p.w_step : nullptr;
    r.gate = p.gate ? p.gate + group * p.gate_step : nullptr;
    return r;
}

template <typename T, int V, int J, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? kAddBlock : kAddThreads) add_fwd_kernel(const AddParams p) {
    using A = Cols<V>;
    using W = typename A::W;
    constexpr int H = A::H;
    constexpr bool KEEP = J * V <= 8;   // vectors stay in registers over a part's rows
    __shared__ float slots[2][4][1][32];   // taken in turn by the rows: a row's sums may be one
    int turn = 0;
    const int l = BLOCK ? threadIdx.x : (threadIdx.x & (p.team - 1));
    const int mine = BLOCK ? 0 : threadIdx.x / p.team, teams = BLOCK ? 1 : kAddThreads / p.team;
    const bool post = p.post != NA_NORM_NONE, norm = p.norm != NA_NORM_NONE;
    for (int part = blockIdx.x; part < p.groups * p.per_group; part += gridDim.x) {
        const Part rows = part_of(p, part, teams);
        W ka[KEEP ? J : 1][H], kc[KEEP ? J : 1][H], kw[KEEP ? J : 1][H], kb[KEEP ? J : 1][H];
        auto vectors = [&](int j, int at) {
            const int i = KEEP ? j : 0;
            float a[V], c[V];
            gate_weights<V>(p, rows.gate, at, a, c);
            A::from(a, ka[i]);
            A::from(c, kc[i]);
        };
        auto weights = [&](int j, int at) {
            const int i = KEEP ? j : 0;
            float w[V], b[V];
            load_weights<V>(at < p.C ? rows.w : nullptr, at, w, 1.f);
            load_weights<V>(at < p.C ? rows.b : nullptr, at, b, 0.f);
            A::from(w, kw[i]);
            A::from(b, kb[i]);
        };
        if (KEEP) {
#pragma unroll
            for (int j = 0; j < J; ++j) {
                vectors(j, (l + p.team * j) * V);
                weights(j, (l + p.team * j) * V);
            }
        }
        for (long long r0 = rows.first; r0 < rows.end; r0 += static_cast<long long>(teams) * p.per_group, turn ^= 1) {
            const bool live = r0 + mine < rows.end;   // whole warps stay together, for the sums
            const long long row = live ? r0 + mine : rows.end - 1;
            Chunk<T, V> rx[J], ry[J];
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const long long at = row * p.C + min((l + p.team * j) * V, p.C - V);
                ry[j].load(p.y, at);
                rx[j].load(p.x, at);
            }
            W s[J][H];
            float r = 1.f;
#pragma unroll
            for (int j = 0; j < J; ++j) {
                float f[V];
                ry[j].get(f);
                A::from(f, s[j]);
            }
            auto inside = [&](int j) { return (l + p.team * j) * V < p.C; };
            // Centres s on its mean for layer norm, and the inverse deviation of what is left.
            auto moments = [&](int kind, int at, float& mean) {
                mean = 0.f;
                if (kind == NA_NORM_LAYER) {
                    W t = 0;
#pragma unroll
                    for (int j = 0; j < J; ++j)
#pragma unroll
                        for (int e = 0; e < H; ++e)
                            if (inside(j)) t = A::add(t, s[j][e]);
                    float sum[1] = {A::sum(t)};
                    team_sum<1, BLOCK>(sum, p.team, slots[turn][at]);
                    mean = sum[0] * p.inv_c;
                    const W m = A::both(-mean);
#pragma unroll
                    for (int j = 0; j < J; ++j)
#pragma unroll
                        for (int e = 0; e < H; ++e) s[j][e] = A::add(s[j][e], m);
                }
                W t = 0;
#pragma unroll
                for (int j = 0; j < J; ++j)
#pragma unroll
                    for (int e = 0; e < H; ++e)
                        if (inside(j)) t = A::fma(s[j][e], s[j][e], t);
                float sum[1] = {A::sum(t)};
                team_sum<1, BLOCK>(sum, p.team, slots[turn][at + 1]);
                return rsqrtf(fmaf(sum[0], p.inv_c, p.eps));
            };
            if (post) {
                float mean;
                r = moments(p.post, 0, mean);
                if (live && l == 0 && p.post_rstd) {
                    p.post_rstd[row] = r;
                    if (p.post == NA_NORM_LAYER) p.post_mean[row] = mean;
                }
            }
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const int at = (l + p.team * j) * V, i = KEEP ? j : 0;
                if (!KEEP) vectors(j, at);
                float f[V];
                rx[j].get(f);
                W x[H];
                A::from(f, x);
#pragma unroll
                for (int e = 0; e < H; ++e)
                    s[j][e] = A::fma(A::mul(s[j][e], A::both(r)), ka[i][e], A::fma(x[e], A::both(p.residual), kc[i][e]));
                if (live && p.s && at < p.C) {
                    A::to(s[j], f);
                    store_chunk<T, V>(p.s, row * p.C + at, f);
                }
            }
            if (!norm) continue;
            float mean;
            r = moments(p.norm, 2, mean);
            if (live && l == 0 && p.rstd) {
                p.rstd[row] = r;
                if (p.norm == NA_NORM_LAYER) p.mean[row] = mean;
            }
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const int at = (l + p.team * j) * V, i = KEEP ? j : 0;
                if (!KEEP) weights(j, at);
                float f[V];
                W h[H];
#pragma unroll
                for (int e = 0; e < H; ++e) h[e] = A::fma(A::mul(s[j][e], A::both(r)), kw[i][e], kb[i][e]);
                if (live && at < p.C) {
                    A::to(h, f);
                    store_chunk<T, V>(p.h, row * p.C + at, f);
                }
            }
        }
    }
}

// A part's sums of one kind.  Warp teams: the warp's teams by shuffles, then the warps through shared memory ([warp][C]).
template <int V, int J, bool BLOCK>
__device__ __forceinline__ void store_sums(const AddParams& p, int part, int slot, const typename Cols<V>::W (&t)[J][Cols<V>::H], int l, float* cols) {
    float* out = p.partial + (static_cast<long long>(part) * p.sums + slot) * p.C;
    float f[J][V];
#pragma unroll
    for (int j = 0; j < J; ++j) Cols<V>::to(t[j], f[j]);
    if constexpr (BLOCK) {
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int c = (l + p.team * j) * V;
#pragma unroll
            for (int e = 0; e < V; ++e)
                if (c < p.C) out[c + e] = f[j][e];
        }
    } else {
#pragma unroll
        for (int m = 16; m >= 1; m >>= 1)
            if (m >= p.team) {
#pragma unroll
                for (int j = 0; j < J; ++j)
#pragma unroll
                    for (int e = 0; e < V; ++e) f[j][e] += __shfl_xor_sync(0xffffffffu, f[j][e], m);
            }
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        __syncthreads();   // the sums before have been read
        if (lane < p.team) {
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const int c = (l + p.team * j) * V;
#pragma unroll
                for (int e = 0; e < V; ++e)
                    if (c < p.C) cols[warp * p.C + c + e] = f[j][e];
            }
        }
        __syncthreads();
        for (int c = threadIdx.x; c < p.C; c += kAddThreads) {
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < kAddThreads / 32; ++i) s += cols[i * p.C + c];
            out[c] = s;
        }
    }
}

template <typename T, int V, int J, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? kAddBlock : kAddThreads) add_bwd_kernel(const AddParams p) {
    using A = Cols<V>;
    using W = typename A::W;
    constexpr int H = A::H;
    constexpr bool KEEP = J * V <= 8;
    __shared__ float slots[2][2][2][32];   // taken in turn by the rows: a row's sums may be one
    int turn = 0;
    extern __shared__ float cols[];   // warp teams: [warp][C]
    const int l = BLOCK ? threadIdx.x : (threadIdx.x & (p.team - 1));
    const int mine = BLOCK ? 0 : threadIdx.x / p.team, teams = BLOCK ? 1 : kAddThreads / p.team;
    const bool post = p.post != NA_NORM_NONE, norm = p.norm != NA_NORM_NONE;
    auto inside = [&](int j) { return (l + p.team * j) * V < p.C; };
    for (int part = blockIdx.x; part < p.groups * p.per_group; part += gridDim.x) {
        const Part rows = part_of(p, part, teams);
        W ka[KEEP ? J : 1][H], kw[KEEP ? J : 1][H];
        W t0[J][H], t1[J][H], t2[J][H], t3[J][H];   // sums of dh e, dh, D f, D
        auto vectors = [&](int j) {
            float a[V], c[V];
            gate_weights<V>(p, rows.gate, (l + p.team * j) * V, a, c);
            A::from(a, ka[KEEP ? j : 0]);
        };
        auto weights = [&](int j) {
            float w[V];
            load_weights<V>(inside(j) ? rows.w : nullptr, (l + p.team * j) * V, w, 1.f);
            A::from(w, kw[KEEP ? j : 0]);
        };
#pragma unroll
        for (int j = 0; j < J; ++j) {
            if (KEEP) {
                vectors(j);
                weights(j);
            }
#pragma unroll
            for (int e = 0; e < H; ++e) t0[j][e] = t1[j][e] = t2[j][e] = t3[j][e] = 0;
        }
        for (long long r0 = rows.first; r0 < rows.end; r0 += static_cast<long long>(teams) * p.per_group, turn ^= 1) {
            const bool live = r0 + mine < rows.end;
            const long long row = live ? r0 + mine : rows.end - 1;
            Chunk<T, V> rdh[J], rds[J], rs[J], ry[J];
            // places past the end are zeros made of zeros: what stands there need not be finite, and may be an output already
            auto read = [&](const Chunk<T, V>& raw, bool there, int j, W (&v)[H]) {
                float f[V];
                raw.get(f);
                A::from(f, v);
#pragma unroll
                for (int e = 0; e < H; ++e)
                    if (!there || !live || !inside(j)) v[e] = 0;
            };
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const long long at = row * p.C + min((l + p.team * j) * V, p.C - V);
                rdh[j].load(p.dh ? p.dh : p.s_in ? p.s_in : p.y, at);
                rs[j].load(p.s_in ? p.s_in : p.y, at);
                rds[j].load(p.ds ? p.ds : p.y, at);
                ry[j].load(p.y, at);
            }
            W d[J][H];
#pragma unroll
            for (int j = 0; j < J; ++j) read(rds[j], p.ds != nullptr, j, d[j]);
            if (norm) {
                const float mean = p.norm == NA_NORM_LAYER ? p.mean[row] : 0.f, rstd = p.rstd[row];
                W e_[J][H], g[J][H], s0 = 0, s1 = 0;
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    if (!KEEP) weights(j);
                    W dh[H];
                    read(rdh[j], p.dh != nullptr, j, dh);
                    read(rs[j], true, j, e_[j]);
#pragma unroll
                    for (int e = 0; e < H; ++e) {
                        e_[j][e] = A::mul(A::add(e_[j][e], A::both(-mean)), A::both(rstd));
                        if (!live || !inside(j)) e_[j][e] = 0;
                        t0[j][e] = A::fma(dh[e], e_[j][e], t0[j][e]);
                        t1[j][e] = A::add(t1[j][e], dh[e]);
                        g[j][e] = A::mul(dh[e], kw[KEEP ? j : 0][e]);
                        s0 = A::add(s0, g[j][e]);
                        s1 = A::fma(g[j][e], e_[j][e], s1);
                    }
                }
                float s[2] = {A::sum(s0), A::sum(s1)};
                team_sum<2, BLOCK>(s, p.team, slots[turn][0]);
                const W k0 = A::both(p.norm == NA_NORM_LAYER ? -rstd * (s[0] * p.inv_c) : 0.f), k1 = A::both(-rstd * (s[1] * p.inv_c));
#pragma unroll
                for (int j = 0; j < J; ++j)
#pragma unroll
                    for (int e = 0; e < H; ++e)
                        d[j][e] = A::add(d[j][e], A::fma(e_[j][e], k1, A::fma(g[j][e], A::both(rstd), k0)));
            }
            W f_[J][H], s0 = 0, s1 = 0;
            const float mean = p.post == NA_NORM_LAYER ? p.post_mean[row] : 0.f, rstd = post ? p.post_rstd[row] : 1.f;
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const int at = (l + p.team * j) * V;
                if (!KEEP) vectors(j);
                read(ry[j], true, j, f_[j]);
                W o[H];
#pragma unroll
                for (int e = 0; e < H; ++e) {
                    o[e] = A::mul(d[j][e], A::both(p.residual));
                    if (!live || !inside(j)) d[j][e] = 0;
                    f_[j][e] = A::mul(A::add(f_[j][e], A::both(-mean)), A::both(rstd));
                    if (!live || !inside(j)) f_[j][e] = 0;
                    t2[j][e] = A::fma(d[j][e], f_[j][e], t2[j][e]);
                    t3[j][e] = A::add(t3[j][e], d[j][e]);
                    d[j][e] = A::mul(d[j][e], ka[KEEP ? j : 0][e]);
                    s0 = A::add(s0, d[j][e]);
                    s1 = A::fma(d[j][e], f_[j][e], s1);
                }
                if (live && at < p.C) {
                    float f[V];
                    A::to(o, f);
                    store_chunk<T, V>(p.dx, row * p.C + at, f);
                }
            }
            W k0 = 0, k1 = 0;
            if (post) {
                float s[2] = {A::sum(s0), A::sum(s1)};
                team_sum<2, BLOCK>(s, p.team, slots[turn][1]);
                k0 = A::both(p.post == NA_NORM_LAYER ? -rstd * (s[0] * p.inv_c) : 0.f);
                k1 = A::both(-rstd * (s[1] * p.inv_c));
            }
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const int at = (l + p.team * j) * V;
                W o[H];
#pragma unroll
                for (int e = 0; e < H; ++e) o[e] = A::fma(f_[j][e], k1, A::fma(d[j][e], A::both(rstd), k0));
                if (live && at < p.C) {
                    float f[V];
                    A::to(o, f);
                    store_chunk<T, V>(p.dy, row * p.C + at, f);
                }
            }
        }
        if (p.slot[0] >= 0) store_sums<V, J, BLOCK>(p, part, p.slot[0], t0, l, cols);
        if (p.slot[1] >= 0) store_sums<V, J, BLOCK>(p, part, p.slot[1], t1, l, cols);
        if (p.slot[2] >= 0) store_sums<V, J, BLOCK>(p, part, p.slot[2], t2, l, cols);
        if (p.slot[3] >= 0) store_sums<V, J, BLOCK>(p, part, p.slot[3], t3, l, cols);
    }
}

// The gradients of the vectors from the parts' sums.  Blocks of the first launch row (if any vector is shared by all groups)
// add all parts, a part's D sums times its group's gate where that has several; the others each add one group's parts.  A
// block takes eight columns (a sector of each partial row), four parts a warp.
struct SumParams {
    const float* partial;
    const float* gate;       // backward's gate, at i * gate_step
    const float* post_w;
    const float* post_b;
    float* dw;
    float* db;
    float* dgate;
    float* dpost_w;
    float* dpost_b;
    long long gate_step;
    int slot[4], sums;
    int C, groups, per_group;
    int all;                 // the first launch row adds all parts
    int w_many, gate_many;   // w and b, gate: one vector a group
    float scale;
};

constexpr int kSumThreads = 1024;
__global__ void __launch_bounds__(kSumThreads) add_sum_kernel(const SumParams p) {
    __shared__ float part[4][kSumThreads / 32][8];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 8 + (lane & 7);
    const bool all = p.all && blockIdx.y == 0;
    const int group = all ? 0 : static_cast<int>(blockIdx.y) - p.all;
    const int first = all ? 0 : group * p.per_group, end = all ? p.groups * p.per_group : first + p.per_group;
    float t[4] = {0.f, 0.f, 0.f, 0.f};
    if (c < p.C) {
#pragma unroll 2
        for (int r = first + (threadIdx.x >> 3); r < end; r += kSumThreads / 8) {
            const float* at = p.partial + static_cast<long long>(r) * p.sums * p.C + c;
            const float gate = all && p.gate_many ? p.gate[r / p.per_group * p.gate_step + c] : 1.f;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (p.slot[i] >= 0) t[i] = fmaf(at[static_cast<long long>(p.slot[i]) * p.C], i < 2 ? 1.f : gate, t[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        t[i] += __shfl_xor_sync(0xffffffffu, t[i], 8);
        t[i] += __shfl_xor_sync(0xffffffffu, t[i], 16);
        if (lane < 8) part[i][warp][lane] = t[i];
    }
    __syncthreads();
    if (warp >= 8) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        t[i] = part[i][lane][warp];
#pragma unroll
        for (int m = 16; m >= 1; m >>= 1) t[i] += __shfl_xor_sync(0xffffffffu, t[i], m);
    }
    const int at = blockIdx.x * 8 + warp;
    if (lane != 0 || at >= p.C) return;
    const long long mine = static_cast<long long>(group) * p.C + at;
    if (all != (p.w_many != 0)) {
        if (p.dw) p.dw[mine] = t[0];
        if (p.db) p.db[mine] = t[1];
    }
    if (p.dgate && all != (p.gate_many != 0))
        p.dgate[mine] = p.scale * fmaf(p.post_w ? p.post_w[at] : 1.f, t[2], p.post_b ? p.post_b[at] * t[3] : 0.f);
    if (all) {
        const float g = p.scale * (p.gate && !p.gate_many ? p.gate[at] : 1.f);
        if (p.dpost_w) p.dpost_w[at] = g * t[2];
        if (p.dpost_b) p.dpost_b[at] = g * t[3];
    }
}

// How a problem is laid out: chunk width, chunks per thread, threads per row, blocks, parts of a group.
struct AddPlan {
    bool vec, block;
    int j, team, blocks, per_group;
};

AddPlan plan_add(long long group_rows, long long groups, int C, int es, bool bwd) {
    AddPlan n{};
    const int V = C % (16 / es) == 0 ? 16 / es : 1;
    n.vec = V > 1;
    const int chunks = C / V;
    const int warp_j = V == 8 ? 1 : (V == 4 ? 2 : 4);
    n.block = chunks > 32 * warp_j;
    int teams = 1, per_sm;
    if (!n.block) {
        n.team = 1;
        while (n.team < chunks && n.team < 32) n.team *= 2;
        n.j = 1;
        while (n.j * n.team < chunks) n.j *= 2;
        if (!n.vec) n.j = 4;
        teams = kAddThreads / n.team;
        per_sm = bwd ? 2 : 4;
    } else {
        n.j = n.vec ? 2 : 4;
        while (n.j * kAddBlock < chunks) n.j *= n.vec ? 2 : 4;
        n.team = ((chunks + n.j - 1) / n.j + 31) / 32 * 32;
        per_sm = std::max(1, std::min(16, (bwd ? 512 : 1024) / n.team));
    }
    const long long tiles = (group_rows + teams - 1) / teams, most = static_cast<long long>(kSms) * per_sm;
    // in the backward a part's sums cost about as much as a few rows of its own
    const long long least = bwd && n.block ? 4 : 1;
    n.per_group = static_cast<int>(std::max(1LL, std::min((tiles + least - 1) / least, most / groups)));
    n.blocks = static_cast<int>(std::min(groups * n.per_group, most));
    return n;
}

template <typename T, int V, int J, bool BLOCK, bool BWD>
na_status run_add(const AddParams& p, const AddPlan& n, cudaStream_t s) {
    const int threads = BLOCK ? n.team : kAddThreads;
    if constexpr (BWD) {
        const size_t smem = BLOCK || !p.partial ? 0 : static_cast<size_t>(kAddThreads / 32) * p.C * sizeof(float);   // at most 8 KB
        add_bwd_kernel<T, V, J, BLOCK><<<n.blocks, threads, smem, s>>>(p);
    } else {
        add_fwd_kernel<T, V, J, BLOCK><<<n.blocks, threads, 0, s>>>(p);
    }
    return launch_result();
}

template <typename T, bool BWD>
na_status launch_add(const AddParams& p, const AddPlan& n, cudaStream_t s) {
    constexpr int V = Elem<T>::EPC;
    if (n.vec && !n.block) {
        if (n.j == 1) return run_add<T, V, 1, false, BWD>(p, n, s);
        if constexpr (V == 4) return run_add<T, V, 2, false, BWD>(p, n, s);
    } else if (n.vec) {
        if (n.j == 2) return run_add<T, V, 2, true, BWD>(p, n, s);
        if constexpr (V == 4) return run_add<T, V, 4, true, BWD>(p, n, s);
    } else if (!n.block) {
        return run_add<T, 1, 4, false, BWD>(p, n, s);
    }
    return n.j == 4 ? run_add<T, 1, 4, true, BWD>(p, n, s) : run_add<T, 1, 16, true, BWD>(p, n, s);
}

template <bool BWD>
na_status dispatch_add(const AddParams& p, const AddPlan& n, na_dtype dtype, cudaStream_t s) {
    if (dtype == NA_BF16) return launch_add<__nv_bfloat16, BWD>(p, n, s);
    if (dtype == NA_FP16) return launch_add<__half, BWD>(p, n, s);
    return launch_add<float, BWD>(p, n, s);
}

bool known_norm(na_norm_kind k) { return k == NA_NORM_NONE || k == NA_NORM_LAYER || k == NA_NORM_RMS; }

// Sizes and kinds that both directions share; groups receives the number of vectors.
na_status add_sizes(long long rows, int C, long long w_groups, long long gate_groups, na_norm_kind norm, na_norm_kind post,
                    float scale, float residual, na_dtype dtype, long long& groups) {
    if (rows < 1 || C < 1 || w_groups < 1 || gate_groups < 1 || !known_dtype(dtype) || !known_norm(norm) || !known_norm(post) ||
        !std::isfinite(scale) || !std::isfinite(residual))
        return NA_ERR_INVALID_ARG;
    if (w_groups > 1 && gate_groups > 1 && w_groups != gate_groups) return NA_ERR_INVALID_ARG;
    groups = std::max(w_groups, gate_groups);
    if (rows % groups != 0) return NA_ERR_INVALID_ARG;
    if (C > kAddMaxC || rows > (1LL << 40) / C || groups > kAddMaxGroups) return NA_ERR_UNSUPPORTED;
    return NA_OK;
}

// A norm's statistics go together: both for layer norm, the inverse deviation alone for root mean square, none without a norm.
bool statistics_fit(na_norm_kind kind, const float* mean, const float* rstd, bool needed) {
    if (kind == NA_NORM_NONE) return !mean && !rstd;
    if (needed && !rstd) return false;
    return kind == NA_NORM_LAYER ? (mean == nullptr) == (rstd == nullptr) : !mean;
}

size_t add_workspace(const AddPlan& n, long long groups, int C, int sums) {
    return (static_cast<size_t>(groups) * n.per_group * sums * C * sizeof(float) + 255) / 256 * 256;
}

}  // namespace
}  // namespace na

extern "C" {

na_status na_addnorm(const void* x, const void* y, void* s, void* h, const float* w, const float* b, const float* gate,
                     const float* post_w, const float* post_b, float* mean, float* rstd, float* post_mean, float* post_rstd,
                     int64_t rows, int C, int64_t w_groups, int64_t gate_groups, na_norm_kind norm, na_norm_kind post,
                     float scale, float residual, float eps, na_dtype dtype, void* stream) {
    using namespace na;
    long long groups;
    const na_status st = add_sizes(rows, C, w_groups, gate_groups, norm, post, scale, residual, dtype, groups);
    if (st != NA_OK) return st;
    if (!x || !y || (!s && !h) || (h != nullptr) != (norm != NA_NORM_NONE) || !std::isfinite(eps) || eps < 0.f ||
        !statistics_fit(norm, mean, rstd, false) || !statistics_fit(post, post_mean, post_rstd, false) ||
        ((w || b) && norm == NA_NORM_NONE) || ((post_w || post_b) && post == NA_NORM_NONE) || (!w && !b && w_groups > 1) ||
        (!gate && gate_groups > 1))
        return NA_ERR_INVALID_ARG;
    for (const void* q : {x, y, static_cast<const void*>(s), static_cast<const void*>(h), static_cast<const void*>(w),
                          static_cast<const void*>(b), static_cast<const void*>(gate), static_cast<const void*>(post_w),
                          static_cast<const void*>(post_b)})
        if (!ptr_aligned(q, 16)) return NA_ERR_ALIGNMENT;
    for (const float* q : {mean, rstd, post_mean, post_rstd})
        if (!ptr_aligned(q, 4)) return NA_ERR_ALIGNMENT;
    const long long bytes = rows * C * elem_bytes(dtype), row = 4LL * C;
    const Span sx{x, bytes}, sy{y, bytes}, ss{s, bytes}, sh{h, bytes}, sw{w, row * w_groups}, sb{b, row * w_groups},
        sg{gate, row * gate_groups}, spw{post_w, row}, spb{post_b, row}, sm{mean, 4 * rows}, sr{rstd, 4 * rows},
        spm{post_mean, 4 * rows}, spr{post_rstd, 4 * rows};
    if (!output_clear(ss, {sx, sy}, {sh, sw, sb, sg, spw, spb, sm, sr, spm, spr}) ||
        !output_clear(sh, {sx, sy}, {sw, sb, sg, spw, spb, sm, sr, spm, spr}) ||
        !output_clear(sm, {}, {sx, sy, sw, sb, sg, spw, spb, sr, spm, spr}) ||
        !output_clear(sr, {}, {sx, sy, sw, sb, sg, spw, spb, spm, spr}) ||
        !output_clear(spm, {}, {sx, sy, sw, sb, sg, spw, spb, spr}) || !output_clear(spr, {}, {sx, sy, sw, sb, sg, spw, spb}))
        return NA_ERR_INVALID_ARG;
    AddParams p{};
    p.x = x;
    p.y = y;
    p.s = s;
    p.h = h;
    p.w = w;
    p.b = b;
    p.gate = gate;
    p.post_w = post_w;
    p.post_b = post_b;
    p.w_step = w_groups > 1 ? C : 0;
    p.gate_step = gate_groups > 1 ? C : 0;
    p.mean = mean;
    p.rstd = rstd;
    p.post_mean = post_mean;
    p.post_rstd = post_rstd;
    p.norm = norm;
    p.post = post;
    p.scale = scale;
    p.residual = residual;
    p.eps = eps;
    p.inv_c = 1.f / static_cast<float>(C);
    p.C = C;
    p.rows = rows;
    p.group_rows = rows / groups;
    p.groups = static_cast<int>(groups);
    const AddPlan n = plan_add(p.group_rows, groups, C, elem_bytes(dtype), false);
    p.team = n.team;
    p.per_group = n.per_group;
    return dispatch_add<false>(p, n, dtype, static_cast<cudaStream_t>(stream));
}

size_t na_addnorm_bwd_workspace_size(int64_t rows, int C, int64_t w_groups, int64_t gate_groups, na_dtype dtype) {
    using namespace na;
    long long groups;
    if (add_sizes(rows, C, w_groups, gate_groups, NA_NORM_LAYER, NA_NORM_LAYER, 1.f, 1.f, dtype, groups) != NA_OK) return 0;
    return add_workspace(plan_add(rows / groups, groups, C, elem_bytes(dtype), true), groups, C, 4);
}

na_status na_addnorm_bwd(const void* dh, const void* ds, const void* s, const void* y, const float* w, const float* gate,
                         const float* post_w, const float* post_b, const float* mean, const float* rstd,
                         const float* post_mean, const float* post_rstd, void* dx, void* dy, float* dw, float* db,
                         float* dgate, float* dpost_w, float* dpost_b, int64_t rows, int C, int64_t w_groups,
                         int64_t gate_groups, na_norm_kind norm, na_norm_kind post, float scale, float residual,
                         na_dtype dtype, void* workspace, size_t workspace_bytes, void* stream) {
    using namespace na;
    long long groups;
    na_status st = add_sizes(rows, C, w_groups, gate_groups, norm, post, scale, residual, dtype, groups);
    if (st != NA_OK) return st;
    const bool normed = norm != NA_NORM_NONE, posted = post != NA_NORM_NONE;
    if (!dx || !dy || !y || (dh != nullptr) != normed || (s != nullptr) != normed || (!normed && !ds) ||
        !statistics_fit(norm, mean, rstd, true) || !statistics_fit(post, post_mean, post_rstd, true) ||
        ((w || dw || db) && !normed) || ((post_w || post_b || dpost_w || dpost_b) && !posted) ||
        (!w && !dw && !db && w_groups > 1) || (!gate && gate_groups > 1) || (dgate && !gate))
        return NA_ERR_INVALID_ARG;
    for (const void* q : {dh, ds, s, y, static_cast<const void*>(w), static_cast<const void*>(gate), static_cast<const void*>(post_w),
                          static_cast<const void*>(post_b), static_cast<const void*>(dx), static_cast<const void*>(dy)})
        if (!ptr_aligned(q, 16)) return NA_ERR_ALIGNMENT;
    for (const float* q : {mean, rstd, post_mean, post_rstd, static_cast<const float*>(dw), static_cast<const float*>(db),
                           static_cast<const float*>(dgate), static_cast<const float*>(dpost_w), static_cast<const float*>(dpost_b)})
        if (!ptr_aligned(q, 4)) return NA_ERR_ALIGNMENT;
    const long long bytes = rows * C * elem_bytes(dtype), row = 4LL * C;
    const Span in[] = {{dh, bytes}, {ds, bytes}, {s, bytes}, {y, bytes}};
    const Span fixed[] = {{w, row * w_groups}, {gate, row * gate_groups}, {post_w, row}, {post_b, row}, {mean, 4 * rows},
                          {rstd, 4 * rows}, {post_mean, 4 * rows}, {post_rstd, 4 * rows}};
    const Span made[] = {{dw, row * w_groups}, {db, row * w_groups}, {dgate, row * gate_groups}, {dpost_w, row}, {dpost_b, row}};
    const Span sdx{dx, bytes}, sdy{dy, bytes};
    // dx is written before y is read
    bool clear = output_clear(sdx, {in[0], in[1], in[2]}, {in[3], sdy}) && output_clear(sdy, {in[0], in[1], in[2], in[3]}, {});
    for (const Span& q : fixed) clear = clear && !spans_overlap(sdx, q) && !spans_overlap(sdy, q);
    for (int i = 0; i < 5; ++i) {
        clear = clear && !spans_overlap(made[i], sdx) && !spans_overlap(made[i], sdy);
        for (const Span& q : in) clear = clear && !spans_overlap(made[i], q);
        for (const Span& q : fixed) clear = clear && !spans_overlap(made[i], q);
        for (int k = 0; k < i; ++k) clear = clear && !spans_overlap(made[i], made[k]);
    }
    if (!clear) return NA_ERR_INVALID_ARG;
    AddParams p{};
    p.dh = dh;
    p.ds = ds;
    p.s_in = s;
    p.y = y;
    p.dx = dx;
    p.dy = dy;
    p.w = w;
    p.gate = gate;
    p.post_w = post_w;
    p.post_b = post_b;
    p.w_step = w_groups > 1 ? C : 0;
    p.gate_step = gate_groups > 1 ? C : 0;
    p.mean = const_cast<float*>(mean);
    p.rstd = const_cast<float*>(rstd);
    p.post_mean = const_cast<float*>(post_mean);
    p.post_rstd = const_cast<float*>(post_rstd);
    p.norm = norm;
    p.post = post;
    p.scale = scale;
    p.residual = residual;
    p.inv_c = 1.f / static_cast<float>(C);
    p.C = C;
    p.rows = rows;
    p.group_rows = rows / groups;
    p.groups = static_cast<int>(groups);
    const AddPlan n = plan_add(p.group_rows, groups, C, elem_bytes(dtype), true);
    p.team = n.team;
    p.per_group = n.per_group;
    const bool wanted[4] = {dw != nullptr, db != nullptr, dgate || dpost_w, dpost_b || (dgate && post_b)};
    for (int i = 0; i < 4; ++i) p.slot[i] = wanted[i] ? p.sums++ : -1;
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    const size_t need = add_workspace(n, groups, C, p.sums);
    void* ws = p.sums ? workspace : nullptr;
    bool owned = false;
    if (ws) {
        if (workspace_bytes < need) return NA_ERR_WORKSPACE;
        if (!ptr_aligned(ws, 16)) return NA_ERR_ALIGNMENT;
        const Span sws{ws, static_cast<long long>(need)};
        bool apart = !spans_overlap(sws, sdx) && !spans_overlap(sws, sdy);
        for (const Span& q : in) apart = apart && !spans_overlap(sws, q);
        for (const Span& q : fixed) apart = apart && !spans_overlap(sws, q);
        for (const Span& q : made) apart = apart && !spans_overlap(sws, q);
        if (!apart) return NA_ERR_INVALID_ARG;
    } else if (p.sums) {
        if (cudaMallocAsync(&ws, need, cs) != cudaSuccess) return NA_ERR_WORKSPACE;
        owned = true;
    }
    p.partial = static_cast<float*>(ws);
    st = dispatch_add<true>(p, n, dtype, cs);
    if (st == NA_OK && p.sums) {
        SumParams q{};
        q.partial = p.partial;
        q.gate = gate;
        q.post_w = post_w;
        q.post_b = post_b;
        q.dw = dw;
        q.db = db;
        q.dgate = dgate;
        q.dpost_w = dpost_w;
        q.dpost_b = dpost_b;
        q.gate_step = p.gate_step;
        for (int i = 0; i < 4; ++i) q.slot[i] = p.slot[i];
        q.sums = p.sums;
        q.C = C;
        q.groups = p.groups;
        q.per_group = n.per_group;
        q.w_many = w_groups > 1;
        q.gate_many = gate_groups > 1;
        q.scale = scale;
        q.all = ((dw || db) && !q.w_many) || (dgate && !q.gate_many) || dpost_w || dpost_b;
        const bool many = ((dw || db) && q.w_many) || (dgate && q.gate_many);
        add_sum_kernel<<<dim3((C + 7) / 8, q.all + (many ? p.groups : 0)), kSumThreads, 0, cs>>>(q);
        st = launch_result();
    }
    if (owned && cudaFreeAsync(ws, cs) != cudaSuccess && st == NA_OK) st = NA_ERR_CUDA;
    return st;
}

}  // extern "C"
