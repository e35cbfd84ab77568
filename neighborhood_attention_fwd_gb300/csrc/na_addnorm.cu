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

#include "na_add.h"

namespace na {
using namespace add;

namespace {

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

constexpr int kSumThreads = 256;
__global__ void __launch_bounds__(kSumThreads) add_sum_kernel(const SumParams p) {
    after_previous();
    __shared__ float part[4][kSumThreads / 32][8];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 8 + (lane & 7);
    const bool all = p.all && blockIdx.y == 0;
    const int group = all ? 0 : static_cast<int>(blockIdx.y) - p.all;
    const int first = all ? 0 : group * p.per_group, end = all ? p.groups * p.per_group : first + p.per_group;
    const bool w_here = all != (p.w_many != 0), gate_here = all != (p.gate_many != 0);
    const bool want[4] = {w_here && p.slot[0] >= 0, w_here && p.slot[1] >= 0, (all || gate_here) && p.slot[2] >= 0, (all || gate_here) && p.slot[3] >= 0};
    float t[4] = {0.f, 0.f, 0.f, 0.f};
    if (c < p.C) {
        const float* gates = all && p.gate_many ? p.gate : nullptr;
#pragma unroll 4
        for (int r = first + (threadIdx.x >> 3); r < end; r += kSumThreads / 8) {
            const float* at = p.partial + static_cast<long long>(r) * p.sums * p.C + c;
            const float gate = gates ? gates[r / p.per_group * p.gate_step + c] : 1.f;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (want[i]) t[i] = fmaf(at[static_cast<long long>(p.slot[i]) * p.C], i < 2 ? 1.f : gate, t[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        t[i] += __shfl_xor_sync(0xffffffffu, t[i], 8);
        t[i] += __shfl_xor_sync(0xffffffffu, t[i], 16);
        if (lane < 8) part[i][warp][lane] = t[i];
    }
    __syncthreads();
    const int at = blockIdx.x * 8 + threadIdx.x;
    if (threadIdx.x >= 8 || at >= p.C) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        t[i] = 0.f;
#pragma unroll
        for (int k = 0; k < kSumThreads / 32; ++k) t[i] += part[i][k][threadIdx.x];
    }
    const long long mine = static_cast<long long>(group) * p.C + at;
    if (w_here) {
        if (p.dw) p.dw[mine] = t[0];
        if (p.db) p.db[mine] = t[1];
    }
    if (p.dgate && gate_here)
        p.dgate[mine] = p.scale * fmaf(p.post_w ? p.post_w[at] : 1.f, t[2], p.post_b ? p.post_b[at] * t[3] : 0.f);
    if (all) {
        const float g = p.scale * (p.gate && !p.gate_many ? p.gate[at] : 1.f);
        if (p.dpost_w) p.dpost_w[at] = g * t[2];
        if (p.dpost_b) p.dpost_b[at] = g * t[3];
    }
}

AddPlan plan_add(long long group_rows, long long groups, int C, int es, bool bwd, bool lean = false) {
    AddPlan n{};
    const int V = C % (16 / es) == 0 ? 16 / es : 1;
    n.vec = V > 1;
    const int chunks = C / V;
    // chunks per thread of a warp team, at most (the backward holds 8 channels to a thread, the forward 16); longer rows are a block's
    const int warp_j = V == 1 ? 8 : (bwd ? 8 / V : 16 / V);
    n.block = chunks > 32 * warp_j;
    int teams = 1, per_sm, units = 1;
    if (!n.block) {
        n.j = 1;
        if (n.vec) {
            while (n.j * 32 < chunks) n.j *= 2;
        } else {
            n.j = chunks > 128 ? 8 : 4;
        }
        n.team = 1;
        while (n.team * n.j < chunks) n.team *= 2;
        teams = 32 / n.team;
        units = kAddThreads / 32;
        per_sm = bwd ? 2 : add_fwd_blocks(n.j * V, lean && n.vec);
    } else {
        n.j = V == 8 ? 1 : (V == 4 ? 2 : 4);
        while (n.j * kAddBlock < chunks) n.j *= 2;
        n.team = ((chunks + n.j - 1) / n.j + 31) / 32 * 32;
        per_sm = std::max(1, std::min(16, (bwd ? 512 : 1024) / n.team));
    }
    n.tile = teams;
    const int arrays = bwd ? 4 : 2, row = C * es;
    const size_t sums = bwd && !n.block ? static_cast<size_t>(kAddThreads / 32) * C * 4 : 0;
    // As many rows of a unit as `per_sm` blocks have room for, of at most kAddTileBytes an array.  A pass of a warp's teams is at most
    // 1 KB an array (2 KB forward): two stages of it, the sums and what else a block holds always fit.
    const size_t room = ((224 * 1024) / per_sm - sums - 4 * 1024) / units;
    auto stages = [&](int passes) { return static_cast<size_t>(kAddStages) * arrays * ring_pitch(teams * passes * row, n.vec); };
    // A ring costs its filling: blocks that have one row each take it straight from memory (333 rows of 1024, 2 bytes, forward: 3.4 ->
    // 3.1 us), rows that are not whole chunks, copied with their edges, up to 16 each (backward, 2 bytes, 1001
    // wide, 2000 rows: 18.5 us, with the ring 22.0; 20000 rows: 128, with the ring 91).
    const bool few = n.block && groups * group_rows <= static_cast<long long>(kSms) * per_sm * (n.vec || n.j == 16 ? 1 : 16);
    if (room >= stages(1) && !few) {
        n.ring = true;
        int passes = std::max(1, std::min(kAddTileBytes / (teams * row), kAddTileRows / teams));
        // fewer rows a tile where there is no room, or where the grid is small
        while (passes > 1 && (stages(passes) > room ||
                              groups * group_rows < static_cast<long long>(teams) * passes * units * kSms * per_sm * kAddStages))
            --passes;
        n.tile = teams * passes;
        n.ring_bytes = stages(passes) * units;
    }
    const long long tiles = (group_rows + n.tile - 1) / n.tile, most = static_cast<long long>(kSms) * per_sm;
    // in the backward a part's sums cost about as much as a few rows of its own
    const long long least = units * (bwd && n.block ? 4 : 1);
    n.per_group = static_cast<int>(std::max(1LL, std::min((tiles + least - 1) / least, most / groups)));
    n.blocks = static_cast<int>(std::min(groups * n.per_group, most));
    return n;
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
    na_status st = add_sizes(rows, C, w_groups, gate_groups, norm, post, scale, residual, dtype, groups);
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
    const AddPlan n = plan_add(p.group_rows, groups, C, elem_bytes(dtype), false, lean_forward(p));
    p.team = n.team;
    p.per_group = n.per_group;
    p.tile = n.tile;
    p.wait_ns = wait_limit_ns();
    p.withhold = wait_withhold();
    if (n.ring && (st = device_status_word(&p.err)) != NA_OK) return st;
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
    p.tile = n.tile;
    p.wait_ns = wait_limit_ns();
    p.withhold = wait_withhold();
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
    }
    if (n.ring && (st = device_status_word(&p.err)) != NA_OK) return st;
    if (p.sums && !ws) {
        if (!taken(cudaMallocAsync(&ws, need, cs))) return NA_ERR_WORKSPACE;
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
        st = launch_after(add_sum_kernel, dim3((C + 7) / 8, q.all + (many ? p.groups : 0)), kSumThreads, cs, q);
    }
    if (owned && cudaFreeAsync(ws, cs) != cudaSuccess && st == NA_OK) st = NA_ERR_CUDA;
    return st;
}

}  // extern "C"
