// na_glu.cu -- the gated feed-forward product h = act(x Wg^T + bg) * (x Wu^T + bu) and its gradients: host side, plans and
// copies.  The tensor-core kernels are in na_glu_tc.cuh; those on FMA units (fp32 tensors, and small 2-byte ones whose rows
// are not whole 16-byte chunks) and the sums that follow the products in na_glu_fma.cuh.
//
//   g = x Wg^T + bg,  u = x Wu^T + bu,  h = act(g) u
//   dg = dh u act'(g),  du = dh act(g);  dx = dg Wg + du Wu,  dWg = dg^T x,  dWu = du^T x,  dbg, dbu = column sums of dg, du
//
// Nothing is kept from the forward: the backward makes g and u again (4 T D F of its 12 T D F operations), so training holds
// no array of T F elements between the passes.  dg and du go through the workspace in the tensors' type: beside 2-byte x and
// weights the tensor cores take no wider operands.  A sum over them keeps the relative size of that rounding, and it is as large as
// the result's own: against 64 bits the gradients are off by 0.00234 (bf16) and 0.00029 (fp16) where fp32 dg and du would leave 0.00166
// and 0.00021.  Each as the sum of two values of the type would avoid it for 20 instead of 12 T D F operations.  dbg and dbu need no
// operands: they are sums of the fp32 values, made over a tile's rows as the tile is and then added up.
#include <algorithm>

#include "na_block.cuh"
#include "na_device.cuh"
#include "na_glu.h"

namespace na {
using namespace dev;
using namespace glu;

namespace {

na_status glu_sizes(long long rows, int D, int F, na_dtype dtype) {
    if (rows < 1 || D < 1 || F < 1 || !known_dtype(dtype)) return NA_ERR_INVALID_ARG;
    if (D > kGluMaxWidth || F > kGluMaxWidth || rows > kGluMaxRows || rows > (1LL << 40) / D || rows > (1LL << 40) / F) return NA_ERR_UNSUPPORTED;
    return NA_OK;
}

// Rows of D 2-byte elements to rows of W, a multiple of 8, with zeros past D, or back.  A thread has a 16-byte chunk of the W.
template <bool WIDEN>
__global__ void __launch_bounds__(256) glu_copy_kernel(const GluCopies c) {
    const int i = blockIdx.y, per = c.W / 8;
    const long long chunks = c.rows[i] * per;
    for (long long k = blockIdx.x * 256LL + threadIdx.x; k < chunks; k += gridDim.x * 256LL) {
        const long long row = k / per;
        const int col = static_cast<int>(k - row * per) * 8;
        if constexpr (WIDEN) {
            const uint16_t* from = static_cast<const uint16_t*>(c.from[i]) + row * c.D;
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int a = col + 2 * e;
                w[e] = (a < c.D ? from[a] : 0u) | (a + 1 < c.D ? static_cast<uint32_t>(from[a + 1]) << 16 : 0u);
            }
            static_cast<uint4*>(c.to[i])[k] = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
            const uint4 v = static_cast<const uint4*>(c.from[i])[k];
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
            uint16_t* to = static_cast<uint16_t*>(c.to[i]) + row * c.D;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (col + e < c.D) to[col + e] = static_cast<uint16_t>(w[e / 2] >> (16 * (e & 1)));
        }
    }
}

na_status launch_copies(const GluCopies& c, bool widen, cudaStream_t s) {
    const long long most = std::max(c.rows[0], std::max(c.rows[1], c.rows[2])) * (c.W / 8);
    if (most == 0) return NA_OK;
    const dim3 grid(static_cast<unsigned>(std::min((most + 255) / 256, 8LL * kSms)), 3);
    if (widen) glu_copy_kernel<true><<<grid, 256, 0, s>>>(c);
    else glu_copy_kernel<false><<<grid, 256, 0, s>>>(c);
    return launch_result();
}

bool known_act(na_glu_act a) { return a >= NA_ACT_SILU && a <= NA_ACT_SIGMOID; }

// A product on tensor cores: its tensor maps, boxes of 64 (or 32) elements by as many rows as one copy brings (na_glu_tc.cuh).
// n: its plan, of kBoth the tokens'; w: of kBoth the weights'.
na_status launch_tensor(const GluParams& p, Product which, const GluTiles& n, na_dtype dtype, cudaStream_t s, const GluTiles* w = nullptr) {
    GluTcParams q{};
    const bool pair = which == kForward || which == kSlopes;
    const uint64_t D = p.D, F = p.F, T = p.T, pitch = 2 * static_cast<uint64_t>(p.pitch);
    na_status st = device_status_word(&q.err);
    auto map = [&](CUtensorMap& m, const void* base, uint64_t inner, uint64_t rows, uint64_t row_bytes, uint32_t box, uint32_t wide = 64) {
        const uint64_t sizes[2] = {inner, rows};
        if (st == NA_OK) st = encode_box(&m, base, dtype, sizes, row_bytes, wide, box);
    };
    q.wide = p.F % 8 == 0;
    if (pair) {
        const uint32_t b_rows = n.pairs ? 128 : 64;
        map(q.a[0], p.x, D, T, 2 * D, n.few ? n.few : 128);
        map(q.b[0], p.wg, D, F, 2 * D, b_rows);
        map(q.b[1], p.wu, D, F, 2 * D, b_rows);
        if (!n.few) {   // results and dh: boxes of 32 by 32
            map(q.b[2], p.wg, D, F, 2 * D, n.last_nf);
            map(q.b[3], p.wu, D, F, 2 * D, n.last_nf);
            if (which == kSlopes) {
                if (q.wide) map(q.in, p.dh, F, T, 2 * F, 32, 32);
                else map(q.in, p.dg, F, T, pitch, 32, 32);
                map(q.out[0], p.dg, F, T, pitch, 32, 32);
                map(q.out[1], p.du, F, T, pitch, 32, 32);
            } else if (q.wide) {
                map(q.out[0], p.h, F, T, 2 * F, 32, 32);
            }
        }
        q.rows = n.rows;
        q.cols = n.cols;
        q.steps = n.steps;
        q.run = n.run;
        q.splits = n.splits;
        q.last_nf = n.last_nf;
        q.span = n.span;
        q.groups = n.groups;
    } else {
        map(q.a[0], p.dg, F, T, pitch, 64);
        map(q.a[1], p.du, F, T, pitch, 64);
        if (which != kWeights) {
            map(q.b[0], p.wg, D, F, 2 * D, 64);
            map(q.b[1], p.wu, D, F, 2 * D, 64);
        }
        if (which != kTokens) map(q.b[2], p.x, D, T, 2 * D, 64);
        const GluTiles& weights = w ? *w : n;
        q.job[0] = {n.rows, n.cols, n.splits, n.ways, n.run, n.steps};
        q.job[1] = {weights.rows, weights.cols, weights.splits, weights.ways, weights.run, weights.steps};
        q.token_workers = n.workers;
    }
    if (st != NA_OK) return st;
    q.bg = p.bg;
    q.bu = p.bu;
    q.dh = p.dh;
    q.h = p.h;
    q.dg = p.dg;
    q.du = p.du;
    q.dx = p.dx;
    q.dwg = p.dwg;
    q.dwu = p.dwu;
    q.partial = p.partial;
    q.sums = p.sums;
    q.sum_pitch = p.sum_pitch;
    q.pitch = p.pitch;
    q.T = static_cast<int>(p.T);
    q.D = p.D;
    q.F = p.F;
    q.act = p.act;
    q.wait_ns = wait_limit_ns();
    q.withhold = wait_withhold();
    const bool f16 = dtype == NA_FP16;
    const int blocks = n.pairs ? 2 : 1;
    switch (which) {
        case kForward:
            if (n.few) return f16 ? launch_few<kForward, __half>(q, n.few, s) : launch_few<kForward, __nv_bfloat16>(q, n.few, s);
            return f16 ? launch_tiles<kForward, __half>(q, blocks, s) : launch_tiles<kForward, __nv_bfloat16>(q, blocks, s);
        case kSlopes:
            if (n.few) return f16 ? launch_few<kSlopes, __half>(q, n.few, s) : launch_few<kSlopes, __nv_bfloat16>(q, n.few, s);
            return f16 ? launch_tiles<kSlopes, __half>(q, blocks, s) : launch_tiles<kSlopes, __nv_bfloat16>(q, blocks, s);
        case kTokens: return f16 ? launch_tiles<kTokens, __half>(q, blocks, s) : launch_tiles<kTokens, __nv_bfloat16>(q, blocks, s);
        case kWeights: return f16 ? launch_tiles<kWeights, __half>(q, blocks, s) : launch_tiles<kWeights, __nv_bfloat16>(q, blocks, s);
        default: return f16 ? launch_tiles<kBoth, __half>(q, 2, s) : launch_tiles<kBoth, __nv_bfloat16>(q, 2, s);
    }
}

na_status fma_product(GluParams p, Product which, const FmaTile& tile, na_dtype dtype, cudaStream_t s) {
    p.splits = tile.splits;
    p.run = tile.run;
    if (dtype == NA_BF16) return launch_fma<__nv_bfloat16>(p, which, tile, s);
    if (dtype == NA_FP16) return launch_fma<__half>(p, which, tile, s);
    return launch_fma<float>(p, which, tile, s);
}

na_status sum_runs(const float* partial, int runs, long long n, long long cut, void* out0, void* out1, na_dtype dtype, cudaStream_t s) {
    if (dtype == NA_BF16) return launch_sum<__nv_bfloat16>(partial, runs, n, cut, out0, out1, s);
    if (dtype == NA_FP16) return launch_sum<__half>(partial, runs, n, cut, out0, out1, s);
    return launch_sum<float>(partial, runs, n, cut, out0, out1, s);
}

// Sums of the tiles' rows of sums over runs of them: partial[run][2][F].  A lane takes a chunk of 16 bytes of every eighth row.
__global__ void __launch_bounds__(256) glu_column_kernel(const float* tiles, long long rows, int F, int pitch, long long run, float* partial) {
    after_previous();
    next_may_start();
    __shared__ __align__(16) float sums[8][128];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int first_col = blockIdx.x * 128, c = first_col + lane * 4;
    const float* from = tiles + static_cast<long long>(blockIdx.z) * pitch + c;
    const long long first = blockIdx.y * run, end = min(first + run, rows);
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (c < pitch)
#pragma unroll 4
        for (long long r = first + warp; r < end; r += 8) {
            const float4 f = *reinterpret_cast<const float4*>(from + r * 2 * pitch);
            s.x += f.x, s.y += f.y, s.z += f.z, s.w += f.w;
        }
    *reinterpret_cast<float4*>(&sums[warp][lane * 4]) = s;
    __syncthreads();
    const int i = threadIdx.x;
    if (i >= 128 || first_col + i >= F) return;
    float t = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) t += sums[w][i];
    partial[(blockIdx.y * 2LL + blockIdx.z) * F + first_col + i] = t;
}

// dbg and dbu from the sums that the slopes' kernel has made.
na_status column_sums(const GluParams& p, const GluPlan& n, void* dbg, void* dbu, na_dtype dtype, cudaStream_t s) {
    float* runs = p.sums + n.sums / sizeof(float);
    const na_status st = launch_after(glu_column_kernel, dim3(up(p.F, 128), n.runs, 2), 256, s, p.sums, n.sum_rows, p.F, n.sum_pitch, n.column_run, runs);
    return st == NA_OK ? sum_runs(runs, n.runs, 2LL * p.F, p.F, dbg, dbu, dtype, s) : st;
}

}  // namespace
}  // namespace na

extern "C" {

na_status na_glu(const void* x, const void* wg, const void* wu, const void* bg, const void* bu, void* h, int64_t rows, int D,
                 int F, na_glu_act act, na_dtype dtype, void* stream) {
    using namespace na;
    na_status st = glu_sizes(rows, D, F, dtype);
    if (st != NA_OK) return st;
    if (!x || !wg || !wu || !h || !known_act(act)) return NA_ERR_INVALID_ARG;
    for (const void* q : {x, wg, wu, bg, bu, static_cast<const void*>(h)})
        if (!ptr_aligned(q, 16)) return NA_ERR_ALIGNMENT;
    const long long es = elem_bytes(dtype), wide = es * F * D;
    if (!output_clear({h, rows * F * es}, {}, {{x, rows * D * es}, {wg, wide}, {wu, wide}, {bg, F * es}, {bu, F * es}})) return NA_ERR_INVALID_ARG;
    GluParams p{};
    p.x = x;
    p.wg = wg;
    p.wu = wu;
    p.bg = bg;
    p.bu = bu;
    p.h = h;
    p.T = rows;
    p.D = D;
    p.F = F;
    p.act = act;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int width = tensor_width(rows, D, F, dtype);
    if (width == 0) return fma_product(p, kForward, plan_fma(kForward, rows, D, F), dtype, s);
    if (width == D) return launch_tensor(p, kForward, plan_tiles(kForward, rows, D, F), dtype, s);
    const size_t tokens = up256(static_cast<size_t>(rows) * width * es), weights = up256(static_cast<size_t>(F) * width * es);
    void* ws = nullptr;
    if (!taken(cudaMallocAsync(&ws, tokens + 2 * weights, s))) return NA_ERR_WORKSPACE;
    char* at = static_cast<char*>(ws);
    const GluCopies copies{{x, wg, wu}, {at, at + tokens, at + tokens + weights}, {rows, F, F}, D, width};
    st = launch_copies(copies, true, s);
    p.x = copies.to[0];
    p.wg = copies.to[1];
    p.wu = copies.to[2];
    p.D = width;
    if (st == NA_OK) st = launch_tensor(p, kForward, plan_tiles(kForward, rows, width, F), dtype, s);
    if (cudaFreeAsync(ws, s) != cudaSuccess && st == NA_OK) st = NA_ERR_CUDA;
    return st;
}

size_t na_glu_bwd_workspace_size(int64_t rows, int D, int F, na_dtype dtype) {
    using namespace na;
    if (glu_sizes(rows, D, F, dtype) != NA_OK) return 0;
    return glu_workspace(plan_glu(rows, D, F, dtype));
}

na_status na_glu_bwd(const void* dh, const void* x, const void* wg, const void* wu, const void* bg, const void* bu, void* dx,
                     void* dwg, void* dwu, void* dbg, void* dbu, int64_t rows, int D, int F, na_glu_act act, na_dtype dtype,
                     void* workspace, size_t workspace_bytes, void* stream) {
    using namespace na;
    na_status st = glu_sizes(rows, D, F, dtype);
    if (st != NA_OK) return st;
    if (!dh || !x || !wg || !wu || (dwg == nullptr) != (dwu == nullptr) || (dbg && !bg) || (dbu && !bu) || (!dx && !dwg && !dbg && !dbu) ||
        !known_act(act))
        return NA_ERR_INVALID_ARG;
    for (const void* q : {dh, x, wg, wu, bg, bu, static_cast<const void*>(dx), static_cast<const void*>(dwg), static_cast<const void*>(dwu),
                          static_cast<const void*>(dbg), static_cast<const void*>(dbu)})
        if (!ptr_aligned(q, 16)) return NA_ERR_ALIGNMENT;
    const long long es = elem_bytes(dtype), wide = es * F * D;
    const Span in[] = {{dh, rows * F * es}, {x, rows * D * es}, {wg, wide}, {wu, wide}, {bg, F * es}, {bu, F * es}};
    const Span out[] = {{dx, rows * D * es}, {dwg, wide}, {dwu, wide}, {dbg, F * es}, {dbu, F * es}};
    for (int i = 0; i < 5; ++i) {
        for (const Span& q : in)
            if (spans_overlap(out[i], q)) return NA_ERR_INVALID_ARG;
        for (int k = 0; k < i; ++k)
            if (spans_overlap(out[i], out[k])) return NA_ERR_INVALID_ARG;
    }
    const GluPlan n = plan_glu(rows, D, F, dtype);
    const size_t need = glu_workspace(n);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    void* ws = workspace;
    if (ws) {
        if (workspace_bytes < need) return NA_ERR_WORKSPACE;
        if (!ptr_aligned(ws, 16)) return NA_ERR_ALIGNMENT;
        const Span sws{ws, static_cast<long long>(need)};
        for (const Span& q : in)
            if (spans_overlap(sws, q)) return NA_ERR_INVALID_ARG;
        for (const Span& q : out)
            if (spans_overlap(sws, q)) return NA_ERR_INVALID_ARG;
    } else if (!taken(cudaMallocAsync(&ws, need, s))) {
        return NA_ERR_WORKSPACE;
    }
    GluParams p{};
    p.dh = dh;
    p.x = x;
    p.wg = wg;
    p.wu = wu;
    p.bg = bg;
    p.bu = bu;
    p.dx = dx;
    p.dwg = dwg;
    p.dwu = dwu;
    p.dg = ws;
    p.du = static_cast<char*>(ws) + n.array;
    p.partial = reinterpret_cast<float*>(static_cast<char*>(ws) + 2 * n.array);
    if (dbg || dbu) p.sums = p.partial;   // added up before anything else is put there
    p.sum_pitch = n.sum_pitch;
    p.T = rows;
    p.pitch = n.pitch;
    p.D = n.width;
    p.F = F;
    p.act = act;
    const bool copied = n.width != D;
    if (copied) {   // the products' own tensors, in whole chunks
        char* at = static_cast<char*>(ws) + 2 * n.array + n.partial;
        const GluCopies in_copies{{x, wg, wu}, {at, at + n.tokens_copy, at + n.tokens_copy + n.weights_copy}, {rows, F, F}, D, n.width};
        st = launch_copies(in_copies, true, s);
        p.x = in_copies.to[0];
        p.wg = in_copies.to[1];
        p.wu = in_copies.to[2];
        at += n.tokens_copy + 2 * n.weights_copy;
        if (dx) p.dx = at;
        if (dwg) {
            p.dwg = at + n.tokens_copy;
            p.dwu = at + n.tokens_copy + n.weights_copy;
        }
    }
    const long long size = static_cast<long long>(F) * n.width, tokens_size = rows * n.width;
    if (n.tensor) {
        // rows of dh that are not whole chunks go to dg's place first
        if (st == NA_OK && !n.slopes.few && F % 8 != 0) st = launch_copies({{dh, nullptr, nullptr}, {p.dg, nullptr, nullptr}, {rows, 0, 0}, F, static_cast<int>(n.pitch)}, true, s);
        if (st == NA_OK) st = launch_tensor(p, kSlopes, n.slopes, dtype, s);
    } else {
        st = fma_product(p, kSlopes, n.slopes_fma, dtype, s);
    }
    if (st == NA_OK && p.sums) st = column_sums(p, n, dbg, dbu, dtype, s);
    const bool both = dx && dwg && n.tensor && n.tokens.workers;
    if (st == NA_OK && both) st = launch_tensor(p, kBoth, n.tokens, dtype, s, &n.weights);
    if (st == NA_OK && dx) {
        if (!both) st = n.tensor ? launch_tensor(p, kTokens, n.tokens, dtype, s) : fma_product(p, kTokens, n.tokens_fma, dtype, s);
        const int splits = n.tensor ? static_cast<int>(n.tokens.splits) : n.tokens_fma.splits;
        if (st == NA_OK && splits > 1)
            st = sum_runs(p.partial, splits, tokens_size, tokens_size, p.dx, nullptr, dtype, s);
    }
    if (st == NA_OK && dwg) {
        if (!both) st = n.tensor ? launch_tensor(p, kWeights, n.weights, dtype, s) : fma_product(p, kWeights, n.weights_fma, dtype, s);
        const int splits = n.tensor ? static_cast<int>(n.weights.splits) : n.weights_fma.splits;
        if (st == NA_OK && splits > 1) st = sum_runs(p.partial, splits, 2 * size, size, p.dwg, p.dwu, dtype, s);
    }
    if (st == NA_OK && copied) st = launch_copies({{p.dx, p.dwg, p.dwu}, {dx, dwg, dwu}, {dx ? rows : 0, dwg ? F : 0, dwg ? F : 0}, D, n.width}, false, s);
    if (!workspace && cudaFreeAsync(ws, s) != cudaSuccess && st == NA_OK) st = NA_ERR_CUDA;
    return st;
}

}  // extern "C"
