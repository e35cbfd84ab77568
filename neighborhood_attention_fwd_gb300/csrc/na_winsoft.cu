// na_winsoft.cu -- dropout of a tensor, and the entry points of the window softmax with dropout and of the
// differential window softmax (kernels in na_win_impl.cuh).
#include <algorithm>
#include <cmath>

#include "na_block.cuh"
#include "na_win.h"

namespace na {
namespace {

constexpr int kThreads = 256;       // of the per-head sums
constexpr int kDropThreads = 128;   // of the dropout (256: 2^28 elements of bf16 166 us instead of 156)

// Sums of a [n, heads] matrix over n, per_block rows of it to each block: out[block][heads].
__global__ void __launch_bounds__(kThreads) head_sum_kernel(const float* in, long long n, int heads, long long per_block,
                                                              float* out) {
    __shared__ float part[kThreads];
    const long long r0 = blockIdx.x * per_block, r1 = min(r0 + per_block, n);
    float* to = out + static_cast<long long>(blockIdx.x) * heads;
    if (heads > kThreads) {
        for (int h = threadIdx.x; h < heads; h += kThreads) {
            float s = 0.f;
            for (long long r = r0; r < r1; ++r) s += in[r * heads + h];
            to[h] = s;
        }
        return;
    }
    const int lanes = kThreads / heads, use = lanes * heads;
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

// Dropout of a tensor: y = gain x where the generator keeps the element, else 0 (y may be x).  A thread takes kOct octets of
// a block's run: it loads them all, works out the generator's constants meanwhile, then draws.  Memory-bound: 2^28 elements
// of bf16 in 157 us (101% of the copy rate), of fp32 in 325 us (97%).
template <typename T>
constexpr int kOct = sizeof(T) == 4 ? 2 : 4;

template <typename T, typename Bits>
__device__ __forceinline__ void dropout_run(const T* x, T* y, long long n, const Dropout& d, long long o0, Bits bits) {
    using E = Elem<T>;
    constexpr int C = sizeof(T) == 4 ? 2 : 1, V = E::EPC;
    uint4 r[kOct<T>][C];
#pragma unroll
    for (int j = 0; j < kOct<T>; ++j) {
        const long long o = o0 + j * kDropThreads;
        if (o * 8 + 8 <= n)
#pragma unroll
            for (int c = 0; c < C; ++c) r[j][c] = ld_stream(x + o * 8 + c * V);
    }
    const auto draw = bits();
#pragma unroll
    for (int j = 0; j < kOct<T>; ++j) {
        const long long o = o0 + j * kDropThreads;
        if (o * 8 + 8 <= n) {
#pragma unroll
            for (int c = 0; c < C; ++c) {
                float f[V];
                E::unpack(r[j][c], f);
#pragma unroll
                for (int e = 0; e < V; ++e) f[e] *= d.gain;
                r[j][c] = E::pack(f);
            }
            if (d.state) {
                if constexpr (C == 2) drop_words(r[j][0], r[j][1], draw(o), d.steps);
                else drop_words(r[j][0], draw(o), d.steps);
            }
#pragma unroll
            for (int c = 0; c < C; ++c) st_stream(y + o * 8 + c * V, r[j][c]);
        } else if (o * 8 < n) {   // the tensor ends inside this octet
            uint4 m = make_uint4(~0u, ~0u, ~0u, ~0u);
            if (d.state) drop_words(m, draw(o), d.steps);
            for (int e = 0; o * 8 + e < n; ++e) {
                const float v = E::get(x[o * 8 + e]) * d.gain;
                y[o * 8 + e] = E::put(keep_of(m, e) ? v : 0.f);
            }
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(kDropThreads) dropout_kernel(const T* x, T* y, long long n, Dropout d) {
    const long long first = static_cast<long long>(blockIdx.x) * (kDropThreads * kOct<T>);
    const RngState rng = d.state ? rng_load(d.state) : RngState{};
    if (first + kDropThreads * kOct<T> <= (1LL << 32)) {
        dropout_run(x, y, n, d, first + threadIdx.x, [&] {
            const RngPlan plan = rng_plan(rng);
            return [plan](long long o) { return rng_block(plan, static_cast<uint32_t>(o)); };
        });
    } else {
        dropout_run(x, y, n, d, first + threadIdx.x, [&] {
            return [rng](long long o) { return rng_block(rng, static_cast<unsigned long long>(o)); };
        });
    }
}

// ---------------------------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------------------------

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
    p.wait_ns = wait_limit_ns();
    p.withhold = wait_withhold();
    return NA_OK;
}

na_status launch_win(WinParams& p, na_dtype dtype, bool diff, bool bwd, cudaStream_t s) {
    using Launch = na_status (*)(WinParams&, cudaStream_t);
    static constexpr Launch kForms[2][2][3] = {
        {{launch_soft_fwd_bf16, launch_soft_fwd_f32, launch_soft_fwd_f16}, {launch_soft_bwd_bf16, launch_soft_bwd_f32, launch_soft_bwd_f16}},
        {{launch_diff_fwd_bf16, launch_diff_fwd_f32, launch_diff_fwd_f16}, {launch_diff_bwd_bf16, launch_diff_bwd_f32, launch_diff_bwd_f16}},
    };
    return kForms[diff][bwd][dtype](p, s);   // NA_BF16, NA_FP32, NA_FP16
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
// Tokens of a block: at least sixteen values for every thread, so that small grids take one block and one launch.
long long sum_tokens(long long tokens, int heads) {
    const long long share = (tokens + kSumBlocks - 1) / kSumBlocks, least = std::max(1, 16 * kThreads / heads);
    return std::max(share, least);
}

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
    const long long per = 8LL * kDropThreads * (dtype == NA_FP32 ? kOct<float> : kOct<__half>), blocks = (n + per - 1) / per;
    if (blocks > 0x7fffffffLL) return NA_ERR_UNSUPPORTED;
    const unsigned nb = static_cast<unsigned>(blocks);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == NA_BF16)
        dropout_kernel<<<nb, kDropThreads, 0, s>>>(static_cast<const __nv_bfloat16*>(x), static_cast<__nv_bfloat16*>(y), n, d);
    else if (dtype == NA_FP16)
        dropout_kernel<<<nb, kDropThreads, 0, s>>>(static_cast<const __half*>(x), static_cast<__half*>(y), n, d);
    else
        dropout_kernel<<<nb, kDropThreads, 0, s>>>(static_cast<const float*>(x), static_cast<float*>(y), n, d);
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
    return launch_win(w, dtype, false, false, static_cast<cudaStream_t>(stream));
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
    return launch_win(w, dtype, false, true, static_cast<cudaStream_t>(stream));
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
    return launch_win(w, dtype, true, false, static_cast<cudaStream_t>(stream));
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
        if (!taken(cudaMallocAsync(&ws, diff_workspace(w), s))) return NA_ERR_WORKSPACE;
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
    st = launch_win(w, dtype, true, true, s);
    if (st == NA_OK && !lam_per_row) {
        // the rows' values [tokens, heads] summed over the tokens, in two steps of a fixed order
        const long long tokens = w.rows / heads, per = sum_tokens(tokens, heads);
        const int blocks = static_cast<int>((tokens + per - 1) / per);
        float* partial = w.dlam + (w.rows + 63) / 64 * 64;
        head_sum_kernel<<<blocks, kThreads, 0, s>>>(w.dlam, tokens, heads, per, blocks == 1 ? dlam : partial);
        if (blocks > 1) head_sum_kernel<<<1, kThreads, 0, s>>>(partial, blocks, heads, blocks, dlam);
        st = launch_result();
    }
    if (owned && cudaFreeAsync(ws, s) != cudaSuccess && st == NA_OK) st = NA_ERR_CUDA;
    return st;
}

}  // extern "C"
