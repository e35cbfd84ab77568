// na_rope.cu -- rotary positions of queries and keys on a grid, forward and backward.
//
// Every spatial axis a owns a block of rot[a] channels of the head (blocks follow one another from
// channel 0; channels behind the last block pass through).  Pair i of the block at position x along the
// axis turns by theta = (origin[a] + x) f_{a,i}:  (u, v) -> amp (u cos theta - v sin theta, u sin theta +
// v cos theta); the backward pass turns by -theta.  Pairs are (i, i + rot/2) or (2 i, 2 i + 1) of the block.
//
// Angles.  A far position times a frequency loses the angle in fp32 (at position 10^6 the fp32 spacing of
// the product is 0.06 rad).  Frequencies are held as turns per position in 64-bit fixed point; position times
// frequency modulo 2^64 is then the exact phase of that frequency, whatever the position, and its top 32
// bits go to sincospif.  The host splits f / 2 pi into two doubles, so the fixed-point value is
// good to 2^-64 turns.
//
// What bounds it.  Every element is read and written once: memory.  A block takes consecutive tokens, computes the
// tokens' angles once into shared memory (all heads of q and k share them) while its first loads are in
// flight, and then streams the tokens' rows in 16-byte chunks.  Measured: bf16 q and k of 1024x1024 x 8 heads of 32, 330 us,
// 6.5 TB/s (96% of the copy rate); fp16, 131071 tokens of 16 + 4 heads of 128, half of them turned, 197 us (100%).
#include <algorithm>
#include <cmath>

#include "na_block.cuh"

namespace na {
namespace {

constexpr int kRopeThreads = 128;   // 256: queries and keys of 1024x1024 x 8 heads of 32 in 340 us instead of 332
constexpr int kMaxPairs = 64;   // D / 2 at D = 128
constexpr int kMaxTokens = 64;  // tokens of a block
constexpr int kRopeBytes = 32 * 1024;   // rows of a block, about

struct RopeParams {
    const void* x[2];          // q, k (k null: heads_k = 0)
    void* y[2];
    long long tokens;
    uint32_t upt[2];           // units per token of q and k (all heads)
    FastDiv fd_upt[2];
    int L[3];
    FastDiv fd_L[3], fd_np;
    unsigned long long origin[3];
    unsigned long long turns[kMaxPairs];   // turns per position, 64-bit fixed point
    int pair_end[3];           // pairs of axes 0 .. a
    int np;                    // pairs in all
    int row;                   // entries of a token's row of angles
    int cph;                   // 16-byte chunks per head row
    int lu;                    // log2 of the units per head row
    int tt;                    // tokens per block
    float amp, sgn;            // amplitude; -1 for the backward rotation
    // half layout, whole chunks: unit u holds chunks a and b (channels c and c + rot/2 of a block), pairs from p0
    // (0xff: passes through)
    uint8_t ua[16], ub[16], up[16];
    // half layout, any even rot: partner and pair of every channel (pair 0xff: passes through)
    uint8_t partner[128], pair[128];
};

// The grid positions of the block's tokens, one token per thread (a block has at most kMaxTokens).
__device__ __forceinline__ void fill_positions(const RopeParams& p, int (*pos)[kMaxTokens], long long tok0, int tt) {
    if (static_cast<int>(threadIdx.x) >= tt) return;
    const long long tok = tok0 + threadIdx.x;
    if (p.tokens < (1LL << 32)) {
        const uint32_t r = static_cast<uint32_t>(tok), q2 = fdiv(r, p.fd_L[2]), q1 = fdiv(q2, p.fd_L[1]), q0 = fdiv(q1, p.fd_L[0]);
        pos[2][threadIdx.x] = static_cast<int>(r - q2 * p.L[2]);
        pos[1][threadIdx.x] = static_cast<int>(q2 - q1 * p.L[1]);
        pos[0][threadIdx.x] = static_cast<int>(q1 - q0 * p.L[0]);
    } else {
        const long long q2 = tok / p.L[2], q1 = q2 / p.L[1];
        pos[2][threadIdx.x] = static_cast<int>(tok - q2 * p.L[2]);
        pos[1][threadIdx.x] = static_cast<int>(q2 - q1 * p.L[1]);
        pos[0][threadIdx.x] = static_cast<int>(q1 % p.L[0]);
    }
}

// The frequencies in shared memory: lanes that read different entries of a kernel parameter do so one by one.
__device__ __forceinline__ void fill_turns(const RopeParams& p, unsigned long long* turns) {
    if (static_cast<int>(threadIdx.x) < p.np) turns[threadIdx.x] = p.turns[threadIdx.x];
}

__device__ __forceinline__ int axis_of(const RopeParams& p, int pair) {
    return pair < p.pair_end[0] ? 0 : (pair < p.pair_end[1] ? 1 : 2);
}

// cos and sin, times the amplitude, of a pair at grid position x of its axis.
__device__ __forceinline__ float2 angle_of(const RopeParams& p, int axis, unsigned long long turns, int x) {
    const unsigned long long o = axis == 0 ? p.origin[0] : (axis == 1 ? p.origin[1] : p.origin[2]);
    const unsigned long long phase = (o + static_cast<unsigned long long>(x)) * turns;
    float s, c;
    sincospif(static_cast<float>(static_cast<int32_t>(phase >> 32)) * 4.656612873077393e-10f, &s, &c);   // 2^-31 half turns
    return make_float2(c * p.amp, s * p.amp * p.sgn);
}

// Where a pair's angle lies in its token's row of the table: units of G pairs, two entries apart where a unit is longer
// than 16 bytes, so that the lanes of a head row, a unit each, read different banks.
template <int G>
__host__ __device__ constexpr int angle_at(int pair) { return pair + (G >= 4 ? pair / G * 2 : 0); }

// The angles of every pair of the block's tokens.
template <int G>
__device__ __forceinline__ void fill_angles(const RopeParams& p, float2* tab, const unsigned long long* turns,
                                            const int (*pos)[kMaxTokens], int tt) {
    for (uint32_t i = threadIdx.x; i < static_cast<uint32_t>(tt * p.np); i += kRopeThreads) {
        const uint32_t t = fdiv(i, p.fd_np);
        const int pair = static_cast<int>(i - t * static_cast<uint32_t>(p.np)), a = axis_of(p, pair);
        tab[t * p.row + angle_at<G>(pair)] = angle_of(p, a, turns[pair], pos[a][t]);
    }
}

// Units of whole chunks: one chunk of pairs (2 i, 2 i + 1), or two chunks of pairs (i, i + rot/2).  A
// thread keeps four or eight units in flight; the first ones are loaded before the angles are computed.
template <typename T, bool INTER>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams p) {
    using E = Elem<T>;
    constexpr int V = E::EPC, NC = INTER ? 1 : 2, U = INTER ? 8 : 4, NP = INTER ? V / 2 : V;
    extern __shared__ __align__(16) float2 tab[];
    __shared__ int pos[3][kMaxTokens];
    __shared__ unsigned long long turns[kMaxPairs];
    const long long tok0 = static_cast<long long>(blockIdx.x) * p.tt;
    const int tt = static_cast<int>(min(static_cast<long long>(p.tt), p.tokens - tok0));
    const uint32_t nq = static_cast<uint32_t>(tt) * p.upt[0], n = nq + static_cast<uint32_t>(tt) * p.upt[1];
    const uint32_t u = threadIdx.x & ((1u << p.lu) - 1u);   // a block's threads are whole head rows
    const int ca = INTER ? static_cast<int>(u) : p.ua[u], cb = INTER ? 0 : p.ub[u];
    const int p0 = INTER ? static_cast<int>(u) * NP : (p.up[u] == 0xff ? p.np : p.up[u]);
    const uint4* xs[2];
    uint4* ys[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const long long at = tok0 * p.upt[i] * NC;
        xs[i] = static_cast<const uint4*>(p.x[i]) + at;
        ys[i] = static_cast<uint4*>(p.y[i]) + at;
    }
    uint4 r[U][NC];
    auto load = [&](uint32_t base) {
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const uint32_t i = base + j * kRopeThreads;
            if (i < n) {
                const int w = i >= nq;
                const uint4* x = xs[w] + static_cast<long long>((w ? i - nq : i) >> p.lu) * p.cph;
                r[j][0] = ld_stream(x + ca);
                if (!INTER) r[j][NC - 1] = ld_stream(x + cb);
            }
        }
    };
    load(threadIdx.x);
    fill_positions(p, pos, tok0, tt);
    fill_turns(p, turns);
    __syncthreads();
    fill_angles<NP>(p, tab, turns, pos, tt);
    __syncthreads();
    for (uint32_t base = threadIdx.x;;) {
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const uint32_t i = base + j * kRopeThreads;
            if (i < n) {
                const int w = i >= nq;
                const uint32_t k = w ? i - nq : i;
                uint4* y = ys[w] + static_cast<long long>(k >> p.lu) * p.cph;
                if (p0 < p.np) {
                    const float2* cs = tab + fdiv(k, p.fd_upt[w]) * p.row + angle_at<NP>(p0);
                    float f[NC][V];
                    E::unpack(r[j][0], f[0]);
                    if (!INTER) E::unpack(r[j][NC - 1], f[NC - 1]);
#pragma unroll
                    for (int e = 0; e < NP; ++e) {
                        if (!INTER || p0 + e < p.np) {
                            const float2 t = cs[e];
                            float& a = INTER ? f[0][2 * e] : f[0][e];
                            float& b = INTER ? f[0][2 * e + 1] : f[NC - 1][e];
                            const float va = a, vb = b;
                            a = va * t.x - vb * t.y;
                            b = va * t.y + vb * t.x;
                        }
                    }
                    const uint4 turned = E::pack(f[0]);
                    if (INTER && p0 + NP > p.np) {   // a chunk turned in part keeps the other pairs' bits
                        constexpr int WP = 4 / NP;   // words per pair
                        uint32_t* to = reinterpret_cast<uint32_t*>(&r[j][0]);
                        const uint32_t* from = reinterpret_cast<const uint32_t*>(&turned);
#pragma unroll
                        for (int i2 = 0; i2 < 4; ++i2)
                            if (p0 + i2 / WP < p.np) to[i2] = from[i2];
                    } else {
                        r[j][0] = turned;
                    }
                    if (!INTER) r[j][NC - 1] = E::pack(f[NC - 1]);
                }
                st_stream(y + ca, r[j][0]);
                if (!INTER) st_stream(y + cb, r[j][NC - 1]);
            }
        }
        base += U * kRopeThreads;
        if (base >= n) break;
        load(base);
    }
}

// Half layout with a block whose halves are not whole chunks: a chunk's partners lie anywhere in its head's row, so the
// rows pass through shared memory, kSplit chunks (whole head rows) per thread at a time, the next ones on
// their way meanwhile.  The angles are kept per channel, the sine with the sign it takes there:
// y = x cos + partner sin.
// PAIRED: 2-byte elements whose blocks' halves are even, so that partners lie in whole words (bf16, 8 heads of 64,
// 20x20x24 channels: 71% of the copy rate; 20x22x22, whose partners are gathered one by one: 59%).
constexpr int kSplit = 4;
template <typename T, bool PAIRED>
__global__ void __launch_bounds__(kRopeThreads) rope_split_kernel(const __grid_constant__ RopeParams p) {
    using E = Elem<T>;
    constexpr int V = E::EPC;
    extern __shared__ __align__(16) float2 tab[];   // [token][pair of elements of the chunk][chunk][2]: lanes read one after another
    __shared__ uint4 rows[kSplit * kRopeThreads];
    __shared__ int pos[3][kMaxTokens];
    __shared__ unsigned long long turns[kMaxPairs];
    __shared__ int where[2][kMaxPairs];   // a pair's two channels, as places in a token's row of the table
    const long long tok0 = static_cast<long long>(blockIdx.x) * p.tt;
    const int tt = static_cast<int>(min(static_cast<long long>(p.tt), p.tokens - tok0));
    const int D = p.cph * V, c = threadIdx.x & (p.cph - 1);
    const uint32_t nq = static_cast<uint32_t>(tt) * p.upt[0], n = nq + static_cast<uint32_t>(tt) * p.upt[1];
    const uint4* xs[2] = {static_cast<const uint4*>(p.x[0]) + tok0 * p.upt[0], static_cast<const uint4*>(p.x[1]) + tok0 * p.upt[1]};
    uint4* ys[2] = {static_cast<uint4*>(p.y[0]) + tok0 * p.upt[0], static_cast<uint4*>(p.y[1]) + tok0 * p.upt[1]};
    uint4 r[kSplit];
    auto load = [&](uint32_t base) {
#pragma unroll
        for (int j = 0; j < kSplit; ++j) {
            const uint32_t i = base + j * kRopeThreads;
            if (i < n) r[j] = i < nq ? ld_stream(xs[0] + i) : ld_stream(xs[1] + (i - nq));
        }
    };
    load(threadIdx.x);
    fill_positions(p, pos, tok0, tt);
    fill_turns(p, turns);
    auto place = [&](int ch) { return (ch % V / 2 * p.cph + ch / V) * 2 + ch % 2; };
    if (static_cast<int>(threadIdx.x) < D) {
        const int ch = threadIdx.x, pair = p.pair[ch];
        if (pair != 0xff) where[p.partner[ch] < ch][pair] = place(ch);
    }
    // of the thread's channels, which are the same in every turn: partners, and the bits of those that turn
    int partner[V];
    uint32_t keep[4] = {0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < V; ++e) {
        const bool turned = p.pair[c * V + e] != 0xff;
        partner[e] = turned ? p.partner[c * V + e] : c * V + e;
        if (turned) keep[e * static_cast<int>(sizeof(T)) / 4] |= sizeof(T) == 4 ? ~0u : 0xffffu << (16 * (e & 1));
    }
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < static_cast<uint32_t>(tt * p.np); i += kRopeThreads) {
        const uint32_t t = fdiv(i, p.fd_np);
        const int pair = static_cast<int>(i - t * static_cast<uint32_t>(p.np)), a = axis_of(p, pair);
        const float2 cs = angle_of(p, a, turns[pair], pos[a][t]);
        tab[t * p.row + where[0][pair]] = make_float2(cs.x, -cs.y);
        tab[t * p.row + where[1][pair]] = cs;
    }
    for (uint32_t base = threadIdx.x;;) {
#pragma unroll
        for (int j = 0; j < kSplit; ++j) rows[j * kRopeThreads + threadIdx.x] = r[j];
        __syncthreads();   // the rows, and in the first turn the angles
#pragma unroll
        for (int j = 0; j < kSplit; ++j) {
            const uint32_t i = base + j * kRopeThreads;
            if (i >= n) continue;
            const int w = i >= nq;
            const uint32_t k = w ? i - nq : i;
            const float2* cs = tab + fdiv(k, p.fd_upt[w]) * p.row + 2 * c;
            const T* head = reinterpret_cast<const T*>(rows + j * kRopeThreads + (threadIdx.x - c));
            float f[V];
            E::unpack(r[j], f);
#pragma unroll
            for (int e = 0; e < V; e += 2) {
                const float4 t = *reinterpret_cast<const float4*>(cs + e * p.cph);
                float o[2];
                if constexpr (PAIRED) {
                    E::two(*reinterpret_cast<const uint32_t*>(head + partner[e]), o[0], o[1]);
                } else {
                    o[0] = E::get(head[partner[e]]);
                    o[1] = E::get(head[partner[e + 1]]);
                }
                f[e] = fmaf(o[0], t.y, f[e] * t.x);
                f[e + 1] = fmaf(o[1], t.w, f[e + 1] * t.z);
            }
            const uint4 y = E::pack(f);
            // channels that do not turn keep their bits
            st_stream(ys[w] + k, make_uint4((y.x & keep[0]) | (r[j].x & ~keep[0]), (y.y & keep[1]) | (r[j].y & ~keep[1]),
                                            (y.z & keep[2]) | (r[j].z & ~keep[2]), (y.w & keep[3]) | (r[j].w & ~keep[3])));
        }
        base += kSplit * kRopeThreads;
        if (base - threadIdx.x >= n) break;
        load(base);
        __syncthreads();   // the rows have been read
    }
}

// f / (2 pi) modulo 1 in units of 2^-64: the quotient as a sum of two doubles (1 / 2 pi = kInvHi + kInvLo).
unsigned long long fixed_turns(double f) {
    constexpr double kInvHi = 0.15915494309189535, kInvLo = -9.839338337591243e-18, kUnit = 18446744073709551616.0;
    const double m = std::fabs(f), hi = m * kInvHi;
    const double lo = std::fma(m, kInvHi, -hi) + m * kInvLo;
    const double frac = (hi - std::floor(hi)) * kUnit;   // exact and below 2^64; lo is far smaller
    const unsigned long long t = static_cast<unsigned long long>(frac) +
                                 static_cast<unsigned long long>(static_cast<long long>(std::nearbyint(lo * kUnit)));
    return f < 0 ? 0ull - t : t;
}

template <typename T>
void launch_rope_t(const RopeParams& p, bool inter, bool split, bool even, unsigned blocks, size_t smem, cudaStream_t s) {
    if constexpr (sizeof(T) == 2)
        if (split && even) {
            rope_split_kernel<T, true><<<blocks, kRopeThreads, smem, s>>>(p);
            return;
        }
    if (split) rope_split_kernel<T, false><<<blocks, kRopeThreads, smem, s>>>(p);
    else if (inter) rope_kernel<T, true><<<blocks, kRopeThreads, smem, s>>>(p);
    else rope_kernel<T, false><<<blocks, kRopeThreads, smem, s>>>(p);
}

na_status rope(const void* q, const void* k, void* q_out, void* k_out, int B, int ndim, const int* spatial, int heads_q,
               int heads_k, int D, const int* rot, const double* freq, const int64_t* origin, float amp,
               na_rope_layout layout, na_dtype dtype, bool back, void* stream) {
    RopeParams p{};
    na_status st = grid_tokens(B, ndim, spatial, heads_q, D, p.L, p.tokens);
    if (st != NA_OK) return st;
    if (heads_k < 0 || !rot || !freq || !std::isfinite(amp) || !known_dtype(dtype)) return NA_ERR_INVALID_ARG;
    if (layout != NA_ROPE_HALF && layout != NA_ROPE_INTERLEAVED) return NA_ERR_INVALID_ARG;
    int L[3];
    long long tokens = 0;
    if (heads_k > 0 && (st = grid_tokens(B, ndim, spatial, heads_k, D, L, tokens)) != NA_OK) return st;
    int channels = 0;
    for (int a = 0; a < ndim; ++a) {
        if (rot[a] < 0 || rot[a] % 2 != 0 || rot[a] > D - channels) return NA_ERR_INVALID_ARG;
        channels += rot[a];
    }
    if (channels == 0) return NA_ERR_INVALID_ARG;
    if (D != 16 && D != 32 && D != 64 && D != 128) return NA_ERR_UNSUPPORTED;
    for (int i = 0; i < channels / 2; ++i)
        if (!std::isfinite(freq[i]) || std::fabs(freq[i]) > 1e6) return NA_ERR_INVALID_ARG;
    if (!q || !q_out || (heads_k > 0) != (k != nullptr) || (heads_k > 0) != (k_out != nullptr)) return NA_ERR_INVALID_ARG;
    for (const void* x : {q, k, static_cast<const void*>(q_out), static_cast<const void*>(k_out)})
        if (!ptr_aligned(x, 16)) return NA_ERR_ALIGNMENT;
    const int es = elem_bytes(dtype), V = 16 / es;
    const Span sq{q, p.tokens * heads_q * D * es}, sk{k, p.tokens * heads_k * D * es}, oq{q_out, sq.bytes}, ok{k_out, sk.bytes};
    if (!output_clear(oq, {sq}, {sk, ok}) || !output_clear(ok, {sk}, {sq})) return NA_ERR_INVALID_ARG;

    p.x[0] = q;
    p.x[1] = k;
    p.y[0] = q_out;
    p.y[1] = k_out;
    p.np = channels / 2;
    int done = 0;
    for (int a = 0; a < 3; ++a) {   // leading embedded axes own no channels
        if (a >= 3 - ndim) {
            done += rot[a - (3 - ndim)] / 2;
            p.origin[a] = origin ? static_cast<unsigned long long>(origin[a - (3 - ndim)]) : 0ull;
        }
        p.pair_end[a] = done;
        p.fd_L[a] = make_fastdiv(static_cast<uint32_t>(p.L[a]));
    }
    for (int i = 0; i < p.np; ++i) p.turns[i] = fixed_turns(freq[i]);
    p.fd_np = make_fastdiv(static_cast<uint32_t>(p.np));
    p.amp = amp;
    p.sgn = back ? -1.f : 1.f;
    p.cph = D / V;
    const bool inter = layout == NA_ROPE_INTERLEAVED;
    bool split = false, even = true;
    if (!inter)
        for (int a = 0; a < ndim; ++a) {
            split |= (rot[a] / 2) % V != 0;
            even &= (rot[a] / 2) % 2 == 0;
        }
    int upr = p.cph;   // units per head row
    if (!inter && !split) {
        upr = p.cph / 2;
        int u = 0, ch = 0, pr = 0;
        for (int a = 0; a < ndim; ++a) {
            for (int i = 0; i < rot[a] / 2; i += V, ++u, pr += V) {
                p.ua[u] = static_cast<uint8_t>((ch + i) / V);
                p.ub[u] = static_cast<uint8_t>((ch + rot[a] / 2 + i) / V);
                p.up[u] = static_cast<uint8_t>(pr);
            }
            ch += rot[a];
        }
        for (; u < upr; ++u, ch += 2 * V) {
            p.ua[u] = static_cast<uint8_t>(ch / V);
            p.ub[u] = static_cast<uint8_t>(ch / V + 1);
            p.up[u] = 0xff;
        }
    }
    if (split) {
        for (int c = 0; c < D; ++c) p.pair[c] = 0xff;
        int ch = 0, pr = 0;
        for (int a = 0; a < ndim; ++a) {
            for (int i = 0; i < rot[a] / 2; ++i, ++pr) {
                const int lo = ch + i, hi = ch + rot[a] / 2 + i;
                p.partner[lo] = static_cast<uint8_t>(hi);
                p.partner[hi] = static_cast<uint8_t>(lo);
                p.pair[lo] = p.pair[hi] = static_cast<uint8_t>(pr);
            }
            ch += rot[a];
        }
    }
    while ((1 << p.lu) < upr) ++p.lu;
    const long long upt_q = static_cast<long long>(heads_q) * upr, upt_k = static_cast<long long>(heads_k) * upr;
    // tokens per block: about kRopeBytes of rows and at most 24 KB of angles; fewer where the grid would
    // not fill the multiprocessors twice
    const long long row = (static_cast<long long>(heads_q) + heads_k) * D * es;
    const int g = inter ? V / 2 : V;   // pairs of a unit
    p.row = split ? D : p.np + (g >= 4 ? (p.np + g - 1) / g * 2 : 0);
    const long long angles = p.row * static_cast<long long>(sizeof(float2));
    long long tt = std::min<long long>({kRopeBytes / row, kMaxTokens, 24 * 1024 / angles});
    tt = tt < 1 ? 1 : tt;
    const long long fill = p.tokens / (2 * kSms);
    if (tt > fill) tt = fill < 1 ? 1 : fill;
    const long long blocks = (p.tokens + tt - 1) / tt;
    if (blocks > 0x7fffffffLL || tt * (upt_q + upt_k) > 0x3fffffffLL) return NA_ERR_UNSUPPORTED;
    p.upt[0] = static_cast<uint32_t>(upt_q);
    p.upt[1] = static_cast<uint32_t>(upt_k);
    for (int i = 0; i < 2; ++i) p.fd_upt[i] = make_fastdiv(p.upt[i]);
    p.tt = static_cast<int>(tt);
    const size_t smem = static_cast<size_t>(tt * angles);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const unsigned nb = static_cast<unsigned>(blocks);
    if (dtype == NA_BF16) launch_rope_t<__nv_bfloat16>(p, inter, split, even, nb, smem, s);
    else if (dtype == NA_FP16) launch_rope_t<__half>(p, inter, split, even, nb, smem, s);
    else launch_rope_t<float>(p, inter, split, even, nb, smem, s);
    return launch_result();
}

}  // namespace
}  // namespace na

extern "C" {

na_status na_rope(const void* q, const void* k, void* q_out, void* k_out, int B, int ndim, const int* spatial, int heads_q,
                  int heads_k, int D, const int* rot, const double* freq, const int64_t* origin, float amplitude,
                  na_rope_layout layout, na_dtype dtype, void* stream) {
    return na::rope(q, k, q_out, k_out, B, ndim, spatial, heads_q, heads_k, D, rot, freq, origin, amplitude, layout, dtype,
                    false, stream);
}

na_status na_rope_bwd(const void* dq_out, const void* dk_out, void* dq, void* dk, int B, int ndim, const int* spatial,
                      int heads_q, int heads_k, int D, const int* rot, const double* freq, const int64_t* origin,
                      float amplitude, na_rope_layout layout, na_dtype dtype, void* stream) {
    return na::rope(dq_out, dk_out, dq, dk, B, ndim, spatial, heads_q, heads_k, D, rot, freq, origin, amplitude, layout,
                    dtype, true, stream);
}

}  // extern "C"
