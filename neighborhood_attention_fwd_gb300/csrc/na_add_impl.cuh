// na_add_impl.cuh -- kernels of the residual add between norms, forward and backward (see na_addnorm.cu).
#pragma once

#include "na_add.h"
#include "na_rows.cuh"

namespace na {
namespace add {

using namespace rows;

// The coefficients of the unit rows in z scaled and gated: z = f a + c.  Zeros past the row, where they leave nothing in a sum.
template <int V>
__device__ __forceinline__ void gate_weights(const AddParams& p, const float* gate, int at, float (&a)[V], float (&c)[V]) {
    float g[V], w[V], b[V];
    const bool in = at < p.C;
    load_weights<V>(in ? gate : nullptr, at, g, 1.f);
    load_weights<V>(in ? p.post_w : nullptr, at, w, 1.f);
    load_weights<V>(in ? p.post_b : nullptr, at, b, 0.f);
#pragma unroll
    for (int e = 0; e < V; ++e) {
        a[e] = in ? p.scale * g[e] * w[e] : 0.f;
        c[e] = in ? p.scale * g[e] * b[e] : 0.f;
    }
}

// Parts and tiles.  A block takes parts part, part + grid, ..; a part is a group's tiles of `tile` rows, every per_group-th run of
// `units` of them, one for each of the block's units: a warp, or of rows a block wide the block.
struct Walk {
    const AddParams& p;
    int unit, units, part, group;
    long long step, row, end;   // rows to the next tile; the tile's first row, the end of the group
    __device__ __forceinline__ Walk(const AddParams& q, int u, int n)
        : p(q), unit(u), units(n), part(blockIdx.x), step(static_cast<long long>(q.tile) * q.per_group * n) {
        open();
    }
    __device__ __forceinline__ bool parts() const { return part < p.groups * p.per_group; }
    __device__ __forceinline__ void open() {
        if (!parts()) return;
        group = part / p.per_group;
        row = group * p.group_rows + (static_cast<long long>(part - group * p.per_group) * units + unit) * p.tile;
        end = (group + 1) * p.group_rows;
    }
    __device__ __forceinline__ bool here() const { return row < end; }   // the part has this tile
    __device__ __forceinline__ int rows() const { return static_cast<int>(min(static_cast<long long>(p.tile), end - row)); }
    __device__ __forceinline__ void next() { row += step; }
    __device__ __forceinline__ void next_part() {
        part += gridDim.x;
        open();
    }
    // the next tile in any part
    __device__ __forceinline__ void settle() {
        while (parts() && !here()) next_part();
    }
    __device__ __forceinline__ const float* at(const float* v, long long step) const { return v ? v + group * step : nullptr; }
};

// A unit's rows of several arrays through a ring of tiles in shared memory (cp.async.bulk): registers alone do not keep enough
// loads under way beside the sums.  A tile is one run of bytes of each array.  Rows that are not whole chunks start anywhere: then
// the run is widened to 16 bytes on both sides (what it brings of other rows is not read), and the tensor's last bytes, which it
// must not pass, are copied one by one.  The unit's first thread fills a stage again once the unit has read it.
template <int N, bool BLOCK, bool WHOLE>
struct Ring {
    uint64_t* full;                // shared: a barrier a stage
    unsigned char* smem;           // [stage][array][tile]
    const void* from[N];           // null: left out
    uint32_t row_bytes;
    bool first;                    // the unit's first thread; it alone uses what follows
    int issued, lost;              // tiles loaded; the first one whose copy did not land in time (-1: none)
    int s;
    uint32_t parity;

    static __device__ __forceinline__ void sync() {
        if (BLOCK) __syncthreads();
        else __syncwarp();
    }
    __device__ __forceinline__ uint32_t pitch(const AddParams& p) const { return ring_pitch(p.tile * row_bytes, WHOLE); }
    __device__ __forceinline__ void load(const AddParams& p, Walk& w, int stage) {   // the tile at w, if there is one
        w.settle();
        if (!w.parts()) return;
        unsigned char* to = smem + static_cast<size_t>(stage) * N * pitch(p);
        uint32_t bytes = row_bytes * w.rows();
        long long start = w.row * row_bytes;
        if (!WHOLE) {
            const long long end = start + bytes, stop = min((end + 15) & ~15ll, (p.rows * row_bytes) & ~15ll);
            start &= ~15ll;
            for (long long o = stop; o < end; o += 2)
#pragma unroll
                for (int i = 0; i < N; ++i)
                    if (from[i])
                        *reinterpret_cast<uint16_t*>(to + static_cast<size_t>(i) * pitch(p) + (o - start)) =
                            *reinterpret_cast<const uint16_t*>(static_cast<const char*>(from[i]) + o);
            bytes = static_cast<uint32_t>(stop - start);
        }
        int arrays = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) arrays += from[i] != nullptr;
        mbar_arrive_expect_tx(&full[stage], arrays * bytes);
        if (!(p.withhold && blockIdx.x == 0 && issued == 0) && (WHOLE || bytes))   // test hook: the first copy never lands
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (from[i]) bulk_load(to + static_cast<size_t>(i) * pitch(p), static_cast<const char*>(from[i]) + start, bytes, &full[stage]);
        ++issued;
        w.next();
    }
    __device__ __forceinline__ void start(const AddParams& p, Walk& ahead) {
        s = 0;
        parity = 0;
        issued = 0;
        lost = -1;
        if (first) {
            for (int i = 0; i < kAddStages; ++i) mbar_init(&full[i], 1);
            fence_barrier_init();
            for (int i = 0; i < kAddStages; ++i) load(p, ahead, i);
        }
        sync();
    }
    // A wait that runs out records itself; the unit then goes on to its end without copies.
    __device__ __forceinline__ void wait(const AddParams& p, int step) {
        if (!mbar_wait(&full[s], parity, WaitGuard{p.err, p.wait_ns}, kSiteNorm) && lost < 0) lost = step;
    }
    __device__ __forceinline__ const unsigned char* at(const AddParams& p, const Walk& w, int array, int row) const {   // of the tile at w
        if (WHOLE) return smem + static_cast<uint32_t>((s * N + array) * p.tile + row) * row_bytes;
        return smem + (s * N + array) * pitch(p) + (static_cast<uint32_t>(w.row * row_bytes) & 15u) + static_cast<uint32_t>(row) * row_bytes;
    }
    __device__ __forceinline__ void done(const AddParams& p, Walk& ahead) {   // the unit has read the tile
        sync();
        if (first && lost < 0) load(p, ahead, s);
        if (++s == kAddStages) {
            s = 0;
            parity ^= 1u;
        }
    }
    __device__ __forceinline__ void finish(const AddParams& p) {   // the copies in flight have to land before the memory is given back
        if (first && lost >= 0)
            for (int i = lost; i < issued; ++i) mbar_drain(&full[i % kAddStages], (i / kAddStages) & 1, p.wait_ns);
    }
};

// Sums over a row's team; of a block's, every thread adds the warps' sums itself (slots: [value][warp], zeros of warps that are
// not there), which is shorter than a second round of shuffles.
template <int N, bool BLOCK>
__device__ __forceinline__ void row_sum(float (&v)[N], int team, float (*slot)[16]) {
    if constexpr (!BLOCK) {
        team_sum<N, false>(v, team, nullptr);
    } else {
#pragma unroll
        for (int m = 16; m >= 1; m >>= 1)
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], m);
        if ((threadIdx.x & 31) == 0) {
#pragma unroll
            for (int i = 0; i < N; ++i) slot[i][threadIdx.x >> 5] = v[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            v[i] = 0.f;
            for (int w = 0; w < static_cast<int>(blockDim.x >> 5); w += 4) {
                const float4 t = *reinterpret_cast<const float4*>(&slot[i][w]);
                v[i] += (t.x + t.y) + (t.z + t.w);
            }
        }
    }
}

// A chunk of a row, of the ring or of memory; zeros where it is not there.
template <typename T, int V, bool RING>
__device__ __forceinline__ void take(Chunk<T, V>& c, bool there, const unsigned char* row, const void* from, long long base, int at) {
    if constexpr (!RING) c.load(from, base + at);
    else if constexpr (V == 1) c.raw = *reinterpret_cast<const T*>(row + at * sizeof(T));
    else c.raw = *reinterpret_cast<const uint4*>(row + at * sizeof(T));
    if (!there) c = Chunk<T, V>{};
}

// LEAN: neither norm has a mean, and there are no shifts.
template <typename T, int V, int J, bool BLOCK, bool RING, bool LEAN>
__global__ void __launch_bounds__(BLOCK ? kAddBlock : kAddThreads, BLOCK || !RING ? 1 : add_fwd_blocks(J * V, LEAN)) add_fwd_kernel(const AddParams p) {
    using A = Cols<V>;
    using W = typename A::W;
    constexpr int H = A::H;
    constexpr bool KEEP = J * V <= 8;   // vectors stay in registers over a part's rows
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ __align__(16) float slots[2][4][1][16];   // taken in turn by the rows: a row's sums may be one
    constexpr int UNITS = BLOCK ? 1 : kAddThreads / 32;
    __shared__ uint64_t full[UNITS][kAddStages];
    const int l = BLOCK ? threadIdx.x : (threadIdx.x & (p.team - 1)), unit = BLOCK ? 0 : threadIdx.x >> 5;
    const int mine = BLOCK ? 0 : (threadIdx.x & 31) / p.team, teams = BLOCK ? 1 : 32 / p.team;   // of the unit
    const bool post = p.post != NA_NORM_NONE, norm = p.norm != NA_NORM_NONE;
    auto inside = [&](int j) { return (l + p.team * j) * V < p.C; };
    Walk w(p, unit, UNITS), ahead(w);
    const uint32_t row_bytes = p.C * static_cast<uint32_t>(sizeof(T));
    Ring<2, BLOCK, (V > 1)> ring{full[unit], smem + static_cast<size_t>(unit) * kAddStages * 2 * ring_pitch(p.tile * row_bytes, V > 1), {p.y, p.x}, row_bytes,
                                 BLOCK ? threadIdx.x == 0 : (threadIdx.x & 31) == 0};
    if constexpr (BLOCK) {
        for (int i = threadIdx.x; i < static_cast<int>(sizeof slots / sizeof(float)); i += blockDim.x) (&slots[0][0][0][0])[i] = 0.f;
        __syncthreads();
    }
    if constexpr (RING) ring.start(p, ahead);
    W ka[KEEP ? J : 1][H], kc[KEEP ? J : 1][H], kw[KEEP ? J : 1][H], kb[KEEP ? J : 1][H];
    const float *gate = nullptr, *weight = nullptr, *shift = nullptr;
    auto vectors = [&](int j, int at) {
        const int i = KEEP ? j : 0;
        float a[V], c[V];
        gate_weights<V>(p, gate, at, a, c);
        A::from(a, ka[i]);
        A::from(c, kc[i]);
    };
    auto weights = [&](int j, int at) {
        const int i = KEEP ? j : 0;
        float wt[V], b[V];
        load_weights<V>(at < p.C ? weight : nullptr, at, wt, 1.f);
        load_weights<V>(at < p.C ? shift : nullptr, at, b, 0.f);
        A::from(wt, kw[i]);
        A::from(b, kb[i]);
    };
    int turn = 0, group = -1;
    w.settle();
    for (int step = 0; w.parts(); ++step, w.next(), w.settle()) {
        if (w.group != group) {
            group = w.group;
            gate = w.at(p.gate, p.gate_step);
            weight = w.at(p.w, p.w_step);
            shift = w.at(p.b, p.w_step);
            if (KEEP) {
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    vectors(j, (l + p.team * j) * V);
                    weights(j, (l + p.team * j) * V);
                }
            }
        }
        const int n = w.rows();
        if constexpr (RING) ring.wait(p, step);
        for (int r0 = mine; r0 - mine < n; r0 += teams, turn ^= 1) {
            const bool live = r0 < n;   // whole warps stay together, for the sums
            const int ri = live ? r0 : n - 1;
            const long long row = w.row + ri;
            Chunk<T, V> rx[J], ry[J];
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const int at = min((l + p.team * j) * V, p.C - V);
                take<T, V, RING>(ry[j], inside(j), RING ? ring.at(p, w, 0, ri) : nullptr, p.y, row * p.C, at);
                take<T, V, RING>(rx[j], inside(j), RING ? ring.at(p, w, 1, ri) : nullptr, p.x, row * p.C, at);
            }
            W s[J][H];
            float r = 1.f;
#pragma unroll
            for (int j = 0; j < J; ++j) {
                float f[V];
                ry[j].get(f);
                A::from(f, s[j]);
            }
            // Centres s on its mean for layer norm, and the inverse deviation of what is left.
            auto moments = [&](int kind, int at, float& mean) {
                mean = 0.f;
                if (!LEAN && kind == NA_NORM_LAYER) {
                    W t = 0;
#pragma unroll
                    for (int j = 0; j < J; ++j)
#pragma unroll
                        for (int e = 0; e < H; ++e) t = A::add(t, s[j][e]);
                    float sum[1] = {A::sum(t)};
                    row_sum<1, BLOCK>(sum, p.team, slots[turn][at]);
                    mean = sum[0] * p.inv_c;
#pragma unroll
                    for (int j = 0; j < J; ++j) {
                        const W m = A::both(inside(j) ? -mean : 0.f);
#pragma unroll
                        for (int e = 0; e < H; ++e) s[j][e] = A::add(s[j][e], m);
                    }
                }
                W t = 0;
#pragma unroll
                for (int j = 0; j < J; ++j)
#pragma unroll
                    for (int e = 0; e < H; ++e) t = A::fma(s[j][e], s[j][e], t);
                float sum[1] = {A::sum(t)};
                row_sum<1, BLOCK>(sum, p.team, slots[turn][at + 1]);
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
                    s[j][e] = A::fma(A::mul(s[j][e], A::both(r)), ka[i][e], LEAN ? A::mul(x[e], A::both(p.residual)) : A::fma(x[e], A::both(p.residual), kc[i][e]));
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
                for (int e = 0; e < H; ++e) h[e] = LEAN ? A::mul(A::mul(s[j][e], A::both(r)), kw[i][e]) : A::fma(A::mul(s[j][e], A::both(r)), kw[i][e], kb[i][e]);
                if (live && at < p.C) {
                    A::to(h, f);
                    store_chunk<T, V>(p.h, row * p.C + at, f);
                }
            }
        }
        if constexpr (RING) ring.done(p, ahead);
    }
    if constexpr (RING) ring.finish(p);
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

// LEAN: neither norm has a mean and neither db nor dpost_b is wanted: without their sums, a third of the instructions that
// bound rows of 2-byte channels.
template <typename T, int V, int J, bool BLOCK, bool RING, bool LEAN>
__global__ void __launch_bounds__(BLOCK ? kAddBlock : kAddThreads, BLOCK ? 1 : 2) add_bwd_kernel(const AddParams p) {
    next_may_start();
    using A = Cols<V>;
    using W = typename A::W;
    constexpr int H = A::H;
    constexpr bool KEEP = J * V <= 8;
    extern __shared__ __align__(128) unsigned char smem[];   // rings; then, of warp teams, the sums: [warp][C]
    __shared__ __align__(16) float slots[2][2][2][16];   // taken in turn by the rows: a row's sums may be one
    constexpr int UNITS = BLOCK ? 1 : kAddThreads / 32;
    __shared__ uint64_t full[UNITS][kAddStages];
    const uint32_t row_bytes = p.C * static_cast<uint32_t>(sizeof(T));
    const size_t ring_bytes = RING ? static_cast<size_t>(kAddStages) * 4 * ring_pitch(p.tile * row_bytes, V > 1) : 0;
    float* cols = reinterpret_cast<float*>(smem + UNITS * ring_bytes);
    const int lane = threadIdx.x & 31, l = BLOCK ? threadIdx.x : (threadIdx.x & (p.team - 1)), unit = BLOCK ? 0 : threadIdx.x >> 5;
    const int mine = BLOCK ? 0 : lane / p.team, teams = BLOCK ? 1 : 32 / p.team;   // of the unit
    const bool post = p.post != NA_NORM_NONE, norm = p.norm != NA_NORM_NONE;
    auto inside = [&](int j) { return (l + p.team * j) * V < p.C; };
    Walk w(p, unit, UNITS), ahead(w), next(w);
    Ring<4, BLOCK, (V > 1)> ring{full[unit], smem + unit * ring_bytes, {p.dh, p.s_in, p.ds, p.y}, row_bytes, BLOCK ? threadIdx.x == 0 : lane == 0};
    // a tile's statistics, a tile ahead: lane r holds those of row r
    float ahead_stats[4];
    auto read_stats = [&](float (&t)[4]) {
        next.settle();
        const bool there = next.parts() && lane < next.rows();
        const float* from[4] = {LEAN ? nullptr : p.mean, p.rstd, LEAN ? nullptr : p.post_mean, p.post_rstd};
#pragma unroll
        for (int i = 0; i < 4; ++i) t[i] = there && from[i] ? from[i][next.row + lane] : 0.f;
        next.next();
    };
    if constexpr (BLOCK) {
        for (int i = threadIdx.x; i < static_cast<int>(sizeof slots / sizeof(float)); i += blockDim.x) (&slots[0][0][0][0])[i] = 0.f;
        __syncthreads();
    }
    read_stats(ahead_stats);
    if constexpr (RING) ring.start(p, ahead);
    W ka[KEEP ? J : 1][H], kw[KEEP ? J : 1][H];
    W t0[J][H], t1[J][H], t2[J][H], t3[J][H];   // sums of dh e, dh, D f, D
    const float *gate = nullptr, *weight = nullptr;
    auto vectors = [&](int j) {
        float a[V], c[V];
        gate_weights<V>(p, gate, (l + p.team * j) * V, a, c);
        A::from(a, ka[KEEP ? j : 0]);
    };
    auto weights = [&](int j) {
        float wt[V];
        load_weights<V>(inside(j) ? weight : nullptr, (l + p.team * j) * V, wt, 1.f);
        A::from(wt, kw[KEEP ? j : 0]);
    };
    int turn = 0, step = 0;
    for (; w.parts(); w.next_part()) {
        gate = w.at(p.gate, p.gate_step);
        weight = w.at(p.w, p.w_step);
#pragma unroll
        for (int j = 0; j < J; ++j) {
            if (KEEP) {
                vectors(j);
                weights(j);
            }
#pragma unroll
            for (int e = 0; e < H; ++e) t0[j][e] = t1[j][e] = t2[j][e] = t3[j][e] = 0;
        }
        for (; w.here(); ++step, w.next()) {
            const int n = w.rows();
            float stats[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) stats[i] = ahead_stats[i];
            read_stats(ahead_stats);
            if constexpr (RING) ring.wait(p, step);
            for (int r0 = mine; r0 - mine < n; r0 += teams, turn ^= 1) {
                const bool live = r0 < n;
                const int ri = live ? r0 : n - 1;
                const long long row = w.row + ri;
                // From memory all loads go out at once; from the ring each is read where it is used.  Places past the end are zeros made of
                // zeros, with statistics of zero: what stands there need not be finite, and may be an output already.
                Chunk<T, V> raw[RING ? 1 : 4][J];
                if constexpr (!RING) {
                    const void* from[4] = {p.dh, p.s_in, p.ds, p.y};
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int j = 0; j < J; ++j)
                            if (from[i]) raw[i][j].load(from[i], row * p.C + min((l + p.team * j) * V, p.C - V));
                }
                auto read = [&](int array, int j, W (&v)[H]) {
                    float f[V];
                    Chunk<T, V> c;
                    if constexpr (RING) take<T, V, true>(c, true, ring.at(p, w, array, ri), nullptr, 0, min((l + p.team * j) * V, p.C - V));
                    else c = raw[array][j];
                    if (!live || !inside(j)) c = Chunk<T, V>{};
                    c.get(f);
                    A::from(f, v);
                };
                auto stat = [&](int i, const float* from, float none) {
                    const float v = __shfl_sync(0xffffffffu, stats[i], ri);
                    return !live ? 0.f : !from ? none : v;
                };
                const float norm_mean = LEAN ? 0.f : stat(0, p.mean, 0.f), norm_rstd = stat(1, p.rstd, 1.f);
                const float mean = LEAN ? 0.f : stat(2, p.post_mean, 0.f), rstd = stat(3, p.post_rstd, 1.f);
                // unit rows: (v - mean) rstd
                auto unit = [&](W (&v)[H], float m, float r) {
#pragma unroll
                    for (int e = 0; e < H; ++e) v[e] = A::mul(LEAN ? v[e] : A::add(v[e], A::both(-m)), A::both(r));
                };
                W d[J][H];
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    if (p.ds) read(2, j, d[j]);
                    else
#pragma unroll
                        for (int e = 0; e < H; ++e) d[j][e] = 0;
                }
                if (norm) {
                    W e_[J][H], g[J][H], s0 = 0, s1 = 0;
#pragma unroll
                    for (int j = 0; j < J; ++j) {
                        if (!KEEP) weights(j);
                        W dh[H];
                        read(0, j, dh);
                        read(1, j, e_[j]);
                        unit(e_[j], norm_mean, norm_rstd);
#pragma unroll
                        for (int e = 0; e < H; ++e) {
                            t0[j][e] = A::fma(dh[e], e_[j][e], t0[j][e]);
                            if (!LEAN) t1[j][e] = A::add(t1[j][e], dh[e]);
                            g[j][e] = A::mul(dh[e], kw[KEEP ? j : 0][e]);
                            if (!LEAN) s0 = A::add(s0, g[j][e]);
                            s1 = A::fma(g[j][e], e_[j][e], s1);
                        }
                    }
                    float k0 = 0.f, k1;
                    if constexpr (LEAN) {
                        float s[1] = {A::sum(s1)};
                        row_sum<1, BLOCK>(s, p.team, slots[turn][0]);
                        k1 = -norm_rstd * (s[0] * p.inv_c);
                    } else {
                        float s[2] = {A::sum(s0), A::sum(s1)};
                        row_sum<2, BLOCK>(s, p.team, slots[turn][0]);
                        if (p.norm == NA_NORM_LAYER) k0 = -norm_rstd * (s[0] * p.inv_c);
                        k1 = -norm_rstd * (s[1] * p.inv_c);
                    }
#pragma unroll
                    for (int j = 0; j < J; ++j)
#pragma unroll
                        for (int e = 0; e < H; ++e) {
                            if (!LEAN) d[j][e] = A::add(d[j][e], A::both(k0));
                            d[j][e] = A::fma(e_[j][e], A::both(k1), A::fma(g[j][e], A::both(norm_rstd), d[j][e]));
                        }
                }
                W f_[J][H], s0 = 0, s1 = 0;
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    const int at = (l + p.team * j) * V;
                    if (!KEEP) vectors(j);
                    read(3, j, f_[j]);
                    unit(f_[j], mean, rstd);
                    W o[H];
#pragma unroll
                    for (int e = 0; e < H; ++e) {
                        o[e] = A::mul(d[j][e], A::both(p.residual));
                        t2[j][e] = A::fma(d[j][e], f_[j][e], t2[j][e]);
                        if (!LEAN) t3[j][e] = A::add(t3[j][e], d[j][e]);
                        d[j][e] = A::mul(d[j][e], ka[KEEP ? j : 0][e]);
                        if (!LEAN) s0 = A::add(s0, d[j][e]);
                        s1 = A::fma(d[j][e], f_[j][e], s1);
                    }
                    if (live && at < p.C) {
                        float f[V];
                        A::to(o, f);
                        store_chunk<T, V>(p.dx, row * p.C + at, f);
                    }
                }
                float k0 = 0.f, k1 = 0.f;
                if (post) {
                    if constexpr (LEAN) {
                        float s[1] = {A::sum(s1)};
                        row_sum<1, BLOCK>(s, p.team, slots[turn][1]);
                        k1 = -rstd * (s[0] * p.inv_c);
                    } else {
                        float s[2] = {A::sum(s0), A::sum(s1)};
                        row_sum<2, BLOCK>(s, p.team, slots[turn][1]);
                        if (p.post == NA_NORM_LAYER) k0 = -rstd * (s[0] * p.inv_c);
                        k1 = -rstd * (s[1] * p.inv_c);
                    }
                }
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    const int at = (l + p.team * j) * V;
                    W o[H];
#pragma unroll
                    for (int e = 0; e < H; ++e) {
                        o[e] = LEAN ? A::mul(d[j][e], A::both(rstd)) : A::fma(d[j][e], A::both(rstd), A::both(k0));
                        o[e] = A::fma(f_[j][e], A::both(k1), o[e]);
                    }
                    if (live && at < p.C) {
                        float f[V];
                        A::to(o, f);
                        store_chunk<T, V>(p.dy, row * p.C + at, f);
                    }
                }
            }
            if constexpr (RING) ring.done(p, ahead);
        }
        if (p.slot[0] >= 0) store_sums<V, J, BLOCK>(p, w.part, p.slot[0], t0, l, cols);
        if (!LEAN && p.slot[1] >= 0) store_sums<V, J, BLOCK>(p, w.part, p.slot[1], t1, l, cols);
        if (p.slot[2] >= 0) store_sums<V, J, BLOCK>(p, w.part, p.slot[2], t2, l, cols);
        if (!LEAN && p.slot[3] >= 0) store_sums<V, J, BLOCK>(p, w.part, p.slot[3], t3, l, cols);
    }
    if constexpr (RING) ring.finish(p);
}

template <typename Kernel>
na_status start_add(Kernel* kernel, const AddParams& p, const AddPlan& n, size_t smem, cudaStream_t s) {
    if (smem > 32 * 1024 && !allow_shared(reinterpret_cast<const void*>(kernel))) return NA_ERR_CUDA;
    kernel<<<n.blocks, n.block ? n.team : kAddThreads, smem, s>>>(p);
    return launch_result();
}

template <typename T, int V, int J, bool BLOCK, bool BWD, bool RING>
na_status run_add(const AddParams& p, const AddPlan& n, cudaStream_t s) {
    if constexpr (BWD) {
        const size_t smem = n.ring_bytes + (BLOCK || !p.partial ? 0 : static_cast<size_t>(kAddThreads / 32) * p.C * sizeof(float));
        const bool lean = p.norm != NA_NORM_LAYER && p.post != NA_NORM_LAYER && p.slot[1] < 0 && p.slot[3] < 0;
        if constexpr (V > 1)
            if (lean) return start_add(add_bwd_kernel<T, V, J, BLOCK, RING, true>, p, n, smem, s);
        return start_add(add_bwd_kernel<T, V, J, BLOCK, RING, false>, p, n, smem, s);
    } else {
        if constexpr (V > 1)
            if (lean_forward(p)) return start_add(add_fwd_kernel<T, V, J, BLOCK, RING, true>, p, n, n.ring_bytes, s);
        return start_add(add_fwd_kernel<T, V, J, BLOCK, RING, false>, p, n, n.ring_bytes, s);
    }
}

template <typename T, int V, int J, bool BWD>
na_status run_block(const AddParams& p, const AddPlan& n, cudaStream_t s) {
    return n.ring ? run_add<T, V, J, true, BWD, true>(p, n, s) : run_add<T, V, J, true, BWD, false>(p, n, s);
}

template <typename T, bool BWD>
na_status launch_add(const AddParams& p, const AddPlan& n, cudaStream_t s) {
    constexpr int V = Elem<T>::EPC;
    if (!n.block) {
        if (!n.ring) return NA_ERR_UNSUPPORTED;   // never: see plan_add
        if (!n.vec) {
            return n.j == 4 ? run_add<T, 1, 4, false, BWD, true>(p, n, s) : run_add<T, 1, 8, false, BWD, true>(p, n, s);
        }
        if (n.j == 1) return run_add<T, V, 1, false, BWD, true>(p, n, s);
        if constexpr (V == 4 || !BWD)
            if (n.j == 2) return run_add<T, V, 2, false, BWD, true>(p, n, s);
        if constexpr (V == 4 && !BWD) return run_add<T, V, 4, false, BWD, true>(p, n, s);
        return NA_ERR_UNSUPPORTED;   // never: see plan_add
    }
    if (!n.vec) {
        if (n.j == 4) return run_block<T, 1, 4, BWD>(p, n, s);
        return n.j == 8 ? run_block<T, 1, 8, BWD>(p, n, s) : run_block<T, 1, 16, BWD>(p, n, s);
    }
    if constexpr (V == 8)
        if (n.j == 1) return run_block<T, V, 1, BWD>(p, n, s);
    if (n.j == 2) return run_block<T, V, 2, BWD>(p, n, s);
    if constexpr (V == 4) return run_block<T, V, 4, BWD>(p, n, s);
    return NA_ERR_UNSUPPORTED;   // never: see plan_add
}

}  // namespace add
}  // namespace na
