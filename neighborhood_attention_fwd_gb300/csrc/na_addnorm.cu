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
constexpr int kAddTileBytes = 8 * 1024;   // of a tile of the ring, an array
constexpr int kAddTileRows = 32;         // most rows of a tile: a lane holds a row's statistics
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
    int tile;                 // rows of a turn of a unit
    unsigned* err;            // ring: device status word
    unsigned long long wait_ns;
    uint32_t withhold;        // ring: test hook, block 0 leaves out its first copy
};

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

// A unit's rows of several arrays through a ring of tiles in shared memory (cp.async.bulk; rows are whole chunks, so a tile is one
// run of bytes of each array): registers alone do not keep enough loads under way beside the sums.  The unit's first thread
// fills a stage again once the unit has read it.
constexpr int kAddStages = 2;
template <int N, bool BLOCK>
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
    __device__ __forceinline__ void load(const AddParams& p, Walk& w, int stage) {   // the tile at w, if there is one
        w.settle();
        if (!w.parts()) return;
        const uint32_t bytes = row_bytes * w.rows();
        unsigned char* to = smem + static_cast<size_t>(stage) * N * p.tile * row_bytes;
        int arrays = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) arrays += from[i] != nullptr;
        mbar_arrive_expect_tx(&full[stage], arrays * bytes);
        if (!(p.withhold && blockIdx.x == 0 && issued == 0))   // test hook: the first copy never lands
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (from[i]) bulk_load(to + static_cast<size_t>(i) * p.tile * row_bytes, static_cast<const char*>(from[i]) + w.row * row_bytes, bytes, &full[stage]);
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
    __device__ __forceinline__ const unsigned char* at(const AddParams& p, int array, int row) const {
        return smem + static_cast<uint32_t>((s * N + array) * p.tile + row) * row_bytes;
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

// Blocks of the forward's warp teams per multiprocessor that the registers leave room for, with E channels to a thread.
__host__ __device__ constexpr int add_fwd_blocks(int E, bool lean) { return E <= 8 && lean ? 3 : 2; }

// A chunk of a row, of the ring or of memory; zeros where it is not there.
template <typename T, int V, bool RING>
__device__ __forceinline__ void take(Chunk<T, V>& c, bool there, const unsigned char* tile, const void* base, long long at, int col) {
    if constexpr (RING) c.raw = *reinterpret_cast<const uint4*>(tile + col * sizeof(T));
    else c.load(base, at + col);
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
    Ring<2, BLOCK> ring{full[unit], smem + static_cast<size_t>(unit) * kAddStages * 2 * p.tile * row_bytes, {p.y, p.x}, row_bytes,
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
                take<T, V, RING>(ry[j], inside(j), RING ? ring.at(p, 0, ri) : nullptr, p.y, row * p.C, at);
                take<T, V, RING>(rx[j], inside(j), RING ? ring.at(p, 1, ri) : nullptr, p.x, row * p.C, at);
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
    using A = Cols<V>;
    using W = typename A::W;
    constexpr int H = A::H;
    constexpr bool KEEP = J * V <= 8;
    extern __shared__ __align__(128) unsigned char smem[];   // rings; then, of warp teams, the sums: [warp][C]
    __shared__ __align__(16) float slots[2][2][2][16];   // taken in turn by the rows: a row's sums may be one
    constexpr int UNITS = BLOCK ? 1 : kAddThreads / 32;
    __shared__ uint64_t full[UNITS][kAddStages];
    const uint32_t row_bytes = p.C * static_cast<uint32_t>(sizeof(T));
    const size_t ring_bytes = RING ? static_cast<size_t>(kAddStages) * 4 * p.tile * row_bytes : 0;
    float* cols = reinterpret_cast<float*>(smem + UNITS * ring_bytes);
    const int lane = threadIdx.x & 31, l = BLOCK ? threadIdx.x : (threadIdx.x & (p.team - 1)), unit = BLOCK ? 0 : threadIdx.x >> 5;
    const int mine = BLOCK ? 0 : lane / p.team, teams = BLOCK ? 1 : 32 / p.team;   // of the unit
    const bool post = p.post != NA_NORM_NONE, norm = p.norm != NA_NORM_NONE;
    auto inside = [&](int j) { return (l + p.team * j) * V < p.C; };
    Walk w(p, unit, UNITS), ahead(w), next(w);
    Ring<4, BLOCK> ring{full[unit], smem + unit * ring_bytes, {p.dh, p.s_in, p.ds, p.y}, row_bytes, BLOCK ? threadIdx.x == 0 : lane == 0};
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
                    if constexpr (RING) c.raw = *reinterpret_cast<const uint4*>(ring.at(p, array, ri) + min((l + p.team * j) * V, p.C - V) * sizeof(T));
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

// How a problem is laid out: chunk width, chunks per thread, threads per row, blocks, parts of a group, rows of a tile.
struct AddPlan {
    bool vec, block, ring;
    int j, team, blocks, per_group, tile;
    size_t ring_bytes;
};

AddPlan plan_add(long long group_rows, long long groups, int C, int es, bool bwd, bool lean = false) {
    AddPlan n{};
    const int V = C % (16 / es) == 0 ? 16 / es : 1;
    n.vec = V > 1;
    const int chunks = C / V;
    // chunks per thread of a warp team, at most; longer rows are a block's
    const int warp_j = V == 8 || (bwd && V == 4) ? 2 : 4;
    n.block = chunks > 32 * warp_j;
    int teams = 1, per_sm, units = 1;
    if (!n.block) {
        n.team = 1;
        while (n.team < chunks && n.team < 32) n.team *= 2;
        n.j = 1;
        while (n.j * n.team < chunks) n.j *= 2;
        if (!n.vec) n.j = 4;
        teams = 32 / n.team;
        units = kAddThreads / 32;
        per_sm = bwd ? 2 : (n.vec ? add_fwd_blocks(n.j * V, lean) : 4);
    } else {
        n.j = V == 8 ? 1 : (V == 4 ? 2 : 4);
        while (n.j * kAddBlock < chunks) n.j *= n.vec ? 2 : 4;
        n.team = ((chunks + n.j - 1) / n.j + 31) / 32 * 32;
        per_sm = std::max(1, std::min(16, (bwd ? 512 : 1024) / n.team));
    }
    n.tile = teams;
    const int arrays = bwd ? 4 : 2, row = C * es;
    const size_t sums = bwd && !n.block ? static_cast<size_t>(kAddThreads / 32) * C * 4 : 0;
    if (n.vec) {
        // As many rows of a unit as `per_sm` blocks have room for, of at most kAddTileBytes an array.  A pass of a warp's teams is at most
        // 1 KB an array (2 KB forward): two stages of it, the sums and what else a block holds always fit.
        const size_t room = ((224 * 1024) / per_sm - sums - 4 * 1024) / units, pass = static_cast<size_t>(kAddStages) * teams * row * arrays;
        if (room >= pass) {
            n.ring = true;
            int passes = std::max(1, std::min({static_cast<int>(room / pass), kAddTileBytes / (teams * row), kAddTileRows / teams}));
            // fewer rows a tile where the grid is small
            while (passes > 1 && groups * group_rows < static_cast<long long>(teams) * passes * units * kSms * per_sm * kAddStages) --passes;
            n.tile = teams * passes;
            n.ring_bytes = passes * pass * units;
        }
    }
    const long long tiles = (group_rows + n.tile - 1) / n.tile, most = static_cast<long long>(kSms) * per_sm;
    // in the backward a part's sums cost about as much as a few rows of its own
    const long long least = units * (bwd && n.block ? 4 : 1);
    n.per_group = static_cast<int>(std::max(1LL, std::min((tiles + least - 1) / least, most / groups)));
    n.blocks = static_cast<int>(std::min(groups * n.per_group, most));
    return n;
}

bool lean_forward(const AddParams& p) { return p.norm != NA_NORM_LAYER && p.post != NA_NORM_LAYER && !p.b && !p.post_b; }

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

template <typename T, bool BWD>
na_status launch_add(const AddParams& p, const AddPlan& n, cudaStream_t s) {
    constexpr int V = Elem<T>::EPC;
    if (n.vec && !n.block) {
        if (!n.ring) return NA_ERR_UNSUPPORTED;   // never: see plan_add
        if (n.j == 1) return run_add<T, V, 1, false, BWD, true>(p, n, s);
        if (n.j == 2) return run_add<T, V, 2, false, BWD, true>(p, n, s);
        if constexpr (V == 4 && !BWD) return run_add<T, V, 4, false, BWD, true>(p, n, s);
    } else if (n.vec) {
        if constexpr (V == 8)
            if (n.j == 1) return n.ring ? run_add<T, V, 1, true, BWD, true>(p, n, s) : run_add<T, V, 1, true, BWD, false>(p, n, s);
        if (n.j == 2) return n.ring ? run_add<T, V, 2, true, BWD, true>(p, n, s) : run_add<T, V, 2, true, BWD, false>(p, n, s);
        if constexpr (V == 4) return n.ring ? run_add<T, V, 4, true, BWD, true>(p, n, s) : run_add<T, V, 4, true, BWD, false>(p, n, s);
    } else if (!n.block) {
        return run_add<T, 1, 4, false, BWD, false>(p, n, s);
    }
    return n.j == 4 ? run_add<T, 1, 4, true, BWD, false>(p, n, s) : run_add<T, 1, 16, true, BWD, false>(p, n, s);
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
    if (n.ring && (st = device_status_word(&p.err)) != NA_OK) return st;
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
