// na_glu_tc.cuh -- tensor-core kernels of the gated feed-forward product (bf16 or fp16 operands, fp32 accumulators).
//
// A product's result is cut into tiles, 256 x 256 for a pair of blocks (tcgen05.mma with cta_group::2: each block holds 128
// rows and half of the columns' operand) or 128 x 128 for one block.  Blocks stay and take tiles in turn.  Per tile, steps of
// 64 along the summed axis come by TMA through a ring of stages (128-byte swizzle), one thread issues the products, and eight
// (or four) warps take the finished accumulators from TMEM while the next tile's products fill the other half of it.
//   forward, slopes   rows: tokens; columns: as many of g as of u, so that both factors of an element meet in one thread
//   tokens            dx: rows: tokens; columns: channels; summed over the columns of dg, then of du
//   weights           dWg, dWu: rows: columns of dg or du; columns: channels; summed over tokens, operands turned by the
//                     descriptors (both run along the other axis in memory)
// Results leave through shared memory by TMA (32 rows of 128 bytes a warp), which also cuts them at the ragged edges.
// Few tokens have a kernel of their own (glu_few_kernel), which streams the weights as the rows of the product.
//
// Every wait is bounded (na_device.cuh).
#pragma once

#include <type_traits>

#include "na_block.cuh"
#include "na_device.cuh"
#include "na_glu.h"

namespace na {
namespace glu {

using namespace dev;

// ---------------------------------------------------------------------------------------------
// Pairs of blocks, and wider TMEM loads
// ---------------------------------------------------------------------------------------------

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Shared-cluster address of the same place in another block of the cluster.
__device__ __forceinline__ uint32_t peer_address(uint32_t local, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(local), "r"(rank));
    return r;
}
__device__ __forceinline__ void arrive_remote(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ float ld_cluster(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// A wait on a barrier that the other block of a pair arrives on: acquire at cluster scope.
__device__ __forceinline__ bool mbar_spin_cluster(uint64_t* bar, uint32_t parity, const WaitGuard& err, unsigned site) {
    const unsigned long long t0 = globaltimer();
    for (uint32_t i = 1;; ++i) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(smem_u32(bar)), "r"(parity)
            : "memory");
        if (ok) return true;
        if ((i & 63u) == 0u && (ld_volatile(err.word) != 0u || globaltimer() - t0 > err.limit_ns)) {
            record_error(err.word, site);
            return false;
        }
    }
}

template <int CG>
__device__ __forceinline__ void tmem_take(uint32_t* dst, uint32_t cols) {
    if constexpr (CG == 1) {
        tmem_alloc(dst, cols);
        tmem_relinquish();
    } else {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "r"(cols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
}
template <int CG>
__device__ __forceinline__ void tmem_give(uint32_t taddr, uint32_t cols) {
    if constexpr (CG == 1) tmem_dealloc(taddr, cols);
    else asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(cols) : "memory");
}

template <int CG>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    if constexpr (CG == 1) {
        umma_bf16(d, a, b, idesc, accumulate);
    } else {
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
            : "memory");
    }
}
// Arrive on `bar` (of both blocks of a pair) when every product issued so far has completed.
template <int CG>
__device__ __forceinline__ void commit(uint64_t* bar) {
    if constexpr (CG == 1) {
        umma_commit(bar);
    } else {
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                         smem_u32(bar)),
                     "h"(static_cast<uint16_t>(3))
                     : "memory");
    }
}

// A box of two axes into this block's shared memory; the bytes count on `bar`, an address of either block of a pair.
template <int CG>
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y) {
    if constexpr (CG == 1) {
        asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
                     "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
                     : "memory");
    } else {
        asm volatile(
            "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
            : "memory");
    }
}
__device__ __forceinline__ void store_box(const CUtensorMap* map, uint32_t src, int x, int y) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(reinterpret_cast<uint64_t>(map)),
                 "r"(src), "r"(x), "r"(y)
                 : "memory");
}
__device__ __forceinline__ void store_box(const CUtensorMap* map, uint32_t src, int x, int y, int z) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(reinterpret_cast<uint64_t>(map)),
                 "r"(src), "r"(x), "r"(y), "r"(z)
                 : "memory");
}

// 32 lanes x 16 columns of 32 bits (one row per lane).
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
          "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}
// No use of the registers moves above it (follows tmem_ld_wait_all).
__device__ __forceinline__ void reg_fence16(uint32_t (&r)[16]) {
    asm volatile(""
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]),
                   "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :
                 : "memory");
}

// Raw elements of T (bf16 or fp16) widened.
template <typename T>
__device__ __forceinline__ float widen(const void* base, long long at) {
    float lo, hi;
    Elem<T>::two(static_cast<const uint16_t*>(base)[at], lo, hi);
    return lo;
}
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}

// After a wait that ran out: time for what is in flight into this block's memory to land.
__device__ __forceinline__ void settle() {
    const unsigned long long t0 = globaltimer();
    while (globaltimer() - t0 < 1000000ull) __nanosleep(1000);
}

// ---------------------------------------------------------------------------------------------
// Tiles
// ---------------------------------------------------------------------------------------------

constexpr uint32_t kBand = 16;   // rows of tiles that are finished together: their operand and all columns' stay in L2

template <int WHICH, int CG, int NT>
struct TileShape {
    static constexpr bool PAIR = WHICH == kForward || WHICH == kSlopes;
    static constexpr int NF = NT / 2;                            // PAIR: columns of g (and of u) of a tile
    static constexpr int M = 128 * CG;                           // rows of a tile
    static constexpr uint32_t A_BYTES = 128 * 128, B_BYTES = NT / CG * 128, STAGE = A_BYTES + B_BYTES;
    static constexpr int WARPS = PAIR ? NF / 16 : 8;             // of the epilogue
    static constexpr int OUT = PAIR ? 64 : NT / 2;               // columns of a warp
    static constexpr int BUFFERS = WHICH == kForward ? 1 : 2;    // of 4 KB, a warp's
    static constexpr int STAGES = CG == 1 ? 5 : (WHICH == kSlopes ? 4 : 5);
    static constexpr int THREADS = 128 + 32 * WARPS;
    static constexpr uint32_t STAGING = STAGES * STAGE, BIAS = STAGING + WARPS * BUFFERS * 4096;
    static constexpr uint32_t BYTES = BIAS + (PAIR ? WARPS * 128 * 4 : 0) + 1024;   // 1024: to align the start
};

struct Tile {
    unsigned row, col, first, last, split;   // steps [first, last)
};
template <int WHICH>
__device__ __forceinline__ Tile tile_of(const GluTcParams& p, unsigned i) {
    const unsigned per = p.rows * p.cols;
    Tile t;
    t.split = i / per;
    i -= t.split * per;
    const unsigned band = i / (kBand * p.cols), base = band * kBand, height = min(kBand, p.rows - base);
    i -= base * p.cols;
    t.col = i / height;
    t.row = base + i - t.col * height;
    t.first = t.split * p.run;
    t.last = min(p.steps, t.first + p.run);
    return t;
}

template <int WHICH, int CG, int NT, typename T>
__global__ void __launch_bounds__(TileShape<WHICH, CG, NT>::THREADS, 1) glu_tile_kernel(const __grid_constant__ GluTcParams p) {
    using S = TileShape<WHICH, CG, NT>;
    constexpr bool PAIR = S::PAIR, WEIGHTS = WHICH == kWeights;
    extern __shared__ uint8_t raw_smem[];
    __shared__ uint64_t full[S::STAGES], empty[S::STAGES], acc_full[2], acc_empty[2], dh_full[S::WARPS];
    __shared__ uint32_t tmem_base;
    const uint32_t smem = (smem_u32(raw_smem) + 1023u) & ~1023u;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = CG == 2 ? cluster_rank() : 0u;
    const unsigned mine = blockIdx.x / CG, all = gridDim.x / CG, tiles = p.rows * p.cols * p.splits;
    const WaitGuard guard{p.err, p.wait_ns};
    if (threadIdx.x == 0) {
        for (int s = 0; s < S::STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_empty[i], CG * S::WARPS);
        }
        for (int i = 0; i < S::WARPS; ++i) mbar_init(&dh_full[i], 1);
        fence_barrier_init();
    }
    if (warp == 2) tmem_take<CG>(&tmem_base, 2 * NT);
    tc_fence_before();
    __syncthreads();
    if constexpr (CG == 2) cluster_sync();
    tc_fence_after();
    const uint32_t tmem = tmem_base;

    if (warp == 0 && lane == 0) {
        // copies
        const uint32_t full_at = CG == 2 ? peer_address(smem_u32(full), 0) : smem_u32(full);   // the leading block's barriers
        int s = 0;
        uint32_t parity = 1;
        bool ok = true, withhold = p.withhold && blockIdx.x == 0;
        for (unsigned i = mine; ok && i < tiles; i += all) {
            const Tile t = tile_of<WHICH>(p, i);
            for (unsigned k = t.first; k < t.last; ++k) {
                ok = CG == 2 ? mbar_spin_cluster(&empty[s], parity, guard, kSiteEmpty) : mbar_spin(&empty[s], parity, guard, kSiteEmpty);
                if (!ok) break;
                const uint32_t to = smem + s * S::STAGE;
                const uint32_t bar = full_at + s * 8;
                if (rank == 0) mbar_arrive_expect_tx(&full[s], CG * S::STAGE);
                if (withhold) {   // test hook: the first copy never lands
                    withhold = false;
                } else if constexpr (PAIR) {
                    load_box<CG>(to, &p.a[0], bar, k * 64, t.row * S::M + rank * 128);
                    if constexpr (CG == 2) {
                        load_box<CG>(to + S::A_BYTES, &p.b[rank], bar, k * 64, t.col * S::NF);
                    } else {
                        load_box<CG>(to + S::A_BYTES, &p.b[0], bar, k * 64, t.col * S::NF);
                        load_box<CG>(to + S::A_BYTES + S::B_BYTES / 2, &p.b[1], bar, k * 64, t.col * S::NF);
                    }
                } else if constexpr (WHICH == kTokens) {
                    const unsigned half = k >= p.steps / 2, at = (k - half * (p.steps / 2)) * 64;
                    load_box<CG>(to, &p.a[half], bar, at, t.row * S::M + rank * 128);
#pragma unroll
                    for (int j = 0; j < NT / CG / 64; ++j)
                        load_box<CG>(to + S::A_BYTES + j * 8192, &p.b[half], bar, t.col * NT + rank * (NT / 2) + j * 64, at);
                } else {
                    const unsigned half = t.row >= p.rows / 2, row = (t.row - half * (p.rows / 2)) * S::M + rank * 128;
#pragma unroll
                    for (int j = 0; j < 2; ++j) load_box<CG>(to + j * 8192, &p.a[half], bar, row + j * 64, k * 64);
#pragma unroll
                    for (int j = 0; j < NT / CG / 64; ++j)
                        load_box<CG>(to + S::A_BYTES + j * 8192, &p.b[0], bar, t.col * NT + rank * (NT / 2) + j * 64, k * 64);
                }
                if (++s == S::STAGES) {
                    s = 0;
                    parity ^= 1u;
                }
            }
        }
        if (!ok) settle();
    } else if (warp == 1 && lane == 0 && rank == 0) {
        // products
        const uint32_t bf = idesc_bf16(S::M, NT, WEIGHTS, !PAIR), idesc = std::is_same<T, __half>::value ? bf & ~((7u << 7) | (7u << 10)) : bf;
        // rows of 128 bytes: eight make an atom of the swizzle.  Along the summed axis 16 elements are 32 bytes of a row, or where
        // the operand runs along the other axis 16 rows; there the next 64 of that axis are 8 KB on
        const uint64_t da = sdesc(0u, WEIGHTS ? 8192u : 16u, 1024u, 2u), db = sdesc(0u, PAIR ? 16u : 8192u, 1024u, 2u);
        constexpr uint32_t KA = WEIGHTS ? 2048 : 32, KB = PAIR ? 32 : 2048;
        int s = 0;
        uint32_t parity = 0, n = 0;
        bool ok = true;
        for (unsigned i = mine; ok && i < tiles; i += all, ++n) {
            const Tile t = tile_of<WHICH>(p, i);
            const uint32_t buf = n & 1u, acc = tmem + buf * NT;
            ok = CG == 2 ? mbar_spin_cluster(&acc_empty[buf], ((n >> 1) & 1u) ^ 1u, guard, kSiteP)
                         : mbar_spin(&acc_empty[buf], ((n >> 1) & 1u) ^ 1u, guard, kSiteP);
            if (!ok) break;
            tc_fence_after();
            for (unsigned k = t.first; k < t.last; ++k) {
                ok = CG == 2 ? mbar_spin_cluster(&full[s], parity, guard, kSiteKV) : mbar_spin(&full[s], parity, guard, kSiteKV);
                if (!ok) break;
                tc_fence_after();
                const uint32_t at = smem + s * S::STAGE;
#pragma unroll
                for (uint32_t j = 0; j < 4; ++j)
                    mma<CG>(acc, da + ((at + j * KA) >> 4), db + ((at + S::A_BYTES + j * KB) >> 4), idesc, k > t.first || j > 0);
                commit<CG>(&empty[s]);
                if (++s == S::STAGES) {
                    s = 0;
                    parity ^= 1u;
                }
            }
            if (ok) commit<CG>(&acc_full[buf]);
        }
        if (!ok) settle();
    } else if (warp >= 4) {
        // results: warp e takes rows 32 (e & 3) .. of the block and the (e / 4)-th run of columns
        const int e = warp - 4, quarter = e & 3, part = e >> 2;
        const uint32_t staging = smem + S::STAGING + e * S::BUFFERS * 4096;
        float* bias = reinterpret_cast<float*>(raw_smem + (smem - smem_u32(raw_smem)) + S::BIAS) + e * 128;
        const uint32_t row = staging + lane * 128, sw = lane & 7;
        uint32_t n = 0;
        const uint32_t acc_at = CG == 2 ? peer_address(smem_u32(acc_empty), 0) : 0u;
        auto release = [&](uint32_t buf) {   // this warp has read its accumulators
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if constexpr (CG == 2) arrive_remote(acc_at + buf * 8);
                else mbar_arrive(&acc_empty[buf]);
            }
        };
        for (unsigned i = mine; i < tiles; i += all, ++n) {
            const Tile t = tile_of<WHICH>(p, i);
            const uint32_t buf = n & 1u;
            const int m0 = static_cast<int>((WEIGHTS && t.row >= p.rows / 2 ? t.row - p.rows / 2 : t.row) * S::M + rank * 128 + quarter * 32);
            const uint32_t taddr = tmem + buf * NT + (static_cast<uint32_t>(quarter * 32) << 16);
            if constexpr (PAIR) {
                const int f0 = static_cast<int>(t.col * S::NF + part * 64);
                // what the tile needs besides its products
                if (lane == 0) tma_store_wait_read();
                __syncwarp();
                if constexpr (WHICH == kSlopes) {
                    if (p.wide) {
                        if (lane == 0) {
                            mbar_arrive_expect_tx(&dh_full[e], 4096);
                            load_box<1>(staging, &p.in, smem_u32(&dh_full[e]), f0, m0);
                        }
                    } else {
                        const uint16_t* from = static_cast<const uint16_t*>(p.dh);
                        for (int r = 0; r < 32; ++r) {
                            uint32_t w = 0;
#pragma unroll
                            for (int j = 0; j < 2; ++j)
                                if (m0 + r < p.T && f0 + 2 * lane + j < p.F)
                                    w |= static_cast<uint32_t>(from[static_cast<long long>(m0 + r) * p.F + f0 + 2 * lane + j]) << (16 * j);
                            asm volatile("st.shared.b32 [%0], %1;" ::"r"(staging + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4), "r"(w) : "memory");
                        }
                    }
                }
                if (p.bg || p.bu) {
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int f = f0 + lane + 32 * j;
                        bias[lane + 32 * j] = p.bg && f < p.F ? widen<T>(p.bg, f) : 0.f;
                        bias[64 + lane + 32 * j] = p.bu && f < p.F ? widen<T>(p.bu, f) : 0.f;
                    }
                }
                __syncwarp();
                bool ok = mbar_wait(&acc_full[buf], (n >> 1) & 1u, guard, kSiteFinal);
                if constexpr (WHICH == kSlopes)
                    if (p.wide) ok = ok && mbar_wait(&dh_full[e], n & 1u, guard, kSiteQ);
                if (!__all_sync(0xffffffffu, ok)) {
                    settle();
                    break;
                }
                tc_fence_after();
                uint32_t g[2][16], u[2][16];
                tmem_ld16(taddr + part * 64, g[0]);
                tmem_ld16(taddr + S::NF + part * 64, u[0]);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    tmem_ld_wait_all();
                    reg_fence16(g[c & 1]);
                    reg_fence16(u[c & 1]);
                    if (c < 3) {
                        tmem_ld16(taddr + part * 64 + (c + 1) * 16, g[(c + 1) & 1]);
                        tmem_ld16(taddr + S::NF + part * 64 + (c + 1) * 16, u[(c + 1) & 1]);
                    } else {
                        release(buf);
                    }
                    float fg[16], fu[16];
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        fg[k] = __uint_as_float(g[c & 1][k]);
                        fu[k] = __uint_as_float(u[c & 1][k]);
                    }
                    if (p.bg || p.bu) {
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            fg[k] += bias[c * 16 + k];
                            fu[k] += bias[64 + c * 16 + k];
                        }
                    }
                    const uint32_t at0 = row + ((2 * c) ^ sw) * 16, at1 = row + ((2 * c + 1) ^ sw) * 16;
                    uint32_t w[8], v[8];
                    if constexpr (WHICH == kSlopes) {
                        const uint4 a = ld_shared_v4(at0), b = ld_shared_v4(at1);
                        w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
                    }
                    with_act(p.act, [&](auto tag) {
                        constexpr int ACT = decltype(tag)::value;
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            float a0, a1, s0, s1;
                            activate<ACT, true>(fg[2 * k], a0, s0);
                            activate<ACT, true>(fg[2 * k + 1], a1, s1);
                            if constexpr (WHICH == kForward) {
                                w[k] = Elem<T>::pair(a0 * fu[2 * k], a1 * fu[2 * k + 1]);
                            } else {
                                float d0, d1;
                                Elem<T>::two(w[k], d0, d1);
                                w[k] = Elem<T>::pair(d0 * fu[2 * k] * s0, d1 * fu[2 * k + 1] * s1);
                                v[k] = Elem<T>::pair(d0 * a0, d1 * a1);
                            }
                        }
                    });
                    st_shared_v4(at0, w[0], w[1], w[2], w[3]);
                    st_shared_v4(at1, w[4], w[5], w[6], w[7]);
                    if constexpr (WHICH == kSlopes) {
                        st_shared_v4(at0 + 4096, v[0], v[1], v[2], v[3]);
                        st_shared_v4(at1 + 4096, v[4], v[5], v[6], v[7]);
                    }
                }
                if (WHICH == kSlopes || p.wide) {
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        if (f0 < p.F && m0 < p.T) {
                            store_box(&p.out[0], staging, f0, m0);
                            if constexpr (WHICH == kSlopes) store_box(&p.out[1], staging + 4096, f0, m0);
                        }
                        tma_store_commit();
                    }
                } else {
                    __syncwarp();
                    uint16_t* to = static_cast<uint16_t*>(p.h);
                    for (int r = 0; r < 32 && m0 + r < p.T; ++r) {
                        uint32_t w;
                        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w) : "r"(staging + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4) : "memory");
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            if (f0 + 2 * lane + j < p.F) to[static_cast<long long>(m0 + r) * p.F + f0 + 2 * lane + j] = static_cast<uint16_t>(w >> (16 * j));
                    }
                }
            } else {
                const int c0 = static_cast<int>(t.col * NT + part * S::OUT);
                if (!__all_sync(0xffffffffu, mbar_wait(&acc_full[buf], (n >> 1) & 1u, guard, kSiteFinal))) {
                    settle();
                    break;
                }
                tc_fence_after();
                const unsigned half = WEIGHTS && t.row >= p.rows / 2;
                uint32_t v[2][16];
                tmem_ld16(taddr + part * S::OUT, v[0]);
                constexpr int PIECES = S::OUT / 16;
#pragma unroll
                for (int c = 0; c < PIECES; ++c) {
                    // a buffer holds 64 columns of 2 bytes or 32 of 4
                    const int per = p.split ? 2 : 4, at = c % per;
                    const uint32_t box = (c / per) & 1;
                    if (at == 0) {   // the store before the last has read this buffer
                        if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
                        __syncwarp();
                    }
                    tmem_ld_wait_all();
                    reg_fence16(v[c & 1]);
                    if (c + 1 < PIECES) tmem_ld16(taddr + part * S::OUT + (c + 1) * 16, v[(c + 1) & 1]);
                    else release(buf);
                    const uint32_t to = row + box * 4096;
                    if (p.split) {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            st_shared_v4(to + ((4 * at + j) ^ sw) * 16, v[c & 1][4 * j], v[c & 1][4 * j + 1], v[c & 1][4 * j + 2], v[c & 1][4 * j + 3]);
                    } else {
                        uint32_t w[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j) w[j] = Elem<T>::pair(__uint_as_float(v[c & 1][2 * j]), __uint_as_float(v[c & 1][2 * j + 1]));
                        st_shared_v4(to + ((2 * at) ^ sw) * 16, w[0], w[1], w[2], w[3]);
                        st_shared_v4(to + ((2 * at + 1) ^ sw) * 16, w[4], w[5], w[6], w[7]);
                    }
                    if (at == per - 1) {
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            const int x = c0 + (c / per) * per * 16;
                            if (x < p.D && m0 < (WEIGHTS ? p.F : p.T)) {
                                if (p.split) store_box(&p.out[0], staging + box * 4096, x, m0, WEIGHTS ? t.split * 2 + half : t.split);
                                else store_box(&p.out[half], staging + box * 4096, x, m0);
                            }
                            tma_store_commit();   // an empty group too: the waits count groups
                        }
                    }
                }
            }
        }
        if (lane == 0) tma_store_wait_all();
        tc_fence_before();
    }
    __syncwarp();
    if constexpr (CG == 2) cluster_sync();
    else __syncthreads();
    tc_fence_after();
    if (warp == 2) tmem_give<CG>(tmem, 2 * NT);
}

// ---------------------------------------------------------------------------------------------
// Few tokens (forward and slopes): the weights are the rows of the product, 64 of Wg above 64 of Wu, and the NTOK tokens its
// columns, so a step of 64 along the summed axis brings 16 KB of weights, read once, beside 2 KB of 16 tokens.  A tile's sum
// is cut over the blocks of a cluster where there are few tiles; the others' sums come to the first one by distributed shared
// memory, in order.  The factors of an element are then in rows 64 apart: u goes through shared memory.
// ---------------------------------------------------------------------------------------------

template <int NTOK>
struct FewShape {
    static constexpr uint32_t A_BYTES = 128 * 128, STAGE = A_BYTES + NTOK * 128;
    static constexpr int STAGES = NTOK == 16 ? 6 : (NTOK == 64 ? 4 : 3);   // two blocks to a multiprocessor
    static constexpr int COLS = NTOK < 32 ? 32 : NTOK;                       // of TMEM
    static constexpr int THREADS = 192;
    static constexpr uint32_t BYTES = STAGES * STAGE + 1024;
    static_assert(NTOK * (512 + 256) <= STAGES * STAGE, "the sums and u of a tile take the stages' place");
};

template <int WHICH, int NTOK, typename T>
__global__ void __launch_bounds__(192) glu_few_kernel(const __grid_constant__ GluTcParams p) {
    using S = FewShape<NTOK>;
    extern __shared__ uint8_t raw_smem[];
    __shared__ uint64_t full[S::STAGES], empty[S::STAGES], done;
    __shared__ uint32_t tmem_base;
    const uint32_t smem = (smem_u32(raw_smem) + 1023u) & ~1023u;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const unsigned rank = p.splits > 1 ? cluster_rank() : 0u;
    const int f0 = static_cast<int>(blockIdx.x / p.splits * 64);
    const unsigned first = rank * p.run, last = min(p.steps, first + p.run);
    const WaitGuard guard{p.err, p.wait_ns};
    if (threadIdx.x == 0) {
        for (int s = 0; s < S::STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(&done, 1);
        fence_barrier_init();
    }
    if (warp == 1) tmem_take<1>(&tmem_base, S::COLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base;
    bool ok = true;
    if (warp == 0 && lane == 0) {
        bool withhold = p.withhold && blockIdx.x == 0;
        for (unsigned k = first; k < last; ++k) {
            const unsigned n = k - first, s = n % S::STAGES;
            if (!(ok = mbar_spin(&empty[s], (n / S::STAGES & 1u) ^ 1u, guard, kSiteEmpty))) break;
            const uint32_t to = smem + s * S::STAGE, bar = smem_u32(&full[s]);
            mbar_arrive_expect_tx(&full[s], S::STAGE);
            if (withhold) {   // test hook: the first copy never lands
                withhold = false;
                continue;
            }
            load_box<1>(to, &p.b[0], bar, k * 64, f0);
            load_box<1>(to + 8192, &p.b[1], bar, k * 64, f0);
            load_box<1>(to + S::A_BYTES, &p.a[0], bar, k * 64, 0);
        }
        if (!ok) settle();
    } else if (warp == 1 && lane == 0) {
        const uint32_t bf = idesc_bf16(128, NTOK, false, false), idesc = std::is_same<T, __half>::value ? bf & ~((7u << 7) | (7u << 10)) : bf;
        const uint64_t d = sdesc(0u, 16u, 1024u, 2u);
        for (unsigned k = first; k < last; ++k) {
            const unsigned n = k - first, s = n % S::STAGES;
            if (!(ok = mbar_spin(&full[s], n / S::STAGES & 1u, guard, kSiteKV))) break;
            tc_fence_after();
            const uint32_t at = smem + s * S::STAGE;
#pragma unroll
            for (uint32_t j = 0; j < 4; ++j) umma_bf16(tmem, d + ((at + j * 32) >> 4), d + ((at + S::A_BYTES + j * 32) >> 4), idesc, n > 0 || j > 0);
            umma_commit(&empty[s]);
        }
        if (ok) umma_commit(&done);
        else settle();
    } else if (warp >= 2) {
        ok = __all_sync(0xffffffffu, mbar_wait(&done, 0, guard, kSiteFinal));
        if (!ok) settle();
        tc_fence_after();
    }
    __syncwarp();
    // every copy of this block has landed and been read: the stages' memory holds the sums [token][row], then u [token][column]
    const int quarter = warp & 3, row = quarter * 32 + lane;
    const uint32_t taddr = tmem + (static_cast<uint32_t>(quarter * 32) << 16), sums = smem, us = smem + NTOK * 512;
    if (p.splits > 1) {
        if (warp >= 2 && rank > 0) {
#pragma unroll 1
            for (int c = 0; c < NTOK; c += 16) {
                uint32_t v[16];
                tmem_ld16(taddr + c, v);
                tmem_ld_wait_all();
                reg_fence16(v);
#pragma unroll
                for (int k = 0; k < 16; ++k) st_shared_f32(sums + ((c + k) * 128 + row) * 4, __uint_as_float(v[k]));
            }
        }
        __syncwarp();
        cluster_sync();
    }
    if (warp >= 2 && rank == 0) {
        const int f = f0 + (row & 63);
        const bool gate = row < 64;
        const void* b = gate ? p.bg : p.bu;
        const float bias = b && f < p.F ? widen<T>(b, f) : 0.f;
        auto sixteen = [&](int c, float (&v)[16]) {
            uint32_t r[16];
            tmem_ld16(taddr + c, r);
            tmem_ld_wait_all();
            reg_fence16(r);
#pragma unroll
            for (int k = 0; k < 16; ++k) v[k] = __uint_as_float(r[k]);
            for (unsigned q = 1; q < p.splits; ++q) {
                const uint32_t from = peer_address(sums + (c * 128 + row) * 4, q);
#pragma unroll
                for (int k = 0; k < 16; ++k) v[k] += ld_cluster(from + k * 512);
            }
#pragma unroll
            for (int k = 0; k < 16; ++k) v[k] += bias;
        };
        if (!gate) {
#pragma unroll 1
            for (int c = 0; c < NTOK; c += 16) {
                if (c >= p.T) break;
                float u[16];
                sixteen(c, u);
#pragma unroll
                for (int k = 0; k < 16; ++k) st_shared_f32(us + ((c + k) * 64 + row - 64) * 4, u[k]);
            }
        }
        named_bar_sync(1, 128);
        if (gate) {
#pragma unroll 1
            for (int c = 0; c < NTOK; c += 16) {
                if (c >= p.T) break;
                float g[16];
                sixteen(c, g);
                with_act(p.act, [&](auto tag) {
                    constexpr int ACT = decltype(tag)::value;
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        const long long t = c + k;
                        if (t >= p.T || f >= p.F || !ok) break;
                        float u, a, slope;
                        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(u) : "r"(us + ((c + k) * 64 + row) * 4) : "memory");
                        activate<ACT, true>(g[k], a, slope);
                        if constexpr (WHICH == kForward) {
                            static_cast<T*>(p.h)[t * p.F + f] = Elem<T>::put(a * u);
                        } else {
                            const float dh = widen<T>(p.dh, t * p.F + f);
                            static_cast<T*>(p.dg)[t * p.pitch + f] = Elem<T>::put(dh * u * slope);
                            static_cast<T*>(p.du)[t * p.pitch + f] = Elem<T>::put(dh * a);
                        }
                    }
                });
            }
        }
        tc_fence_before();
    }
    __syncwarp();
    if (p.splits > 1) cluster_sync();   // the first block has read the others' sums
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_give<1>(tmem, S::COLS);
}

// ---------------------------------------------------------------------------------------------
// Launches (instances: na_glu_*.cu)
// ---------------------------------------------------------------------------------------------

template <typename Kernel>
na_status launch_glu(Kernel* kernel, const GluTcParams& p, unsigned blocks, int cluster, int threads, uint32_t bytes, cudaStream_t s) {
    if (!allow_shared(reinterpret_cast<const void*>(kernel))) return NA_ERR_CUDA;
    cudaLaunchConfig_t c{};
    c.gridDim = dim3(blocks);
    c.blockDim = dim3(threads);
    c.dynamicSmemBytes = bytes;
    c.stream = s;
    cudaLaunchAttribute a{};
    a.id = cudaLaunchAttributeClusterDimension;
    a.val.clusterDim.x = cluster;
    a.val.clusterDim.y = a.val.clusterDim.z = 1;
    c.attrs = &a;
    c.numAttrs = cluster > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&c, kernel, p) == cudaSuccess ? NA_OK : NA_ERR_CUDA;
}

// pairs: tiles of 256 x 256 on pairs of blocks, else of 128 x 128.
template <int WHICH, typename T>
na_status launch_tiles(const GluTcParams& p, bool pairs, cudaStream_t s) {
    const unsigned tiles = p.rows * p.cols * p.splits;
    if (pairs) {
        using S = TileShape<WHICH, 2, 256>;
        return launch_glu(glu_tile_kernel<WHICH, 2, 256, T>, p, 2 * (tiles < kSms / 2 ? tiles : kSms / 2), 2, S::THREADS, S::BYTES, s);
    }
    using S = TileShape<WHICH, 1, 128>;
    return launch_glu(glu_tile_kernel<WHICH, 1, 128, T>, p, tiles < kSms ? tiles : kSms, 1, S::THREADS, S::BYTES, s);
}

template <int WHICH, typename T>
na_status launch_few(const GluTcParams& p, int tokens, cudaStream_t s) {
    const unsigned blocks = p.rows * p.splits;
    if (tokens == 16) return launch_glu(glu_few_kernel<WHICH, 16, T>, p, blocks, p.splits, 192, FewShape<16>::BYTES, s);
    if (tokens == 64) return launch_glu(glu_few_kernel<WHICH, 64, T>, p, blocks, p.splits, 192, FewShape<64>::BYTES, s);
    return launch_glu(glu_few_kernel<WHICH, 128, T>, p, blocks, p.splits, 192, FewShape<128>::BYTES, s);
}

}  // namespace glu
}  // namespace na
