// na_glu_tc.cuh -- tensor-core kernels of the gated feed-forward product (bf16 or fp16 operands, fp32 accumulators).
//
// A product's result is cut into tiles, up to 256 x 256 for a pair of blocks (tcgen05.mma with cta_group::2: each block holds 128
// rows and half of the columns' operand) or 128 x 128 for one block.  Blocks stay and take tiles in turn.  Per tile, steps of
// 64 along the summed axis come by TMA through rings in shared memory (128-byte swizzle), one thread issues the products, and
// eight to sixteen warps take the finished accumulators from TMEM while the next tile's products fill the other half of it.
//   forward, slopes   rows: tokens; columns: as many of g as of u, so that both factors of an element meet in one thread
//   tokens            dx: rows: tokens; columns: channels; summed over the columns of dg, then of du
//   weights           dWg, dWu: rows: columns of dg or du; columns: channels; summed over tokens, operands turned by the
//                     descriptors (both run along the other axis in memory)
// Few tokens have a kernel of their own (glu_few_kernel), which streams the weights as the rows of the product (1 token, 1024 ->
// 2736: 5.5 us; the weights' bytes alone take 1.7).
//
// Every wait is bounded (na_device.cuh).
#pragma once

#include <algorithm>
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
// Relaxed: what it tells of, loads from TMEM, is ordered by the tcgen05 fences.  A release to the cluster waits for the warp's
// stores to global memory first (most of the warps' time: 756 us against 651 for the 1024^2 tokens when this was changed).
__device__ __forceinline__ void arrive_remote(uint32_t bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ float ld_cluster(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// The warps that issue copies and products run as whole warps, one elected lane issuing: operands then stay in uniform registers
// (one lane alone spent 70 cycles on a product, and its 285 a step bounded the kernel).  A spinning wait of a whole warp; its
// clock is first read after 64 tests: these warps wait at every step, mostly shorter than that read takes.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const WaitGuard& err, unsigned site) {
    unsigned long long t0 = 0;
    for (uint32_t i = 1;; ++i) {
        if (__all_sync(0xffffffffu, mbar_test(bar, parity))) return true;
        if ((i & 63u) == 0u) {
            const unsigned long long now = globaltimer();
            if (t0 == 0) t0 = now;
            if (__any_sync(0xffffffffu, ld_volatile(err.word) != 0u || now - t0 > err.limit_ns)) {
                record_error(err.word, site);
                return false;
            }
        }
    }
}
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
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
__device__ __forceinline__ void st_shared_b32(uint32_t addr, uint32_t v) { asm volatile("st.shared.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory"); }
__device__ __forceinline__ uint32_t ld_shared_b32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
// Word w of row r of a buffer with rows of 64 bytes in 64-byte swizzle.
__device__ __forceinline__ uint32_t word_at(uint32_t base, int r, int w) { return base + r * 64 + (((w >> 2) ^ ((r >> 1) & 3)) << 4) + (w & 3) * 4; }
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}

// The sums over a warp's lanes of eight columns, of column lane / 4 to each lane: lanes hand one another the half of the columns that
// is not theirs (nine shuffles for 40).
__device__ __forceinline__ float columns_sum(float (&v)[8], int lane) {
#pragma unroll
    for (int half = 4; half >= 1; half /= 2) {
        const bool upper = lane & 4 * half;
#pragma unroll
        for (int k = 0; k < half; ++k) {
            const float away = upper ? v[k] : v[k + half];
            v[k] = (upper ? v[k + half] : v[k]) + __shfl_xor_sync(0xffffffffu, away, 4 * half);
        }
    }
    v[0] += __shfl_xor_sync(0xffffffffu, v[0], 2);
    return v[0] + __shfl_xor_sync(0xffffffffu, v[0], 1);
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

// Item i of rows x cols, by bands of rows, down the columns of a band.
struct Place {
    unsigned row, col;
};
__device__ __forceinline__ Place place_of(unsigned i, unsigned rows, unsigned cols) {
    const unsigned band = i / (kBand * cols), base = band * kBand, height = min(kBand, rows - base);
    i -= base * cols;
    return {base + i % height, i / height};
}

// ---------------------------------------------------------------------------------------------
// Forward and slopes.  A tile: 128 CG rows of tokens, 64 CG columns of g and the same of u, fewer of them in the last of a row.  The
// rows' and the columns' operand have rings of their own: where all of a row of tiles' operand (its steps of 64) fits its ring,
// it is brought once for the `span` columns of tiles that a block takes in a row, which halves what comes out of L2, the bound
// of short sums (1024^2 tokens, 256 -> 688, 2-byte: 535 us, 13 TB/s).  Long sums run at 1560 TFLOP/s (4095 tokens, 4096 -> 11008:
// 472 us).  The epilogue has sixteen (eight) warps, each for 32 rows by 32 columns.  Every block copies what it and its pair
// read itself: the library also runs as one of several ranks, each on a GPU of its own, and no load of it goes to several blocks.
// ---------------------------------------------------------------------------------------------

template <int WHICH, int CG>
struct PairShape {
    static constexpr int NF = 64 * CG;                           // most columns of g of a tile
    static constexpr int M = 128 * CG;                           // rows of a tile
    static constexpr uint32_t SLOT = 128 * 128;                  // either ring's
    static constexpr int ROWS = kPairRows<WHICH>, COLS = WHICH == kForward ? 5 : 4;   // slots
    static constexpr int PARTS = NF / 32, WARPS = 4 * PARTS;     // of the epilogue
    static constexpr uint32_t WARP_STAGING = WHICH == kForward ? 2048 : 4096;   // 32 rows of 64 bytes: results; dh
    static constexpr int THREADS = 128 + 32 * WARPS;
    static constexpr uint32_t TMEM = 256;                        // columns of one of the two accumulators
    static constexpr uint32_t STAGING = (ROWS + COLS) * SLOT, BIAS = STAGING + WARPS * WARP_STAGING;
    static constexpr uint32_t BYTES = BIAS + WARPS * 64 * 4 + 1024;   // 1024: to align the start
    static_assert(BYTES <= 227 * 1024 - 512, "more than a block's shared memory");
};

// The tiles of a block, in order.
template <int CG>
struct PairWalk {
    const GluTcParams& p;
    unsigned item, items, row, col, end;   // tile (row, col); the item ends before column `end`
    __device__ __forceinline__ explicit PairWalk(const GluTcParams& q) : p(q), item(blockIdx.x / CG), items(q.rows * q.groups) { open(); }
    __device__ __forceinline__ void open() {
        if (item >= items) return;
        const Place at = place_of(item, p.rows, p.groups);
        row = at.row;
        col = at.col * p.span;
        end = min(p.cols, col + p.span);
    }
    __device__ __forceinline__ bool more() const { return item < items; }
    __device__ __forceinline__ void next() {
        if (++col < end) return;
        item += gridDim.x / CG;
        open();
    }
};

// SUMS: also the sums of dg and du over a warp's 32 rows.
template <int WHICH, int CG, bool SUMS, typename T>
__global__ void __launch_bounds__(PairShape<WHICH, CG>::THREADS, 1) glu_pair_kernel(const __grid_constant__ GluTcParams p) {
    using S = PairShape<WHICH, CG>;
    using Walk = PairWalk<CG>;
    extern __shared__ uint8_t raw_smem[];
    __shared__ uint64_t rows_full[S::ROWS], rows_empty[S::ROWS], cols_full[S::COLS], cols_empty[S::COLS], acc_full[2], acc_empty[2], dh_full[S::WARPS];
    __shared__ uint32_t tmem_base;
    const uint32_t smem = (smem_u32(raw_smem) + 1023u) & ~1023u;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = CG == 2 ? cluster_rank() : 0u;   // the block in its pair
    const WaitGuard guard{p.err, p.wait_ns};
    if (threadIdx.x == 0) {
        for (int s = 0; s < S::ROWS; ++s) {
            mbar_init(&rows_full[s], 1);
            mbar_init(&rows_empty[s], 1);
        }
        for (int s = 0; s < S::COLS; ++s) {
            mbar_init(&cols_full[s], 1);
            mbar_init(&cols_empty[s], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_empty[i], CG * S::WARPS);
        }
        for (int i = 0; i < S::WARPS; ++i) mbar_init(&dh_full[i], 1);
        fence_barrier_init();
    }
    if (warp == 2) tmem_take<CG>(&tmem_base, 2 * S::TMEM);
    tc_fence_before();
    __syncthreads();
    if constexpr (CG == 2) cluster_sync();
    tc_fence_after();
    const uint32_t tmem = tmem_base;
    if constexpr (WHICH == kSlopes) next_may_start();

    if (warp == 0) {
        // copies
        const uint32_t rows_at = CG == 2 ? peer_address(smem_u32(rows_full), 0) : smem_u32(rows_full);   // the leading block's barriers
        const uint32_t cols_at = CG == 2 ? peer_address(smem_u32(cols_full), 0) : smem_u32(cols_full);
        uint32_t sa = 0, pa = 1, sb = 0, pb = 1;
        const bool leader = elect_one();
        bool ok = true, withhold = p.withhold && blockIdx.x == 0, fresh = true;
        for (Walk w(p); ok && w.more();) {
            for (unsigned k = 0; k < p.steps; ++k) {
                if (fresh) {
                    if (!(ok = warp_wait(&rows_empty[sa], pa, guard, kSiteEmpty))) break;
                    if (leader) {
                        if (rank == 0) mbar_arrive_expect_tx(&rows_full[sa], CG * S::SLOT);
                        // test hook: the first copy never lands
                        if (!withhold) load_box<CG>(smem + sa * S::SLOT, &p.a[0], rows_at + sa * 8, k * 64, w.row * S::M + rank * 128);
                    }
                    withhold = false;
                    if (++sa == S::ROWS) {
                        sa = 0;
                        pa ^= 1u;
                    }
                }
                if (!(ok = warp_wait(&cols_empty[sb], pb, guard, kSiteEmpty))) break;
                const unsigned at = w.col + 1 == p.cols ? 2 : 0, nf = at ? p.last_nf : S::NF;
                const uint32_t to = smem + (S::ROWS + sb) * S::SLOT, bar = cols_at + sb * 8;
                if (leader) {
                    if (rank == 0) mbar_arrive_expect_tx(&cols_full[sb], 2 * nf * 128);   // of both blocks
                    if constexpr (CG == 2) {
                        load_box<CG>(to, &p.b[at + rank], bar, k * 64, w.col * S::NF);
                    } else {
                        load_box<CG>(to, &p.b[at], bar, k * 64, w.col * S::NF);
                        load_box<CG>(to + nf * 128, &p.b[at + 1], bar, k * 64, w.col * S::NF);
                    }
                }
                if (++sb == S::COLS) {
                    sb = 0;
                    pb ^= 1u;
                }
            }
            const unsigned item = w.item;
            w.next();
            fresh = w.item != item;
        }
        if (!ok) settle();
    } else if (warp == 1 && rank == 0) {
        // products.  Rows of 128 bytes, eight to an atom of the swizzle; 16 elements along the summed axis are 32 bytes of a row
        constexpr uint32_t TYPES = std::is_same<T, __half>::value ? ~((7u << 7) | (7u << 10)) : ~0u;
        const uint64_t desc = sdesc(0u, 16u, 1024u, 2u);
        uint32_t sa0 = 0, pa0 = 0, sb = 0, pb = 0, n = 0;   // sa0, pa0: of the item's first step
        const bool leader = elect_one();
        bool ok = true, fresh = true;
        for (Walk w(p); ok && w.more(); ++n) {
            const uint32_t buf = n & 1u, acc = tmem + buf * S::TMEM;
            if (!(ok = warp_wait(&acc_empty[buf], ((n >> 1) & 1u) ^ 1u, guard, kSiteP))) break;
            tc_fence_after();
            const bool last = w.col + 1 == w.end;
            const uint32_t idesc = idesc_bf16(S::M, 2 * (w.col + 1 == p.cols ? p.last_nf : S::NF), false, false) & TYPES;
            uint32_t sa = sa0, pa = pa0;
            for (unsigned k = 0; k < p.steps; ++k) {
                if (fresh && !(ok = warp_wait(&rows_full[sa], pa, guard, kSiteKV))) break;
                if (!(ok = warp_wait(&cols_full[sb], pb, guard, kSiteKV))) break;
                tc_fence_after();
                const uint32_t at = smem + sa * S::SLOT, bt = smem + (S::ROWS + sb) * S::SLOT;
                if (leader) {
#pragma unroll
                    for (uint32_t j = 0; j < 4; ++j) mma<CG>(acc, desc + ((at + j * 32) >> 4), desc + ((bt + j * 32) >> 4), idesc, k > 0 || j > 0);
                    commit<CG>(&cols_empty[sb]);
                    if (last) commit<CG>(&rows_empty[sa]);
                }
                if (++sa == S::ROWS) {
                    sa = 0;
                    pa ^= 1u;
                }
                if (++sb == S::COLS) {
                    sb = 0;
                    pb ^= 1u;
                }
            }
            if (ok && leader) commit<CG>(&acc_full[buf]);
            const unsigned item = w.item;
            w.next();
            fresh = w.item != item;
            if (fresh) {
                sa0 = sa;
                pa0 = pa;
            }
        }
        if (!ok) settle();
    } else if (warp >= 4) {
        // results: warp e takes rows 32 (e & 3) .. of the block and 32 columns
        const int e = warp - 4, quarter = e & 3, part = e >> 2;
        const uint32_t staging = smem + S::STAGING + e * S::WARP_STAGING, dh_at = staging + 2048;
        float* bias = reinterpret_cast<float*>(raw_smem + (smem - smem_u32(raw_smem)) + S::BIAS) + e * 64;
        const uint32_t acc_at = CG == 2 ? peer_address(smem_u32(acc_empty), 0) : 0u;
        auto release = [&](uint32_t buf) {   // this warp has read its accumulators
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if constexpr (CG == 2) arrive_remote(acc_at + buf * 8);
                else mbar_arrive(&acc_empty[buf]);
            }
        };
        auto row_of = [&](const Walk& w) { return static_cast<int>(w.row * S::M + rank * 128 + quarter * 32); };
        auto col_of = [&](const Walk& w) { return static_cast<int>(w.col * S::NF + part * 32); };
        auto fetch = [&](const Walk& w) {   // a tile's dh, ahead of it
            if (lane == 0 && w.more()) {
                mbar_arrive_expect_tx(&dh_full[e], 2048);
                load_box<1>(dh_at, &p.in, smem_u32(&dh_full[e]), col_of(w), row_of(w));
            }
        };
        // where rows are not whole chunks: two rows at a time, a lane two columns, as a word if rows are whole words
        auto by_elements = [&](int m0, int f0) {
            __syncwarp();
            const int r0 = lane >> 4, c = 2 * (lane & 15), n = min(32, p.T - m0);
            const bool first = f0 + c < p.F, second = f0 + c + 1 < p.F, words = p.F % 2 == 0;
            uint16_t* out = static_cast<uint16_t*>(p.h) + static_cast<long long>(m0 + r0) * p.F + f0 + c;
            const long long step = 2LL * p.F;
#pragma unroll
            for (int r = 0; r < 32; r += 2, out += step) {
                const uint32_t w = ld_shared_b32(word_at(staging, r + r0, lane & 15));
                if (r + r0 >= n) continue;
                if (words) {
                    if (first) *reinterpret_cast<uint32_t*>(out) = w;
                } else {
                    if (first) out[0] = static_cast<uint16_t>(w);
                    if (second) out[1] = static_cast<uint16_t>(w >> 16);
                }
            }
            __syncwarp();
        };
        auto by_tma = [&](const CUtensorMap* map, int m0, int f0) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                store_box(map, staging, f0, m0);
                tma_store_commit();
            }
        };
        const uint32_t row = staging + lane * 64, dh_row = dh_at + lane * 64, sw = (lane >> 1) & 3;   // rows of 64 bytes in 64-byte swizzle
        const bool biased = p.bg || p.bu;
        // a loop for each activation: only one is run
        auto results = [&](auto tag) {
            constexpr int ACT = decltype(tag)::value;
            Walk w(p);
            if constexpr (WHICH == kSlopes) fetch(w);
            for (uint32_t n = 0; w.more(); ++n) {
                const uint32_t buf = n & 1u;
                const int m0 = row_of(w), f0 = col_of(w);
                const uint32_t nf = w.col + 1 == p.cols ? p.last_nf : S::NF;
                const uint32_t taddr = tmem + buf * S::TMEM + (static_cast<uint32_t>(quarter * 32) << 16) + part * 32;
                const bool there = f0 < p.F && m0 < p.T;   // else nothing but to give the accumulators back
                w.next();
                uint32_t dh[16];
                if constexpr (WHICH == kSlopes) {
                    if (!__all_sync(0xffffffffu, mbar_wait(&dh_full[e], n & 1u, guard, kSiteQ))) {
                        settle();
                        break;
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint4 v = ld_shared_v4(dh_row + (j ^ sw) * 16);
                        dh[4 * j] = v.x, dh[4 * j + 1] = v.y, dh[4 * j + 2] = v.z, dh[4 * j + 3] = v.w;
                    }
                    __syncwarp();
                    fetch(w);
                }
                if (biased) {
                    __syncwarp();
                    const bool in = f0 + lane < p.F;
                    bias[lane] = in && p.bg ? widen<T>(p.bg, f0 + lane) : 0.f;
                    bias[32 + lane] = in && p.bu ? widen<T>(p.bu, f0 + lane) : 0.f;
                }
                if (lane == 0) tma_store_wait_read();   // the results before have left the staging
                __syncwarp();
                if (!__all_sync(0xffffffffu, mbar_wait(&acc_full[buf], (n >> 1) & 1u, guard, kSiteFinal))) {
                    settle();
                    break;
                }
                tc_fence_after();
                if (!there) {
                    release(buf);
                    continue;
                }
                // eight columns at a time, the next ones on their way
                uint32_t du[16], rg[2][8], ru[2][8];
                float sum_g = 0.f, sum_u = 0.f;   // of column 8 (lane % 4) + lane / 4
                tmem_ld8(taddr, rg[0]);
                tmem_ld8(taddr + nf, ru[0]);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    tmem_ld_wait2(rg[c & 1], ru[c & 1]);
                    if (c < 3) {
                        tmem_ld8(taddr + (c + 1) * 8, rg[(c + 1) & 1]);
                        tmem_ld8(taddr + nf + (c + 1) * 8, ru[(c + 1) & 1]);
                    } else {
                        release(buf);
                    }
                    float g[8], u[8], a[8], slope[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        g[k] = __uint_as_float(rg[c & 1][k]);
                        u[k] = __uint_as_float(ru[c & 1][k]);
                    }
                    if (biased) {
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            g[k] += bias[c * 8 + k];
                            u[k] += bias[32 + c * 8 + k];
                        }
                    }
                    activate8<ACT>(g, a, slope);
                    uint32_t v[4];
                    float dg8[SUMS ? 8 : 1], du8[SUMS ? 8 : 1];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        if constexpr (WHICH == kForward) {
                            v[k] = Elem<T>::pair(a[2 * k] * u[2 * k], a[2 * k + 1] * u[2 * k + 1]);
                        } else {
                            float d0, d1;
                            Elem<T>::two(dh[4 * c + k], d0, d1);
                            const float dg0 = d0 * u[2 * k] * slope[2 * k], dg1 = d1 * u[2 * k + 1] * slope[2 * k + 1];
                            const float du0 = d0 * a[2 * k], du1 = d1 * a[2 * k + 1];
                            v[k] = Elem<T>::pair(dg0, dg1);
                            du[4 * c + k] = Elem<T>::pair(du0, du1);
                            if constexpr (SUMS) {   // rows past the last token are not there: a bias may make them infinite
                                const bool in = m0 + lane < p.T;
                                dg8[2 * k] = in ? dg0 : 0.f, dg8[2 * k + 1] = in ? dg1 : 0.f;
                                du8[2 * k] = in ? du0 : 0.f, du8[2 * k + 1] = in ? du1 : 0.f;
                            }
                        }
                    }
                    if constexpr (SUMS) {
                        const float tg = columns_sum(dg8, lane), tu = columns_sum(du8, lane);
                        if ((lane & 3) == c) {
                            sum_g = tg;
                            sum_u = tu;
                        }
                    }
                    st_shared_v4(row + (c ^ sw) * 16, v[0], v[1], v[2], v[3]);
                }
                if constexpr (WHICH == kForward) {
                    if (p.wide) by_tma(&p.out[0], m0, f0);
                    else by_elements(m0, f0);
                } else {
                    if constexpr (SUMS) {
                        const int f = f0 + (lane & 3) * 8 + (lane >> 2);
                        float* to = p.sums + static_cast<long long>(m0 / 32) * 2 * p.sum_pitch + f;
                        if (f < p.F) {
                            to[0] = sum_g;
                            to[p.sum_pitch] = sum_u;
                        }
                    }
                    // dg, then du through the same staging
                    by_tma(&p.out[0], m0, f0);
                    if (lane == 0) tma_store_wait_read();
                    __syncwarp();
#pragma unroll
                    for (int j = 0; j < 4; ++j) st_shared_v4(row + (j ^ sw) * 16, du[4 * j], du[4 * j + 1], du[4 * j + 2], du[4 * j + 3]);
                    by_tma(&p.out[1], m0, f0);
                }
            }
        };
        with_act(p.act, results);
        if (lane == 0) tma_store_wait_all();
        tc_fence_before();
    }
    __syncwarp();
    if constexpr (CG == 2) cluster_sync();
    else __syncthreads();
    tc_fence_after();
    if (warp == 2) tmem_give<CG>(tmem, 2 * S::TMEM);
}

// ---------------------------------------------------------------------------------------------
// Tokens and weights: plain products, 256 x 256 on pairs of blocks or 128 x 128.  Where there are few tiles, or the summed axis is
// long, it is cut into splits (their fp32 sums are added by another kernel): `ways` of them side by side, each taking every
// ways-th step, for `run` steps, then the next ones.
// Both products read all of dg and du.  Where these do not fit L2, one launch makes both side by side: some blocks go down the rows
// of dx, the others down the tokens of the weights' sums at the same pace, so that what one side reads the other finds in L2
// (262144 tokens, 256 -> 688: 137 + 136 us one after the other, both bound by memory; 225 together).
// ---------------------------------------------------------------------------------------------

template <int CG>
struct TileShape {
    static constexpr int N = 128 * CG, M = 128 * CG;
    static constexpr uint32_t A_BYTES = 128 * 128, STAGE = 2 * A_BYTES;
    static constexpr int WARPS = 8, OUT = N / 2;                 // of the epilogue; columns of a warp
    static constexpr int STAGES = 5, THREADS = 128 + 32 * WARPS;
    static constexpr uint32_t STAGING = STAGES * STAGE;          // 4 KB a warp: 32 rows of 128 bytes
    static constexpr uint32_t BYTES = STAGING + WARPS * 4096 + 1024;
    static_assert(BYTES <= 227 * 1024 - 512, "more than a block's shared memory");
};

template <int STAGES>
struct TileBarriers {
    uint64_t full[STAGES], empty[STAGES], acc_full[2], acc_empty[2];
};

struct Tile {
    unsigned row, col, split, first, end;   // steps first, first + ways, .. below end
};
__device__ __forceinline__ Tile tile_of(const GluJob& job, unsigned i) {
    const unsigned per = job.rows * job.cols, split = i / per, turn = split / job.ways;
    const Place at = place_of(i - split * per, job.rows, job.cols);
    const unsigned first = turn * job.run * job.ways + split - turn * job.ways;
    return {at.row, at.col, split, first, min(job.steps, first + job.run * job.ways)};
}

// A block's part in one of the products: worker `mine` of `all`.
template <int WHICH, int CG, typename T>
__device__ __forceinline__ void tile_work(const GluTcParams& p, unsigned mine, unsigned all, uint32_t smem, TileBarriers<TileShape<CG>::STAGES>& bars,
                                          uint32_t tmem, uint32_t rank) {
    using S = TileShape<CG>;
    constexpr bool WEIGHTS = WHICH == kWeights;
    const GluJob& job = p.job[WEIGHTS];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const unsigned tiles = job.rows * job.cols * job.splits;
    const WaitGuard guard{p.err, p.wait_ns};
    // dg and du, Wg and Wu are halves: of the summed axis (tokens), of the rows of tiles (weights)
    if (warp == 0) {
        // copies
        const uint32_t full_at = CG == 2 ? peer_address(smem_u32(bars.full), 0) : smem_u32(bars.full);   // the leading block's barriers
        int s = 0;
        uint32_t parity = 1;
        const bool leader = elect_one();
        bool ok = true, withhold = p.withhold && blockIdx.x == 0;
        for (unsigned i = mine; ok && i < tiles; i += all) {
            const Tile t = tile_of(job, i);
            for (unsigned k = t.first; k < t.end; k += job.ways) {
                if (!(ok = warp_wait(&bars.empty[s], parity, guard, kSiteEmpty))) break;
                const uint32_t to = smem + s * S::STAGE, bar = full_at + s * 8;
                const unsigned half = WEIGHTS ? t.row >= job.rows / 2 : k >= job.steps / 2;
                const unsigned row = (WEIGHTS ? t.row - half * (job.rows / 2) : t.row) * S::M + rank * 128, col = t.col * S::N + rank * 128;
                const unsigned at = (WEIGHTS ? k : k - half * (job.steps / 2)) * 64;
                if (leader) {
                    if (rank == 0) mbar_arrive_expect_tx(&bars.full[s], CG * S::STAGE);
                    if (!withhold) {   // test hook: the first copy never lands
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            if constexpr (WEIGHTS) {
                                load_box<CG>(to + j * 8192, &p.a[half], bar, row + j * 64, at);
                                load_box<CG>(to + S::A_BYTES + j * 8192, &p.b[2], bar, col + j * 64, at);
                            } else {
                                load_box<CG>(to + j * 8192, &p.a[half], bar, at, row + j * 64);
                                load_box<CG>(to + S::A_BYTES + j * 8192, &p.b[half], bar, col + j * 64, at);
                            }
                        }
                    }
                }
                withhold = false;
                if (++s == S::STAGES) {
                    s = 0;
                    parity ^= 1u;
                }
            }
        }
        if (!ok) settle();
    } else if (warp == 1 && rank == 0) {
        // products
        const uint32_t bf = idesc_bf16(S::M, S::N, WEIGHTS, true), idesc = std::is_same<T, __half>::value ? bf & ~((7u << 7) | (7u << 10)) : bf;
        // rows of 128 bytes: eight make an atom of the swizzle.  Along the summed axis 16 elements are 32 bytes of a row, or where
        // the operand runs along the other axis 16 rows; there the next 64 of that axis are 8 KB on
        const uint64_t da = sdesc(0u, WEIGHTS ? 8192u : 16u, 1024u, 2u), db = sdesc(0u, 8192u, 1024u, 2u);
        constexpr uint32_t KA = WEIGHTS ? 2048 : 32, KB = 2048;
        int s = 0;
        uint32_t parity = 0, n = 0;
        const bool leader = elect_one();
        bool ok = true;
        for (unsigned i = mine; ok && i < tiles; i += all, ++n) {
            const Tile t = tile_of(job, i);
            const uint32_t buf = n & 1u, acc = tmem + buf * S::N;
            if (!(ok = warp_wait(&bars.acc_empty[buf], ((n >> 1) & 1u) ^ 1u, guard, kSiteP))) break;
            tc_fence_after();
            for (unsigned k = t.first; k < t.end; k += job.ways) {
                if (!(ok = warp_wait(&bars.full[s], parity, guard, kSiteKV))) break;
                tc_fence_after();
                const uint32_t at = smem + s * S::STAGE;
                if (leader) {
#pragma unroll
                    for (uint32_t j = 0; j < 4; ++j)
                        mma<CG>(acc, da + ((at + j * KA) >> 4), db + ((at + S::A_BYTES + j * KB) >> 4), idesc, k > t.first || j > 0);
                    commit<CG>(&bars.empty[s]);
                }
                if (++s == S::STAGES) {
                    s = 0;
                    parity ^= 1u;
                }
            }
            if (ok && leader) commit<CG>(&bars.acc_full[buf]);
        }
        if (!ok) settle();
    } else if (warp >= 4) {
        // results: warp e takes rows 32 (e & 3) .. of the block and the (e / 4)-th half of its columns
        const int e = warp - 4, quarter = e & 3, part = e >> 2;
        const uint32_t staging = smem + S::STAGING + e * 4096;
        const uint32_t row = staging + lane * 128, sw = lane & 7;   // rows of 128 bytes in 128-byte swizzle
        const uint32_t acc_at = CG == 2 ? peer_address(smem_u32(bars.acc_empty), 0) : 0u;
        const bool split = job.splits > 1;
        uint32_t n = 0;
        for (unsigned i = mine; i < tiles; i += all, ++n) {
            const Tile t = tile_of(job, i);
            const uint32_t buf = n & 1u, taddr = tmem + buf * S::N + (static_cast<uint32_t>(quarter * 32) << 16) + part * S::OUT;
            const unsigned half = WEIGHTS && t.row >= job.rows / 2;
            const int m0 = static_cast<int>((t.row - half * (job.rows / 2)) * S::M + rank * 128 + quarter * 32), last_row = WEIGHTS ? p.F : p.T;
            const int c0 = static_cast<int>(t.col * S::N + part * S::OUT);
            float* sums = p.partial + static_cast<long long>(WEIGHTS ? t.split * 2 + half : t.split) * last_row * p.D;
            T* result = static_cast<T*>(!WEIGHTS ? p.dx : half ? p.dwu : p.dwg);
            if (!__all_sync(0xffffffffu, mbar_wait(&bars.acc_full[buf], (n >> 1) & 1u, guard, kSiteFinal))) {
                settle();
                break;
            }
            tc_fence_after();
            uint32_t v[2][16];
            tmem_ld16(taddr, v[0]);
            constexpr int PIECES = S::OUT / 16;
#pragma unroll
            for (int c = 0; c < PIECES; ++c) {
                const int per = split ? 2 : 4, at = c % per;   // the staging holds 64 columns of 2 bytes or 32 of 4
                tmem_ld_wait_all();
                reg_fence16(v[c & 1]);
                if (c + 1 < PIECES) {
                    tmem_ld16(taddr + (c + 1) * 16, v[(c + 1) & 1]);
                } else {   // this warp has read its accumulators
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if constexpr (CG == 2) arrive_remote(acc_at + buf * 8);
                        else mbar_arrive(&bars.acc_empty[buf]);
                    }
                }
                if (split) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        st_shared_v4(row + ((4 * at + j) ^ sw) * 16, v[c & 1][4 * j], v[c & 1][4 * j + 1], v[c & 1][4 * j + 2], v[c & 1][4 * j + 3]);
                } else {
                    uint32_t w[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) w[j] = Elem<T>::pair(__uint_as_float(v[c & 1][2 * j]), __uint_as_float(v[c & 1][2 * j + 1]));
                    st_shared_v4(row + ((2 * at) ^ sw) * 16, w[0], w[1], w[2], w[3]);
                    st_shared_v4(row + ((2 * at + 1) ^ sw) * 16, w[4], w[5], w[6], w[7]);
                }
                if (at == per - 1) {   // out by rows: eight lanes a row
                    __syncwarp();
                    const int r = lane >> 3, col = c0 + (c / per) * per * 16 + (lane & 7) * (split ? 4 : 8);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const uint4 w = ld_shared_v4(staging + (r + 4 * j) * 128 + (((lane & 7) ^ ((r + 4 * j) & 7)) << 4));
                        const long long to = static_cast<long long>(m0 + r + 4 * j) * p.D + col;
                        if (m0 + r + 4 * j < last_row && col < p.D) {
                            if (split) st_stream(sums + to, w);
                            else st_stream(result + to, w);
                        }
                    }
                    __syncwarp();
                }
            }
        }
        tc_fence_before();
    }
}

template <int WHICH, int CG, typename T>
__global__ void __launch_bounds__(TileShape<CG>::THREADS, 1) glu_tile_kernel(const __grid_constant__ GluTcParams p) {
    using S = TileShape<CG>;
    extern __shared__ uint8_t raw_smem[];
    __shared__ TileBarriers<S::STAGES> bars;
    __shared__ uint32_t tmem_base;
    const uint32_t smem = (smem_u32(raw_smem) + 1023u) & ~1023u;
    const int warp = threadIdx.x >> 5;
    const uint32_t rank = CG == 2 ? cluster_rank() : 0u;
    const unsigned mine = blockIdx.x / CG, all = gridDim.x / CG;
    if (threadIdx.x == 0) {
        for (int s = 0; s < S::STAGES; ++s) {
            mbar_init(&bars.full[s], 1);
            mbar_init(&bars.empty[s], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars.acc_full[i], 1);
            mbar_init(&bars.acc_empty[i], CG * S::WARPS);
        }
        fence_barrier_init();
    }
    if (warp == 2) tmem_take<CG>(&tmem_base, 2 * S::N);
    tc_fence_before();
    __syncthreads();
    if constexpr (CG == 2) cluster_sync();
    tc_fence_after();
    const uint32_t tmem = tmem_base;
    after_previous();
    next_may_start();
    if constexpr (WHICH != kBoth) tile_work<WHICH, CG, T>(p, mine, all, smem, bars, tmem, rank);
    else if (mine < p.token_workers) tile_work<kTokens, CG, T>(p, mine, p.token_workers, smem, bars, tmem, rank);
    else tile_work<kWeights, CG, T>(p, mine - p.token_workers, all - p.token_workers, smem, bars, tmem, rank);
    __syncwarp();
    if constexpr (CG == 2) cluster_sync();
    else __syncthreads();
    tc_fence_after();
    if (warp == 2) tmem_give<CG>(tmem, 2 * S::N);
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
    // one step's copies: both weights' rows and the tokens'
    auto load = [&](unsigned k, unsigned s, bool withhold) {
        const uint32_t to = smem + s * S::STAGE, bar = smem_u32(&full[s]);
        mbar_arrive_expect_tx(&full[s], S::STAGE);
        if (withhold) return;   // test hook: the first copy never lands
        load_box<1>(to, &p.b[0], bar, k * 64, f0);
        load_box<1>(to + 8192, &p.b[1], bar, k * 64, f0);
        load_box<1>(to + S::A_BYTES, &p.a[0], bar, k * 64, 0);
    };
    const unsigned ahead = min(last - first, static_cast<unsigned>(S::STAGES));
    if (warp == 0 && elect_one()) {
        for (int s = 0; s < S::STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(&done, 1);
        fence_barrier_init();
        // the first stages need nobody else: their copies are on their way while the block sets up
        for (unsigned n = 0; n < ahead; ++n) load(first + n, n, n == 0 && p.withhold && blockIdx.x == 0);
    }
    if (warp == 1) tmem_take<1>(&tmem_base, S::COLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base;
    bool ok = true;
    if (warp == 0) {
        const bool leader = elect_one();
        for (unsigned n = ahead; n < last - first; ++n) {
            const unsigned s = n % S::STAGES;
            if (!(ok = warp_wait(&empty[s], (n / S::STAGES & 1u) ^ 1u, guard, kSiteEmpty))) break;
            if (leader) load(first + n, s, false);
        }
        if (!ok) settle();
    } else if (warp == 1) {
        const uint32_t bf = idesc_bf16(128, NTOK, false, false), idesc = std::is_same<T, __half>::value ? bf & ~((7u << 7) | (7u << 10)) : bf;
        const uint64_t d = sdesc(0u, 16u, 1024u, 2u);
        const bool leader = elect_one();
        for (unsigned k = first; k < last; ++k) {
            const unsigned n = k - first, s = n % S::STAGES;
            if (!(ok = warp_wait(&full[s], n / S::STAGES & 1u, guard, kSiteKV))) break;
            tc_fence_after();
            const uint32_t at = smem + s * S::STAGE;
            if (leader) {
#pragma unroll
                for (uint32_t j = 0; j < 4; ++j) umma_bf16(tmem, d + ((at + j * 32) >> 4), d + ((at + S::A_BYTES + j * 32) >> 4), idesc, n > 0 || j > 0);
                umma_commit(&empty[s]);
            }
        }
        if (!ok) settle();
        else if (leader) umma_commit(&done);
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
            float sum_g = 0.f, sum_u = 0.f;   // of dg and du over the tokens
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
                            const float dg = dh * u * slope, du = dh * a;
                            static_cast<T*>(p.dg)[t * p.pitch + f] = Elem<T>::put(dg);
                            static_cast<T*>(p.du)[t * p.pitch + f] = Elem<T>::put(du);
                            sum_g += dg;
                            sum_u += du;
                        }
                    }
                });
            }
            if constexpr (WHICH == kSlopes)
                if (p.sums && f < p.F && ok) {
                    p.sums[f] = sum_g;
                    p.sums[p.sum_pitch + f] = sum_u;
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
na_status launch_glu(Kernel* kernel, const GluTcParams& p, unsigned blocks, int cluster, int threads, uint32_t bytes, cudaStream_t s, bool after = false) {
    if (!allow_shared(reinterpret_cast<const void*>(kernel))) return NA_ERR_CUDA;
    cudaLaunchConfig_t c{};
    c.gridDim = dim3(blocks);
    c.blockDim = dim3(threads);
    c.dynamicSmemBytes = bytes;
    c.stream = s;
    cudaLaunchAttribute a[2]{};
    c.attrs = a;
    if (cluster > 1) {
        a[c.numAttrs].id = cudaLaunchAttributeClusterDimension;
        a[c.numAttrs].val.clusterDim.x = cluster;
        a[c.numAttrs].val.clusterDim.y = a[c.numAttrs].val.clusterDim.z = 1;
        ++c.numAttrs;
    }
    if (after) {   // behind another kernel of the call
        a[c.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        a[c.numAttrs].val.programmaticStreamSerializationAllowed = 1;
        ++c.numAttrs;
    }
    return taken(cudaLaunchKernelEx(&c, kernel, p)) ? NA_OK : NA_ERR_CUDA;
}

template <int WHICH, int CG, typename T>
na_status launch_tiles(const GluTcParams& p, unsigned tiles, cudaStream_t s) {
    const unsigned blocks = CG * std::min<unsigned>(tiles, kSms / CG);
    if constexpr (WHICH == kSlopes)
        if (p.sums) return launch_glu(glu_pair_kernel<WHICH, CG, true, T>, p, blocks, CG, PairShape<WHICH, CG>::THREADS, PairShape<WHICH, CG>::BYTES, s);
    if constexpr (WHICH == kForward || WHICH == kSlopes)
        return launch_glu(glu_pair_kernel<WHICH, CG, false, T>, p, blocks, CG, PairShape<WHICH, CG>::THREADS, PairShape<WHICH, CG>::BYTES, s);
    else
        return launch_glu(glu_tile_kernel<WHICH, CG, T>, p, blocks, CG, TileShape<CG>::THREADS, TileShape<CG>::BYTES, s, true);
}

template <int WHICH, typename T>
na_status launch_tiles(const GluTcParams& p, int blocks, cudaStream_t s) {
    if constexpr (WHICH == kBoth) {
        return launch_tiles<kBoth, 2, T>(p, static_cast<unsigned>(kSms / 2), s);
    } else if constexpr (WHICH == kForward || WHICH == kSlopes) {
        const unsigned items = p.rows * p.groups;
        return blocks == 2 ? launch_tiles<WHICH, 2, T>(p, items, s) : launch_tiles<WHICH, 1, T>(p, items, s);
    } else {
        const GluJob& job = p.job[WHICH == kWeights];
        const unsigned tiles = job.rows * job.cols * job.splits;
        return blocks == 2 ? launch_tiles<WHICH, 2, T>(p, tiles, s) : launch_tiles<WHICH, 1, T>(p, tiles, s);
    }
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
