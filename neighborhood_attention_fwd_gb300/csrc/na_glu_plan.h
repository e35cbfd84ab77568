// na_glu_plan.h -- how the gated feed-forward product and its gradients are cut into tiles, splits and launches, and what their
// workspace holds.  Host code alone, without CUDA: a test compiles it by itself.
#pragma once

#include <algorithm>
#include <cstddef>

#include "../../include/na.h"
#include "na_machine.h"

namespace na {
namespace glu {

// The products.  kForward: h from x and both weights.  kSlopes: the same product again, and dg, du from it and dh.
// kTokens: dx = dg Wg + du Wu.  kWeights: dWg = dg^T x, dWu = du^T x.
// kBoth: these two in one launch.
enum Product { kForward = 0, kSlopes = 1, kTokens = 2, kWeights = 3, kBoth = 4 };

// Steps of the rows' operand that a block of the forward or of the slopes holds.
template <int WHICH>
constexpr int kPairRows = WHICH == kForward ? 6 : 5;

inline unsigned up(long long n, long long by) { return static_cast<unsigned>((n + by - 1) / by); }

// How a product is cut on CUDA cores: tiles of 128 or 32 rows and columns, splits of the summed axis (run: kWeights: tokens of one,
// kTokens: pieces of 16 columns of dg, then du).
struct FmaTile {
    int rows, cols, splits;
    long long run;
};

// Blocks of a product on CUDA cores: tiles of rows, tiles of columns, splits (kWeights: of dWg and dWu each).  A grid has 65535 places
// along z: past 32767 splits (over 2^28 tokens) the others follow along x, behind the rows.
constexpr int kMostZ = 32767;
// Products in one fp32 sum of FMA units at most.  A longer sequence of additions of one value is off by more than a sum's parts add up
// to: 0.3 x 0.7 over 2^18 channels came out 0.3% too small.
constexpr int kMostProducts = 8192;
struct FmaGrid {
    unsigned x, y, z;
};
inline FmaGrid fma_grid(Product which, long long T, int D, int F, const FmaTile& n) {
    if (which == kForward || which == kSlopes) return {up(T, n.rows), up(F, n.cols / 2), 1};
    if (which == kTokens) return {up(T, n.rows), up(D, n.cols), static_cast<unsigned>(n.splits)};
    return {up(F, n.rows) * up(n.splits, kMostZ), up(D, n.cols), 2u * std::min(n.splits, kMostZ)};
}

constexpr int kGluMaxWidth = 1 << 20;              // of D and F
constexpr long long kGluMaxRows = (1LL << 31) - 256;   // a tile's rows are counted in 31 bits

// How a product is cut on tensor cores.
struct GluTiles {
    bool pairs;              // tiles of 256 x 256 on pairs of blocks, else of 128 x 128
    int few;                 // 16, 64, 128: the kernel of few tokens
    unsigned rows, cols, steps, run, splits, ways;
    unsigned last_nf, span, groups;   // forward, slopes
    unsigned workers;                 // tokens and weights in one launch: pairs of blocks for the tokens, 0: apart
    double time;                      // estimated nanoseconds
};

// Nanoseconds of a step of 64 along the summed axis of a tile, for pairs of blocks and for one, and of what a tile takes besides.
constexpr long long kPairStep = 280, kOneStep = 190, kTileTime = 1000;
// Bytes that one product leaves in L2 for the next.
constexpr double kFitsL2 = 80e6;
// The same where the rows' operand stays for several columns of tiles.
constexpr long long kPairStay = 230, kOneStay = 160;
// Steps of 64 products summed in one accumulator at most.  The tensor cores cut their sums instead of rounding them: sums of
// 43691 products of one sign came out 2.5e-4 of their value too small; 24576 are 1.4e-4, about half of fp16's rounding.
constexpr unsigned kMostSteps = 384;

// Cuts the steps into `ways` parts side by side of at most kMostSteps each, and turns of them; false if a part would be empty.
inline bool cut_steps(GluTiles& t, unsigned ways) {
    const unsigned most = up(t.steps, ways), least = t.steps / ways;   // steps of a way
    if (least == 0) return false;
    for (unsigned turns = up(most, kMostSteps); turns <= most; ++turns) {
        t.ways = ways;
        t.run = up(most, turns);
        const unsigned n = up(most, t.run);
        t.splits = ways * n;
        if ((n - 1) * t.run < least) return true;
    }
    return false;
}

inline GluTiles plan_tiles(Product which, long long T, int D, int F) {
    const bool pair = which == kForward || which == kSlopes;
    GluTiles best{};
    if (pair && T <= 128) {
        // As many blocks to a tile's sum as make it shortest, two blocks to a multiprocessor: a step of 64 takes about 0.12 us, a
        // block 8 steps' time to start and end, a cluster of 2 another 7, of 4 another 24 (1 token, 2736 x 1024: 5.7, 5.5 and 7.1 us;
        // of 8 17.7).
        best.few = T <= 16 ? 16 : (T <= 64 ? 64 : 128);
        best.rows = up(F, 64);
        best.cols = 1;
        best.steps = up(D, 64);
        const long long extra[3] = {0, 7, 24};
        long long least = 0;
        for (unsigned i = 0, s = 1; i < 3 && s <= best.steps; ++i, s *= 2) {
            const unsigned run = up(best.steps, s);
            if (up(best.steps, run) != s) continue;   // every block has steps
            const long long time = static_cast<long long>(up(static_cast<long long>(best.rows) * s, 2 * kSms)) * (run + 8) + extra[i];
            if (s == 1 || time < least) {
                least = time;
                best.run = run;
                best.splits = s;
            }
        }
        return best;
    }
    double least = 0;
    for (bool pairs : {false, true}) {
        const int m = pairs ? 256 : 128, slots = pairs ? kSms / 2 : kSms;
        GluTiles t{};
        t.pairs = pairs;
        t.splits = 1;
        if (pair) {
            // a row's last tile is only as wide as it has to be: a product of pairs takes 32 columns (16 of g) at a time, of one
            // block 16
            t.rows = up(T, m);
            t.cols = up(F, m / 2);
            t.last_nf = up(F - (t.cols - 1) * (m / 2), pairs ? 16 : 8) * (pairs ? 16 : 8);
            t.steps = t.run = up(D, 64);
            const unsigned stay = which == kForward ? kPairRows<kForward> : kPairRows<kSlopes>;
            for (unsigned span = 1; span <= t.cols; ++span) {
                if (span > 1 && (t.steps > stay || span > 64)) break;
                const unsigned groups = up(t.cols, span);
                if (span > 1 && up(t.cols, span - 1) == groups) continue;   // no fewer items than with the shorter run
                const double waves = static_cast<double>((static_cast<long long>(t.rows) * groups + slots - 1) / slots);
                const long long step = span > 1 ? (pairs ? kPairStay : kOneStay) : (pairs ? kPairStep : kOneStep);
                const double time = waves * std::min<double>(span, static_cast<double>(F) / (m / 2)) * t.steps * step + kTileTime;
                if (best.groups == 0 || time < least) {
                    least = time;
                    best = t;
                    best.span = span;
                    best.groups = groups;
                }
            }
            continue;
        }
        t.rows = which == kWeights ? 2 * up(F, m) : up(T, m);
        t.cols = up(D, m);
        t.steps = which == kWeights ? up(T, 64) : 2 * up(F, 64);
        const long long tiles = static_cast<long long>(t.rows) * t.cols;
        const double size = which == kWeights ? 2.0 * F * D : static_cast<double>(T) * D;
        const double arrays = 4.0 * T * F, memory = arrays > kFitsL2 ? arrays / 6000 : 0;
        for (unsigned ways = 1; ways <= std::max(1u, std::min(64u, t.steps / 4)); ++ways) {
            if (!cut_steps(t, ways)) continue;
            const double waves = static_cast<double>((tiles * t.splits + slots - 1) / slots);
            // no faster than dg and du come from memory; sums of several splits are written and read again by another kernel
            const double time = std::max(waves * (t.run * (pairs ? kPairStep : kOneStep) + kTileTime), memory) +
                                (t.splits > 1 ? 3000 + 8.0 * size * t.splits / 5000 : 0);
            if (best.splits == 0 || time < least) {
                least = time;
                best = t;
                best.time = time;
            }
        }
    }
    return best;
}

// Tokens and weights in one launch where that is estimated shorter: of the splits that leave the tokens 16 of the pairs of blocks at
// least, those with which both sides end soonest.  A call that wants one of the two alone keeps this cut, and so its bits (dx or dwg, dwu
// alone of 262144 x 256 x 688 take 374 and 376 us, both 478).
inline void plan_both(long long T, int D, int F, GluTiles& tokens, GluTiles& weights) {
    const unsigned slots = kSms / 2, steps_t = 2 * up(F, 64), steps_w = up(T, 64);
    const unsigned tiles_w = 2 * up(F, 256) * up(D, 256);
    if (4.0 * T * F <= kFitsL2 || tiles_w > slots / 2) return;
    const long long tiles_t = static_cast<long long>(up(T, 256)) * up(D, 256);
    GluTiles t{}, w{};
    t.pairs = w.pairs = true;
    t.rows = up(T, 256);
    w.rows = 2 * up(F, 256);
    t.cols = w.cols = up(D, 256);
    t.steps = steps_t;
    w.steps = steps_w;
    if (!cut_steps(t, 1) || t.splits > 1) return;
    double least = tokens.time + weights.time;
    for (unsigned ways = 1; ways * tiles_w <= slots - 16; ++ways) {
        if (!cut_steps(w, ways)) continue;
        t.workers = slots - ways * tiles_w;
        const double first = static_cast<double>(up(tiles_t, t.workers)) * (steps_t * kPairStep + kTileTime);
        const double second = static_cast<double>(up(steps_w, ways)) * kPairStep + static_cast<double>(w.splits / ways) * kTileTime;
        const double time = std::max(first, second) + 3000 + 16.0 * F * D * w.splits / 5000;
        if (time < least) {
            least = time;
            tokens = t;
            weights = w;
        }
    }
}

// How a problem is laid out: the workspace's arrays, and how the weights' gradients are cut.
struct GluPlan {
    bool tensor;                     // tensor cores
    int width;                       // channels of the products, as tensor_width
    size_t tokens_copy, weights_copy;   // bytes of x or dx, of Wg, Wu, dWg or dWu in that width; 0 where it is D
    long long pitch;                 // of a row of dg and du
    size_t array;                    // bytes of one of them
    FmaTile slopes_fma, tokens_fma, weights_fma;   // CUDA cores
    GluTiles slopes, tokens, weights;              // tensor cores
    long long sum_rows;              // dbg and dbu: sums of dg and du over the rows of a tile, [sum_rows][2][sum_pitch]
    int sum_pitch;                   // F up to whole 16-byte chunks
    int runs;                        // of those rows
    long long column_run;
    size_t sums;                     // bytes of the sums of tiles, at the start of the partial ones
    size_t partial;                  // bytes
};

// Tiles and splits of a product on CUDA cores.  Cycles of a multiprocessor for a step of a tile: 128 x 128 are bound by FMA, the
// others by shared memory; one block alone takes 40 (32 x 32) to 115 for the latency of its loads.  The summed axis is cut where the
// tiles leave multiprocessors idle, and to at most kMostProducts in one sum; longer ones of kForward and kSlopes are added up in such
// runs within a block, in kernels of square tiles.
inline FmaTile plan_fma(Product which, long long T, int D, int F) {
    const bool pair = which == kForward || which == kSlopes;
    const long long rows = which == kWeights ? F : T, cols = pair ? 2LL * F : D, depth = pair ? D : (which == kWeights ? T : 2LL * up(F, 16) * 16);
    FmaTile best{};
    double least = 0;
    for (int r : {128, 32})
        for (int c : {128, 32}) {
            const double cycles = r == 128 ? (c == 128 ? 128 : 40) : (c == 128 ? 48 : 36);
            const long long tiles = static_cast<long long>(up(rows, r)) * up(cols, c) * (which == kWeights ? 2 : 1);
            if (up(cols, c) > 65535) continue;   // a launch's columns
            if (pair && D > kMostProducts && r != c) continue;
            const long long fewest = pair ? 1 : (depth + kMostProducts - 1) / kMostProducts;
            const long long most = pair ? 1 : std::max(fewest, std::min({depth / 128, (2 * kSms + tiles - 1) / tiles, 1024LL}));
            for (long long splits : {fewest, (fewest + most) / 2, most}) {
                if (splits < 1) continue;
                const long long blocks = tiles * splits, waves = (blocks + kSms - 1) / kSms;
                // nanoseconds; alone on its multiprocessor a block waits for its operands
                double time = std::max(waves * cycles, r + c > 64 ? 115.0 : 40.0) * (static_cast<double>(depth) / splits + 32) / 1.9;
                if (splits > 1) time += 3000 + 8.0 * rows * D * (which == kWeights ? 2 : 1) * splits / 5000;
                if (best.rows == 0 || time < least) {
                    least = time;
                    best = {r, c, static_cast<int>(splits), 0};
                }
            }
        }
    if (which == kWeights) {
        best.run = ((T + best.splits - 1) / best.splits + 15) / 16 * 16;
        best.splits = static_cast<int>((T + best.run - 1) / best.run);
    } else if (which == kTokens) {
        const long long pieces = 2LL * up(F, 16);
        best.run = (pieces + best.splits - 1) / best.splits;
        best.splits = static_cast<int>((pieces + best.run - 1) / best.run);
    }
    return best;
}

inline size_t up256(size_t n) { return (n + 255) / 256 * 256; }

// Channels that the tensor cores work on: D, or for 2-byte rows that are not whole 16-byte chunks D with zeros up to the next chunk,
// in copies, from 5e7 operations on (bf16, forward and gradients, FMA units -> copies: 100 x 499 x 501 25 -> 24 us, 97 -> 55; 300 x
// 999 x 1001 145 -> 27, 455 -> 59; 2000 x 1001 x 3001 543 -> 50, 1876 -> 138).  0: none, the product runs on FMA units, as fp32
// does, and sums over more channels than an accumulator of the tensor cores takes within the type's rounding (kMostSteps; 2^16 of one
// sign come out 3.7e-4 too small, and fp16 rounds by 4.9e-4).
inline int tensor_width(long long T, int D, int F, na_dtype dtype) {
    if (dtype == NA_FP32 || D > (dtype == NA_FP16 ? 1 << 16 : 1 << 18)) return 0;
    if (D % 8 == 0) return D;
    return 4.0 * T * D * F >= 5e7 ? (D + 7) / 8 * 8 : 0;
}

inline GluPlan plan_glu(long long T, int D, int F, na_dtype dtype) {
    GluPlan n{};
    const int es = dtype == NA_FP32 ? 4 : 2, chunk = 16 / es;
    const int width = tensor_width(T, D, F, dtype);
    n.tensor = width > 0;
    n.width = n.tensor ? width : D;
    if (n.width != D) {
        n.tokens_copy = up256(static_cast<size_t>(T) * n.width * es);
        n.weights_copy = up256(static_cast<size_t>(F) * n.width * es);
    }
    D = n.width;
    n.pitch = (static_cast<long long>(F) + chunk - 1) / chunk * chunk;
    n.array = up256(static_cast<size_t>(T) * n.pitch * es);
    size_t floats = 0;
    if (n.tensor) {
        n.slopes = plan_tiles(kSlopes, T, D, F);
        n.tokens = plan_tiles(kTokens, T, D, F);
        n.weights = plan_tiles(kWeights, T, D, F);
        plan_both(T, D, F, n.tokens, n.weights);
        if (n.tokens.splits > 1) floats = static_cast<size_t>(n.tokens.splits) * T * D;
        if (n.weights.splits > 1) floats = std::max(floats, static_cast<size_t>(n.weights.splits) * 2 * F * D);
    } else {
        n.slopes_fma = plan_fma(kSlopes, T, D, F);
        n.tokens_fma = plan_fma(kTokens, T, D, F);
        n.weights_fma = plan_fma(kWeights, T, D, F);
        if (n.tokens_fma.splits > 1) floats = static_cast<size_t>(n.tokens_fma.splits) * T * D;
        if (n.weights_fma.splits > 1) floats = std::max(floats, static_cast<size_t>(n.weights_fma.splits) * 2 * F * D);
    }
    // sums of dg and du: over the rows of a tile as it is made (all of few tokens; else a warp's 32 on tensor cores, a block's on CUDA
    // cores), then runs of those rows: four blocks a multiprocessor, at least 64 rows each, at most 8192, of which a thread adds every
    // eighth
    n.sum_rows = n.tensor ? (n.slopes.few ? 1 : up(T, 32)) : up(T, n.slopes_fma.rows);
    n.sum_pitch = (F + 3) / 4 * 4;
    const long long columns = 2LL * up(F, 128);
    const long long runs = std::max((n.sum_rows + 8191) / 8192, std::min((n.sum_rows + 63) / 64, (4 * kSms + columns - 1) / columns));
    n.column_run = (n.sum_rows + runs - 1) / runs;
    n.runs = static_cast<int>((n.sum_rows + n.column_run - 1) / n.column_run);
    n.sums = up256(static_cast<size_t>(n.sum_rows) * 2 * n.sum_pitch * sizeof(float));
    n.partial = std::max(up256(floats * sizeof(float)), n.sums + up256(static_cast<size_t>(n.runs) * 2 * F * sizeof(float)));
    return n;
}

inline size_t glu_workspace(const GluPlan& n) { return 2 * n.array + n.partial + 2 * n.tokens_copy + 4 * n.weights_copy; }

}  // namespace glu
}  // namespace na
