// na_add.h -- parameters and plan of the residual add between norms, shared by its host code (na_addnorm.cu) and its kernels
// (na_add_impl.cuh; one na_add_*.cu per direction and type).
#pragma once

#include "na_block.cuh"

namespace na {
namespace add {

constexpr int kAddThreads = 256;   // blocks of warp teams
constexpr int kAddBlock = 512;     // most threads of a row's block (128 registers each)
constexpr int kAddMaxC = 8192;
constexpr int kAddStages = 2;            // of a ring
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

// Blocks of the forward's warp teams per multiprocessor that the registers leave room for, with E channels to a thread.
__host__ __device__ constexpr int add_fwd_blocks(int E, bool lean) { return E <= 8 && lean ? 3 : 2; }

// How a problem is laid out: chunk width, chunks per thread, threads per row, blocks, parts of a group, rows of a tile.
struct AddPlan {
    bool vec, block, ring;
    int j, team, blocks, per_group, tile;
    size_t ring_bytes;
};

// Bytes of a tile in a ring: rows that are not whole chunks are copied with up to 15 bytes on both sides.
__host__ __device__ constexpr uint32_t ring_pitch(uint32_t bytes, bool whole) { return whole ? bytes : (bytes + 30u) & ~15u; }

inline bool lean_forward(const AddParams& p) { return p.norm != NA_NORM_LAYER && p.post != NA_NORM_LAYER && !p.b && !p.post_b; }

template <typename T, bool BWD>
na_status launch_add(const AddParams& p, const AddPlan& n, cudaStream_t s);

}  // namespace add
}  // namespace na
