// na_win.h -- parameters and launchers of the window softmax kernels (na_win_impl.cuh).
#pragma once

#include "na_block.cuh"

namespace na {

constexpr int kWinThreads = 256;

struct WinParams {
    const void* x1;
    const void* x2;
    const void* dy;
    const float* lam;      // [heads], or [rows] with lam_rows
    void* out1;            // y; dx1
    void* out2;            // dx2
    float* dlam;           // backward: -r_2 of every row
    long long rows, tiles;
    int K, heads;
    int lanes, log_lanes;  // lanes per row (a power of two)
    int tile;              // rows per tile (a multiple of 8)
    int stages;            // tiles of a block's ring
    uint32_t lam_rows, rows32;
    FastDiv fd_heads;
    Dropout drop;
    unsigned* err;         // device status word
    unsigned long long wait_ns;
};

// One instance per type: `diff` the difference of two maps, `bwd` the gradients.
na_status launch_win_bf16(WinParams& p, bool diff, bool bwd, cudaStream_t s);
na_status launch_win_f16(WinParams& p, bool diff, bool bwd, cudaStream_t s);
na_status launch_win_f32(WinParams& p, bool diff, bool bwd, cudaStream_t s);

}  // namespace na
