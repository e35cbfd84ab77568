// na_win.h -- parameters and launchers of the window softmax kernels (na_win_impl.cuh).
#pragma once

#include "na_block.cuh"

namespace na {

constexpr int kWinThreads = 128;

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
    int tile;              // rows per tile (a multiple of 8)
    int stages;            // tiles of a block's ring
    uint32_t lam_rows;
    Dropout drop;
    unsigned* err;         // device status word
    unsigned long long wait_ns;
    uint32_t withhold;     // test hook: block 0 leaves out its first copy
};

// Kernels of one type and form: `diff` the difference of two maps, `bwd` the gradients.
na_status launch_soft_fwd_bf16(WinParams& p, cudaStream_t s);
na_status launch_soft_fwd_f16(WinParams& p, cudaStream_t s);
na_status launch_soft_fwd_f32(WinParams& p, cudaStream_t s);
na_status launch_soft_bwd_bf16(WinParams& p, cudaStream_t s);
na_status launch_soft_bwd_f16(WinParams& p, cudaStream_t s);
na_status launch_soft_bwd_f32(WinParams& p, cudaStream_t s);
na_status launch_diff_fwd_bf16(WinParams& p, cudaStream_t s);
na_status launch_diff_fwd_f16(WinParams& p, cudaStream_t s);
na_status launch_diff_fwd_f32(WinParams& p, cudaStream_t s);
na_status launch_diff_bwd_bf16(WinParams& p, cudaStream_t s);
na_status launch_diff_bwd_f16(WinParams& p, cudaStream_t s);
na_status launch_diff_bwd_f32(WinParams& p, cudaStream_t s);

}  // namespace na
