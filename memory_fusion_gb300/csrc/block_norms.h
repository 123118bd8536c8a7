// block_norms.h -- launchers of the norms before and after a block (block_norms.cu), shared with the C-ABI layer.  Not
// part of the public ABI.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace cf {

constexpr int kBlockNormsMaxCols = 32768;

// what the rows' ring in shared memory needs to know
struct RingArgs {
    int depth;  // stages (the launcher's)
    uint32_t extra_arrivals;  // test hook: arrivals that the stages' barriers wait for in vain
    unsigned long long timeout_ns;
    uint32_t *err;
};

struct BlockNormsArgs {
    const void *h, *x, *gate;  // x, gate: or null
    const float *post_weight, *post_bias, *pre_weight, *pre_bias;  // or null
    void *x_out, *y;           // either or null
    int64_t rows;
    uint32_t rows_per_gate;
    int cols, post, pre, dtype;
    float scale, alpha, eps;
    int gates;
    int lanes, chunk, gates_along;  // threads of a row, rows of them, a gate with every row (the launcher's)
    RingArgs ring;
};
// vec: columns a multiple of 8, everything 16-byte aligned
cudaError_t launch_block_norms(BlockNormsArgs a, bool vec, int sms, bool pdl, cudaStream_t stream);

struct BlockNormsGradArgs {
    const void *dy, *dx_out, *h, *x_out, *gate;  // all but h: or null (x_out where dy is)
    const float *post_weight, *post_bias, *pre_weight;  // or null
    void *dh, *dx, *dgate;     // the last two: or null
    int sum_at[4];             // place of dpost_weight, dpost_bias, dpre_weight, dpre_bias in the partial sums, -1: not wanted
    float *sum_out[4];
    float *partials;           // [sums][sets][cols]
    float *slots;              // [workers][2][cols] sums of gates that begin before a worker's rows, or end behind them
    int64_t rows;
    uint32_t rows_per_gate;
    int cols, post, pre, dtype;
    float scale, alpha, eps;
    int64_t chunk;             // rows of a worker (the plan's, set by the launcher, as are the next)
    int lanes, cluster, sets;
    RingArgs ring;
};
// A worker is a group of threads that holds a row, its rows a stretch of neighbours; a set the workers of a CTA (or of a
// cluster, which has one).
struct BlockNormsGradPlan {
    int pieces, lanes, cluster, threads, sets, workers;
    int64_t chunk;
};
BlockNormsGradPlan plan_block_norms_grad(int64_t rows, int64_t cols, int sms, bool lean, int dtype);
// neither LayerNorms nor biases, and aligned rows
bool block_norms_grad_lean(const BlockNormsGradArgs &a, bool vec);
cudaError_t launch_block_norms_grad(BlockNormsGradArgs a, const BlockNormsGradPlan &p, bool vec, bool pdl,
                                    cudaStream_t stream);

}  // namespace cf
