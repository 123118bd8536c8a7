// grouped_internal.h -- the grouped GEMM and low-rank adapter launchers
// (gemm_grouped.cu), shared with the C-ABI layer.  Not part of the public ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace cf {

enum GroupedKind : int {
    GR_FORWARD = 0,  // Y = act(X_g . W_g), optionally keeping the pre-activation
    GR_DGRAD = 1,    // dX = (dY_g . W_g^T) (* act'(Z))
    GR_WGRAD = 2,    // dW_g = X_g^T . dY_g
    GR_SHRINK = 3,   // H = scale[a] * X_g . A_a (adapters: groups are requests), as two 16-bit parts
    GR_LORA = 4,     // Y = X . W + bias + H . B_a
};

constexpr int kGroupedMaxSmem = 232448;   // dynamic shared memory of a CTA (227 KB)
constexpr int kGroupedMaxGroups = 1024;  // the group table lives in shared memory
constexpr int kGroupedSplitTiles = 1024; // tiles whose contraction may be divided among CTAs
constexpr int kGroupedWorkers = 160;     // CTAs that may hold a piece of a tile (a GB300 has 152 SMs)
// Cycles that the host's choice of tiles and the device's plan both count with (about 1.8 GHz under load): an MMA block
// of 64 in the contraction takes 2.35 a column, and 290 at least (370 in a pair); dividing tiles (writing, adding,
// finishing pieces) 1500 and 70 a column.
constexpr int kMmaCycles20Columns = 47, kMmaCyclesLeast = 290, kMmaCyclesLeastPair = 370;
constexpr int kDivideCycles = 1500, kDivideCyclesColumn = 70;
// blocks of 64 that a worker takes at least (2, 4 and 8: 10.4, 10.4 and 10.4 us in the geometric mean over 35 calls of up
// to 4099 rows, so nothing finer is looked for)
constexpr int kMinStretch = 4;
// Rows up to which a request's X . A runs on the CUDA cores, and the most parts of their contraction (geometric mean over
// 28 batches: 30.4 us with 2 rows, 30.7 with 4, 31.7 with 8; 30.6 with 4 parts, 30.7 with 8, 30.8 with 16)
constexpr int kLoraShortRows = 4;
constexpr int kLoraMaxSplit = 8;
constexpr int kLoraMaxRank = 128;        // one tile of features in the first product

// Columns that an MMA multiplies come in steps: 16 for one CTA (M = 128), 32 for a pair (M = 256 over two CTAs), each of
// which stages half of them.  (WGRAD pairs: whole 64-column blocks in either CTA.)
__host__ __device__ constexpr int grouped_column_step(int kind, bool pair) {
    return pair ? (kind == GR_WGRAD ? 128 : 32) : 16;
}
// Rows of each of the `tiles` row tiles (two at least) that a group's rows are cut into evenly, in whole steps.  (Rows
// plus tiles may pass 2^31.)
__host__ __device__ constexpr int grouped_rows_per_tile(int rows, int tiles, int step) {
    return ((rows - 1) / tiles + step) & ~(step - 1);
}
// LORA, a tile of several requests: of the `own` rows at its start that are one long request's, those whose low-rank
// product runs on the tensor cores, in whole steps; the rest of them go with the other rows
__host__ __device__ constexpr int lora_tensor_columns(int own, bool pair) {
    return own & ~(grouped_column_step(GR_LORA, pair) - 1);
}

struct GroupedArgs {
    CUtensorMap tmap_a;    // the operand whose features become accumulator lanes: W (WGRAD: X)
    CUtensorMap tmap_b;    // the operand whose rows become accumulator columns: X or dY (WGRAD: dY)
    CUtensorMap tmap_b2;   // the same with boxes of half the rows (not WGRAD)
    CUtensorMap tmap_lb;   // LORA: B of the adapters, as tmap_a
    CUtensorMap tmap_h;    // LORA: H, as tmap_b
    int a_blocks;          // 64-feature blocks staged: 1 where there are no more than 64 features, else 2
    int a_split, b_split;  // 1: rows of 64-column blocks do not tile the matrix, so one block a copy (a length % 64)
    const int32_t *offsets;  // [groups + 1] rows of each group (LORA: of each request)
    const int32_t *windex;   // SHRINK, LORA: [groups] adapter of each request, -1 for none
    void *out;               // Y / dX / dW / H [T, 2, rank]
    void *preact;            // FORWARD: Z written; DGRAD: Z read; or null
    const float *bias;       // LORA: [F] or null
    const float *scale;      // SHRINK: [nweights] or null
    const void *low;         // LORA: H [T, 2, rank] 16-bit, upper parts and rests
    int after_shrink;        // LORA: the launch before is the SHRINK that makes H (it waits for what came before it)
    const void *x, *lora_a;  // SHRINK: X [T, C], A [nweights, C, F]
    float *low_parts;        // SHRINK: [request and 64 ranks][low_split][kLoraShortRows][64] parts of short requests' H
    uint32_t *low_counters;  // SHRINK: parts arrived, zero between launches
    int low_split;           // SHRINK: parts of a short request's contraction
    const void *lora_b;      // LORA: B [nweights, rank, F]
    uint32_t *err;
    uint32_t *counters;      // [kGroupedSplitTiles] pieces arrived, zero between launches
    float *partials;         // [2 * kGroupedWorkers][bn][128] pieces of tiles, or null: whole tiles only
    int T;                   // rows of X / dY
    int F;                   // features: length of the accumulator-lane axis of the result
    int C;                   // contraction length (WGRAD: the groups' rows instead)
    int N;                   // WGRAD: columns of dW
    int groups;
    int nweights;            // weights that windex may name
    int rank;                // LORA
    int long_rows;           // LORA: rows from which a request has tiles of its own
    int fp16;                // 16-bit type of every operand: 0 bf16, 1 fp16
    int act;                 // FORWARD: 1 = GELU(tanh)
    int bn;                  // columns of one accumulator tile (16, 32, 64, 128 or 256)
    int stages;
    int copy_cycles;         // what a block's copies take
    int wait_cycles;         // LORA: what H takes, about
    int pair;                // CTA pairs, one cta_group::2 MMA stream over 256 features (not SHRINK)
    int extra_arrivals;      // test hook: arrivals that the accumulator-ready barriers wait for in vain
    unsigned long long timeout_ns;
};

int grouped_smem_bytes(int kind, bool pair, int stages, int bn, int groups, int a_blocks);
cudaError_t launch_grouped(int kind, const GroupedArgs &a, int ctas, int smem, bool pdl, cudaStream_t stream);

}  // namespace cf
