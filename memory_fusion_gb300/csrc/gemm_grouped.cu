// gemm_grouped.cu -- products whose rows choose their weights, on tcgen05:
//     FORWARD  Y = act(X_g . W_g)             rows [offsets[g], offsets[g+1]) of X with W[g]
//     DGRAD    dX = (dY_g . W_g^T) * act'(Z)
//     WGRAD    dW_g = X_g^T . dY_g            a sum over the group's rows
//     SHRINK   H = scale[a] * X_g . A[a]      groups are requests, a their adapter
//     LORA     Y = X . W + bias + H . B[a]    the shared projection with the adapters' second product
//
// Design:
//  * Features are the accumulator's lanes and rows of the batch its columns:
//    D^T[128 features, n rows] = W^T . X^T.  A group of a few rows then costs an
//    MMA of N = 16 and a 2 KB row tile instead of a 128-row tile that is mostly
//    padding: a decode batch reads weights and little else.  The last tile of a
//    group takes the N it needs (multiples of 16), and a group's tiles are cut
//    evenly.  Columns behind a group's rows hold its neighbour's products: a
//    column depends on its own row alone, so they are not stored and nothing
//    of them (a NaN, say) can reach the group.
//  * WGRAD sums over rows, so there the neighbour's rows must not take part:
//    the last block of a group issues the MMAs that hold its rows and zeroes, in
//    shared memory, what is left of the last 16.
//  * Group sizes are device data.  Every CTA scans the offsets into a table in
//    shared memory and walks the same tile list; no host synchronisation.
//    Offsets that decrease or pass T are clamped and reported
//    (CF_ERR_DEVICE_BOUNDS), so no read or write leaves its array.
//  * Warp roles as in the fused GEMM: warp 0 issues TMA loads into a ring, warp
//    1 the MMAs into one of two accumulators, warps 2..9 the epilogue of tile i
//    while tile i + 1 is multiplied; every wait is bounded.  The first two run
//    their loops as whole warps and issue by an elected lane: a loop of one lane
//    spent some 600 cycles a block on its own control flow (16384 rows over 8
//    groups of 2048 x 8192: 351 us, now 317).
//  * CTA pairs (M = 256, cta_group::2) where there are tiles enough for them:
//    each CTA stages its own 128 features and half of the rows, so a block costs
//    an SM 32 KB of copies in place of 48 (single CTAs 356 us there).
//  * Few tiles with a long contraction are divided among the SMs: pieces of fp32
//    accumulators in the workspace, added in a fixed order by the last arriver.
//
// What bounds each form, and what it measured on a GB300 in a CUDA graph, more than twice L2 between two uses of an input
// (at 2070 MHz; in brackets over two seconds, where the power cap takes the long ones to 1560 MHz):
//     FORWARD  16384 rows, 8 groups of 2048 x 8192, GELU: the tensor pipe, 317 us (1.73 PFLOP/s) [372, 1.48];
//              250 rows, 32 groups of 2048 x 4096: HBM, 72 us (6.6 TB/s); 4099 rows, 64 groups of 1000 x 2056: HBM,
//              49 us (5.3 TB/s); 2 rows, 8 groups of 1024 x 2048: latency, 7.1 us (launch 2, table 1.2, first copy 1,
//              16 blocks in pieces 1, joining them 1.5)
//     DGRAD    16384 rows, 16 groups of 4096 x 2048, GELU': the tensor pipe, 191 to 200 us (1.38 to 1.44 PFLOP/s)
//              [203, 1.36]; 333 rows, 12 groups of 520 x 1032: latency, 7.0 to 7.9 us
//     WGRAD    16384 rows, 8 groups of 2048 x 8192: the tensor pipe, 326 us (1.69 PFLOP/s) [368, 1.50]; 1003 rows,
//              24 groups of 520 x 1032: the epilogues of its 600 tiles, 14 us (2.1 TB/s)
//     LORA     with its SHRINK, 8192 rows of 8 requests, 4096 x 4096, rank 64: the tensor pipe, 165 us (1.72 PFLOP/s)
//              [184, 1.54]; one row, rank 16: 14.6 us, 64 requests of one row: 25 us (the chain X . A, join, H . B, join
//              beside 33 MB of W); 1537 rows of 40 requests, 2048 x 2056, rank 24: 43 us (the chain, then row tiles
//              that requests do not fill)
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "../../include/cf.h"
#include "cf_internal.h"
#include "grouped_internal.h"
#include "ptx.cuh"
#include "umma.cuh"

namespace cf {

// ---------------------------------------------------------------------------
// Primitives that only these kernels use (the shared ones are in ptx.cuh)
// ---------------------------------------------------------------------------
namespace ptx {

// bring the line holding p into L2
__device__ __forceinline__ void prefetch_l2(const void *p) {
    asm volatile("prefetch.global.L2 [%0];" ::"l"(reinterpret_cast<uint64_t>(p)));
}
// 3-D and 4-D tiled TMA loads without a cache policy; _pair: completing on an mbarrier of either CTA of the pair
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void *tmap, uint32_t bar, int32_t x, int32_t y,
                                            int32_t z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}
__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const void *tmap, uint32_t bar_cluster, int32_t x,
                                                 int32_t y, int32_t z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar_cluster), "r"(x), "r"(y), "r"(z)
        : "memory");
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void *tmap, uint32_t bar, int32_t x, int32_t y,
                                            int32_t z, int32_t w) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w)
        : "memory");
}
__device__ __forceinline__ void tma_load_4d_pair(uint32_t dst, const void *tmap, uint32_t bar_cluster, int32_t x,
                                                 int32_t y, int32_t z, int32_t w) {
    asm volatile(
        "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar_cluster), "r"(x), "r"(y), "r"(z), "r"(w)
        : "memory");
}
// arrive on an mbarrier of another CTA of the cluster without release semantics: nothing this thread wrote is handed
// over.  (A release per pipeline stage waits for the thread's own copies: the weight gradient ran at half the speed.)
__device__ __forceinline__ void mbar_arrive_cluster_relaxed(uint32_t bar_cluster) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar_cluster) : "memory");
}

// 32 columns of 32 lanes of tensor memory in 8 x 8 blocks: of lanes 8b..8b+7 and columns 8k..8k+7, thread t holds lane
// t / 4 and columns 2 (t % 4) and the next, in v[16 (b / 2) + 4 k + 2 (b % 2)] and the next
__device__ __forceinline__ void tmem_ld_blocks(uint32_t taddr, uint32_t (&v)[32]) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
        asm volatile(
            "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
            "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
            : "=r"(v[16 * h]), "=r"(v[16 * h + 1]), "=r"(v[16 * h + 2]), "=r"(v[16 * h + 3]), "=r"(v[16 * h + 4]),
              "=r"(v[16 * h + 5]), "=r"(v[16 * h + 6]), "=r"(v[16 * h + 7]), "=r"(v[16 * h + 8]),
              "=r"(v[16 * h + 9]), "=r"(v[16 * h + 10]), "=r"(v[16 * h + 11]), "=r"(v[16 * h + 12]),
              "=r"(v[16 * h + 13]), "=r"(v[16 * h + 14]), "=r"(v[16 * h + 15])
            : "r"(taddr + (uint32_t(16 * h) << 16))
            : "memory");
}
// the wait for loads into v, which is theirs until then.  (A wait that does not name them orders memory alone: arithmetic
// on v may be moved in front of it.)
__device__ __forceinline__ void tmem_ld_wait(uint32_t (&v)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                   "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]),
                   "+r"(v[15]), "+r"(v[16]), "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]),
                   "+r"(v[22]), "+r"(v[23]), "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]),
                   "+r"(v[29]), "+r"(v[30]), "+r"(v[31])::"memory");
}
// four 8 x 8 blocks of 16-bit numbers to and from shared memory, transposed: thread t holds row t / 4, columns
// 2 (t % 4) and the next of each block; thread 8m + j gives the 16 bytes that are column j of block m
__device__ __forceinline__ void stmatrix4_t(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b),
                 "r"(c), "r"(d)
                 : "memory");
}
__device__ __forceinline__ void ldmatrix4_t(uint32_t addr, uint32_t &a, uint32_t &b, uint32_t &c, uint32_t &d) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(a), "=r"(b), "=r"(c), "=r"(d)
                 : "r"(addr)
                 : "memory");
}

// one lane of a converged warp, the same one every time
__device__ __forceinline__ bool elect_one() {
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e != 0u;
}

}  // namespace ptx

namespace {

// instruction descriptor: kind::f16, A and B both bf16 or both fp16, D = fp32, either operand MN-major or K-major,
// M = m, N = n
__device__ __forceinline__ uint32_t idesc_f16(int m, int n, bool fp16, bool a_mn, bool b_mn) {
    return (1u << 4) | (fp16 ? 0u : (1u << 7) | (1u << 10)) | (uint32_t(a_mn) << 15) | (uint32_t(b_mn) << 16) |
           (uint32_t(n >> 3) << 17) | (uint32_t(m >> 4) << 24);
}


// Epilogue warps, from warp 2 on: two halves of 4 (128 lanes each); SHRINK one, and two more warps that only help
// with its short requests.
__host__ __device__ constexpr int epi_warps(int kind) { return kind == GR_SHRINK ? 4 : 8; }
__host__ __device__ constexpr int threads_of(int kind) { return kind == GR_SHRINK ? 256 : 320; }
// Ten warps are three on a quarter of the SM: 168 registers each.  (Fewer, so that a CTA of LORA fits beside one of
// SHRINK, gained nothing: 64 requests 22.4 us, 21.8 without.)
__host__ __device__ constexpr int registers_of(int kind) { return kind == GR_SHRINK ? 128 : 168; }
constexpr int kShortWarps = 6;
constexpr int kBK = 64;         // contraction per stage (128 bytes: one swizzle atom)
constexpr int kFB = 128;        // features per tile (accumulator lanes)
// row tiles walked before the next feature tile (the forward and the input gradient of 16384 rows, one after another:
// 368 and 201 us with 4, 358 and 193 with 16, 359 and 193 with 64)
constexpr int kRasterRows = 16;
// LORA: rows up to which a run of shorter requests joins the long one before it (a run of its own costs a row tile; one
// that joins ends the tile's part on the tensor cores.  Geometric mean over 28 batches with 0, 16, 32 and 64 rows: 31.4,
// 30.8, 30.7 and 30.8 us; 1537 rows of 40 requests, 2048 x 2056: 52 us with 0, 43 with the others)
constexpr int kRunRows = 32;
constexpr int kShortRows = kLoraShortRows;

// The waits for an accumulator and for a group's last block have this much more time for each 64-deep block before it.
// (A block takes 0.15 to 0.4 us, 2 where every SM's copies come from HBM at once: a tile that is not divided may sum for
// seconds.)
constexpr uint64_t kBlockNs = 4000;

constexpr uint32_t kInfoProducer = 0x10000000u;
constexpr uint32_t kInfoMma = 0x20000000u;
constexpr uint32_t kInfoEpi = 0x30000000u;
constexpr uint32_t kInfoTable = 0x70000000u;
constexpr uint32_t kInfoRange = 0x71000000u;

struct GrLayout {
    uint32_t a_bytes, stage_bytes, table, stg, bars, total;
};

// int32 arrays of the group table behind the Plan, groups + 1 long
__host__ __device__ constexpr int table_arrays(int kind) { return kind == GR_LORA ? 6 : kind == GR_SHRINK ? 3 : 2; }

__host__ __device__ inline GrLayout gr_layout(int kind, bool pair, int stages, int bn, int groups, int a_blocks) {
    GrLayout L;
    // a CTA of a pair stages its own 128 features and half of the tile's columns
    L.a_bytes = uint32_t(a_blocks) * 8192u;
    L.stage_bytes = L.a_bytes + uint32_t((pair ? bn / 2 : bn) * kBK * 2);
    uint32_t off = uint32_t(stages) * L.stage_bytes;
    // (with one block of features the MMA reads another 8 KB behind it, into lanes that nobody stores)
    if (a_blocks == 1 && L.stage_bytes < 16384u) off += 16384u - L.stage_bytes;
    L.table = off;
    off += (32u + uint32_t(table_arrays(kind) * (groups + 1)) * 4u + 15u) & ~15u;
    // per epilogue warp: 16-bit [32 rows][32 features]; LORA: fp32; WGRAD: 16-bit [32 features][64 columns];
    // SHRINK: before that, the warps' sums of 4 rows x 64 ranks
    L.stg = off;
    off += (kind == GR_LORA || kind == GR_WGRAD) ? 8u * 4096u : kind == GR_SHRINK ? 4u * 2048u : 8u * 2048u;
    static_assert(kShortWarps * 4 * 64 * 4 <= 4 * 2048, "sums of the short requests");
    L.bars = (off + 15u) & ~15u;
    L.total = L.bars + 256u;
    return L;
}

struct GrBars {
    uint32_t full0, empty0, tmem_full0, tmem_empty0, mma_done, misc;
};
__device__ __forceinline__ GrBars gr_bars(uint32_t base, int stages) {
    GrBars b;
    b.full0 = base;
    b.empty0 = base + 8 * stages;
    b.tmem_full0 = base + 16 * stages;
    b.tmem_empty0 = b.tmem_full0 + 16;
    b.mma_done = b.tmem_empty0 + 16;
    b.misc = b.mma_done + 8;
    return b;
}
static_assert(16 * 12 + 16 + 16 + 8 + 20 <= 256, "barrier area");

template <bool kPair>
__device__ __forceinline__ int feature_tiles(const GroupedArgs &a) {
    return kPair ? (a.F + 2 * kFB - 1) / (2 * kFB) : (a.F + kFB - 1) / kFB;
}

// one piece of work: a tile, or the part of its contraction that falls to this CTA
struct Tile {
    int id;     // tile number
    int g;      // group
    int w;      // its weights
    int f0;     // first feature of this CTA
    int col0;   // first accumulator column's row of the batch (WGRAD: column of dW)
    int n;      // columns that exist
    int nm;     // columns multiplied (n rounded up; a pair: half of them staged by each CTA)
    int nk;     // 64-deep blocks of the tile's contraction
    int kb0, kb1;  // the blocks of this piece
    int row0;   // WGRAD: first row of the group
    int rows;   // WGRAD: rows of the group
    int extra;  // LORA: blocks of the low-rank product behind the tile's own (pieces: with the last)
    int ad;     // LORA: the adapter of the first nx columns' rows, -1 none
    int nx;     // LORA: columns whose low-rank product runs on the tensor cores: all of the tile (nm), or a long
                // request's in whole steps of the MMA's columns
    bool mixed; // LORA: the columns behind them are of several requests
    int first, last;  // workers that hold pieces of the tile
    int slot;   // which of its two workspace slots this worker's piece goes to
    __device__ bool whole() const { return first == last; }
};

// How the launch divides its work, decided on the device once the sizes are known (every CTA decides alike).
// Whole tiles dealt out in turn; or, where the tiles are few or their last round is poorly filled, the blocks of all
// tiles in one row, cut into equal stretches: a worker's stretch starts and ends inside a tile at most once each.
// The pieces of a tile are added in the workspace in worker order (so equal calls give equal bits) by the
// worker whose piece arrives last; nobody waits.
struct Plan {
    int split;      // stretches
    int workers;    // that take part
    int tiles;
    int ways;       // split: stretches of each tile, or 0 where they run over tiles:
    int base, rem;  // then a worker's stretch is base blocks, of the first rem workers one more
    int groups;     // LORA: long requests and runs of short ones; else the groups
};
static_assert(sizeof(Plan) <= 32, "table layout");

// The group table in shared memory.
struct Table {
    Plan *plan;
    int *off;   // [groups + 1] first row of each group (LORA: request)
    int *pre;   // [plan groups + 1] tiles of the groups before (WGRAD: blocks of one tile of each)
    int *ad;    // SHRINK, LORA: adapter of each request, -1 for none
    int *goff;  // LORA: [plan groups + 1] first row of each plan group: a long request, or a run of short ones
    int *gad;   // LORA: its adapter, -1 none, -2 a run
    int *turn;  // LORA: [groups] changes of the adapter up to each request
    __device__ Table(uint8_t *p, int kind, int groups) {
        plan = reinterpret_cast<Plan *>(p);
        off = reinterpret_cast<int *>(p + 32);
        pre = off + groups + 1;
        ad = pre + groups + 1;
        goff = kind == GR_LORA ? ad + groups + 1 : off;
        gad = goff + groups + 1;
        turn = gad + groups + 1;
    }
};

// The request of a row of the batch: the last that starts at or before it.
__device__ __forceinline__ int request_of(const Table &tab, int groups, int row) {
    int lo = 0, hi = groups - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (tab.off[mid] <= row) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// LORA: rows of the run of short requests behind plan group g that join it
__device__ __forceinline__ int joined_rows(const Table &tab, int ngroups, int g) {
    if (tab.gad[g] == -2 || g + 1 >= ngroups || tab.gad[g + 1] != -2) return 0;
    const int rows = tab.goff[g + 2] - tab.goff[g + 1];
    return rows <= kRunRows ? rows : 0;
}

template <int KIND, bool kPair>
struct Walk {
    const Table tab;
    const GroupedArgs &a;
    const Plan plan;
    int ft;      // feature tiles
    int per_group;  // WGRAD: tiles of a group
    int shift;   // log2(a.bn)
    int nkc;     // blocks of C
    int g;       // group of the current tile (tiles are visited in ascending order)
    int half;    // features of this CTA behind the tile's first: 0, or 128 in the second CTA of a pair
    int worker, cur, end;  // tile, or unit and the end of this worker's stretch

    __device__ Walk(const Table &t, const GroupedArgs &a_, int worker_, int half_)
        : tab(t), a(a_), plan(*t.plan), g(0), half(half_), worker(worker_) {
        ft = feature_tiles<kPair>(a);
        shift = 31 - __clz(a.bn);
        nkc = (a.C + kBK - 1) / kBK;
        per_group = KIND == GR_WGRAD ? ft * ((a.N + a.bn - 1) >> shift) : 0;
        cur = worker;
        end = plan.tiles;
        if (!kPair && plan.split) {
            if (plan.ways != 0) {  // one piece: of tile worker / ways
                end = cur + (worker < plan.workers ? 1 : 0);
            } else {
                cur = unit_of(worker);
                end = worker < plan.workers ? unit_of(worker + 1) : cur;
            }
        }
    }
    static constexpr int kTileF = kPair ? 2 * kFB : kFB;
    static constexpr int kGran = grouped_column_step(KIND, kPair);
    __device__ int unit_of(int w) const { return w * plan.base + min(w, plan.rem); }
    __device__ int worker_of(int u) const {
        const int wide = plan.rem * (plan.base + 1);
        return u < wide ? u / (plan.base + 1) : plan.rem + (u - wide) / plan.base;
    }

    __device__ bool next(Tile &r) {
        if (cur >= end) return false;
        int local, kb = 0;
        if constexpr (KIND == GR_WGRAD) {
            // (an empty group counts one block a tile, which holds no rows)
            if (!kPair && plan.split) {
                while (cur >= per_group * tab.pre[g + 1]) ++g;
                const int nk = tab.pre[g + 1] - tab.pre[g], at = cur - per_group * tab.pre[g];
                local = at / nk;
                kb = at % nk;
            } else {
                g = cur / per_group;
                local = cur % per_group;
            }
            r.id = g * per_group + local;
        } else {
            r.id = cur;
            if (!kPair && plan.split) {
                if (plan.ways != 0) {
                    r.id = cur / plan.ways;
                } else {
                    r.id = cur / nkc;
                    kb = cur - r.id * nkc;
                }
            }
            // the last group that starts at or before the tile: 32 at a time, by the whole warp
            for (int passed = 32; passed == 32;) {
                const int at = min(g + 1 + int(threadIdx.x & 31), plan.groups);  // (pre of the last is above any tile)
                passed = __popc(__ballot_sync(0xffffffffu, r.id >= tab.pre[at]));
                g += passed;
            }
            local = r.id - tab.pre[g];
        }
        r.g = g;
        r.w = KIND == GR_SHRINK ? tab.ad[g] : (KIND == GR_LORA ? 0 : g);
        const int lo = tab.goff[g];
        const int rows = tab.goff[g + 1] - lo + (KIND == GR_LORA ? joined_rows(tab, plan.groups, g) : 0);
        int blocks;  // of the tile, one at least
        if constexpr (KIND == GR_WGRAD) {
            const int nt = (a.N + a.bn - 1) >> shift;
            r.f0 = (local / nt) * kTileF + half;
            r.col0 = (local % nt) * a.bn;
            r.n = min(a.bn, a.N - r.col0);
            r.row0 = lo;
            r.rows = rows;
            r.nk = (rows + kBK - 1) / kBK;
            blocks = max(r.nk, 1);
        } else {
            const int rt = (rows + a.bn - 1) >> shift;  // row tiles of the group, cut evenly
            if (rt == 1) {
                r.f0 = local * kTileF + half;
                r.col0 = lo;
                r.n = rows;
            } else {
                const int per = grouped_rows_per_tile(rows, rt, kGran);
                const int chunk = local / (kRasterRows * ft);
                const int wide = min(kRasterRows, rt - chunk * kRasterRows);
                const int in = local - chunk * kRasterRows * ft;
                const int ftile = in / wide;
                const int rtile = chunk * kRasterRows + in - ftile * wide;
                r.f0 = ftile * kTileF + half;
                r.col0 = lo + rtile * per;
                r.n = min(per, rows - rtile * per);
            }
            r.row0 = r.rows = 0;
            r.nk = blocks = nkc;
        }
        r.nm = (r.n + kGran - 1) & ~(kGran - 1);
        r.ad = -1;
        r.nx = 0;
        r.mixed = false;
        if constexpr (KIND == GR_LORA) {
            const int own = tab.gad[g] == -2 ? 0 : min(max(tab.goff[g + 1] - r.col0, 0), r.n);  // a long request's rows
            if (own == r.n) {
                r.ad = tab.gad[g];
                r.nx = r.nm;
            } else {  // requests in a row may share an adapter
                const int s0 = request_of(tab, a.groups, r.col0), s1 = request_of(tab, a.groups, r.col0 + r.n - 1);
                r.mixed = tab.turn[s0] != tab.turn[s1];
                r.nx = r.mixed ? lora_tensor_columns(own, kPair) : r.nm;
                if (r.nx > 0) r.ad = tab.ad[s0];
            }
        }
        r.kb0 = kb;
        r.kb1 = r.nk;
        r.first = r.last = worker;
        r.slot = 0;
        if (!kPair && plan.split && plan.ways != 0) {
            r.first = r.id * plan.ways;
            r.last = r.first + plan.ways - 1;
            r.kb0 = (worker - r.first) * nkc / plan.ways;
            r.kb1 = (worker - r.first + 1) * nkc / plan.ways;
            ++cur;
        } else if (!kPair && plan.split) {
            const int u0 = cur - kb;  // the tile's first unit
            const int take = min(blocks - kb, end - cur);
            r.kb1 = min(kb + take, r.nk);
            if (take < blocks) {
                r.first = worker_of(u0);
                r.last = worker_of(u0 + blocks - 1);
                r.slot = slot_of(worker, u0);
            }
            cur += take;
        } else {
            cur += plan.workers;
        }
        r.extra = KIND == GR_LORA && r.ad >= 0 && r.kb1 == r.nk ? 2 * ((a.rank + kBK - 1) / kBK) : 0;
        return true;
    }
    // a worker's first piece goes to its slot 0 unless its stretch began in an earlier tile
    __device__ int slot_of(int w, int u0) const { return plan.ways != 0 || unit_of(w) >= u0 ? 0 : 1; }
};

// GELU in the tanh form is z * p with p = 1 / (1 + exp(-2u)), u = sqrt(2/pi)(z + 0.044715 z^3):
// no cancellation in the left tail, where 1 + tanh(u) would lose every digit
__device__ __forceinline__ float gelu_p(float z) {
    const float u = 0.7978845608028654f * fmaf(0.044715f * z, z * z, z);
    return __fdividef(1.f, 1.f + ptx::ex2_approx(-2.885390081777927f * u));
}
__device__ __forceinline__ float gelu(float z) { return z * gelu_p(z); }
// d/dz of that: p + 2 z p (1 - p) u'.  Beyond |z| = 12, p is 0 or 1 to fp32 and the second term
// vanishes; the clamp keeps z^2 finite there (and a NaN stays one)
__device__ __forceinline__ float gelu_slope(float z) {
    const float c = fabsf(z) > 12.f ? copysignf(12.f, z) : z;
    const float p = gelu_p(c);
    const float du = 0.7978845608028654f * fmaf(0.134145f * c, c, 1.f);
    return fmaf(2.f * c * p * (1.f - p), du, p);
}

__device__ __forceinline__ uint16_t to16(float v, bool fp16) {
    return fp16 ? __half_as_ushort(__float2half_rn(v)) : __bfloat16_as_ushort(__float2bfloat16_rn(v));
}
__device__ __forceinline__ uint32_t pack16(float lo, float hi, bool fp16) {
    return uint32_t(to16(lo, fp16)) | (uint32_t(to16(hi, fp16)) << 16);
}
__device__ __forceinline__ float from16(uint16_t v, bool fp16) {
    return fp16 ? __half2float(__ushort_as_half(v)) : __uint_as_float(uint32_t(v) << 16);
}

// two numbers rounded to 16 bits, and back
template <bool kFp16>
__device__ __forceinline__ uint32_t pack_pair(float lo, float hi) {
    if constexpr (kFp16) {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
}

constexpr float kFloatMax = 3.402823466e38f;
// a finite number, no larger than the type's largest (bf16: numbers that would round to infinity lie behind that)
template <bool kFp16>
__device__ __forceinline__ float fits(float h) {
    constexpr float kMost = kFp16 ? 65504.f : 0x1.fep127f;
    return fabsf(h) > kMost && fabsf(h) <= kFloatMax ? copysignf(kMost, h) : h;
}

// H in two 16-bit parts, upper and rest: 16 bits and more of mantissa (fp16: 22, within twice its range, behind which H
// saturates, which is reported; an infinity or NaN goes to the upper part), so that the second product can run on the
// tensor cores
template <bool kFp16>
__device__ __forceinline__ void split_pair(uint32_t &up, uint32_t &rest, float lo, float hi) {
    up = pack_pair<kFp16>(fits<kFp16>(lo), fits<kFp16>(hi));
    const float rl = lo - from16(uint16_t(up), kFp16), rh = hi - from16(uint16_t(up >> 16), kFp16);
    rest = pack_pair<kFp16>(fabsf(lo) <= kFloatMax ? fits<kFp16>(rl) : 0.f,
                            fabsf(hi) <= kFloatMax ? fits<kFp16>(rh) : 0.f);
}
// fp16: a finite number that its two parts cannot hold
__device__ __forceinline__ bool beyond_parts(float h) { return fabsf(h) > 131008.f && fabsf(h) <= kFloatMax; }
__device__ __forceinline__ void report_range(const GroupedArgs &a) {
    ptx::record_error(a.err, 8u /*CF_ERR_DEVICE_BOUNDS*/, kInfoRange);
}
__device__ __forceinline__ void store_low(const GroupedArgs &a, int row, int r, float h) {
    if (a.fp16 && beyond_parts(h)) report_range(a);
    uint32_t up, rest;
    if (a.fp16) split_pair<true>(up, rest, h, 0.f);
    else split_pair<false>(up, rest, h, 0.f);
    uint16_t *y = static_cast<uint16_t *>(a.out) + size_t(row) * (2 * a.F) + r;
    y[0] = uint16_t(up);
    y[a.F] = uint16_t(rest);
}

// A warp's fragment, 32 rows of the batch x 32 features, on its way between the accumulator's layout and memory's.  In
// registers, as tmem_ld_blocks hands it out; in the warp's 2 KB of shared memory 64 bytes a row, its four 16-byte
// pieces at piece ^ row / 2 % 4, so that neither side meets bank conflicts; lane l then holds piece l % 4 of rows
// l / 4, + 8, + 16, + 24, and global memory is read and written in 16-byte pieces, 64 bytes a row.  (Turned a 16-bit
// value at a time, 6792 rows of 55 groups of 96 x 5344 took 54 us, now 49.)
struct Fragment {
    uint8_t *stg;
    int lane, cols;
    bool live;        // the piece's features exist
    size_t at, step;  // element of the first piece, and from a piece to the next
    __device__ uint8_t *piece(int i) const { return stg + i * 512 + ((lane >> 2) * 4 + ((lane ^ lane >> 3) & 3)) * 16; }
    __device__ uint32_t block(int k) const {
        return ptx::smem_u32(stg) + uint32_t(k * 512 + ((lane & 7) * 4 + ((lane >> 3 ^ lane >> 1) & 3)) * 16);
    }
    // memory's pieces in, the pairs of column block k and feature block b out, at p[4 k + b]
    __device__ void load(const uint4 (&z)[4], uint32_t (&p)[16]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4 *>(piece(i)) = z[i];
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 4; ++k) ptx::ldmatrix4_t(block(k), p[4 * k], p[4 * k + 1], p[4 * k + 2], p[4 * k + 3]);
        __syncwarp();
    }
    // the same back to memory
    __device__ void store(void *out, const uint32_t (&p)[16]) const {
#pragma unroll
        for (int k = 0; k < 4; ++k) ptx::stmatrix4_t(block(k), p[4 * k], p[4 * k + 1], p[4 * k + 2], p[4 * k + 3]);
        __syncwarp();
        uint16_t *y = static_cast<uint16_t *>(out) + at;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (live && (lane >> 2) + 8 * i < cols)
                *reinterpret_cast<uint4 *>(y + i * step) = *reinterpret_cast<const uint4 *>(piece(i));
        __syncwarp();
    }
    // index of the first of the two accumulators that make p[4 k + b]
    __device__ static constexpr int pair(int k, int b) { return 16 * (b / 2) + 4 * k + 2 * (b % 2); }
    // the accumulators, rounded
    template <bool kFp16>
    __device__ static void pack(uint32_t (&p)[16], const uint32_t (&v)[32]) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int j = pair(i / 4, i % 4);
            p[i] = pack_pair<kFp16>(__uint_as_float(v[j]), __uint_as_float(v[j + 1]));
        }
    }
    __device__ void store_rounded(void *out, const uint32_t (&v)[32], bool fp16) const {
        uint32_t p[16];
        if (fp16) pack<true>(p, v);
        else pack<false>(p, v);
        store(out, p);
    }
    // the accumulators times scale, split
    template <bool kFp16>
    __device__ static void split(uint32_t (&up)[16], uint32_t (&rest)[16], const uint32_t (&v)[32], float scale) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int j = pair(i / 4, i % 4);
            split_pair<kFp16>(up[i], rest[i], scale * __uint_as_float(v[j]), scale * __uint_as_float(v[j + 1]));
        }
    }
};

// WGRAD: 32 of a 64-column block's columns of this lane's row of dW into the warp's 4 KB of shared memory (16-byte pieces
// at piece ^ row % 8, so that neither side of the turn meets bank conflicts): the first (hi 0) or the second (4) half
template <bool kFp16>
__device__ __forceinline__ void put_columns(const uint32_t (&v)[32], uint4 *stg, int hi, int lane) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            p[i] = pack_pair<kFp16>(__uint_as_float(v[8 * j + 2 * i]), __uint_as_float(v[8 * j + 2 * i + 1]));
        stg[lane * 8 + ((hi + j) ^ (lane & 7))] = make_uint4(p[0], p[1], p[2], p[3]);
    }
}
// ... and the block's rows out of it, 128 bytes each
__device__ __forceinline__ void store_columns(const GroupedArgs &a, const Tile &w, int c0, const uint4 *stg, int q,
                                              int lane, bool ok) {
    __syncwarp();
    const int piece = lane & 7, f0 = w.f0 + q * 32 + (lane >> 3);
    uint16_t *y = static_cast<uint16_t *>(a.out) + (size_t(w.g) * a.F + f0) * a.N + w.col0 + c0 + piece * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int row = (lane >> 3) + 4 * i;
        if (ok && f0 + 4 * i < a.F && c0 + piece * 8 < w.n)  // N is a multiple of 8
            *reinterpret_cast<uint4 *>(y + size_t(4 * i) * a.N) = stg[row * 8 + (piece ^ (row & 7))];
    }
    __syncwarp();
}

// a fragment in registers (32 rows of this lane's feature) turned in the warp's 4 KB of shared memory ...
__device__ __forceinline__ void turn(const uint32_t (&v)[32], float *stg, int lane) {
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 32; ++j) stg[j * 32 + lane] = __uint_as_float(v[j]);
    __syncwarp();
}
// ... and read back as 8 features of row lane / 4 + 8i, features (lane % 4) * 8 and on
__device__ __forceinline__ void turned(float (&x)[8], const float *stg, int lane, int i) {
    const float4 *s = reinterpret_cast<const float4 *>(stg + ((lane >> 2) + 8 * i) * 32 + (lane & 3) * 8);
    const float4 l = s[0], h = s[1];
    x[0] = l.x, x[1] = l.y, x[2] = l.z, x[3] = l.w;
    x[4] = h.x, x[5] = h.y, x[6] = h.z, x[7] = h.w;
}

// the pieces of the pre-activation's fragment at column c of the tile (zeros outside)
__device__ __forceinline__ void load_fragment(uint4 (&z)[4], const GroupedArgs &a, const Tile &w, int c, int q,
                                              int lane, bool ok) {
    const int f = w.f0 + q * 32 + (lane & 3) * 8;
    const uint16_t *p = static_cast<const uint16_t *>(a.preact) + size_t(w.col0 + c + (lane >> 2)) * a.F + f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        z[i] = ok && f < a.F && c + (lane >> 2) + 8 * i < w.n
                   ? *reinterpret_cast<const uint4 *>(p + size_t(8 * i) * a.F) : make_uint4(0u, 0u, 0u, 0u);
}

// The group table from the raw offsets (in off[]) and adapters (in ad[]), by one warp: offsets clamped to [0, T] and
// to not decrease, adapters outside -1 .. L-1 made -1, the running numbers of tiles, the plan.  It stands between the
// offsets' arrival and the first copy, so it is short: one pass of 32 groups at a time, no 64-bit division.
template <int KIND, bool kPair>
__device__ void scan_table(const Table &tab, const GroupedArgs &a, int workers, uint32_t *err) {
    const int lane = threadIdx.x & 31;
    const int ft = feature_tiles<kPair>(a);
    const int shift = 31 - __clz(a.bn);
    constexpr uint32_t kAll = 0xffffffffu;
    const int raw0 = tab.off[0];
    int lo_all = min(max(raw0, 0), a.T);  // end of the groups before, clamped
    bool bad = raw0 != lo_all;
    const int first = lo_all;
    int carry = 0, longest = 0, ngroups = 0;
    uint32_t long_before = 1u;
    int turns = 0, last_ad = -1;  // LORA
    // No branches on the lane from here to the plan: lanes behind the last group repeat its end, count nothing and
    // store what is stored there anyway.  (With branches between them the shuffles took 2000 cycles and more.)
    tab.off[0] = first;
    for (int i0 = 0; i0 < a.groups; i0 += 32) {
        const int i = i0 + lane;
        const bool in = i < a.groups;
        const int at = in ? i : a.groups - 1;
        const int raw = tab.off[at + 1];
        int v = min(max(raw, lo_all), a.T);
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(kAll, v, d);
            v = lane >= d ? max(v, o) : v;
        }
        const int up = __shfl_up_sync(kAll, v, 1);
        const int lo = lane == 0 ? lo_all : up;
        lo_all = __shfl_sync(kAll, v, 31);
        const int rows = in ? v - lo : 0;
        bad |= in && v != raw;
        tab.off[at + 1] = v;
        int count;
        if constexpr (KIND == GR_WGRAD) {
            count = in ? max((rows + kBK - 1) / kBK, 1) : 0;
            longest = max(longest, count);
        } else {
            count = ft * ((rows + a.bn - 1) >> shift);
        }
        if constexpr (KIND == GR_SHRINK || KIND == GR_LORA) {
            int w = tab.ad[at];
            const bool wrong = w < -1 || w >= a.nweights;
            bad |= in && wrong;
            w = wrong ? -1 : w;
            tab.ad[at] = w;
            count = KIND == GR_SHRINK && (w < 0 || rows <= kShortRows) ? 0 : count;
            if constexpr (KIND == GR_LORA) {
                // a long request is a group of its own, a run of short ones another
                const uint32_t longs = __ballot_sync(kAll, rows >= a.long_rows);
                const uint32_t some = __ballot_sync(kAll, in);
                const uint32_t m = (longs | (longs << 1) | long_before) & some;  // groups start here
                long_before = longs >> 31;
                const int gi = m >> lane & 1u ? ngroups + __popc(m & ((1u << lane) - 1u)) : a.groups;
                tab.goff[gi] = lo;  // (the last entry is a dummy, or written below)
                tab.gad[gi] = rows >= a.long_rows ? w : -2;
                ngroups += __popc(m);
                const int left = __shfl_up_sync(kAll, w, 1);
                const uint32_t changes = __ballot_sync(kAll, w != (lane == 0 ? last_ad : left));
                tab.turn[at] = turns + __popc(changes & (0xffffffffu >> (31 - lane)));
                turns += __popc(changes);
                last_ad = __shfl_sync(kAll, w, 31);
            }
        }
        if constexpr (KIND != GR_LORA) {
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int o = __shfl_up_sync(kAll, count, d);
                count += lane >= d ? o : 0;
            }
            tab.pre[at + 1] = carry + count;
            carry += __shfl_sync(kAll, count, 31);
        }
    }
    if constexpr (KIND == GR_LORA) {
        __syncwarp();
        tab.goff[ngroups] = lo_all;
        __syncwarp();
        for (int i0 = 0; i0 < a.groups; i0 += 32) {
            const int i = i0 + lane;
            const int at = i < ngroups ? i : ngroups - 1;
            // a run that joins the long request before it (there is one, but for the first group) has no tiles
            const int here = tab.gad[at], behind = tab.gad[min(at + 1, ngroups - 1)];
            const int own = tab.goff[at + 1] - tab.goff[at], run = tab.goff[min(at + 2, ngroups)] - tab.goff[at + 1];
            const bool joins = here == -2 && at > 0 && own <= kRunRows;
            const bool takes = here != -2 && behind == -2 && run <= kRunRows;
            const int rows = (joins ? 0 : own) + (takes ? run : 0);
            int count = i < ngroups ? ft * ((rows + a.bn - 1) >> shift) : 0;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int o = __shfl_up_sync(kAll, count, d);
                count += lane >= d ? o : 0;
            }
            tab.pre[at + 1] = carry + count;
            carry += __shfl_sync(kAll, count, 31);
        }
    } else {
        ngroups = a.groups;
    }
    if constexpr (KIND == GR_WGRAD) longest = __reduce_max_sync(kAll, longest);
    // Rounds of whole tiles against equal stretches, in blocks; what adding pieces costs is in the host's plan
    // (grouped_cycles), which chose the tiles.  Every lane decides alike; divisions that do not need one another are
    // worked out side by side, a lane each (in a row they took 600 cycles of a launch of 10000).
    const int rows_all = lo_all - first;
    constexpr long long kMost = 1 << 30;  // blocks of all tiles: sums of them and of the workers then fit an int
    const int per_tile = KIND == GR_WGRAD ? ft * ((a.N + a.bn - 1) >> shift) : 1;
    const int nkc = (a.C + kBK - 1) / kBK;
    Plan p;
    p.split = 0;
    p.workers = workers;
    p.tiles = KIND == GR_WGRAD ? ngroups * per_tile : carry;
    p.ways = p.base = p.rem = 0;
    p.groups = ngroups;
    const bool few = KIND == GR_WGRAD ? ngroups <= kGroupedSplitTiles && per_tile <= kGroupedSplitTiles &&
                                            p.tiles <= kGroupedSplitTiles &&
                                            static_cast<long long>(per_tile) * carry <= kMost
                                      : carry <= kGroupedSplitTiles && static_cast<long long>(p.tiles) * nkc <= kMost;
    if (!kPair && a.partials != nullptr && few && p.tiles > 0) {
        auto divide = [&](int n0, int d0, int n1, int d1, int n2, int d2, int n3, int d3) {
            const int n = lane == 0 ? n0 : lane == 1 ? n1 : lane == 2 ? n2 : n3;
            const int d = lane == 0 ? d0 : lane == 1 ? d1 : lane == 2 ? d2 : d3;
            const int q = n / d;
            return make_int4(__shfl_sync(kAll, q, 0), __shfl_sync(kAll, q, 1), __shfl_sync(kAll, q, 2),
                             __shfl_sync(kAll, q, 3));
        };
        const int units = KIND == GR_WGRAD ? per_tile * carry : p.tiles * nkc;
        const int4 of = divide(units + workers - 1, workers, p.tiles + workers - 1, workers,
                               KIND == GR_WGRAD ? units + p.tiles - 1 : workers, p.tiles,
                               KIND == GR_WGRAD ? 0 : rows_all + ngroups - 1, ngroups);
        const int share = of.x, rounds = of.y;
        const int stretch = max(share, kMinStretch);
        // WGRAD: of mean tiles, or the longest one
        const int whole0 = max(rounds * (KIND == GR_WGRAD ? of.z : nkc), longest);
        // Equal parts of every tile, where there are workers for two at least: a worker then has one piece, not the
        // end of one tile and the start of another, each of which costs what adding a piece costs.
        const int most = KIND == GR_WGRAD ? 0 : min(of.z, nkc / kMinStretch);
        const int cols = KIND == GR_WGRAD ? a.bn : min(a.bn, of.w + 15);  // columns of a tile, about
        const int block = max(max(kMmaCycles20Columns * cols / 20, kMmaCyclesLeast), a.copy_cycles);
        const int4 in = divide(kDivideCycles + kDivideCyclesColumn * cols, block, a.wait_cycles, block, nkc + most - 1,
                               max(most, 1), units, stretch);
        const int adding = in.x + 1, least = in.y;  // no tile can be finished before
        const int whole = max(whole0, least);
        const int even = most >= 2 ? max(in.z, least) + adding : 1 << 30;
        const int mixed = max(stretch, least) + adding + adding / 2;
        if (whole > min(even, mixed)) {
            p.split = 1;
            if (even <= mixed) {
                p.ways = most;
                p.workers = p.tiles * most;
            } else {
                p.workers = stretch == share ? workers : max(in.w, 1);
                p.base = units / p.workers;
                p.rem = units - p.base * p.workers;
            }
        }
    }
    if (lane == 0) {
        tab.pre[0] = 0;
        *tab.plan = p;
    }
    if (__any_sync(kAll, bad) && lane == 0 && blockIdx.x == 0)
        ptx::record_error(err, 8u /*CF_ERR_DEVICE_BOUNDS*/, kInfoTable);
}

// A block of the contraction stages 16 KB of the feature operand (8 KB where there are no more than 64 features; what
// is behind the last feature is zero or stale, in lanes that are never stored) and the tile's columns: one box of rows,
// of the full width or of half of it.  (An SM takes 75 B of copies a cycle: a group of up to 128 rows at 256 columns
// takes 440 cycles a block by half boxes, 650 by full ones.)  Rows of a box behind the tile's are its neighbour's, in
// columns that are not multiplied or not stored.  WGRAD: 64-column blocks to fill.
template <bool kPair>
__device__ __forceinline__ bool half_box(const GroupedArgs &a, const Tile &w) {
    return kPair ? w.nm <= a.bn / 2 : 2 * w.nm <= a.bn;
}
template <int KIND, bool kPair>
__device__ __forceinline__ int b_blocks(const GroupedArgs &a, const Tile &w) {
    const int cols = kPair ? w.nm / 2 : w.nm;
    return KIND == GR_WGRAD ? (a.b_split ? (cols + 63) / 64 : (kPair ? a.bn / 2 : a.bn) / 64) : 1;
}
template <int KIND, bool kPair>
__device__ __forceinline__ uint32_t b_bytes(const GroupedArgs &a, int blocks, bool half) {
    return KIND == GR_WGRAD ? uint32_t(blocks) * 8192u : uint32_t(kPair ? a.bn / 2 : a.bn) * (half ? 64u : 128u);
}

// WGRAD: rows left .. 16*steps - 1 of every 64-column block of the stage (a row is 128 bytes of a block) become
// zeros, by one warp; then the async proxy may read them
__device__ __forceinline__ void zero_tail(uint8_t *st, int left, int steps, int blocks, int lane) {
    const int per = (16 * steps - left) * 8;  // 16-byte pieces per block; the blocks of X, then those of dY
    for (int blk = 0; blk < blocks; ++blk)
        for (int p = lane; p < per; p += 32)
            *reinterpret_cast<uint4 *>(st + blk * 8192 + left * 128 + p * 16) = make_uint4(0u, 0u, 0u, 0u);
    ptx::fence_proxy_async_smem();
    __syncwarp();
}

// Where the pieces of a divided tile lie: the first may be the second slot of its worker, every later one starts its
// worker's stretch.
struct Pieces {
    const float *p0, *p;  // of the first piece, of the second
    size_t step;          // from the second on
    int more;             // pieces behind the first
};
template <int KIND, bool kPair>
__device__ __forceinline__ Pieces pieces_of(const GroupedArgs &a, const Walk<KIND, kPair> &walk, const Tile &w) {
    const int u0 = KIND == GR_WGRAD
                       ? walk.per_group * walk.tab.pre[w.g] + (w.id - w.g * walk.per_group) * max(w.nk, 1)
                       : w.id * w.nk;
    const size_t piece = size_t(kFB) * a.bn;
    return Pieces{a.partials + size_t(2 * w.first + walk.slot_of(w.first, u0)) * piece,
                  a.partials + size_t(2 * (w.first + 1)) * piece, 2 * piece, w.last - w.first};
}

// WGRAD: the pieces at 32 columns from c on of one lane, added in worker order
__device__ __forceinline__ void sum_pieces(uint32_t (&v)[32], const Pieces &pc, int c, int n, int l) {
    const int cols = min(32, n - c);
    const size_t at = size_t(c) * kFB + l;
    float s[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) s[j] = j < cols ? __ldcg(pc.p0 + at + j * kFB) : 0.f;
    for (int k = 0; k < pc.more; k += 2) {  // two pieces' loads in flight
        float x[2][32];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 32; ++j)
                x[i][j] = k + i < pc.more && j < cols ? __ldcg(pc.p + (k + i) * pc.step + at + j * kFB) : 0.f;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 32; ++j) s[j] += x[i][j];
    }
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(s[j]);
}

// Four features of one row, finished and stored: s holds the products.
template <int KIND>
__device__ __forceinline__ void finish_row(const GroupedArgs &a, const Tile &w, int row, int f, float4 s4) {
    const bool fp16 = a.fp16 != 0;
    float s[4] = {s4.x, s4.y, s4.z, s4.w};
    if constexpr (KIND == GR_SHRINK) {
        const float sc = a.scale ? __ldg(a.scale + w.w) : 1.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) store_low(a, row, f + i, sc * s[i]);
        return;
    }
    const size_t at = size_t(row) * a.F + f;
    if (KIND == GR_FORWARD && a.preact)
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.preact) + at) =
            make_uint2(pack16(s[0], s[1], fp16), pack16(s[2], s[3], fp16));
    if (KIND == GR_FORWARD && a.act) {
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] = gelu(s[i]);
    }
    if (KIND == GR_DGRAD && a.preact) {
        const uint2 z = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(a.preact) + at);
        const uint32_t zw[2] = {z.x, z.y};
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] *= gelu_slope(from16(uint16_t(zw[i / 2] >> ((i & 1) * 16)), fp16));
    }
    if (KIND == GR_LORA && a.bias) {
        const float4 b = __ldg(reinterpret_cast<const float4 *>(a.bias + f));
        s[0] += b.x, s[1] += b.y, s[2] += b.z, s[3] += b.w;
    }
    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) + at) =
        make_uint2(pack16(s[0], s[1], fp16), pack16(s[2], s[3], fp16));
}

// The pieces of a divided tile added in worker order and finished (all kinds but WGRAD).  A warp takes whole columns,
// that is rows of the batch: a lane 4 neighbouring features, so the loads are 512 bytes a warp and the stores whole
// rows, and nothing needs turning.  kCols columns of four pieces are in flight.
template <int KIND, int kCols>
__device__ __forceinline__ void finish_columns(const GroupedArgs &a, const Tile &w, const Pieces &pc, int e, int lane) {
    constexpr int kWarps = epi_warps(KIND), kFly = 4;
    const int f = w.f0 + 4 * lane;
    if (f >= a.F) return;
#pragma unroll 1
    for (int j = e; j < w.n; j += kCols * kWarps) {
        const size_t at = size_t(j) * kFB + 4 * lane;
        float4 s[kCols];
#pragma unroll
        for (int h = 0; h < kCols; ++h) s[h] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
        for (int k = 0; k <= pc.more; k += kFly) {
            float4 x[kFly][kCols];
#pragma unroll
            for (int i = 0; i < kFly; ++i) {
                const float *p = (k + i == 0 ? pc.p0 : pc.p + (k + i - 1) * pc.step) + at;
#pragma unroll
                for (int h = 0; h < kCols; ++h)
                    x[i][h] = k + i <= pc.more && j + h * kWarps < w.n
                                  ? __ldcg(reinterpret_cast<const float4 *>(p + h * kWarps * kFB))
                                  : make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll
            for (int i = 0; i < kFly; ++i)
#pragma unroll
                for (int h = 0; h < kCols; ++h)
                    s[h].x += x[i][h].x, s[h].y += x[i][h].y, s[h].z += x[i][h].z, s[h].w += x[i][h].w;
        }
#pragma unroll
        for (int h = 0; h < kCols; ++h)
            if (j + h * kWarps < w.n) finish_row<KIND>(a, w, w.col0 + j + h * kWarps, f, s[h]);
    }
}
template <int KIND>
__device__ __forceinline__ void finish_pieces(const GroupedArgs &a, const Tile &w, const Pieces &pc, int e, int lane) {
    if constexpr (KIND == GR_SHRINK) {  // few features: lanes go over rows and features alike
        const int nf = a.F / 4;
        for (int i = e * 32 + lane; i < w.n * nf; i += 128) {
            const int j = i / nf, f = (i - j * nf) * 4;
            const size_t at = size_t(j) * kFB + f;
            float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int k = 0; k <= pc.more; k += 8) {
                float4 x[8];
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    x[q] = k + q <= pc.more ? __ldcg(reinterpret_cast<const float4 *>(
                                                  (k + q == 0 ? pc.p0 : pc.p + (k + q - 1) * pc.step) + at))
                                            : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int q = 0; q < 8; ++q) s.x += x[q].x, s.y += x[q].y, s.z += x[q].z, s.w += x[q].w;
            }
            finish_row<KIND>(a, w, w.col0 + j, f, s);
        }
    } else {  // (as few columns at a time as there are: code that is run once or twice is mostly fetched)
        if (w.n <= epi_warps(KIND)) finish_columns<KIND, 1>(a, w, pc, e, lane);
        else finish_columns<KIND, 4>(a, w, pc, e, lane);
    }
}

// LORA, a tile with rows of several requests: the adapters' second product on the CUDA cores, in fp32.  Each row takes
// its own adapter's B and nothing of another's, so a NaN in an adapter stays with its requests.
// x: this lane's 8 features (from f on) of one row; four lanes cover a row's 32 features, eight rows go side by side
// with an adapter each, and lanes of one adapter read the same addresses.  L2's latency bounds it, 1000 cycles for 8
// ranks; from rank 32 on 16 are in flight (13434 rows of 27 requests at rank 64: 67 us, now 58).
template <int kRanks>
__device__ __forceinline__ void low_rank_step(float (&x)[8], const uint16_t *b, const uint16_t *h, int rank, int step,
                                              bool fp16) {
    uint4 bv[kRanks], up[kRanks / 8], rest[kRanks / 8];
#pragma unroll
    for (int k = 0; k < kRanks; ++k) bv[k] = __ldg(reinterpret_cast<const uint4 *>(b + size_t(k) * step));
#pragma unroll
    for (int g = 0; g < kRanks / 8; ++g) {
        up[g] = __ldcg(reinterpret_cast<const uint4 *>(h + 8 * g));
        rest[g] = __ldcg(reinterpret_cast<const uint4 *>(h + rank + 8 * g));
    }
#pragma unroll
    for (int k = 0; k < kRanks; ++k) {
        const uint4 u = up[k / 8], l = rest[k / 8];
        const uint32_t uw[4] = {u.x, u.y, u.z, u.w}, lw[4] = {l.x, l.y, l.z, l.w};
        const float hk = from16(uint16_t(uw[k % 8 / 2] >> ((k & 1) * 16)), fp16) +
                         from16(uint16_t(lw[k % 8 / 2] >> ((k & 1) * 16)), fp16);
        const uint32_t w[4] = {bv[k].x, bv[k].y, bv[k].z, bv[k].w};
#pragma unroll
        for (int p = 0; p < 4; ++p)
            ptx::fma2(x[2 * p], x[2 * p + 1], hk, hk, from16(uint16_t(w[p]), fp16),
                      from16(uint16_t(w[p] >> 16), fp16), x[2 * p], x[2 * p + 1]);
    }
}
__device__ __forceinline__ void add_low_rank(float (&x)[8], const GroupedArgs &a, int ad, int row, int f) {
    if (ad < 0) return;
    const int rank = a.rank;
    const bool fp16 = a.fp16 != 0;
    const uint16_t *b = static_cast<const uint16_t *>(a.lora_b) + size_t(ad) * rank * a.F + f;
    const uint16_t *h = static_cast<const uint16_t *>(a.low) + size_t(row) * (2 * rank);
    int r = 0;
    if (rank >= 32) {
#pragma unroll 1
        for (; r + 16 <= rank; r += 16) low_rank_step<16>(x, b + size_t(r) * a.F, h + r, rank, a.F, fp16);
    }
#pragma unroll 1
    for (; r < rank; r += 8) low_rank_step<8>(x, b + size_t(r) * a.F, h + r, rank, a.F, fp16);
}

// One lane's share of a short request: rows of A (8 ranks, a 16-byte piece) `step` apart, `left` rows until the end,
// against up to kRows rows of X; the lanes of a warp that hold the same ranks are then added, in a fixed order, into
// sums[row][64].  kFly pieces in flight: one row takes fewer registers for its sums, so more loads (beside the
// projection, which saturates HBM at the same time, each turn of the loop costs about 2000 cycles).
template <int kRows, int kFly>
__device__ __forceinline__ void short_sums(const GroupedArgs &a, const uint16_t *wa, const uint16_t *x, int left,
                                           int step, int rows, int shift, int lane, float *sums, bool live) {
    const bool fp16 = a.fp16 != 0;
    float acc[8 * kRows];
#pragma unroll
    for (int i = 0; i < 8 * kRows; ++i) acc[i] = 0.f;
#pragma unroll 1
    for (int k = 0; k < left; k += kFly * step) {
        uint4 w[kFly];
        uint16_t xs[kFly];
#pragma unroll
        for (int i = 0; i < kFly; ++i) {
            const bool in = k + i * step < left;
            w[i] = in ? __ldg(reinterpret_cast<const uint4 *>(wa + size_t(k + i * step) * a.F))
                      : make_uint4(0u, 0u, 0u, 0u);
            xs[i] = in ? __ldg(x + k + i * step) : uint16_t(0);
        }
#pragma unroll
        for (int j = 0; j < kRows; ++j) {
            if (j >= rows) break;
            if (j > 0) {
#pragma unroll
                for (int i = 0; i < kFly; ++i)
                    xs[i] = k + i * step < left ? __ldg(x + size_t(j) * a.C + k + i * step) : uint16_t(0);
            }
#pragma unroll
            for (int i = 0; i < kFly; ++i) {
                const float xv = from16(xs[i], fp16);
                const uint32_t ww[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
                for (int p = 0; p < 4; ++p)
                    ptx::fma2(acc[8 * j + 2 * p], acc[8 * j + 2 * p + 1], xv, xv, from16(uint16_t(ww[p]), fp16),
                              from16(uint16_t(ww[p] >> 16), fp16), acc[8 * j + 2 * p], acc[8 * j + 2 * p + 1]);
            }
        }
    }
    __syncwarp();
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) {
#pragma unroll
        for (int i = 0; i < 8 * kRows; ++i) {
            const float o = __shfl_xor_sync(0xffffffffu, acc[i], d);
            acc[i] = d >= (1 << shift) ? acc[i] + o : acc[i];
        }
    }
    if (lane < (1 << shift) && live) {
#pragma unroll
        for (int i = 0; i < 8 * kRows; ++i) sums[(i / 8) * 64 + (i & 7)] = acc[i];
    }
}

// SHRINK, short requests: H on the CUDA cores, in fp32, by the warps from 2 on (192 threads).  A unit is a request, up
// to 64 ranks and one of low_split parts of the contraction (added by the last to arrive): neighbouring lanes take
// neighbouring 16-byte pieces of A's rows, for up to 4 rows of X at a time; the sums are folded over the lanes of equal
// ranks, then over the warps.  (As tiles, a request of one row took a copy of 64 rows of 32 bytes per block at rank
// 16, some 640 cycles of copy engine each.)
__device__ void shrink_short(const GroupedArgs &a, const Table &tab, float *sums, volatile uint32_t *verdict) {
    const int tid = threadIdx.x - 64, lane = tid & 31, warp = tid >> 5;
    const int chunks = (a.F + 63) / 64;
    const bool fp16 = a.fp16 != 0;
    const int span = ((a.C / 8 + a.low_split - 1) / a.low_split) * 8;
    for (int u = blockIdx.x; u < a.groups * chunks * a.low_split; u += gridDim.x) {
        const int part = u % a.low_split, uc = u / a.low_split;
        const int s = uc / chunks, r0 = (uc - s * chunks) * 64;
        const int lo = tab.off[s];
        // (one for the warp, and known to be: see the group table on shuffles)
        const int rows = __shfl_sync(0xffffffffu, tab.off[s + 1] - lo, 0), ad = __shfl_sync(0xffffffffu, tab.ad[s], 0);
        if (ad < 0 || rows == 0 || rows > kShortRows) continue;
        // pieces of 8 ranks in a row of the unit: lane = (row of A) * 2^shift + piece
        const int pieces = min(a.F - r0, 64) / 8;
        const int shift = pieces > 4 ? 3 : pieces > 2 ? 2 : pieces - 1;
        const int piece = lane & ((1 << shift) - 1);
        const bool live = piece < pieces;
        const int step = (kShortWarps * 32) >> shift;  // rows of A side by side
        const uint16_t *wa =
            static_cast<const uint16_t *>(a.lora_a) + size_t(ad) * a.C * a.F + r0 + (live ? piece * 8 : 0);
        const int k_end = min(a.C, (part + 1) * span);
        for (int t0 = 0; t0 < rows; t0 += 4) {
            const uint16_t *x = static_cast<const uint16_t *>(a.x) + size_t(lo + t0) * a.C;
            const int k0 = part * span + (tid >> shift);
            const uint16_t *row = wa + size_t(k0) * a.F;
            float *const mine = sums + warp * 256 + piece * 8;
            if (rows == 1) short_sums<1, 12>(a, row, x + k0, k_end - k0, step, 1, shift, lane, mine, live);
            else short_sums<4, 6>(a, row, x + k0, k_end - k0, step, rows - t0, shift, lane, mine, live);
            ptx::named_bar_sync(4, kShortWarps * 32);
            for (int i = tid; i < 4 * pieces * 8; i += kShortWarps * 32) {
                const int j = i / (pieces * 8), r = i - j * pieces * 8;
                if (t0 + j < rows) {
                    float h = 0.f;
#pragma unroll
                    for (int g = 0; g < kShortWarps; ++g) h += sums[(g * 4 + j) * 64 + r];
                    float *const parts = a.low_parts + (size_t(uc) * a.low_split + part) * (kShortRows * 64);
                    if (a.low_split > 1) __stcg(parts + (t0 + j) * 64 + r, h);
                    else store_low(a, lo + t0 + j, r0 + r, a.scale ? h * __ldg(a.scale + ad) : h);
                }
            }
            ptx::named_bar_sync(4, kShortWarps * 32);
        }
        if (a.low_split > 1) {  // the parts, added in order by whoever comes last
            if (tid == 0) {
                const bool last = ptx::atom_add_acq_rel_gpu(a.low_counters + uc, 1u) == uint32_t(a.low_split - 1);
                if (last) ptx::st_relaxed_gpu(a.low_counters + uc, 0u);
                *verdict = last;
            }
            ptx::named_bar_sync(4, kShortWarps * 32);
            if (*verdict != 0u) {
                const float sc = a.scale ? __ldg(a.scale + ad) : 1.f;
                for (int i = tid; i < rows * pieces * 8; i += kShortWarps * 32) {
                    const int j = i / (pieces * 8), r = i - j * pieces * 8;
                    const float *p = a.low_parts + size_t(uc) * a.low_split * (kShortRows * 64) + j * 64 + r;
                    float x[kLoraMaxSplit], h = 0.f;
#pragma unroll
                    for (int k = 0; k < kLoraMaxSplit; ++k)
                        x[k] = k < a.low_split ? __ldcg(p + k * (kShortRows * 64)) : 0.f;
#pragma unroll
                    for (int k = 0; k < kLoraMaxSplit; ++k) h += x[k];
                    store_low(a, lo + j, r0 + r, h * sc);
                }
            }
            ptx::named_bar_sync(4, kShortWarps * 32);
        }
    }
}

template <bool kPair>
__device__ __forceinline__ void issue_mma(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t accumulate) {
    if constexpr (kPair) ptx::mma_bf16_pair(d, ad, bd, idesc, accumulate);
    else ptx::mma_bf16(d, ad, bd, idesc, accumulate);
}
// arrive when the MMAs issued so far are complete (a pair: on both CTAs' barrier)
template <bool kPair>
__device__ __forceinline__ void issue_commit(uint32_t bar) {
    if constexpr (kPair) ptx::mma_commit_pair_mc(bar, 3);
    else ptx::mma_commit(bar);
}
// The four MMAs of a 64-deep block and the commit that frees its stage (pair: in both CTAs), issued by one elected lane
// of a converged warp.  kA, kB: from 16 of the contraction to the next, in descriptor units.
template <bool kPair, int kA, int kB>
__device__ __forceinline__ void mma_block(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t accumulate,
                                          uint32_t bar) {
    if constexpr (kPair) {
        asm volatile(
            "{\n\t.reg .pred e, p, t;\n\t.reg .b64 a, b;\n\t.reg .b16 m;\n\t"
            "elect.sync _|e, 0xffffffff;\n\t"
            "setp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 t, 0, 0;\n\tmov.b16 m, 3;\n\t"
            "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t"
            "add.s64 a, %1, %6;\n\tadd.s64 b, %2, %7;\n\t"
            "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %3, t;\n\t"
            "add.s64 a, %1, %8;\n\tadd.s64 b, %2, %9;\n\t"
            "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %3, t;\n\t"
            "add.s64 a, %1, %10;\n\tadd.s64 b, %2, %11;\n\t"
            "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %3, t;\n\t"
            "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%5], m;\n\t}"
            ::"r"(d), "l"(ad), "l"(bd), "r"(idesc), "r"(accumulate), "r"(bar), "n"(kA), "n"(kB), "n"(2 * kA),
            "n"(2 * kB), "n"(3 * kA), "n"(3 * kB)
            : "memory");
    } else {
        asm volatile(
            "{\n\t.reg .pred e, p, t;\n\t.reg .b64 a, b;\n\t"
            "elect.sync _|e, 0xffffffff;\n\t"
            "setp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
            "add.s64 a, %1, %6;\n\tadd.s64 b, %2, %7;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
            "add.s64 a, %1, %8;\n\tadd.s64 b, %2, %9;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
            "add.s64 a, %1, %10;\n\tadd.s64 b, %2, %11;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
            "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%5];\n\t}"
            ::"r"(d), "l"(ad), "l"(bd), "r"(idesc), "r"(accumulate), "r"(bar), "n"(kA), "n"(kB), "n"(2 * kA),
            "n"(2 * kB), "n"(3 * kA), "n"(3 * kB)
            : "memory");
    }
}

// the 32-column fragment behind c of those that a half takes: spans of kSpan columns, one of kHalves
template <int kSpan, int kHalves>
__device__ __forceinline__ int next_fragment(int c) {
    return kSpan == 64 && (c & 32) == 0 ? c + 32 : c + 32 + (kHalves - 1) * kSpan;
}

// The copies of block kb into a stage, completing on `bar` (kShared: a barrier of either CTA of the pair)
template <int KIND, bool kShared>
__device__ __forceinline__ void stage_loads(const GroupedArgs &a, const Tile &w, uint32_t sa, uint32_t sb, uint32_t bar,
                                            int kb, int col0, int blocks, bool half) {
    const int k0 = kb * kBK;
    if constexpr (KIND == GR_WGRAD) {
        const int y = w.row0 + k0;
        if (a.a_split) {
            for (int i = 0; i < a.a_blocks; ++i) {
                if constexpr (kShared) ptx::tma_load_2d_pair(sa + i * 8192, &a.tmap_a, bar, w.f0 + 64 * i, y);
                else ptx::tma_load_2d(sa + i * 8192, &a.tmap_a, bar, w.f0 + 64 * i, y);
            }
        } else {
            if constexpr (kShared) ptx::tma_load_3d_pair(sa, &a.tmap_a, bar, 0, y, w.f0 / 64);
            else ptx::tma_load_3d(sa, &a.tmap_a, bar, 0, y, w.f0 / 64);
        }
        if (a.b_split) {
            for (int i = 0; i < blocks; ++i) {
                if constexpr (kShared) ptx::tma_load_2d_pair(sb + i * 8192, &a.tmap_b, bar, col0 + 64 * i, y);
                else ptx::tma_load_2d(sb + i * 8192, &a.tmap_b, bar, col0 + 64 * i, y);
            }
        } else {
            if constexpr (kShared) ptx::tma_load_3d_pair(sb, &a.tmap_b, bar, 0, y, col0 / 64);
            else ptx::tma_load_3d(sb, &a.tmap_b, bar, 0, y, col0 / 64);
        }
    } else {
        if constexpr (KIND == GR_DGRAD) {
            if constexpr (kShared) ptx::tma_load_3d_pair(sa, &a.tmap_a, bar, k0, w.f0, w.w);
            else ptx::tma_load_3d(sa, &a.tmap_a, bar, k0, w.f0, w.w);
        } else if (a.a_split) {
            for (int i = 0; i < a.a_blocks; ++i) {
                if constexpr (kShared) ptx::tma_load_3d_pair(sa + i * 8192, &a.tmap_a, bar, w.f0 + 64 * i, k0, w.w);
                else ptx::tma_load_3d(sa + i * 8192, &a.tmap_a, bar, w.f0 + 64 * i, k0, w.w);
            }
        } else {
            if constexpr (kShared) ptx::tma_load_4d_pair(sa, &a.tmap_a, bar, 0, k0, w.f0 / 64, w.w);
            else ptx::tma_load_4d(sa, &a.tmap_a, bar, 0, k0, w.f0 / 64, w.w);
        }
        const CUtensorMap *const rows = half ? &a.tmap_b2 : &a.tmap_b;
        if constexpr (kShared) ptx::tma_load_2d_pair(sb, rows, bar, k0, col0);
        else ptx::tma_load_2d(sb, rows, bar, k0, col0);
    }
}

// A value that every lane of the warp holds alike, known to be.
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }

// The bounded wait of a whole warp, one verdict.
template <bool kClusterScope = false>
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, uint64_t tmo, volatile uint32_t *abort,
                                          uint32_t *err, uint32_t info) {
    const bool now = kClusterScope ? ptx::mbar_try_wait_cluster(bar, parity) : ptx::mbar_try_wait(bar, parity);
    if (__all_sync(0xffffffffu, now)) return true;
    return __all_sync(0xffffffffu, ptx::mbar_wait_bounded<kClusterScope>(bar, parity, tmo, abort, err, info)) != 0;
}

// The producer loop, of a whole warp with an elected lane that issues (as in the MMA loop).
template <int KIND, bool kPair>
__device__ __forceinline__ void produce(const GroupedArgs &a, Walk<KIND, kPair> &walk, const GrLayout &L,
                                        const GrBars &B, uint32_t base, uint32_t crank, uint64_t tmo,
                                        volatile uint32_t *abort) {
    const int stages = a.stages;
    const bool leader = crank == 0u;
    const uint32_t full_lead = kPair ? ptx::mapa(B.full0, 0u) : B.full0;
    const bool elected = ptx::elect_one();
    uint32_t it = 0, s = 0, ph = 0;
    bool ok = true;
    // the low-rank product of a tile's first nx columns, of one adapter: blocks of 64 ranks, H's upper parts, then its
    // lower ones, against the same rows of B
    auto load_low_rank = [&](const Tile &t) {
        const int extra = uniform(t.extra);
        if (extra > 0) ptx::griddep_wait();  // H is the previous grid's
        for (int x = 0; x < extra && ok; ++x) {
            ok = wait_warp(B.empty0 + 8 * s, ph ^ 1u, tmo, abort, a.err, kInfoProducer | s);
            if (!ok) break;
            const int r0 = (x >> 1) * kBK;
            const uint32_t sa = base + s * L.stage_bytes;
            const uint32_t bar = full_lead + 8 * s;
            if (elected) {
                const uint32_t own = uint32_t(a.a_blocks) * 8192u + b_bytes<KIND, kPair>(a, 1, false);
                if (leader) ptx::mbar_arrive_expect_tx(B.full0 + 8 * s, kPair ? 2 * own : own);
                if (a.a_split) {
                    for (int i = 0; i < a.a_blocks; ++i) {
                        if constexpr (kPair)
                            ptx::tma_load_3d_pair(sa + i * 8192, &a.tmap_lb, bar, t.f0 + 64 * i, r0, t.ad);
                        else ptx::tma_load_3d(sa + i * 8192, &a.tmap_lb, bar, t.f0 + 64 * i, r0, t.ad);
                    }
                } else {
                    if constexpr (kPair) ptx::tma_load_4d_pair(sa, &a.tmap_lb, bar, 0, r0, t.f0 / 64, t.ad);
                    else ptx::tma_load_4d(sa, &a.tmap_lb, bar, 0, r0, t.f0 / 64, t.ad);
                }
                const int xh = (x & 1) * a.rank + r0, y = t.col0 + (kPair ? int(crank) * (t.nx / 2) : 0);
                if constexpr (kPair) ptx::tma_load_2d_pair(sa + L.a_bytes, &a.tmap_h, bar, xh, y);
                else ptx::tma_load_2d(sa + L.a_bytes, &a.tmap_h, bar, xh, y);
            }
            __syncwarp();
            ++it;
            if (++s == uint32_t(stages)) {
                s = 0;
                ph ^= 1u;
            }
        }
    };
    Tile w;
    while (ok && walk.next(w)) {
        const int kb0 = uniform(w.kb0), kb1 = uniform(w.kb1);
        const int cols = kPair ? w.nm / 2 : w.nm;  // columns this CTA stages
        const int col0 = w.col0 + int(crank) * cols;
        const int blocks = b_blocks<KIND, kPair>(a, w);
        const bool half = KIND != GR_WGRAD && half_box<kPair>(a, w);
        const uint32_t own = uint32_t(a.a_blocks) * 8192u + b_bytes<KIND, kPair>(a, blocks, half);
        for (int kb = kb0; kb < kb1; ++kb) {
            ok = wait_warp(B.empty0 + 8 * s, ph ^ 1u, tmo, abort, a.err, kInfoProducer | s);
            if (!ok) break;
            const uint32_t sa = base + s * L.stage_bytes;
            const uint32_t sb = sa + L.a_bytes;
            if (elected) {
                // A pair's loads complete on the leader's barrier.  (WGRAD: but for a group's last block where it
                // has to be zeroed behind the rows; the second CTA's part then completes on its own barrier, its
                // warp 1 zeroes and arrives.)
                const bool tail = kPair && KIND == GR_WGRAD && kb == w.nk - 1 && (w.rows & 15) != 0;
                if (!kPair || leader) {
                    ptx::mbar_arrive_expect_tx(B.full0 + 8 * s, kPair && !tail ? 2 * own : own);
                } else if (KIND == GR_WGRAD) {
                    if (tail) ptx::mbar_arrive_expect_tx(B.full0 + 8 * s, own);
                    else ptx::mbar_arrive_cluster_relaxed(full_lead + 8 * s);  // the loads count bytes
                }
                if (kPair && !(tail && !leader))
                    stage_loads<KIND, true>(a, w, sa, sb, full_lead + 8 * s, kb, col0, blocks, half);
                else stage_loads<KIND, false>(a, w, sa, sb, B.full0 + 8 * s, kb, col0, blocks, half);
            }
            __syncwarp();
            ++it;
            if (++s == uint32_t(stages)) {
                s = 0;
                ph ^= 1u;
            }
        }
        if constexpr (KIND == GR_LORA) load_low_rank(w);
    }
    // every load has landed and been read before the CTA may leave
    const uint32_t first = it > uint32_t(stages) ? it - uint32_t(stages) : 0u;
    for (uint32_t i = first; i < it; ++i) {
        volatile uint32_t local_abort = 0;
        ptx::mbar_wait_bounded(B.empty0 + 8 * (i % uint32_t(stages)), (i / uint32_t(stages)) & 1u, tmo, &local_abort,
                               nullptr, 0);
    }
}

template <int KIND, bool kPair>
__global__ void __maxnreg__(registers_of(KIND)) grouped_kernel(const __grid_constant__ GroupedArgs a) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t base = ptx::smem_u32(smem_raw);
    if ((base & 1023u) != 0u) {  // the swizzled operand tiles need it; see the fused GEMM
        ptx::griddep_wait();
        if (threadIdx.x == 0) ptx::record_error(a.err, 8u, 0x60000000u | (base & 1023u));
        return;
    }
    constexpr int kEpiWarps = epi_warps(KIND), kThreads = threads_of(KIND), kHalves = kEpiWarps / 4,
                  kSpan = KIND == GR_WGRAD ? 64 : 32;
    constexpr bool kAMn = KIND != GR_DGRAD;  // features contiguous in memory: A is MN-major
    constexpr bool kBMn = KIND == GR_WGRAD;
    const int stages = a.stages;
    const GrLayout L = gr_layout(KIND, kPair, stages, a.bn, a.groups, a.a_blocks);
    const GrBars B = gr_bars(base + L.bars, stages);
    const Table tab(smem_raw + L.table, KIND, a.groups);
    volatile uint32_t *misc = reinterpret_cast<volatile uint32_t *>(smem_raw + (B.misc - base));
    volatile uint32_t *abort = misc + 1;
    const uint64_t tmo = a.timeout_ns;
    const int warp = __shfl_sync(0xffffffffu, int(threadIdx.x >> 5), 0);  // one for the warp, and known to be
    const int lane = threadIdx.x & 31;
    const uint32_t tmem_cols = uint32_t(max(2 * a.bn, 64));  // (a fragment of the second accumulator's is 32 wide)
    // A pair (two CTAs of a cluster) works on one tile of 256 features: the even CTA issues MMAs of M = 256 that
    // read both CTAs' shared memory and write both tensor memories (128 features each).
    const uint32_t crank = kPair ? ptx::cluster_ctarank() : 0u;
    const bool leader = crank == 0u;
    const int worker = int(blockIdx.x) / (kPair ? 2 : 1), workers = int(gridDim.x) / (kPair ? 2 : 1);

    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) {
            // WGRAD pairs: the second CTA arrives too, when its part of the stage is ready
            ptx::mbar_init(B.full0 + 8 * s, kPair && KIND == GR_WGRAD && leader ? 2 : 1);
            ptx::mbar_init(B.empty0 + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            ptx::mbar_init(B.tmem_full0 + 8 * b, 1 + uint32_t(a.extra_arrivals));
            ptx::mbar_init(B.tmem_empty0 + 8 * b, kPair ? 2 * kEpiWarps : kEpiWarps);
        }
        ptx::mbar_init(B.mma_done, 1);
        misc[1] = 0u;
        ptx::fence_mbarrier_init_cluster();
    }
    if (warp == 1) {
        if constexpr (kPair) {
            ptx::tmem_alloc_pair(B.misc, tmem_cols);
            ptx::tmem_relinquish_pair();
        } else {
            ptx::tmem_alloc(B.misc, tmem_cols);
            ptx::tmem_relinquish();
        }
    }
    if (threadIdx.x == 0) {
        ptx::prefetch_tensormap(&a.tmap_a);
        ptx::prefetch_tensormap(&a.tmap_b);
    }
    // The next grid may start only once this CTA holds its tensor memory: a dependent CTA that took it first
    // would wait for this grid while this grid waited for the columns.
    __syncthreads();
    if constexpr (KIND == GR_SHRINK) {
        // LORA, launched next, reads what came before this grid without waiting: it must not start earlier
        ptx::griddep_wait();
        ptx::griddep_launch_dependents();
    } else {
        ptx::griddep_launch_dependents();
        if (KIND != GR_LORA || !a.after_shrink) ptx::griddep_wait();
    }
    // (LORA has not waited itself: nothing that another launch may have written is read through L1 before it has)
    for (int i = threadIdx.x; i <= a.groups; i += kThreads) {
        tab.off[i] = __ldcg(a.offsets + i);
        if constexpr (KIND == GR_SHRINK || KIND == GR_LORA)
            if (i < a.groups) tab.ad[i] = __ldcg(a.windex + i);
    }
    __syncthreads();
    if (warp == 0) scan_table<KIND, kPair>(tab, a, workers, a.err);
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if constexpr (kPair) ptx::cluster_sync();  // the peer's barriers are initialised before anything signals them
    const uint32_t tmem_base = misc[0];
    Walk<KIND, kPair> walk(tab, a, worker, int(crank) * kFB);
    Tile w;

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        produce<KIND, kPair>(a, walk, L, B, base, crank, tmo, abort);
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        // (WGRAD: the whole warp, which zeroes the rows behind a group in its last block)
        if (!leader) {
            if constexpr (kPair && KIND == GR_WGRAD) {
                // the second CTA of a pair: zero its part of each group's last block
                uint32_t s = 0, ph = 0;  // ring position of the tile's first block; a phase bit per stage
                while (walk.next(w)) {
                    if (w.nk > 0 && (w.rows & 15) != 0) {
                        const uint32_t at = (s + uint32_t(w.nk) - 1u) % uint32_t(stages);
                        const bool ok =
                            ptx::mbar_wait_bounded(B.full0 + 8 * at, (ph >> at) & 1u, tmo + uint64_t(w.nk) * kBlockNs,
                                                   abort, a.err, kInfoMma | 0x200u | at);
                        if (!__all_sync(0xffffffffu, ok)) break;
                        ph ^= 1u << at;
                        const int left = w.rows - (w.nk - 1) * kBK;
                        zero_tail(smem_raw + at * L.stage_bytes, left, (left + 15) / 16,
                                  a.a_blocks + (w.nm / 2 + 63) / 64, lane);
                        if (lane == 0) ptx::mbar_arrive_cluster(ptx::mapa(B.full0 + 8 * at, 0u));
                    }
                    s = (s + uint32_t(w.nk)) % uint32_t(stages);
                }
            }
        } else {
            // The whole warp runs the loop, and one lane of it issues: control flow and descriptors that are the warp's
            // own keep the work between MMA groups short, so that the tensor pipe's queue does not run dry.
            const uint64_t ad0 = kAMn ? sw128_desc(base, 8192, 1024) : sw128_desc(base, 16, 1024);
            const uint64_t bd0 =
                kBMn ? sw128_desc(base + L.a_bytes, 8192, 1024) : sw128_desc(base + L.a_bytes, 16, 1024);
            constexpr int kAStep = kAMn ? 128 : 2, kBStep = kBMn ? 128 : 2;  // of 16 in the contraction
            const uint32_t stage_step = L.stage_bytes >> 4;
            const bool elected = ptx::elect_one();  // the same lane as in mma_block: commits cover their thread's MMAs
            uint32_t s = 0, ph = 0;
            // the low-rank product of a tile's first nx columns, and the commit that hands the accumulator over
            auto finish = [&](const Tile &t, uint32_t buf) {
                const int extra = uniform(t.extra);
                const uint32_t d = tmem_base + buf * uint32_t(a.bn);
                const uint32_t idesc = idesc_f16(kPair ? 2 * kFB : kFB, uniform(t.nx), a.fp16 != 0, kAMn, kBMn);
                for (int x = 0; KIND == GR_LORA && x < extra; ++x) {
                    if (!wait_warp(B.full0 + 8 * s, ph, tmo, abort, a.err, kInfoMma | 0x400u | s)) return false;
                    ptx::tc_fence_after();
                    const int ranks = a.rank - (x >> 1) * kBK;
                    const int steps = ranks >= kBK ? kBK / 16 : (ranks + 15) / 16;
                    const uint64_t so = uint64_t(s * stage_step);
                    if (elected) {
                        for (int k = 0; k < steps; ++k)
                            issue_mma<kPair>(d, ad0 + so + uint64_t(k * kAStep), bd0 + so + uint64_t(k * kBStep), idesc,
                                             1u);
                        issue_commit<kPair>(B.empty0 + 8 * s);
                    }
                    __syncwarp();
                    if (++s == uint32_t(stages)) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
                if (elected) issue_commit<kPair>(B.tmem_full0 + 8 * buf);
                __syncwarp();
                return true;
            };
            for (int tile = 0; walk.next(w); ++tile) {
                const uint32_t buf = uint32_t(tile & 1), tph = (uint32_t(tile) >> 1) & 1u;
                const uint32_t d = tmem_base + buf * uint32_t(a.bn);
                const uint32_t idesc = idesc_f16(kPair ? 2 * kFB : kFB, uniform(w.nm), a.fp16 != 0, kAMn, kBMn);
                const int length = KIND == GR_WGRAD ? uniform(w.rows) : a.C;
                const int kb0 = uniform(w.kb0), kb1 = uniform(w.kb1);
                // blocks of 64, and where the piece ends with the contraction the shorter one behind them
                const int whole = min(kb1, length / kBK);
                const int left = kb1 > whole ? length - whole * kBK : 0;
                if (!wait_warp(B.tmem_empty0 + 8 * buf, tph ^ 1u, tmo, abort, a.err, kInfoMma | buf)) break;
                ptx::tc_fence_after();
                bool ok = true;
                for (int kb = kb0; kb < whole; ++kb) {
                    ok = wait_warp(B.full0 + 8 * s, ph, tmo, abort, a.err, kInfoMma | 0x100u | s);
                    if (!ok) break;
                    ptx::tc_fence_after();
                    const uint64_t so = uint64_t(s * stage_step);
                    mma_block<kPair, kAStep, kBStep>(d, ad0 + so, bd0 + so, idesc, kb > kb0 ? 1u : 0u,
                                                     B.empty0 + 8 * s);
                    if (++s == uint32_t(stages)) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
                if (ok && left > 0) {
                    const int steps = (left + 15) / 16;
                    // (a WGRAD pair: the peer's zeroes are behind its arrival)
                    ok = wait_warp<kPair && KIND == GR_WGRAD>(B.full0 + 8 * s, ph, tmo, abort, a.err,
                                                              kInfoMma | 0x100u | s);
                    if (ok) {
                        if constexpr (KIND == GR_WGRAD) {
                            if ((left & 15) != 0)
                                zero_tail(smem_raw + s * L.stage_bytes, left, steps,
                                          a.a_blocks + ((kPair ? w.nm / 2 : w.nm) + 63) / 64, lane);
                        }
                        ptx::tc_fence_after();
                        const uint64_t so = uint64_t(s * stage_step);
                        if (elected) {
                            for (int k = 0; k < steps; ++k)
                                issue_mma<kPair>(d, ad0 + so + uint64_t(k * kAStep), bd0 + so + uint64_t(k * kBStep),
                                                 idesc, whole > kb0 || k > 0 ? 1u : 0u);
                            issue_commit<kPair>(B.empty0 + 8 * s);
                        }
                        __syncwarp();
                    }
                    if (++s == uint32_t(stages)) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
                if (!ok || !finish(w, buf)) break;
            }
            if (elected) {
                if constexpr (kPair) ptx::mma_commit_pair_mc(B.mma_done, 1);
                else ptx::mma_commit(B.mma_done);
                volatile uint32_t local_abort = 0;
                ptx::mbar_wait_bounded(B.mma_done, 0, tmo, &local_abort, nullptr, 0);
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ epilogue
        // thread = one feature (TMEM lane); the two halves of 4 warps take alternate 32-column fragments
        const int e = warp - 2;
        const int half = e >> 2;
        const int q = warp & 3;
        const bool fp16 = a.fp16 != 0;
        if constexpr (KIND == GR_SHRINK) shrink_short(a, tab, reinterpret_cast<float *>(smem_raw + L.stg), misc + 4);
        for (int tile = 0; e < kEpiWarps && walk.next(w); ++tile) {
            const uint32_t buf = uint32_t(tile & 1), tph = (uint32_t(tile) >> 1) & 1u;
            uint4 zv[4];  // DGRAD: the next fragment's pre-activations, on their way before the accumulator is ready
            if constexpr (KIND == GR_DGRAD)
                if (a.preact && half * 32 < w.n && w.whole()) load_fragment(zv, a, w, half * 32, q, lane, true);
            // LORA, a tile of several requests: this worker adds the low-rank product of every parts-th eight rows
            int parts = 0, part = 0;
            if constexpr (KIND == GR_LORA) {
                if (w.mixed) {
                    parts = w.last - w.first + 1;
                    part = worker - w.first;
                    // the other rows' slices of B on their way to L2 while the projection is multiplied
                    for (int c = half * 32; c < w.n; c += 64) {
                        for (int i = 0; i < 4; ++i) {
                            const int j = c + (lane >> 2) + 8 * i;
                            if (c + 8 * i < w.nx || (c / 8 + i) % parts != part || j >= w.n) continue;
                            const int ad = tab.ad[request_of(tab, a.groups, w.col0 + j)];
                            const int f8 = w.f0 + q * 32 + (lane & 3) * 8;
                            if (ad < 0 || f8 >= a.F) continue;
                            const uint16_t *b =
                                static_cast<const uint16_t *>(a.lora_b) + size_t(ad) * a.rank * a.F + f8;
                            for (int r = lane & 3; r < a.rank; r += 4)
                                ptx::prefetch_l2(b + size_t(r) * a.F - (lane & 3) * 8);
                        }
                    }
                }
            }
            // The first eight of those rows that fall to this warp are worked out now, while the projection is
            // multiplied.
            int early = -1;  // which eight of the tile's
            float low[8];
            if constexpr (KIND == GR_LORA) {
                if (parts > 0) {
                    ptx::griddep_wait();  // H is the previous grid's
                    int c = half * 32;
                    while (c + 32 <= w.nx) c += 64;
                    for (int i = 3; i >= 0; --i)
                        if (c + 8 * i >= w.nx && c + 8 * i < w.n && (c / 8 + i) % parts == part) early = c / 8 + i;
                    if (early >= 0) {
#pragma unroll
                        for (int k = 0; k < 8; ++k) low[k] = 0.f;
                        const int j = early * 8 + (lane >> 2), f8 = w.f0 + q * 32 + (lane & 3) * 8;
                        if (j < w.n && f8 < a.F)
                            add_low_rank(low, a, tab.ad[request_of(tab, a.groups, w.col0 + j)], w.col0 + j, f8);
                    }
                }
            }
            const bool ok = ptx::mbar_wait_bounded(B.tmem_full0 + 8 * buf, tph, tmo + uint64_t(w.kb1 - w.kb0) * kBlockNs,
                                                   abort, a.err, kInfoEpi | buf);
            ptx::tc_fence_after();
            if constexpr (KIND == GR_LORA) ptx::griddep_wait();  // the bias is read through L1
            const uint32_t tacc = tmem_base + (uint32_t(q * 32) << 16) + buf * uint32_t(a.bn);
            const int f = w.f0 + q * 32 + lane;
            const bool live = f < a.F && ok;
            bool held = true;  // the accumulator is still this tile's
            if (!kPair && !w.whole()) {
                // a piece of the tile: to the workspace, [column][lane]; the last to arrive goes on with the sum
                float *const mine = a.partials + size_t(2 * worker + w.slot) * size_t(kFB * a.bn) + q * 32 + lane;
                for (int c = half * kSpan; c < w.n; c = next_fragment<kSpan, kHalves>(c)) {
                    uint32_t v[32];
                    ptx::tmem_ld32(tacc + uint32_t(c), v);
                    ptx::tmem_ld_wait(v);
                    const int cols = min(32, w.n - c);
                    if constexpr (KIND == GR_LORA) {
                        if (parts > 0) {
                            float *const stg = reinterpret_cast<float *>(smem_raw + L.stg) + e * 1024;
                            turn(v, stg, lane);
                            const int f8 = w.f0 + q * 32 + (lane & 3) * 8;
                            float *p = a.partials + size_t(2 * worker + w.slot) * size_t(kFB * a.bn) +
                                       size_t(c + (lane >> 2)) * kFB + q * 32 + (lane & 3) * 8;
#pragma unroll 1
                            for (int i = 0; i < 4; ++i, p += 8 * kFB) {
                                if ((lane >> 2) + 8 * i >= cols || f8 >= a.F) continue;
                                float x[8];
                                turned(x, stg, lane, i);
                                const int row = w.col0 + c + (lane >> 2) + 8 * i;
                                if (c / 8 + i == early) {
#pragma unroll
                                    for (int k = 0; k < 8; ++k) x[k] += low[k];
                                } else if (c + 8 * i >= w.nx && (c / 8 + i) % parts == part) {
                                    add_low_rank(x, a, tab.ad[request_of(tab, a.groups, row)], row, f8);
                                }
                                float4 *d = reinterpret_cast<float4 *>(p);
                                __stcg(d, make_float4(x[0], x[1], x[2], x[3]));
                                __stcg(d + 1, make_float4(x[4], x[5], x[6], x[7]));
                            }
                            continue;
                        }
                    }
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (j < cols && live) __stcg(mine + (c + j) * kFB, __uint_as_float(v[j]));
                }
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(B.tmem_empty0 + 8 * buf);
                held = false;
                // thread 64's release covers what the others wrote before the barrier, its acquire what they read after
                ptx::named_bar_sync(3, kEpiWarps * 32);
                volatile uint32_t *const verdict = misc + 2 + (tile & 1);  // read before the one after next is written
                if (threadIdx.x == 64) {
                    const uint32_t before = ptx::atom_add_acq_rel_gpu(a.counters + w.id, 1u);
                    const bool last = before == uint32_t(w.last - w.first);
                    if (last) ptx::st_relaxed_gpu(a.counters + w.id, 0u);  // for the next launch
                    *verdict = last;
                }
                ptx::named_bar_sync(3, kEpiWarps * 32);
                if (*verdict == 0u) continue;
                if constexpr (KIND != GR_WGRAD) {
                    finish_pieces<KIND>(a, w, pieces_of(a, walk, w), e, lane);
                    continue;
                }
            }
            if constexpr (KIND == GR_SHRINK) {
                const float sc = a.scale ? __ldg(a.scale + w.w) : 1.f;
                bool over = false;
#pragma unroll 1
                for (int c = 0; c < w.n; c += 32) {
                    uint32_t v[32], up[16], rest[16];
                    ptx::tmem_ld_blocks(tacc + uint32_t(c), v);
                    ptx::tmem_ld_wait(v);
                    if (fp16) {  // (of this request's rows and the ranks that there are)
                        const int fb = w.f0 + q * 32 + (lane >> 2), left = w.n - c - 2 * (lane & 3);
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            const int k = i / 8, b = i / 2 % 4;
                            over |= beyond_parts(sc * __uint_as_float(v[Fragment::pair(k, b) + i % 2])) &&
                                    8 * k + i % 2 < left && fb + 8 * b < a.F;
                        }
                    }
                    if (fp16) Fragment::split<true>(up, rest, v, sc);
                    else Fragment::split<false>(up, rest, v, sc);
                    const int f8 = w.f0 + q * 32 + (lane & 3) * 8;
                    const Fragment fr{smem_raw + L.stg + e * 2048, lane, w.n - c, f8 < a.F && ok,
                                      size_t(w.col0 + c + (lane >> 2)) * (2 * a.F) + f8, size_t(16) * a.F};
                    fr.store(a.out, up);
                    fr.store(static_cast<uint16_t *>(a.out) + a.F, rest);
                }
                if (over && ok) report_range(a);
            }
            float bias[4] = {0.f, 0.f, 0.f, 0.f};  // LORA: of a fragment's features in blocks
            if constexpr (KIND == GR_LORA) {
                const int fb = w.f0 + q * 32 + (lane >> 2);
#pragma unroll
                for (int b = 0; b < 4; ++b)
                    if (a.bias && fb + 8 * b < a.F) bias[b] = __ldg(a.bias + fb + 8 * b);
            }
            if constexpr (KIND == GR_WGRAD) {  // the halves take alternate 64-column blocks
                uint4 *const stg = reinterpret_cast<uint4 *>(smem_raw + L.stg + e * 4096);
                for (int c = half * 64; c < w.n; c += 128) {
                    uint32_t v[2][32];
                    const int two = c + 32 < w.n ? 2 : 1;
                    if (kPair || w.whole()) {
                        ptx::tmem_ld32(tacc + uint32_t(c), v[0]);
                        if (two == 2) ptx::tmem_ld32(tacc + uint32_t(c + 32), v[1]);
                        ptx::tmem_ld_wait(v[0]);
                        ptx::tmem_ld_wait(v[1]);
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (h >= two) break;
                        if (!kPair && !w.whole()) sum_pieces(v[h], pieces_of(a, walk, w), c + 32 * h, w.n, q * 32 + lane);
                        if (w.nk == 0) {  // an empty group's sum is zero
#pragma unroll
                            for (int j = 0; j < 32; ++j) v[h][j] = 0u;
                        }
                        if (fp16) put_columns<true>(v[h], stg, 4 * h, lane);
                        else put_columns<false>(v[h], stg, 4 * h, lane);
                    }
                    store_columns(a, w, c, stg, q, lane, ok);
                }
            }
            constexpr bool kFragments = KIND == GR_FORWARD || KIND == GR_DGRAD || KIND == GR_LORA;
            for (int c = half * 32; kFragments && c < w.n; c += 64) {
                uint32_t v[32];
                const int cols = min(32, w.n - c);
                if (KIND == GR_LORA && parts > 0 && c + 32 > w.nx) {
                    // rows with adapters of their own
                    ptx::tmem_ld32(tacc + uint32_t(c), v);
                    ptx::tmem_ld_wait(v);
                    float *const stg = reinterpret_cast<float *>(smem_raw + L.stg) + e * 1024;
                    turn(v, stg, lane);
                    const int f8 = w.f0 + q * 32 + (lane & 3) * 8;
                    uint16_t *y = static_cast<uint16_t *>(a.out) + size_t(w.col0 + c + (lane >> 2)) * a.F + f8;
#pragma unroll 1
                    for (int i = 0; i < 4; ++i, y += size_t(8) * a.F) {
                        if ((lane >> 2) + 8 * i >= cols || f8 >= a.F || !ok) continue;
                        float x[8];
                        turned(x, stg, lane, i);
                        const int row = w.col0 + c + (lane >> 2) + 8 * i;
                        if (c / 8 + i == early) {
#pragma unroll
                            for (int k = 0; k < 8; ++k) x[k] += low[k];
                        } else if (c + 8 * i >= w.nx) {
                            add_low_rank(x, a, tab.ad[request_of(tab, a.groups, row)], row, f8);
                        }
                        if (a.bias) {
                            const float4 b0 = __ldg(reinterpret_cast<const float4 *>(a.bias + f8));
                            const float4 b1 = __ldg(reinterpret_cast<const float4 *>(a.bias + f8) + 1);
                            x[0] += b0.x, x[1] += b0.y, x[2] += b0.z, x[3] += b0.w;
                            x[4] += b1.x, x[5] += b1.y, x[6] += b1.z, x[7] += b1.w;
                        }
                        uint32_t p[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) p[k] = pack16(x[2 * k], x[2 * k + 1], fp16);
                        *reinterpret_cast<uint4 *>(y) = make_uint4(p[0], p[1], p[2], p[3]);
                    }
                    __syncwarp();
                } else {
                    ptx::tmem_ld_blocks(tacc + uint32_t(c), v);
                    ptx::tmem_ld_wait(v);
                    constexpr uint32_t kStg = KIND == GR_LORA ? 4096u : 2048u;
                    const Fragment fr{smem_raw + L.stg + e * kStg, lane, cols,
                                      (w.f0 + q * 32 + (lane & 3) * 8) < a.F && ok,
                                      size_t(w.col0 + c + (lane >> 2)) * a.F + w.f0 + q * 32 + (lane & 3) * 8,
                                      size_t(8) * a.F};
                    if constexpr (KIND == GR_DGRAD) {
                        if (a.preact) {
                            uint32_t z[16];
                            fr.load(zv, z);
                            if (c + 64 < w.n)  // the next fragment's, while this one is worked on
                                load_fragment(zv, a, w, c + 64, q, lane, ok);
#pragma unroll
                            for (int i = 0; i < 32; ++i) {
                                const int j = Fragment::pair(i / 8, i / 2 % 4) + i % 2;
                                v[j] = __float_as_uint(__uint_as_float(v[j]) *
                                                       gelu_slope(from16(uint16_t(z[i / 2] >> (i % 2 * 16)), fp16)));
                            }
                        }
                    }
                    if constexpr (KIND == GR_FORWARD) {
                        if (a.preact) fr.store_rounded(a.preact, v, fp16);
                        if (a.act) {
#pragma unroll
                            for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(gelu(__uint_as_float(v[j])));
                        }
                    }
                    if constexpr (KIND == GR_LORA) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            const int j = Fragment::pair(i / 8, i / 2 % 4) + i % 2;
                            v[j] = __float_as_uint(__uint_as_float(v[j]) + bias[i / 2 % 4]);
                        }
                    }
                    fr.store_rounded(a.out, v, fp16);
                }
            }
            ptx::tc_fence_before();
            __syncwarp();
            if (held && lane == 0) {
                if constexpr (kPair) ptx::mbar_arrive_cluster(ptx::mapa(B.tmem_empty0 + 8 * buf, 0u));
                else ptx::mbar_arrive(B.tmem_empty0 + 8 * buf);
            }
        }
    }
    // this grid's end is the end of the one before it, too
    if constexpr (KIND == GR_LORA) ptx::griddep_wait();
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if constexpr (kPair) ptx::cluster_sync();  // no CTA leaves while its peer may still reach its shared memory
    if (warp == 1) {
        if constexpr (kPair) ptx::tmem_dealloc_pair(tmem_base, tmem_cols);
        else ptx::tmem_dealloc(tmem_base, tmem_cols);
    }
}

template <bool kPair>
void *kernel_for(int kind) {
    switch (kind) {
        case GR_FORWARD: return reinterpret_cast<void *>(&grouped_kernel<GR_FORWARD, kPair>);
        case GR_DGRAD: return reinterpret_cast<void *>(&grouped_kernel<GR_DGRAD, kPair>);
        case GR_WGRAD: return reinterpret_cast<void *>(&grouped_kernel<GR_WGRAD, kPair>);
        case GR_SHRINK: return kPair ? nullptr : reinterpret_cast<void *>(&grouped_kernel<GR_SHRINK, false>);
        case GR_LORA: return reinterpret_cast<void *>(&grouped_kernel<GR_LORA, kPair>);
        default: return nullptr;
    }
}

}  // namespace

int grouped_smem_bytes(int kind, bool pair, int stages, int bn, int groups, int a_blocks) {
    return int(gr_layout(kind, pair, stages, bn, groups, a_blocks).total);
}

cudaError_t launch_grouped(int kind, const GroupedArgs &a, int ctas, int smem, bool pdl, cudaStream_t stream) {
    const bool pair = a.pair != 0;
    void *fn = pair ? kernel_for<true>(kind) : kernel_for<false>(kind);
    if (!fn) return cudaErrorInvalidValue;
    // Once per device and kernel, to the most a launch may ask for: launches from several threads set the same value,
    // and none is set under a capture later.
    static std::atomic<bool> set[64][16];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidValue;
    std::atomic<bool> &done = set[dev][2 * kind + (pair ? 1 : 0)];
    if (!done.load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kGroupedMaxSmem);
        if (e != cudaSuccess) return e;
        done.store(true, std::memory_order_release);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(threads_of(kind));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (pdl) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (pair) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = 2;
        attr[n].val.clusterDim.y = 1;
        attr[n++].val.clusterDim.z = 1;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    void *args[] = {(void *)&a};
    return cudaLaunchKernelExC(&cfg, fn, args);
}

}  // namespace cf
