// block_norms.cu -- what stands between two blocks of a model:
//     x' = alpha x + scale gate Post(h)      h the block's output, x the stream around it
//     y  = Pre(x')                           the next block's input
// Post and Pre are RMSNorm, LayerNorm or nothing, each with a weight and a bias or without; and the gradient of all of
// it.  With t^ the normalised values of a norm, r the reciprocal root, g the gradient behind weight and bias times the
// weight:  dt = r (g - mean(g) - t^ mean(g t^)), RMSNorm without mean(g).  The statistics are not kept by the forward
// pass: both rows are in registers anyway, so working them out again costs no memory traffic.
//
// HBM bounds both passes: the forward one reads h and x and writes x' and y, the gradient reads dy, dx', h and x' and
// writes dh and dx.  A row is held in registers by as many threads as it has pieces of 8 columns (the forward pass: or
// half or a quarter as many); short rows share a warp, wide ones in the gradient are split over a cluster's CTAs.  Sums
// over a row go by shuffles, then through shared memory, of every CTA of the cluster where there are several.  A norm's
// squares are taken about a mean, never about zero, so nothing cancels.
// 16384 x 4096 bf16, RMSNorms, eight gates: forward 94 us (5.7 TB/s), gradient 147 (5.5; 138 and 9 for the sums).  What is
// left are the waits of a row's exchanges, one after another, and the instructions between them.  8192 x 4096 bf16 with
// LayerNorms and biases: forward 83 us, gradient 135, 1.75 and 1.85 times what RMSNorms take of half as many rows as above.
// Rows that start anywhere are read from shared memory and stored number by number: 8192 x 4095 bf16 with RMSNorms 98 and
// 222 us, 2.1 and 3.0 times what aligned ones take; with LayerNorms and biases 133 and 251, 1.6 and 1.9 times.
//
// The gradients of the weights are sums over all rows: a thread keeps its columns' sums in registers over a stretch of
// neighbouring rows, and a second, small launch adds the stretches in order (so equal calls give equal bits).  A gate
// shared by rows has a sum of its own for each of its rows' stretches: what one thread has whole it writes, the rest
// goes to the workspace too.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>

#include "block_norms.h"
#include "pieces.cuh"
#include "ptx.cuh"

namespace cf {
namespace {

constexpr uint32_t kAll = 0xffffffffu;

// The threads of a row: `lanes` of them in a warp, or `warps` whole warps, of `cluster` CTAs.
struct Group {
    int lanes;      // threads of the row in this CTA
    int warps;      // 1: a warp or part of one
    int cluster;
    int t;          // this thread's number among them
    int warp;       // its warp among them
    uint32_t bar;   // named barrier
    uint32_t rank;  // of the CTA in the cluster
    float *slots;   // two halves of `half` numbers, one for every second exchange
    int half;
    int turn;
    float4 *means;             // LayerNorm in the forward pass: its warps' statistics, two halves
    float n_warp, inv_warp;  // and the columns that the warp has
};

// v summed over the threads of the row in this warp
__device__ __forceinline__ float warp_sum(const Group &g, float v) {
    if (g.lanes >= 32) {
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
    } else {
        for (int d = g.lanes >> 1; d >= 1; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
    }
    return v;
}

// v summed over the row (of one CTA); every thread of the row gets the same bits.  The slots behind the last warp's, up
// to a multiple of four, hold zeros.
__device__ __forceinline__ float row_sum(Group &g, float v) {
    v = warp_sum(g, v);
    if (g.warps == 1) return v;
    float *const slots = g.slots + (g.turn & 1) * g.half;
    ++g.turn;
    if ((threadIdx.x & 31) == 0) slots[g.warp] = v;
    ptx::named_bar_sync(g.bar, uint32_t(g.lanes));
    float s = 0.f;
    for (int i = 0; i < g.warps; i += 4) {
        const float4 q = *reinterpret_cast<const float4 *>(slots + i);
        s += (q.x + q.y) + (q.z + q.w);
    }
    return s;
}

// kV (a power of two) values at once, over a cluster's row too.  In a warp each step halves the values that a lane goes
// on with (it hands the others to its partner), so eight values take 9 shuffles where one by one they take 40; then lane
// l holds value place(l % kV) of the warp, and the warps' are added the same way round.
template <int kV>
__device__ __forceinline__ constexpr int place(int lane) {
    int p = 0;
    for (int k = kV / 2, d = 1; k >= 1; k /= 2, d *= 2) p += lane & d ? k : 0;
    return p;
}
template <int kV, bool kCluster>
__device__ __forceinline__ void row_sums(Group &g, float (&v)[kV]) {
    if (!kCluster && g.lanes < 32) {
        for (int d = g.lanes >> 1; d >= 1; d >>= 1) {
#pragma unroll
            for (int i = 0; i < kV; ++i) v[i] += __shfl_xor_sync(kAll, v[i], d);
        }
        return;
    }
    const int lane = threadIdx.x & 31;
    float w[kV];
#pragma unroll
    for (int i = 0; i < kV; ++i) w[i] = v[i];
#pragma unroll
    for (int k = kV / 2, d = 1; k >= 1; k /= 2, d *= 2) {
        const bool upper = lane & d;
#pragma unroll
        for (int i = 0; i < k; ++i)
            w[i] = (upper ? w[i + k] : w[i]) + __shfl_xor_sync(kAll, upper ? w[i] : w[i + k], d);
    }
#pragma unroll
    for (int d = kV; d <= 16; d *= 2) w[0] += __shfl_xor_sync(kAll, w[0], d);
    float s = w[0];
    if (kCluster || g.warps > 1) {
        float *const slots = g.slots + (g.turn & 1) * g.half;
        ++g.turn;
        const int mine = (kCluster ? int(g.rank) * g.warps : 0) + g.warp;
        if constexpr (kCluster) {
            for (int c = lane / kV; c < g.cluster; c += 32 / kV)
                ptx::st_cluster_f32(ptx::mapa(ptx::smem_u32(slots + mine * kV + lane % kV), uint32_t(c)), s);
            ptx::cluster_sync();
        } else {
            if (lane < kV) slots[mine * kV + lane] = s;
            ptx::named_bar_sync(g.bar, uint32_t(g.lanes));
        }
        s = 0.f;
        if constexpr (kCluster) {
            for (int i = lane / kV; i < g.warps * g.cluster; i += 32 / kV) s += slots[i * kV + lane % kV];
        } else {
#pragma unroll
            for (int i = 0; i < 16 * kV / 32; ++i) s += 32 * i < g.half ? slots[lane + 32 * i] : 0.f;
        }
#pragma unroll
        for (int d = kV; d <= 16; d *= 2) s += __shfl_xor_sync(kAll, s, d);
    }
#pragma unroll
    for (int i = 0; i < kV; ++i) v[place<kV>(i)] = __shfl_sync(kAll, s, i);
}

// Columns of a thread's piece p: eight in a row where rows and vectors are 16-byte aligned, else every lanes-th.
template <bool kVec>
struct Columns {
    int c0, lanes, first, n;  // first: of the CTA; n: of the row
    __device__ __forceinline__ int at(int p, int j) const {
        return kVec ? first + (c0 + p * lanes) * 8 + j : first + c0 + (p * 8 + j) * lanes;
    }
    __device__ __forceinline__ bool live(int p, int j) const { return at(p, kVec ? 0 : j) < n; }
};

// (columns behind the last one stay what they were in v)
template <int kDt, bool kVec>
__device__ __forceinline__ void load_piece(Piece<kDt> &v, const void *row, const Columns<kVec> &cols, int p, bool on) {
    using E = typename Element<kDt>::type;
    if constexpr (kVec) {
        if (on && cols.live(p, 0)) v.load(static_cast<const E *>(row) + cols.at(p, 0));
    } else {
        v.zero();
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (on && cols.live(p, j)) v.put(j, static_cast<const E *>(row)[cols.at(p, j)]);
    }
}
template <int kDt, bool kVec>
__device__ __forceinline__ void store_piece(void *row, const Two (&x)[4], const Columns<kVec> &cols, int p, bool on) {
    using E = typename Element<kDt>::type;
    if constexpr (kVec) {
        Piece<kDt> v;
        v.pack(x);
        if (on && cols.live(p, 0)) v.store(static_cast<E *>(row) + cols.at(p, 0));
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float2 q = x[j / 2].parts();
            if (on && cols.live(p, j)) static_cast<E *>(row)[cols.at(p, j)] = from_float<kDt>(j % 2 ? q.y : q.x);
        }
    }
}
// a vector's columns (behind the last one zeros), or `none` where there is no vector
template <bool kVec>
__device__ __forceinline__ void load_vector(Two (&x)[4], const float *v, float none, const Columns<kVec> &cols, int p) {
    if (!v) {
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = Two(none);
    } else if constexpr (kVec) {
        const bool in = cols.live(p, 0);
        const float4 *q = reinterpret_cast<const float4 *>(v + (in ? cols.at(p, 0) : 0));
        const float4 l = in ? __ldg(q) : make_float4(0.f, 0.f, 0.f, 0.f);
        const float4 h = in ? __ldg(q + 1) : make_float4(0.f, 0.f, 0.f, 0.f);
        x[0] = Two(l.x, l.y), x[1] = Two(l.z, l.w), x[2] = Two(h.x, h.y), x[3] = Two(h.z, h.w);
    } else {
#pragma unroll
        for (int j = 0; j < 8; j += 2)
            x[j / 2] = Two(cols.live(p, j) ? __ldg(v + cols.at(p, j)) : 0.f,
                           cols.live(p, j + 1) ? __ldg(v + cols.at(p, j + 1)) : 0.f);
    }
}
// How rows come in.
enum RowMode : int {
    LOOSE = 0,  // numbers that start anywhere, few columns or, forward, over 16384: a thread takes every lanes-th, fp32
                // ones ahead of time, in copies of 4 bytes
    SHORT = 1,  // 16-byte aligned, few columns (copies of 16 bytes ahead of time, by the thread that needs them) or, forward,
                // over 16384 (loads)
    WIDE = 2,   // 16-byte aligned, whole warps: bulk copies ahead of time, one a row
    SHIFTED = 3,  // numbers that start anywhere, whole warps: bulk copies of the 16-byte pieces that hold a row
};
__host__ __device__ constexpr bool is_vec(int mode) { return mode == SHORT || mode == WIDE; }
__host__ __device__ constexpr bool is_bulk(int mode) { return mode == WIDE || mode == SHIFTED; }

constexpr int kMostRingRows = 5;

// Rows on their way, in shared memory, several stages of up to kRows rows (one of each of that many matrices), a row kP
// pieces a thread.  LOOSE and SHORT: a thread fills and reads its own columns alone, so nobody waits for anybody.
__host__ __device__ constexpr int ring_depth(int dt) { return dt == CF_FP32 ? 2 : 4; }
__host__ __device__ constexpr bool has_ring(int dt, int mode, int pieces) {
    return is_bulk(mode) || ((mode == SHORT || dt == CF_FP32) && pieces <= 2);
}
template <int kDt, int kMode, int kRows, int kP>
struct RowRing {
    using E = typename Element<kDt>::type;
    static constexpr bool kVec = is_vec(kMode);
    static constexpr bool kOn = has_ring(kDt, kMode, kP);
    static constexpr int kDepth = ring_depth(kDt);
    static constexpr int kCopies = kVec ? Piece<kDt>::kWords / 4 : 8;  // of a piece
    static constexpr uint32_t kBytes = kVec ? 16 : 4;                                   // of a copy
    const E *src[kRows];  // this thread's first column of the next row; null: zeros
    const Columns<kVec> &cols;
    uint32_t base, step;  // of this thread's copies; from one to the next
    int rows, stage, left;  // rows: of a stage; left: rows to come
    size_t apart;

    __device__ __forceinline__ RowRing(const Columns<kVec> &c, const RingArgs &r, uint8_t *ring, const Group &, int rows_,
                                       int left_, volatile uint32_t *)
        : cols(c), base(ptx::smem_u32(ring) + threadIdx.x * kBytes), step(blockDim.x * kBytes), rows(rows_), stage(0), left(left_),
          apart(size_t(c.n)) {}
    __device__ __forceinline__ void matrix(int k, const void *m, int64_t row, int64_t) {
        src[k] = m ? static_cast<const E *>(m) + (left > 0 ? size_t(row) * apart : 0) +
                         (cols.at(0, 0) < cols.n ? cols.at(0, 0) : 0)
                   : nullptr;
    }
    // a row of each matrix into stage `to`, if there is one
    __device__ __forceinline__ void fetch(int to) {
        if constexpr (kOn) {
            const bool on = left > 0;
#pragma unroll
            for (int k = 0; k < kRows; ++k) {
                if (k >= rows) break;
                uint32_t dst = base + uint32_t((to * rows + k) * (kP * kCopies)) * step;
#pragma unroll
                for (int p = 0; p < kP; ++p)
#pragma unroll
                    for (int j = 0; j < kCopies; ++j, dst += step) {
                        const bool in = on && src[k] != nullptr && cols.live(p, kVec ? 0 : j);
                        const int d = in ? (kVec ? p * cols.lanes * 8 + j * (16 / int(sizeof(E))) : (p * 8 + j) * cols.lanes)
                                         : 0;
                        // (nothing is read where nothing is in)
                        const E *const from = in ? src[k] + d : src[0];
                        if constexpr (kVec) ptx::cp_async_16(dst, from, in ? 16u : 0u);
                        else ptx::cp_async_4(dst, from, in ? 4u : 0u);
                    }
                if (on && src[k] != nullptr) src[k] += apart;
            }
            --left;
            ptx::cp_async_commit();
        }
    }
    __device__ __forceinline__ void start() {
#pragma unroll
        for (int s = 0; s < kDepth - 1; ++s) fetch(s);
    }
    // the row in hand is there, and one more is on its way
    __device__ __forceinline__ void turn() {
        fetch(stage == 0 ? kDepth - 1 : stage - 1);
        if constexpr (kOn) ptx::cp_async_wait<kDepth - 1>();
    }
    __device__ __forceinline__ void take(Piece<kDt> &v, int k, int p) {
        if constexpr (kOn) {
            uint32_t at = base + uint32_t(((stage * rows + k) * kP + p) * kCopies) * step;
#pragma unroll
            for (int j = 0; j < kCopies; ++j, at += step) {
                if constexpr (kVec) {
                    const uint4 q = ptx::ld_shared_v4(at);
                    v.w[4 * j] = q.x, v.w[4 * j + 1] = q.y, v.w[4 * j + 2] = q.z, v.w[4 * j + 3] = q.w;
                } else {
                    v.w[j] = ptx::ld_shared_u32(at);
                }
            }
        } else {
            v.zero();
            if (left > 0 && src[k] != nullptr) {
                const E *const row = src[k] - (cols.at(0, 0) < cols.n ? cols.at(0, 0) : 0);
                load_piece<kDt, kVec>(v, row, cols, p, true);
            }
        }
    }
    // on to the next row
    __device__ __forceinline__ void next() {
        if constexpr (kOn) {
            stage = stage == kDepth - 1 ? 0 : stage + 1;
        } else {
#pragma unroll
            for (int k = 0; k < kRows; ++k)
                if (left > 0 && src[k] != nullptr) src[k] += apart;
            --left;
        }
    }
    __device__ __forceinline__ void release(int) {}
    // Behind the last row the copies write zeros: they have all arrived before the ring's place takes the CTA's sums (a
    // __syncthreads alone does not wait for them), and before the CTA leaves.
    __device__ __forceinline__ void finish() {
        if constexpr (kOn) ptx::cp_async_wait<0>();
    }
};

// WIDE: the row's first thread asks for whole rows (of the CTA's share) in bulk copies, which complete on an mbarrier a
// stage, and refills a stage when the exchange of the row's sums has shown that every thread is through with it.  What it
// alone needs lies in shared memory: the other threads' registers hold the sums.  (With copies by each thread, their
// addresses and predicates were a fifth of the gradient's instructions.)
// SHIFTED: a row's 16-byte pieces, the first and last of which hold a neighbour's numbers, too; where they would reach
// out of the matrix (its first and last row) the leader brings those few numbers itself.  A thread reads its numbers one
// by one, behind the row's start in its first piece.
struct RingState {
    const uint8_t *src[kMostRingRows];                      // the next row's share of this CTA; null: zeros
    const uint8_t *lo[kMostRingRows], *hi[kMostRingRows];  // SHIFTED: the matrix's ends
    int left, fill, issued;  // rows to ask for; the stage to fill next; rows asked for
    uint32_t bytes;          // WIDE: of a stage
};
constexpr uint32_t kRingHead = 2048;  // of up to 8 groups: 8 mbarriers and the leader's state, 256 bytes
static_assert(sizeof(RingState) <= 192, "behind the mbarriers");
// bytes of a row of a ring's stage
__host__ __device__ constexpr int ring_pitch(int dt, int mode, int pieces, int lanes) {
    return lanes * pieces * 8 * type_bytes(dt) + (mode == SHIFTED ? 32 : 0);
}
template <int kDt, int kMode, int kRows, int kP>
struct BulkRing {
    using E = typename Element<kDt>::type;
    static constexpr bool kOn = true, kVec = kMode == WIDE;
    const Columns<kVec> &cols;
    const RingArgs &ring;
    volatile uint32_t *abort;
    RingState *state;
    uint32_t bar, at, pitch;  // of the row in hand: its mbarrier, the thread's numbers; from a row to the next
    uint32_t lead[kVec ? 1 : kRows];  // SHIFTED: of each matrix's row in hand, bytes in front of it in its first piece
    int rows, stage;
    uint32_t phase;
    bool leader;

    __device__ __forceinline__ BulkRing(const Columns<kVec> &c, const RingArgs &r, uint8_t *smem, const Group &g, int rows_,
                                        int left, volatile uint32_t *abort_)
        : cols(c), ring(r), abort(abort_), rows(rows_), stage(0), phase(0), leader(g.t == 0) {
        const int group = int(threadIdx.x) / c.lanes;
        pitch = uint32_t(ring_pitch(kDt, kMode, kP, c.lanes));
        bar = ptx::smem_u32(smem) + uint32_t(group) * 256u;
        state = reinterpret_cast<RingState *>(smem + group * 256 + 64);
        at = ptx::smem_u32(smem) + kRingHead + uint32_t(group * r.depth * rows) * pitch +
             uint32_t(c.c0) * (kVec ? 8 : 1) * sizeof(E);
        if (leader) {
            for (int s = 0; s < r.depth; ++s) ptx::mbar_init(bar + 8 * s, 1 + r.extra_arrivals);
            ptx::fence_mbarrier_init_cluster();
            state->left = left;
            state->fill = state->issued = 0;
            state->bytes = 0;
        }
    }
    __device__ __forceinline__ uint32_t share() const {
        return uint32_t(min(cols.lanes * kP * 8, cols.n - cols.first)) * uint32_t(sizeof(E));
    }
    // (what no copy fills is zero)
    __device__ __forceinline__ void matrix(int k, const void *m, int64_t row, int64_t all) {
        m = k < rows ? m : nullptr;
        const size_t row_bytes = size_t(cols.n) * sizeof(E);
        const uint8_t *const first = static_cast<const uint8_t *>(m) + size_t(row) * row_bytes + cols.first * sizeof(E);
        if (leader) {
            state->src[k] = m && state->left > 0 ? first : nullptr;
            if (m) state->bytes += share();
            state->lo[k] = static_cast<const uint8_t *>(m);
            state->hi[k] = static_cast<const uint8_t *>(m) + size_t(all) * row_bytes;
        }
        if constexpr (!kVec) lead[k] = uint32_t(reinterpret_cast<uintptr_t>(first)) & 15u;
        if (k >= rows) return;
        if constexpr (kVec) {
            for (int p = 0; p < kP; ++p)
                if (!m || !cols.live(p, 0))
                    for (int s = 0; s < ring.depth; ++s)
                        for (uint32_t b = 0; b < 8 * sizeof(E); b += 4)
                            ptx::st_shared_u32(
                                at + uint32_t(s * rows + k) * pitch + uint32_t(p * cols.lanes) * 8 * sizeof(E) + b, 0u);
        } else if (!m) {
            for (int s = 0; s < ring.depth; ++s)
                for (uint32_t b = uint32_t(cols.c0) * 4; b < pitch; b += uint32_t(cols.lanes) * 4)
                    ptx::st_shared_u32(at - uint32_t(cols.c0) * sizeof(E) + uint32_t(s * rows + k) * pitch + b, 0u);
        }
    }
    __device__ __forceinline__ static void issue(RingState *st, const RingArgs &ring, uint32_t bars, uint32_t first,
                                                 uint32_t pitch, int rows, uint32_t share, size_t apart,
                                                 volatile uint32_t *abort, int n) {
        const uint64_t policy = ptx::policy_evict_first();
        for (; n > 0; --n) {
            const int to = st->fill;
            st->fill = to + 1 == ring.depth ? 0 : to + 1;
            if (st->left <= 0 || *abort) return;
            const uint32_t full = bars + 8 * to;
            if constexpr (!kVec) {
                for (int k = 0; k < rows; ++k)
                    if (st->src[k] != nullptr) inner(st, k, share, first + uint32_t(to * rows + k) * pitch);
            }
            if constexpr (kVec) {
                ptx::mbar_arrive_expect_tx(full, st->bytes);
            } else {
                uint32_t bytes = 0;
                for (int k = 0; k < rows; ++k) bytes += st->src[k] == nullptr ? 0u : inner(st, k, share, 0u);
                ptx::mbar_arrive_expect_tx(full, bytes);  // (after the leader's own numbers)
            }
            for (int k = 0; k < rows; ++k) {
                const uint8_t *const src = st->src[k];
                if (src == nullptr) continue;
                uint32_t dst = first + uint32_t(to * rows + k) * pitch, size = share;
                const uint8_t *from = src;
                if constexpr (!kVec) {
                    size = inner(st, k, share, 0u);
                    from = reinterpret_cast<const uint8_t *>(reinterpret_cast<uintptr_t>(src) & ~uintptr_t(15));
                    if (at_end(st, k, share)) {
                        const uint8_t *const piece = from;
                        from = reinterpret_cast<const uint8_t *>((reinterpret_cast<uintptr_t>(src) + 15) & ~uintptr_t(15));
                        dst += uint32_t(from - piece);
                    }
                }
                if (size > 0) ptx::bulk_load_g2s_hint(dst, from, size, full, policy);
                st->src[k] = src + apart;
            }
            --st->left;
            ++st->issued;
        }
    }
    // SHIFTED: whether the row's first or last piece reaches out of the matrix
    __device__ __forceinline__ static bool at_end(const RingState *st, int k, uint32_t share) {
        const uintptr_t a = reinterpret_cast<uintptr_t>(st->src[k]), e = a + share;
        return (a & ~uintptr_t(15)) < reinterpret_cast<uintptr_t>(st->lo[k]) ||
               ((e + 15) & ~uintptr_t(15)) > reinterpret_cast<uintptr_t>(st->hi[k]);
    }
    // Bytes of the row's pieces; where they would reach out of the matrix, of those inside it, and the numbers outside
    // them are brought to `to`, where the row's first piece begins (0: they are not).
    __device__ __forceinline__ static uint32_t inner(const RingState *st, int k, uint32_t share, uint32_t to) {
        const uintptr_t a = reinterpret_cast<uintptr_t>(st->src[k]), e = a + share;
        if (!at_end(st, k, share)) return uint32_t(((e + 15) & ~uintptr_t(15)) - (a & ~uintptr_t(15)));
        const uintptr_t a0 = (a + 15) & ~uintptr_t(15), a1 = max(a0, e & ~uintptr_t(15));
        if (to != 0u) {
            for (uintptr_t b = a; b < min(a0, e); b += sizeof(E))
                put(to + uint32_t(b - (a & ~uintptr_t(15))), *reinterpret_cast<const E *>(b));
            for (uintptr_t b = a1; b < e; b += sizeof(E))
                put(to + uint32_t(b - (a & ~uintptr_t(15))), *reinterpret_cast<const E *>(b));
        }
        return uint32_t(a1 - a0);
    }
    __device__ __forceinline__ static void put(uint32_t addr, E v) {
        if constexpr (sizeof(E) == 4) ptx::st_shared_u32(addr, __float_as_uint(v));
        else ptx::st_shared_u16(addr, v);
    }
    // every thread of the row has taken what it needs of the last n rows.  (Before the first ones: the barriers'
    // initialisation and the zeros are known to all threads.)
    __device__ __forceinline__ void release(int n) {
        if (leader)  // (c0 is 0)
            issue(state, ring, bar - 8 * stage, at - uint32_t(stage * rows) * pitch, pitch, rows, share(),
                  size_t(cols.n) * sizeof(E), abort, n);
        __syncwarp();
    }
    __device__ __forceinline__ void start() { release(ring.depth); }
    __device__ __forceinline__ void turn() {
        ptx::mbar_wait_bounded(bar, phase, ring.timeout_ns, abort, ring.err, 0x76000000u | uint32_t(stage));
    }
    __device__ __forceinline__ void take(Piece<kDt> &v, int k, int p) {
        if constexpr (kVec) {
            const uint32_t from = at + uint32_t(k) * pitch + uint32_t(p * cols.lanes) * 8 * sizeof(E);
#pragma unroll
            for (int j = 0; j < Piece<kDt>::kWords / 4; ++j) {
                const uint4 q = ptx::ld_shared_v4(from + 16 * j);
                v.w[4 * j] = q.x, v.w[4 * j + 1] = q.y, v.w[4 * j + 2] = q.z, v.w[4 * j + 3] = q.w;
            }
        } else {
            uint32_t from = at + uint32_t(k) * pitch + lead[k] + uint32_t(p * 8 * cols.lanes) * sizeof(E);
            v.zero();
#pragma unroll
            for (int j = 0; j < 8; ++j, from += uint32_t(cols.lanes) * sizeof(E)) {
                if constexpr (sizeof(E) == 4) v.w[j] = cols.live(p, j) ? ptx::ld_shared_u32(from) : 0u;
                else v.put(j, cols.live(p, j) ? ptx::ld_shared_u16(from) : uint16_t(0));
            }
        }
    }
    __device__ __forceinline__ void next() {
        at += uint32_t(rows) * pitch;
        bar += 8;
        if constexpr (!kVec) {
            const uint32_t row = uint32_t(cols.n) * uint32_t(sizeof(E));
#pragma unroll
            for (int k = 0; k < kRows; ++k) lead[k] = (lead[k] + row) & 15u;
        }
        if (++stage == ring.depth) {
            stage = 0;
            phase ^= 1u;
            at -= uint32_t(ring.depth * rows) * pitch;
            bar -= 8 * ring.depth;
        }
    }
    // Nothing is on its way when the CTA leaves (after a wait that ran out there might be), and the place is free for the
    // CTA's sums.  (The row's other threads are through with the barriers: each row's exchange is behind its wait.)
    __device__ __forceinline__ void finish() {
        if (!leader) return;
        volatile uint32_t local = 0;
        const int issued = state->issued;
        for (int s = 0; s < ring.depth && s < issued; ++s)
            ptx::mbar_wait_bounded(bar + 8 * (s - stage), uint32_t((issued - 1 - s) / ring.depth) & 1u, ring.timeout_ns,
                                   &local, nullptr, 0);
        for (int s = 0; s < ring.depth; ++s) ptx::mbar_inval(bar + 8 * (s - stage));
    }
};
template <int kDt, int kRows, int kP>
struct RowRing<kDt, WIDE, kRows, kP> : BulkRing<kDt, WIDE, kRows, kP> {
    using BulkRing<kDt, WIDE, kRows, kP>::BulkRing;
};
template <int kDt, int kRows, int kP>
struct RowRing<kDt, SHIFTED, kRows, kP> : BulkRing<kDt, SHIFTED, kRows, kP> {
    using BulkRing<kDt, SHIFTED, kRows, kP>::BulkRing;
};

// x with 0 in the place of columns behind the last one
template <bool kVec>
__device__ __forceinline__ Two live_two(Two x, const Columns<kVec> &cols, int p, int j) {
    const float2 q = x.parts();
    return Two(cols.live(p, 2 * j) ? q.x : 0.f, cols.live(p, 2 * j + 1) ? q.y : 0.f);
}

// 1 / sqrt(v): the hardware's value and one step of Newton's method, good to 2^-23 or so in a few instructions (the
// correctly rounded one takes some 25)
__device__ __forceinline__ float reciprocal_root(float v) {
    const float r = rsqrtf(v);
    const float e = fmaf(v * r, -r, 1.f);
    return fabsf(v) > 1e-30f && v < 1e30f ? fmaf(0.5f * r, e, r) : r;
}

// c added to the columns that there are, the others are zero
template <bool kVec, int kP>
__device__ __forceinline__ void add_live(Two (&x)[kP][4], float c, const Columns<kVec> &cols) {
    const Two k(c);
#pragma unroll
    for (int p = 0; p < kP; ++p)
#pragma unroll
        for (int j = 0; j < 4; ++j) x[p][j] = x[p][j] + k;
    if (cols.live(kP - 1, 7)) return;
#pragma unroll
    for (int p = 0; p < kP; ++p)
#pragma unroll
        for (int j = 0; j < 4; ++j) x[p][j] = live_two(x[p][j], cols, p, j);
}

// The reciprocal root of one norm's row held in x (1: no norm), which loses its mean where the norm takes it.
// kFull: it may be a LayerNorm.  Its squares are taken about the mean of the warp's columns, and one exchange brings every
// warp's mean and squares: with n of them, sums s and q, about the mean c of the first warp
//     sum (x - m)^2 = sum q + n (s / n - c)^2  -  N (m - c)^2,
// where the first sum is at most N / n times the difference (the first warp's n), so no more is lost than that of 2^-24.
// (A mean first, then the squares, two exchanges: 8192 x 4096 bf16 with two LayerNorms 75 us.)
template <bool kVec, int kP, bool kFull>
__device__ __forceinline__ float spread(Group &g, int norm, Two (&x)[kP][4], const Columns<kVec> &cols, float inv_n,
                                        float eps) {
    if (norm == CF_NORM_NONE) return 1.f;
    float mean = 0.f;
    if (kFull && norm == CF_NORM_LAYER) {
        Two s(0.f);
#pragma unroll
        for (int p = 0; p < kP; ++p)
#pragma unroll
            for (int j = 0; j < 4; ++j) s = s + x[p][j];
        mean = warp_sum(g, s.sum()) * g.inv_warp;
        add_live<kVec, kP>(x, -mean, cols);
    }
    Two s(0.f);
#pragma unroll
    for (int p = 0; p < kP; ++p)
#pragma unroll
        for (int j = 0; j < 4; ++j) s = fma(x[p][j], x[p][j], s);
    float q = s.sum();
    if (kFull && norm == CF_NORM_LAYER) {
        q = warp_sum(g, q);
        if (g.warps > 1) {
            float4 *const slots = g.means + (g.turn & 1) * g.warps;
            ++g.turn;
            if ((threadIdx.x & 31) == 0) slots[g.warp] = make_float4(mean, q, g.n_warp, 0.f);
            ptx::named_bar_sync(g.bar, uint32_t(g.lanes));
            const float c = slots[0].x;
            float off = 0.f;  // N (m - c)
            q = 0.f;
#pragma unroll 4
            for (int i = 0; i < g.warps; ++i) {
                const float4 w = slots[i];
                const float d = w.x - c;
                off = fmaf(w.z, d, off);
                q += fmaf(w.z * d, d, w.y);
            }
            off *= inv_n;
            q = fmaf(-off * off, 1.f / inv_n, q);
            q = q < 0.f ? 0.f : q;  // (a NaN stays)
            add_live<kVec, kP>(x, mean - (c + off), cols);
        }
    } else {
        q = row_sum(g, q);
    }
    return reciprocal_root(fmaf(q, inv_n, eps));
}

// Bytes of what the forward pass's threads keep in shared memory
__host__ __device__ constexpr int forward_kept_bytes(bool bias, int pieces, int threads) {
    return threads * pieces * 32 * (pieces == 4 ? 1 : bias ? 2 : 0);
}

// kP pieces a thread.  kFull: LayerNorms or biases, too.  A worker takes a stretch of neighbouring rows, as in the gradient.
template <int kDt, int kMode, int kP, bool kFull>
__global__ void __maxnreg__(kP == 4 && !is_bulk(kMode) ? 64 : 128) block_norms_kernel(const BlockNormsArgs a) {
    constexpr bool kVec = is_vec(kMode);
    constexpr bool kAside = kP == 4;
    extern __shared__ __align__(128) uint8_t smem[];  // what is kept there, the ring
    uint8_t *const ring_smem = smem + forward_kept_bytes(a.post_bias || a.pre_bias, kP, int(blockDim.x));
    __shared__ uint32_t abort;
    if (threadIdx.x == 0) abort = 0u;
    __shared__ float4 means[kFull ? 2 * 32 : 1];           // of up to 32 warps in all
    __shared__ __align__(16) float slots[2 * 32 + 8 * 8];  // of each of up to 8 groups of warps, rounded up to four
    for (int i = threadIdx.x; i < int(sizeof(slots) / 4); i += blockDim.x) slots[i] = 0.f;
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    using E = typename Element<kDt>::type;
    Group g;
    g.lanes = a.lanes;
    g.warps = (a.lanes + 31) / 32;
    g.cluster = 1;
    const int group = int(threadIdx.x) / a.lanes;
    g.t = int(threadIdx.x) - group * a.lanes;
    g.warp = g.t >> 5;
    g.bar = 1 + uint32_t(group);
    g.rank = 0;
    g.half = (g.warps + 3) & ~3;
    g.slots = slots + group * 2 * g.half;
    g.turn = 0;
    g.means = means + (kFull ? group * 2 * g.warps : 0);
    const Columns<kVec> cols{g.t, a.lanes, 0, a.cols};
    const int groups = int(blockDim.x) / a.lanes;
    const float inv_n = 1.f / float(a.cols);
    if constexpr (kFull) {
        float n_warp = 0.f;
#pragma unroll
        for (int p = 0; p < kP; ++p)
#pragma unroll
            for (int j = 0; j < 8; ++j) n_warp += cols.live(p, j) ? 1.f : 0.f;
        g.n_warp = warp_sum(g, n_warp);
        g.inv_warp = 1.f / fmaxf(g.n_warp, 1.f);
    }
    const Two alpha(a.x ? a.alpha : 0.f);
    const int64_t mine = int64_t(blockIdx.x) * groups + group;
    const int first = int(min(a.rows, mine * a.chunk)), last = int(min(a.rows, int64_t(first) + a.chunk));
    // rows that threads of one warp may share a warp's turn with: as many turns as any; else their own
    const int turns = a.lanes < 32 ? a.chunk : last - first;
    RowRing<kDt, kMode, 3, kP> ring(cols, a.ring, ring_smem, g, a.gates_along ? 3 : 2, last - first, &abort);
    ring.matrix(0, a.h, first, a.rows);
    ring.matrix(1, a.x, first, a.rows);
    ring.matrix(2, a.gates_along ? a.gate : nullptr, first, a.rows);
    __syncthreads();
    ring.start();

    Two w1[kAside ? 1 : kP][4], w2[kP][4];  // Post's weight times the gate; Pre's
    int gate_end = 0;                       // the first row behind the rows of the gate in w1
    // Kept in shared memory, which no other thread looks at: with four pieces a thread w1, else the biases, Post's times
    // scale and gate (read from memory at each row, 8192 x 4096 bf16 took 89 us).
    float4 *const kept = reinterpret_cast<float4 *>(smem) + threadIdx.x;
    auto keep = [&](int k, int p, const Two (&v)[4]) {
#pragma unroll
        for (int j = 0; j < 4; j += 2) {
            const float2 l = v[j].parts(), h = v[j + 1].parts();
            kept[((k * kP + p) * 2 + j / 2) * int(blockDim.x)] = make_float4(l.x, l.y, h.x, h.y);
        }
    };
    auto get_kept = [&](int k, int p, Two (&v)[4]) {
#pragma unroll
        for (int j = 0; j < 4; j += 2) {
            const float4 q = kept[((k * kP + p) * 2 + j / 2) * int(blockDim.x)];
            v[j] = Two(q.x, q.y), v[j + 1] = Two(q.z, q.w);
        }
    };
    auto take_gate = [&](int of, bool here) {
        gate_end = int((uint32_t(of) + 1u) * a.rows_per_gate);
#pragma unroll
        for (int p = 0; p < kP; ++p) {
            Two w[4], k[4];
            load_vector<kVec>(w, a.post_weight, 1.f, cols, p);
            if (a.gate) {
                Piece<kDt> q;
                if (here) {
                    ring.take(q, 2, p);
                } else {
                    q.zero();
                    load_piece<kDt, kVec>(q, static_cast<const E *>(a.gate) + size_t(of) * a.cols, cols, p, true);
                }
                q.unpack(k);
#pragma unroll
                for (int j = 0; j < 4; ++j) w[j] = w[j] * k[j];
            }
            if constexpr (kAside) {
                keep(0, p, w);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) w1[p][j] = w[j];
                if (kFull && a.post_bias && !here) {
                    load_vector<kVec>(w, a.post_bias, 0.f, cols, p);
#pragma unroll
                    for (int j = 0; j < 4; ++j) w[j] = w[j] * Two(a.scale) * (a.gate ? k[j] : Two(1.f));
                    keep(0, p, w);
                }
            }
        }
    };
#pragma unroll
    for (int p = 0; p < kP; ++p) {
        load_vector<kVec>(w2[p], a.pre_weight, 1.f, cols, p);
        if (kFull && !kAside) {
            Two b[4];
            if (a.pre_bias) {
                load_vector<kVec>(b, a.pre_bias, 0.f, cols, p);
                keep(1, p, b);
            }
            if (a.post_bias && a.gates_along) {  // (the gate is in the ring, row by row)
                load_vector<kVec>(b, a.post_bias, 0.f, cols, p);
#pragma unroll
                for (int j = 0; j < 4; ++j) b[j] = b[j] * Two(a.scale);
                keep(0, p, b);
            }
        }
    }
    if (!a.gates_along) take_gate(int(uint32_t(first) / a.rows_per_gate < uint32_t(a.gates) ? uint32_t(first) / a.rows_per_gate : 0u), false);
    E *xo = static_cast<E *>(a.x_out), *yo = static_cast<E *>(a.y);
    if (xo) xo += size_t(first) * a.cols;
    if (yo) yo += size_t(first) * a.cols;
    for (int i = 0; i < turns; ++i) {
        const bool on = i < last - first;  // (behind the last row first + i may pass 2^31)
        ring.turn();
        if (a.gates_along) {
            if (on) take_gate(first + i, true);
        } else if (on && first + i == gate_end) {
            take_gate(int(uint32_t(first + i) / a.rows_per_gate), false);
        }
        Two x[kP][4];
#pragma unroll
        for (int p = 0; p < kP; ++p) {
            Piece<kDt> q;
            ring.take(q, 0, p);
            q.unpack(x[p]);
        }
        Two root(a.scale * spread<kVec, kP, kFull>(g, a.post, x, cols, inv_n, a.eps));
#pragma unroll
        for (int p = 0; p < kP; ++p) {
            Two u[4];
            Piece<kDt> q;
            ring.take(q, 1, p);
            q.unpack(u);
#pragma unroll
            for (int j = 0; j < 4; ++j) u[j] = u[j] * alpha;
            if (kFull && a.post_bias) {  // scale gate bias
                Two b[4], k[4];
                if constexpr (kAside) {  // (the bias, and a gate that is not in the ring, from memory again)
                    load_vector<kVec>(b, a.post_bias, 0.f, cols, p);
#pragma unroll
                    for (int j = 0; j < 4; ++j) b[j] = b[j] * Two(a.scale);
                } else {
                    get_kept(0, p, b);
                }
                if (a.gate && (kAside || a.gates_along)) {
                    if (a.gates_along) {
                        ring.take(q, 2, p);
                    } else {
                        q.zero();
                        load_piece<kDt, kVec>(
                            q, static_cast<const E *>(a.gate) + size_t(gate_end / a.rows_per_gate - 1) * a.cols, cols, p,
                            on);
                    }
                    q.unpack(k);
#pragma unroll
                    for (int j = 0; j < 4; ++j) b[j] = b[j] * k[j];
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) u[j] = u[j] + b[j];
            }
            if constexpr (kAside) {
                Two w[4];
                get_kept(0, p, w);
#pragma unroll
                for (int j = 0; j < 4; ++j) x[p][j] = fma(x[p][j] * root, w[j], u[j]);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) x[p][j] = fma(x[p][j] * root, w1[p][j], u[j]);
            }
            if (xo) store_piece<kDt, kVec>(xo, x[p], cols, p, on);
        }
        if (xo) xo += a.cols;
        if (yo == nullptr) {
            if (g.warps > 1) ptx::named_bar_sync(g.bar, uint32_t(g.lanes));
            __syncwarp();
            ring.next();
            ring.release(1);
            continue;
        }
        root = Two(spread<kVec, kP, kFull>(g, a.pre, x, cols, inv_n, a.eps));
        ring.next();
        ring.release(1);
#pragma unroll
        for (int p = 0; p < kP; ++p) {
#pragma unroll
            for (int j = 0; j < 4; ++j) x[p][j] = x[p][j] * root * w2[p][j];
            if (kFull && a.pre_bias) {
                Two b[4];
                if constexpr (kAside) load_vector<kVec>(b, a.pre_bias, 0.f, cols, p);
                else get_kept(1, p, b);
#pragma unroll
                for (int j = 0; j < 4; ++j) x[p][j] = x[p][j] + b[j];
            }
            store_piece<kDt, kVec>(yo, x[p], cols, p, on);
        }
        yo += a.cols;
    }
    ring.finish();
}

// ---------------------------------------------------------------------------
// gradient
// ---------------------------------------------------------------------------
// a thread's columns of a vector of the workspace
template <bool kVec>
__device__ __forceinline__ void store_floats(float *out, const Two (&x)[4], const Columns<kVec> &cols, int p) {
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        const float2 q = x[j / 2].parts();
        if (kVec && cols.live(p, j)) __stcg(reinterpret_cast<float2 *>(out + cols.at(p, j)), q);
        if (!kVec && cols.live(p, j)) __stcg(out + cols.at(p, j), q.x);
        if (!kVec && cols.live(p, j + 1)) __stcg(out + cols.at(p, j + 1), q.y);
    }
}

// Bytes of what the CTA's threads keep in shared memory, each for itself: the sums over all gates and, with two pieces a
// thread, Post's weight (in registers, what did not fit took the gradient of 16384 x 4096 from 154 to 175 us).
__host__ __device__ constexpr int kept_bytes(bool gate, bool full, int pieces, int threads) {
    return threads * pieces * 32 * ((gate ? (full ? 2 : 1) : 0) + (pieces == 2 ? 1 : 0));
}

// With hc and xc the rows without their means (RMSNorm: the rows), g2 = dy w2 and w1 = scale gate weight, every sum that
// the row needs is one over products of what is loaded:
//     sum g2 x^ = r2 sum g2 xc,
//     d  = dx' + r2 (g2 - mean(g2) - x^ mean(g2 x^)),
//     sum w1 d h^ = r1 (sum w1 hc dx' + r2 (sum w1 hc g2 - mean(g2) sum w1 hc - r2 mean(g2 x^) sum w1 hc xc)),
// so one exchange between the threads serves where three would follow one another (16384 x 4096 bf16: 287 us with
// three; fp32 gradients are 1.4e-7 off, where sums one after another in fp32 leave 1.2e-7).  A LayerNorm's means come one
// exchange before: that of the row before, where the ring holds two rows.
// (Rows ahead kept in registers left no room for the sums: 16384 x 4096 bf16 172 us, 158 with the ring in shared memory.)
// kFull: LayerNorms or biases, too.  kGate: a gate, whose rows' sums are closed where the next gate begins.
// kP pieces a thread, up to 512 threads an SM with 128 registers: two where those hold them (not with biases' sums), so
// that a row of 4096 takes half of the SM's threads and the other half, with a row of its own, works while this one
// exchanges its sums.
template <int kDt, int kMode, bool kCluster, bool kGate, bool kFull, int kP>
__global__ void __launch_bounds__(512) block_norms_grad_kernel(const BlockNormsGradArgs a) {
    constexpr bool kVec = is_vec(kMode), kWide = is_bulk(kMode);
    constexpr int kV = kFull ? 16 : 8;
    extern __shared__ __align__(128) uint8_t smem[];  // what is kept there, the ring
    __shared__ uint32_t abort;
    __shared__ float slots[kCluster ? 2 * 16 * kV * 8 : 2 * (16 * kV + 8 * 32)];  // (up to 8 groups, each rounded up to 32)
    using E = typename Element<kDt>::type;
    if (threadIdx.x == 0) abort = 0u;
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    Group g;
    g.lanes = a.lanes;
    g.warps = (a.lanes + 31) / 32;
    g.cluster = a.cluster;
    const int group = int(threadIdx.x) / a.lanes;
    g.t = int(threadIdx.x) - group * a.lanes;
    g.warp = g.t >> 5;
    g.bar = 1 + uint32_t(group);
    g.rank = kCluster ? ptx::cluster_ctarank() : 0u;
    // (whole rounds of 32 numbers; what no warp writes stays zero)
    g.half = (g.warps * kV * (kCluster ? a.cluster : 1) + 31) & ~31;
    g.slots = slots + group * 2 * g.half;
    g.turn = 0;
    if constexpr (!kCluster) {
        for (int i = threadIdx.x; i < int(sizeof(slots) / 4); i += blockDim.x) slots[i] = 0.f;
        __syncthreads();
    }
    const Columns<kVec> cols{g.t, a.lanes, int(g.rank) * a.lanes * kP * 8, a.cols};
    const int groups = int(blockDim.x) / a.lanes;
    const int set = int(blockIdx.x) / a.cluster, worker = set * groups + group;
    const int chunk = int(a.chunk);
    const int first = int(min(a.rows, int64_t(worker) * chunk)), last = int(min(a.rows, int64_t(first) + chunk));
    // rows that threads of one warp may share a warp's turn with: as many turns as any; else their own
    const int turns = a.lanes < 32 ? chunk : last - first;
    const float inv_n = 1.f / float(a.cols);
    const bool lh = kFull && a.post == CF_NORM_LAYER, lx = kFull && a.pre == CF_NORM_LAYER;
    if constexpr (kCluster) ptx::cluster_sync();  // nobody writes into a CTA that has not started

    constexpr bool kAside = kP == 2;
    Two w2[kP][4], w1[kAside ? 1 : kP][4];  // Pre's weight; scale * gate * Post's weight
#pragma unroll
    for (int p = 0; p < kP; ++p) load_vector<kVec>(w2[p], a.pre_weight, 1.f, cols, p);
    // sums over the rows, those of the gate in hand in sa and sb; in shared memory, which no other thread looks at, those
    // of all gates
    Two sa[kP][4], sc[kP][4], sb[kP][4], sd[kP][4];
    float *const done = reinterpret_cast<float *>(smem) + threadIdx.x * 2;
    uint8_t *const ring_smem = smem + kept_bytes(kGate, kFull, kP, int(blockDim.x));
    auto total = [&](int k, int p, int j) -> float2 & {
        return *reinterpret_cast<float2 *>(done + ((k * kP + p) * 4 + j) * 2 * int(blockDim.x));
    };
#pragma unroll
    for (int p = 0; p < kP; ++p)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            sa[p][j] = sb[p][j] = sc[p][j] = sd[p][j] = Two(0.f);
            if constexpr (kGate) {
                total(0, p, j) = make_float2(0.f, 0.f);
                if constexpr (kFull) total(1, p, j) = make_float2(0.f, 0.f);
            }
        }

    auto w1_at = [&](int p, int j) -> float2 & { return total(kGate ? (kFull ? 2 : 1) : 0, p, j); };
    auto w1_of = [&](int p, int j) { return kAside ? Two(w1_at(p, j)) : w1[kAside ? 0 : p][j]; };
    auto set_w1 = [&](int p, int j, Two v) {
        if constexpr (kAside) w1_at(p, j) = v.parts();
        else w1[p][j] = v;
    };

    int gate_at = 0, gate_end = 0;  // the gate in hand, the first row behind its rows
    const bool gates_along = kGate && RowRing<kDt, kMode, 5, kP>::kOn && a.gate && a.rows_per_gate == 1;
    RowRing<kDt, kMode, 5, kP> ring(cols, a.ring, ring_smem, g, gates_along ? 5 : 4, last - first, &abort);
    ring.matrix(0, a.h, first, a.rows);
    ring.matrix(1, a.dy ? a.x_out : nullptr, first, a.rows);
    ring.matrix(2, a.dy, first, a.rows);
    ring.matrix(3, a.dx_out, first, a.rows);
    ring.matrix(4, gates_along ? a.gate : nullptr, first, a.rows);
    __syncthreads();
    ring.start();
    // scale * gate, from memory or from the row of gates in hand
    auto scaled_gate = [&](Two (&k)[4], int of, int p, bool here) {
        Piece<kDt> q;
        q.zero();
        if (here) ring.take(q, 4, p);
        else if (a.gate) load_piece<kDt, kVec>(q, static_cast<const E *>(a.gate) + size_t(of) * a.cols, cols, p, true);
#pragma unroll
        for (int j = 0; j < 4; ++j) k[j] = Two(a.scale) * (a.gate ? Two(q.get(2 * j), q.get(2 * j + 1)) : Two(1.f));
    };
    auto take_gate = [&](int of, bool here) {
        gate_at = of;
        gate_end = int((uint32_t(of) + 1u) * a.rows_per_gate);
#pragma unroll
        for (int p = 0; p < kP; ++p) {
            Two k[4], w[4];
            scaled_gate(k, of, p, here);
            load_vector<kVec>(w, a.post_weight, 1.f, cols, p);
#pragma unroll
            for (int j = 0; j < 4; ++j) set_w1(p, j, live_two(w[j] * k[j], cols, p, j));
        }
    };
    if (kGate && first < last) {
        if (!gates_along) take_gate(int(uint32_t(first) / a.rows_per_gate), false);
    } else {
#pragma unroll
        for (int p = 0; p < kP; ++p) {
            Two w[4];
            load_vector<kVec>(w, a.post_weight, 1.f, cols, p);
#pragma unroll
            for (int j = 0; j < 4; ++j) set_w1(p, j, live_two(w[j] * Two(a.scale), cols, p, j));
        }
    }
    size_t at = first < last ? size_t(first) * a.cols : 0;  // where the row in hand lies
    constexpr bool kAhead = kFull && kMode == WIDE;
    const bool ahead = kAhead && a.ring.depth >= 2 && (lh || lx);
    Two mh(0.f), mx(0.f);  // less the LayerNorms' means
    for (int i = 0; i < turns; ++i) {
        const bool on = kWide || i < last - first;
        const int r = on ? first + i : last;  // (behind the last row first + i may pass 2^31)
        ring.turn();
        if (gates_along && on) take_gate(r, true);
        Piece<kDt> raw[4][kP];
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int p = 0; p < kP; ++p) ring.take(raw[k][p], k, p);
        ring.next();
        // columns 2j and the next of the k-th matrix's row
        auto pair = [&](int k, int p, int j) { return Two(raw[k][p].get(2 * j), raw[k][p].get(2 * j + 1)); };
        if constexpr (!kAhead) mh = mx = Two(0.f);  // (nothing is kept from a row to the next)
        if ((lh || lx) && (!ahead || i == 0)) {
            Two s(0.f), t(0.f);
#pragma unroll
            for (int p = 0; p < kP; ++p)
#pragma unroll
                for (int j = 0; j < 4; ++j) s = s + pair(0, p, j), t = t + pair(1, p, j);
            float v[2] = {s.sum(), t.sum()};
            row_sums<2, kCluster>(g, v);
            mh = Two(lh ? -v[0] * inv_n : 0.f);
            mx = Two(lx ? -v[1] * inv_n : 0.f);
        }
        auto h_of = [&](int p, int j) { return kFull ? live_two(pair(0, p, j) + mh, cols, p, j) : pair(0, p, j); };
        auto x_of = [&](int p, int j) { return kFull ? live_two(pair(1, p, j) + mx, cols, p, j) : pair(1, p, j); };
        constexpr int kSums = kFull ? 12 : 6;
        float v[kV];
        {
            Two s[kSums];
#pragma unroll
            for (int k = 0; k < kSums; ++k) s[k] = Two(0.f);
#pragma unroll
            for (int p = 0; p < kP; ++p)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const Two h = h_of(p, j), x = x_of(p, j), d = pair(3, p, j);
                    const Two w = w1_of(p, j), g2 = pair(2, p, j) * w2[p][j], wh = w * h;
                    s[0] = fma(h, h, s[0]);
                    s[1] = fma(x, x, s[1]);
                    s[2] = fma(g2, x, s[2]);
                    s[3] = fma(wh, d, s[3]);
                    s[4] = fma(wh, g2, s[4]);
                    s[5] = fma(wh, x, s[5]);
                    if constexpr (kFull) {
                        s[6] = s[6] + g2;
                        s[7] = s[7] + wh;
                        s[8] = fma(w, d, s[8]);
                        s[9] = fma(w, g2, s[9]);
                        s[10] = fma(w, x, s[10]);
                        s[11] = s[11] + w;
                    }
                }
#pragma unroll
            for (int k = 0; k < kV; ++k) v[k] = k < kSums ? s[k < kSums ? k : 0].sum() : 0.f;
        }
        if (kAhead && ahead && i + 1 < turns) {
            Two s(0.f), t(0.f);
            ring.turn();
#pragma unroll
            for (int p = 0; p < kP; ++p) {
                Piece<kDt> q;
                ring.take(q, 0, p);
#pragma unroll
                for (int j = 0; j < 4; ++j) s = s + Two(q.get(2 * j), q.get(2 * j + 1));
                ring.take(q, 1, p);
#pragma unroll
                for (int j = 0; j < 4; ++j) t = t + Two(q.get(2 * j), q.get(2 * j + 1));
            }
            v[kV - 2] = s.sum(), v[kV - 1] = t.sum();
        }
        row_sums<kV, kCluster>(g, v);
        ring.release(1);
        if constexpr (kP == 2) {  // (unpacked once more: held as fp32 over the exchange, they do not fit)
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int p = 0; p < kP; ++p) raw[k][p].pin();
        }
        // (an eps of 0 would make a NaN of a row that is not there)
        const float r1 = a.post == CF_NORM_NONE ? 1.f : on ? reciprocal_root(fmaf(v[0], inv_n, a.eps)) : 0.f;
        const float r2 = a.pre == CF_NORM_NONE ? 1.f : on ? reciprocal_root(fmaf(v[1], inv_n, a.eps)) : 0.f;
        const float ma = lx ? v[kFull ? 6 : 0] * inv_n : 0.f;                     // mean(g2)
        const float mb = a.pre == CF_NORM_NONE ? 0.f : r2 * r2 * (v[2] * inv_n);  // r2 mean(g2 x^)
        // r1 mean(w1 d h^), mean(w1 d)
        const float na = a.post == CF_NORM_NONE
                             ? 0.f
                             : r1 * r1 * (v[3] + r2 * (v[4] - (kFull ? ma * v[kFull ? 7 : 0] : 0.f) - mb * v[5])) * inv_n;
        const float nb =
            lh ? (v[kFull ? 8 : 0] + r2 * (v[kFull ? 9 : 0] - ma * v[kFull ? 11 : 0] - mb * v[kFull ? 10 : 0])) * inv_n
               : 0.f;
        const Two k1(r1), k2(r2), kb(-r2 * mb), ka(-r2 * ma), kn(-na), km(-r1 * nb);
#pragma unroll
        for (int p = 0; p < kP; ++p) {
            Two dx[4], dh[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const Two x = x_of(p, j), y = pair(2, p, j);
                Two d = fma(x, kb, fma(y * w2[p][j], k2, pair(3, p, j)));
                if constexpr (kFull) d = d + ka;
                sc[p][j] = fma(y, x * k2, sc[p][j]);
                if constexpr (kFull) sd[p][j] = sd[p][j] + y, sb[p][j] = sb[p][j] + d;
                const Two h = h_of(p, j) * k1;
                sa[p][j] = fma(d, h, sa[p][j]);
                dh[j] = fma(h, kn, (w1_of(p, j) * d) * k1);
                if constexpr (kFull) dh[j] = dh[j] + km;
                dx[j] = d * Two(a.alpha);
            }
            if (a.dx) store_piece<kDt, kVec>(static_cast<E *>(a.dx) + at, dx, cols, p, on);
            store_piece<kDt, kVec>(static_cast<E *>(a.dh) + at, dh, cols, p, on);
        }
        if (kAhead && ahead) {
            mh = Two(lh ? -v[kV - 2] * inv_n : 0.f);
            mx = Two(lx ? -v[kV - 1] * inv_n : 0.f);
        }
        if (on) at += size_t(a.cols);
        if constexpr (kGate) {
            if (on && (r + 1 == last || r + 1 == gate_end)) {  // its last row here
                const int from = gate_end - int(a.rows_per_gate);
#pragma unroll
                for (int p = 0; p < kP; ++p) {
                    Two w[4], b[4], d[4];
                    load_vector<kVec>(w, a.post_weight, 1.f, cols, p);
                    if constexpr (kFull) load_vector<kVec>(b, a.post_bias, 0.f, cols, p);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        d[j] = w[j] * sa[p][j];
                        if constexpr (kFull) d[j] = fma(b[j], sb[p][j], d[j]);
                        d[j] = d[j] * Two(a.scale);
                    }
                    if (a.sum_at[0] >= 0 || a.sum_at[1] >= 0) {
                        Two gate[4];
                        scaled_gate(gate, gate_at, p, false);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            total(0, p, j) = fma(gate[j], sa[p][j], Two(total(0, p, j))).parts();
                            if constexpr (kFull) total(1, p, j) = fma(gate[j], sb[p][j], Two(total(1, p, j))).parts();
                        }
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) sa[p][j] = sb[p][j] = Two(0.f);
                    if (a.dgate && from >= first && gate_end <= last) {
                        store_piece<kDt, kVec>(static_cast<E *>(a.dgate) + size_t(gate_at) * a.cols, d, cols, p, true);
                    } else if (a.dgate) {  // slot 0: begun by a worker before; slot 1: here, and goes on
                        float *const slot = a.slots + (size_t(2) * worker + (from >= first ? 1 : 0)) * a.cols;
                        store_floats<kVec>(slot, d, cols, p);
                    }
                }
                if (r + 1 < last && !gates_along) take_gate(gate_at + 1, false);
            }
        }
    }
    ring.finish();
    // the CTA's sums: those of its groups of threads are added through shared memory, which the ring needs no more
    float *const sums = reinterpret_cast<float *>(ring_smem);
    const int wide = a.lanes * kP * 8;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if (a.sum_at[k] < 0) continue;
        float *const out = a.partials + (size_t(a.sum_at[k]) * a.sets + set) * a.cols;
        if (groups > 1) __syncthreads();
#pragma unroll
        for (int p = 0; p < kP; ++p) {
            Two v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                v[j] = k >= 2                       ? (k == 2 ? sc[p][j] : sd[p][j])
                       : kGate && (kFull || k == 0) ? Two(total(k, p, j))
                                                    : Two(a.scale) * (k == 0 ? sa[p][j] : sb[p][j]);
            if (kCluster || groups == 1) {
                store_floats<kVec>(out, v, cols, p);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float2 q = v[j / 2].parts();
                    if (cols.live(p, j)) sums[group * wide + cols.at(p, j)] = j % 2 ? q.y : q.x;
                }
            }
        }
        if (!kCluster && groups > 1) {
            __syncthreads();
            for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
                float s = 0.f;
                for (int i = 0; i < groups; ++i) s += sums[i * wide + c];
                __stcg(out + c, s);
            }
        }
    }
    if constexpr (kCluster) ptx::cluster_sync();  // no CTA leaves while its peers may still write to it
}

// The workers' sums added in order: 32 columns a CTA, a warp every so many-th term, then the warps.  (335 terms of 1111
// columns by eight warps 10.5 us, which is the loads one after another.)
// Of many terms (a gate that thousands of workers share), kSumLong are in flight.
constexpr int kSumWarps = 32, kSumFly = 8, kSumLong = 32, kSumSms = 152;
__global__ void __launch_bounds__(kSumWarps * 32) block_norms_sums_kernel(const BlockNormsGradArgs a, int nsums, int gates_first) {
    __shared__ float part[kSumWarps][32];
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int blocks = (a.cols + 31) / 32, sum = int(blockIdx.x) / blocks;
    const int c = (int(blockIdx.x) - sum * blocks) * 32 + lane;
    const bool live = c < a.cols;
    int what = sum;
    const float *from, *head = nullptr;  // terms `step` apart; one before them
    size_t step;
    int terms;
    int64_t of = -1;
    if (what < nsums) {
        from = a.partials + size_t(what) * a.sets * a.cols;
        step = a.cols;
        terms = a.sets;
    } else {
        // the gate that begins with one worker and ends with another one
        what -= nsums;
        int64_t w;
        if (gates_first) {
            of = what;
            w = of * int64_t(a.rows_per_gate) / a.chunk;
        } else {
            w = what;
            const int64_t end = min(a.rows, (w + 1) * a.chunk);
            if (end <= w * a.chunk) return;
            of = (end - 1) / int64_t(a.rows_per_gate);
            if (of * int64_t(a.rows_per_gate) < w * a.chunk) return;
        }
        const int64_t last = ((of + 1) * int64_t(a.rows_per_gate) - 1) / a.chunk;
        if (last == w) return;
        head = a.slots + (size_t(2) * w + 1) * a.cols;
        from = a.slots + size_t(2) * (w + 1) * a.cols;
        step = size_t(2) * a.cols;
        terms = int(last - w);
    }
    float s = head && warp == 0 && live ? __ldcg(head + c) : 0.f;
    const int warps = int(blockDim.x) / 32;
    int i = warp;
    for (; i + warps * (kSumLong - 1) < terms; i += warps * kSumLong) {
        float x[kSumLong];
#pragma unroll
        for (int k = 0; k < kSumLong; ++k) x[k] = live ? __ldcg(from + (i + warps * k) * step + c) : 0.f;
#pragma unroll
        for (int k = 0; k < kSumLong; ++k) s += x[k];
    }
    for (; i < terms; i += warps * kSumFly) {
        float x[kSumFly];
#pragma unroll
        for (int k = 0; k < kSumFly; ++k)
            x[k] = live && i + warps * k < terms ? __ldcg(from + (i + warps * k) * step + c) : 0.f;
#pragma unroll
        for (int k = 0; k < kSumFly; ++k) s += x[k];
    }
    part[warp][lane] = s;
    __syncthreads();
    if (warp != 0 || !live) return;
    s = 0.f;
    for (int k = 0; k < warps; ++k) s += part[k][lane];
    if (of < 0) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (a.sum_at[k] == sum) a.sum_out[k][c] = s;
    } else if (a.dtype == CF_FP32) {
        static_cast<float *>(a.dgate)[size_t(of) * a.cols + c] = s;
    } else {
        static_cast<uint16_t *>(a.dgate)[size_t(of) * a.cols + c] =
            a.dtype == CF_FP16 ? from_float<CF_FP16>(s) : from_float<CF_BF16>(s);
    }
}

int round_lanes(int64_t threads) {  // of a row: a power of two in a warp, else whole warps
    if (threads > 32) return int((threads + 31) / 32 * 32);
    int p = 1;
    while (p < threads) p <<= 1;
    return p;
}

cudaError_t launch(const void *fn, dim3 grid, int threads, int cluster, bool pdl, cudaStream_t stream, void **args,
                   int smem = 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.dynamicSmemBytes = size_t(smem);
    cfg.gridDim = grid;
    cfg.blockDim = dim3(unsigned(threads));
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (pdl) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (cluster > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = unsigned(cluster);
        attr[n].val.clusterDim.y = 1;
        attr[n++].val.clusterDim.z = 1;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    return cudaLaunchKernelExC(&cfg, fn, args);
}

// Once per device and kernel, to the most a launch may ask for: launches from several threads set the same value, and
// none is set under a capture later.
constexpr int kMostSmem = 232448;  // of a CTA (227 KB)
cudaError_t allow_smem(const void *fn, int *own) {  // own: the kernel's static shared memory
    struct Entry {
        std::atomic<const void *> fn;
        std::atomic<uint64_t> devices;
        std::atomic<int> own;
    };
    static Entry table[96];  // (60 kernels)
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidValue;
    for (Entry &t : table) {
        const void *at = t.fn.load(std::memory_order_acquire);
        if (at == nullptr && t.fn.compare_exchange_strong(at, fn, std::memory_order_acq_rel)) at = fn;
        if (at != fn) continue;
        if (!(t.devices.load(std::memory_order_acquire) >> dev & 1)) {
            cudaFuncAttributes attr;
            e = cudaFuncGetAttributes(&attr, fn);
            if (e == cudaSuccess)
                e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         kMostSmem - int(attr.sharedSizeBytes));
            if (e != cudaSuccess) return e;
            t.own.store(int(attr.sharedSizeBytes), std::memory_order_release);
            t.devices.fetch_or(uint64_t(1) << dev, std::memory_order_acq_rel);
        }
        *own = t.own.load(std::memory_order_acquire);
        return cudaSuccess;
    }
    return cudaErrorInvalidValue;
}

// (what is rare is compiled in its widest form alone)
template <int kDt>
const void *forward_kernel(int mode, bool full, int pieces) {
    if (mode == LOOSE)
        return pieces == 1 ? reinterpret_cast<const void *>(&block_norms_kernel<kDt, LOOSE, 1, true>)
                           : reinterpret_cast<const void *>(&block_norms_kernel<kDt, LOOSE, 4, true>);
    if (mode == SHIFTED)
        return pieces == 2 ? reinterpret_cast<const void *>(&block_norms_kernel<kDt, SHIFTED, 2, true>)
                           : reinterpret_cast<const void *>(&block_norms_kernel<kDt, SHIFTED, 4, true>);
    if (mode == SHORT)
        return pieces == 1 ? reinterpret_cast<const void *>(&block_norms_kernel<kDt, SHORT, 1, true>)
                           : reinterpret_cast<const void *>(&block_norms_kernel<kDt, SHORT, 4, true>);
    if (pieces == 4) return reinterpret_cast<const void *>(&block_norms_kernel<kDt, WIDE, 4, true>);
    return full ? reinterpret_cast<const void *>(&block_norms_kernel<kDt, WIDE, 2, true>)
                : reinterpret_cast<const void *>(&block_norms_kernel<kDt, WIDE, 2, false>);
}
template <int kDt, int kMode, bool kCluster, bool kGate, bool kFull, int kP>
const void *grad_of() {
    return reinterpret_cast<const void *>(&block_norms_grad_kernel<kDt, kMode, kCluster, kGate, kFull, kP>);
}
template <int kDt>
const void *grad_kernel(int mode, bool cluster, bool gate, bool full, int pieces) {
    if (mode == LOOSE) return grad_of<kDt, LOOSE, false, true, true, 1>();
    if (mode == SHIFTED)
        return cluster ? grad_of<kDt, SHIFTED, true, true, true, 1>() : grad_of<kDt, SHIFTED, false, true, true, 1>();
    if (mode == SHORT) return grad_of<kDt, SHORT, false, true, true, 1>();
    if (cluster) {
        if constexpr (kDt != CF_FP32)
            if (pieces == 2) return grad_of<kDt, WIDE, true, true, false, 2>();
        return full ? grad_of<kDt, WIDE, true, true, true, 1>() : grad_of<kDt, WIDE, true, true, false, 1>();
    }
    if (full) return gate ? grad_of<kDt, WIDE, false, true, true, 1>() : grad_of<kDt, WIDE, false, false, true, 1>();
    if constexpr (kDt != CF_FP32)
        if (pieces == 2)
            return gate ? grad_of<kDt, WIDE, false, true, false, 2>() : grad_of<kDt, WIDE, false, false, false, 2>();
    return grad_of<kDt, WIDE, false, true, false, 1>();
}

// Shared memory of a launch's ring and, in bulk copies, its depth: what fits with `ctas` CTAs an SM, up to r->depth stages (0: three; 2, 3, 4
// and 6 of them, 16384 x 4096 bf16 forward: 97, 93, 95 and 135 us, what they take is missing in L1).
int plan_ring(RingArgs *r, int dt, int mode, int rows, int pieces, int lanes, int threads, int ctas, int own) {
    if (!has_ring(dt, mode, pieces)) return 0;
    const int stage = rows * (threads / lanes) * ring_pitch(dt, mode, pieces, lanes);
    if (!is_bulk(mode)) return ring_depth(dt) * stage;
    const int room = std::min(kMostSmem, (kMostSmem + 1024) / ctas - 1024) - own - int(kRingHead);
    r->depth = std::max(1, std::min(r->depth > 0 ? std::min(r->depth, 8) : 3, room / stage));
    return int(kRingHead) + r->depth * stage;
}

}  // namespace

constexpr int kForwardThreads = 512;  // an SM, with 96 registers each (16384 x 4096 bf16, copies by each thread: 768 with
                                      // 80 117 us, 1024 with 64 200 us, 512 with 128 102 us, with 96 95 us)

cudaError_t launch_block_norms(BlockNormsArgs a, bool vec, int sms, bool pdl, cudaStream_t stream) {
    const int pieces = (a.cols + 7) / 8;
    // a thread's pieces: two, so that what a row costs besides its numbers is shared by more of them
    const int per = pieces < 64 ? 1 : pieces <= 1024 ? 2 : 4;
    a.lanes = round_lanes((pieces + per - 1) / per);
    // (above 16384 columns it takes 1024 threads, which have 64 registers, and no ring fits)
    const bool bulk = per > 1 && a.lanes <= 512;
    const int mode = vec ? (bulk ? WIDE : SHORT) : bulk ? SHIFTED : LOOSE;
    const int groups = std::max(1, 256 / a.lanes), threads = groups * a.lanes;
    // a stretch of rows for each group of threads
    const int per_sm = std::max(1, kForwardThreads / threads);
    int64_t ctas = std::min<int64_t>((a.rows + groups - 1) / groups, int64_t(sms) * per_sm);
    a.chunk = int((a.rows + ctas * groups - 1) / (ctas * groups));
    ctas = (a.rows + int64_t(a.chunk) * groups - 1) / (int64_t(a.chunk) * groups);
    const int kept = forward_kept_bytes(a.post_bias || a.pre_bias, per, threads);
    // (of fp32, three rows of more than 8192 columns do not fit)
    a.gates_along = a.gate && a.rows_per_gate == 1 && has_ring(a.dtype, mode, per) && !(per == 4 && a.dtype == CF_FP32);
    const bool full = a.post == CF_NORM_LAYER || a.pre == CF_NORM_LAYER || a.post_bias || a.pre_bias;
    const void *fn = a.dtype == CF_BF16   ? forward_kernel<CF_BF16>(mode, full, per)
                     : a.dtype == CF_FP16 ? forward_kernel<CF_FP16>(mode, full, per)
                                          : forward_kernel<CF_FP32>(mode, full, per);
    int own;
    const cudaError_t e = allow_smem(fn, &own);
    if (e != cudaSuccess) return e;
    const int smem =
        kept + plan_ring(&a.ring, a.dtype, mode, a.gates_along ? 3 : 2, per, a.lanes, threads, per_sm, own + kept);
    void *args[] = {&a};
    return launch(fn, dim3(unsigned(ctas)), threads, 1, pdl, stream, args, smem);
}

BlockNormsGradPlan plan_block_norms_grad(int64_t rows, int64_t cols, int sms, bool lean, int dtype) {
    BlockNormsGradPlan p;
    const int64_t n = (cols + 7) / 8;
    // (of fp32, two are too many registers; where a cluster has one row at most, more CTAs finish sooner: 1 x 16384 bf16
    // 10 us with one, 14 with two, 2048 x 16384 239 and 109)
    p.pieces = lean && dtype != CF_FP32 && n >= 64 && (n <= 1024 || rows * ((n + 511) / 512) > sms) ? 2 : 1;
    p.cluster = int((n + 512 * p.pieces - 1) / (512 * p.pieces));
    p.lanes = round_lanes((n + p.cluster * p.pieces - 1) / (p.cluster * p.pieces));
    const int groups = p.cluster > 1 ? 1 : std::max(1, 256 / p.lanes);
    p.threads = groups * p.lanes;
    const int64_t most = int64_t(sms) * std::max(1, 512 / p.threads) / p.cluster;
    const int64_t sets = std::max<int64_t>(1, std::min<int64_t>(most, (rows + groups - 1) / groups));
    p.chunk = (rows + sets * groups - 1) / (sets * groups);
    p.sets = int((rows + p.chunk * groups - 1) / (p.chunk * groups));
    p.workers = p.sets * groups;
    return p;
}

bool block_norms_grad_lean(const BlockNormsGradArgs &a, bool vec) {
    return vec && a.post != CF_NORM_LAYER && a.pre != CF_NORM_LAYER && !a.post_bias && a.sum_at[1] < 0 && a.sum_at[3] < 0;
}

cudaError_t launch_block_norms_grad(BlockNormsGradArgs a, const BlockNormsGradPlan &p, bool vec, bool pdl,
                                    cudaStream_t stream) {
    a.lanes = p.lanes;
    a.cluster = p.cluster;
    a.chunk = p.chunk;
    a.sets = p.sets;
    const bool gate = a.gate != nullptr, cluster = p.cluster > 1, full = !block_norms_grad_lean(a, vec);
    const int mode = p.lanes < 32 ? (vec ? SHORT : LOOSE) : vec ? WIDE : SHIFTED;
    const void *fn = a.dtype == CF_BF16   ? grad_kernel<CF_BF16>(mode, cluster, gate, full, p.pieces)
                     : a.dtype == CF_FP16 ? grad_kernel<CF_FP16>(mode, cluster, gate, full, p.pieces)
                                          : grad_kernel<CF_FP32>(mode, cluster, gate, full, p.pieces);
    void *args[] = {&a};
    int own;
    cudaError_t e = allow_smem(fn, &own);
    if (e != cudaSuccess) return e;
    const int rows = a.gate && a.rows_per_gate == 1 ? 5 : 4;
    // (as grad_kernel chooses: what is rare has its gates' sums anyway)
    const int kept = kept_bytes(gate || mode != WIDE || cluster || (!full && p.pieces == 1), full || mode != WIDE,
                                    p.pieces, p.threads);
    // (the ring's place takes the sums of several groups in the end)
    const int smem = kept + std::max(plan_ring(&a.ring, a.dtype, mode, rows, p.pieces, p.lanes, p.threads,
                                                 std::max(1, 512 / p.threads), own + kept),
                                       p.threads == p.lanes ? 0 : p.threads * p.pieces * 8 * 4);
    e = launch(fn, dim3(unsigned(p.sets * p.cluster)), p.threads, p.cluster, pdl, stream, args, smem);
    if (e != cudaSuccess) return e;
    int nsums = 0;
    for (int k = 0; k < 4; ++k) nsums += a.sum_at[k] >= 0;
    const int64_t gates = gate ? a.rows / a.rows_per_gate : 0;
    int gates_first = gates <= p.workers;
    const int shared = gate && a.dgate && a.rows_per_gate > 1 ? int(std::min<int64_t>(gates, p.workers)) : 0;
    if (nsums + shared == 0) return cudaSuccess;
    // as many warps a CTA as there is room for all CTAs at once (eight: 335 terms of 1111 columns 10.5 us, 32: 6.6; 304 of
    // 4096 columns and eight gates the other way round)
    const int64_t blocks = int64_t((a.cols + 31) / 32) * (nsums + shared);
    int warps = 8;
    while (warps < kSumWarps && blocks * warps * 2 <= int64_t(kSumSms) * 64) warps *= 2;
    void *args2[] = {&a, &nsums, &gates_first};
    return launch(reinterpret_cast<const void *>(&block_norms_sums_kernel),
                  dim3(unsigned((a.cols + 31) / 32) * unsigned(nsums + shared)), warps * 32, 1, pdl, stream, args2);
}

}  // namespace cf
