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
// mean is taken before its squares, so nothing cancels.
//
// The gradients of the weights are sums over all rows: a thread keeps its columns' sums in registers over a stretch of
// neighbouring rows, and a second, small launch adds the stretches in order (so equal calls give equal bits).  A gate
// shared by rows has a sum of its own for each of its rows' stretches: what one thread has whole it writes, the rest
// goes to the workspace too.
#include <cuda_runtime.h>

#include <algorithm>
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
    float2 *slots;  // [2][warps * cluster], one half for every second exchange
    int turn;
};

// a and b, each summed over the row; every thread of the row gets the same bits
template <bool kCluster>
__device__ __forceinline__ float2 row_sum(Group &g, float a, float b) {
    if (g.lanes >= 32) {
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1) {
            a += __shfl_xor_sync(kAll, a, d);
            b += __shfl_xor_sync(kAll, b, d);
        }
    } else {
        for (int d = g.lanes >> 1; d >= 1; d >>= 1) {
            a += __shfl_xor_sync(kAll, a, d);
            b += __shfl_xor_sync(kAll, b, d);
        }
    }
    if (g.warps == 1 && !kCluster) return make_float2(a, b);
    const int all = g.warps * (kCluster ? g.cluster : 1);
    float2 *const slots = g.slots + (g.turn & 1) * all;
    ++g.turn;
    if constexpr (kCluster) {
        // lane l tells CTA l of the cluster
        const int lane = threadIdx.x & 31;
        if (lane < g.cluster)
            ptx::st_cluster_v2f32(ptx::mapa(ptx::smem_u32(slots + g.rank * g.warps + g.warp), uint32_t(lane)), a, b);
        ptx::cluster_sync();
    } else {
        if ((threadIdx.x & 31) == 0) slots[g.warp] = make_float2(a, b);
        ptx::named_bar_sync(g.bar, uint32_t(g.lanes));
    }
    float2 s = make_float2(0.f, 0.f);
    for (int i = 0; i < all; ++i) {
        const float2 v = slots[i];
        s.x += v.x, s.y += v.y;
    }
    return s;
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

template <int kDt, bool kVec>
__device__ __forceinline__ void load_piece(Piece<kDt> &v, const void *row, const Columns<kVec> &cols, int p, bool on) {
    using E = typename Element<kDt>::type;
    v.zero();
    if constexpr (kVec) {
        if (on && cols.live(p, 0)) v.load(static_cast<const E *>(row) + cols.at(p, 0));
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (on && cols.live(p, j)) v.put(j, static_cast<const E *>(row)[cols.at(p, j)]);
    }
}
template <int kDt, bool kVec>
__device__ __forceinline__ void store_piece(void *row, const float (&x)[8], const Columns<kVec> &cols, int p, bool on) {
    using E = typename Element<kDt>::type;
    if constexpr (kVec) {
        Piece<kDt> v;
        v.pack(x);
        if (on && cols.live(p, 0)) v.store(static_cast<E *>(row) + cols.at(p, 0));
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (on && cols.live(p, j)) static_cast<E *>(row)[cols.at(p, j)] = from_float<kDt>(x[j]);
    }
}
// a vector's columns, `none` where there is no vector
template <bool kVec>
__device__ __forceinline__ void load_vector(float (&x)[8], const float *v, float none, const Columns<kVec> &cols,
                                            int p) {
    if (!v) {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = none;
    } else if constexpr (kVec) {
        const bool in = cols.live(p, 0);
        const float4 *q = reinterpret_cast<const float4 *>(v + (in ? cols.at(p, 0) : 0));
        const float4 l = in ? __ldg(q) : make_float4(0.f, 0.f, 0.f, 0.f);
        const float4 h = in ? __ldg(q + 1) : make_float4(0.f, 0.f, 0.f, 0.f);
        x[0] = l.x, x[1] = l.y, x[2] = l.z, x[3] = l.w, x[4] = h.x, x[5] = h.y, x[6] = h.z, x[7] = h.w;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = cols.live(p, j) ? __ldg(v + cols.at(p, j)) : 0.f;
    }
}

// mean and reciprocal root of one norm's row held in x (0 and 1: no norm)
template <bool kVec, int kP>
__device__ __forceinline__ float2 spread(Group &g, int norm, const float (&x)[kP][8], const Columns<kVec> &cols,
                                         float inv_n, float eps) {
    if (norm == CF_NORM_NONE) return make_float2(0.f, 1.f);
    float mean = 0.f;
    if (norm == CF_NORM_LAYER) {
        float s = 0.f;
#pragma unroll
        for (int p = 0; p < kP; ++p)
#pragma unroll
            for (int j = 0; j < 8; ++j) s += x[p][j];
        mean = row_sum<false>(g, s, 0.f).x * inv_n;
    }
    float s = 0.f;
#pragma unroll
    for (int p = 0; p < kP; ++p)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float d = cols.live(p, j) ? x[p][j] - mean : 0.f;
            s = fmaf(d, d, s);
        }
    return make_float2(mean, __frsqrt_rn(fmaf(row_sum<false>(g, s, 0.f).x, inv_n, eps)));
}

template <int kDt, bool kVec, int kP>
__global__ void __launch_bounds__(kP == 4 ? 1024 : 512) block_norms_kernel(const BlockNormsArgs a) {
    __shared__ float2 slots[64];
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
    g.slots = slots + group * 2 * g.warps;
    g.turn = 0;
    const Columns<kVec> cols{g.t, a.lanes, 0, a.cols};
    const int groups = int(blockDim.x) / a.lanes;
    const float inv_n = 1.f / float(a.cols);
    // (every thread of a warp makes the same turns)
    for (int64_t r0 = int64_t(blockIdx.x) * groups; r0 < a.rows; r0 += int64_t(gridDim.x) * groups) {
        const int64_t r = r0 + group;
        const bool on = r < a.rows;
        const size_t at = on ? size_t(r) * a.cols : 0;
        Piece<kDt> hp[kP], xp[kP], gp[kP];
        const E *const gate =
            a.gate ? static_cast<const E *>(a.gate) + size_t(on ? uint32_t(r) / a.rows_per_gate : 0u) * a.cols : nullptr;
#pragma unroll
        for (int p = 0; p < kP; ++p) load_piece<kDt, kVec>(hp[p], static_cast<const E *>(a.h) + at, cols, p, on);
#pragma unroll
        for (int p = 0; p < kP; ++p) load_piece<kDt, kVec>(xp[p], static_cast<const E *>(a.x) + at, cols, p, on && a.x);
#pragma unroll
        for (int p = 0; p < kP; ++p) load_piece<kDt, kVec>(gp[p], gate, cols, p, on && gate);
        float x[kP][8];
#pragma unroll
        for (int p = 0; p < kP; ++p) hp[p].unpack(x[p]);
        float2 s = spread<kVec, kP>(g, a.post, x, cols, inv_n, a.eps);
#pragma unroll
        for (int p = 0; p < kP; ++p) {
            float w[8], b[8];
            load_vector<kVec>(w, a.post_weight, 1.f, cols, p);
            load_vector<kVec>(b, a.post_bias, 0.f, cols, p);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float v = a.scale * fmaf((x[p][j] - s.x) * s.y, w[j], b[j]);
                const float old = a.x ? a.alpha * xp[p].get(j) : 0.f;
                x[p][j] = cols.live(p, j) ? (gate ? fmaf(v, gp[p].get(j), old) : v + old) : 0.f;
            }
            if (a.x_out) store_piece<kDt, kVec>(static_cast<E *>(a.x_out) + at, x[p], cols, p, on);
        }
        if (a.y == nullptr) continue;
        s = spread<kVec, kP>(g, a.pre, x, cols, inv_n, a.eps);
#pragma unroll
        for (int p = 0; p < kP; ++p) {
            float w[8], b[8];
            load_vector<kVec>(w, a.pre_weight, 1.f, cols, p);
            load_vector<kVec>(b, a.pre_bias, 0.f, cols, p);
#pragma unroll
            for (int j = 0; j < 8; ++j) x[p][j] = fmaf((x[p][j] - s.x) * s.y, w[j], b[j]);
            store_piece<kDt, kVec>(static_cast<E *>(a.y) + at, x[p], cols, p, on);
        }
    }
}

// ---------------------------------------------------------------------------
// gradient
// ---------------------------------------------------------------------------
// Means and reciprocal roots of both norms' rows (h and x'), in two exchanges, one without a LayerNorm.
template <bool kVec, bool kCluster>
__device__ __forceinline__ void spreads(Group &g, int post, int pre, const float (&h)[8], const float (&x)[8],
                                        const Columns<kVec> &cols, float inv_n, float eps, float2 &sh, float2 &sx) {
    sh = sx = make_float2(0.f, 1.f);
    if (post == CF_NORM_NONE && pre == CF_NORM_NONE) return;
    if (post == CF_NORM_LAYER || pre == CF_NORM_LAYER) {
        float a = 0.f, b = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) a += h[j], b += x[j];
        const float2 s = row_sum<kCluster>(g, a, b);
        if (post == CF_NORM_LAYER) sh.x = s.x * inv_n;
        if (pre == CF_NORM_LAYER) sx.x = s.y * inv_n;
    }
    float a = 0.f, b = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const bool live = cols.live(0, j);
        const float dh = live ? h[j] - sh.x : 0.f, dx = live ? x[j] - sx.x : 0.f;
        a = fmaf(dh, dh, a);
        b = fmaf(dx, dx, b);
    }
    const float2 s = row_sum<kCluster>(g, a, b);
    if (post != CF_NORM_NONE) sh.y = __frsqrt_rn(fmaf(s.x, inv_n, eps));
    if (pre != CF_NORM_NONE) sx.y = __frsqrt_rn(fmaf(s.y, inv_n, eps));
}

// kShift: sums for the biases, too.  kGate: a gate, whose rows' sums are closed where the next gate begins.
template <int kDt, bool kVec, bool kCluster, bool kGate, bool kShift>
__global__ void __launch_bounds__(512) block_norms_grad_kernel(const BlockNormsGradArgs a) {
    __shared__ float2 slots[2 * 16 * 8];
    __shared__ float sums[kCluster ? 1 : 512 * 8];
    using E = typename Element<kDt>::type;
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
    g.slots = slots + group * 2 * g.warps;
    g.turn = 0;
    const Columns<kVec> cols{g.t, a.lanes, int(g.rank) * a.lanes * 8, a.cols};
    const int groups = int(blockDim.x) / a.lanes;
    const int set = int(blockIdx.x) / a.cluster, worker = set * groups + group;
    const int64_t first = worker * a.chunk, last = min(a.rows, first + a.chunk);
    const float inv_n = 1.f / float(a.cols);
    if constexpr (kCluster) ptx::cluster_sync();  // nobody writes into a CTA that has not started

    float w2[8], w1[8];  // Pre's weight; scale * gate * Post's weight
    load_vector<kVec>(w2, a.pre_weight, 1.f, cols, 0);
    load_vector<kVec>(w1, a.post_weight, 1.f, cols, 0);
#pragma unroll
    for (int j = 0; j < 8; ++j) w1[j] *= a.scale;
    float sa[8], sb[8], sc[8], sd[8], ta[8], tb[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) sa[j] = sb[j] = sc[j] = sd[j] = ta[j] = tb[j] = 0.f;

    Piece<kDt> gate, next[4];
    int64_t gate_at = 0, gate_end = 0;  // the gate in hand, the first row behind its rows
    auto take_gate = [&](int64_t of) {
        gate_at = of;
        gate_end = (of + 1) * int64_t(a.rows_per_gate);
        load_piece<kDt, kVec>(gate, static_cast<const E *>(a.gate) + size_t(of) * a.cols, cols, 0, true);
        load_vector<kVec>(w1, a.post_weight, 1.f, cols, 0);
#pragma unroll
        for (int j = 0; j < 8; ++j) w1[j] *= a.scale * gate.get(j);
    };
    gate.zero();
    if (kGate && first < last) take_gate(uint32_t(first) / a.rows_per_gate);
    auto fetch = [&](int64_t r, bool on) {
        const size_t at = on ? size_t(r) * a.cols : 0;
        load_piece<kDt, kVec>(next[0], static_cast<const E *>(a.h) + at, cols, 0, on);
        load_piece<kDt, kVec>(next[1], static_cast<const E *>(a.x_out) + at, cols, 0, on && a.dy);
        load_piece<kDt, kVec>(next[2], static_cast<const E *>(a.dy) + at, cols, 0, on && a.dy);
        load_piece<kDt, kVec>(next[3], static_cast<const E *>(a.dx_out) + at, cols, 0, on && a.dx_out);
    };
    fetch(first, first < last);
    // (every thread of a warp makes the same turns)
    for (int64_t i = 0; i < a.chunk; ++i) {
        const int64_t r = first + i;
        const bool on = r < last;
        float h[8], x[8], dy[8], dx[8];
        next[0].unpack(h), next[1].unpack(x), next[2].unpack(dy), next[3].unpack(dx);
        fetch(r + 1, r + 1 < last);
        const size_t at = on ? size_t(r) * a.cols : 0;
        float2 sh, sx;
        spreads<kVec, kCluster>(g, a.post, a.pre, h, x, cols, inv_n, a.eps, sh, sx);
        if (!on) sh.y = sx.y = 0.f;  // (an eps of 0 would make a NaN of a row that is not there)
        if (a.dy) {
            float s0 = 0.f, s1 = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                x[j] = cols.live(0, j) ? (x[j] - sx.x) * sx.y : 0.f;
                sc[j] = fmaf(dy[j], x[j], sc[j]);
                if constexpr (kShift) sd[j] += dy[j];
                dy[j] *= w2[j];
                s0 += dy[j];
                s1 = fmaf(dy[j], x[j], s1);
            }
            float2 m = make_float2(0.f, 0.f);
            if (a.pre != CF_NORM_NONE) m = row_sum<kCluster>(g, s0, s1);
            m.x = a.pre == CF_NORM_LAYER ? m.x * inv_n : 0.f;
            m.y *= inv_n;
#pragma unroll
            for (int j = 0; j < 8; ++j) dx[j] = fmaf(sx.y, dy[j] - m.x - x[j] * m.y, dx[j]);
        }
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            h[j] = cols.live(0, j) ? (h[j] - sh.x) * sh.y : 0.f;
            sa[j] = fmaf(dx[j], h[j], sa[j]);
            if constexpr (kShift) sb[j] += cols.live(0, j) ? dx[j] : 0.f;
            x[j] = dx[j] * w1[j];
            s0 += cols.live(0, j) ? x[j] : 0.f;
            s1 = fmaf(x[j], h[j], s1);
            dx[j] *= a.alpha;
        }
        if (a.dx) store_piece<kDt, kVec>(static_cast<E *>(a.dx) + at, dx, cols, 0, on);
        float2 m = make_float2(0.f, 0.f);
        if (a.post != CF_NORM_NONE) m = row_sum<kCluster>(g, s0, s1);
        m.x = a.post == CF_NORM_LAYER ? m.x * inv_n : 0.f;
        m.y *= inv_n;
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = sh.y * (x[j] - m.x - h[j] * m.y);
        store_piece<kDt, kVec>(static_cast<E *>(a.dh) + at, x, cols, 0, on);
        if constexpr (kGate) {
            if (on && (r + 1 == last || r + 1 == gate_end)) {  // its last row here
                float v[8], w[8], b[8];
                load_vector<kVec>(w, a.post_weight, 1.f, cols, 0);
                load_vector<kVec>(b, a.post_bias, 0.f, cols, 0);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    v[j] = a.scale * fmaf(w[j], sa[j], kShift ? b[j] * sb[j] : 0.f);
                    const float k = a.scale * gate.get(j);
                    ta[j] = fmaf(k, sa[j], ta[j]);
                    if constexpr (kShift) tb[j] = fmaf(k, sb[j], tb[j]);
                    sa[j] = sb[j] = 0.f;
                }
                const int64_t from = gate_end - int64_t(a.rows_per_gate);
                if (a.dgate && from >= first && gate_end <= last) {
                    store_piece<kDt, kVec>(static_cast<E *>(a.dgate) + size_t(gate_at) * a.cols, v, cols, 0, true);
                } else if (a.dgate) {  // slot 0: begun by a worker before; slot 1: here, and goes on
                    float *const slot = a.slots + (size_t(2) * worker + (from >= first ? 1 : 0)) * a.cols;
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (cols.live(0, j)) __stcg(slot + cols.at(0, j), v[j]);
                }
                if (r + 1 < last) take_gate(gate_at + 1);
            }
        }
    }
    // the CTA's sums: those of its groups of threads are added through shared memory
    const bool wanted[4] = {a.sum_at[0] >= 0, a.sum_at[1] >= 0, a.sum_at[2] >= 0, a.sum_at[3] >= 0};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if (!wanted[k]) continue;
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] = k == 0 ? (kGate ? ta[j] : a.scale * sa[j])
                   : k == 1 ? (kGate ? tb[j] : a.scale * sb[j]) : k == 2 ? sc[j] : sd[j];
        float *const out = a.partials + (size_t(a.sum_at[k]) * a.sets + set) * a.cols;
        if (kCluster || groups == 1) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (cols.live(0, j)) __stcg(out + cols.at(0, j), v[j]);
        } else {
            __syncthreads();
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (cols.live(0, j)) sums[group * a.lanes * 8 + cols.at(0, j)] = v[j];
            __syncthreads();
            for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
                float s = 0.f;
                for (int i = 0; i < groups; ++i) s += sums[i * a.lanes * 8 + c];
                __stcg(out + c, s);
            }
        }
    }
    if constexpr (kCluster) ptx::cluster_sync();  // no CTA leaves while its peers may still write to it
}

// The workers' sums added in order: 32 columns a CTA, a warp every 32nd term, then the warps.
__global__ void __launch_bounds__(1024) block_norms_sums_kernel(const BlockNormsGradArgs a, int nsums, int gates_first) {
    __shared__ float part[32][33];
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
    for (int i = warp; i < terms; i += 128) {
        float x[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            x[k] = live && i + 32 * k < terms ? __ldcg(from + (i + 32 * k) * step + c) : 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) s += x[k];
    }
    part[warp][lane] = s;
    __syncthreads();
    if (warp != 0 || !live) return;
    s = 0.f;
#pragma unroll
    for (int k = 0; k < 32; ++k) s += part[k][lane];
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

cudaError_t launch(const void *fn, dim3 grid, int threads, int cluster, bool pdl, cudaStream_t stream, void **args) {
    cudaLaunchConfig_t cfg = {};
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

template <int kDt, bool kVec>
const void *forward_kernel(int pieces) {
    return pieces == 1   ? reinterpret_cast<const void *>(&block_norms_kernel<kDt, kVec, 1>)
           : pieces == 2 ? reinterpret_cast<const void *>(&block_norms_kernel<kDt, kVec, 2>)
                         : reinterpret_cast<const void *>(&block_norms_kernel<kDt, kVec, 4>);
}
template <int kDt, bool kVec, bool kCluster>
const void *grad_kernel(bool gate, bool shift) {
    if (gate)
        return shift ? reinterpret_cast<const void *>(&block_norms_grad_kernel<kDt, kVec, kCluster, true, true>)
                     : reinterpret_cast<const void *>(&block_norms_grad_kernel<kDt, kVec, kCluster, true, false>);
    return shift ? reinterpret_cast<const void *>(&block_norms_grad_kernel<kDt, kVec, kCluster, false, true>)
                 : reinterpret_cast<const void *>(&block_norms_grad_kernel<kDt, kVec, kCluster, false, false>);
}
template <int kDt>
const void *grad_kernel_of(bool vec, bool cluster, bool gate, bool shift) {
    if (cluster)
        return vec ? grad_kernel<kDt, true, true>(gate, shift) : grad_kernel<kDt, false, true>(gate, shift);
    return vec ? grad_kernel<kDt, true, false>(gate, shift) : grad_kernel<kDt, false, false>(gate, shift);
}

}  // namespace

cudaError_t launch_block_norms(BlockNormsArgs a, bool vec, int sms, bool pdl, cudaStream_t stream) {
    const int pieces = (a.cols + 7) / 8;
    const int per = pieces <= 32 ? 1 : pieces <= 1024 ? 2 : 4;
    a.lanes = round_lanes((pieces + per - 1) / per);
    const int groups = std::max(1, 256 / a.lanes), threads = groups * a.lanes;
    const int64_t ctas = std::min<int64_t>((a.rows + groups - 1) / groups, int64_t(sms) * (2048 / threads) * 4);
    const void *fn = a.dtype == CF_BF16   ? (vec ? forward_kernel<CF_BF16, true>(per) : forward_kernel<CF_BF16, false>(per))
                     : a.dtype == CF_FP16 ? (vec ? forward_kernel<CF_FP16, true>(per) : forward_kernel<CF_FP16, false>(per))
                                          : (vec ? forward_kernel<CF_FP32, true>(per) : forward_kernel<CF_FP32, false>(per));
    void *args[] = {&a};
    return launch(fn, dim3(unsigned(ctas)), threads, 1, pdl, stream, args);
}

BlockNormsGradPlan plan_block_norms_grad(int64_t rows, int64_t cols, int sms) {
    BlockNormsGradPlan p;
    const int64_t pieces = (cols + 7) / 8;
    p.cluster = int((pieces + 511) / 512);
    p.lanes = round_lanes((pieces + p.cluster - 1) / p.cluster);
    const int groups = p.cluster > 1 ? 1 : std::max(1, 256 / p.lanes);
    p.threads = groups * p.lanes;
    const int64_t most = int64_t(sms) * std::max(1, 512 / p.threads) / p.cluster;
    const int64_t sets = std::max<int64_t>(1, std::min<int64_t>(most, (rows + groups - 1) / groups));
    p.chunk = (rows + sets * groups - 1) / (sets * groups);
    p.sets = int((rows + p.chunk * groups - 1) / (p.chunk * groups));
    p.workers = p.sets * groups;
    return p;
}

cudaError_t launch_block_norms_grad(BlockNormsGradArgs a, const BlockNormsGradPlan &p, bool vec, bool pdl,
                                    cudaStream_t stream) {
    a.lanes = p.lanes;
    a.cluster = p.cluster;
    a.chunk = p.chunk;
    a.sets = p.sets;
    const bool gate = a.gate != nullptr, shift = a.post_bias || a.sum_at[1] >= 0 || a.sum_at[3] >= 0;
    const bool cluster = p.cluster > 1;
    const void *fn = a.dtype == CF_BF16   ? grad_kernel_of<CF_BF16>(vec, cluster, gate, shift)
                     : a.dtype == CF_FP16 ? grad_kernel_of<CF_FP16>(vec, cluster, gate, shift)
                                          : grad_kernel_of<CF_FP32>(vec, cluster, gate, shift);
    void *args[] = {&a};
    cudaError_t e = launch(fn, dim3(unsigned(p.sets * p.cluster)), p.threads, p.cluster, pdl, stream, args);
    if (e != cudaSuccess) return e;
    int nsums = 0;
    for (int k = 0; k < 4; ++k) nsums += a.sum_at[k] >= 0;
    const int64_t gates = gate ? a.rows / a.rows_per_gate : 0;
    int gates_first = gates <= p.workers;
    const int shared = gate && a.dgate && a.rows_per_gate > 1 ? int(std::min<int64_t>(gates, p.workers)) : 0;
    if (nsums + shared == 0) return cudaSuccess;
    void *args2[] = {&a, &nsums, &gates_first};
    return launch(reinterpret_cast<const void *>(&block_norms_sums_kernel),
                  dim3(unsigned((a.cols + 31) / 32) * unsigned(nsums + shared)), 1024, 1, pdl, stream, args2);
}

}  // namespace cf
