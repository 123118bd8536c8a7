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
    float *slots;   // two halves of `half` numbers, one for every second exchange
    int half;
    int turn;
};

// v summed over the row (of one CTA); every thread of the row gets the same bits.  The slots behind the last warp's, up
// to a multiple of four, hold zeros.
__device__ __forceinline__ float row_sum(Group &g, float v) {
    if (g.lanes >= 32) {
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
    } else {
        for (int d = g.lanes >> 1; d >= 1; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
    }
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
        const int all = g.warps * (kCluster ? g.cluster : 1);
        s = 0.f;
        for (int i = lane / kV; i < all; i += 32 / kV) s += slots[i * kV + lane % kV];
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
// x with 0 in the place of columns behind the last one
template <bool kVec>
__device__ __forceinline__ Two live_two(Two x, const Columns<kVec> &cols, int p, int j) {
    const float2 q = x.parts();
    return Two(cols.live(p, 2 * j) ? q.x : 0.f, cols.live(p, 2 * j + 1) ? q.y : 0.f);
}

// The reciprocal root of one norm's row held in x (1: no norm), which loses its mean where the norm takes it.
// kFull: it may be a LayerNorm.
template <bool kVec, int kP, bool kFull>
__device__ __forceinline__ float spread(Group &g, int norm, Two (&x)[kP][4], const Columns<kVec> &cols, float inv_n,
                                        float eps) {
    if (norm == CF_NORM_NONE) return 1.f;
    if (kFull && norm == CF_NORM_LAYER) {
        Two s(0.f);
#pragma unroll
        for (int p = 0; p < kP; ++p)
#pragma unroll
            for (int j = 0; j < 4; ++j) s = s + x[p][j];
        const Two mean(-row_sum(g, s.sum()) * inv_n);
#pragma unroll
        for (int p = 0; p < kP; ++p)
#pragma unroll
            for (int j = 0; j < 4; ++j) x[p][j] = live_two(x[p][j] + mean, cols, p, j);
    }
    Two s(0.f);
#pragma unroll
    for (int p = 0; p < kP; ++p)
#pragma unroll
        for (int j = 0; j < 4; ++j) s = fma(x[p][j], x[p][j], s);
    return __frsqrt_rn(fmaf(row_sum(g, s.sum()), inv_n, eps));
}

// kP pieces a thread.  kFull: LayerNorms or biases, too.
template <int kDt, bool kVec, int kP, bool kFull>
__global__ void __launch_bounds__(kP == 4 ? 1024 : 512, kP == 4 ? 1 : 2) block_norms_kernel(const BlockNormsArgs a) {
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
    __syncthreads();
    const Columns<kVec> cols{g.t, a.lanes, 0, a.cols};
    const int groups = int(blockDim.x) / a.lanes;
    const float inv_n = 1.f / float(a.cols);
    const Two alpha(a.x ? a.alpha : 0.f);
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
        Two x[kP][4];
#pragma unroll
        for (int p = 0; p < kP; ++p) hp[p].unpack(x[p]);
        Two root(a.scale * spread<kVec, kP, kFull>(g, a.post, x, cols, inv_n, a.eps));
#pragma unroll
        for (int p = 0; p < kP; ++p) {
            Two w[4], u[4];
            load_vector<kVec>(w, a.post_weight, 1.f, cols, p);
            xp[p].unpack(u);
#pragma unroll
            for (int j = 0; j < 4; ++j) x[p][j] = x[p][j] * root;
            if (kFull && a.post_bias) {  // root has the scale
                Two b[4];
                load_vector<kVec>(b, a.post_bias, 0.f, cols, p);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    x[p][j] = fma(x[p][j], w[j], b[j] * Two(a.scale));
                    w[j] = Two(1.f);
                }
            }
            if (gate) {
                Two k[4];
                gp[p].unpack(k);
#pragma unroll
                for (int j = 0; j < 4; ++j) w[j] = w[j] * k[j];
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[p][j] = fma(x[p][j], w[j], u[j] * alpha);
                // (behind the last column a weight that is not there would be 1, but what it multiplies is 0)
            }
            if (a.x_out) store_piece<kDt, kVec>(static_cast<E *>(a.x_out) + at, x[p], cols, p, on);
        }
        if (a.y == nullptr) continue;
        root = Two(spread<kVec, kP, kFull>(g, a.pre, x, cols, inv_n, a.eps));
#pragma unroll
        for (int p = 0; p < kP; ++p) {
            Two w[4], b[4];
            load_vector<kVec>(w, a.pre_weight, 1.f, cols, p);
            if constexpr (kFull) load_vector<kVec>(b, a.pre_bias, 0.f, cols, p);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[p][j] = x[p][j] * root;
                x[p][j] = kFull ? fma(x[p][j], w[j], b[j]) : x[p][j] * w[j];
            }
            store_piece<kDt, kVec>(static_cast<E *>(a.y) + at, x[p], cols, p, on);
        }
    }
}

// ---------------------------------------------------------------------------
// gradient
// ---------------------------------------------------------------------------
// a thread's columns of a vector of the workspace
template <bool kVec>
__device__ __forceinline__ void store_floats(float *out, const Two (&x)[4], const Columns<kVec> &cols) {
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        const float2 q = x[j / 2].parts();
        if (kVec && cols.live(0, j)) __stcg(reinterpret_cast<float2 *>(out + cols.at(0, j)), q);
        if (!kVec && cols.live(0, j)) __stcg(out + cols.at(0, j), q.x);
        if (!kVec && cols.live(0, j + 1)) __stcg(out + cols.at(0, j + 1), q.y);
    }
}

// With hc and xc the rows without their means (RMSNorm: the rows), g2 = dy w2 and w1 = scale gate weight, every sum that
// the row needs is one over products of what is loaded:
//     sum g2 x^ = r2 sum g2 xc,
//     d  = dx' + r2 (g2 - mean(g2) - x^ mean(g2 x^)),
//     sum w1 d h^ = r1 (sum w1 hc dx' + r2 (sum w1 hc g2 - mean(g2) sum w1 hc - r2 mean(g2 x^) sum w1 hc xc)),
// so one exchange between the threads serves where three would follow one another (16384 x 4096 bf16: 287 us with
// three).  A LayerNorm's means come one exchange before.
// kFull: LayerNorms or biases, too.  kGate: a gate, whose rows' sums are closed where the next gate begins.
template <int kDt, bool kVec, bool kCluster, bool kGate, bool kFull>
__global__ void __launch_bounds__(512) block_norms_grad_kernel(const BlockNormsGradArgs a) {
    constexpr int kV = kFull ? 16 : 8;
    __shared__ float slots[2 * 16 * kV * (kCluster ? 8 : 1)];
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
    g.half = g.warps * kV * (kCluster ? a.cluster : 1);
    g.slots = slots + group * 2 * g.half;
    g.turn = 0;
    const Columns<kVec> cols{g.t, a.lanes, int(g.rank) * a.lanes * 8, a.cols};
    const int groups = int(blockDim.x) / a.lanes;
    const int set = int(blockIdx.x) / a.cluster, worker = set * groups + group;
    const int64_t first = worker * a.chunk, last = min(a.rows, first + a.chunk);
    const float inv_n = 1.f / float(a.cols);
    const bool lh = kFull && a.post == CF_NORM_LAYER, lx = kFull && a.pre == CF_NORM_LAYER;
    if constexpr (kCluster) ptx::cluster_sync();  // nobody writes into a CTA that has not started

    Two w2[4], w1[4];  // Pre's weight; scale * gate * Post's weight
    load_vector<kVec>(w2, a.pre_weight, 1.f, cols, 0);
    Two sa[4], sb[4], sc[4], sd[4], ta[4], tb[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) sa[j] = sb[j] = sc[j] = sd[j] = ta[j] = tb[j] = Two(0.f);

    Piece<kDt> gate, next[4];
    int64_t gate_at = 0, gate_end = 0;  // the gate in hand, the first row behind its rows
    auto scaled_gate = [&](int j) {
        return Two(a.scale) * (a.gate ? Two(gate.get(2 * j), gate.get(2 * j + 1)) : Two(1.f));
    };
    auto take_gate = [&](int64_t of) {
        gate_at = of;
        gate_end = (of + 1) * int64_t(a.rows_per_gate);
        load_piece<kDt, kVec>(gate, static_cast<const E *>(a.gate) + size_t(of) * a.cols, cols, 0, a.gate != nullptr);
        load_vector<kVec>(w1, a.post_weight, 1.f, cols, 0);
#pragma unroll
        for (int j = 0; j < 4; ++j) w1[j] = live_two(w1[j] * scaled_gate(j), cols, 0, j);
    };
    gate.zero();
    if (kGate && first < last) {
        take_gate(uint32_t(first) / a.rows_per_gate);
    } else {
        load_vector<kVec>(w1, a.post_weight, 1.f, cols, 0);
#pragma unroll
        for (int j = 0; j < 4; ++j) w1[j] = live_two(w1[j] * Two(a.scale), cols, 0, j);
    }
    size_t ahead = first < last ? size_t(first) * a.cols : 0;  // where the next row to fetch lies
    auto fetch = [&](bool on) {
        load_piece<kDt, kVec>(next[0], static_cast<const E *>(a.h) + ahead, cols, 0, on);
        load_piece<kDt, kVec>(next[1], static_cast<const E *>(a.x_out) + ahead, cols, 0, on && a.dy);
        load_piece<kDt, kVec>(next[2], static_cast<const E *>(a.dy) + ahead, cols, 0, on && a.dy);
        load_piece<kDt, kVec>(next[3], static_cast<const E *>(a.dx_out) + ahead, cols, 0, on && a.dx_out);
        if (on) ahead += size_t(a.cols);
    };
    size_t at = ahead;  // where the row in hand lies
    fetch(first < last);
    // (every thread of a warp makes the same turns)
    for (int64_t i = 0; i < a.chunk; ++i) {
        const int64_t r = first + i;
        const bool on = r < last;
        Two h[4], x[4], y[4], d[4];
        next[0].unpack(h), next[1].unpack(x), next[2].unpack(y), next[3].unpack(d);
        fetch(r + 1 < last);
        if (lh || lx) {
            Two s(0.f), t(0.f);
#pragma unroll
            for (int j = 0; j < 4; ++j) s = s + h[j], t = t + x[j];
            float v[2] = {s.sum(), t.sum()};
            row_sums<2, kCluster>(g, v);
            const Two mh(lh ? -v[0] * inv_n : 0.f), mx(lx ? -v[1] * inv_n : 0.f);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                h[j] = live_two(h[j] + mh, cols, 0, j);
                x[j] = live_two(x[j] + mx, cols, 0, j);
            }
        }
        constexpr int kSums = kFull ? 12 : 6;
        Two p[kSums];
#pragma unroll
        for (int k = 0; k < kSums; ++k) p[k] = Two(0.f);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const Two g2 = y[j] * w2[j], wh = w1[j] * h[j];
            p[0] = fma(h[j], h[j], p[0]);
            p[1] = fma(x[j], x[j], p[1]);
            p[2] = fma(g2, x[j], p[2]);
            p[3] = fma(wh, d[j], p[3]);
            p[4] = fma(wh, g2, p[4]);
            p[5] = fma(wh, x[j], p[5]);
            if constexpr (kFull) {
                p[6] = p[6] + g2;
                p[7] = p[7] + wh;
                p[8] = fma(w1[j], d[j], p[8]);
                p[9] = fma(w1[j], g2, p[9]);
                p[10] = fma(w1[j], x[j], p[10]);
                p[11] = p[11] + w1[j];
            }
        }
        float v[kV];
#pragma unroll
        for (int k = 0; k < kV; ++k) v[k] = k < kSums ? p[k < kSums ? k : 0].sum() : 0.f;
        row_sums<kV, kCluster>(g, v);
        // (an eps of 0 would make a NaN of a row that is not there)
        const float r1 = a.post == CF_NORM_NONE ? 1.f : on ? __frsqrt_rn(fmaf(v[0], inv_n, a.eps)) : 0.f;
        const float r2 = a.pre == CF_NORM_NONE ? 1.f : on ? __frsqrt_rn(fmaf(v[1], inv_n, a.eps)) : 0.f;
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
        for (int j = 0; j < 4; ++j) {
            d[j] = fma(x[j], kb, fma(y[j] * w2[j], k2, d[j]));
            if constexpr (kFull) d[j] = d[j] + ka;
            sc[j] = fma(y[j], x[j] * k2, sc[j]);
            if constexpr (kFull) sd[j] = sd[j] + y[j], sb[j] = sb[j] + d[j];
            h[j] = h[j] * k1;
            sa[j] = fma(d[j], h[j], sa[j]);
            h[j] = fma(h[j], kn, (w1[j] * d[j]) * k1);
            if constexpr (kFull) h[j] = h[j] + km;
            d[j] = d[j] * Two(a.alpha);
        }
        if (a.dx) store_piece<kDt, kVec>(static_cast<E *>(a.dx) + at, d, cols, 0, on);
        store_piece<kDt, kVec>(static_cast<E *>(a.dh) + at, h, cols, 0, on);
        if (on) at += size_t(a.cols);
        if constexpr (kGate) {
            if (on && (r + 1 == last || r + 1 == gate_end)) {  // its last row here
                Two w[4], b[4];
                load_vector<kVec>(w, a.post_weight, 1.f, cols, 0);
                if constexpr (kFull) load_vector<kVec>(b, a.post_bias, 0.f, cols, 0);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const Two k = scaled_gate(j);
                    ta[j] = fma(k, sa[j], ta[j]);
                    d[j] = w[j] * sa[j];
                    if constexpr (kFull) {
                        d[j] = fma(b[j], sb[j], d[j]);
                        tb[j] = fma(k, sb[j], tb[j]);
                        sb[j] = Two(0.f);
                    }
                    d[j] = d[j] * Two(a.scale);
                    sa[j] = Two(0.f);
                }
                const int64_t from = gate_end - int64_t(a.rows_per_gate);
                if (a.dgate && from >= first && gate_end <= last) {
                    store_piece<kDt, kVec>(static_cast<E *>(a.dgate) + size_t(gate_at) * a.cols, d, cols, 0, true);
                } else if (a.dgate) {  // slot 0: begun by a worker before; slot 1: here, and goes on
                    float *const slot = a.slots + (size_t(2) * worker + (from >= first ? 1 : 0)) * a.cols;
                    store_floats<kVec>(slot, d, cols);
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
        Two v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            v[j] = k == 0 ? (kGate ? ta[j] : Two(a.scale) * sa[j])
                   : k == 1 ? (kGate ? tb[j] : Two(a.scale) * sb[j]) : k == 2 ? sc[j] : sd[j];
        float *const out = a.partials + (size_t(a.sum_at[k]) * a.sets + set) * a.cols;
        if (kCluster || groups == 1) {
            store_floats<kVec>(out, v, cols);
        } else {
            __syncthreads();
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float2 q = v[j / 2].parts();
                if (cols.live(0, j)) sums[group * a.lanes * 8 + cols.at(0, j)] = j % 2 ? q.y : q.x;
            }
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

// The workers' sums added in order: 32 columns a CTA, a warp every kSumWarps-th term, then the warps.
constexpr int kSumWarps = 8, kSumFly = 8;
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
    for (int i = warp; i < terms; i += kSumWarps * kSumFly) {
        float x[kSumFly];
#pragma unroll
        for (int k = 0; k < kSumFly; ++k)
            x[k] = live && i + kSumWarps * k < terms ? __ldcg(from + (i + kSumWarps * k) * step + c) : 0.f;
#pragma unroll
        for (int k = 0; k < kSumFly; ++k) s += x[k];
    }
    part[warp][lane] = s;
    __syncthreads();
    if (warp != 0 || !live) return;
    s = 0.f;
#pragma unroll
    for (int k = 0; k < kSumWarps; ++k) s += part[k][lane];
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

template <int kDt, bool kVec, bool kFull>
const void *forward_kernel(int pieces) {
    return pieces == 1   ? reinterpret_cast<const void *>(&block_norms_kernel<kDt, kVec, 1, kFull>)
           : pieces == 2 ? reinterpret_cast<const void *>(&block_norms_kernel<kDt, kVec, 2, kFull>)
                         : reinterpret_cast<const void *>(&block_norms_kernel<kDt, kVec, 4, kFull>);
}
template <int kDt>
const void *forward_kernel(bool vec, bool full, int pieces) {
    if (!vec) return forward_kernel<kDt, false, true>(pieces);
    return full ? forward_kernel<kDt, true, true>(pieces) : forward_kernel<kDt, true, false>(pieces);
}
// (what is rare is compiled in its widest form alone)
template <int kDt>
const void *grad_kernel(bool vec, bool cluster, bool gate, bool full) {
    if (!vec)
        return cluster ? reinterpret_cast<const void *>(&block_norms_grad_kernel<kDt, false, true, true, true>)
                       : reinterpret_cast<const void *>(&block_norms_grad_kernel<kDt, false, false, true, true>);
    if (cluster)
        return full ? reinterpret_cast<const void *>(&block_norms_grad_kernel<kDt, true, true, true, true>)
                    : reinterpret_cast<const void *>(&block_norms_grad_kernel<kDt, true, true, true, false>);
    if (gate)
        return full ? reinterpret_cast<const void *>(&block_norms_grad_kernel<kDt, true, false, true, true>)
                    : reinterpret_cast<const void *>(&block_norms_grad_kernel<kDt, true, false, true, false>);
    return full ? reinterpret_cast<const void *>(&block_norms_grad_kernel<kDt, true, false, false, true>)
                : reinterpret_cast<const void *>(&block_norms_grad_kernel<kDt, true, false, false, false>);
}

}  // namespace

cudaError_t launch_block_norms(BlockNormsArgs a, bool vec, int sms, bool pdl, cudaStream_t stream) {
    const int pieces = (a.cols + 7) / 8;
    const int per = pieces <= 32 ? 1 : pieces <= 1024 ? 2 : 4;
    a.lanes = round_lanes((pieces + per - 1) / per);
    const int groups = std::max(1, 256 / a.lanes), threads = groups * a.lanes;
    const int64_t ctas = std::min<int64_t>((a.rows + groups - 1) / groups, int64_t(sms) * (2048 / threads) * 4);
    const bool full = a.post == CF_NORM_LAYER || a.pre == CF_NORM_LAYER || a.post_bias || a.pre_bias;
    const void *fn = a.dtype == CF_BF16   ? forward_kernel<CF_BF16>(vec, full, per)
                     : a.dtype == CF_FP16 ? forward_kernel<CF_FP16>(vec, full, per)
                                          : forward_kernel<CF_FP32>(vec, full, per);
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
    const bool gate = a.gate != nullptr, cluster = p.cluster > 1;
    const bool full = a.post_bias || a.sum_at[1] >= 0 || a.sum_at[3] >= 0 || a.post == CF_NORM_LAYER ||
                      a.pre == CF_NORM_LAYER;
    const void *fn = a.dtype == CF_BF16   ? grad_kernel<CF_BF16>(vec, cluster, gate, full)
                     : a.dtype == CF_FP16 ? grad_kernel<CF_FP16>(vec, cluster, gate, full)
                                          : grad_kernel<CF_FP32>(vec, cluster, gate, full);
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
                  dim3(unsigned((a.cols + 31) / 32) * unsigned(nsums + shared)), kSumWarps * 32, 1, pdl, stream, args2);
}

}  // namespace cf
