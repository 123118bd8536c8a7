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
#include <atomic>
#include <cstdint>

#include "block_norms.h"
#include "pieces.cuh"
#include "ptx.cuh"

#ifndef NREG
#define NREG 96
#define NTHR 512
#endif
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
// Rows on their way, in shared memory: a thread fills and reads its own columns alone, so nobody waits for anybody.  The
// ring has kDepth stages of up to kRows rows (one of each of that many matrices), a row kP pieces a thread.  (16-bit
// numbers that start anywhere cannot be copied so; theirs are loaded when they are needed.)
__host__ __device__ constexpr int ring_depth(int dt) { return dt == CF_FP32 ? 2 : 4; }
__host__ __device__ constexpr bool has_ring(int dt, bool vec, int pieces) { return (vec || dt == CF_FP32) && pieces <= 2; }
constexpr int kMostSmem = 232448;  // of a CTA (227 KB)
inline int ring_bytes(int dt, bool vec, int rows, int pieces, int threads) {
    return has_ring(dt, vec, pieces) ? ring_depth(dt) * rows * threads * pieces * 8 * type_bytes(dt) : 0;
}
template <int kDt, bool kVec, int kRows, int kP>
struct RowRing {
    using E = typename Element<kDt>::type;
    static constexpr bool kOn = has_ring(kDt, kVec, kP);
    static constexpr int kDepth = ring_depth(kDt);
    static constexpr int kCopies = kVec ? Piece<kDt>::kWords / 4 : 8;  // of a piece
    static constexpr uint32_t kBytes = kVec ? 16 : 4;                  // of a copy
    const E *src[kRows];  // this thread's first column of the next row; null: zeros
    const Columns<kVec> &cols;
    uint32_t base, step;  // of this thread's copies; from one to the next
    int rows, stage, left;  // rows: of a stage; left: rows to come
    size_t apart;

    __device__ __forceinline__ RowRing(const Columns<kVec> &c, uint32_t ring, int rows_, int left_)
        : cols(c), base(ring + threadIdx.x * kBytes), step(blockDim.x * kBytes), rows(rows_), stage(0), left(left_),
          apart(size_t(c.n)) {}
    __device__ __forceinline__ void matrix(int k, const void *m, int64_t row) {
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
    return reciprocal_root(fmaf(row_sum(g, s.sum()), inv_n, eps));
}

// kP pieces a thread.  kFull: LayerNorms or biases, too.  A worker takes a stretch of neighbouring rows, as in the gradient.
template <int kDt, bool kVec, int kP, bool kFull>
__global__ void __maxnreg__(kP == 4 ? 64 : NREG) block_norms_kernel(const BlockNormsArgs a) {
    extern __shared__ __align__(16) uint8_t ring_smem[];
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
    const int64_t mine = int64_t(blockIdx.x) * groups + group;
    const int first = int(min(a.rows, mine * a.chunk)), last = int(min(a.rows, int64_t(first) + a.chunk));
    // rows that threads of one warp may share a warp's turn with: as many turns as any; else their own
    const int turns = a.lanes < 32 ? a.chunk : last - first;
    RowRing<kDt, kVec, 3, kP> ring(cols, ptx::smem_u32(ring_smem), a.gates_along ? 3 : 2, last - first);
    ring.matrix(0, a.h, first);
    ring.matrix(1, a.x, first);
    ring.matrix(2, a.gates_along ? a.gate : nullptr, first);
    ring.start();

    Two w1[kP][4], w2[kP][4];  // Post's weight times the gate; Pre's
    int gate_end = 0;          // the first row behind the rows of the gate in w1
    auto take_gate = [&](int of, bool here) {
        gate_end = int((uint32_t(of) + 1u) * a.rows_per_gate);
#pragma unroll
        for (int p = 0; p < kP; ++p) {
            load_vector<kVec>(w1[p], a.post_weight, 1.f, cols, p);
            if (!a.gate) continue;
            Piece<kDt> q;
            if (here) {
                ring.take(q, 2, p);
            } else {
                q.zero();
                load_piece<kDt, kVec>(q, static_cast<const E *>(a.gate) + size_t(of) * a.cols, cols, p, true);
            }
            Two k[4];
            q.unpack(k);
#pragma unroll
            for (int j = 0; j < 4; ++j) w1[p][j] = w1[p][j] * k[j];
        }
    };
#pragma unroll
    for (int p = 0; p < kP; ++p) load_vector<kVec>(w2[p], a.pre_weight, 1.f, cols, p);
    if (!a.gates_along) take_gate(int(uint32_t(first) / a.rows_per_gate < uint32_t(a.gates) ? uint32_t(first) / a.rows_per_gate : 0u), false);
    E *xo = static_cast<E *>(a.x_out), *yo = static_cast<E *>(a.y);
    if (xo) xo += size_t(first) * a.cols;
    if (yo) yo += size_t(first) * a.cols;
    for (int i = 0; i < turns; ++i) {
        const bool on = first + i < last;
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
            for (int j = 0; j < 4; ++j) x[p][j] = fma(x[p][j] * root, w1[p][j], u[j] * alpha);
            if (kFull && a.post_bias) {  // scale gate bias; the gate from memory again
                Two b[4];
                load_vector<kVec>(b, a.post_bias, 0.f, cols, p);
                if (a.gate) {
                    if (a.gates_along) {
                        ring.take(q, 2, p);
                    } else {
                        q.zero();
                        load_piece<kDt, kVec>(
                            q, static_cast<const E *>(a.gate) + size_t(gate_end / a.rows_per_gate - 1) * a.cols, cols, p,
                            on);
                    }
                    q.unpack(u);
#pragma unroll
                    for (int j = 0; j < 4; ++j) b[j] = b[j] * u[j];
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) x[p][j] = fma(b[j], Two(a.scale), x[p][j]);
            }
            if (xo) store_piece<kDt, kVec>(xo, x[p], cols, p, on);
        }
        ring.next();
        if (xo) xo += a.cols;
        if (yo == nullptr) continue;
        root = Two(spread<kVec, kP, kFull>(g, a.pre, x, cols, inv_n, a.eps));
#pragma unroll
        for (int p = 0; p < kP; ++p) {
            Two b[4];
            if constexpr (kFull) load_vector<kVec>(b, a.pre_bias, 0.f, cols, p);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[p][j] = x[p][j] * root;
                x[p][j] = kFull ? fma(x[p][j], w2[p][j], b[j]) : x[p][j] * w2[p][j];
            }
            store_piece<kDt, kVec>(yo, x[p], cols, p, on);
        }
        yo += a.cols;
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
// Rows ahead go through a ring in shared memory, of which a thread fills and reads its own columns alone, so nobody waits
// for anybody: kept in registers on their way, they left no room for the sums (16384 x 4096 bf16: 172 us).
// kFull: LayerNorms or biases, too.  kGate: a gate, whose rows' sums are closed where the next gate begins.
template <int kDt, bool kVec, bool kCluster, bool kGate, bool kFull>
__global__ void __launch_bounds__(512) block_norms_grad_kernel(const BlockNormsGradArgs a) {
    constexpr int kV = kFull ? 16 : 8;
    extern __shared__ __align__(16) uint8_t ring_smem[];
    __shared__ float slots[2 * (16 * kV + 8 * 32) * (kCluster ? 8 : 1)];  // of up to 8 groups, each rounded up to 32
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
    // (whole rounds of 32 numbers; what no warp writes stays zero)
    g.half = (g.warps * kV * (kCluster ? a.cluster : 1) + 31) & ~31;
    g.slots = slots + group * 2 * g.half;
    g.turn = 0;
    if constexpr (!kCluster) {
        for (int i = threadIdx.x; i < int(sizeof(slots) / 4); i += blockDim.x) slots[i] = 0.f;
        __syncthreads();
    }
    const Columns<kVec> cols{g.t, a.lanes, int(g.rank) * a.lanes * 8, a.cols};
    const int groups = int(blockDim.x) / a.lanes;
    const int set = int(blockIdx.x) / a.cluster, worker = set * groups + group;
    const int chunk = int(a.chunk);
    const int first = int(min(a.rows, int64_t(worker) * chunk)), last = int(min(a.rows, int64_t(first) + chunk));
    // rows that threads of one warp may share a warp's turn with: as many turns as any; else their own
    const int turns = a.lanes < 32 ? chunk : last - first;
    const float inv_n = 1.f / float(a.cols);
    const bool lh = kFull && a.post == CF_NORM_LAYER, lx = kFull && a.pre == CF_NORM_LAYER;
    if constexpr (kCluster) ptx::cluster_sync();  // nobody writes into a CTA that has not started

    Two w2[4], w1[4];  // Pre's weight; scale * gate * Post's weight
    load_vector<kVec>(w2, a.pre_weight, 1.f, cols, 0);
    Two sa[4], sb[4], sc[4], sd[4], ta[4], tb[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) sa[j] = sb[j] = sc[j] = sd[j] = ta[j] = tb[j] = Two(0.f);

    Piece<kDt> gate;
    int gate_at = 0, gate_end = 0;  // the gate in hand, the first row behind its rows
    auto scaled_gate = [&](int j) {
        return Two(a.scale) * (a.gate ? Two(gate.get(2 * j), gate.get(2 * j + 1)) : Two(1.f));
    };
    auto take_gate = [&](int of, bool here) {  // here: it lies in `gate`
        gate_at = of;
        gate_end = int((uint32_t(of) + 1u) * a.rows_per_gate);
        if (a.gate && !here)
            load_piece<kDt, kVec>(gate, static_cast<const E *>(a.gate) + size_t(of) * a.cols, cols, 0, true);
        load_vector<kVec>(w1, a.post_weight, 1.f, cols, 0);
#pragma unroll
        for (int j = 0; j < 4; ++j) w1[j] = live_two(w1[j] * scaled_gate(j), cols, 0, j);
    };
    gate.zero();
    const bool gates_along = kGate && RowRing<kDt, kVec, 5, 1>::kOn && a.gate && a.rows_per_gate == 1;
    if (kGate && !gates_along && first < last) {
        take_gate(int(uint32_t(first) / a.rows_per_gate), false);
    } else if (!kGate) {
        load_vector<kVec>(w1, a.post_weight, 1.f, cols, 0);
#pragma unroll
        for (int j = 0; j < 4; ++j) w1[j] = live_two(w1[j] * Two(a.scale), cols, 0, j);
    }

    RowRing<kDt, kVec, 5, 1> ring(cols, ptx::smem_u32(ring_smem), gates_along ? 5 : 4, last - first);
    ring.matrix(0, a.h, first);
    ring.matrix(1, a.dy ? a.x_out : nullptr, first);
    ring.matrix(2, a.dy, first);
    ring.matrix(3, a.dx_out, first);
    ring.matrix(4, gates_along ? a.gate : nullptr, first);
    ring.start();
    size_t at = first < last ? size_t(first) * a.cols : 0;  // where the row in hand lies
    for (int i = 0; i < turns; ++i) {
        const int r = first + i;
        const bool on = r < last;
        ring.turn();
        Piece<kDt> raw[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) ring.take(raw[k], k, 0);
        if (gates_along && on) {
            ring.take(gate, 4, 0);
            take_gate(r, true);
        }
        ring.next();
        Two h[4], x[4], y[4], d[4];
        raw[0].unpack(h), raw[1].unpack(x), raw[2].unpack(y), raw[3].unpack(d);
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
                const int from = gate_end - int(a.rows_per_gate);
                if (a.dgate && from >= first && gate_end <= last) {
                    store_piece<kDt, kVec>(static_cast<E *>(a.dgate) + size_t(gate_at) * a.cols, d, cols, 0, true);
                } else if (a.dgate) {  // slot 0: begun by a worker before; slot 1: here, and goes on
                    float *const slot = a.slots + (size_t(2) * worker + (from >= first ? 1 : 0)) * a.cols;
                    store_floats<kVec>(slot, d, cols);
                }
                if (r + 1 < last && !gates_along) take_gate(gate_at + 1, false);
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
cudaError_t allow_smem(const void *fn) {
    struct Entry {
        std::atomic<const void *> fn;
        std::atomic<uint64_t> devices;
    };
    static Entry table[128];  // (51 kernels)
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidValue;
    for (Entry &t : table) {
        const void *at = t.fn.load(std::memory_order_acquire);
        if (at == nullptr && t.fn.compare_exchange_strong(at, fn, std::memory_order_acq_rel)) at = fn;
        if (at != fn) continue;
        if (t.devices.load(std::memory_order_acquire) >> dev & 1) return cudaSuccess;
        cudaFuncAttributes attr;
        e = cudaFuncGetAttributes(&attr, fn);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     kMostSmem - int(attr.sharedSizeBytes));
        if (e == cudaSuccess) t.devices.fetch_or(uint64_t(1) << dev, std::memory_order_acq_rel);
        return e;
    }
    return cudaErrorInvalidValue;
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

constexpr int kForwardThreads = NTHR;

cudaError_t launch_block_norms(BlockNormsArgs a, bool vec, int sms, bool pdl, cudaStream_t stream) {
    const int pieces = (a.cols + 7) / 8;
    const int per = pieces <= 32 ? 1 : pieces <= 1024 && (pieces + 63) / 64 * 32 <= 512 ? 2 : 4;
    a.lanes = round_lanes((pieces + per - 1) / per);
    const int groups = std::max(1, 256 / a.lanes), threads = groups * a.lanes;
    // CTAs of up to kForwardThreads an SM, of a stretch of rows each
    int64_t ctas = std::min<int64_t>((a.rows + groups - 1) / groups, int64_t(sms) * std::max(1, kForwardThreads / threads));
    a.chunk = int((a.rows + ctas * groups - 1) / (ctas * groups));
    ctas = (a.rows + int64_t(a.chunk) * groups - 1) / (int64_t(a.chunk) * groups);
    a.gates_along = a.gate && a.rows_per_gate == 1 && has_ring(a.dtype, vec, per);
    const bool full = a.post == CF_NORM_LAYER || a.pre == CF_NORM_LAYER || a.post_bias || a.pre_bias;
    const void *fn = a.dtype == CF_BF16   ? forward_kernel<CF_BF16>(vec, full, per)
                     : a.dtype == CF_FP16 ? forward_kernel<CF_FP16>(vec, full, per)
                                          : forward_kernel<CF_FP32>(vec, full, per);
    void *args[] = {&a};
    const int smem = ring_bytes(a.dtype, vec, a.gates_along ? 3 : 2, per, threads);
    const cudaError_t e = allow_smem(fn);
    return e != cudaSuccess ? e : launch(fn, dim3(unsigned(ctas)), threads, 1, pdl, stream, args, smem);
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
    const int smem = ring_bytes(a.dtype, vec, a.gate && a.rows_per_gate == 1 ? 5 : 4, 1, p.threads);
    cudaError_t e = allow_smem(fn);
    if (e != cudaSuccess) return e;
    e = launch(fn, dim3(unsigned(p.sets * p.cluster)), p.threads, p.cluster, pdl, stream, args, smem);
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
