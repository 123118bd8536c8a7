// logprobs.cu -- what a model's logits are asked for: of z = scale * logits, a row,
//     lse      = log sum exp z
//     logprob  = z[target] - lse
//     entropy  = lse - sum p z,  p = exp(z - lse)
//     the top tokens and their log probabilities
// in one pass over the row, and the gradient
//     dlogits  = scale (dlogprob (1[target] - p) + dlse p - dentropy p (z - lse + entropy)).
//
// HBM bounds both: the logits are read once (the gradient: and written once).  A thread carries the running maximum m of
// its logits, s = sum 2^d and t = sum d 2^d with d = (z - m) log2 e, so that lse = m + ln s and entropy = ln s - ln2 t / s
// lose nothing to a large m.  (The difference comes first, the scale second: a row of the type's lowest number does not
// overflow.)  Where few rows leave SMs idle a cluster of CTAs shares a row.
//
// Rows start anywhere: a row is cut at 16-byte boundaries of its memory into windows, the first and last of which may be
// partial and are read number by number.  The gradient's windows are the logits': into rows that start elsewhere in 16
// bytes it stores number by number (4096 x 32003 bf16 of rows 32064 apart: into rows as far apart 82 us, into contiguous
// ones 310; fp32 into contiguous ones 178, floor 156).
//
// What stands between the loads and HBM's rate is the instructions: 17 a number at first (322 us for 4096 x 128000 bf16), 10
// now (200 us with eight top tokens, 5.2 TB/s; without top tokens 163, 6.4 TB/s; without the entropy either 158; the
// gradient 308, the copy's rate, without the entropy's 305).
// d is the difference times scale log2 e, a factor rounded once, and 2^d the hardware's: two steps of fp32 (2^-22) and 3
// half steps of |d| ln 2 of each term, which is what the log probabilities are off by (some 8e-8 of their size).
// So numbers are worked on in pairs, maxima are taken of 16-bit pairs as they are, and -inf, whose 0 times -inf would be a
// NaN in the entropy, is raised to a low finite number as a pair too, where the running maximum shows that this changes
// nothing; elsewhere (rows of nothing but masks) number by number.
//
// Top tokens: a thread also remembers its largest logit and the first window that holds it.  A bound that k of the
// threads' (largest, window) pairs reach is one below which no top token can lie, and where hardly more than k reach it,
// only those threads have anything on the bound or above it: in that one window, or, where the largest of the others shows
// it, in any.  These windows are read again, and what reaches the bound, little more than k numbers, is ranked by counting.  Pairs order equal logits by window, so equal logits in any number (a masked row) change nothing.
// Rows made so that more than kCandidates numbers reach the bound are searched once for each of the k.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstddef>
#include <cstdint>

#include "logprobs.h"
#include "pieces.cuh"
#include "ptx.cuh"

namespace cf {
namespace {

constexpr uint32_t kAll = 0xffffffffu;
constexpr float kLog2E = 1.4426950408889634f, kLn2F = 0.6931471805599453f;
constexpr int kMaxThreads = 256, kMaxCluster = 8;
constexpr int kCandidates = 1024;
constexpr int kSlack = 8;  // threads more than top tokens that may be looked at again
constexpr int kFly = 4;  // windows in flight
constexpr uint32_t kInfoTarget = 0x72000000u;

__device__ __forceinline__ float inf() { return __int_as_float(0x7f800000); }
// the larger one; a NaN stays one
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// An order of all numbers as unsigned ones: -inf lowest, NaN above everything, the zeros alike.
__device__ __forceinline__ uint32_t order(float v) {
    const uint32_t b = __float_as_uint(v + 0.f);
    if ((b & 0x7fffffffu) > 0x7f800000u) return kAll;
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t o) {
    if (o == kAll) return __uint_as_float(0x7fc00000u);
    return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}
// larger first, of equals the lower index
__device__ __forceinline__ uint64_t pair_of(uint32_t o, uint32_t index) { return uint64_t(o) << 32 | uint32_t(~index); }

// 16 bytes of numbers
template <int kDt>
struct Pack {
    static constexpr int kN = kDt == CF_FP32 ? 4 : 8;
    uint32_t u[4];

    __device__ __forceinline__ float get(int j) const {
        if constexpr (kDt == CF_FP32) return __uint_as_float(u[j]);
        else if constexpr (kDt == CF_FP16) return __half2float(__ushort_as_half(uint16_t(u[j / 2] >> (j % 2 * 16))));
        else return __uint_as_float(j % 2 ? u[j / 2] & 0xffff0000u : u[j / 2] << 16);
    }
    __device__ __forceinline__ void set(int j, float v) {
        if constexpr (kDt == CF_FP32) {
            u[j] = __float_as_uint(v);
        } else {
            const uint32_t h = from_float<kDt>(v);
            u[j / 2] = j % 2 ? (u[j / 2] & 0xffffu) | h << 16 : (u[j / 2] & 0xffff0000u) | h;
        }
    }
    __device__ __forceinline__ Two pair(int j) const { return Two(get(2 * j), get(2 * j + 1)); }
    __device__ __forceinline__ void set_pair(int j, Two v) {
        const float2 p = v.parts();
        if constexpr (kDt == CF_FP32) {
            u[2 * j] = __float_as_uint(p.x), u[2 * j + 1] = __float_as_uint(p.y);
        } else if constexpr (kDt == CF_FP16) {
            const __half2 h = __floats2half2_rn(p.x, p.y);
            u[j] = *reinterpret_cast<const uint32_t *>(&h);
        } else {
            u[j] = ptx::pack_bf16x2(p.x, p.y);
        }
    }
    // the larger ones of two words' numbers; NaNs stay
    __device__ __forceinline__ static uint32_t larger(uint32_t a, uint32_t b) {
        uint32_t r;
        if constexpr (kDt == CF_FP32) asm("max.NaN.f32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        else if constexpr (kDt == CF_FP16) asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        else asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    __device__ __forceinline__ float largest() const {
        Pack m;
        m.u[0] = larger(larger(u[0], u[1]), larger(u[2], u[3]));
        return kDt == CF_FP32 ? m.get(0) : max_nan(m.get(0), m.get(1));
    }
    __device__ __forceinline__ void raise(uint32_t low) {
#pragma unroll
        for (int i = 0; i < 4; ++i) u[i] = larger(u[i], low);
    }
    // What -inf is raised to, as a word; and the sizes that m and m + the distance to it must keep to for this to be
    // right: above `least`, which is so far above it that what it stands for counts 0, and below `most`, so that m s2 is
    // finite.
    __device__ __forceinline__ static uint32_t low() {
        return kDt == CF_FP32 ? 0xf2fc6f7cu /* -1e31 */ : kDt == CF_FP16 ? 0xfbfffbffu /* -65504 */ : 0xf2fcf2fcu;
    }
    __device__ __forceinline__ static float least(float s2) {
        return (kDt == CF_FP16 ? -65504.f : kDt == CF_FP32 ? -1e31f : __uint_as_float(0xf2fc0000u)) + 160.f / s2;
    }
    __device__ __forceinline__ static float most(float s2) { return s2 < 1e7f ? 1e30f : 0.f; }
};

// The windows of a row: 16 bytes of memory each, from the one that holds the row's first number.
template <int kDt>
struct Windows {
    using E = typename Element<kDt>::type;
    static constexpr int kN = 16 / int(sizeof(E));  // numbers of a window
    const E *row;
    int vocab, lead, count;  // lead: numbers of the first window that lie in front of the row
    __device__ Windows(const E *r, int v) : row(r), vocab(v) {
        lead = int((reinterpret_cast<uintptr_t>(r) & 15u) / sizeof(E));
        count = int((int64_t(v) + lead + kN - 1) / kN);
    }
    __device__ __forceinline__ int first(int w) const { return w * kN - lead; }  // index of its first number
    __device__ __forceinline__ int full0() const { return lead > 0 ? 1 : 0; }    // the first whole window
    __device__ __forceinline__ int full1() const { return (vocab + lead) / kN; }  // the one behind the last whole window
    __device__ __forceinline__ Pack<kDt> whole(int w) const {
        const uint4 v = __ldcs(reinterpret_cast<const uint4 *>(row + first(w)));
        return Pack<kDt>{{v.x, v.y, v.z, v.w}};
    }
    // any window, and none; what is not of the row is -inf
    __device__ __forceinline__ Pack<kDt> any(int w) const {
        if (w >= full0() && w < full1()) return whole(w);
        Pack<kDt> p{};
        const int i0 = first(w);
#pragma unroll
        for (int i = 0; i < kN; ++i)
            p.set(i, w < count && i0 + i >= 0 && i0 + i < vocab ? to_float<kDt>(row[i0 + i]) : -inf());
        return p;
    }
};

// running maximum, sum and weighted sum (16 bytes: a CTA sends m and s to another one as a pair)
struct __align__(16) Stats {
    float m, s, t;
    __device__ __forceinline__ float ref() const { return m == -inf() ? 0.f : m; }
    // the same with a larger maximum
    __device__ __forceinline__ void raise(float to, float s2) {
        if (to > m) {
            if (s != 0.f) {
                // (from 200 on r is 0, and 0 times an infinite d would be a NaN)
                const float d = fminf((to - m) * s2, 200.f), r = ptx::ex2_approx(-d);
                t = r * (t - d * s);
                s *= r;
            }
            m = to;
        }
    }
    __device__ __forceinline__ void add(Stats o, float s2) {
        raise(o.m, s2);
        o.raise(m, s2);
        s += o.s;
        t += o.t;
    }
};

// One CTA's share of a row: window 0, where it is partial, is the first thread's of the first CTA; the others go round.
template <int kDt>
struct Share {
    Windows<kDt> w;
    int part, parts;  // this CTA of the row's
    __device__ __forceinline__ int round() const { return parts * int(blockDim.x); }  // windows from a step to the next
    __device__ __forceinline__ int window(int step, int t) const {  // step -1: the partial one
        if (step < 0) return part == 0 && t == 0 && w.full0() > 0 ? 0 : w.count;
        return w.full0() + (step * parts + part) * int(blockDim.x) + t;
    }
    __device__ __forceinline__ int steps() const { return (w.count - w.full0() + round() - 1) / round(); }  // of any thread
};

template <int kDt>
__device__ void search_tops(const Share<kDt> &sh, int k, uint64_t *top, uint64_t *scratch) {
    // every pair in turn: the largest below the one before
    uint64_t below = ~uint64_t(0);
    for (int i = 0; i < k; ++i) {
        uint64_t best = 0;
        for (int step = -1; step < sh.steps(); ++step) {
            const int w = sh.window(step, int(threadIdx.x));
            if (w >= sh.w.count) continue;
            const Pack<kDt> x = sh.w.any(w);
#pragma unroll
            for (int j = 0; j < Windows<kDt>::kN; ++j) {
                const int at = sh.w.first(w) + j;
                const uint64_t p = pair_of(order(x.get(j)), uint32_t(at));
                if (at >= 0 && at < sh.w.vocab && p < below && p > best) best = p;
            }
        }
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1) best = max(best, __shfl_xor_sync(kAll, best, d));
        if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = best;
        __syncthreads();
        for (int j = 0; j < int(blockDim.x >> 5); ++j) best = max(best, scratch[j]);
        if (threadIdx.x == 0) top[i] = best;
        below = best;
        __syncthreads();
    }
}

// most: the thread's largest logit with its first window, a pair (0: none); second: the order of its other windows' largest
template <int kDt>
__device__ void find_tops(const Share<kDt> &sh, uint64_t most, uint32_t second, int k, uint64_t *top, uint64_t *pairs,
                          uint32_t *seconds, int *chosen, uint64_t *bound, int *found, int *many) {
    const int tid = int(threadIdx.x), n = int(blockDim.x);
    pairs[tid] = most;
    seconds[tid] = second;
    if (tid == 0) *found = 0;
    if (tid < k) top[tid] = 0;
    __syncthreads();
    // One warp looks for an order that at least k pairs reach and hardly more, halving the range that is left; where many
    // are on the bound itself, so it does for their window.  (The k largest in turn were 3.4 us for each of the k for
    // 4096 x 128000 bf16; every thread counting the pairs above its own took a sixth of the kernel's instructions.
    // Threads without a window have no pair; where fewer than k have one, everything is a candidate.)
    constexpr int kShift = kDt == CF_FP32 ? 0 : kDt == CF_FP16 ? 13 : 16;  // an order's bits that are always the same
    if (tid < 32) {
        uint32_t order_of[kMaxThreads / 32], window_of[kMaxThreads / 32], low = kAll, high = 0;
        int have = 0;
#pragma unroll
        for (int i = 0; i < kMaxThreads / 32; ++i) {
            const uint64_t p = tid + 32 * i < n ? pairs[tid + 32 * i] : 0;
            order_of[i] = uint32_t(p >> 32) >> kShift;
            window_of[i] = uint32_t(~p);
            if (p == 0) continue;
            ++have;
            low = min(low, order_of[i]);
            high = max(high, order_of[i]);
        }
        have = __reduce_add_sync(kAll, have);
        low = __reduce_min_sync(kAll, low);
        high = __reduce_max_sync(kAll, high);
        // pairs that have an order above o, or o itself and a window of at most w
        auto count = [&](uint32_t o, uint32_t w) {
            int c = 0;
#pragma unroll
            for (int i = 0; i < kMaxThreads / 32; ++i) c += order_of[i] > o || (order_of[i] == o && window_of[i] <= w);
            return __reduce_add_sync(kAll, c);
        };
        uint32_t last = kAll;
        if (have < k) {
            low = 0;
        } else if (have > k + kSlack) {
            while (low < high) {
                const uint32_t mid = low + (high - low + 1) / 2;
                const int c = count(mid, kAll);
                if (c < k) {
                    high = mid - 1;
                } else {
                    low = mid;
                    have = c;
                    if (c <= k + kSlack) break;
                }
            }
            if (have > k + kSlack) {
                uint32_t from = 0;
                last = uint32_t(sh.w.count);
                while (from < last) {
                    const uint32_t mid = from + (last - from) / 2;
                    const int c = count(low, mid);
                    if (c < k) {
                        from = mid + 1;
                    } else {
                        last = mid;
                        if (c <= k + kSlack) break;
                    }
                }
            }
        }
        // from the front the windows of those that have no other one of interest, from the back the others' threads
        int front = 0, back = 0;
#pragma unroll
        for (int i = 0; i < kMaxThreads / 32; ++i) {
            const bool on = order_of[i] != 0 && (order_of[i] > low || (order_of[i] == low && window_of[i] <= last));
            const bool more = on && seconds[tid + 32 * i] >> kShift >= low;
            const uint32_t one = __ballot_sync(kAll, on && !more), all = __ballot_sync(kAll, more);
            const uint32_t before = (1u << tid) - 1u;
            if (on && !more) chosen[front + __popc(one & before)] = int(window_of[i]);
            if (more) chosen[kLogprobsMaxTop + kSlack - 1 - back - __popc(all & before)] = tid + 32 * i;
            front += __popc(one);
            back += __popc(all);
        }
        if (tid == 0) {
            *bound = uint64_t(low) << 32 | last;
            many[0] = front;
            many[1] = back;
        }
    }
    __syncthreads();
    const int ones = many[0];
    const uint32_t least = uint32_t(*bound >> 32), last = uint32_t(*bound);
    const int steps = sh.steps() + 1;
    for (int i = tid; i < ones + many[1] * steps; i += n) {
        int w;
        if (i < ones) {
            w = chosen[i];
        } else {
            const int who = (i - ones) / steps;
            w = sh.window(i - ones - who * steps - 1, chosen[kLogprobsMaxTop + kSlack - 1 - who]);
        }
        if (w >= sh.w.count) continue;
        const Pack<kDt> x = sh.w.any(w);
#pragma unroll
        for (int j = 0; j < Windows<kDt>::kN; ++j) {
            const int at = sh.w.first(w) + j;
            const uint32_t o = order(x.get(j));
            if (at < 0 || at >= sh.w.vocab) continue;
            if (o >> kShift > least || (o >> kShift == least && uint32_t(w) <= last)) {
                const int slot = atomicAdd(found, 1);
                if (slot < kCandidates) pairs[slot] = pair_of(o, uint32_t(at));
            }
        }
    }
    __syncthreads();
    const int all = *found;
    if (all > kCandidates) {
        search_tops(sh, k, top, pairs);
        return;
    }
    for (int c = tid; c < all; c += n) {
        const uint64_t p = pairs[c];
        int r = 0;
        for (int i = 0; i < all; ++i) r += pairs[i] > p;
        if (r < k) top[r] = p;
    }
    __syncthreads();
}

template <int kDt, bool kEntropy, bool kTop>
__global__ void __launch_bounds__(kMaxThreads, 4) logprobs_kernel(const LogprobsArgs a) {
    __shared__ Stats warp_stats[kMaxThreads / 32];
    __shared__ Stats cta_stats[kMaxCluster];
    __shared__ uint64_t pairs[kTop ? kCandidates : 1];
    __shared__ uint64_t tops[kTop ? kMaxCluster * kLogprobsMaxTop : 1];  // of the row's CTAs, in the first one
    __shared__ int chosen[kLogprobsMaxTop + kSlack];
    __shared__ uint64_t bound;
    __shared__ uint32_t seconds[kTop ? kMaxThreads : 1];
    __shared__ int found, many[2];
    static_assert(kCandidates >= kMaxThreads, "one pair a thread");
    static_assert(sizeof(Stats) == 16 && offsetof(Stats, m) == 0 && offsetof(Stats, s) == 4 && offsetof(Stats, t) == 8,
                  "sent as a pair and a number");
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    using E = typename Element<kDt>::type;
    constexpr int kN = Windows<kDt>::kN;
    const int tid = int(threadIdx.x), lane = tid & 31, warp = tid >> 5;
    const int64_t r = int64_t(blockIdx.x) / a.cluster;
    const int part = int(int64_t(blockIdx.x) - r * a.cluster);
    const E *const row = static_cast<const E *>(a.logits) + r * a.stride;
    const Share<kDt> sh{Windows<kDt>(row, a.vocab), part, a.cluster};
    const float s2 = a.scale * kLog2E;

    int64_t target = -1;
    float given = 0.f;
    if (part == 0 && tid == 0 && a.targets) {
        target = a.targets[r];
        if (target < -1 || target >= a.vocab) {
            ptx::record_error(a.err, 8u /*CF_ERR_DEVICE_BOUNDS*/, kInfoTarget);
            target = -1;
        }
        if (target >= 0) given = to_float<kDt>(row[target]);
    }

    Stats st{-inf(), 0.f, 0.f};
    // the largest logit, in an order of signed numbers (a maximum's NaN is a positive one, so it is above everything; no
    // logit has the lowest number), and its first window
    int most_order = int(0x80000000u), second_order = int(0x80000000u);
    uint32_t most_window = 0;
    using P = Pack<kDt>;
    const uint32_t low = P::low();
    const float least = P::least(s2), beyond = P::most(s2);
    // n windows from w on, `step` apart
    auto take = [&](P (&x)[kFly], int n, int w, int step) {
        float high = -inf();
#pragma unroll
        for (int i = 0; i < kFly; ++i) {
            if (i >= n) break;
            const float m = x[i].largest();
            if constexpr (kTop) {
                const int bits = __float_as_int(m + 0.f), o = bits ^ (bits >> 31 & 0x7fffffff);
                second_order = max(second_order, min(most_order, o));
                if (o > most_order) {
                    most_order = o;
                    most_window = uint32_t(w + i * step);
                }
            }
            high = fmaxf(high, m);
        }
        st.raise(high, s2);
        if (st.m > least && fabsf(st.m) < beyond) {
            const Two k(s2), c(-st.m);
            Two sum(0.f), weighted(0.f);
#pragma unroll
            for (int i = 0; i < kFly; ++i) {
                if (i >= n) break;
                if constexpr (kEntropy) x[i].raise(low);
#pragma unroll
                for (int j = 0; j < kN / 2; ++j) {
                    const Two d = (x[i].pair(j) + c) * k;  // (the difference first: m s2 would be rounded)
                    const float2 p = d.parts();
                    const Two e(ptx::ex2_approx(p.x), ptx::ex2_approx(p.y));
                    sum = sum + e;
                    if constexpr (kEntropy) weighted = fma(e, d, weighted);
                }
            }
            st.s += sum.sum();
            if constexpr (kEntropy) st.t += weighted.sum();
        } else {
            const float ref = st.ref();
#pragma unroll 1
            for (int i = 0; i < n; ++i)
#pragma unroll
                for (int j = 0; j < kN; ++j) {
                    float v = x[0].get(j);
#pragma unroll
                    for (int q = 1; q < kFly; ++q) v = i == q ? x[q].get(j) : v;
                    const float d = max_nan((v - ref) * s2, -200.f);  // (of -inf: 2^-200 is 0, and 0 times it)
                    const float e = ptx::ex2_approx(d);
                    st.s += e;
                    st.t = fmaf(e, d, st.t);
                }
        }
    };
    const int round = sh.round(), w0 = sh.window(0, tid);
    P x[kFly];
    if (sh.window(-1, tid) == 0) {
        x[0] = sh.w.any(0);
        take(x, 1, 0, 0);
    }
    // windows that are whole for every thread of the CTA, kFly at a time, the next ones on their way
    int w = w0, g = 0;
    const int whole = (sh.w.full1() - (w0 - tid) - int(blockDim.x) + round) / round;  // steps whose last thread's is whole
    const int turns = max(0, whole) / kFly;
    if (turns > 0) {
        // (two sets of registers that take turns: moving one to the other costs half an instruction a number)
        const uint4 *from = reinterpret_cast<const uint4 *>(sh.w.row + sh.w.first(w));
        auto fetch = [&](P (&to)[kFly]) {
#pragma unroll
            for (int i = 0; i < kFly; ++i) {
                const uint4 v = __ldcs(from + i * round);
                to[i] = P{{v.x, v.y, v.z, v.w}};
            }
            from += kFly * round;
        };
        P y[kFly];
        fetch(x);
#pragma unroll 1
        for (;;) {
            if (g + 1 < turns) fetch(y);
            take(x, kFly, w, round);
            w += kFly * round;
            if (++g >= turns) break;
            if (g + 1 < turns) fetch(x);
            take(y, kFly, w, round);
            w += kFly * round;
            if (++g >= turns) break;
        }
    }
#pragma unroll 1
    for (; w < sh.w.count; w += kFly * round) {
#pragma unroll
        for (int i = 0; i < kFly; ++i) x[i] = sh.w.any(w + i * round);
        const int n = min(kFly, (sh.w.count - w + round - 1) / round);
        take(x, n, w, round);
    }
    auto unsigned_order = [](int o) {
        return o == int(0x80000000u) ? 0u : order(__int_as_float(o ^ (o >> 31 & 0x7fffffff)));
    };
    const uint64_t most = most_order == int(0x80000000u) ? 0 : pair_of(unsigned_order(most_order), most_window);
    const uint32_t second = unsigned_order(second_order);
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1)
        st.add(Stats{__shfl_xor_sync(kAll, st.m, d), __shfl_xor_sync(kAll, st.s, d), __shfl_xor_sync(kAll, st.t, d)}, s2);
    if (lane == 0) warp_stats[warp] = st;
    if constexpr (kTop) find_tops(sh, most, second, a.top, tops + part * kLogprobsMaxTop, pairs, seconds, chosen, &bound, &found, many);
    __syncthreads();
    if (tid == 0) {
        for (int i = 1; i < int(blockDim.x >> 5); ++i) st.add(warp_stats[i], s2);
        cta_stats[part] = st;
    }
    if (a.cluster > 1) {
        ptx::cluster_sync();  // every CTA has started
        if (part != 0) {
            if (tid == 0) {
                const uint32_t to = ptx::mapa(ptx::smem_u32(cta_stats + part), 0u);
                ptx::st_cluster_v2f32(to, st.m, st.s);
                ptx::st_cluster_f32(to + 8, st.t);
            }
            if (kTop && tid < a.top) {
                const uint64_t p = tops[part * kLogprobsMaxTop + tid];
                ptx::st_cluster_v2f32(ptx::mapa(ptx::smem_u32(tops + part * kLogprobsMaxTop + tid), 0u),
                                      __uint_as_float(uint32_t(p)), __uint_as_float(uint32_t(p >> 32)));
            }
        }
        ptx::cluster_sync();
        if (part != 0) return;
        if (tid == 0)
            for (int i = 1; i < a.cluster; ++i) st.add(cta_stats[i], s2);
    }
    if (tid == 0) {
        warp_stats[0] = st;
        const float log_s = logf(st.s);
        const bool none = st.s == 0.f;  // nothing but -inf
        if (a.lse) a.lse[r] = none ? -inf() : fmaf(st.ref(), a.scale, log_s);
        if (a.logprob)
            a.logprob[r] = target < 0 ? 0.f : none ? -inf() : (given - st.ref()) * a.scale - log_s;
        if (kEntropy && a.entropy) a.entropy[r] = none ? 0.f : log_s - kLn2F * (st.t / st.s);
    }
    if constexpr (kTop) {
        __syncthreads();
        st = warp_stats[0];
        const float log_s = logf(st.s);
        for (int c = tid; c < a.cluster * a.top; c += int(blockDim.x)) {
            const int at = c / a.top * kLogprobsMaxTop + c % a.top;
            const uint64_t p = tops[at];
            int rank = c % a.top;
            if (a.cluster > 1) {
                rank = 0;
                for (int i = 0; i < a.cluster; ++i)
                    for (int j = 0; j < a.top; ++j) rank += tops[i * kLogprobsMaxTop + j] > p;
            }
            if (p != 0 && rank < a.top) {
                const size_t out = size_t(r) * a.top + rank;
                if (a.top_ids) a.top_ids[out] = uint32_t(~p);
                if (a.top_logprobs)
                    a.top_logprobs[out] =
                        st.s == 0.f ? -inf() : (value_of(uint32_t(p >> 32)) - st.ref()) * a.scale - log_s;
            }
        }
    }
}

// ---------------------------------------------------------------------------
// gradient
// ---------------------------------------------------------------------------
constexpr int kGradThreads = 256;

template <int kDt, bool kEntropy>
__global__ void __launch_bounds__(kGradThreads) logprobs_grad_kernel(const LogprobsGradArgs a) {
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    using E = typename Element<kDt>::type;
    using P = Pack<kDt>;
    constexpr int kN = P::kN;
    const int64_t r = int64_t(blockIdx.x) / a.chunks;
    const int chunk = int(int64_t(blockIdx.x) - r * a.chunks);
    const Windows<kDt> win(static_cast<const E *>(a.logits) + r * a.stride, a.vocab);
    E *const out = static_cast<E *>(a.dlogits) + r * a.dstride;
    const bool same = (reinterpret_cast<uintptr_t>(out) & 15u) == (reinterpret_cast<uintptr_t>(win.row) & 15u);
    int w = chunk * (a.turns * kFly * kGradThreads) + int(threadIdx.x);
    const int end = min(win.count, (chunk + 1) * (a.turns * kFly * kGradThreads));
    P next[kFly];
#pragma unroll
    for (int i = 0; i < kFly; ++i) next[i] = win.any(w + i * kGradThreads);
    int64_t target = a.targets ? a.targets[r] : -1;
    if (target < -1 || target >= a.vocab) {
        if (threadIdx.x == 0) ptx::record_error(a.err, 8u /*CF_ERR_DEVICE_BOUNDS*/, kInfoTarget);
        target = -1;
    }
    const float lse = a.lse[r];
    const float given = target >= 0 && a.dlogprob ? a.dlogprob[r] * a.scale : 0.f;
    const float dh = kEntropy ? a.dentropy[r] * a.scale : 0.f;
    // p times (c0 + c1 d), d = z - lse
    const float c0 = (a.dlse ? a.dlse[r] * a.scale : 0.f) - given - (kEntropy ? dh * a.entropy[r] : 0.f);
    const bool none = lse == -inf();
    // -inf may count as a low finite number (see Pack) where its distance from lse is large, and finite
    const float least = P::least(a.scale * kLog2E) * a.scale;
    const uint32_t low = P::low();
    // (... and where c0 + c1 d, too, is finite there, or 0 times it would be a NaN)
    const float lowest = P{{low, low, low, low}}.get(0);
    const bool finite = !kEntropy || fabsf(fmaf(-dh, fmaf(lowest, a.scale, -lse), c0)) < 3e38f;
    const bool plain = lse > least && fabsf(lse) < P::most(a.scale) && !none && finite;
    const Two scale(a.scale), shift(-lse), log2e(kLog2E), k0(c0), k1(-dh);
#pragma unroll 1
    for (; w < end; w += kFly * kGradThreads) {
        P x[kFly];
#pragma unroll
        for (int i = 0; i < kFly; ++i) x[i] = next[i];
        if (w + kFly * kGradThreads < end) {
#pragma unroll
            for (int i = 0; i < kFly; ++i) next[i] = win.any(w + (kFly + i) * kGradThreads);
        }
#pragma unroll
        for (int i = 0; i < kFly; ++i) {
            const int v = w + i * kGradThreads, i0 = win.first(v);
            if (v >= end) break;
            if (plain) {
                if constexpr (kEntropy) x[i].raise(low);
#pragma unroll
                for (int j = 0; j < kN / 2; ++j) {
                    const Two d = fma(x[i].pair(j), scale, shift);
                    const float2 q = (d * log2e).parts();
                    const Two p(ptx::ex2_approx(q.x), ptx::ex2_approx(q.y));
                    Two g = p * (kEntropy ? fma(k1, d, k0) : k0);
                    const int at = i0 + 2 * j;
                    if (uint32_t(int(target) - at) < 2u) {
                        const float2 h = g.parts();
                        g = int(target) == at ? Two(h.x + given, h.y) : Two(h.x, h.y + given);
                    }
                    x[i].set_pair(j, g);
                }
            } else {
#pragma unroll
                for (int j = 0; j < kN; ++j) {
                    float d = fmaf(x[i].get(j), a.scale, -lse);
                    if constexpr (kEntropy) d = max_nan(d, -200.f);  // (of -inf: 2^-288 is 0, and 0 times it)
                    float g = ptx::ex2_approx(d * kLog2E) * (kEntropy ? fmaf(-dh, d, c0) : c0);
                    if (i0 + j == target) g += given;
                    x[i].set(j, none ? 0.f : g);
                }
            }
            if (same && i0 >= 0 && i0 + kN <= a.vocab) {
                __stcs(reinterpret_cast<uint4 *>(out + i0), make_uint4(x[i].u[0], x[i].u[1], x[i].u[2], x[i].u[3]));
            } else {
#pragma unroll
                for (int j = 0; j < kN; ++j)
                    if (i0 + j >= 0 && i0 + j < a.vocab) out[i0 + j] = from_float<kDt>(x[i].get(j));
            }
        }
    }
}

template <int kDt>
const void *forward_kernel(bool entropy, bool top) {
    if (entropy)
        return top ? reinterpret_cast<const void *>(&logprobs_kernel<kDt, true, true>)
                   : reinterpret_cast<const void *>(&logprobs_kernel<kDt, true, false>);
    return top ? reinterpret_cast<const void *>(&logprobs_kernel<kDt, false, true>)
               : reinterpret_cast<const void *>(&logprobs_kernel<kDt, false, false>);
}
template <int kDt>
const void *grad_kernel(bool entropy) {
    return entropy ? reinterpret_cast<const void *>(&logprobs_grad_kernel<kDt, true>)
                   : reinterpret_cast<const void *>(&logprobs_grad_kernel<kDt, false>);
}

cudaError_t launch(const void *fn, unsigned ctas, int threads, int cluster, bool pdl, cudaStream_t stream, void **args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
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

}  // namespace

cudaError_t launch_logprobs(LogprobsArgs a, int sms, bool pdl, cudaStream_t stream) {
    const int per = 16 / type_bytes(a.dtype);
    const int64_t windows = (int64_t(a.vocab) + 2 * per - 2) / per;  // the most a row can have
    int cluster = 1;
    while (cluster < kMaxCluster && 2 * cluster * a.rows <= 2 * sms && windows > 64 * cluster) cluster *= 2;
    const int64_t mine = (windows + cluster - 1) / cluster;
    int threads = 64;
    while (threads < 256 && threads * kFly < mine) threads *= 2;
    // Fewer where that still fills the SMs (1024 threads each, at 64 registers): what a row costs besides its numbers, the
    // waits of one row, then goes beside more rows' reading (4096 rows bf16, 8 top tokens: of 10000 logits 64 us with 256
    // threads and 36 with 64, of 32003 95 and, with 128, 78).  Not below two threads for each of a thread's windows, or
    // more threads have several windows of interest (128000 logits: 201 us with 256 threads, 243 with 64).
    while (threads > 64 && a.rows * cluster * (threads / 2) * 5 >= int64_t(sms) * 1024 * 4 && mine <= threads / 2 * (threads / 4))
        threads /= 2;
    a.cluster = cluster;
    const bool entropy = a.entropy != nullptr, top = a.top > 0;
    const void *fn = a.dtype == CF_BF16   ? forward_kernel<CF_BF16>(entropy, top)
                     : a.dtype == CF_FP16 ? forward_kernel<CF_FP16>(entropy, top)
                                          : forward_kernel<CF_FP32>(entropy, top);
    void *args[] = {&a};
    return launch(fn, unsigned(a.rows * cluster), threads, cluster, pdl, stream, args);
}

// turns of kFly windows that a thread of the gradient takes: few where there are few CTAs, else up to eight
static int grad_turns(int64_t rows, int64_t windows) {
    int turns = 1;
    while (turns < 8 && rows * ((windows + 2 * turns * kFly * kGradThreads - 1) / (2 * turns * kFly * kGradThreads)) >= 1216)
        turns *= 2;
    return turns;
}
static int64_t grad_windows(int64_t vocab, int dtype) {
    const int per = 16 / type_bytes(dtype);
    return (vocab + 2 * per - 2) / per;  // the most a row can have
}

int64_t logprobs_grad_ctas(int64_t rows, int64_t vocab, int dtype) {
    const int64_t windows = grad_windows(vocab, dtype), each = int64_t(grad_turns(rows, windows)) * kFly * kGradThreads;
    return rows * ((windows + each - 1) / each);
}

cudaError_t launch_logprobs_grad(LogprobsGradArgs a, bool pdl, cudaStream_t stream) {
    const int64_t ctas = logprobs_grad_ctas(a.rows, a.vocab, a.dtype);
    a.chunks = int(ctas / a.rows);
    a.turns = grad_turns(a.rows, grad_windows(a.vocab, a.dtype));
    const bool entropy = a.dentropy != nullptr;
    const void *fn = a.dtype == CF_BF16   ? grad_kernel<CF_BF16>(entropy)
                     : a.dtype == CF_FP16 ? grad_kernel<CF_FP16>(entropy)
                                          : grad_kernel<CF_FP32>(entropy);
    void *args[] = {&a};
    return launch(fn, unsigned(ctas), kGradThreads, 1, pdl, stream, args);
}

}  // namespace cf
