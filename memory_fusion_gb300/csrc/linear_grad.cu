// linear_grad.cu -- what the gradient of a dense layer needs beside its two products:
//     dZ = dY * act'(Z)      the gradient behind the activation, 16 bits
//     sums = sum over the rows of dZ  (fp32, of the unrounded values): the gradient of the bias
// dZ is rounded because the two products' tensor cores take 16 bits of it: dX and dW are then about sqrt(2) times as far
// from the exact ones as their own rounding puts them (bf16 0.00235 of their size against 0.00166, fp16 0.00029 against
// 0.00021).  Its rest in a second pair of products would take that away and double their time.
//
// HBM bounds it: dY and Z are read once and dZ is written once.  A CTA takes a strip of 256 columns (a warp's lane 8
// of them, a 16-byte piece) and a chunk of the rows, a warp every eighth row and four of them in flight; the warps' sums
// meet in shared memory, the chunks' in the workspace, where the last CTA of a strip to arrive adds them in order, so
// that equal calls give equal bits.  8192 x 8192 bf16, GELU': 69 to 76 us (5.3 to 5.8 TB/s, DRAM 65 % busy; 0.58
// instructions a cycle and scheduler, most of them the slope's), with its two products of 2048 x 8192 407 to 415 us.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "activations.cuh"
#include "grouped_internal.h"
#include "pieces.cuh"
#include "ptx.cuh"

namespace cf {
namespace {

constexpr int kWarps = 8, kFly = 4;

// numbers of 16 bits kept within +-end (a word of two); NaNs stay
template <bool kFp16>
__device__ __forceinline__ uint32_t within(uint32_t v, uint32_t end) {
    uint32_t r;
    if constexpr (kFp16) {
        asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(end));
        asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(r), "r"(end ^ 0x80008000u));
    } else {
        asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(end));
        asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(r), "r"(end ^ 0x80008000u));
    }
    return r;
}

template <bool kFp16>
__global__ void __launch_bounds__(kWarps * 32, 4) linear_sums_kernel(const LinearSumsArgs a) {
    __shared__ float part[kWarps][kLinearStrip];
    __shared__ uint32_t last;
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int strip = int(blockIdx.x % unsigned(a.strips)), chunk = int(blockIdx.x / unsigned(a.strips));
    const int c = strip * kLinearStrip + lane * 8;
    const bool live = c < a.cols;  // cols is a multiple of 8
    const int64_t r1 = min(a.rows, (chunk + 1) * a.rows_per_chunk);
    constexpr int kDt = kFp16 ? CF_FP16 : CF_BF16;
    using P = Piece<kDt>;
    Two sum[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) sum[j] = Two(0.f);
    const uint32_t end16 = from_float<kDt>(slope_end(a.act)), end = end16 | end16 << 16;
    const uint16_t *dy = static_cast<const uint16_t *>(a.dy), *z = static_cast<const uint16_t *>(a.z);
#pragma unroll 1
    for (int64_t r = chunk * a.rows_per_chunk + warp; live && r < r1; r += kFly * kWarps) {
        P g[kFly], p[kFly];
#pragma unroll
        for (int i = 0; i < kFly; ++i) {
            const size_t at = size_t(r + i * kWarps) * a.cols + c;
            g[i].zero();
            p[i].zero();
            if (r + i * kWarps < r1) {
                g[i].load(dy + at);
                if (z) p[i].load(z + at);
            }
        }
#pragma unroll
        for (int i = 0; i < kFly; ++i) {
            Two x[4], y[4];
            g[i].unpack(x);
            if (z) {
                if (a.act != 3) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) p[i].w[j] = within<kFp16>(p[i].w[j], end);
                }
                p[i].unpack(y);
#pragma unroll
                for (int j = 0; j < 4; ++j) x[j] = times_slope(x[j], y[j], a.act);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) sum[j] = sum[j] + x[j];
            if (a.dz && r + i * kWarps < r1) {
                g[i].pack(x);
                g[i].store(static_cast<uint16_t *>(a.dz) + size_t(r + i * kWarps) * a.cols + c);
            }
        }
    }
    if (!a.sums) return;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 v = sum[j].parts();
        part[warp][lane * 8 + 2 * j] = v.x, part[warp][lane * 8 + 2 * j + 1] = v.y;
    }
    __syncthreads();
    const int col = strip * kLinearStrip + int(threadIdx.x);
    float total = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) total += part[w][threadIdx.x];
    if (a.chunks == 1) {
        if (col < a.cols) a.sums[col] = total;
        return;
    }
    if (col < a.cols) __stcg(a.partials + size_t(chunk) * a.cols + col, total);
    __syncthreads();  // thread 0's release covers what the others wrote before it, its acquire what they read after
    if (threadIdx.x == 0) {
        last = ptx::atom_add_acq_rel_gpu(a.counters + strip, 1u) == uint32_t(a.chunks - 1);
        if (last) ptx::st_relaxed_gpu(a.counters + strip, 0u);  // for the next launch
    }
    __syncthreads();
    if (last == 0u || col >= a.cols) return;
    total = 0.f;
    for (int k = 0; k < a.chunks; k += 8) {
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            x[i] = k + i < a.chunks ? __ldcg(a.partials + size_t(k + i) * a.cols + col) : 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) total += x[i];
    }
    a.sums[col] = total;
}

}  // namespace

void plan_linear_sums(int64_t rows, int64_t cols, int sms, LinearSumsArgs *a) {
    a->rows = rows;
    a->cols = int(cols);
    a->strips = int((cols + kLinearStrip - 1) / kLinearStrip);
    // four CTAs an SM; a chunk of one turn of the loop at least
    int64_t chunks = std::max<int64_t>(1, int64_t(4) * sms / a->strips);
    chunks = std::min<int64_t>(chunks, (rows + kFly * kWarps - 1) / (kFly * kWarps));
    chunks = std::max<int64_t>(chunks, 1);
    a->rows_per_chunk = std::max<int64_t>(1, (rows + chunks - 1) / chunks);
    a->chunks = int(std::max<int64_t>(1, (rows + a->rows_per_chunk - 1) / a->rows_per_chunk));
}

cudaError_t launch_linear_sums(const LinearSumsArgs &a, bool pdl, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(a.strips) * unsigned(a.chunks));
    cfg.blockDim = dim3(kWarps * 32);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return a.fp16 ? cudaLaunchKernelEx(&cfg, linear_sums_kernel<true>, a)
                  : cudaLaunchKernelEx(&cfg, linear_sums_kernel<false>, a);
}

}  // namespace cf
