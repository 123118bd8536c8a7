// linear_grad.cu -- what the gradient of a dense layer needs beside its two products:
//     dZ = dY * act'(Z)      the gradient behind the activation, 16 bits
//     sums = sum over the rows of dZ  (fp32, of the unrounded values): the gradient of the bias
//
// HBM bounds it: dY and Z are read once and dZ is written once.  A CTA takes a strip of 256 columns (a warp's lane 8
// of them, a 16-byte piece) and a chunk of the rows, a warp every eighth row and four of them in flight; the warps' sums
// meet in shared memory, the chunks' in the workspace, where the last CTA of a strip to arrive adds them in order, so
// that equal calls give equal bits.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "activations.cuh"
#include "grouped_internal.h"
#include "ptx.cuh"

namespace cf {
namespace {

constexpr int kWarps = 8, kFly = 4;

template <bool kFp16>
__device__ __forceinline__ void unpack8(float (&x)[8], uint4 v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (kFp16) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
            x[2 * i] = f.x, x[2 * i + 1] = f.y;
        } else {
            x[2 * i] = __uint_as_float(w[i] << 16), x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
}
template <bool kFp16>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (kFp16) {
            const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        } else {
            w[i] = ptx::pack_bf16x2(x[2 * i], x[2 * i + 1]);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <bool kFp16>
__global__ void __launch_bounds__(kWarps * 32) linear_sums_kernel(const LinearSumsArgs a) {
    __shared__ float part[kWarps][kLinearStrip];
    __shared__ uint32_t last;
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int strip = int(blockIdx.x % unsigned(a.strips)), chunk = int(blockIdx.x / unsigned(a.strips));
    const int c = strip * kLinearStrip + lane * 8;
    const bool live = c < a.cols;  // cols is a multiple of 8
    const int64_t r1 = min(a.rows, (chunk + 1) * a.rows_per_chunk);
    float sum[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) sum[j] = 0.f;
    const uint16_t *dy = static_cast<const uint16_t *>(a.dy), *z = static_cast<const uint16_t *>(a.z);
#pragma unroll 1
    for (int64_t r = chunk * a.rows_per_chunk + warp; live && r < r1; r += kFly * kWarps) {
        uint4 g[kFly], p[kFly];
#pragma unroll
        for (int i = 0; i < kFly; ++i) {
            const bool in = r + i * kWarps < r1;
            const size_t at = size_t(r + i * kWarps) * a.cols + c;
            g[i] = in ? *reinterpret_cast<const uint4 *>(dy + at) : make_uint4(0u, 0u, 0u, 0u);
            p[i] = in && z ? *reinterpret_cast<const uint4 *>(z + at) : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int i = 0; i < kFly; ++i) {
            float x[8], y[8];
            unpack8<kFp16>(x, g[i]);
            if (z) {
                unpack8<kFp16>(y, p[i]);
                times_slope(x, y, a.act);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) sum[j] += x[j];
            if (a.dz && r + i * kWarps < r1)
                *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.dz) + size_t(r + i * kWarps) * a.cols + c) =
                    pack8<kFp16>(x);
        }
    }
    if (!a.sums) return;
#pragma unroll
    for (int j = 0; j < 8; ++j) part[warp][lane * 8 + j] = sum[j];
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
