// pieces.cuh -- rows of 16-bit or 32-bit numbers in pieces of 8, as the row kernels hold them in registers.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/cf.h"
#include "ptx.cuh"

namespace cf {

constexpr __host__ __device__ int type_bytes(int dt) { return dt == CF_FP32 ? 4 : 2; }

template <int kDt>
struct Element {
    using type = uint16_t;
};
template <>
struct Element<CF_FP32> {
    using type = float;
};

template <int kDt>
__device__ __forceinline__ float to_float(typename Element<kDt>::type v) {
    if constexpr (kDt == CF_FP32) return v;
    else if constexpr (kDt == CF_FP16) return __half2float(__ushort_as_half(v));
    else return __uint_as_float(uint32_t(v) << 16);
}
template <int kDt>
__device__ __forceinline__ typename Element<kDt>::type from_float(float v) {
    if constexpr (kDt == CF_FP32) return v;
    else if constexpr (kDt == CF_FP16) return __half_as_ushort(__float2half_rn(v));
    else return __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

// Two fp32 numbers, worked on by one instruction.
struct Two {
    float2 v;
    __device__ __forceinline__ Two() {}
    __device__ __forceinline__ explicit Two(float2 p) : v(p) {}
    __device__ __forceinline__ Two(float lo, float hi) : v(make_float2(lo, hi)) {}
    __device__ __forceinline__ explicit Two(float both) : v(make_float2(both, both)) {}
    __device__ __forceinline__ float2 parts() const { return v; }
    __device__ __forceinline__ float sum() const { return v.x + v.y; }
};
__device__ __forceinline__ Two fma(Two a, Two b, Two c) { return Two(__ffma2_rn(a.v, b.v, c.v)); }
__device__ __forceinline__ Two operator*(Two a, Two b) { return Two(__fmul2_rn(a.v, b.v)); }
__device__ __forceinline__ Two operator+(Two a, Two b) { return Two(__fadd2_rn(a.v, b.v)); }

// eight numbers, as stored
template <int kDt>
struct Piece {
    static constexpr int kWords = kDt == CF_FP32 ? 8 : 4;
    uint32_t w[kWords];

    // what was worked out from the words before is worked out again behind this
    __device__ __forceinline__ void pin() {
#pragma unroll
        for (int i = 0; i < kWords; ++i) asm volatile("" : "+r"(w[i]));
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0u;
    }
    __device__ __forceinline__ float get(int j) const {
        if constexpr (kDt == CF_FP32) return __uint_as_float(w[j]);
        else if constexpr (kDt == CF_FP16) return __half2float(__ushort_as_half(uint16_t(w[j / 2] >> (j % 2 * 16))));
        else return __uint_as_float(j % 2 ? w[j / 2] & 0xffff0000u : w[j / 2] << 16);
    }
    __device__ __forceinline__ void unpack(Two (&x)[4]) const {
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = Two(get(2 * j), get(2 * j + 1));
    }
    __device__ __forceinline__ void pack(const Two (&x)[4]) {
        float f[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 p = x[j].parts();
            f[2 * j] = p.x, f[2 * j + 1] = p.y;
        }
        pack(f);
    }
    __device__ __forceinline__ void pack(const float (&x)[8]) {
#pragma unroll
        for (int j = 0; j < 8; j += (kDt == CF_FP32 ? 1 : 2)) {
            if constexpr (kDt == CF_FP32) {
                w[j] = __float_as_uint(x[j]);
            } else if constexpr (kDt == CF_FP16) {
                const __half2 h = __floats2half2_rn(x[j], x[j + 1]);
                w[j / 2] = *reinterpret_cast<const uint32_t *>(&h);
            } else {
                w[j / 2] = ptx::pack_bf16x2(x[j], x[j + 1]);
            }
        }
    }
    // from and to 16-byte aligned memory
    __device__ __forceinline__ void load(const void *p) {
#pragma unroll
        for (int i = 0; i < kWords / 4; ++i) {
            const uint4 v = __ldcs(reinterpret_cast<const uint4 *>(p) + i);
            w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
        }
    }
    __device__ __forceinline__ void store(void *p) const {
#pragma unroll
        for (int i = 0; i < kWords / 4; ++i)
            reinterpret_cast<uint4 *>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    }
    __device__ __forceinline__ void put(int j, typename Element<kDt>::type v) {
        if constexpr (kDt == CF_FP32) w[j] = __float_as_uint(v);
        else w[j / 2] |= uint32_t(v) << (j % 2 * 16);  // of a zeroed piece
    }
};

}  // namespace cf
