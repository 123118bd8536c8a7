// activations.cuh -- the activation nodes of the products' epilogues and their slopes.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "pieces.cuh"
#include "ptx.cuh"

namespace cf {

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

// SiLU is z * p with p = 1 / (1 + exp(-z)); its slope p (1 + z (1 - p)).  (From |z| = 88 on exp(-z) is infinite or zero,
// and so p; an infinite z times p = 0 would be a NaN where the limit is 0.)
__device__ __forceinline__ float silu_p(float z) { return __fdividef(1.f, 1.f + ptx::ex2_approx(-1.4426950408889634f * z)); }
__device__ __forceinline__ float silu(float z) { return z < -120.f ? 0.f : z * silu_p(z); }
// act (cf_activation) of every value of an array, floats or their bits; one branch for all of them
__device__ __forceinline__ float as_float(float v) { return v; }
__device__ __forceinline__ float as_float(uint32_t v) { return __uint_as_float(v); }
__device__ __forceinline__ void set_float(float &v, float x) { v = x; }
__device__ __forceinline__ void set_float(uint32_t &v, float x) { v = __float_as_uint(x); }
template <class T, int n>
__device__ __forceinline__ void activate(T (&v)[n], int act) {
    if (act == 1) {
#pragma unroll
        for (int j = 0; j < n; ++j) set_float(v[j], gelu(as_float(v[j])));
    } else if (act == 2) {
#pragma unroll
        for (int j = 0; j < n; ++j) set_float(v[j], silu(as_float(v[j])));
    } else if (act == 3) {  // (a NaN stays one)
#pragma unroll
        for (int j = 0; j < n; ++j) set_float(v[j], as_float(v[j]) < 0.f ? 0.f : as_float(v[j]));
    }
}
// x * act'(z), pair by pair, z no larger than slope_end(act) in size (beyond it the slope is 0 or 1 to fp32, and the
// products below would leave fp32's range).
// GELU: with p = 1 / (1 + exp(-2u)), z p (1 - p) 2 u' + p.  (One by one, with the clamp in fp32, the slopes bound the
// kernel: 8192 x 8192 bf16 75 us.)
__device__ __forceinline__ float slope_end(int act) { return act == 1 ? 12.f : 120.f; }
__device__ __forceinline__ Two times_slope(Two x, Two z, int act) {
    if (act == 3) {  // the slope at 0 is 0; a NaN stays one
        const float2 a = x.parts(), v = z.parts();
        return Two(a.x * (v.x > 0.f ? 1.f : (v.x == v.x ? 0.f : v.x)), a.y * (v.y > 0.f ? 1.f : (v.y == v.y ? 0.f : v.y)));
    }
    Two u, du;  // the exponent, to the base 2; 2 u'
    if (act == 1) {
        const Two z2 = z * z;
        u = z * fma(z2, Two(-2.885390081777927f * 0.7978845608028654f * 0.044715f), Two(-2.885390081777927f * 0.7978845608028654f));
        du = fma(z2, Two(2.f * 0.7978845608028654f * 0.134145f), Two(2.f * 0.7978845608028654f));
    } else {
        u = z * Two(-1.4426950408889634f);
        du = Two(1.f);
    }
    const float2 e = u.parts();
    const Two p(__fdividef(1.f, 1.f + ptx::ex2_approx(e.x)), __fdividef(1.f, 1.f + ptx::ex2_approx(e.y)));
    const Two t = z * p;
    return x * fma(fma(Two(-1.f) * t, p, t), du, p);
}

}  // namespace cf
