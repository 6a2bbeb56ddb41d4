// Epilogue of the linear products (fp8_linear, fp8_w8a16_linear): bias,
// activation (plain or gated), residual addition and the output cast, on
// float32 sums in registers.
//
//   z = acc * scale + bias(n)
//   plain   t[n] = act(z[n])
//   gated   t[n] = act(z[n]) * z[N/2 + n]      (gate rows first, then up rows)
//   y = cast(t + residual)
//
// Everything is float32 and rounded once, by the output cast.  The logistic
// forms are written as z / (1 + e^-u): no cancellation for negative z, and an
// overflowing exponential gives the right limit 0.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"

namespace fp8l {

// What a product's epilogue does (kernel argument).
struct Epilogue {
    const void *bias;      // [N] of bias_dtype, or null
    int bias_dtype;        // FP8L_F16, FP8L_BF16 or FP8L_F32
    int act;               // FP8L_ACT_* without the gate bit
    const void *residual;  // [M, width] of the output's 16-bit type, or null
    const float *out_scale;
    void *y;  // [M, width]
    int out_dtype;
    int width;  // columns of y: N, or N / 2 when gated
};

namespace {

__device__ __forceinline__ float silu_of(float z) { return __fdividef(z, 1.0f + __expf(-z)); }

// z Phi(z) = max(z, 0) - |z| h(|z|), h(a) = erfc(a / sqrt 2) / 2: no
// cancellation for negative z.  h(a) = e^(-a^2 / 2) t R(t), t = 1 / (1 + 0.36
// a), which maps a >= 0 to (0, 1] and gives the right decay 1 / a; R is the
// polynomial of degree 6 with the least largest relative error over 0 <= a <=
// 14, fitted by reweighted least squares: 9e-7, below the exponential's own
// error.  (erfcf in its place cost 20 to 30 % of a product with K = 4096: 1024
// x 28672 112 us against 80 without an activation; this form takes 97.)
// The tail's argument stops at z = 20, where it is zero beside z: of an
// infinite z it would be infinity times 0.  (Minus infinity and NaN stay: NaN,
// the formula's infinity times 0.)
__device__ __forceinline__ float gelu_of(float z) {
    float a;
    asm("min.NaN.f32 %0, %1, 0f41A00000;" : "=f"(a) : "f"(z));
    a = fabsf(a);
    const float t = __fdividef(1.0f, fmaf(0.36f, a, 1.0f));
    float r = 0.047059460972601275f;
    r = fmaf(r, t, -0.1797755885232244f);
    r = fmaf(r, t, 0.18096890501073565f);
    r = fmaf(r, t, 0.02653901863037719f);
    r = fmaf(r, t, 0.13972304963865187f);
    r = fmaf(r, t, 0.14177175868564995f);
    r = fmaf(r, t, 0.14371309497733017f);
    const float e = __expf(-0.5f * a * a);
    return fmaf(-a * e, t * r, fmaxf(z, 0.0f));
}

// z (1 + tanh u) / 2 with u = sqrt(2 / pi) (z + 0.044715 z^3) is z times the
// logistic function of 2 u
__device__ __forceinline__ float gelu_tanh_of(float z) {
    const float u2 = z * fmaf(z * z, 0.07135481282970f, 1.59576912160573f);
    return __fdividef(z, 1.0f + __expf(-u2));
}

// COUNT values through the activation; one branch for all of them
template <int COUNT>
__device__ __forceinline__ void activate(float (&v)[COUNT], int act) {
    if (act == FP8L_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < COUNT; ++i) v[i] = silu_of(v[i]);
    } else if (act == FP8L_ACT_GELU_TANH) {
#pragma unroll
        for (int i = 0; i < COUNT; ++i) v[i] = gelu_tanh_of(v[i]);
    } else if (act == FP8L_ACT_GELU) {
#pragma unroll
        for (int i = 0; i < COUNT; ++i) v[i] = gelu_of(v[i]);
    } else if (act == FP8L_ACT_RELU) {
#pragma unroll
        for (int i = 0; i < COUNT; ++i) v[i] = v[i] < 0.0f ? 0.0f : v[i];
    }
}

// Codes of t / out_scale: t times the rounded reciprocal (2^-23 of t off the
// quotient at most, where t itself carries the product's float32 rounding),
// the division itself where the reciprocal leaves the normal range.  (The
// correctly rounded quotient of fp8_scaled_mm takes eight instructions for
// this one: 0.5 us of a tile's epilogue.)
struct OutScale {
    float os, inv;
    __device__ __forceinline__ static OutScale make(float os) {
        const bool plain = os >= 0x1p-120f && os <= 0x1p120f;
        return OutScale{os, plain ? __frcp_rn(os) : 0.0f};
    }
    __device__ __forceinline__ float of(float t) const { return inv != 0.0f ? t * inv : __fdiv_rn(t, os); }
    // four codes, the first in the low byte
    __device__ __forceinline__ uint32_t codes(float a, float b, float c, float d) const {
        return static_cast<uint32_t>(
                   __nv_cvt_float2_to_fp8x2(make_float2(of(a), of(b)), __NV_SATFINITE, __NV_E4M3)) |
               (static_cast<uint32_t>(
                    __nv_cvt_float2_to_fp8x2(make_float2(of(c), of(d)), __NV_SATFINITE, __NV_E4M3))
                << 16);
    }
};

// Loads of what the preceding kernel on the stream may have written:
// coherent, and kept after griddepcontrol.wait.
__device__ __forceinline__ float epi_ld_f32(const float *p) {
    float v;
    asm volatile("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(p) : "memory");
    return v;
}

__device__ __forceinline__ float epi_ld_16(const void *p, int64_t i, int dtype) {
    unsigned short u;
    asm volatile("ld.global.u16 %0, [%1];"
                 : "=h"(u)
                 : "l"(static_cast<const unsigned short *>(p) + i)
                 : "memory");
    return dtype == FP8L_BF16 ? __uint_as_float(static_cast<uint32_t>(u) << 16)
                              : __half2float(__ushort_as_half(u));
}

// a pair of 16-bit values (the first in the low half)
__device__ __forceinline__ float2 widen_pair(uint32_t w, int dtype) {
    if (dtype == FP8L_BF16)
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}

__device__ __forceinline__ float epi_bias(const Epilogue &e, int64_t n) {
    if (e.bias == nullptr) return 0.0f;
    return e.bias_dtype == FP8L_F32 ? epi_ld_f32(static_cast<const float *>(e.bias) + n)
                                    : epi_ld_16(e.bias, n, e.bias_dtype);
}

}  // namespace
}  // namespace fp8l
