// Arguments and output steps shared by the attention kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kv_device.cuh"
#include "quant_device.cuh"
#include "tc_device.cuh"

namespace fp8l {

struct AttnParams {
    const uint16_t *q;
    int tokens;
    int64_t q_stride;
    int q_heads, kv_heads;
    const uint8_t *k_cache, *v_cache;
    const float *k_scale, *v_scale;
    int num_pages, page_shift;
    const int32_t *block_table;
    int table_width;
    const int32_t *q_offsets, *kv_lens;
    int requests;
    float score_scale;  // sm_scale * log2(e)
    int window;
    const float *out_scale;
    void *out;
    int out_dtype;
    float *lse;
    int stages;
    float *partials;
    unsigned *counters, *status;
    long long wait_cycles;
    unsigned stall;
};

namespace {

constexpr float kLn2 = 0.693147180559945309f;

// VALS consecutive outputs of a row from dimension d on
template <int VALS>
__device__ __forceinline__ void attn_store(const AttnParams &p, int token, int head, int dim, int d,
                                           const float (&o)[VALS]) {
    const int64_t at = (static_cast<int64_t>(token) * p.q_heads + head) * dim + d;
    if (p.out_dtype == FP8L_E4M3) {
        const float s = p.out_scale[0];
        uint8_t *y = static_cast<uint8_t *>(p.out) + at;
        if constexpr (VALS < 4) {
#pragma unroll
            for (int i = 0; i < VALS; ++i) y[i] = code_of(o[i], s);
        } else {
            const Quot d = Quot::make<FP8L_F32>(s);
            uint32_t c[VALS / 4];
#pragma unroll
            for (int i = 0; i < VALS / 4; ++i)
                c[i] = codes_of_word<FP8L_F32, true>(
                           make_uint4(__float_as_uint(o[4 * i]), __float_as_uint(o[4 * i + 1]),
                                      __float_as_uint(o[4 * i + 2]), __float_as_uint(o[4 * i + 3])), d).x;
            if constexpr (VALS % 16 == 0) {
#pragma unroll
                for (int i = 0; i < VALS / 4; i += 4)
                    *reinterpret_cast<uint4 *>(y + 4 * i) = make_uint4(c[i], c[i + 1], c[i + 2], c[i + 3]);
            } else {
#pragma unroll
                for (int i = 0; i < VALS / 4; ++i) *reinterpret_cast<uint32_t *>(y + 4 * i) = c[i];
            }
        }
    } else {
        uint16_t *y = static_cast<uint16_t *>(p.out) + at;
        if constexpr (VALS == 1) {
            *y = static_cast<uint16_t>(pack_out16(o[0], o[0], p.out_dtype) & 0xFFFFu);
        } else {
            uint32_t w[VALS / 2];
#pragma unroll
            for (int i = 0; i < VALS / 2; ++i) w[i] = pack_out16(o[2 * i], o[2 * i + 1], p.out_dtype);
            if constexpr (VALS == 2) {
                *reinterpret_cast<uint32_t *>(y) = w[0];
            } else if constexpr (VALS == 4) {
                *reinterpret_cast<uint2 *>(y) = make_uint2(w[0], w[1]);
            } else {
#pragma unroll
                for (int i = 0; i < VALS / 2; i += 4)
                    *reinterpret_cast<uint4 *>(y + 2 * i) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
            }
        }
    }
}

// lse from the reference m (base 2) and the sum l = sum 2^(s - m)
__device__ __forceinline__ void attn_store_lse(const AttnParams &p, int token, int head, float m, float l) {
    p.lse[static_cast<int64_t>(token) * p.q_heads + head] = l > 0.0f ? (m + log2f(l)) * kLn2 : -INFINITY;
}

}  // namespace
}  // namespace fp8l
