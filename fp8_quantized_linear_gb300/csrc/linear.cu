// Entry points of the linear products with a fused epilogue: W8A8
// (fp8_linear) and W8A16 (fp8_w8a16_linear).
//
// ("[Kernel][FP8] Initial support with dynamic per-tensor scaling" and
// "Marlin fp8": the products themselves, which replace nn.Linear with its
// bias; "RFC: FP8 Quantization Schema in vLLM": an E4M3 result through
// output_scale.)
#include <cuda_fp8.h>

#include "common.cuh"
#include "epilogue.cuh"

namespace fp8l {
namespace {

struct SimpleArgs {
    const void *x;
    const uint8_t *w;
    int M, N, K;
    int packed;
    const float *a_scale;
    int a_per_token;
    const float *w_scale;
    int w_per_channel;
    int gated;
    Epilogue e;
};

__device__ __forceinline__ float e4m3_value(uint8_t c) {
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E4M3)));
}

template <int XDT>
__device__ __forceinline__ float x_value(const void *x, size_t i) {
    if constexpr (XDT == FP8L_E4M3) return e4m3_value(static_cast<const uint8_t *>(x)[i]);
    if constexpr (XDT == FP8L_BF16) return __bfloat162float(static_cast<const __nv_bfloat16 *>(x)[i]);
    return __half2float(static_cast<const __half *>(x)[i]);
}

__device__ __forceinline__ size_t packed_at(int n, int k, int K) {
    const int chunks = (K + 63) / 64, c = k / 64, t = (k & 63) / 16, j = k & 15;
    return (static_cast<size_t>(n / 16) * chunks + c) * 1024 + ((n >> 3) & 1) * 512 +
           ((n & 7) * 4 + t) * 16 + j;
}

// 16 x 16 outputs per block, 16 k at a time through shared memory.
template <int XDT>
__global__ void __launch_bounds__(256) linear_simple_kernel(const SimpleArgs p) {
    __shared__ float xs[16][17], ws[2][16][17];
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int m = blockIdx.y * 16 + ty, n = blockIdx.x * 16 + tx;
    const int wrow = blockIdx.x * 16 + ty;
    float acc0 = 0.0f, acc1 = 0.0f;
    for (int k0 = 0; k0 < p.K; k0 += 16) {
        xs[ty][tx] = m < p.M ? x_value<XDT>(p.x, static_cast<size_t>(m) * p.K + k0 + tx) : 0.0f;
        for (int g = 0; g <= p.gated; ++g) {
            const int row = wrow + g * p.e.width;
            const size_t at = p.packed ? packed_at(row, k0 + tx, p.K)
                                       : static_cast<size_t>(row) * p.K + k0 + tx;
            ws[g][ty][tx] = e4m3_value(p.w[at]);
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            acc0 = fmaf(xs[ty][k], ws[0][tx][k], acc0);
            if (p.gated) acc1 = fmaf(xs[ty][k], ws[1][tx][k], acc1);
        }
        __syncthreads();
    }
    if (m >= p.M) return;
    const float sa = p.a_scale == nullptr ? 1.0f : epi_ld_f32(p.a_scale + (p.a_per_token ? m : 0));
    auto scaled = [&](float acc, int row) {
        return acc * (sa * epi_ld_f32(p.w_scale + (p.w_per_channel ? row : 0))) + epi_bias(p.e, row);
    };
    float v[1] = {scaled(acc0, n)};
    activate(v, p.e.act);
    if (p.gated) v[0] *= scaled(acc1, n + p.e.width);
    const size_t o = static_cast<size_t>(m) * p.e.width + n;
    if (p.e.residual != nullptr) v[0] += epi_ld_16(p.e.residual, o, p.e.out_dtype);
    if (p.e.out_dtype == FP8L_F16)
        static_cast<__half *>(p.e.y)[o] = __float2half_rn(v[0]);
    else if (p.e.out_dtype == FP8L_BF16)
        static_cast<__nv_bfloat16 *>(p.e.y)[o] = __float2bfloat16_rn(v[0]);
    else
        static_cast<uint8_t *>(p.e.y)[o] = static_cast<uint8_t>(__nv_cvt_float_to_fp8(
            __fdiv_rn(v[0], epi_ld_f32(p.e.out_scale)), __NV_SATFINITE, __NV_E4M3));
}

template <int XDT>
int launch_simple(const SimpleArgs &p, cudaStream_t stream) {
    const int blocks_m = (p.M + 15) / 16;
    if (blocks_m > 65535) return FP8L_ESHAPE;
    linear_simple_kernel<XDT><<<dim3(p.e.width / 16, blocks_m), 256, 0, stream>>>(p);
    return launch_status();
}

bool misaligned(const void *p, unsigned bytes) {
    return (reinterpret_cast<uintptr_t>(p) & (bytes - 1u)) != 0;
}

// Whether [p, p + n) and [q, q + m) share a byte (null ranges share none).
bool overlap(const void *p, size_t n, const void *q, size_t m) {
    if (p == nullptr || q == nullptr || n == 0 || m == 0) return false;
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    return a < b + m && b < a + n;
}

// The arguments both products share, checked; fills the epilogue.
int check_epilogue(int64_t M, int64_t N, int64_t K, const void *bias, int bias_dtype, int activation,
                   const void *residual, const float *out_scale, void *y, int out_dtype, Epilogue *e,
                   int *gated) {
    const int act = activation & ~FP8L_ACT_GATED;
    if (act < FP8L_ACT_NONE || act > FP8L_ACT_GELU_TANH) return FP8L_EINVAL;
    *gated = (activation & FP8L_ACT_GATED) != 0 ? 1 : 0;
    if (bias != nullptr && bias_dtype != FP8L_F16 && bias_dtype != FP8L_BF16 && bias_dtype != FP8L_F32)
        return FP8L_EINVAL;
    if (residual != nullptr && out_dtype == FP8L_E4M3) return FP8L_EINVAL;
    if (M < 0 || M > 0x7FFFFFFF || N <= 0 || K <= 0 || N > (1 << 20) || K > (1 << 20) ||
        N % (*gated ? 32 : 16) != 0 || K % 16 != 0)
        return FP8L_ESHAPE;
    if (M > 0 && y == nullptr) return FP8L_EINVAL;
    if (misaligned(bias, bias_dtype == FP8L_F32 ? 4 : 2) ||
        (M > 0 && (!aligned16(y) || !aligned16(residual))))
        return FP8L_EALIGN;
    e->bias = bias;
    e->bias_dtype = bias_dtype;
    e->act = act;
    e->residual = residual;
    e->out_scale = out_scale;
    e->y = y;
    e->out_dtype = out_dtype;
    e->width = static_cast<int>(*gated ? N / 2 : N);
    return FP8L_OK;
}

// The output may be the residual itself (added in place) but shares no byte
// with anything else that is read.
int check_output(const Epilogue &e, int64_t M, int64_t N, const void *x, size_t x_bytes, const void *w,
                 size_t w_bytes, const float *a_scale, size_t a_scales, const float *w_scale,
                 size_t w_scales) {
    const size_t elems = static_cast<size_t>(M) * static_cast<size_t>(e.width);
    const size_t bytes = elems * (e.out_dtype == FP8L_E4M3 ? 1 : 2);
    if (overlap(e.y, bytes, x, x_bytes) || overlap(e.y, bytes, w, w_bytes) ||
        overlap(e.y, bytes, a_scale, 4 * a_scales) || overlap(e.y, bytes, w_scale, 4 * w_scales) ||
        overlap(e.y, bytes, e.bias, static_cast<size_t>(N) * (e.bias_dtype == FP8L_F32 ? 4 : 2)) ||
        (e.out_dtype == FP8L_E4M3 && overlap(e.y, bytes, e.out_scale, 4)) ||
        (e.residual != e.y && overlap(e.y, bytes, e.residual, 2 * elems)))
        return FP8L_EINVAL;
    return FP8L_OK;
}

}  // namespace
}  // namespace fp8l

extern "C" int fp8_linear(const uint8_t *a, const uint8_t *w, int64_t M, int64_t N, int64_t K,
                          const float *a_scale, const float *w_scale, int w_per_channel,
                          const void *bias, int bias_dtype, int activation, const void *residual,
                          const float *out_scale, void *y, int out_dtype, void *workspace,
                          unsigned flags, void *stream) {
    using namespace fp8l;
    if (out_dtype != FP8L_F16 && out_dtype != FP8L_BF16 && out_dtype != FP8L_E4M3) return FP8L_EINVAL;
    if ((flags & ~(FP8L_WEIGHTS_STABLE | FP8L_A_PER_TOKEN | FP8L_KERNEL_MASK)) != 0u) return FP8L_EINVAL;
    if (a_scale == nullptr || w_scale == nullptr || workspace == nullptr || w == nullptr)
        return FP8L_EINVAL;
    if (out_dtype == FP8L_E4M3 && out_scale == nullptr) return FP8L_EINVAL;
    SimpleArgs p{};
    int st = check_epilogue(M, N, K, bias, bias_dtype, activation, residual, out_scale, y, out_dtype,
                            &p.e, &p.gated);
    if (st != FP8L_OK) return st;
    if (M > 0 && a == nullptr) return FP8L_EINVAL;
    if (!aligned16(w) || !aligned16(workspace) || (M > 0 && !aligned16(a)) || misaligned(a_scale, 4) ||
        misaligned(w_scale, 4) || (out_dtype == FP8L_E4M3 && misaligned(out_scale, 4)))
        return FP8L_EALIGN;
    const int pt = (flags & FP8L_A_PER_TOKEN) != 0u ? 1 : 0, pc = w_per_channel ? 1 : 0;
    st = check_output(p.e, M, N, a, static_cast<size_t>(M) * K, w, static_cast<size_t>(N) * K, a_scale,
                      pt ? M : 1, w_scale, pc ? N : 1);
    if (st != FP8L_OK) return st;
    if (bias == nullptr && activation == FP8L_ACT_NONE && residual == nullptr)
        return fp8_scaled_mm(a, w, M, N, K, a_scale, w_scale, w_per_channel, out_scale, y, out_dtype,
                             workspace, flags, stream);
    st = check_device(nullptr);
    if (st != FP8L_OK) return st;
    if (M == 0) return FP8L_OK;
    p.x = a;
    p.w = w;
    p.M = static_cast<int>(M);
    p.N = static_cast<int>(N);
    p.K = static_cast<int>(K);
    p.a_scale = a_scale;
    p.a_per_token = pt;
    p.w_scale = w_scale;
    p.w_per_channel = pc;
    return launch_simple<FP8L_E4M3>(p, as_stream(stream));
}

extern "C" int fp8_w8a16_linear(const void *x, int x_dtype, const uint8_t *w, const float *w_scale,
                                int64_t M, int64_t N, int64_t K, const void *bias, int bias_dtype,
                                int activation, const void *residual, void *y, unsigned flags,
                                void *stream) {
    using namespace fp8l;
    if (x_dtype != FP8L_F16 && x_dtype != FP8L_BF16) return FP8L_EINVAL;
    if ((flags & ~(FP8L_WEIGHTS_STABLE | FP8L_WEIGHTS_PACKED | FP8L_KERNEL_MASK)) != 0u)
        return FP8L_EINVAL;
    if (w == nullptr || w_scale == nullptr) return FP8L_EINVAL;
    SimpleArgs p{};
    int st = check_epilogue(M, N, K, bias, bias_dtype, activation, residual, nullptr, y, x_dtype, &p.e,
                            &p.gated);
    if (st != FP8L_OK) return st;
    if (M > 0 && x == nullptr) return FP8L_EINVAL;
    if (!aligned16(w) || (M > 0 && !aligned16(x)) || misaligned(w_scale, 4)) return FP8L_EALIGN;
    p.packed = (flags & FP8L_WEIGHTS_PACKED) != 0u ? 1 : 0;
    st = check_output(p.e, M, N, x, static_cast<size_t>(M) * K * 2, w,
                      p.packed ? fp8_packed_weight_bytes(N, K) : static_cast<size_t>(N) * K, nullptr, 0,
                      w_scale, N);
    if (st != FP8L_OK) return st;
    if (bias == nullptr && activation == FP8L_ACT_NONE && residual == nullptr)
        return fp8_w8a16_mm(x, x_dtype, w, w_scale, M, N, K, y, flags, stream);
    st = check_device(nullptr);
    if (st != FP8L_OK) return st;
    if (M == 0) return FP8L_OK;
    p.x = x;
    p.w = w;
    p.M = static_cast<int>(M);
    p.N = static_cast<int>(N);
    p.K = static_cast<int>(K);
    p.w_scale = w_scale;
    p.w_per_channel = 1;
    return x_dtype == FP8L_BF16 ? launch_simple<FP8L_BF16>(p, as_stream(stream))
                                : launch_simple<FP8L_F16>(p, as_stream(stream));
}
