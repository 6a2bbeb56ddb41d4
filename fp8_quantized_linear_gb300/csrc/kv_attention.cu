// Causal attention over the paged FP8 cache (fp8_kv_attention).
//
//   s_j = sm_scale q . k_j,   out = sum_j exp(s_j) v_j / sum_j exp(s_j)
//
// One block per (token, query head): tiles of 128 keys, one key per thread
// for the scores, one dimension per thread for the weighted values, with the
// running maximum m and sum l of the softmax carried from tile to tile
// (a larger maximum rescales l and the accumulator by exp(m_old - m_new)).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kv_device.cuh"
#include "quant_device.cuh"
#include "tc_device.cuh"

namespace fp8l {
namespace {

constexpr int kAttThreads = 128;

struct AttnParams {
    const uint16_t *q;
    int tokens;
    int64_t q_stride;
    int q_heads, kv_heads, dim;
    const uint8_t *k_cache, *v_cache;
    const float *k_scale, *v_scale;
    int num_pages, page_shift;
    const int32_t *block_table;
    int table_width;
    const int32_t *q_offsets, *kv_lens;
    int requests;
    float sm_scale;
    int window;
    const float *out_scale;
    void *out;
    int q_dtype, out_dtype;
    float *lse;
};

__device__ __forceinline__ float e4m3_value(uint8_t c) {
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E4M3)));
}

__global__ void __launch_bounds__(kAttThreads) kv_attention_kernel(const AttnParams p) {
    __shared__ float qs[128], ws[kAttThreads], red[8];
    grid_dependency_sync();
    const int t = static_cast<int>(blockIdx.x) / p.q_heads, h = static_cast<int>(blockIdx.x) % p.q_heads;
    if (t < p.q_offsets[0] || t >= p.q_offsets[p.requests]) return;
    int lo = 0, hi = p.requests;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.q_offsets[mid] <= t)
            lo = mid;
        else
            hi = mid;
    }
    const int r = lo, tid = static_cast<int>(threadIdx.x);
    const int last = p.kv_lens[r] - (p.q_offsets[r + 1] - t);
    const int first = p.window > 0 ? max(0, last - p.window + 1) : 0;
    const int g = h / (p.q_heads / p.kv_heads);
    const int P = 1 << p.page_shift;
    if (tid < p.dim) {
        const uint16_t raw = p.q[static_cast<int64_t>(t) * p.q_stride + h * p.dim + tid];
        qs[tid] = (p.q_dtype == FP8L_BF16 ? __uint_as_float(static_cast<uint32_t>(raw) << 16)
                                          : __half2float(__ushort_as_half(raw))) * p.sm_scale;
    }
    float m = -INFINITY, l = 0.0f, acc = 0.0f;
    __syncthreads();
    for (int j0 = first & ~(kAttThreads - 1); j0 <= last; j0 += kAttThreads) {
        const int j = j0 + tid;
        float s = -INFINITY;
        int64_t ph = 0;
        if (j >= first && j <= last) {
            const int page = min(max(p.block_table[static_cast<int64_t>(r) * p.table_width + (j >> p.page_shift)], 0),
                                 p.num_pages - 1);
            ph = static_cast<int64_t>(page) * p.kv_heads + g;
            float dot = 0.0f;
            for (int c = 0; c < p.dim / 16; ++c) {
                const uint4 u = *reinterpret_cast<const uint4 *>(
                    p.k_cache + kv_chunk_offset(ph, P, p.dim, j & (P - 1), c));
                const uint8_t *b = reinterpret_cast<const uint8_t *>(&u);
#pragma unroll
                for (int i = 0; i < 16; ++i) dot = fmaf(qs[16 * c + i], e4m3_value(b[i]), dot);
            }
            s = dot * p.k_scale[ph];
        }
        float mt = s;
        for (int o = 16; o > 0; o >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xFFFFFFFFu, mt, o));
        if ((tid & 31) == 0) red[tid >> 5] = mt;
        __syncthreads();
        mt = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
        const float mn = fmaxf(m, mt);
        const float keep = m == -INFINITY ? 0.0f : expf(m - mn);
        const float w = s == -INFINITY ? 0.0f : expf(s - mn);
        ws[tid] = w;
        float sum = w;
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        if ((tid & 31) == 0) red[4 + (tid >> 5)] = sum;
        __syncthreads();
        l = l * keep + ((red[4] + red[5]) + (red[6] + red[7]));
        acc *= keep;
        m = mn;
        if (tid < p.dim) {
            for (int i = max(first - j0, 0); i < min(kAttThreads, last + 1 - j0); ++i) {
                const int k = j0 + i;
                const int page = min(max(p.block_table[static_cast<int64_t>(r) * p.table_width + (k >> p.page_shift)], 0),
                                     p.num_pages - 1);
                const int64_t vh = static_cast<int64_t>(page) * p.kv_heads + g;
                const uint8_t c = p.v_cache[kv_chunk_offset(vh, P, p.dim, k & (P - 1), tid >> 4) + (tid & 15)];
                acc = fmaf(ws[i] * p.v_scale[vh], e4m3_value(c), acc);
            }
        }
        __syncthreads();
    }
    const float o = l > 0.0f ? acc / l : 0.0f;
    const int64_t at = (static_cast<int64_t>(t) * p.q_heads + h);
    if (tid < p.dim) {
        if (p.out_dtype == FP8L_E4M3)
            static_cast<uint8_t *>(p.out)[at * p.dim + tid] = code_of(o, p.out_scale[0]);
        else
            static_cast<uint16_t *>(p.out)[at * p.dim + tid] =
                static_cast<uint16_t>(pack_out16(o, o, p.out_dtype) & 0xFFFFu);
    }
    if (tid == 0 && p.lse != nullptr) p.lse[at] = l > 0.0f ? m + logf(l) : -INFINITY;
}

constexpr size_t kAttnZeroBytes = 4096;
constexpr size_t kAttnWorkspaceBytes = 4096;

}  // namespace
}  // namespace fp8l

extern "C" {

size_t fp8_kv_attention_workspace_bytes(void) { return fp8l::kAttnWorkspaceBytes; }
size_t fp8_kv_attention_workspace_zero_bytes(void) { return fp8l::kAttnZeroBytes; }

int fp8_kv_attention(const void *q, int q_dtype, int64_t tokens, int64_t q_stride, int64_t q_heads,
                     int64_t kv_heads, int64_t head_dim, const uint8_t *k_cache, const uint8_t *v_cache,
                     const float *k_scale, const float *v_scale, int64_t num_pages, int64_t page_size,
                     const int32_t *block_table, int64_t table_width, const int32_t *q_offsets,
                     const int32_t *kv_lens, int64_t requests, int64_t max_q_len, float sm_scale,
                     int64_t window, const float *out_scale, void *out, int out_dtype, float *lse,
                     void *workspace, void *stream) {
    using namespace fp8l;
    if ((q_dtype != FP8L_F16 && q_dtype != FP8L_BF16) || (out_dtype != q_dtype && out_dtype != FP8L_E4M3) ||
        !(sm_scale > 0.0f) || sm_scale > 3.0e38f)
        return FP8L_EINVAL;
    if (tokens < 0 || tokens > INT32_MAX || (head_dim != 64 && head_dim != 128) || kv_heads < 1 ||
        q_heads < kv_heads || q_heads % kv_heads != 0 || q_heads * head_dim > (1 << 20) ||
        q_stride < q_heads * head_dim || q_stride % 8 != 0 || !kv_page_size_ok(page_size) || num_pages < 1 ||
        num_pages > INT32_MAX / page_size || table_width < 1 || table_width > INT32_MAX || requests < 1 ||
        requests > kKvMaxRequests || max_q_len < 0 || window < 0)
        return FP8L_ESHAPE;
    if (!k_cache || !v_cache || !k_scale || !v_scale || !block_table || !q_offsets || !kv_lens || !workspace ||
        (out_dtype == FP8L_E4M3 && !out_scale) || (tokens > 0 && (!q || !out)))
        return FP8L_EINVAL;
    if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) ||
        !aligned16(workspace) || !aligned4(k_scale) || !aligned4(v_scale) || !aligned4(block_table) ||
        !aligned4(q_offsets) || !aligned4(kv_lens) || !aligned4(out_scale) || !aligned4(lse))
        return FP8L_EALIGN;
    int sms = 0;
    if (int st = check_device(&sms); st != FP8L_OK) return st;
    if (tokens == 0 || max_q_len == 0) return FP8L_OK;
    if (tokens * q_heads > INT32_MAX) return FP8L_ESHAPE;
    AttnParams p;
    p.q = static_cast<const uint16_t *>(q);
    p.tokens = static_cast<int>(tokens);
    p.q_stride = q_stride;
    p.q_heads = static_cast<int>(q_heads);
    p.kv_heads = static_cast<int>(kv_heads);
    p.dim = static_cast<int>(head_dim);
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.num_pages = static_cast<int>(num_pages);
    p.page_shift = __builtin_ctzll(static_cast<unsigned long long>(page_size));
    p.block_table = block_table;
    p.table_width = static_cast<int>(table_width);
    p.q_offsets = q_offsets;
    p.kv_lens = kv_lens;
    p.requests = static_cast<int>(requests);
    p.sm_scale = sm_scale;
    p.window = static_cast<int>(window < INT32_MAX ? window : 0);
    p.out_scale = out_scale;
    p.out = out;
    p.q_dtype = q_dtype;
    p.out_dtype = out_dtype;
    p.lse = lse;
    return launch_dependent(kv_attention_kernel, dim3(static_cast<unsigned>(tokens * q_heads)), kAttThreads, 0,
                            as_stream(stream), p);
}

}  // extern "C"
