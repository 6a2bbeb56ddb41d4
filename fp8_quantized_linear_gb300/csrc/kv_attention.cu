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

#include <atomic>

#include "kv_attention_decode.cuh"
#include "kv_attention_params.cuh"

namespace fp8l {
namespace {

constexpr int kAttThreads = 128;

__device__ __forceinline__ float e4m3_value(uint8_t c) {
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E4M3)));
}

template <int QDT, int DIM>
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
    if (tid < DIM) {
        const uint16_t raw = p.q[static_cast<int64_t>(t) * p.q_stride + h * DIM + tid];
        qs[tid] = (QDT == FP8L_BF16 ? __uint_as_float(static_cast<uint32_t>(raw) << 16)
                                          : __half2float(__ushort_as_half(raw))) * p.score_scale;
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
            for (int c = 0; c < DIM / 16; ++c) {
                const uint4 u = *reinterpret_cast<const uint4 *>(
                    p.k_cache + kv_chunk_offset(ph, P, DIM, j & (P - 1), c));
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
        const float keep = m == -INFINITY ? 0.0f : exp2f(m - mn);
        const float w = s == -INFINITY ? 0.0f : exp2f(s - mn);
        ws[tid] = w;
        float sum = w;
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        if ((tid & 31) == 0) red[4 + (tid >> 5)] = sum;
        __syncthreads();
        l = l * keep + ((red[4] + red[5]) + (red[6] + red[7]));
        acc *= keep;
        m = mn;
        if (tid < DIM) {
            for (int i = max(first - j0, 0); i < min(kAttThreads, last + 1 - j0); ++i) {
                const int k = j0 + i;
                const int page = min(max(p.block_table[static_cast<int64_t>(r) * p.table_width + (k >> p.page_shift)], 0),
                                     p.num_pages - 1);
                const int64_t vh = static_cast<int64_t>(page) * p.kv_heads + g;
                const uint8_t c = p.v_cache[kv_chunk_offset(vh, P, DIM, k & (P - 1), tid >> 4) + (tid & 15)];
                acc = fmaf(ws[i] * p.v_scale[vh], e4m3_value(c), acc);
            }
        }
        __syncthreads();
    }
    const float o = l > 0.0f ? acc / l : 0.0f;
    const float x[1] = {o};
    if (tid < DIM) attn_store<1>(p, t, h, DIM, tid, x);
    if (tid == 0 && p.lse != nullptr) attn_store_lse(p, t, h, m, l);
}

// Workspace: status word, merge counters (zero between calls), partials
constexpr size_t kAttnCountersOffset = 64;
constexpr size_t kAttnZeroBytes = 2048;
constexpr int kDecMaxRows = 16;
constexpr size_t kAttnWorkspaceBytes =
    kAttnZeroBytes + sizeof(float) * 2 * kDecMaxCtas * kDecMaxRows * (128 + 2);
static_assert(kAttnCountersOffset + 4 * kDecMaxCtas <= kAttnZeroBytes, "counters fit");

constexpr int kDecSmemPerCta = 113 * 1024 - 512;  // two CTAs per SM

template <int QDT, int DIM, int ROWS>
int launch_decode(AttnParams p, int sms, cudaStream_t stream) {
    using Sm = DecSmem<QDT, DIM, ROWS>;
    int stages = (kDecSmemPerCta - Sm::kFixedBytes) / Sm::kStageBytes;
    stages = stages < kDecMaxStages ? stages : kDecMaxStages;
    p.stages = stages;
    const int smem = stages * Sm::kStageBytes + Sm::kFixedBytes;
    auto kernel = kv_attention_decode_kernel<QDT, DIM, ROWS>;
    static std::atomic<unsigned> ready{0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return FP8L_ECUDA;
    if (!(ready.load(std::memory_order_acquire) >> dev & 1u)) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess ||
            cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, 100) != cudaSuccess)
            return FP8L_ECUDA;
        ready.fetch_or(1u << dev, std::memory_order_release);
    }
    const int ctas = 2 * sms < kDecMaxCtas ? 2 * sms : kDecMaxCtas;
    return launch_dependent(kernel, dim3(static_cast<unsigned>(ctas)), kDecThreads, smem, stream, p);
}

template <int QDT, int DIM>
int launch_attention(const AttnParams &p, int64_t rows, int sms, cudaStream_t stream) {
    if (rows <= 8) return launch_decode<QDT, DIM, 8>(p, sms, stream);
    if (rows <= 16) return launch_decode<QDT, DIM, 16>(p, sms, stream);
    return launch_dependent(kv_attention_kernel<QDT, DIM>, dim3(static_cast<unsigned>(p.tokens) * p.q_heads),
                            kAttThreads, 0, stream, p);
}

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
    p.score_scale = sm_scale * 1.44269504088896341f;
    p.window = static_cast<int>(window < INT32_MAX ? window : 0);
    p.out_scale = out_scale;
    p.out = out;
    p.out_dtype = out_dtype;
    p.lse = lse;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    p.status = status_word(workspace);
    p.counters = reinterpret_cast<unsigned *>(ws + kAttnCountersOffset);
    p.partials = reinterpret_cast<float *>(ws + kAttnZeroBytes);
    const WaitConfig waits = wait_config();
    p.wait_cycles = waits.cycles;
    p.stall = waits.stall;
    p.stages = 0;
    // query rows of one request and kv head at most
    const int64_t rows = (max_q_len < tokens ? max_q_len : tokens) * (q_heads / kv_heads);
    const cudaStream_t s = as_stream(stream);
    if (q_dtype == FP8L_BF16)
        return head_dim == 128 ? launch_attention<FP8L_BF16, 128>(p, rows, sms, s)
                               : launch_attention<FP8L_BF16, 64>(p, rows, sms, s);
    return head_dim == 128 ? launch_attention<FP8L_F16, 128>(p, rows, sms, s)
                           : launch_attention<FP8L_F16, 64>(p, rows, sms, s);
}

}  // extern "C"
