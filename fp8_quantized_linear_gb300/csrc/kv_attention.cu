// Causal attention over the paged FP8 cache (fp8_kv_attention).
//
// Few query rows per request and kv head go to the decode kernel
// (kv_attention_decode.cuh), more to the prompt kernel
// (kv_attention_prompt.cuh); this file checks the arguments and chooses.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kv_attention_decode.cuh"
#include "kv_attention_params.cuh"
#include "kv_attention_prompt.cuh"

namespace fp8l {
namespace {

// Workspace: status word, merge counters (zero between calls), partials
constexpr size_t kAttnCountersOffset = 64;
constexpr size_t kAttnZeroBytes = 16384;
constexpr size_t kDecPartials = static_cast<size_t>(2) * kDecMaxCtas * 16 * (128 + 2);  // or half the CTAs, 32 rows
constexpr size_t kProPartials = static_cast<size_t>(2) * kProMaxCtas * kProRows * (128 + 2);
constexpr size_t kAttnWorkspaceBytes =
    kAttnZeroBytes + sizeof(float) * (kDecPartials > kProPartials ? kDecPartials : kProPartials);
// decode: per merge level, two pieces of a CTA, two softmax groups (four of half the CTAs)
static_assert(kAttnCountersOffset + 4 * kDecLevels * 2 * 2 * kDecMaxCtas <= kAttnZeroBytes &&
                  kAttnCountersOffset + 4 * kProLevels * 2 * 2 * kProMaxCtas <= kAttnZeroBytes,
              "counters fit");

constexpr int kSmemPerSm = 227 * 1024;  // what the CTAs of an SM can ask for, each with 1 KB of its own

template <int QDT, int DIM, int GROUPS, int WPARTS>
int launch_decode(AttnParams p, int sms, cudaStream_t stream) {
    using Sh = DecShape<QDT, DIM, GROUPS, WPARTS>;
    constexpr int kBudget = kSmemPerSm / Sh::kCtasPerSm - 1024;
    constexpr int kFit = (kBudget - Sh::kFixedBytes) / Sh::kStageBytes;
    static_assert(kFit >= 2, "two stages at least");
    p.stages = kFit < kDecMaxStages ? kFit : kDecMaxStages;
    const int smem = p.stages * Sh::kStageBytes + Sh::kFixedBytes;
    static std::atomic<unsigned long long> ready{0};
    auto kernel = kv_attention_decode_kernel<QDT, DIM, GROUPS, WPARTS>;
    if (int st = allow_smem(kernel, smem, ready, true); st != FP8L_OK) return st;
    const int most = kDecMaxCtas / 2 * Sh::kCtasPerSm, ctas = Sh::kCtasPerSm * sms;
    return launch_dependent(kernel, dim3(static_cast<unsigned>(ctas < most ? ctas : most)), Sh::kThreads, smem, stream,
                            p);
}

template <int QDT, int DIM>
int launch_prompt(const AttnParams &p, int sms, cudaStream_t stream) {
    constexpr int smem = ProSmem<QDT, DIM>::kBytes;
    static std::atomic<unsigned long long> ready{0};
    auto kernel = kv_attention_prompt_kernel<QDT, DIM>;
    if (int st = allow_smem(kernel, smem, ready, true); st != FP8L_OK) return st;
    return launch_dependent(kernel, dim3(static_cast<unsigned>(sms < kProMaxCtas ? sms : kProMaxCtas)), kProThreads,
                            smem, stream, p);
}

// The kernel for the most rows a request has per kv head.  A group of eight rows
// more than needed costs time, and the prompt kernel's halves of 128 rows pay
// from 33 rows, where a row tile of the decode kernel would read the keys twice.
// One request above 32 rows takes all to the prompt kernel: 64 decoding (8 rows)
// beside a chunk of 512 tokens 267 us, 90 + 43 apart.
// Measured over 64 sequences of 0.1-8k keys, 8 kv heads of 128:
//   8 rows: 88 us with one group, 99 with two;   16: 106 with two, 145 with four;
//   20 rows: 153 us, 244 with the prompt kernel;  32: 160 against 238.
//
// Outputs in codes: a value near a code's border shows the weights' rounding,
// which a 16-bit output's own covers.  Of 262144 codes over the same sequences 96
// differ from the 64-bit value's with 12-bit weights, 4 with 16 bits (13 with
// 32-bit weights and no other rounding).  Up to eight rows the fourth part's columns
// are there anyway and cost 1 % (88.3 -> 89.2 us; 2.5 % at D = 64); with 16 rows 2.5 %,
// with 32 4.5 %, and there the three parts stay.
template <int QDT, int DIM>
int launch_attention(const AttnParams &p, int64_t rows, int sms, cudaStream_t stream) {
    if (rows <= 8)
        return p.out_dtype == FP8L_E4M3 ? launch_decode<QDT, DIM, 1, 4>(p, sms, stream)
                                        : launch_decode<QDT, DIM, 1, 3>(p, sms, stream);
    if (rows <= 16) return launch_decode<QDT, DIM, 2, 3>(p, sms, stream);
    if (rows <= 32) return launch_decode<QDT, DIM, 4, 3>(p, sms, stream);
    return launch_prompt<QDT, DIM>(p, sms, stream);
}

}  // namespace
}  // namespace fp8l

extern "C" {

size_t fp8_kv_attention_workspace_bytes(void) { return fp8l::kAttnWorkspaceBytes; }
size_t fp8_kv_attention_workspace_zero_bytes(void) { return fp8l::kAttnZeroBytes; }

int fp8l_capture_id(void *stream, unsigned long long *id) {
    if (id == nullptr) return FP8L_EINVAL;
    *id = 0;
    if (stream == nullptr) return FP8L_OK;
    cudaStreamCaptureStatus status = cudaStreamCaptureStatusNone;
    unsigned long long capture = 0;
    if (cudaStreamGetCaptureInfo(fp8l::as_stream(stream), &status, &capture) != cudaSuccess)
        return fp8l::cuda_failed();
    if (status == cudaStreamCaptureStatusActive) *id = capture;
    return FP8L_OK;
}

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
        q_heads < kv_heads || q_heads > (1 << 20) || q_heads % kv_heads != 0 || q_heads * head_dim > (1 << 20) ||
        tokens * q_heads > INT32_MAX - kProRows || q_stride < q_heads * head_dim || q_stride % 8 != 0 || !kv_page_size_ok(page_size) || num_pages < 1 ||
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
    // a window that holds every key the table can is none (and negative positions
    // less a window stay in 32 bits)
    p.window = static_cast<int>(window <= INT32_MAX - tokens && window < table_width * page_size ? window : 0);
    p.out_scale = out_scale;
    p.out = out;
    p.out_dtype = out_dtype;
    p.lse = lse;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    p.status = status_word(workspace);
    if (library_status_word(&p.library_status) != FP8L_OK) return cuda_failed();
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
