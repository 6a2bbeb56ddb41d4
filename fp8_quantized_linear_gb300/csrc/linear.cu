// Entry points of the linear products with a fused epilogue: W8A8
// (fp8_linear) and W8A16 (fp8_w8a16_linear).
//
// ("[Kernel][FP8] Initial support with dynamic per-tensor scaling" and
// "Marlin fp8": the products themselves, which replace nn.Linear with its
// bias; "RFC: FP8 Quantization Schema in vLLM": an E4M3 result through
// output_scale.)
#include "linear_launch.cuh"

namespace fp8l {
namespace {

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

// The kernel of fp8_linear (times of each product alone in a replayed graph
// over rotating operands, us):
//   - weights streamed through registers for a few tokens and small weights,
//     whose time is the start of the kernel (M = 1 at 4096 x 4096 5.1 against
//     7.4 swapped, M = 8 at 8192 x 4096 9.5 against 9.9; but M = 8 at 5120 x
//     8192 12.5 against 11.1, M = 1 at 6144 x 6144 gated 11.7 against 10.6, M =
//     16 at 6144 x 4096 11.3 against 9.5); up to 4096 weight rows all CTAs run
//     at once and it pays for longer (M = 8 at 4096 x 11008 10.6 against 11.6);
//     a CTA reads its rows whole, so not where they are long (M = 8 at 2048 x
//     22016 15.4 against 12.9, x 12288 9.4 against 9.8; M = 16 at 1024 x 8192
//     9.0 against 6.7, x 4096 4.4 against 5.7);
//   - swapped operands up to 128 tokens, and beyond while tokens x weight rows
//     stay below 2^20, too few 256 x 256 tiles for the SM pairs (M = 256 at
//     4096 x 4096 13.5 against 14.3 tiled, M = 192 at 11008 x 4096 21.3 against
//     17.6, M = 128 at 28672 x 4096 31.1 against 32.7);
//   - swapped operands, too, where the 256 x 256 tiles begin a second round
//     over the pairs and two CTAs an SM hold all 128 x 128 tiles (M = 333 at
//     11008 x 4096 22.9 against 26.9 tiled, at 12288 x 12288 53 against 70; M =
//     400, a second wave, 39.6 against 27.3), if rows of K fill their 128-byte
//     lines (K = 4112 33.4 against 29.4: each box row takes two lines, and
//     smaller tiles load more of them);
//   - tiles over SM pairs otherwise.
unsigned choose_linear(int64_t M, int64_t N, int64_t K, int sms) {
    const int64_t wbytes = N * K, few = int64_t(N <= 4096 ? 48 : 32) << 20;
    if (M <= 8 ? wbytes <= few && K < 16384 : M <= 16 && wbytes <= (int64_t(16) << 20) && K <= 4096)
        return FP8L_KERNEL_STREAM;
    if (M <= 128 || M * N <= (1 << 20)) return FP8L_KERNEL_SWAPPED;
    const int64_t pair_tiles = ((M + 255) / 256) * ((N + 255) / 256);
    const int64_t swapped_tiles = ((M + 127) / 128) * ((N + 127) / 128);
    return K % 128 == 0 && pair_tiles > sms / 2 && swapped_tiles <= 2 * int64_t(sms) ? FP8L_KERNEL_SWAPPED
                                                                                      : FP8L_KERNEL_TILED;
}

// The kernel of fp8_w8a16_linear: weights streamed through registers for a few
// tokens (M = 1 at 12288 x 4096, packed, 11.2 us against 13.1 swapped), up to 8
// for any weights, since it takes the tokens whole (at most 8 % are lost by
// that: M = 5 at 28672 x 8192 42.3 us against 42.3, M = 8 45.4 against 42.3), up
// to 16 where it is the faster one (4096 x 4096 6.8 against 9.5, 2048 x 6144 8.0
// against 9.2, but 2048 x 12288 13.4 against 11.7), else tokens in parts through
// the swapped-operand kernel (M = 16 at 4096 x 11008 14.0 against 14.1 to 18.2,
// at 22016 x 4096 gated 20.6 against 25.0; M = 32 at 4096 x 11008 15.7 against
// 26.6).
unsigned choose_w8a16_linear(int64_t M, int64_t N, int64_t K, unsigned flags) {
    const unsigned k = flags & FP8L_KERNEL_MASK;
    if (k != FP8L_KERNEL_AUTO) return k;
    return M <= 8 || (M <= 16 && N * K <= (int64_t(32) << 20) && K <= 8192) ? FP8L_KERNEL_STREAM
                                                                            : FP8L_KERNEL_SWAPPED;
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
    const int pt = (flags & FP8L_A_PER_TOKEN) != 0u ? 1 : 0, pc = w_per_channel ? 1 : 0;
    if ((a_scale == nullptr && !(pt && M == 0)) || w_scale == nullptr || w == nullptr) return FP8L_EINVAL;
    if (out_dtype == FP8L_E4M3 && out_scale == nullptr) return FP8L_EINVAL;
    LinearCall c{};
    int st = check_epilogue(M, N, K, bias, bias_dtype, activation, residual, out_scale, y, out_dtype,
                            &c.e, &c.gated);
    if (st != FP8L_OK) return st;
    if (M > 0 && a == nullptr) return FP8L_EINVAL;
    if (!aligned16(w) || !aligned16(workspace) || (M > 0 && !aligned16(a)) || misaligned(a_scale, 4) ||
        misaligned(w_scale, 4) || (out_dtype == FP8L_E4M3 && misaligned(out_scale, 4)))
        return FP8L_EALIGN;
    st = check_output(c.e, M, N, a, static_cast<size_t>(M) * K, w, static_cast<size_t>(N) * K, a_scale,
                      pt ? M : 1, w_scale, pc ? N : 1);
    if (st != FP8L_OK) return st;
    if (overlap(y, static_cast<size_t>(M) * c.e.width * (out_dtype == FP8L_E4M3 ? 1 : 2), workspace,
                workspace != nullptr ? kWorkspaceBytes : 0))
        return FP8L_EINVAL;
    st = check_device(&c.sms);
    if (st != FP8L_OK) return st;
    if (M == 0) return FP8L_OK;
    unsigned *status = nullptr;
    if (workspace == nullptr) {  // the library's status word in its place
        if (library_status_word(&status) != FP8L_OK) return FP8L_ECUDA;
        workspace = status;
    }
    const unsigned choice = flags & FP8L_KERNEL_MASK;
    if (choice == FP8L_KERNEL_AUTO && bias == nullptr && activation == FP8L_ACT_NONE && residual == nullptr)
        return fp8_scaled_mm(a, w, M, N, K, a_scale, w_scale, w_per_channel, out_scale, y, out_dtype,
                             workspace, flags, stream);
    c.x = a;
    c.x_dtype = FP8L_E4M3;
    c.w = w;
    c.M = static_cast<int>(M);
    c.N = static_cast<int>(N);
    c.K = static_cast<int>(K);
    c.a_scale = a_scale;
    c.a_per_token = pt;
    c.w_scale = w_scale;
    c.w_per_channel = pc;
    c.status = status_word(workspace);
    c.stable = (flags & FP8L_WEIGHTS_STABLE) != 0u;
    c.stream = as_stream(stream);
    const unsigned kernel = choice != FP8L_KERNEL_AUTO ? choice : choose_linear(M, N, K, c.sms);
    if (kernel == FP8L_KERNEL_STREAM) return launch_linear_stream(c);
    if (kernel == FP8L_KERNEL_TILED) return launch_linear_pair(c);
    return launch_linear_swapped(c, 1, a_scale);
}

extern "C" size_t fp8_w8a16_linear_workspace_bytes(int x_dtype, int64_t M, int64_t N, int64_t K,
                                                   unsigned flags) {
    if (fp8l::choose_w8a16_linear(M, N, K, flags) != FP8L_KERNEL_SWAPPED) return 0;
    if ((x_dtype != FP8L_F16 && x_dtype != FP8L_BF16) || M <= 0 || M > 0x7FFFFFFF || K <= 0 ||
        K > (1 << 20) || K % 16 != 0)
        return 0;
    return fp8l::linear_parts_bytes(x_dtype, M, K);
}

extern "C" int fp8_w8a16_linear(const void *x, int x_dtype, const uint8_t *w, const float *w_scale,
                                int64_t M, int64_t N, int64_t K, const void *bias, int bias_dtype,
                                int activation, const void *residual, void *y, void *workspace,
                                unsigned flags, void *stream) {
    using namespace fp8l;
    if (x_dtype != FP8L_F16 && x_dtype != FP8L_BF16) return FP8L_EINVAL;
    if ((flags & ~(FP8L_WEIGHTS_STABLE | FP8L_WEIGHTS_PACKED | FP8L_KERNEL_MASK)) != 0u)
        return FP8L_EINVAL;
    const unsigned kernel = choose_w8a16_linear(M, N, K, flags);
    if (kernel == FP8L_KERNEL_TILED) return FP8L_EINVAL;
    if (w == nullptr || w_scale == nullptr) return FP8L_EINVAL;
    LinearCall c{};
    int st = check_epilogue(M, N, K, bias, bias_dtype, activation, residual, nullptr, y, x_dtype, &c.e,
                            &c.gated);
    if (st != FP8L_OK) return st;
    // what the kernels' grids and tensor maps count, before the tokens are split
    if (kernel == FP8L_KERNEL_STREAM ? M > kLinearStreamTokens : M > 0 && !linear_parts_fit(x_dtype, M, N))
        return FP8L_ESHAPE;
    if (M > 0 && x == nullptr) return FP8L_EINVAL;
    if (!aligned16(w) || (M > 0 && !aligned16(x)) || misaligned(w_scale, 4)) return FP8L_EALIGN;
    c.packed = (flags & FP8L_WEIGHTS_PACKED) != 0u ? 1 : 0;
    st = check_output(c.e, M, N, x, static_cast<size_t>(M) * K * 2, w,
                      c.packed ? fp8_packed_weight_bytes(N, K) : static_cast<size_t>(N) * K, nullptr, 0,
                      w_scale, N);
    if (st != FP8L_OK) return st;
    // (beyond, its other kernels take longer than the parts: 64 bf16 tokens of
    // 11008 x 4096 27 us for 18, 128 85 for 23, 64 fp16 ones 18 for 21)
    if ((flags & FP8L_KERNEL_MASK) == FP8L_KERNEL_AUTO && bias == nullptr &&
        activation == FP8L_ACT_NONE && residual == nullptr && M <= (x_dtype == FP8L_F16 ? 64 : 16))
        return fp8_w8a16_mm(x, x_dtype, w, w_scale, M, N, K, y, flags, stream);
    const size_t scratch = M > 0 ? fp8_w8a16_linear_workspace_bytes(x_dtype, M, N, K, flags) : 0;
    if (scratch > 0 && workspace == nullptr) return FP8L_EINVAL;
    if (!aligned16(workspace)) return FP8L_EALIGN;
    const size_t w_bytes = c.packed ? fp8_packed_weight_bytes(N, K) : static_cast<size_t>(N) * K;
    const size_t y_bytes = static_cast<size_t>(M) * static_cast<size_t>(c.e.width) * 2;
    if (overlap(workspace, scratch, x, static_cast<size_t>(M) * K * 2) ||
        overlap(workspace, scratch, w, w_bytes) || overlap(workspace, scratch, y, y_bytes) ||
        overlap(workspace, scratch, residual, y_bytes) || overlap(workspace, scratch, w_scale, 4 * N) ||
        overlap(workspace, scratch, bias, static_cast<size_t>(N) * (bias_dtype == FP8L_F32 ? 4 : 2)))
        return FP8L_EINVAL;
    st = check_device(&c.sms);
    if (st != FP8L_OK) return st;
    if (M == 0) return FP8L_OK;
    c.x = x;
    c.x_dtype = x_dtype;
    c.w = w;
    c.M = static_cast<int>(M);
    c.N = static_cast<int>(N);
    c.K = static_cast<int>(K);
    c.w_scale = w_scale;
    c.w_per_channel = 1;
    c.stable = (flags & FP8L_WEIGHTS_STABLE) != 0u;
    c.stream = as_stream(stream);
    if (kernel == FP8L_KERNEL_STREAM) return launch_linear_stream(c);
    if (library_status_word(&c.status) != FP8L_OK) return FP8L_ECUDA;
    const float *token_scale = nullptr;
    st = linear_split_tokens(c, workspace, &token_scale);
    if (st != FP8L_OK) return st;
    c.x = workspace;
    return launch_linear_swapped(c, linear_parts(x_dtype), token_scale);
}
