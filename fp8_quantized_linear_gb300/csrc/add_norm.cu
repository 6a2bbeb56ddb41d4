// Residual addition, RMS normalization and activation quantization in one
// pass over the residual stream.
//
// "Condition to achieve linear speedup?" (the QQQ issue): the activation
// quantization of a W8A8 layer is fused into the element-wise kernel before
// it, such as RMSNorm; in a decoder layer that kernel also adds the previous
// product's output to the residual stream.  Per row m of x, res [M, K]:
//   t[m,k] = RN16( x[m,k] + res[m,k] )                (the new stream, written)
//   r[m]   = 1 / sqrt( (1/K) sum_k t[m,k]^2 + eps )
//   h[m,k] = RN16( (t[m,k] * r[m]) * gamma[k] )
//   codes  = the E4M3 quantization of h (dynamic per tensor, static, per
//            token, or none), as in fp8_rmsnorm_quant
//
// 7 bytes an element cross HBM (two 16-bit reads, one 16-bit write, one
// code), so the kernels are streams.  A row lives in the registers of its
// threads from the loads to the stores; nothing is staged in shared memory
// and nothing is read twice.  Enough rows are in flight on an SM (2048
// threads of 2 to 8 pending 16-byte loads each) to cover HBM's latency
// without a copy pipeline.
//   add_norm_rows      static, per token, norm only: one row per block (a
//                      warp per row up to 1024 columns, where a block's
//                      barriers would cost more than the row).
//   add_norm_dynamic   one scale for the tensor: blocks persist over their
//                      rows, meet at a grid maximum (cooperative launch, the
//                      workspace's barrier words), then cast.  Rows whose h
//                      fits shared memory are kept there; the others are
//                      read again from the stream just written, newest
//                      first, and normalized with the same operations.
#include <atomic>

#include "quant_device.cuh"
#include "skinny_device.cuh"

namespace fp8l {
namespace {

constexpr int kAddMaxK = 32768;
constexpr int kAddSmemBudget = 200 * 1024;  // of held rows, per SM
constexpr int kAddMaxDevices = 64;

struct AddNormArgs {
    const void *x, *res, *gamma;
    float eps;
    int M, K;
    void *total;
    uint8_t *q;
    float *scale;
    void *h;
    int mode;
    unsigned *epoch, *arrive, *amax, *status, *lib_status;
    int slots;  // dynamic: rows a block holds in shared memory
    long long wait_cycles;
    unsigned stall;
};

// streamed 16 bytes that this kernel reads once (the preceding kernel may
// have written them: coherent)
__device__ __forceinline__ uint4 ld_once16(const void *p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

template <int DT>
__device__ __forceinline__ uint32_t narrow_pair(uint64_t f) {
    const float a = __uint_as_float(static_cast<uint32_t>(f));
    const float b = __uint_as_float(static_cast<uint32_t>(f >> 32));
    if constexpr (DT == FP8L_BF16) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&v);
    } else {
        const __half2 v = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
}

// RN16(x + res), eight elements
template <int DT>
__device__ __forceinline__ uint4 add_word(const uint4 &x, const uint4 &r) {
    return make_uint4(narrow_pair<DT>(f2_add(widen16<DT>(x.x), widen16<DT>(r.x))),
                      narrow_pair<DT>(f2_add(widen16<DT>(x.y), widen16<DT>(r.y))),
                      narrow_pair<DT>(f2_add(widen16<DT>(x.z), widen16<DT>(r.z))),
                      narrow_pair<DT>(f2_add(widen16<DT>(x.w), widen16<DT>(r.w))));
}

// squares (exact in float32) added to a pair of sums
template <int DT>
__device__ __forceinline__ uint64_t add_squares(const uint4 &v, uint64_t acc) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint64_t f = widen16<DT>(w[i]);
        acc = f2_fma(f, f, acc);
    }
    return acc;
}

// RN16((t r) gamma), eight elements
template <int DT>
__device__ __forceinline__ uint4 scaled_word(const uint4 &t, const uint4 &g, uint64_t r2) {
    const uint32_t tw[4] = {t.x, t.y, t.z, t.w}, gw[4] = {g.x, g.y, g.z, g.w};
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        h[i] = narrow_pair<DT>(f2_mul(f2_mul(widen16<DT>(tw[i]), r2), widen16<DT>(gw[i])));
    return make_uint4(h[0], h[1], h[2], h[3]);
}

// Sum and maximum over the WARPS warps that share a row (one warp: shuffles
// only; else one block barrier each, the partials in arrays of their own and
// added in the same order by every thread).
template <int WARPS>
__device__ __forceinline__ float row_sum(float v, float *part) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if constexpr (WARPS > 1) {
        if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
        __syncthreads();
        v = 0.0f;
#pragma unroll
        for (int i = 0; i < WARPS; ++i) v += part[i];
    }
    return v;
}

template <int WARPS>
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t *part) {
    v = __reduce_max_sync(0xFFFFFFFFu, v);
    if constexpr (WARPS > 1) {
        if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
        __syncthreads();
        v = 0;
#pragma unroll
        for (int i = 0; i < WARPS; ++i) v = max(v, part[i]);
    }
    return v;
}

__device__ __forceinline__ uint64_t rms_factor(float ss, int K, float eps) {
    const float r = __frcp_rn(__fsqrt_rn(__fadd_rn(__fdiv_rn(ss, static_cast<float>(K)), eps)));
    return f2_pack(__float_as_uint(r), __float_as_uint(r));
}

__device__ __forceinline__ float pair_sum(uint64_t acc) {
    return __fadd_rn(__uint_as_float(static_cast<uint32_t>(acc)),
                     __uint_as_float(static_cast<uint32_t>(acc >> 32)));
}

// WARPS warps a row, ROWS rows a block (WARPS == 1, or ROWS == 1), NW words
// (of 8 elements) a thread.
template <int DT, int WARPS, int ROWS, int NW>
__global__ void __launch_bounds__(32 * WARPS * ROWS) add_norm_rows(const AddNormArgs a) {
    static_assert(WARPS == 1 || ROWS == 1, "a block is one row, or a warp is");
    __shared__ float fpart[WARPS];
    __shared__ uint32_t upart[WARPS];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    constexpr int kSpan = 32 * WARPS;  // threads of a row
    const int tid = WARPS == 1 ? (threadIdx.x & 31) : threadIdx.x;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * ROWS + (WARPS == 1 ? threadIdx.x >> 5 : 0);
    pdl_wait();
    if (row >= a.M) return;  // a whole warp (ROWS > 1) or no thread
    const int words = a.K / 8;
    const uint4 *x = static_cast<const uint4 *>(a.x) + row * words;
    const uint4 *res = static_cast<const uint4 *>(a.res) + row * words;
    uint4 t[NW], g[NW];
    {
        uint4 xv[NW], rv[NW];
#pragma unroll
        for (int j = 0; j < NW; ++j) {
            const int w = tid + j * kSpan;
            xv[j] = rv[j] = g[j] = make_uint4(0, 0, 0, 0);
            if (w < words) {
                xv[j] = ld_once16(x + w);
                rv[j] = ld_once16(res + w);
            }
        }
#pragma unroll
        for (int j = 0; j < NW; ++j) {
            const int w = tid + j * kSpan;
            if (w < words) g[j] = ld_act16(static_cast<const uint4 *>(a.gamma) + w);
        }
        uint64_t acc = 0;
#pragma unroll
        for (int j = 0; j < NW; ++j) {
            t[j] = add_word<DT>(xv[j], rv[j]);
            acc = add_squares<DT>(t[j], acc);
        }
        // (the stream's stores before the barrier: they drain while it waits)
        uint4 *total = static_cast<uint4 *>(a.total) + row * words;
#pragma unroll
        for (int j = 0; j < NW; ++j) {
            const int w = tid + j * kSpan;
            if (w < words) total[w] = t[j];
        }
        const uint64_t r2 = rms_factor(row_sum<WARPS>(pair_sum(acc), fpart), a.K, a.eps);
#pragma unroll
        for (int j = 0; j < NW; ++j) t[j] = scaled_word<DT>(t[j], g[j], r2);
    }
    if (a.h != nullptr) {
        uint4 *h = static_cast<uint4 *>(a.h) + row * words;
#pragma unroll
        for (int j = 0; j < NW; ++j) {
            const int w = tid + j * kSpan;
            if (w < words) h[w] = t[j];
        }
    }
    if (a.mode == FP8L_NQ_NORM_ONLY) return;
    float s;
    if (a.mode == FP8L_NQ_PER_TOKEN) {
        uint32_t m = 0;  // words beyond the row are zeros
#pragma unroll
        for (int j = 0; j < NW; ++j) m = word_mag_max<DT>(t[j], m);
        s = scale_from_amax(mag_bits_to_float<DT>(row_max<WARPS>(fold_mag<DT>(m), upart)));
        if (tid == 0) a.scale[row] = s;
    } else {
        s = ld_act_f32(a.scale);
    }
    const Quot d = Quot::make<DT>(s);
    uint2 *q = reinterpret_cast<uint2 *>(a.q) + row * words;
    if (a.mode == FP8L_NQ_STATIC) {
#pragma unroll
        for (int j = 0; j < NW; ++j) {
            const int w = tid + j * kSpan;
            if (w < words) q[w] = codes_of_word<DT, true>(t[j], d);
        }
    } else {
#pragma unroll
        for (int j = 0; j < NW; ++j) {
            const int w = tid + j * kSpan;
            if (w < words) q[w] = codes_of_word<DT, false>(t[j], d);
        }
    }
}

template <int DT, int WARPS, int NW>
__global__ void __launch_bounds__(32 * WARPS) add_norm_dynamic(const AddNormArgs a) {
    extern __shared__ __align__(16) uint4 held[];  // [slots][words], h of a block's first rows
    __shared__ float fpart[2][WARPS];
    __shared__ uint32_t red[33];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    constexpr int kSpan = 32 * WARPS;
    const int tid = threadIdx.x, words = a.K / 8;
    const int64_t G = gridDim.x, b = blockIdx.x;
    const unsigned epoch = *reinterpret_cast<volatile unsigned *>(a.epoch), pair = epoch & 1u;
    if (b == 0 && tid == 0) {
        a.arrive[pair ^ 1u] = 0u;
        a.amax[pair ^ 1u] = 0u;
    }
    uint4 g[NW];
#pragma unroll
    for (int j = 0; j < NW; ++j) {
        const int w = tid + j * kSpan;
        g[j] = w < words ? ld_act16(static_cast<const uint4 *>(a.gamma) + w) : make_uint4(0, 0, 0, 0);
    }
    int flip = 0;
    // h of a row of the stream, in place of t; the partials alternate between
    // two arrays, so one barrier a row is enough
    auto normalize = [&](uint4(&t)[NW]) {
        uint64_t acc = 0;
#pragma unroll
        for (int j = 0; j < NW; ++j) acc = add_squares<DT>(t[j], acc);
        const uint64_t r2 = rms_factor(row_sum<WARPS>(pair_sum(acc), fpart[flip]), a.K, a.eps);
        flip ^= 1;
#pragma unroll
        for (int j = 0; j < NW; ++j) t[j] = scaled_word<DT>(t[j], g[j], r2);
    };
    uint32_t m = 0;
    int i = 0;
    for (int64_t row = b; row < a.M; row += G, ++i) {
        const size_t at = static_cast<size_t>(row) * words;
        uint4 xv[NW], t[NW];
#pragma unroll
        for (int j = 0; j < NW; ++j) {
            const int w = tid + j * kSpan;
            xv[j] = t[j] = make_uint4(0, 0, 0, 0);
            if (w < words) {
                xv[j] = ld_once16(static_cast<const uint4 *>(a.x) + at + w);
                t[j] = ld_once16(static_cast<const uint4 *>(a.res) + at + w);
            }
        }
#pragma unroll
        for (int j = 0; j < NW; ++j) {
            const int w = tid + j * kSpan;
            t[j] = add_word<DT>(xv[j], t[j]);
            if (w < words) static_cast<uint4 *>(a.total)[at + w] = t[j];
        }
        normalize(t);
#pragma unroll
        for (int j = 0; j < NW; ++j) {
            const int w = tid + j * kSpan;
            m = word_mag_max<DT>(t[j], m);
            if (w >= words) continue;
            if (a.h != nullptr) static_cast<uint4 *>(a.h)[at + w] = t[j];
            // (each thread reads back only its own words)
            if (i < a.slots) held[static_cast<size_t>(i) * words + w] = t[j];
        }
    }
    const uint32_t bm = block_max_u32(fold_mag<DT>(m), red);
    const unsigned stalled = (a.stall & kStallGrid) != 0u ? 1u : 0u;
    const bool barrier = G > 1 || stalled != 0u;  // a single block has the maximum already
    uint32_t mm = bm;
    if (barrier && !grid_max(a.arrive + pair, a.amax + pair, bm, a.status, &mm,
                             static_cast<unsigned>(G) + stalled, a.wait_cycles)) {
        // (a capture's workspace is read by nobody: the library's word too)
        if (tid == 0) flag_timeout(a.lib_status);
        return;
    }
    const float s = scale_from_amax(mag_bits_to_float<DT>(mm));
    if (b == 0 && tid == 0) {
        *a.scale = s;
        if (barrier) *a.epoch = epoch + 1u;
    }
    const Quot d = Quot::make<DT>(s);
    for (int k = i - 1; k >= 0; --k) {
        const size_t at = static_cast<size_t>(b + G * k) * words;
        uint4 t[NW];
        if (k < a.slots) {
#pragma unroll
            for (int j = 0; j < NW; ++j) {
                const int w = tid + j * kSpan;
                t[j] = w < words ? held[static_cast<size_t>(k) * words + w] : make_uint4(0, 0, 0, 0);
            }
        } else {
            // the stream this thread wrote
#pragma unroll
            for (int j = 0; j < NW; ++j) {
                const int w = tid + j * kSpan;
                t[j] = w < words ? ld_once16(static_cast<const uint4 *>(a.total) + at + w)
                                 : make_uint4(0, 0, 0, 0);
            }
            normalize(t);
        }
#pragma unroll
        for (int j = 0; j < NW; ++j) {
            const int w = tid + j * kSpan;
            if (w < words) reinterpret_cast<uint2 *>(a.q)[at + w] = codes_of_word<DT, false>(t[j], d);
        }
    }
}

__global__ void add_norm_empty_scale(float *scale) { *scale = 1.0f; }

template <int DT, int WARPS, int ROWS, int NW>
int launch_rows(const AddNormArgs &a, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((int64_t(a.M) + ROWS - 1) / ROWS), 1, 1);
    cfg.blockDim = dim3(32 * WARPS * ROWS, 1, 1);
    cfg.stream = stream;
    if (cudaLaunchKernelEx(&cfg, add_norm_rows<DT, WARPS, ROWS, NW>, a) != cudaSuccess) return FP8L_ECUDA;
    return launch_status();
}

// Every block of the grid is resident (cooperative launch): at most one per
// row, and as many per SM as 2048 threads and the held rows allow.
template <int DT, int WARPS, int NW>
int launch_dynamic(AddNormArgs a, int sms, cudaStream_t stream) {
    auto kernel = add_norm_dynamic<DT, WARPS, NW>;
    static std::atomic<int> ready[kAddMaxDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kAddMaxDevices) return FP8L_ECUDA;
    if (!ready[dev].load(std::memory_order_acquire)) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kAddSmemBudget) !=
            cudaSuccess)
            return FP8L_ECUDA;
        ready[dev].store(1, std::memory_order_release);
    }
    const size_t row_bytes = static_cast<size_t>(a.K) * 2;
    int per_sm = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, 32 * WARPS, 0) != cudaSuccess ||
        per_sm < 1)
        return FP8L_ECUDA;
    // rows held: as many as every block's share of the budget takes, and no
    // more than it has
    const int64_t most = int64_t(per_sm) * sms;
    int64_t grid = a.M < most ? a.M : most;
    const int64_t rows = (a.M + grid - 1) / grid;
    const int on_sm = static_cast<int>((grid + sms - 1) / sms);
    int64_t slots = static_cast<int64_t>((kAddSmemBudget / on_sm) / row_bytes);
    if (slots > rows) slots = rows;
    int fit = 0;
    while (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&fit, kernel, 32 * WARPS, slots * row_bytes) ==
               cudaSuccess &&
           int64_t(fit) * sms < grid && slots > 0)
        --slots;
    if (int64_t(fit) * sms < grid) return FP8L_ECUDA;
    a.slots = static_cast<int>(slots);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    cfg.blockDim = dim3(32 * WARPS, 1, 1);
    cfg.dynamicSmemBytes = slots * row_bytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kernel, a) != cudaSuccess) return FP8L_ECUDA;
    return launch_status();
}

template <int DT>
int dispatch_add_norm(const AddNormArgs &a, int sms, cudaStream_t s) {
    const int words = a.K / 8;
    if (a.mode == FP8L_NQ_DYNAMIC) {
        if (words <= 128) return launch_dynamic<DT, 4, 1>(a, sms, s);
        if (words <= 512) return launch_dynamic<DT, 8, 2>(a, sms, s);
        if (words <= 1024) return launch_dynamic<DT, 8, 4>(a, sms, s);
        if (words <= 2048) return launch_dynamic<DT, 16, 4>(a, sms, s);
        return launch_dynamic<DT, 32, 4>(a, sms, s);
    }
    if (words <= 32) return launch_rows<DT, 1, 8, 1>(a, s);
    if (words <= 128) return launch_rows<DT, 1, 8, 4>(a, s);
    if (words <= 256) return launch_rows<DT, 4, 1, 2>(a, s);
    if (words <= 512) return launch_rows<DT, 8, 1, 2>(a, s);
    if (words <= 1024) return launch_rows<DT, 8, 1, 4>(a, s);
    if (words <= 2048) return launch_rows<DT, 16, 1, 4>(a, s);
    return launch_rows<DT, 32, 1, 4>(a, s);
}

// Whether [p, p + n) and [q, q + m) share a byte (a null range shares none).
bool overlap(const void *p, size_t n, const void *q, size_t m) {
    if (p == nullptr || q == nullptr || n == 0 || m == 0) return false;
    const uintptr_t u = reinterpret_cast<uintptr_t>(p), v = reinterpret_cast<uintptr_t>(q);
    return u < v + m && v < u + n;
}

}  // namespace
}  // namespace fp8l

extern "C" int fp8_add_rmsnorm_quant(const void *x, const void *residual, int x_dtype,
                                     const void *gamma, float eps, int64_t M, int64_t K, void *total,
                                     uint8_t *q, float *scale, int mode, void *h, void *workspace,
                                     void *stream) {
    using namespace fp8l;
    if (x_dtype != FP8L_F16 && x_dtype != FP8L_BF16) return FP8L_EINVAL;
    if (mode < FP8L_NQ_DYNAMIC || mode > FP8L_NQ_NORM_ONLY) return FP8L_EINVAL;
    if (!(eps >= 0.0f) || eps > 3.0e38f) return FP8L_EINVAL;  // also rejects NaN
    if (M < 0 || M > 0x7FFFFFFF || K <= 0 || K % 16 != 0 || K > kAddMaxK) return FP8L_ESHAPE;
    const bool codes = mode != FP8L_NQ_NORM_ONLY;
    if (gamma == nullptr || (codes && scale == nullptr && !(M == 0 && mode == FP8L_NQ_PER_TOKEN)))
        return FP8L_EINVAL;
    if (M > 0 && (x == nullptr || residual == nullptr || total == nullptr ||
                  (codes ? q == nullptr : h == nullptr)))
        return FP8L_EINVAL;
    if (mode == FP8L_NQ_DYNAMIC && workspace == nullptr) return FP8L_EINVAL;
    if (!aligned16(gamma) || (M > 0 && (!aligned16(x) || !aligned16(residual) || !aligned16(total) ||
                                        (codes && !aligned16(q)) || !aligned16(h))) ||
        !aligned16(workspace) || (codes && (reinterpret_cast<uintptr_t>(scale) & 3u) != 0))
        return FP8L_EALIGN;
    // outputs share no byte with an input or each other, but the stream may
    // be updated in place
    const size_t n16 = static_cast<size_t>(M) * K * 2, n8 = n16 / 2;
    struct Range {
        const void *p;
        size_t n;
    };
    const bool scale_out = mode == FP8L_NQ_DYNAMIC || mode == FP8L_NQ_PER_TOKEN;
    const Range in[5] = {{x, n16}, {residual, n16}, {gamma, static_cast<size_t>(K) * 2},
                         {mode == FP8L_NQ_STATIC ? scale : nullptr, 4},
                         {mode == FP8L_NQ_DYNAMIC ? workspace : nullptr, kWorkspaceBytes}};
    const Range out[4] = {{total, n16}, {codes ? q : nullptr, n8}, {h, n16},
                          {scale_out ? scale : nullptr, mode == FP8L_NQ_DYNAMIC ? 4 : size_t(M) * 4}};
    for (int i = 0; i < 4; ++i) {
        for (int j = 0; j < 5; ++j)
            if (!(i == 0 && j < 2 && in[j].p == total) && overlap(out[i].p, out[i].n, in[j].p, in[j].n))
                return FP8L_EINVAL;
        for (int j = i + 1; j < 4; ++j)
            if (overlap(out[i].p, out[i].n, out[j].p, out[j].n)) return FP8L_EINVAL;
    }
    int sms = 0;
    const int st = check_device(&sms);
    if (st != FP8L_OK) return st;
    const cudaStream_t s = as_stream(stream);
    if (M == 0) {
        if (mode != FP8L_NQ_DYNAMIC) return FP8L_OK;
        add_norm_empty_scale<<<1, 1, 0, s>>>(scale);
        return launch_status();
    }
    AddNormArgs a{};
    a.x = x;
    a.res = residual;
    a.gamma = gamma;
    a.eps = eps;
    a.M = static_cast<int>(M);
    a.K = static_cast<int>(K);
    a.total = total;
    a.q = q;
    a.scale = scale;
    a.h = h;
    a.mode = mode;
    if (mode == FP8L_NQ_DYNAMIC) {
        a.epoch = epoch_word(workspace);
        a.arrive = arrive_words(workspace);
        a.amax = amax_words(workspace);
        a.status = status_word(workspace);
        if (library_status_word(&a.lib_status) != FP8L_OK) return FP8L_ECUDA;
    }
    const WaitConfig wc = wait_config();
    a.wait_cycles = wc.cycles;
    a.stall = wc.stall;
    return x_dtype == FP8L_BF16 ? dispatch_add_norm<FP8L_BF16>(a, sms, s)
                                : dispatch_add_norm<FP8L_F16>(a, sms, s);
}
