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
// and nothing is read twice.  Enough rows are in flight on an SM (threads of
// 2 to 8 pending 16-byte loads each) to cover HBM's latency without a copy
// pipeline.
//   add_norm_rows  one row per block (a warp per row up to 1024 columns, where
//                  a block's barriers would cost more than the row).
//   add_norm_max, add_norm_cast
//                  one scale for the whole tensor: the first leaves the
//                  tensor's maximum in the workspace and a row's factor r in
//                  the row of q that its codes will fill; the second, a
//                  programmatic dependent, casts h, or makes it again from the
//                  stream just written, the newest rows (still in L2) first.
//   add_norm_cluster
//                  the same for so few rows that one cluster of CTAs holds
//                  them: the maximum goes through distributed shared memory.
// Measured (GB300, replayed graphs, of the copy bandwidth): 16384 x 8192
// static or per token 138.5 us, 0.997; 1021 x 8192 per token 10.3 us, 0.84; 16
// x 4096 per token 1.9 us (launch and one round trip).  Dynamic: 16384 x 8192
// 188 us (177 for 7 bytes an element and the stream read again), 1021 x 8192
// with h 16.4 us for 11.1 of traffic, 16 x 4096 2.6 us (4.2 in two kernels).
// One cooperative kernel with a grid barrier between the halves and h held in
// shared memory took 221, 17.2 and 4.1 us, and had a wait in it.
#include <atomic>

#include "quant_device.cuh"
#include "skinny_device.cuh"

namespace fp8l {
namespace {

constexpr int kAddMaxK = 32768;
// Workspace words of the dynamic mode: a call counter, the half of the pair of
// magnitude maxima that the call uses (counter mod 2), and that pair, whose
// unused half is zero between calls.  add_norm_max reads the counter and names
// the half; add_norm_cast clears the other half and advances the counter: no
// word is written in a kernel that other blocks of it still read.  (Counting
// the blocks that had read the maximum instead, one atomic each, took 4096 x
// 4096 from 25 to 40 us.)
constexpr size_t kAddWordsOffset = 32;
struct AddNormWords {
    unsigned counter, half, amax[2];
};
constexpr int kAddMaxCluster = 16;  // CTAs (above 8 opted in)
constexpr int kAddMaxDevices = 64;
static_assert(kAddWordsOffset >= kBarrierAreaBytes && kAddWordsOffset + sizeof(AddNormWords) <= kPartialsOffset,
              "words of their own in the workspace");

struct AddNormArgs {
    const void *x, *res, *gamma;
    float eps;
    int M, K;
    void *total;
    uint8_t *q;
    float *scale;
    void *h;
    int mode;
    AddNormWords *words;  // dynamic
};

__device__ __forceinline__ uint32_t ld_relaxed(const unsigned *p) {
    uint32_t v;
    asm volatile("ld.relaxed.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}

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
        if ((threadIdx.x & 31) == 0) part[(threadIdx.x >> 5) % WARPS] = v;
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

// r = 1 / sqrt(ms): a reciprocal of a root, and one Newton step with the
// residual 1 - ms y^2 to twice the precision (ms y = hi + lo), which leaves
// little more than r's own rounding
__device__ __forceinline__ uint64_t rms_factor(float ss, int K, float eps) {
    const float ms = __fadd_rn(__fdiv_rn(ss, static_cast<float>(K)), eps);
    const float y = __frcp_rn(__fsqrt_rn(ms));
    const float hi = __fmul_rn(ms, y), lo = __fmaf_rn(ms, y, -hi);
    const float e = __fmaf_rn(-lo, y, __fmaf_rn(-hi, y, 1.0f));
    // (a zero row without eps has y infinite and stays that; a mean square past
    // float32's range has y = 0 and stays that, as in fp8_rmsnorm_quant: ms y
    // would be infinity times 0)
    const float r = ms > 0x1p-100f && ms <= 3.4e38f ? __fmaf_rn(0.5f * y, e, y) : y;
    return f2_pack(__float_as_uint(r), __float_as_uint(r));
}

__device__ __forceinline__ float pair_sum(uint64_t acc) {
    return __fadd_rn(__uint_as_float(static_cast<uint32_t>(acc)),
                     __uint_as_float(static_cast<uint32_t>(acc >> 32)));
}

// What a row's threads do, WARPS warps a row, NW words (of 8 elements) a
// thread, words tid, tid + 32 WARPS, ...  All of a thread's loads are on their
// way before the first is used.
template <int DT, int WARPS, int NW>
struct Row {
    static constexpr int kSpan = 32 * WARPS;

    // the sum x + res, stored as the new stream; words beyond the row are zeros
    __device__ __forceinline__ static void add(const AddNormArgs &a, size_t at, int tid, int words,
                                               uint4 (&t)[NW]) {
        uint4 x[NW], r[NW];
#pragma unroll
        for (int j = 0; j < NW; ++j) {
            const int w = tid + j * kSpan;
            x[j] = r[j] = make_uint4(0, 0, 0, 0);
            if (w < words) {
                x[j] = ld_once16(static_cast<const uint4 *>(a.x) + at + w);
                r[j] = ld_once16(static_cast<const uint4 *>(a.res) + at + w);
            }
        }
#pragma unroll
        for (int j = 0; j < NW; ++j) {
            const int w = tid + j * kSpan;
            t[j] = add_word<DT>(x[j], r[j]);
            if (w < words) static_cast<uint4 *>(a.total)[at + w] = t[j];
        }
    }

    // its float pair of squares' sums
    __device__ __forceinline__ static float squares(const uint4 (&t)[NW]) {
        uint64_t acc = 0;
#pragma unroll
        for (int j = 0; j < NW; ++j) acc = add_squares<DT>(t[j], acc);
        return pair_sum(acc);
    }

    // h in place of t
    __device__ __forceinline__ static void scale(const AddNormArgs &a, int tid, int words, uint64_t r2,
                                                 uint4 (&t)[NW]) {
        uint4 g[NW];
#pragma unroll
        for (int j = 0; j < NW; ++j) {
            const int w = tid + j * kSpan;
            g[j] = w < words ? ld_act16(static_cast<const uint4 *>(a.gamma) + w) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int j = 0; j < NW; ++j) t[j] = scaled_word<DT>(t[j], g[j], r2);
    }

    __device__ __forceinline__ static uint32_t magnitude(const uint4 (&t)[NW], uint32_t m) {
#pragma unroll
        for (int j = 0; j < NW; ++j) m = word_mag_max<DT>(t[j], m);
        return m;
    }

    __device__ __forceinline__ static void store_h(const AddNormArgs &a, size_t at, int tid, int words,
                                                   const uint4 (&t)[NW]) {
        if (a.h == nullptr) return;
#pragma unroll
        for (int j = 0; j < NW; ++j) {
            const int w = tid + j * kSpan;
            if (w < words) static_cast<uint4 *>(a.h)[at + w] = t[j];
        }
    }

    template <bool CLAMP>
    __device__ __forceinline__ static void store_codes(const AddNormArgs &a, size_t at, int tid, int words,
                                                       const uint4 (&t)[NW], const Quot &d) {
#pragma unroll
        for (int j = 0; j < NW; ++j) {
            const int w = tid + j * kSpan;
            if (w < words) reinterpret_cast<uint2 *>(a.q)[at + w] = codes_of_word<DT, CLAMP>(t[j], d);
        }
    }
};

// ROWS rows a block (a warp each), or one row (WARPS warps).
template <int DT, int WARPS, int ROWS, int NW, int BLOCKS>
__global__ void __launch_bounds__(32 * WARPS * ROWS, BLOCKS) add_norm_rows(const AddNormArgs a) {
    static_assert(WARPS == 1 || ROWS == 1, "a block is one row, or a warp is");
    using R = Row<DT, WARPS, NW>;
    __shared__ float fpart[WARPS];
    __shared__ uint32_t upart[WARPS];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tid = WARPS == 1 ? (threadIdx.x & 31) : threadIdx.x;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * ROWS + (WARPS == 1 ? threadIdx.x >> 5 : 0);
    pdl_wait();
    if (row >= a.M) return;  // a whole warp (ROWS > 1) or no thread
    const int words = a.K / 8;
    const size_t at = static_cast<size_t>(row) * words;
    uint4 t[NW];
    R::add(a, at, tid, words, t);
    const uint64_t r2 = rms_factor(row_sum<WARPS>(R::squares(t), fpart), a.K, a.eps);
    R::scale(a, tid, words, r2, t);
    R::store_h(a, at, tid, words, t);
    if (a.mode == FP8L_NQ_NORM_ONLY) return;
    if (a.mode == FP8L_NQ_PER_TOKEN) {
        const uint32_t m = fold_mag<DT>(R::magnitude(t, 0));
        const float s = scale_from_amax(mag_bits_to_float<DT>(row_max<WARPS>(m, upart)));
        if (tid == 0) a.scale[row] = s;
        R::template store_codes<false>(a, at, tid, words, t, Quot::make<DT>(s));
    } else {
        R::template store_codes<true>(a, at, tid, words, t, Quot::make<DT>(ld_act_f32(a.scale)));
    }
}

// The dynamic mode for a few rows, one cluster of CTAs (ROWS rows each): every
// CTA pushes its maximum to all, and the rows never leave the registers.
template <int DT, int WARPS, int ROWS, int NW>
__global__ void __launch_bounds__(32 * WARPS * ROWS, 1) add_norm_cluster(const AddNormArgs a) {
    using R = Row<DT, WARPS, NW>;
    __shared__ float fpart[ROWS][WARPS];
    __shared__ uint32_t red[33], peak[kAddMaxCluster];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // (arrived here, waited for before a peer's memory is written)
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    const int tid = threadIdx.x % (32 * WARPS), sub = threadIdx.x / (32 * WARPS);
    const int row = static_cast<int>(blockIdx.x) * ROWS + sub;
    const bool in = row < a.M;
    const int words = in ? a.K / 8 : 0;  // a row beyond the last has none
    const size_t at = static_cast<size_t>(row) * (a.K / 8);
    uint4 t[NW];
    pdl_wait();
    R::add(a, at, tid, words, t);
    const uint64_t r2 = rms_factor(row_sum<WARPS>(R::squares(t), fpart[sub]), a.K, a.eps);
    R::scale(a, tid, words, r2, t);
    const uint32_t m = block_max_u32(in ? fold_mag<DT>(R::magnitude(t, 0)) : 0u, red);
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    const unsigned ctas = gridDim.x;  // one cluster
    if (threadIdx.x < ctas) {
        uint32_t remote = static_cast<uint32_t>(__cvta_generic_to_shared(&peak[blockIdx.x]));
        asm volatile("mapa.shared::cluster.u32 %0, %0, %1;" : "+r"(remote) : "r"(threadIdx.x));
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(remote), "r"(m) : "memory");
    }
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    R::store_h(a, at, tid, words, t);
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    const unsigned lane = threadIdx.x & 31;
    const uint32_t all = __reduce_max_sync(0xFFFFFFFFu, lane < ctas ? peak[lane] : 0u);
    const float s = scale_from_amax(mag_bits_to_float<DT>(all));
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.scale = s;
    R::template store_codes<false>(a, at, tid, words, t, Quot::make<DT>(s));
}

// The dynamic mode's first half: the stream, h when it is wanted, the factors
// and the maximum.  As many blocks as fit at once go through the rows, so that
// few of them touch the workspace's words (one block a row, 4096 of them, took
// longer to read those words than to do the rest).
template <int DT, int WARPS, int ROWS, int NW, int BLOCKS>
__global__ void __launch_bounds__(32 * WARPS * ROWS, BLOCKS) add_norm_max(const AddNormArgs a) {
    using R = Row<DT, WARPS, NW>;
    __shared__ float fpart[2][WARPS];
    __shared__ uint32_t red[33];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tid = WARPS == 1 ? (threadIdx.x & 31) : threadIdx.x, words = a.K / 8;
    pdl_wait();
    const int64_t first = static_cast<int64_t>(blockIdx.x) * ROWS + (WARPS == 1 ? threadIdx.x >> 5 : 0);
    uint32_t m = 0;
    int flip = 0;  // the partials alternate between two arrays: one barrier a row is enough
    for (int64_t row = first; row < a.M; row += static_cast<int64_t>(gridDim.x) * ROWS) {
        const size_t at = static_cast<size_t>(row) * words;
        uint4 t[NW];
        R::add(a, at, tid, words, t);
        const uint64_t r2 = rms_factor(row_sum<WARPS>(R::squares(t), fpart[flip]), a.K, a.eps);
        flip ^= 1;
        R::scale(a, tid, words, r2, t);
        m = R::magnitude(t, m);
        if (a.h != nullptr)
            R::store_h(a, at, tid, words, t);
        else if (tid == 0)
            *reinterpret_cast<uint32_t *>(a.q + at * 8) = static_cast<uint32_t>(r2);
    }
    m = block_max_u32(fold_mag<DT>(m), red);
    if (threadIdx.x == 0) {
        const unsigned half = ld_relaxed(&a.words->counter) & 1u;
        if (blockIdx.x == 0) a.words->half = half;
        atomicMax(&a.words->amax[half], m);
    }
}

// Its second half: the scale from the maximum, and the codes.
template <int DT, int WARPS, int ROWS, int NW, int BLOCKS>
__global__ void __launch_bounds__(32 * WARPS * ROWS, BLOCKS) add_norm_cast(const AddNormArgs a) {
    using R = Row<DT, WARPS, NW>;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tid = WARPS == 1 ? (threadIdx.x & 31) : threadIdx.x, words = a.K / 8;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * ROWS + (WARPS == 1 ? threadIdx.x >> 5 : 0);
    pdl_wait();
    const unsigned half = ld_relaxed(&a.words->half);
    const float s = scale_from_amax(mag_bits_to_float<DT>(ld_relaxed(&a.words->amax[half])));
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        *a.scale = s;
        a.words->amax[half ^ 1u] = 0u;
        a.words->counter += 1u;
    }
    const Quot d = Quot::make<DT>(s);
    for (int64_t i = first; i < a.M; i += static_cast<int64_t>(gridDim.x) * ROWS) {
        const size_t at = static_cast<size_t>(a.M - 1 - i) * words;
        uint4 t[NW];
        const uint4 *src = static_cast<const uint4 *>(a.h != nullptr ? a.h : a.total) + at;
#pragma unroll
        for (int j = 0; j < NW; ++j) {
            const int w = tid + j * R::kSpan;
            t[j] = w < words ? ld_once16(src + w) : make_uint4(0, 0, 0, 0);
        }
        if (a.h == nullptr) {
            const uint32_t r = __float_as_uint(ld_act_f32(reinterpret_cast<const float *>(a.q + at * 8)));
            // every thread has the row's factor before codes overwrite it
            if constexpr (WARPS > 1)
                __syncthreads();
            else
                __syncwarp();
            R::scale(a, tid, words, f2_pack(r, r), t);
        }
        R::template store_codes<false>(a, at, tid, words, t, d);
    }
}

__global__ void add_norm_empty_scale(float *scale) { *scale = 1.0f; }

// The largest cluster of add_norm_cluster that the GPU holds, 16, 8 or 1.
template <int DT, int WARPS, int ROWS, int NW>
int largest_cluster() {
    static std::atomic<int> known[kAddMaxDevices];  // 0: not asked yet
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kAddMaxDevices) return 1;
    int most = known[dev].load(std::memory_order_relaxed);
    if (most > 0) return most;
    const auto kernel = add_norm_cluster<DT, WARPS, ROWS, NW>;
    most = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess
               ? kAddMaxCluster : 8;
    for (; most > 1; most = most > 8 ? 8 : 1) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(most), 1, 1);
        cfg.blockDim = dim3(32 * WARPS * ROWS, 1, 1);
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = static_cast<unsigned>(most);
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) == cudaSuccess && n > 0) break;
        (void)cudaGetLastError();
    }
    known[dev].store(most, std::memory_order_relaxed);
    return most;
}

// One cluster's launch, where its CTAs hold all rows and the GPU holds it.
template <int DT, int WARPS, int ROWS, int NW>
bool launch_cluster(const AddNormArgs &a, cudaStream_t stream, int *status) {
    const int ctas = static_cast<int>((int64_t(a.M) + ROWS - 1) / ROWS);
    if (ctas > kAddMaxCluster || ctas > largest_cluster<DT, WARPS, ROWS, NW>()) return false;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas), 1, 1);
    cfg.blockDim = dim3(32 * WARPS * ROWS, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cfg.gridDim.x;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    *status = cudaLaunchKernelEx(&cfg, add_norm_cluster<DT, WARPS, ROWS, NW>, a) == cudaSuccess
                  ? launch_status() : FP8L_ECUDA;
    return true;
}

// By the row's length and the rows that 16 CTAs hold: few threads a CTA first
// (17 rows of 4096: two a CTA 3.0 us, four 4.1, in two kernels 4.2; 17 of 8192
// 3.9, four a CTA 5.8, in two kernels 4.7; 128 of 128 2.2, 512 2.9 and 3.9).
template <int DT>
bool dispatch_cluster(const AddNormArgs &a, cudaStream_t s, int *st) {
    const int words = a.K / 8;
    if (words <= 32) return launch_cluster<DT, 1, 8, 1>(a, s, st) || launch_cluster<DT, 1, 32, 1>(a, s, st);
    if (words <= 128) return launch_cluster<DT, 4, 4, 1>(a, s, st) || launch_cluster<DT, 1, 8, 4>(a, s, st);
    if (words <= 256)
        return launch_cluster<DT, 4, 1, 2>(a, s, st) || launch_cluster<DT, 4, 2, 2>(a, s, st) ||
               launch_cluster<DT, 4, 4, 2>(a, s, st);
    if (words <= 512) return launch_cluster<DT, 8, 1, 2>(a, s, st) || launch_cluster<DT, 8, 2, 2>(a, s, st);
    if (words <= 1024) return launch_cluster<DT, 8, 1, 4>(a, s, st) || launch_cluster<DT, 8, 2, 4>(a, s, st);
    if (words <= 2048) return launch_cluster<DT, 16, 1, 4>(a, s, st);
    return launch_cluster<DT, 32, 1, 4>(a, s, st);
}

template <int DT, int WARPS, int ROWS, int NW, int BLOCKS>
int launch_rows(const AddNormArgs &a, int sms, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((int64_t(a.M) + ROWS - 1) / ROWS), 1, 1);
    cfg.blockDim = dim3(32 * WARPS * ROWS, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    // (the kernels wait for the preceding one before they touch memory)
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (a.mode == FP8L_NQ_DYNAMIC) {
        if (cfg.gridDim.x > static_cast<unsigned>(sms * BLOCKS)) cfg.gridDim.x = sms * BLOCKS;
        if (cudaLaunchKernelEx(&cfg, add_norm_max<DT, WARPS, ROWS, NW, BLOCKS>, a) != cudaSuccess ||
            cudaLaunchKernelEx(&cfg, add_norm_cast<DT, WARPS, ROWS, NW, BLOCKS>, a) != cudaSuccess)
            return FP8L_ECUDA;
    } else if (cudaLaunchKernelEx(&cfg, add_norm_rows<DT, WARPS, ROWS, NW, BLOCKS>, a) != cudaSuccess) {
        return FP8L_ECUDA;
    }
    return launch_status();
}

// Threads and words a thread by the row's length: rows up to 1024 elements a
// warp each (a block's barriers would cost more than the row), then the least
// threads that hold a row in two to four words, with as many blocks an SM as
// 64 to 80 registers a thread leave.
template <int DT>
int dispatch_add_norm(const AddNormArgs &a, int sms, cudaStream_t s) {
    const int words = a.K / 8;
    int st = FP8L_OK;
    if (a.mode == FP8L_NQ_DYNAMIC && dispatch_cluster<DT>(a, s, &st)) return st;
    if (words <= 32) return launch_rows<DT, 1, 8, 1, 6>(a, sms, s);
    if (words <= 128) return launch_rows<DT, 1, 8, 4, 3>(a, sms, s);
    if (words <= 256) return launch_rows<DT, 4, 1, 2, 8>(a, sms, s);
    if (words <= 512) return launch_rows<DT, 8, 1, 2, 4>(a, sms, s);
    if (words <= 1024) return launch_rows<DT, 8, 1, 4, 3>(a, sms, s);
    if (words <= 2048) return launch_rows<DT, 16, 1, 4, 2>(a, sms, s);
    return launch_rows<DT, 32, 1, 4, 1>(a, sms, s);
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
    for (int j = 0; j < 3; ++j)  // (the workspace is written too)
        if (overlap(in[j].p, in[j].n, in[4].p, in[4].n)) return FP8L_EINVAL;
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
        a.words = reinterpret_cast<AddNormWords *>(static_cast<char *>(workspace) + kAddWordsOffset);
    }
    return x_dtype == FP8L_BF16 ? dispatch_add_norm<FP8L_BF16>(a, sms, s)
                                : dispatch_add_norm<FP8L_F16>(a, sms, s);
}
