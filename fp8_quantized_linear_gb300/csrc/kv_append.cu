// Norms of queries and keys per head, the position rotation, and the write
// of keys and values into the paged FP8 cache, in one pass over the q/k/v
// product's output (fp8_qk_norm_rope_append).
//
//   r    = 1 / sqrt(mean_d x_d^2 + eps),  x <- x r gamma_d        (q, k)
//   (a, b) <- (a cos - b sin, b cos + a sin)                     (q, k)
//   s    = max over the page's new tokens of amax / 448 (and s_old when the
//          page already holds tokens),  code = E4M3(x / s)       (k, v)
//
// The pass is bound by HBM once there are thousands of tokens (it reads qkv
// once and writes q and the codes once) and by latency in a decode step.  A
// row (one token, one head) is 8 elements in each of DIM / 8 lanes, so every
// global access is 16 bytes, the norm's sum is a shuffle tree inside the
// group and a rotation partner is one shuffle away (or in the same thread).
//
// Blocks first take the cache's units, then the queries.  A unit is a chunk
// of tokens of one kv head, keys or values; the runs of slots that start in
// the chunk are found from the slots alone (ballots of "first slot of a run"
// and "continues a run"), so no list of pages has to be built first.  Runs of
// one or two tokens (decode) go to one group each; longer runs (prompts) are
// spread over the whole block, the rows staying in registers between the
// maximum and the cast.  Tokens that a page already holds are re-cast by the
// whole block when the scale grew: a group alone would read up to 127 rows
// one after the other.
#include "kv_device.cuh"
#include "quant_device.cuh"

namespace fp8l {
namespace {

constexpr int kAppThreads = 256;
constexpr int kAppMaxPage = 128;
constexpr int kAppMaxChunk = 64;    // tokens whose runs one block starts
constexpr int kAppHeadsPerGroup = 4;  // query heads of a token per group: loads in flight

struct AppendParams {
    const uint16_t *qkv;
    int tokens;
    int64_t stride;
    int q_heads, kv_heads;
    const uint16_t *q_gamma, *k_gamma;
    float eps;
    const float *cos_sin;
    int max_positions, rot, interleaved;
    const int32_t *positions, *slots;
    uint16_t *q_out;
    uint8_t *k_cache, *v_cache;
    float *k_scale, *v_scale;
    int num_slots, page_shift;
    int chunk;      // tokens per kv block
    int kv_blocks;  // blocks [0, kv_blocks) take keys and values
    int head_groups;  // ceil(q_heads / kAppHeadsPerGroup)
};

// The pages' blocks of a scale: values are never quantized with less
constexpr float kKvMinScale = FP8L_KV_MIN_SCALE;

struct Row {
    float x[8];
};

template <int DT>
__device__ __forceinline__ Row widen_row(const uint4 &u) {
    Row r;
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint64_t f = widen16<DT>(w[i]);
        r.x[2 * i] = __uint_as_float(static_cast<uint32_t>(f));
        r.x[2 * i + 1] = __uint_as_float(static_cast<uint32_t>(f >> 32));
    }
    return r;
}

template <int DT>
__device__ __forceinline__ uint32_t narrow2(float a, float b) {
    if constexpr (DT == FP8L_BF16) {
        __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<uint32_t *>(&h);
    } else {
        __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<uint32_t *>(&h);
    }
}

// cosines and sines of a token for the eight dimensions [8 l, 8 l + 8) of a
// lane (four pairs in c[0..3], s[0..3] when interleaved)
struct Turn {
    float c[8], s[8];
    int half8;  // rot / 16: lanes of the rotated first half
    bool on;    // this lane's dimensions rotate
};

__device__ __forceinline__ Turn load_turn(const AppendParams &p, int token, int l) {
    Turn t;
    t.half8 = p.rot >> 4;
    t.on = 8 * l < p.rot;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        t.c[i] = 1.0f;
        t.s[i] = 0.0f;
    }
    if (t.on) {
        const int pos = min(max(p.positions[token], 0), p.max_positions - 1);
        const float *row = p.cos_sin + static_cast<int64_t>(pos) * p.rot;
        const int half = p.rot >> 1;
        const int i0 = p.interleaved ? 4 * l : 8 * (l < t.half8 ? l : l - t.half8);
        const float4 c0 = *reinterpret_cast<const float4 *>(row + i0);
        const float4 s0 = *reinterpret_cast<const float4 *>(row + half + i0);
        t.c[0] = c0.x, t.c[1] = c0.y, t.c[2] = c0.z, t.c[3] = c0.w;
        t.s[0] = s0.x, t.s[1] = s0.y, t.s[2] = s0.z, t.s[3] = s0.w;
        if (!p.interleaved) {
            const float4 c1 = *reinterpret_cast<const float4 *>(row + i0 + 4);
            const float4 s1 = *reinterpret_cast<const float4 *>(row + half + i0 + 4);
            t.c[4] = c1.x, t.c[5] = c1.y, t.c[6] = c1.z, t.c[7] = c1.w;
            t.s[4] = s1.x, t.s[5] = s1.y, t.s[6] = s1.z, t.s[7] = s1.w;
        }
    }
    return t;
}

// The norm (when `gamma`) and the rotation of one row held by the LANES
// lanes of `mask`
template <int LANES>
__device__ __forceinline__ void norm_rotate(Row &r, bool norm, const Row &gamma, float eps, const Turn &t,
                                            bool interleaved, int l, uint32_t mask) {
    if (norm) {
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(r.x[i], r.x[i], ss);
#pragma unroll
        for (int o = LANES / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(mask, ss, o, LANES);
        const float inv = __fdiv_rn(1.0f, __fsqrt_rn(ss * (1.0f / (8 * LANES)) + eps));
#pragma unroll
        for (int i = 0; i < 8; ++i) r.x[i] = (r.x[i] * inv) * gamma.x[i];
    }
    if (interleaved) {
        if (t.on) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float a = r.x[2 * i], b = r.x[2 * i + 1];
                r.x[2 * i] = a * t.c[i] - b * t.s[i];
                r.x[2 * i + 1] = b * t.c[i] + a * t.s[i];
            }
        }
    } else {
        const bool low = l < t.half8;
        const int partner = !t.on ? l : (low ? l + t.half8 : l - t.half8);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float other = __shfl_sync(mask, r.x[i], partner, LANES);
            if (t.on) r.x[i] = low ? r.x[i] * t.c[i] - other * t.s[i] : r.x[i] * t.c[i] + other * t.s[i];
        }
    }
}

__device__ __forceinline__ uint32_t row_mag(const Row &r) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(r.x[i]) & 0x7FFFFFFFu);
    return m;
}

__device__ __forceinline__ uint2 row_codes(const Row &r, const Quot &d) {
    const uint4 a = make_uint4(__float_as_uint(r.x[0]), __float_as_uint(r.x[1]), __float_as_uint(r.x[2]),
                               __float_as_uint(r.x[3]));
    const uint4 b = make_uint4(__float_as_uint(r.x[4]), __float_as_uint(r.x[5]), __float_as_uint(r.x[6]),
                               __float_as_uint(r.x[7]));
    return make_uint2(codes_of_word<FP8L_F32, false>(a, d).x, codes_of_word<FP8L_F32, false>(b, d).x);
}

__device__ __forceinline__ float block_scale(uint32_t amax_bits) {
    return fmaxf(__fdiv_rn(__uint_as_float(amax_bits), kE4M3Max), kKvMinScale);
}

// A page and head whose earlier tokens [0, offset) move to a larger scale
struct Recast {
    int64_t ph;
    int offset;
    float from, to;
};

template <int DIM>
__device__ void recast_block(uint8_t *cache, const Recast &job, int page_size) {
    constexpr int kPerOctet = DIM / 16 * 8;  // 16-byte pieces of an octet
    uint8_t *at = cache + kv_chunk_offset(job.ph, page_size, DIM, 0, 0);
    const Quot d = Quot::make<FP8L_F32>(job.to);
    const int pieces = ((job.offset + 7) >> 3) * kPerOctet;
    for (int i = static_cast<int>(threadIdx.x); i < pieces; i += kAppThreads) {
        if ((i / kPerOctet) * 8 + (i & 7) >= job.offset) continue;
        uint4 u = *reinterpret_cast<const uint4 *>(at + static_cast<int64_t>(i) * 16);
        uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float f[4];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
                    static_cast<__nv_fp8x2_storage_t>((w[j] >> (16 * k)) & 0xFFFFu), __NV_E4M3);
                const float2 v = __half22float2(__half2(h));
                f[2 * k] = v.x * job.from;
                f[2 * k + 1] = v.y * job.from;
            }
            w[j] = codes_of_word<FP8L_F32, false>(make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]),
                                                             __float_as_uint(f[2]), __float_as_uint(f[3])), d).x;
        }
        *reinterpret_cast<uint4 *>(at + static_cast<int64_t>(i) * 16) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

template <int DT, int DIM>
__device__ void append_unit(const AppendParams &p, int unit) {
    constexpr int LANES = DIM / 8, GROUPS = kAppThreads / LANES, ROWS = kAppMaxPage / GROUPS;
    __shared__ uint32_t lead[8], cont[8];
    __shared__ uint32_t red[33];
    __shared__ Recast jobs[kAppMaxChunk];
    __shared__ int num_jobs;
    const int heads2 = 2 * p.kv_heads;
    const int t0 = unit / heads2 * p.chunk;
    const int head = (unit % heads2) >> 1;
    const bool values = unit & 1;
    const int P = 1 << p.page_shift;
    const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5;
    const int g = tid / LANES, l = tid % LANES;
    const uint32_t mask = LANES == 16 ? 0xFFFFu << (tid & 16) : 0xFFu << (tid & 24);

    {
        const int64_t t = static_cast<int64_t>(t0) + tid;
        bool first = false, more = false;
        if (tid < p.chunk + P && t < p.tokens) {
            const int s = p.slots[t];
            const bool valid = s >= 0 && s < p.num_slots;
            first = valid && (t == 0 || (s & (P - 1)) == 0 || p.slots[t - 1] != s - 1);
            more = valid && !first;
        }
        const uint32_t a = __ballot_sync(0xFFFFFFFFu, first && tid < p.chunk);
        const uint32_t b = __ballot_sync(0xFFFFFFFFu, more);
        if ((tid & 31) == 0) {
            lead[warp] = a;
            cont[warp] = b;
        }
        if (tid == 0) num_jobs = 0;
    }
    __syncthreads();
    if ((lead[0] | lead[1]) == 0u) return;
    // tokens of the run that starts at token t0 + i
    auto run_length = [&](int i) {
        int j = i + 1;
        while (j < 256) {
            const uint32_t clear = ~cont[j >> 5] >> (j & 31);
            if (clear != 0u) {
                j += __ffs(static_cast<int>(clear)) - 1;
                break;
            }
            j = (j | 31) + 1;
        }
        return min(j - i, P);
    };

    uint8_t *cache = values ? p.v_cache : p.k_cache;
    float *scales = values ? p.v_scale : p.k_scale;
    const uint16_t *src = p.qkv + (p.q_heads + (values ? p.kv_heads : 0) + head) * DIM + 8 * l;
    const bool norm = !values && p.k_gamma != nullptr;
    Row gamma = {};
    if (norm) gamma = widen_row<DT>(*reinterpret_cast<const uint4 *>(p.k_gamma + 8 * l));
    auto load = [&](int t, uint32_t m) {
        Row r = widen_row<DT>(*reinterpret_cast<const uint4 *>(src + static_cast<int64_t>(t) * p.stride));
        if (!values) norm_rotate<LANES>(r, norm, gamma, p.eps, load_turn(p, t, l), p.interleaved != 0, l, m);
        return r;
    };
    auto store = [&](const Row &r, int64_t ph, int o, const Quot &d) {
        *reinterpret_cast<uint2 *>(cache + kv_chunk_offset(ph, P, DIM, o, l >> 1) + 8 * (l & 1)) = row_codes(r, d);
    };

    // runs of one or two tokens: one group each
    for (int i = g; i < p.chunk; i += GROUPS) {
        if (!(lead[i >> 5] >> (i & 31) & 1u)) continue;
        const int n = run_length(i);
        if (n > 2) continue;
        const int t = t0 + i, slot = p.slots[t], o = slot & (P - 1);
        const int64_t ph = static_cast<int64_t>(slot >> p.page_shift) * p.kv_heads + head;
        const float old = o > 0 ? scales[ph] : 0.0f;
        Row a = load(t, mask), b = a;
        if (n == 2) b = load(t + 1, mask);
        uint32_t m = max(row_mag(a), row_mag(b));
#pragma unroll
        for (int x = LANES / 2; x > 0; x >>= 1) m = max(m, __shfl_xor_sync(mask, m, x, LANES));
        const float s = fmaxf(block_scale(m), old);
        const Quot d = Quot::make<FP8L_F32>(s);
        store(a, ph, o, d);
        if (n == 2) store(b, ph, o + 1, d);
        if (l == 0) {
            scales[ph] = s;
            if (o > 0 && s > old) jobs[atomicAdd(&num_jobs, 1)] = Recast{ph, o, old, s};
        }
    }
    // longer runs: the block's groups take rows g, g + GROUPS, ...
    for (int w = 0; w < 2; ++w) {
        for (uint32_t bits = lead[w]; bits != 0u; bits &= bits - 1u) {
            const int i = 32 * w + __ffs(static_cast<int>(bits)) - 1;
            const int n = run_length(i);
            if (n <= 2) continue;
            const int t = t0 + i, slot = p.slots[t], o = slot & (P - 1);
            const int64_t ph = static_cast<int64_t>(slot >> p.page_shift) * p.kv_heads + head;
            const float old = o > 0 ? scales[ph] : 0.0f;
            Row x[ROWS];
            uint32_t m = 0;
#pragma unroll
            for (int j = 0; j < ROWS; ++j) {
                if (g + j * GROUPS < n) {
                    x[j] = load(t + g + j * GROUPS, mask);
                    m = max(m, row_mag(x[j]));
                }
            }
            m = block_max_u32(m, red);
            const float s = fmaxf(block_scale(m), old);
            const Quot d = Quot::make<FP8L_F32>(s);
#pragma unroll
            for (int j = 0; j < ROWS; ++j)
                if (g + j * GROUPS < n) store(x[j], ph, o + g + j * GROUPS, d);
            if (o > 0 && s > old) recast_block<DIM>(cache, Recast{ph, o, old, s}, P);
            __syncthreads();  // every thread has read the old scale and the block maximum
            if (tid == 0) scales[ph] = s;
        }
    }
    __syncthreads();
    for (int j = 0; j < num_jobs; ++j) recast_block<DIM>(cache, jobs[j], P);
}

template <int DT, int DIM>
__device__ void query_rows(const AppendParams &p, int block) {
    constexpr int LANES = DIM / 8, GROUPS = kAppThreads / LANES;
    const int tid = static_cast<int>(threadIdx.x);
    const int l = tid % LANES;
    const uint32_t mask = LANES == 16 ? 0xFFFFu << (tid & 16) : 0xFFu << (tid & 24);
    const int64_t item = static_cast<int64_t>(block) * GROUPS + tid / LANES;
    const int64_t t64 = item / p.head_groups;
    if (t64 >= p.tokens) return;
    const int t = static_cast<int>(t64);
    const int h0 = static_cast<int>(item % p.head_groups) * kAppHeadsPerGroup;
    const int n = min(kAppHeadsPerGroup, p.q_heads - h0);
    const uint16_t *src = p.qkv + static_cast<int64_t>(t) * p.stride + h0 * DIM + 8 * l;
    uint4 u[kAppHeadsPerGroup];
#pragma unroll
    for (int h = 0; h < kAppHeadsPerGroup; ++h)
        u[h] = h < n ? *reinterpret_cast<const uint4 *>(src + h * DIM) : make_uint4(0u, 0u, 0u, 0u);
    const bool norm = p.q_gamma != nullptr;
    Row gamma = {};
    if (norm) gamma = widen_row<DT>(*reinterpret_cast<const uint4 *>(p.q_gamma + 8 * l));
    const Turn turn = load_turn(p, t, l);
    uint16_t *dst = p.q_out + (static_cast<int64_t>(t) * p.q_heads + h0) * DIM + 8 * l;
#pragma unroll
    for (int h = 0; h < kAppHeadsPerGroup; ++h) {
        Row r = widen_row<DT>(u[h]);
        norm_rotate<LANES>(r, norm, gamma, p.eps, turn, p.interleaved != 0, l, mask);
        if (h < n)
            *reinterpret_cast<uint4 *>(dst + h * DIM) =
                make_uint4(narrow2<DT>(r.x[0], r.x[1]), narrow2<DT>(r.x[2], r.x[3]),
                           narrow2<DT>(r.x[4], r.x[5]), narrow2<DT>(r.x[6], r.x[7]));
    }
}

template <int DT, int DIM>
__global__ void __launch_bounds__(kAppThreads) qk_norm_rope_append_kernel(const AppendParams p) {
    grid_dependency_sync();
    const int b = static_cast<int>(blockIdx.x);
    if (b < p.kv_blocks)
        append_unit<DT, DIM>(p, b);
    else
        query_rows<DT, DIM>(p, b - p.kv_blocks);
}

}  // namespace
}  // namespace fp8l

extern "C" int fp8_qk_norm_rope_append(const void *qkv, int dtype, int64_t tokens, int64_t qkv_stride,
                                       int64_t q_heads, int64_t kv_heads, int64_t head_dim,
                                       const void *q_gamma, const void *k_gamma, float eps,
                                       const float *cos_sin, int64_t max_positions, int64_t rot,
                                       int interleaved, const int32_t *positions, const int32_t *slots,
                                       void *q_out, uint8_t *k_cache, uint8_t *v_cache, float *k_scale,
                                       float *v_scale, int64_t num_pages, int64_t page_size, void *stream) {
    using namespace fp8l;
    if (dtype != FP8L_F16 && dtype != FP8L_BF16) return FP8L_EINVAL;
    if (!(eps >= 0.0f) || eps > 3.0e38f) return FP8L_EINVAL;
    if (tokens < 0 || tokens > INT32_MAX || (head_dim != 64 && head_dim != 128) || kv_heads < 1 ||
        q_heads < kv_heads || q_heads % kv_heads != 0 || (q_heads + 2 * kv_heads) * head_dim > (1 << 20) ||
        qkv_stride < (q_heads + 2 * kv_heads) * head_dim || qkv_stride % 8 != 0 || rot < 0 || rot > head_dim ||
        rot % 16 != 0 || (rot > 0 && (max_positions < 1 || max_positions > INT32_MAX)) ||
        !kv_page_size_ok(page_size) || num_pages < 1 || num_pages > INT32_MAX / page_size)
        return FP8L_ESHAPE;
    if (!k_cache || !v_cache || !k_scale || !v_scale || (rot > 0 && (!cos_sin || (!positions && tokens > 0))) ||
        (tokens > 0 && (!qkv || !q_out || !slots)))
        return FP8L_EINVAL;
    if (!aligned16(qkv) || !aligned16(q_gamma) || !aligned16(k_gamma) || !aligned16(cos_sin) ||
        !aligned16(q_out) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned4(k_scale) ||
        !aligned4(v_scale) || !aligned4(positions) || !aligned4(slots))
        return FP8L_EALIGN;
    if (int st = check_device(nullptr); st != FP8L_OK) return st;
    if (tokens == 0) return FP8L_OK;
    AppendParams p;
    p.qkv = static_cast<const uint16_t *>(qkv);
    p.tokens = static_cast<int>(tokens);
    p.stride = qkv_stride;
    p.q_heads = static_cast<int>(q_heads);
    p.kv_heads = static_cast<int>(kv_heads);
    p.q_gamma = static_cast<const uint16_t *>(q_gamma);
    p.k_gamma = static_cast<const uint16_t *>(k_gamma);
    p.eps = eps;
    p.cos_sin = cos_sin;
    p.max_positions = static_cast<int>(max_positions);
    p.rot = static_cast<int>(rot);
    p.interleaved = interleaved;
    p.positions = positions;
    p.slots = slots;
    p.q_out = static_cast<uint16_t *>(q_out);
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.num_slots = static_cast<int>(num_pages * page_size);
    p.page_shift = __builtin_ctzll(static_cast<unsigned long long>(page_size));
    const int groups = kAppThreads / static_cast<int>(head_dim / 8);
    // few tokens: one run per group of a block; many: longer chunks, since in
    // a prompt only every page_size-th token starts a run
    p.chunk = tokens <= 2048 ? groups : kAppMaxChunk;
    const int64_t kv_blocks = (tokens + p.chunk - 1) / p.chunk * 2 * kv_heads;
    p.head_groups = static_cast<int>((q_heads + kAppHeadsPerGroup - 1) / kAppHeadsPerGroup);
    const int64_t q_blocks = (tokens * p.head_groups + groups - 1) / groups;
    if (kv_blocks + q_blocks > INT32_MAX) return FP8L_ESHAPE;
    p.kv_blocks = static_cast<int>(kv_blocks);
    const dim3 grid(static_cast<unsigned>(kv_blocks + q_blocks));
    auto kernel = dtype == FP8L_BF16 ? (head_dim == 128 ? qk_norm_rope_append_kernel<FP8L_BF16, 128>
                                                        : qk_norm_rope_append_kernel<FP8L_BF16, 64>)
                                     : (head_dim == 128 ? qk_norm_rope_append_kernel<FP8L_F16, 128>
                                                        : qk_norm_rope_append_kernel<FP8L_F16, 64>);
    return launch_dependent(kernel, grid, kAppThreads, 0, as_stream(stream), p);
}
