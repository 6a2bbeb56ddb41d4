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
// spread over the whole block, which reads them twice (maximum, cast), the
// second time from L1.  Tokens that a page already holds are re-cast by the
// whole block when the scale grew: a group alone would read up to 127 rows
// one after the other.
//
// Measured (GB300, replayed from a graph; 8 kv heads of 128, bf16, norms and a
// full rotation): 72 us for 13741 tokens with 32 query heads in pages of 128,
// 4.3 TB/s of the 311 MB it has to move (a plain copy of qkv takes 51 us);
// queries alone take 42 us, 5.4 TB/s, keys and values the rest, bound by
// instructions (two readings, the exact quotient: 0.63 of the issue slots).
// 7.3 us for one token each of 256 sequences with 64 query heads, 3.3 us for
// one: the same append replayed, so that no scale grows.  With the cache put
// back before each call the 256 take 9.1 us when no scale grows, 12.8 when those
// of a random cache do, 23 when every page and head re-casts its earlier tokens
// (a block's pages one after the other).  Holding the rows between the readings took 128 registers and 87 us;
// alternating units and queries over the grid changed nothing.
//
// Codes against a 64-bit computation: of 17.2 M each for 13741 tokens, 17 of
// the keys differ (float32 norm and rotation; 24 with a rounding after every
// operation) and about 10^4 of the values.  Those are ties: a 16-bit
// value over its block's amax / 448 is halfway between two codes in 1 of 190
// cases, and the last bit of either quotient, here or in 64 bits, decides.
#include "kv_device.cuh"
#include "quant_device.cuh"

namespace fp8l {
namespace {

constexpr int kAppThreads = 256;
constexpr int kAppMaxChunk = 64;    // tokens whose runs one block starts
constexpr int kAppHeadsPerGroup = 8;  // query heads of a token per group: loads in flight

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

// One row (a token's head) in a group of DIM / 8 lanes, eight dimensions each
// as float pairs.  kSplit: a lane holds dimensions 4 l .. 4 l + 3 and
// DIM / 2 + 4 l .. + 3, so that a rotation over the whole head in halves has
// both dimensions of a pair in one thread; otherwise 8 l .. 8 l + 7.
enum Layout { kContiguous = 0, kSplit = 1 };

struct Row {
    uint64_t p[4];
};

struct Raw {
    uint32_t w[4];
};

template <int DIM, int LAYOUT>
__device__ __forceinline__ Raw load_raw(const uint16_t *row, int l) {
    Raw r;
    if constexpr (LAYOUT == kSplit) {
        const uint2 a = *reinterpret_cast<const uint2 *>(row + 4 * l);
        const uint2 b = *reinterpret_cast<const uint2 *>(row + DIM / 2 + 4 * l);
        r.w[0] = a.x, r.w[1] = a.y, r.w[2] = b.x, r.w[3] = b.y;
    } else {
        const uint4 a = *reinterpret_cast<const uint4 *>(row + 8 * l);
        r.w[0] = a.x, r.w[1] = a.y, r.w[2] = a.z, r.w[3] = a.w;
    }
    return r;
}

template <int DT>
__device__ __forceinline__ Row widen_row(const Raw &u) {
    Row r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r.p[i] = widen16<DT>(u.w[i]);
    return r;
}

__device__ __forceinline__ float lo_f(uint64_t p) { return __uint_as_float(static_cast<uint32_t>(p)); }
__device__ __forceinline__ float hi_f(uint64_t p) { return __uint_as_float(static_cast<uint32_t>(p >> 32)); }
__device__ __forceinline__ uint64_t pair_of(float a, float b) { return f2_pack(__float_as_uint(a), __float_as_uint(b)); }
__device__ __forceinline__ uint64_t f2_neg(uint64_t a) { return a ^ 0x8000000080000000ull; }

template <int DT>
__device__ __forceinline__ uint32_t narrow2(uint64_t p) {
    if constexpr (DT == FP8L_BF16) {
        __nv_bfloat162 h = __floats2bfloat162_rn(lo_f(p), hi_f(p));
        return *reinterpret_cast<uint32_t *>(&h);
    } else {
        __half2 h = __floats2half2_rn(lo_f(p), hi_f(p));
        return *reinterpret_cast<uint32_t *>(&h);
    }
}

template <int DT, int DIM, int LAYOUT>
__device__ __forceinline__ void store_row16(uint16_t *row, int l, const Row &r) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = narrow2<DT>(r.p[i]);
    if constexpr (LAYOUT == kSplit) {
        *reinterpret_cast<uint2 *>(row + 4 * l) = make_uint2(w[0], w[1]);
        *reinterpret_cast<uint2 *>(row + DIM / 2 + 4 * l) = make_uint2(w[2], w[3]);
    } else {
        *reinterpret_cast<uint4 *>(row + 8 * l) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// Cosines and sines of a token for a lane's rotation pairs: the float pairs
// of its four (kSplit: dimensions 4 l .. of the first half; interleaved:
// pairs 4 l ..) or eight (a partner lane holds the other dimension) angles.
template <int LAYOUT>
struct Turn {
    static constexpr int kPairs = LAYOUT == kSplit ? 2 : 4;
    uint64_t c[kPairs], s[kPairs];
    int half8;  // rot / 16: lanes of the rotated first half (contiguous)
    bool on;    // this lane's dimensions rotate
};

template <int LAYOUT>
__device__ __forceinline__ Turn<LAYOUT> load_turn(const AppendParams &p, int token, int l) {
    Turn<LAYOUT> t;
    t.half8 = p.rot >> 4;
    t.on = 8 * l < p.rot || (LAYOUT == kSplit && p.rot > 0);
#pragma unroll
    for (int i = 0; i < Turn<LAYOUT>::kPairs; ++i) {
        t.c[i] = pair_of(1.0f, 1.0f);
        t.s[i] = 0;
    }
    if (t.on) {
        const int pos = min(max(p.positions[token], 0), p.max_positions - 1);
        const float *row = p.cos_sin + static_cast<int64_t>(pos) * p.rot;
        const float *sin = row + (p.rot >> 1);
        const int i0 = LAYOUT == kSplit || p.interleaved ? 4 * l : 8 * (l < t.half8 ? l : l - t.half8);
        const float4 c0 = *reinterpret_cast<const float4 *>(row + i0);
        const float4 s0 = *reinterpret_cast<const float4 *>(sin + i0);
        t.c[0] = pair_of(c0.x, c0.y), t.c[1] = pair_of(c0.z, c0.w);
        t.s[0] = pair_of(s0.x, s0.y), t.s[1] = pair_of(s0.z, s0.w);
        if constexpr (LAYOUT == kContiguous) {
            if (!p.interleaved) {
                const float4 c1 = *reinterpret_cast<const float4 *>(row + i0 + 4);
                const float4 s1 = *reinterpret_cast<const float4 *>(sin + i0 + 4);
                t.c[2] = pair_of(c1.x, c1.y), t.c[3] = pair_of(c1.z, c1.w);
                t.s[2] = pair_of(s1.x, s1.y), t.s[3] = pair_of(s1.z, s1.w);
            }
        }
    }
    return t;
}

// 1 / sqrt(mean of squares + eps) of the row held by the lanes of `mask`
template <int LANES>
__device__ __forceinline__ float row_rms(const Row &r, float eps, uint32_t mask) {
    const uint64_t a = f2_fma(r.p[1], r.p[1], f2_mul(r.p[0], r.p[0]));
    const uint64_t b = f2_fma(r.p[3], r.p[3], f2_mul(r.p[2], r.p[2]));
    float ss = (lo_f(a) + hi_f(a)) + (lo_f(b) + hi_f(b));
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(mask, ss, o, LANES);
    return rsqrtf(ss * (1.0f / (8 * LANES)) + eps);
}

// x r gamma, gamma first: the product of two 16-bit numbers is exact in float32
__device__ __forceinline__ void scale_row(Row &r, float inv, const Row &gamma) {
    const uint64_t i2 = pair_of(inv, inv);
#pragma unroll
    for (int i = 0; i < 4; ++i) r.p[i] = f2_mul(f2_mul(r.p[i], gamma.p[i]), i2);
}

// (a, b) <- (a cos - b sin, b cos + a sin)
template <int LANES, int LAYOUT>
__device__ __forceinline__ void rotate_row(Row &r, const Turn<LAYOUT> &t, bool interleaved, int l, uint32_t mask) {
    if constexpr (LAYOUT == kSplit) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint64_t a = r.p[i], b = r.p[i + 2];
            r.p[i] = f2_fma(f2_neg(b), t.s[i], f2_mul(a, t.c[i]));
            r.p[i + 2] = f2_fma(a, t.s[i], f2_mul(b, t.c[i]));
        }
    } else if (interleaved) {
        if (t.on) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float a = lo_f(r.p[i]), b = hi_f(r.p[i]);
                const float c = i & 1 ? hi_f(t.c[i >> 1]) : lo_f(t.c[i >> 1]);
                const float s = i & 1 ? hi_f(t.s[i >> 1]) : lo_f(t.s[i >> 1]);
                r.p[i] = pair_of(a * c - b * s, b * c + a * s);
            }
        }
    } else {
        const bool low = l < t.half8;
        const int partner = !t.on ? l : (low ? l + t.half8 : l - t.half8);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint64_t other = __shfl_sync(mask, r.p[i], partner, LANES);
            if (t.on) r.p[i] = f2_fma(low ? f2_neg(other) : other, t.s[i], f2_mul(r.p[i], t.c[i]));
        }
    }
}

__device__ __forceinline__ uint32_t row_mag(const Row &r) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        m = max(m, max(static_cast<uint32_t>(r.p[i]) & 0x7FFFFFFFu, static_cast<uint32_t>(r.p[i] >> 32) & 0x7FFFFFFFu));
    return m;
}

__device__ __forceinline__ uint2 row_codes(const Row &r, const Quot &d) {
    const uint4 a = make_uint4(static_cast<uint32_t>(r.p[0]), static_cast<uint32_t>(r.p[0] >> 32),
                               static_cast<uint32_t>(r.p[1]), static_cast<uint32_t>(r.p[1] >> 32));
    const uint4 b = make_uint4(static_cast<uint32_t>(r.p[2]), static_cast<uint32_t>(r.p[2] >> 32),
                               static_cast<uint32_t>(r.p[3]), static_cast<uint32_t>(r.p[3] >> 32));
    return make_uint2(codes_of_word<FP8L_F32, false>(a, d).x, codes_of_word<FP8L_F32, false>(b, d).x);
}

// The scale of a block of this largest magnitude.  A NaN among the values (the
// largest of all bit patterns) stays in it: dropped, it would leave the
// smallest scale, and the block's other values would be crushed by it.
__device__ __forceinline__ float block_scale(uint32_t amax_bits) {
    return max_nan(__fdiv_rn(__uint_as_float(amax_bits), kE4M3Max), kKvMinScale);
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

template <int DT, int DIM, int LAYOUT>
__device__ void append_unit(const AppendParams &p, int unit) {
    constexpr int LANES = DIM / 8, GROUPS = kAppThreads / LANES, BATCH = 2;
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
    const uint16_t *src = p.qkv + (p.q_heads + (values ? p.kv_heads : 0) + head) * DIM;
    const bool norm = !values && p.k_gamma != nullptr;
    Row gamma = {};
    if (norm) gamma = widen_row<DT>(load_raw<DIM, LAYOUT>(p.k_gamma, l));
    auto load = [&](int t) { return load_raw<DIM, LAYOUT>(src + static_cast<int64_t>(t) * p.stride, l); };
    // the float32 row of a token
    auto finish = [&](const Raw &u, const Turn<LAYOUT> &turn) {
        Row r = widen_row<DT>(u);
        if (norm) scale_row(r, row_rms<LANES>(r, p.eps, mask), gamma);
        if (!values && p.rot > 0) rotate_row<LANES, LAYOUT>(r, turn, p.interleaved != 0, l, mask);
        return r;
    };
    const Turn<LAYOUT> none = {};
    auto store = [&](const Row &r, int64_t ph, int o, const Quot &d) {
        const uint2 c = row_codes(r, d);
        if constexpr (LAYOUT == kSplit) {
            uint8_t *at = cache + kv_chunk_offset(ph, P, DIM, o, l >> 2) + 4 * (l & 3);
            *reinterpret_cast<uint32_t *>(at) = c.x;
            *reinterpret_cast<uint32_t *>(at + DIM / 32 * 128) = c.y;
        } else {
            *reinterpret_cast<uint2 *>(cache + kv_chunk_offset(ph, P, DIM, o, l >> 1) + 8 * (l & 1)) = c;
        }
    };

    // runs of one or two tokens: one group each
    for (int i = g; i < p.chunk; i += GROUPS) {
        if (!(lead[i >> 5] >> (i & 31) & 1u)) continue;
        const int n = run_length(i);
        if (n > 2) continue;
        const int t = t0 + i, slot = p.slots[t], o = slot & (P - 1);
        const int64_t ph = static_cast<int64_t>(slot >> p.page_shift) * p.kv_heads + head;
        const float old = o > 0 ? scales[ph] : 0.0f;
        const Row a = finish(load(t), values ? none : load_turn<LAYOUT>(p, t, l));
        const Row b = n == 2 ? finish(load(t + 1), values ? none : load_turn<LAYOUT>(p, t + 1, l)) : a;
        uint32_t m = max(row_mag(a), row_mag(b));
#pragma unroll
        for (int x = LANES / 2; x > 0; x >>= 1) m = max(m, __shfl_xor_sync(mask, m, x, LANES));
        const float s = max_nan(block_scale(m), old);
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
            // rows in batches, twice: the second reading finds them in L1 (a
            // page's rows of a head are 32 KB at most), and few registers
            // leave room for the blocks of queries on the SM
            auto each_row = [&](auto &&use) {
#pragma unroll 1
                for (int j0 = g; j0 < n; j0 += BATCH * GROUPS) {
                    Raw u[BATCH];
#pragma unroll
                    for (int j = 0; j < BATCH; ++j)
                        if (j0 + j * GROUPS < n) u[j] = load(t + j0 + j * GROUPS);
#pragma unroll
                    for (int j = 0; j < BATCH; ++j) {
                        const int i = j0 + j * GROUPS;
                        if (i < n) use(finish(u[j], values ? none : load_turn<LAYOUT>(p, t + i, l)), i);
                    }
                }
            };
            uint32_t m = 0;
            each_row([&](const Row &r, int) { m = max(m, row_mag(r)); });
            m = block_max_u32(m, red);
            const float s = max_nan(block_scale(m), old);
            const Quot d = Quot::make<FP8L_F32>(s);
            each_row([&](const Row &r, int i) { store(r, ph, o + i, d); });
            if (o > 0 && s > old) recast_block<DIM>(cache, Recast{ph, o, old, s}, P);
            __syncthreads();  // every thread has read the old scale and the block maximum
            if (tid == 0) scales[ph] = s;
        }
    }
    __syncthreads();
    for (int j = 0; j < num_jobs; ++j) recast_block<DIM>(cache, jobs[j], P);
}

template <int DT, int DIM, int LAYOUT>
__device__ void query_rows(const AppendParams &p, int block) {
    constexpr int LANES = DIM / 8, GROUPS = kAppThreads / LANES;
    const int tid = static_cast<int>(threadIdx.x);
    const int l = tid % LANES;
    const uint32_t mask = LANES == 16 ? 0xFFFFu << (tid & 16) : 0xFFu << (tid & 24);
    const int64_t item = static_cast<int64_t>(block) * GROUPS + tid / LANES;
    const int64_t t64 = item / p.head_groups;
    if (t64 >= p.tokens) return;
    const int t = static_cast<int>(t64);
    const int h0 = static_cast<int>(item - t64 * p.head_groups) * kAppHeadsPerGroup;
    const int n = min(kAppHeadsPerGroup, p.q_heads - h0);
    const uint16_t *src = p.qkv + static_cast<int64_t>(t) * p.stride + h0 * DIM;
    Raw u[kAppHeadsPerGroup];
#pragma unroll
    for (int h = 0; h < kAppHeadsPerGroup; ++h) u[h] = load_raw<DIM, LAYOUT>(src + (h < n ? h : 0) * DIM, l);
    const bool norm = p.q_gamma != nullptr;
    Row gamma = {};
    if (norm) gamma = widen_row<DT>(load_raw<DIM, LAYOUT>(p.q_gamma, l));
    Turn<LAYOUT> turn;
    if (p.rot > 0) turn = load_turn<LAYOUT>(p, t, l);
    uint16_t *dst = p.q_out + (static_cast<int64_t>(t) * p.q_heads + h0) * DIM;
#pragma unroll
    for (int h = 0; h < kAppHeadsPerGroup; ++h) {
        Row r = widen_row<DT>(u[h]);
        if (norm) scale_row(r, row_rms<LANES>(r, p.eps, mask), gamma);
        if (p.rot > 0) rotate_row<LANES, LAYOUT>(r, turn, p.interleaved != 0, l, mask);
        if (h < n) store_row16<DT, DIM, LAYOUT>(dst + h * DIM, l, r);
    }
}

template <int DT, int DIM, int LAYOUT>
__global__ void __launch_bounds__(kAppThreads, 4) qk_norm_rope_append_kernel(const AppendParams p) {
    grid_dependency_sync();
    const int b = static_cast<int>(blockIdx.x);
    if (b < p.kv_blocks)
        append_unit<DT, DIM, LAYOUT>(p, b);
    else
        query_rows<DT, DIM, LAYOUT>(p, b - p.kv_blocks);
}

template <int DT, int DIM>
int launch_append(const AppendParams &p, dim3 grid, cudaStream_t stream) {
    // both dimensions of a rotation pair in one thread, where the halves of
    // the whole head rotate against each other: 72 us against 104 for 13741
    // tokens, 7.2 against 8.2 for 256 decoding
    if (p.rot == DIM && !p.interleaved)
        return launch_dependent(qk_norm_rope_append_kernel<DT, DIM, kSplit>, grid, kAppThreads, 0, stream, p);
    return launch_dependent(qk_norm_rope_append_kernel<DT, DIM, kContiguous>, grid, kAppThreads, 0, stream, p);
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
        q_heads < kv_heads || q_heads > (1 << 20) || q_heads % kv_heads != 0 ||
        (q_heads + 2 * kv_heads) * head_dim > (1 << 20) ||
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
    // a prompt only every page_size-th token starts a run.  Measured (us, short
    // chunks / long): 256 decoding 7.2 / 17.7, seven prompts of 250 tokens 16.9 /
    // 19.0, of 400 tokens 20.9 / 18.9, of 900 42 / 35, 13741 tokens 87 / 72
    p.chunk = tokens <= 2048 ? groups : kAppMaxChunk;
    const int64_t kv_blocks = (tokens + p.chunk - 1) / p.chunk * 2 * kv_heads;
    p.head_groups = static_cast<int>((q_heads + kAppHeadsPerGroup - 1) / kAppHeadsPerGroup);
    const int64_t q_blocks = (tokens * p.head_groups + groups - 1) / groups;
    if (kv_blocks + q_blocks > INT32_MAX) return FP8L_ESHAPE;
    p.kv_blocks = static_cast<int>(kv_blocks);
    const dim3 grid(static_cast<unsigned>(kv_blocks + q_blocks));
    const cudaStream_t st = as_stream(stream);
    if (dtype == FP8L_BF16)
        return head_dim == 128 ? launch_append<FP8L_BF16, 128>(p, grid, st) : launch_append<FP8L_BF16, 64>(p, grid, st);
    return head_dim == 128 ? launch_append<FP8L_F16, 128>(p, grid, st) : launch_append<FP8L_F16, 64>(p, grid, st);
}
