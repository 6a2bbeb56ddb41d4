// Attention of a few query rows per kv head (decode, drafted tokens) on the
// tcgen05 tensor cores, straight from the cache's codes.
//
// A unit of work is a tile of 128 keys of one request and kv head.  Its
// query rows (tokens x heads of the group, at most ROWS) are the MMA's N side
// and the keys its M side, so the tile's scores land transposed in tensor
// memory, one key per lane:
//   S^T [128 keys x rows]  = K [128 x D] Q^T        (kind::f8f6f4, D / 32 MMAs)
//   O^T [D x rows]        += V^T [D x 128] W^T      (kind::f8f6f4, 4 MMAs)
// K is read as a K-major operand and V as an M-major one from the same
// 128-byte core matrices, exactly as the cache stores them: no code is ever
// widened by a CUDA core, and a tile costs its bytes.
//
// Precision.  The 16-bit query and the float32 weights enter as sums of E4M3
// parts in columns of their own, each part the rounding of 16 times what the
// parts before it left over: q, scaled by a power of two, is exact in two
// parts for bf16 (an 8-bit significand is 4 + 4 bits with a sign) and in
// three for fp16 (11 bits); a weight in three parts has 12 bits, or 2^-25 of
// the running maximum.  The part columns are summed in float32.
//
// Softmax with block scales.  With k_j = sk c_j and v_j = sv d_j per page,
//   t_j = log2(e) sm_scale q.k_j + log2 sv_j,   w_j = 2^(t_j - m),  m ~ max t
//   O = sum_j w_j d_j,   l = sum_j w_j / sv_j,   out = O / l
// so a weight that multiplies codes is at most 2 whatever the scales of the
// pages, and no scale has to be applied to V.  The reference m moves only
// when a score passes it by more than 1 (found by an OR over the tile's
// threads in the barrier that a maximum would need anyway); then l and the
// accumulator in tensor memory are rescaled.
//
// Work.  The tiles of all requests and kv heads are one line, cut into equal
// pieces for the CTAs of one resident wave, whatever the lengths.  A request
// and head inside one piece is written out directly; one that spans pieces
// leaves its partial (m, l, O) in the workspace and the last CTA to arrive
// adds the partials in CTA order, so the result does not depend on timing.
//
// Roles (192 threads, two CTAs per SM): warps 0-3 softmax and epilogue (warp
// w owns tensor-memory lanes 32 w ..), warp 4 copies (one untiled bulk copy
// per page, keys and values; the page's scales by cp.async), warp 5 issues the
// MMAs, the next tile's scores before this tile's values.
#pragma once

#include "kv_attention_params.cuh"

namespace fp8l {
namespace {

constexpr int kDecTile = 128;      // keys per tile = MMA M
constexpr int kDecThreads = 192;
constexpr int kDecMaxStages = 6;
constexpr int kDecMinTiles = 2;    // tiles per CTA below which fewer CTAs run
constexpr int kDecMaxCtas = 2 * 160;

template <int QDT, int ROWS>
struct DecShape {
    static constexpr int kQParts = QDT == FP8L_BF16 ? 2 : 3;
    static constexpr int kWParts = 3;
    static constexpr int kSCols = (ROWS * kQParts + 15) / 16 * 16;
    static constexpr int kOCols = (ROWS * kWParts + 15) / 16 * 16;
    // two score buffers, one when they would not fit half the tensor memory
    static constexpr int kSBufs = 2 * kSCols + kOCols <= 256 ? 2 : 1;
    static constexpr int kUsedCols = kSBufs * kSCols + kOCols;
    static constexpr int kTmemCols = kUsedCols <= 64 ? 64 : (kUsedCols <= 128 ? 128 : 256);
    static_assert(kUsedCols <= 256, "two CTAs share an SM's tensor memory");
};

// Shared memory after the stages
template <int QDT, int DIM, int ROWS>
struct DecSmem {
    using Sh = DecShape<QDT, ROWS>;
    static constexpr int kStageBytes = 2 * kDecTile * DIM;  // keys, values
    static constexpr int kQBytes = Sh::kSCols * DIM;        // per buffer
    static constexpr int kWBytes = kDecTile * Sh::kOCols;   // per buffer
    static constexpr int kQOff = 0;
    static constexpr int kWOff = kQOff + 2 * kQBytes;
    static constexpr int kScaleOff = kWOff + 2 * kWBytes;                  // [stage][2][8] floats
    static constexpr int kQfOff = kScaleOff + kDecMaxStages * 16 * 4;      // [2][ROWS] floats
    static constexpr int kRedOff = kQfOff + 2 * ROWS * 4;                  // [4][ROWS] floats
    static constexpr int kRefOff = kRedOff + 4 * ROWS * 4;                 // [2][ROWS] floats: m, l
    static constexpr int kBarOff = (kRefOff + 2 * ROWS * 4 + 15) / 16 * 16;
    static constexpr int kBars = 2 * kDecMaxStages + 4 + 4 + 2 + 1;
    static constexpr int kMiscOff = kBarOff + kBars * 8;
    static constexpr int kFixedBytes = kMiscOff + 64;
    // the M-side read of a 64-dimension V covers 512 bytes past the last stage
    static_assert(2 * kQBytes >= 512, "reads past the last stage stay inside");
};

__device__ __forceinline__ uint64_t core_desc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
    return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(lbo >> 4) << 16) |
           (static_cast<uint64_t>(sbo >> 4) << 32) | (static_cast<uint64_t>(1) << 46);
}

__device__ __forceinline__ void dec_mma(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc,
                                        uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void bulk_copy(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
        "l"(src), "r"(bytes), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void tmem_ld_n(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

__device__ __forceinline__ void tmem_st_n(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// COLS columns of this thread's lane
template <int COLS>
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, float (&v)[COLS]) {
    static_assert(COLS % 16 == 0, "");
    uint32_t r[COLS / 16][16];
#pragma unroll
    for (int c = 0; c < COLS / 16; ++c) tmem_ld_n(taddr + 16 * c, r[c]);
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int c = 0; c < COLS; ++c) v[c] = __uint_as_float(r[c / 16][c % 16]);
}

// barrier over the 128 softmax threads
__device__ __forceinline__ void softmax_sync() { asm volatile("barrier.cta.sync 1, 128;" ::: "memory"); }

__device__ __forceinline__ bool softmax_any(bool x) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, 1, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(x ? 1u : 0u)
        : "memory");
    return r != 0u;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// E4M3 codes of two values (a in the low byte) and what they leave over,
// times 16
__device__ __forceinline__ uint32_t take_part(float &a, float &b) {
    uint32_t c;
    asm("{\n\t.reg .b16 h;\n\tcvt.rn.satfinite.e4m3x2.f32 h, %2, %1;\n\tcvt.u32.u16 %0, h;\n\t}"
        : "=r"(c)
        : "f"(a), "f"(b));
    uint32_t f;
    asm("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(f) : "r"(c));
    const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&f));
    a = (a - v.x) * 16.0f;
    b = (b - v.y) * 16.0f;
    return c;
}

// Exponent e with 2^7 <= m 2^e < 2^8, at most 120 (rows below 2^-113 lose
// their last bits) so that 2^-e stays a normal float32; m >= 0
__device__ __forceinline__ int part_exponent(float m) {
    return min(134 - static_cast<int>(__float_as_uint(m) >> 23), 120);
}

// A piece of one request and kv head: key tiles [tile, end) of its [begin, stop)
struct DecSegment {
    int r, g;
    int n, row0;        // the request's new tokens, their first row
    int first, keys;    // first visible key, end of the keys
    int tile, end, begin, stop;
    long long at;       // number of `tile` in the line of tiles
};

struct DecRange {
    int n, row0, first, keys, begin, tiles;
};

// The key tiles of a request (0 when it has no rows); a request whose rows
// see nothing has one tile with no valid key, which writes its zeros.
__device__ __forceinline__ DecRange dec_range(const AttnParams &p, int r) {
    DecRange d;
    const int a = min(max(p.q_offsets[r], 0), p.tokens), b = min(max(p.q_offsets[r + 1], 0), p.tokens);
    const int64_t cap = static_cast<int64_t>(p.table_width) << p.page_shift;
    const int L = max(p.kv_lens[r], 0);
    d.keys = static_cast<int64_t>(L) < cap ? L : static_cast<int>(cap);
    d.n = b - a;
    d.row0 = a;
    const int pos = d.keys - d.n;
    d.first = p.window > 0 ? max(0, pos - p.window + 1) : 0;
    d.begin = d.first / kDecTile;
    d.tiles = d.n > 0 ? max((d.keys + kDecTile - 1) / kDecTile - d.begin, 1) : 0;
    return d;
}

// Walks the segments of a CTA's piece [at, end) of the line of tiles.
struct DecWalk {
    long long at, left;  // number of the next tile, tiles still to hand out
    int r, g, offset;    // next tile: offset in request r, head g
    __device__ __forceinline__ bool next(const AttnParams &p, DecSegment &s) {
        if (left <= 0) return false;
        DecRange d = dec_range(p, r);
        while (d.tiles == 0) {
            if (++r >= p.requests) return false;
            d = dec_range(p, r);
        }
        s.r = r;
        s.g = g;
        s.n = d.n;
        s.row0 = d.row0;
        s.first = d.first;
        s.keys = d.keys;
        s.begin = d.begin;
        s.stop = d.begin + d.tiles;
        s.tile = d.begin + offset;
        const long long take = min(static_cast<long long>(d.tiles - offset), left);
        s.end = s.tile + static_cast<int>(take);
        s.at = at;
        at += take;
        left -= take;
        offset += static_cast<int>(take);
        if (offset == d.tiles) {
            offset = 0;
            if (++g == p.kv_heads) {
                g = 0;
                ++r;
                if (r >= p.requests) left = 0;
            }
        }
        return true;
    }
};

// Exclusive prefix (plus the block's total in *total) of one value per thread
__device__ __forceinline__ long long dec_scan(long long v, long long *red, long long *total) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    long long inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xFFFFFFFFu, inc, o);
        if (lane >= o) inc += x;
    }
    __syncthreads();
    if (lane == 31) red[warp] = inc;
    __syncthreads();
    long long before = 0, sum = 0;
#pragma unroll
    for (int w = 0; w < kDecThreads / 32; ++w) {
        if (w < warp) before += red[w];
        sum += red[w];
    }
    *total = sum;
    return before + inc - v;
}

// out and lse of a request and head from its CTAs' partials c0 .. c1, in CTA
// order: a warp per row, DIM / 32 dimensions per lane, 32 partials' factors
// at a time in the lanes.
template <int DIM, int ROWS, typename Partial>
__device__ __forceinline__ void merge_partials(const AttnParams &p, const DecSegment &s, int rows, int group,
                                               long long c0, long long c1, const Partial &partial) {
    constexpr int V = DIM / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int parts = static_cast<int>(c1 - c0 + 1);
    for (int r = warp; r < rows; r += 4) {
        float top = -INFINITY;
        for (int c = lane; c < parts; c += 32) top = fmaxf(top, __ldcg(partial(c0 + c) + ROWS * DIM + 2 * r));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
        float sum = 0.0f, acc[V] = {};
        for (int b = 0; b < parts; b += 32) {
            float e = 0.0f;
            if (b + lane < parts) {
                const float *q = partial(c0 + b + lane) + ROWS * DIM + 2 * r;
                const float2 ml = __ldcg(reinterpret_cast<const float2 *>(q));
                e = ml.x == -INFINITY ? 0.0f : ex2(ml.x - top);
                sum = fmaf(ml.y, e, sum);
            }
            const int n = min(32, parts - b);
#pragma unroll 8
            for (int k = 0; k < n; ++k) {
                const float ek = __shfl_sync(0xFFFFFFFFu, e, k);
                const float *q = partial(c0 + b + k) + r * DIM + V * lane;
                if constexpr (V == 4) {
                    const float4 v = __ldcg(reinterpret_cast<const float4 *>(q));
                    acc[0] = fmaf(v.x, ek, acc[0]);
                    acc[1] = fmaf(v.y, ek, acc[1]);
                    acc[2] = fmaf(v.z, ek, acc[2]);
                    acc[3] = fmaf(v.w, ek, acc[3]);
                } else {
                    const float2 v = __ldcg(reinterpret_cast<const float2 *>(q));
                    acc[0] = fmaf(v.x, ek, acc[0]);
                    acc[1] = fmaf(v.y, ek, acc[1]);
                }
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        const int token = s.row0 + r / group, head = s.g * group + r % group;
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = sum > 0.0f ? acc[i] / sum : 0.0f;
        attn_store<V>(p, token, head, DIM, V * lane, acc);
        if (lane == 0 && p.lse != nullptr) attn_store_lse(p, token, head, top, sum);
    }
}

template <int QDT, int DIM, int ROWS>
__global__ void __launch_bounds__(kDecThreads, 2) kv_attention_decode_kernel(const AttnParams p) {
    using Sh = DecShape<QDT, ROWS>;
    using Sm = DecSmem<QDT, DIM, ROWS>;
    extern __shared__ __align__(128) uint8_t dec_smem[];
    __shared__ long long scan_red[kDecThreads / 32];
    __shared__ long long start_left;
    __shared__ int start_r, start_g, start_offset, merge_now;
    const uint32_t sbase = smem_u32(dec_smem);
    const int S = p.stages;
    const uint32_t fixed = sbase + static_cast<uint32_t>(S) * Sm::kStageBytes;
    uint8_t *fixed_ptr = dec_smem + static_cast<size_t>(S) * Sm::kStageBytes;
    const uint32_t bars = fixed + Sm::kBarOff;
    auto full_bar = [&](int s) { return bars + 8u * s; };
    auto empty_bar = [&](int s) { return bars + 8u * (kDecMaxStages + s); };
    auto sfull_bar = [&](int b) { return bars + 8u * (2 * kDecMaxStages + b); };
    auto sempty_bar = [&](int b) { return bars + 8u * (2 * kDecMaxStages + 2 + b); };
    auto wfull_bar = [&](int b) { return bars + 8u * (2 * kDecMaxStages + 4 + b); };
    auto wfree_bar = [&](int b) { return bars + 8u * (2 * kDecMaxStages + 6 + b); };
    auto qfull_bar = [&](int b) { return bars + 8u * (2 * kDecMaxStages + 8 + b); };
    const uint32_t done_bar = bars + 8u * (2 * kDecMaxStages + 10);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(fixed_ptr + Sm::kMiscOff);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full_bar(s), 1 + 32);  // expected bytes, and the lanes' scale copies
            mbar_init(empty_bar(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(sfull_bar(b), 1);
            mbar_init(sempty_bar(b), 128);
            mbar_init(wfull_bar(b), 128);
            mbar_init(wfree_bar(b), 1);
            mbar_init(qfull_bar(b), 128);
        }
        mbar_init(done_bar, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    // columns that no row uses stay zero: queries and weights
    for (int i = static_cast<int>(threadIdx.x); i < (2 * Sm::kQBytes + 2 * Sm::kWBytes) / 16; i += kDecThreads)
        reinterpret_cast<uint4 *>(fixed_ptr)[i] = make_uint4(0u, 0u, 0u, 0u);
    if (warp == 5) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(tmem_slot)),
                     "r"(Sh::kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    grid_dependency_sync();

    // the line of tiles, and this CTA's piece of it
    long long total = 0;
    {
        long long mine = 0;
        for (int r = static_cast<int>(threadIdx.x); r < p.requests; r += kDecThreads)
            mine += static_cast<long long>(dec_range(p, r).tiles) * p.kv_heads;
        dec_scan(mine, scan_red, &total);
    }
    // fewer CTAs when each would get less than kDecMinTiles
    const long long ctas = max(min(static_cast<long long>(gridDim.x), total / kDecMinTiles),
                               min(static_cast<long long>(gridDim.x), min(total, 1LL)));
    const long long cta = static_cast<long long>(blockIdx.x);
    const bool idle = cta >= ctas;
    const long long w0 = idle ? 0 : total * cta / ctas, w1 = idle ? 0 : total * (cta + 1) / ctas;
    if (!idle) {
        long long carry = 0;
        for (int r0 = 0; r0 < p.requests; r0 += kDecThreads) {
            const int r = r0 + static_cast<int>(threadIdx.x);
            const int tiles = r < p.requests ? dec_range(p, r).tiles : 0;
            long long sum;
            const long long n = static_cast<long long>(tiles) * p.kv_heads;
            const long long before = carry + dec_scan(n, scan_red, &sum);
            if (n > 0 && before <= w0 && w0 < before + n) {
                start_r = r;
                start_g = static_cast<int>((w0 - before) / tiles);
                start_offset = static_cast<int>((w0 - before) % tiles);
                start_left = w1 - w0;
            }
            carry += sum;
            if (carry > w0) break;
        }
    } else if (threadIdx.x == 0) {
        start_r = start_g = start_offset = 0;
        start_left = 0;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const uint32_t o_tmem = tmem + Sh::kSBufs * Sh::kSCols;
    DecWalk walk{w0, start_left, start_r, start_g, start_offset};
    const int P = 1 << p.page_shift;
    const int group = p.q_heads / p.kv_heads;

    if (warp == 4) {
        // ---------------------------------------------------------- copies
        int stage = 0;
        uint32_t phase = 0, issued = 0, issued_parity = 0;
        const int per_tile = kDecTile >> p.page_shift;  // pages of a tile, at most 8
        DecSegment s;
        bool ok = true;
        while (ok && walk.next(p, s)) {
            const int32_t *table = p.block_table + static_cast<int64_t>(s.r) * p.table_width;
            // lanes 0-7 keys of page lane, lanes 8-15 values of page lane - 8
            const int i = lane & 7;
            auto block_of = [&](int tile) { return tile * per_tile + i; };
            auto wanted = [&](int tile) {
                const int b = block_of(tile);
                return lane < 16 && i < per_tile && (static_cast<int64_t>(b) << p.page_shift) < s.keys &&
                       (static_cast<int64_t>(b + 1) << p.page_shift) > s.first;
            };
            int page = wanted(s.tile) ? table[block_of(s.tile)] : 0;
            for (int tile = s.tile; tile < s.end; ++tile) {
                const bool mine = wanted(tile);
                const int64_t ph = static_cast<int64_t>(min(max(page, 0), p.num_pages - 1)) * p.kv_heads + s.g;
                // the next tile's pages, while this one waits for its stage
                if (tile + 1 < s.end) page = wanted(tile + 1) ? table[block_of(tile + 1)] : 0;
                uint32_t bytes = 0;
                if (mine) {
                    const int in_page = min(s.keys - (block_of(tile) << p.page_shift), P);
                    bytes = static_cast<uint32_t>((in_page + 7) / 8 * 8 * DIM);
                }
                uint32_t sum = bytes;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
                ok = mbar_wait(empty_bar(stage), phase ^ 1u, abort_flag, p.status, p.wait_cycles);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                const uint32_t dst = sbase + static_cast<uint32_t>(stage) * Sm::kStageBytes +
                                     (lane >= 8 ? kDecTile * DIM : 0) + static_cast<uint32_t>(i * P * DIM);
                if (lane == 0) mbar_expect_tx(full_bar(stage), sum);
                __syncwarp();
                if (mine) {
                    bulk_copy(dst, (lane < 8 ? p.k_cache : p.v_cache) + ph * P * DIM, bytes, full_bar(stage));
                    const float *scale = (lane < 8 ? p.k_scale : p.v_scale) + ph;
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(
                                     fixed + Sm::kScaleOff + static_cast<uint32_t>((stage * 16 + lane) * 4)),
                                 "l"(scale)
                                 : "memory");
                }
                asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(full_bar(stage))
                             : "memory");
                issued |= 1u << stage;
                issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
                if (++stage == S) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
        // every copy lands before the CTA exits
        for (int s2 = 0; s2 < S; ++s2)
            if (issued & (1u << s2)) mbar_wait_drain(full_bar(s2), (issued_parity >> s2) & 1u, p.status);
    } else if (warp == 5) {
        // ---------------------------------------------------------- MMAs
        if (lane == 0) {
            const uint32_t idesc_s = (1u << 4) | (static_cast<uint32_t>(Sh::kSCols >> 3) << 17) | (8u << 24);
            const uint32_t idesc_o = (1u << 4) | (1u << 15) | (1u << 16) |
                                     (static_cast<uint32_t>(Sh::kOCols >> 3) << 17) | (8u << 24);
            bool ok = true;
            if (p.stall & kStallMma) ok = mbar_wait(done_bar, 0, abort_flag, p.status, p.wait_cycles);
            int stage = 0, prev_stage = 0, i = 0, segment = 0;
            uint32_t phase = 0;
            bool prev_first = false;
            auto values = [&](int k) {  // O += V^T W^T of tile number k
                const int b = k & 1;
                if (!mbar_wait_fast(wfull_bar(b), (k >> 1) & 1u, abort_flag, p.status, p.wait_cycles)) return false;
                tc_fence_after();
                const uint32_t v = sbase + static_cast<uint32_t>(prev_stage) * Sm::kStageBytes + kDecTile * DIM;
                const uint32_t w = fixed + Sm::kWOff + static_cast<uint32_t>(b) * Sm::kWBytes;
#pragma unroll
                for (int j = 0; j < kDecTile / 32; ++j)
                    dec_mma(o_tmem, core_desc(v + 32u * DIM * j, 8 * DIM, 128),
                            core_desc(w + 32u * Sh::kOCols * j, 8 * Sh::kOCols, 128), idesc_o,
                            (prev_first && j == 0) ? 0u : 1u);
                mma_commit(wfree_bar(b));
                mma_commit(empty_bar(prev_stage));
                return true;
            };
            DecSegment s;
            while (ok && walk.next(p, s)) {
                const int qb = segment & 1;
                ok = mbar_wait_fast(qfull_bar(qb), (segment >> 1) & 1u, abort_flag, p.status, p.wait_cycles);
                for (int tile = s.tile; ok && tile < s.end; ++tile, ++i) {
                    const int b = Sh::kSBufs == 2 ? (i & 1) : 0;
                    const uint32_t use = static_cast<uint32_t>(Sh::kSBufs == 2 ? i >> 1 : i);
                    ok = mbar_wait_fast(full_bar(stage), phase, abort_flag, p.status, p.wait_cycles) &&
                         mbar_wait_fast(sempty_bar(b), (use & 1u) ^ 1u, abort_flag, p.status, p.wait_cycles);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t k = sbase + static_cast<uint32_t>(stage) * Sm::kStageBytes;
                    const uint32_t q = fixed + Sm::kQOff + static_cast<uint32_t>(qb) * Sm::kQBytes;
#pragma unroll
                    for (int j = 0; j < DIM / 32; ++j)
                        dec_mma(tmem + static_cast<uint32_t>(b * Sh::kSCols), core_desc(k + 256u * j, 128, 8 * DIM),
                                core_desc(q + 256u * j, 128, 8 * DIM), idesc_s, j == 0 ? 0u : 1u);
                    mma_commit(sfull_bar(b));
                    if (i > 0) ok = values(i - 1);
                    prev_stage = stage;
                    prev_first = tile == s.tile;
                    if (++stage == S) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                ++segment;
            }
            if (ok && i > 0) values(i - 1);
            mma_commit(done_bar);
        }
        __syncwarp();
    } else {
        // ---------------------------------------------------------- softmax
        const int tid = static_cast<int>(threadIdx.x);
        const uint32_t lane_addr = static_cast<uint32_t>(warp * 32) << 16;
        float *qf = reinterpret_cast<float *>(fixed_ptr + Sm::kQfOff);
        float *red = reinterpret_cast<float *>(fixed_ptr + Sm::kRedOff);
        float *ref = reinterpret_cast<float *>(fixed_ptr + Sm::kRefOff);
        const float *scales = reinterpret_cast<const float *>(fixed_ptr + Sm::kScaleOff);
        bool ok = true;

        // The segment's queries as E4M3 parts in buffer b, and the factor of
        // each row's scores: LANES lanes hold a row, eight dimensions each.
        auto load_queries = [&](const DecSegment &s, int b) {
            constexpr int LANES = DIM / 8, AT_ONCE = 128 / LANES;
            const int l = tid % LANES;
            const int rows = min(s.n * group, ROWS);
            for (int row = tid / LANES; row < ROWS; row += AT_ONCE) {
                float x[8] = {};
                if (row < rows) {
                    const int token = s.row0 + row / group, head = s.g * group + row % group;
                    const uint4 u = *reinterpret_cast<const uint4 *>(
                        p.q + static_cast<int64_t>(token) * p.q_stride + head * DIM + 8 * l);
                    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint64_t f = widen16<QDT>(w[i]);
                        x[2 * i] = __uint_as_float(static_cast<uint32_t>(f));
                        x[2 * i + 1] = __uint_as_float(static_cast<uint32_t>(f >> 32));
                    }
                }
                float m = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(x[i]));
                // (every lane of the warp is in the loop: ROWS is a multiple
                // of a warp's rows, or the row is a repeat of none)
#pragma unroll
                for (int o = LANES / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o, LANES));
                const int e = part_exponent(m);
                const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] *= up;
                if (l == 0) qf[b * ROWS + row] = p.score_scale * __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
                for (int part = 0; part < Sh::kQParts; ++part) {
                    uint32_t c[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) c[i] = take_part(x[2 * i], x[2 * i + 1]);
                    const int col = part * ROWS + row;
                    uint8_t *dst = fixed_ptr + Sm::kQOff + b * Sm::kQBytes + (col >> 3) * 8 * DIM + (l >> 1) * 128 +
                                   (col & 7) * 16 + 8 * (l & 1);
                    *reinterpret_cast<uint2 *>(dst) = make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
                }
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            mbar_arrive(qfull_bar(b));
        };

        int stage = 0, i = 0, segment = 0;
        uint32_t phase = 0;
        DecSegment s, next;
        bool more = walk.next(p, s);
        if (more) load_queries(s, 0);
        while (more) {
            const int qb = segment & 1;
            const int rows = min(s.n * group, ROWS);
            float l[ROWS], m[ROWS], f[ROWS];
            softmax_sync();  // the row factors of this segment are written
#pragma unroll
            for (int r = 0; r < ROWS; ++r) {
                l[r] = 0.0f;
                m[r] = -INFINITY;
                f[r] = qf[qb * ROWS + r];
            }
            bool have_next = false;
            for (int tile = s.tile; tile < s.end; ++tile, ++i) {
                const int sb = Sh::kSBufs == 2 ? (i & 1) : 0;
                const uint32_t use = static_cast<uint32_t>(Sh::kSBufs == 2 ? i >> 1 : i);
                const int wb = i & 1;
                const int key = tile * kDecTile + tid;
                // scales and codes of the stage, then the scores
                ok = ok && mbar_wait_fast(full_bar(stage), phase, abort_flag, p.status, p.wait_cycles);
                const int pg = tid >> p.page_shift;
                const bool exists = key >= s.first && key < s.keys;
                const float ks = exists ? scales[stage * 16 + pg] : 0.0f;
                const float vs = exists ? scales[stage * 16 + 8 + pg] : 1.0f;
                const float lv = __log2f(vs), rv = __frcp_rn(vs);
                ok = ok && mbar_wait_fast(sfull_bar(sb), use & 1u, abort_flag, p.status, p.wait_cycles);
                tc_fence_after();
                float t[ROWS];
                {
                    float c[Sh::kSCols];
                    tmem_ld_cols<Sh::kSCols>(tmem + lane_addr + static_cast<uint32_t>(sb * Sh::kSCols), c);
                    tc_fence_before();
                    mbar_arrive(sempty_bar(sb));
#pragma unroll
                    for (int r = 0; r < ROWS; ++r) {
                        float x = c[r];
                        if (Sh::kQParts == 3)
                            x = fmaf(fmaf(c[2 * ROWS + r], 0.0625f, c[ROWS + r]), 0.0625f, x);
                        else
                            x = fmaf(c[ROWS + r], 0.0625f, x);
                        t[r] = fmaf(x, f[r] * ks, lv);
                    }
                }
                // rows see keys up to their position; tiles below every row's
                // need no test (nor above the last row's window)
                const int pos0 = s.keys - s.n;
                const bool plain = tile * kDecTile + kDecTile - 1 <= pos0 && tile * kDecTile >= s.first &&
                                   (p.window == 0 || tile * kDecTile > s.keys - 1 - p.window);
                if (!plain) {
                    int pos = pos0, j = 0;
#pragma unroll
                    for (int r = 0; r < ROWS; ++r) {
                        const bool seen = exists && key <= pos && (p.window == 0 || key > pos - p.window);
                        if (!seen) t[r] = -INFINITY;
                        if (++j == group) {
                            j = 0;
                            ++pos;
                        }
                    }
                }
                bool past = false;
#pragma unroll
                for (int r = 0; r < ROWS; ++r) past |= r < rows && t[r] > m[r] + 1.0f;
                if (softmax_any(past)) {
                    // new references: the tile's maxima
#pragma unroll
                    for (int r = 0; r < ROWS; ++r) {
                        float x = t[r];
#pragma unroll
                        for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, o));
                        if (lane == 0) red[warp * ROWS + r] = x;
                    }
                    softmax_sync();
                    float keep[ROWS];
#pragma unroll
                    for (int r = 0; r < ROWS; ++r) {
                        const float x = fmaxf(fmaxf(red[r], red[ROWS + r]), fmaxf(red[2 * ROWS + r], red[3 * ROWS + r]));
                        const float to = fmaxf(m[r], x);
                        keep[r] = m[r] == -INFINITY ? 0.0f : ex2(m[r] - to);
                        l[r] *= keep[r];
                        m[r] = to;
                    }
                    if (tile != s.tile) {
                        // the accumulator holds tiles up to the previous one
                        ok = ok && mbar_wait_fast(wfree_bar((i - 1) & 1), ((i - 1) >> 1) & 1u, abort_flag, p.status,
                                                  p.wait_cycles);
                        tc_fence_after();
                        float o[Sh::kOCols];
                        tmem_ld_cols<Sh::kOCols>(o_tmem + lane_addr, o);
                        uint32_t u[Sh::kOCols / 16][16];
#pragma unroll
                        for (int c = 0; c < Sh::kOCols; ++c)
                            u[c / 16][c % 16] = __float_as_uint(c < 3 * ROWS ? o[c] * keep[c % ROWS] : 0.0f);
#pragma unroll
                        for (int c = 0; c < Sh::kOCols / 16; ++c) tmem_st_n(o_tmem + lane_addr + 16 * c, u[c]);
                        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                        tc_fence_before();
                    }
                }
                // weights, their sums, and their parts
                float w[ROWS];
#pragma unroll
                for (int r = 0; r < ROWS; ++r) {
                    w[r] = ex2(t[r] - (m[r] == -INFINITY ? 0.0f : m[r]));
                    l[r] = fmaf(w[r], rv, l[r]);
                    w[r] *= 128.0f;
                }
                ok = ok && mbar_wait_fast(wfree_bar(wb), ((i >> 1) & 1u) ^ 1u, abort_flag, p.status, p.wait_cycles);
                uint8_t *wrow = fixed_ptr + Sm::kWOff + wb * Sm::kWBytes + (tid >> 3) * 8 * Sh::kOCols + (tid & 7) * 16;
#pragma unroll
                for (int part = 0; part < 3; ++part) {
#pragma unroll
                    for (int r = 0; r < ROWS; r += 4) {
                        const uint32_t lo = take_part(w[r], w[r + 1]), hi = take_part(w[r + 2], w[r + 3]);
                        const int col = part * ROWS + r;
                        *reinterpret_cast<uint32_t *>(wrow + (col >> 4) * 128 + (col & 15)) = lo | (hi << 16);
                    }
                }
                if (!exists) {
                    // keys that are not there: whatever the stage holds
                    // (NaN codes too) must not meet their zero weights
                    uint8_t *v = dec_smem + static_cast<size_t>(stage) * Sm::kStageBytes + kDecTile * DIM +
                                 (tid >> 3) * 8 * DIM + (tid & 7) * 16;
#pragma unroll
                    for (int c = 0; c < DIM / 16; ++c)
                        *reinterpret_cast<uint4 *>(v + c * 128) = make_uint4(0u, 0u, 0u, 0u);
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                mbar_arrive(wfull_bar(wb));
                if (++stage == S) {
                    stage = 0;
                    phase ^= 1u;
                }
                if (tile == s.tile) {
                    // the next segment's queries, so that its scores need not
                    // wait for this one's epilogue
                    have_next = walk.next(p, next);
                    if (have_next) load_queries(next, qb ^ 1);
                }
            }
            ++segment;

            // ------------------------------------------------------ epilogue
            ok = ok && mbar_wait_fast(wfree_bar((i - 1) & 1), ((i - 1) >> 1) & 1u, abort_flag, p.status, p.wait_cycles);
            tc_fence_after();
#pragma unroll
            for (int r = 0; r < ROWS; ++r) {
                float x = l[r];
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
                l[r] = x;
            }
            softmax_sync();  // the maxima in `red` have been read
#pragma unroll
            for (int r = 0; r < ROWS; ++r)
                if (lane == 0) red[warp * ROWS + r] = l[r];
            softmax_sync();
            float o[Sh::kOCols];
            tmem_ld_cols<Sh::kOCols>(o_tmem + lane_addr, o);
            tc_fence_before();
            const bool whole = s.tile == s.begin && s.end == s.stop;
            float *part = nullptr;
            long long c0 = 0, c1 = 0, seg0 = 0;
            if (!whole) {
                // the CTAs that share this request and head
                seg0 = s.at - (s.tile - s.begin);
                const long long seg1 = seg0 + (s.stop - s.begin);
                c0 = ((seg0 + 1) * ctas - 1) / total;
                c1 = (seg1 * ctas - 1) / total;
                const int slot = s.tile != s.begin || seg0 == w0 ? 0 : 1;
                part = p.partials + (cta * 2 + slot) * static_cast<long long>(ROWS * (DIM + 2));
            }
#pragma unroll
            for (int r = 0; r < ROWS; ++r) {
                l[r] = (red[r] + red[ROWS + r]) + (red[2 * ROWS + r] + red[3 * ROWS + r]);
                o[r] = fmaf(fmaf(o[2 * ROWS + r], 0.0625f, o[ROWS + r]), 0.0625f, o[r]) * (1.0f / 128.0f);
            }
            if (whole) {
                if (tid < DIM) {
#pragma unroll
                    for (int r = 0; r < ROWS; ++r) {
                        const float x[1] = {l[r] > 0.0f ? o[r] / l[r] : 0.0f};
                        if (r < rows) attn_store<1>(p, s.row0 + r / group, s.g * group + r % group, DIM, tid, x);
                    }
                }
                if (p.lse != nullptr) {
#pragma unroll
                    for (int r = 0; r < ROWS; ++r)
                        if (tid == r && r < rows)
                            attn_store_lse(p, s.row0 + r / group, s.g * group + r % group, m[r], l[r]);
                }
            } else {
#pragma unroll
                for (int r = 0; r < ROWS; ++r) {
                    if (r < rows) {
                        if (tid < DIM) part[r * DIM + tid] = o[r];
                        if (tid == r) {
                            part[ROWS * DIM + 2 * r] = m[r];
                            part[ROWS * DIM + 2 * r + 1] = l[r];
                        }
                    }
                }
                __threadfence();
                softmax_sync();
                if (tid == 0) {
                    const unsigned parts = static_cast<unsigned>(c1 - c0 + 1);
                    merge_now = atomicInc(p.counters + c0, parts - 1) == parts - 1;  // wraps to 0
                    __threadfence();
                }
                softmax_sync();
                if (merge_now) {
                    auto partial = [&](long long c) {
                        const int slot = c == c0 && seg0 != total * c0 / ctas ? 1 : 0;
                        return p.partials + (c * 2 + slot) * static_cast<long long>(ROWS * (DIM + 2));
                    };
                    merge_partials<DIM, ROWS>(p, s, rows, group, c0, c1, partial);
                }
            }
            more = have_next;
            s = next;
        }
    }

    // MMAs retired, tensor memory free
    mbar_wait_drain(done_bar, 0, p.status);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 5)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(Sh::kTmemCols));
}

}  // namespace
}  // namespace fp8l
