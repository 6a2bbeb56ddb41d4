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
// parts before it left over.  A bf16 query (an 8-bit significand is 4 + 4 bits
// with a sign), scaled so that its largest element is in [2^7, 2^8), is exact
// in two parts from 2^-13 of that element on and within 2^-21 of it below; fp16
// (11 bits) in three parts from 2^-14 on and within 2^-25.  A weight in three
// parts has 12 bits, or 2^-25 of the running maximum; in four, 16 bits or 2^-29.
// The part columns are summed in float32.
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
// leaves its partial (m, l, O) in the workspace.  Of every kDecFan neighbours
// the last to arrive adds the partials in CTA order and carries the sum to the
// next level, so the result does not depend on timing.
//
// Roles: per eight rows a softmax group of four warps (warp w of a group owns
// tensor-memory lanes 32 w ..: a thread is a key, and in the epilogue a
// dimension), independent of the other groups; one warp for copies (one
// untiled bulk copy per page, keys and values; the page's scales by cp.async),
// which also hands the pieces of the line to the others through shared memory;
// one warp that issues the MMAs, the next tile's scores before this tile's
// values.  Two CTAs per SM up to 16 rows, one with 32.
//
// What bounds it is HBM once a CTA has tens of tiles: 153 us for 5 sequences of
// 60-131k keys (8 kv heads of 128, groups of 8: 989 MB, 6.5 TB/s, 0.95 of the
// measured copy rate), 88 us for 64 of 0.1-8k (469 MB, 5.3 TB/s, 0.78: the
// prologue, 3 us, and one boundary in every 28 tiles, where a CTA's softmax
// waits for its epilogue while the SM's other CTA streams).  One tile's softmax
// takes about 1200 cycles (2000 with four groups), which two CTAs hide and one
// does not: 159 us with 20 rows, 105 us with 12.  D = 64 takes 77 us for half the
// bytes, fp16 96: the softmax of a tile costs the same.  7.0 us for one sequence of
// 129 keys, of which the first bytes arrive after 3.
#pragma once

#include "kv_attention_params.cuh"

namespace fp8l {
namespace {

constexpr int kDecTile = 128;      // keys per tile = MMA M
constexpr int kDecMaxStages = 6;
constexpr int kDecMinTiles = 2;    // tiles per CTA below which fewer CTAs run
constexpr int kDecMaxCtas = 2 * 160;
constexpr int kDecFan = 16;        // partials added by one CTA
constexpr int kDecLevels = 3;      // 16^3 CTAs and more
constexpr int kDecSegments = 16;   // pieces between the copy warp and the slowest role (stages + 3 at most)

// GROUPS softmax groups of eight rows; the weights in WPARTS E4M3 parts
template <int QDT, int DIM, int GROUPS, int WPARTS>
struct DecShape {
    static constexpr int kRows = 8 * GROUPS;
    static constexpr int kCtasPerSm = GROUPS <= 2 ? 2 : 1;
    static constexpr int kThreads = 128 * GROUPS + 64;
    static constexpr int kQParts = QDT == FP8L_BF16 ? 2 : 3;
    static constexpr int kSCols = (kRows * kQParts + 15) / 16 * 16;
    static constexpr int kOCols = (kRows * WPARTS + 15) / 16 * 16;
    static constexpr int kUsedCols = 2 * kSCols + kOCols;
    static constexpr int kTmemCols = kUsedCols <= 64 ? 64 : (kUsedCols <= 128 ? 128 : (kUsedCols <= 256 ? 256 : 512));
    static_assert(kUsedCols <= 512 / kCtasPerSm, "the SM's CTAs share its tensor memory");
    // shared memory after the stages; columns that no row uses hold whatever
    // is there: their products land in columns that nobody reads
    static constexpr int kStageBytes = 2 * kDecTile * DIM;  // keys, values
    static constexpr int kQBytes = kSCols * DIM;            // per buffer
    static constexpr int kWBytes = kDecTile * kOCols;       // per buffer
    static constexpr int kQOff = 0;
    static constexpr int kWOff = kQOff + 2 * kQBytes;
    // the epilogue's rows in float32: in the weights' buffers where one group
    // owns them (its weights have been multiplied by then)
    static constexpr int kRowsOff = GROUPS == 1 ? kWOff : kWOff + 2 * kWBytes;
    static constexpr int kScaleOff = kWOff + 2 * kWBytes + (GROUPS == 1 ? 0 : kRows * DIM * 4);  // [stage][2][8]
    static constexpr int kQfOff = kScaleOff + kDecMaxStages * 16 * 4;   // [2][kRows] floats
    static constexpr int kRedOff = kQfOff + 2 * kRows * 4;              // [4][kRows] floats
    // the epilogue's sums, apart from the maxima: a piece's last tile can move
    // the reference, and no barrier lies between its reads and these writes
    static constexpr int kSumOff = kRedOff + 4 * kRows * 4;             // [4][kRows] floats
    static constexpr int kRefOff = kSumOff + 4 * kRows * 4;             // [kRows] floats
    static constexpr int kSegOff = (kRefOff + kRows * 4 + 15) / 16 * 16;  // [kDecSegments] DecSegment
    static constexpr int kBarOff = kSegOff + kDecSegments * 64;
    static constexpr int kBars = 2 * kDecMaxStages + 10 + kDecSegments + 1;
    static constexpr int kMiscOff = kBarOff + kBars * 8;
    static constexpr int kFixedBytes = kMiscOff + 16;
    static_assert(kRows * DIM * 4 <= 2 * kWBytes || GROUPS > 1, "the rows fit the weights' buffers");
    // the M-side read of a 64-dimension V covers 512 bytes past the last stage
    static_assert(2 * kQBytes >= 512, "reads past the last stage stay inside");
};

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

// Sums (or maxima) of eight values over the warp in 3 + 2 steps: each step of
// the first three halves the values a lane keeps.  Lanes with the same
// lane / 4 return value number (bits 4, 3, 2 of the lane).
template <bool MAX>
__device__ __forceinline__ float reduce8(const float (&v)[8], int lane) {
    auto op = [](float a, float b) { return MAX ? fmaxf(a, b) : a + b; };
    float a[4], b[2];
    const bool h4 = lane & 16, h3 = lane & 8, h2 = lane & 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float other = __shfl_xor_sync(0xFFFFFFFFu, h4 ? v[i] : v[i + 4], 16);
        a[i] = op(h4 ? v[i + 4] : v[i], other);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float other = __shfl_xor_sync(0xFFFFFFFFu, h3 ? a[i] : a[i + 2], 8);
        b[i] = op(h3 ? a[i + 2] : a[i], other);
    }
    float c = op(h2 ? b[1] : b[0], __shfl_xor_sync(0xFFFFFFFFu, h2 ? b[0] : b[1], 4));
    c = op(c, __shfl_xor_sync(0xFFFFFFFFu, c, 2));
    return op(c, __shfl_xor_sync(0xFFFFFFFFu, c, 1));
}

// A piece of one request and kv head: key tiles [tile, end) of its [begin,
// stop).  tile == end: there are no more.
struct DecSegment {
    int r, g;
    int n, row0;        // the request's new tokens, their first row
    int first, keys;    // first visible key, end of the keys
    int tile, end, begin, stop;
    int done;           // tiles of the CTA's piece of the line before this one
    int pad[5];
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
    const int L = min(max(p.kv_lens[r], 0), INT32_MAX - 255);  // (a tile's last key fits an int)
    d.keys = static_cast<int64_t>(L) < cap ? L : static_cast<int>(cap);
    d.n = b - a;
    d.row0 = a;
    const int pos = d.keys - d.n;
    d.first = p.window > 0 ? max(0, pos - p.window + 1) : 0;
    d.begin = d.first / kDecTile;
    d.tiles = d.n > 0 ? max((d.keys + kDecTile - 1) / kDecTile - d.begin, 1) : 0;
    return d;
}

// Walks the pieces of a CTA's part of the line of tiles.
struct DecWalk {
    int done, left;    // tiles handed out, still to hand out
    int r, g, offset;  // next tile: offset in request r, head g
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
        const int take = min(d.tiles - offset, left);
        s.end = s.tile + take;
        s.done = done;
        done += take;
        left -= take;
        offset += take;
        if (offset == d.tiles) {
            offset = 0;
            if (++g == p.kv_heads) {
                g = 0;
                if (++r >= p.requests) left = 0;
            }
        }
        return true;
    }
};

// Exclusive prefix (plus the block's total in *total) of one value per thread
template <int THREADS>
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
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) before += red[w];
        sum += red[w];
    }
    *total = sum;
    return before + inc - v;
}

template <int QDT, int DIM, int GROUPS, int WPARTS>
__global__ void __launch_bounds__(DecShape<QDT, DIM, GROUPS, WPARTS>::kThreads,
                                  DecShape<QDT, DIM, GROUPS, WPARTS>::kCtasPerSm)
kv_attention_decode_kernel(const AttnParams p) {
    using Sh = DecShape<QDT, DIM, GROUPS, WPARTS>;
    constexpr int ROWS = Sh::kRows;
    extern __shared__ __align__(128) uint8_t dec_smem[];
    __shared__ long long scan_red[Sh::kThreads / 32];
    __shared__ int start_r, start_g, start_offset, merge_now[GROUPS];
    const uint32_t sbase = smem_u32(dec_smem);
    const int S = p.stages;
    const uint32_t fixed = sbase + static_cast<uint32_t>(S) * Sh::kStageBytes;
    uint8_t *fixed_ptr = dec_smem + static_cast<size_t>(S) * Sh::kStageBytes;
    const uint32_t full = fixed + Sh::kBarOff, empty = full + 8 * kDecMaxStages;
    const uint32_t sfull = empty + 8 * kDecMaxStages, sempty = sfull + 16, wfull = sempty + 16, wfree = wfull + 16;
    const uint32_t qfull = wfree + 16, segfull = qfull + 16, done_bar = segfull + 8 * kDecSegments;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(fixed_ptr + Sh::kMiscOff);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int kCopyWarp = 4 * GROUPS, kMmaWarp = kCopyWarp + 1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full + 8 * s, 1 + 32);  // expected bytes, and the lanes' scale copies
            mbar_init(empty + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(sfull + 8 * b, 1);
            mbar_init(sempty + 8 * b, 128 * GROUPS);
            mbar_init(wfull + 8 * b, 128 * GROUPS);
            mbar_init(wfree + 8 * b, 1);
            mbar_init(qfull + 8 * b, 128 * GROUPS);
        }
        for (int s = 0; s < kDecSegments; ++s) mbar_init(segfull + 8 * s, 1);
        mbar_init(done_bar, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(tmem_slot)),
                     "r"(Sh::kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    grid_dependency_sync();

    // the line of tiles, and this CTA's piece of it: requests in rounds of
    // one per thread, the first round's values kept for the second reading
    const int mine0 = static_cast<int>(threadIdx.x) < p.requests ? dec_range(p, threadIdx.x).tiles : 0;
    long long total = 0, before0 = 0;
    for (int r0 = 0; r0 < p.requests; r0 += Sh::kThreads) {
        const int r = r0 + static_cast<int>(threadIdx.x);
        const int tiles = r0 == 0 ? mine0 : (r < p.requests ? dec_range(p, r).tiles : 0);
        long long sum;
        const long long before = dec_scan<Sh::kThreads>(static_cast<long long>(tiles) * p.kv_heads, scan_red, &sum);
        if (r0 == 0) before0 = before;
        total += sum;
    }
    // fewer CTAs when each would get less than kDecMinTiles: a merge costs about
    // as much as two tiles.  Measured (us, 1 / 2 / 3 tiles): one sequence of 129
    // keys 9.1 / 6.7 / 12.5, 1500 keys 13.2 / 11.6 / 11.6, 4000 keys 17.9 / 15.5 /
    // 17.3, 30000 keys 23.3 / 23.4 / 23.3, eight of up to 1000 12.3 / 15.5 / 17.0
    const long long ctas = max(min(static_cast<long long>(gridDim.x), total / kDecMinTiles),
                               min(static_cast<long long>(gridDim.x), min(total, 1LL)));
    const long long cta = static_cast<long long>(blockIdx.x);
    const bool idle = cta >= ctas;
    const long long w0 = idle ? 0 : piece_begin(total, cta, ctas), w1 = idle ? 0 : piece_begin(total, cta + 1, ctas);
    if (!idle) {
        long long carry = 0;
        for (int r0 = 0; r0 < p.requests; r0 += Sh::kThreads) {
            const int r = r0 + static_cast<int>(threadIdx.x);
            const int tiles = r0 == 0 ? mine0 : (r < p.requests ? dec_range(p, r).tiles : 0);
            const long long n = static_cast<long long>(tiles) * p.kv_heads;
            long long sum = 0, before = before0;
            if (p.requests > Sh::kThreads) before = carry + dec_scan<Sh::kThreads>(n, scan_red, &sum);
            if (n > 0 && before <= w0 && w0 < before + n) {
                start_r = r;
                const unsigned rest = static_cast<unsigned>(w0 - before);  // below tiles * kv_heads
                start_g = static_cast<int>(rest / static_cast<unsigned>(tiles));
                start_offset = static_cast<int>(rest % static_cast<unsigned>(tiles));
            }
            carry += sum;
            if (carry > w0) break;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const uint32_t o_col = 2 * Sh::kSCols;
    const int P = 1 << p.page_shift;
    const int group = p.q_heads / p.kv_heads;
    DecSegment *segs = reinterpret_cast<DecSegment *>(fixed_ptr + Sh::kSegOff);
    // piece number n, or nullptr after the last (or a time-out)
    auto segment_at = [&](int n) -> const DecSegment * {
        if (!kv_wait(segfull + 8 * (n & (kDecSegments - 1)), (n / kDecSegments) & 1u, abort_flag, p.status,
                     p.wait_cycles))
            return nullptr;
        const DecSegment *s = segs + (n & (kDecSegments - 1));
        return s->tile < s->end ? s : nullptr;
    };

    if (warp == kCopyWarp) {
        // ---------------------------------------------------------- copies
        int stage = 0, published = 0;
        uint32_t phase = 0, issued = 0, issued_parity = 0;
        const int per_tile = kDecTile >> p.page_shift;  // pages of a tile, at most 8
        DecWalk walk{0, static_cast<int>(w1 - w0), idle ? 0 : start_r, idle ? 0 : start_g, idle ? 0 : start_offset};
        bool ok = true, more = true;
        // hands out the next piece (or the end)
        auto publish = [&](DecSegment &s) {
            more = more && walk.next(p, s);
            if (!more) s.tile = s.end = 0;
            if (lane == 0) {
                segs[published & (kDecSegments - 1)] = s;
                mbar_arrive(segfull + 8 * (published & (kDecSegments - 1)));
            }
            __syncwarp();
            ++published;
            return more;
        };
        DecSegment s, ahead;
        bool have = publish(s);
        while (ok && have) {
            // one piece ahead: its queries are prepared under this one's tiles
            const bool have_ahead = publish(ahead);
            const int32_t *table = p.block_table + static_cast<int64_t>(s.r) * p.table_width;
            // lanes 0-7 keys of page lane, lanes 8-15 values of page lane - 8
            const int i = lane & 7;
            auto wanted = [&](int tile) {
                const int64_t b = static_cast<int64_t>(tile) * per_tile + i;
                return lane < 16 && i < per_tile && (b << p.page_shift) < s.keys &&
                       ((b + 1) << p.page_shift) > s.first;
            };
            int page = wanted(s.tile) ? table[s.tile * per_tile + i] : 0;
            for (int tile = s.tile; tile < s.end; ++tile) {
                const bool mine = wanted(tile);
                const int64_t ph = static_cast<int64_t>(min(max(page, 0), p.num_pages - 1)) * p.kv_heads + s.g;
                // the next tile's pages, while this one waits for its stage
                if (tile + 1 < s.end) page = wanted(tile + 1) ? table[(tile + 1) * per_tile + i] : 0;
                uint32_t bytes = 0;
                if (mine) {
                    const int in_page = min(s.keys - ((tile * per_tile + i) << p.page_shift), P);
                    bytes = static_cast<uint32_t>((in_page + 7) / 8 * 8 * DIM);
                }
                const uint32_t sum = __reduce_add_sync(0xFFFFFFFFu, bytes);
                ok = __all_sync(0xFFFFFFFFu,
                                kv_wait(empty + 8 * stage, phase ^ 1u, abort_flag, p.status, p.wait_cycles));
                if (!ok) break;
                const uint32_t dst = sbase + static_cast<uint32_t>(stage) * Sh::kStageBytes +
                                     (lane >= 8 ? kDecTile * DIM : 0) + static_cast<uint32_t>(i * P * DIM);
                if (lane == 0) mbar_expect_tx(full + 8 * stage, sum);
                __syncwarp();
                if (mine) {
                    bulk_copy(dst, (lane < 8 ? p.k_cache : p.v_cache) + ph * P * DIM, bytes, full + 8 * stage);
                    const float *scale = (lane < 8 ? p.k_scale : p.v_scale) + ph;
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(
                                     fixed + Sh::kScaleOff + static_cast<uint32_t>((stage * 16 + lane) * 4)),
                                 "l"(scale)
                                 : "memory");
                }
                asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(full + 8 * stage)
                             : "memory");
                issued |= 1u << stage;
                issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
                if (++stage == S) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            s = ahead;
            have = have_ahead;
        }
        // every copy lands before the CTA exits
        asm volatile("cp.async.wait_all;" ::: "memory");
        for (int x = 0; x < S; ++x)
            if (issued & (1u << x)) kv_drain(full + 8 * x, (issued_parity >> x) & 1u, p.status);
    } else if (warp == kMmaWarp) {
        // ---------------------------------------------------------- MMAs
        const bool leader = elect_one();
        const uint32_t tmem_u = __shfl_sync(0xFFFFFFFFu, tmem, 0);
        const uint32_t idesc_s = (1u << 4) | (static_cast<uint32_t>(Sh::kSCols >> 3) << 17) | (8u << 24);
        const uint32_t idesc_o = (1u << 4) | (1u << 15) | (1u << 16) |
                                 (static_cast<uint32_t>(Sh::kOCols >> 3) << 17) | (8u << 24);
        auto wait = [&](uint32_t bar, uint32_t parity) {
            return __all_sync(0xFFFFFFFFu, kv_wait(bar, parity & 1u, abort_flag, p.status, p.wait_cycles));
        };
        bool ok = true;
        if (p.stall & kStallMma) ok = wait(done_bar, 0);
        int stage = 0, prev_stage = 0, i = 0, segment = 0;
        uint32_t phase = 0;
        bool prev_first = false;
        auto values = [&](int k) {  // O += V^T W^T of tile number k
            const int b = k & 1;
            if (!wait(wfull + 8 * b, k >> 1)) return false;
            tc_fence_after();
            if (leader) {
                const uint32_t v = desc_lo(sbase + static_cast<uint32_t>(prev_stage) * Sh::kStageBytes + kDecTile * DIM,
                                           8 * DIM);
                const uint32_t w = desc_lo(fixed + Sh::kWOff + static_cast<uint32_t>(b) * Sh::kWBytes, 8 * Sh::kOCols);
#pragma unroll
                for (int j = 0; j < kDecTile / 32; ++j)
                    mma_f8_desc(tmem_u + o_col, v + 2 * DIM * j, desc_hi(128), w + 2 * Sh::kOCols * j, desc_hi(128),
                                idesc_o, (prev_first && j == 0) ? 0u : 1u);
                mma_commit(wfree + 8 * b);
                mma_commit(empty + 8 * prev_stage);
            }
            return true;
        };
        while (ok) {
            const DecSegment *s = segment_at(segment);
            if (__any_sync(0xFFFFFFFFu, s == nullptr)) break;
            const int qb = segment & 1, tiles = s->end - s->tile;
            ok = wait(qfull + 8 * qb, segment >> 1);
            for (int tile = 0; ok && tile < tiles; ++tile, ++i) {
                const int b = i & 1;
                ok = wait(full + 8 * stage, phase) && wait(sempty + 8 * b, (i >> 1) + 1);
                if (!ok) break;
                tc_fence_after();
                if (leader) {
                    const uint32_t k = desc_lo(sbase + static_cast<uint32_t>(stage) * Sh::kStageBytes, 128);
                    const uint32_t q = desc_lo(fixed + Sh::kQOff + static_cast<uint32_t>(qb) * Sh::kQBytes, 128);
#pragma unroll
                    for (int j = 0; j < DIM / 32; ++j)
                        mma_f8_desc(tmem_u + static_cast<uint32_t>(b * Sh::kSCols), k + 16 * j, desc_hi(8 * DIM),
                                    q + 16 * j, desc_hi(8 * DIM), idesc_s, j == 0 ? 0u : 1u);
                    mma_commit(sfull + 8 * b);
                }
                if (i > 0) ok = values(i - 1);
                prev_stage = stage;
                prev_first = tile == 0;
                if (++stage == S) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            ++segment;
        }
        if (ok && i > 0) values(i - 1);
        if (leader) mma_commit(done_bar);
        __syncwarp();
    } else {
        // ---------------------------------------------------------- softmax
        const int grp = warp >> 2, bar_id = 1 + grp, tid = static_cast<int>(threadIdx.x) & 127;
        const int row_base = 8 * grp;  // the group's rows of the unit
        const uint32_t lane_addr = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t s_tmem = tmem + lane_addr + row_base, o_tmem = tmem + lane_addr + o_col + row_base;
        float *qf = reinterpret_cast<float *>(fixed_ptr + Sh::kQfOff) + row_base;
        float *red = reinterpret_cast<float *>(fixed_ptr + Sh::kRedOff) + row_base;
        float *sums = reinterpret_cast<float *>(fixed_ptr + Sh::kSumOff) + row_base;
        float *ref = reinterpret_cast<float *>(fixed_ptr + Sh::kRefOff) + row_base;
        const float *scales = reinterpret_cast<const float *>(fixed_ptr + Sh::kScaleOff);
        bool ok = true;

        // The piece's queries as E4M3 parts in buffer b, and the factor of
        // each row's scores: LANES lanes hold a row, eight dimensions each.
        auto load_queries = [&](const DecSegment &s, int b) {
            constexpr int LANES = DIM / 8;
            const int l = tid % LANES, row = tid / LANES;
            if (row < 8) {  // (whole warps)
                const int unit_row = row_base + row, token = unit_row / group;
                float x[8] = {};
                if (token < s.n) {
                    const uint4 u = *reinterpret_cast<const uint4 *>(
                        p.q + static_cast<int64_t>(s.row0 + token) * p.q_stride +
                        (s.g * group + unit_row - token * group) * DIM + 8 * l);
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
#pragma unroll
                for (int o = LANES / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o, LANES));
                const int e = part_exponent(m);
                const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] *= up;
                if (l == 0) qf[b * ROWS + row] = part_factor(p.score_scale, m, e);
#pragma unroll
                for (int part = 0; part < Sh::kQParts; ++part) {
                    uint32_t c[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) c[i] = take_part(x[2 * i], x[2 * i + 1]);
                    const int col = part * ROWS + unit_row;
                    uint8_t *dst = fixed_ptr + Sh::kQOff + b * Sh::kQBytes + (col >> 3) * 8 * DIM + (l >> 1) * 128 +
                                   (col & 7) * 16 + 8 * (l & 1);
                    *reinterpret_cast<uint2 *>(dst) = make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
                }
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            mbar_arrive(qfull + 8 * b);
        };

        int stage = 0, i = 0, segment = 0;
        uint32_t phase = 0;
        const DecSegment *s = segment_at(0);
        // one answer for the group's threads, whose barriers need all of them
        // (a wait can give up in one thread and not in another)
        bool more = !group_any(bar_id, s == nullptr);
        if (more) load_queries(*s, 0);
        while (more) {
            const int qb = segment & 1;
            const int begin = s->tile, end = s->end, first = s->first, keys = s->keys;
            const int pos0 = keys - s->n;  // position of the first row's token
            float l[8], m[8];
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                l[r] = 0.0f;
                m[r] = -INFINITY;
            }
            group_sync(bar_id);  // the row factors of this piece are written
            const DecSegment *next = nullptr;
            if (GROUPS > 1 && row_base >= s->n * group) {
                // none of this group's rows exist: only its share of the
                // barriers, and the next piece's queries
                for (int tile = begin; tile < end; ++tile, ++i) {
                    const int b = i & 1;
                    ok = ok && kv_wait(sfull + 8 * b, (i >> 1) & 1u, abort_flag, p.status, p.wait_cycles);
                    mbar_arrive(sempty + 8 * b);
                    ok = ok && kv_wait(wfree + 8 * b, ((i >> 1) & 1u) ^ 1u, abort_flag, p.status, p.wait_cycles);
                    mbar_arrive(wfull + 8 * b);
                    if (++stage == S) {
                        stage = 0;
                        phase ^= 1u;
                    }
                    if (tile == begin) {
                        next = segment_at(segment + 1);
                        if (group_any(bar_id, next == nullptr)) next = nullptr;
                        if (next != nullptr) load_queries(*next, qb ^ 1);
                    }
                }
                ++segment;
                s = next;
                more = next != nullptr;
                continue;
            }
            for (int tile = begin; tile < end; ++tile, ++i) {
                const int b = i & 1;
                const int key = tile * kDecTile + tid;
                // scales and codes of the stage, then the scores
                ok = ok && kv_wait(full + 8 * stage, phase, abort_flag, p.status, p.wait_cycles);
                const int pg = tid >> p.page_shift;
                const bool exists = key >= first && key < keys;
                const float ks = exists ? scales[stage * 16 + pg] : 0.0f;
                const float vs = exists ? value_scale(scales[stage * 16 + 8 + pg]) : 1.0f;
                // (a NaN scale: in t, for the rows that see the key, alone)
                const float lv = __log2f(vs), rv = __isnanf(vs) ? 0.0f : __frcp_rn(vs);
                const float4 f0 = *reinterpret_cast<const float4 *>(qf + qb * ROWS);
                const float4 f1 = *reinterpret_cast<const float4 *>(qf + qb * ROWS + 4);
                const float f[8] = {f0.x, f0.y, f0.z, f0.w, f1.x, f1.y, f1.z, f1.w};
                ok = ok && kv_wait(sfull + 8 * b, (i >> 1) & 1u, abort_flag, p.status, p.wait_cycles);
                tc_fence_after();
                float t[8];
                {
                    uint32_t c[Sh::kQParts][8];
#pragma unroll
                    for (int part = 0; part < Sh::kQParts; ++part)
                        tmem_ld8(s_tmem + static_cast<uint32_t>(b * Sh::kSCols + part * ROWS), c[part]);
                    tmem_wait_ld();
                    tc_fence_before();
                    mbar_arrive(sempty + 8 * b);
#pragma unroll
                    for (int r = 0; r < 8; ++r) {
                        float x = __uint_as_float(c[Sh::kQParts - 1][r]);
#pragma unroll
                        for (int part = Sh::kQParts - 2; part >= 0; --part)
                            x = fmaf(x, 0.0625f, __uint_as_float(c[part][r]));
                        t[r] = fmaf(x, f[r] * ks, lv);
                    }
                }
                // rows see keys up to their position; tiles below every row's
                // need no test (nor above the last row's window)
                if (!(tile * kDecTile + kDecTile - 1 <= pos0 && tile * kDecTile >= first &&
                      (p.window == 0 || tile * kDecTile > keys - 1 - p.window))) {
                    int pos = pos0 + row_base / group, j = row_base % group;
#pragma unroll
                    for (int r = 0; r < 8; ++r) {
                        if (!(exists && key <= pos && (p.window == 0 || key > pos - p.window))) t[r] = -INFINITY;
                        if (++j == group) {
                            j = 0;
                            ++pos;
                        }
                    }
                }
                bool past = false;
#pragma unroll
                for (int r = 0; r < 8; ++r) past |= t[r] > m[r] + 1.0f;
                if (group_any(bar_id, past)) {
                    // new references: the tile's maxima
                    const float top = reduce8<true>(t, lane);
                    if ((lane & 3) == 0) red[(warp & 3) * ROWS + (lane >> 2)] = top;
                    group_sync(bar_id);
                    float keep[8];
#pragma unroll
                    for (int r = 0; r < 8; ++r) {
                        const float x = fmaxf(fmaxf(red[r], red[ROWS + r]), fmaxf(red[2 * ROWS + r], red[3 * ROWS + r]));
                        const float to = fmaxf(m[r], x);
                        keep[r] = m[r] == -INFINITY ? 0.0f : ex2(m[r] - to);
                        l[r] *= keep[r];
                        m[r] = to;
                    }
                    if (tile != begin) {
                        // the accumulator holds tiles up to the previous one
                        ok = ok && kv_wait(wfree + 8 * ((i - 1) & 1), ((i - 1) >> 1) & 1u, abort_flag, p.status,
                                           p.wait_cycles);
                        tc_fence_after();
#pragma unroll 1
                        for (int part = 0; part < WPARTS; ++part) {
                            uint32_t o[8];
                            tmem_ld8(o_tmem + static_cast<uint32_t>(part * ROWS), o);
                            tmem_wait_ld();
#pragma unroll
                            for (int r = 0; r < 8; ++r) o[r] = __float_as_uint(__uint_as_float(o[r]) * keep[r]);
                            tmem_st8(o_tmem + static_cast<uint32_t>(part * ROWS), o);
                        }
                        tmem_wait_st();
                        tc_fence_before();
                    }
                }
                // weights, their sums, and their parts
                float w[8];
#pragma unroll
                for (int r = 0; r < 8; ++r) {
                    w[r] = ex2(t[r] - (m[r] == -INFINITY ? 0.0f : m[r]));
                    l[r] = fmaf(w[r], rv, l[r]);
                    w[r] *= 128.0f;
                }
                ok = ok && kv_wait(wfree + 8 * b, ((i >> 1) & 1u) ^ 1u, abort_flag, p.status, p.wait_cycles);
                uint8_t *wrow = fixed_ptr + Sh::kWOff + b * Sh::kWBytes + (tid >> 3) * 8 * Sh::kOCols + (tid & 7) * 16;
#pragma unroll
                for (int part = 0; part < WPARTS; ++part) {
                    uint32_t c[4];
#pragma unroll
                    for (int r = 0; r < 4; ++r) c[r] = take_part(w[2 * r], w[2 * r + 1]);
                    const int col = part * ROWS + row_base;
                    *reinterpret_cast<uint2 *>(wrow + (col >> 4) * 128 + (col & 15)) =
                        make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
                }
                if (grp == 0 && !exists) {
                    // keys that are not there: whatever the stage holds
                    // (NaN codes too) must not meet their zero weights
                    uint8_t *v = dec_smem + static_cast<size_t>(stage) * Sh::kStageBytes + kDecTile * DIM +
                                 (tid >> 3) * 8 * DIM + (tid & 7) * 16;
#pragma unroll
                    for (int c = 0; c < DIM / 16; ++c)
                        *reinterpret_cast<uint4 *>(v + c * 128) = make_uint4(0u, 0u, 0u, 0u);
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                mbar_arrive(wfull + 8 * b);
                if (++stage == S) {
                    stage = 0;
                    phase ^= 1u;
                }
                if (tile == begin) {
                    // the next piece's queries, so that its scores need not
                    // wait for this one's epilogue
                    next = segment_at(segment + 1);
                    if (group_any(bar_id, next == nullptr)) next = nullptr;
                    if (next != nullptr) load_queries(*next, qb ^ 1);
                }
            }
            ++segment;

            // ------------------------------------------------------ epilogue
            // sums over the keys, and the accumulator turned from a dimension
            // per thread into rows of shared memory
            const float sum = reduce8<false>(l, lane);
            if ((lane & 3) == 0) sums[(warp & 3) * ROWS + (lane >> 2)] = sum;
#pragma unroll
            for (int r = 0; r < 8; ++r)
                if (tid == r) ref[r] = m[r];
            ok = ok && kv_wait(wfree + 8 * ((i - 1) & 1), ((i - 1) >> 1) & 1u, abort_flag, p.status, p.wait_cycles);
            tc_fence_after();
            float *rows = reinterpret_cast<float *>(fixed_ptr + Sh::kRowsOff) + row_base * DIM;
            {
                uint32_t o[WPARTS][8];
#pragma unroll
                for (int part = 0; part < WPARTS; ++part) tmem_ld8(o_tmem + static_cast<uint32_t>(part * ROWS), o[part]);
                tmem_wait_ld();
                tc_fence_before();
                if (tid < DIM) {
#pragma unroll
                    for (int r = 0; r < 8; ++r) {
                        float x = __uint_as_float(o[WPARTS - 1][r]);
#pragma unroll
                        for (int part = WPARTS - 2; part >= 0; --part)
                            x = fmaf(x, 0.0625f, __uint_as_float(o[part][r]));
                        rows[r * DIM + tid] = x * (1.0f / 128.0f);
                    }
                }
            }
            group_sync(bar_id);
            // a row in 16 threads, V dimensions each
            constexpr int V = DIM / 16;
            const int row = tid >> 4, at = (tid & 15) * V;
            const int unit_row = row_base + row, token = unit_row / group, head = s->g * group + unit_row - token * group;
            const bool valid = token < s->n;
            float acc[V], mm = ref[row];
            float ll = (sums[row] + sums[ROWS + row]) + (sums[2 * ROWS + row] + sums[3 * ROWS + row]);
#pragma unroll
            for (int v = 0; v < V; v += 4) {
                const float4 x = *reinterpret_cast<const float4 *>(rows + row * DIM + at + v);
                acc[v] = x.x, acc[v + 1] = x.y, acc[v + 2] = x.z, acc[v + 3] = x.w;
            }
            bool write = begin == s->begin && end == s->stop;
            if (!write) {
                // the CTAs that share this request and head, and their partials
                constexpr long long kPart = ROWS * (DIM + 2);
                const long long seg0 = w0 + s->done - (begin - s->begin), seg1 = seg0 + (s->stop - s->begin);
                const int c0 = piece_of(total, seg0, ctas), c1 = piece_of(total, seg1 - 1, ctas);
                const int parts = c1 - c0 + 1;
                auto slot_of = [&](int c) {
                    return (c0 + c) * 2 + (c == 0 && seg0 != piece_begin(total, c0, ctas) ? 1 : 0);
                };
                auto partial = [&](int c) { return p.partials + slot_of(c) * kPart; };
                auto put = [&](float *to) {
#pragma unroll
                    for (int v = 0; v < V; v += 4)
                        *reinterpret_cast<float4 *>(to + unit_row * DIM + at + v) =
                            make_float4(acc[v], acc[v + 1], acc[v + 2], acc[v + 3]);
                    if ((tid & 15) == 0)
                        *reinterpret_cast<float2 *>(to + ROWS * DIM + 2 * unit_row) = make_float2(mm, ll);
                };
                // whether this CTA is the last of `parts` to count here
                auto last_of = [&](unsigned *counter, int parts) {
                    __threadfence();
                    group_sync(bar_id);
                    if (tid == 0) {
                        merge_now[grp] = atomicInc(counter, static_cast<unsigned>(parts - 1)) ==
                                         static_cast<unsigned>(parts - 1);  // wraps to 0
                        __threadfence();
                    }
                    group_sync(bar_id);
                    return merge_now[grp] != 0;
                };
                // partials c0, c0 + step, ... added in this order: up to
                // kDecFan factors in a row's 16 threads
                auto merge = [&](int first_c, int step, int n) {
                    const int c = tid & 15;
                    const float2 ml = c < n ? __ldcg(reinterpret_cast<const float2 *>(
                                                  partial(first_c + c * step) + ROWS * DIM + 2 * unit_row))
                                            : make_float2(-INFINITY, 0.0f);
                    mm = ml.x;
#pragma unroll
                    for (int o = 8; o > 0; o >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xFFFFFFFFu, mm, o, 16));
                    const float e = ml.x == -INFINITY ? 0.0f : ex2(ml.x - mm);
                    ll = ml.y * e;
#pragma unroll
                    for (int o = 8; o > 0; o >>= 1) ll += __shfl_xor_sync(0xFFFFFFFFu, ll, o, 16);
#pragma unroll
                    for (int v = 0; v < V; ++v) acc[v] = 0.0f;
#pragma unroll 4
                    for (int k = 0; k < n; ++k) {
                        const float ek = __shfl_sync(0xFFFFFFFFu, e, k, 16);
                        const float *q = partial(first_c + k * step) + unit_row * DIM + at;
#pragma unroll
                        for (int v = 0; v < V; v += 4) {
                            const float4 x = __ldcg(reinterpret_cast<const float4 *>(q + v));
                            acc[v] = fmaf(x.x, ek, acc[v]);
                            acc[v + 1] = fmaf(x.y, ek, acc[v + 1]);
                            acc[v + 2] = fmaf(x.z, ek, acc[v + 2]);
                            acc[v + 3] = fmaf(x.w, ek, acc[v + 3]);
                        }
                    }
                };
                // a tree of fan-in kDecFan, one level where the parts are few:
                // a single CTA reads its partials at one SM's rate
                int index = static_cast<int>(cta) - c0, step = 1, n = parts;
                unsigned *counters = p.counters;
                put(partial(index));
                for (;;) {
                    const int node = index / kDecFan * kDecFan, members = min(kDecFan, n - node);
                    write = last_of(counters + slot_of(node * step) * GROUPS + grp, members);
                    if (!write) break;
                    merge(node * step, step, members);
                    if (n <= kDecFan) break;
                    put(partial(node * step));
                    index = node / kDecFan;
                    step *= kDecFan;
                    n = (n + kDecFan - 1) / kDecFan;
                    counters += 2 * kDecMaxCtas * 2;
                    group_sync(bar_id);  // merge_now has been read
                }
            }
            if (write && valid) {
                const float inv = 1.0f / ll;
#pragma unroll
                for (int v = 0; v < V; ++v) acc[v] = ll == 0.0f ? 0.0f : acc[v] * inv;
                attn_store<V>(p, s->row0 + token, head, DIM, at, acc);
                if ((tid & 15) == 0 && p.lse != nullptr) attn_store_lse(p, s->row0 + token, head, mm, ll);
            }
            group_sync(bar_id);  // rows, sums and references have been read
            s = next;
            more = next != nullptr;
        }
    }

    // MMAs retired, tensor memory free
    kv_drain(done_bar, 0, p.status);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    kv_report(abort_flag, p.library_status);
    if (warp == kMmaWarp)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(Sh::kTmemCols));
}

}  // namespace
}  // namespace fp8l
