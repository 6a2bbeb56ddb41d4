// Attention of many query rows per kv head (prompt chunks) on the tcgen05
// tensor cores.
//
// A unit of work is a tile of 256 query rows (tokens x heads of the group, in
// token order) of one request and kv head against a tile of 128 keys; the
// rows are two halves X = 0, 1 of 128 whose softmax and MMAs alternate, so
// the tensor core multiplies for one half while the other half's weights are
// formed:
//   S_X [128 rows x 128 keys] = Q_X K^T     (kind::f8f6f4, parts x D / 32 MMAs)
//   O_X [128 rows x D]       += W_X V       (kind::f16, 8 MMAs, W in tensor memory)
// K is multiplied as stored: a 16-bit query row, scaled so that its largest
// element is in [2^7, 2^8), is a sum of two (bf16, 8 significand bits) or three
// (fp16, 11 bits) E4M3 parts.  They share the accumulator, so no part can be
// scaled up and all stop at E4M3's step of 2^-9: elements from 2^-9 (bf16) or
// 2^-6 (fp16) of the row's largest on are exact, smaller ones within 2^-17 of the
// largest.  Two fp8 MMAs take the time of one 16-bit one and K is never
// widened.  The weights need a 16-bit format's
// range (a first token often draws most of a row's weight, leaving the others
// below 2^-16 of it), so V is widened to fp16, exactly, once per key tile for
// all 256 rows, by four warps of their own.
//
// Softmax with block scales: with k_j = sk c_j and v_j = sv d_j per page,
//   t_j = log2(e) sm_scale q.k_j + log2 sv_j,   w_j = 2^(t_j - m)
//   O = sum_j w_j d_j,  l = sum_j w_j / sv_j,  out = O / l.
// A row is one thread, a page's factors are uniform, so the maximum and the
// sum cost one operation per score and page.  The reference m starts 7 below
// the first tile's maximum and moves (rescaling l and the accumulator) only
// when a score passes it by 15: weights stay below 2^15 and the row's largest
// is at least 2^7, so fp16 keeps 11 bits of a weight down to 2^-21 of the
// largest and is within 2^-32 of the largest below that.
//
// Work: the tiles (request, kv head, row tile, key tile) form one line, cut
// into equal pieces for one CTA per SM; row tiles that span pieces are merged
// as in the decode kernel, by a tree of kProFan.
//
// Roles (512 threads): warps 0-3 and 4-7 softmax, queries and epilogue of
// halves 0 and 1 (warp w owns tensor-memory lanes 32 (w mod 4) ..), warps 8-11
// V to fp16 and the scales' factors, warp 12 copies and hands the pieces of the
// line to the others through shared memory, warp 13 issues the MMAs.
//
// Measured (GB300, 32 query and 8 kv heads of 128, bf16): 865-905 us from one
// GPU to another for 4096 queries of a 20480-token context, 1370-1430 TFLOP/s,
// 0.73-0.77 of the measured 16-bit rate (fp16 944, D = 64 877); 180 us for six ragged prompts of 6294 tokens (0.31: a row tile there
// has about 8 key tiles, and its queries, masked tile and rows' way out weigh
// as much).  A step of 256 rows and 128 keys needs 2048 tensor cycles and takes
// about 3500: within a half scores, maximum, weights and the second product
// follow each other, and the other half covers only part of that.  What moved
// it: the register split, MMAs issued by an elected lane of a converged warp and
// loops kept rolled for the instruction cache (1305 -> 942 us), waits that sleep
// (942 -> 919; later 900 against 867 without the sleep), rows leaving through shared memory
// and the cheaper conversion of V (919 -> 892).  What did not: two threads per
// row (1006), weights against the old reference before any maximum (1007).
#pragma once

#include <type_traits>

#include "kv_attention_params.cuh"

namespace fp8l {
namespace {

constexpr int kProRows = 256;     // query rows per tile, two halves
constexpr int kProKeys = 128;
constexpr int kProThreads = 512;
constexpr int kProWarps = kProThreads / 32;
constexpr int kProMaxKStages = 4;
constexpr int kProMaxVStages = 2;
constexpr int kProScaleSlots = 8;  // tiles whose page scales are held
constexpr int kProSegments = 8;    // pieces between the copy warp and the softmax halves
constexpr int kProMaxCtas = 160;
// registers per thread of the softmax, converter and other warpgroups after
// the split: 2 x 160 + 104 + 88 = 4 x 128, what the block starts with (184,
// 88, 56 measured 1.5 % slower)
constexpr int kProSoftmaxRegs = 160, kProConvertRegs = 104, kProOtherRegs = 88;
constexpr int kProFan = 8;         // partials added by one CTA
constexpr int kProLevels = 3;      // 8^3 CTAs and more
constexpr float kProHead = 7.0f;   // reference below the maximum it was set from
constexpr float kProMove = 15.0f;  // a score this far above moves it

template <int QDT, int DIM>
struct ProSmem {
    static constexpr int kParts = QDT == FP8L_BF16 ? 2 : 3;
    static constexpr int kTileBytes = kProKeys * DIM;          // K or V codes
    static constexpr int kQPart = 128 * DIM;                   // one part of one half
    static constexpr int kQBytes = 2 * kParts * kQPart;
    static constexpr int kV16Bytes = 2 * kProKeys * DIM;       // per buffer
    static constexpr int kKStages = DIM == 64 ? 4 : (QDT == FP8L_BF16 ? 3 : 2);
    static constexpr int kVStages = DIM == 64 || QDT == FP8L_BF16 ? 2 : 1;
    static constexpr int kKOff = kQBytes;
    static constexpr int kVOff = kKOff + kKStages * kTileBytes;
    static constexpr int kV16Off = kVOff + kVStages * kTileBytes;
    static constexpr int kScaleOff = kV16Off + 2 * kV16Bytes;               // [slot][2][8] floats
    static constexpr int kFactorOff = kScaleOff + kProScaleSlots * 16 * 4;  // [slot][8] float4
    static constexpr int kQfOff = kFactorOff + kProScaleSlots * 8 * 16;     // [256] floats
    static constexpr int kSegOff = kQfOff + kProRows * 4;                   // [kProSegments] ProSegment
    static constexpr int kBarOff = kSegOff + kProSegments * 64;
    static constexpr int kBars =
        2 * kProMaxKStages + 2 * kProMaxVStages + 2 * kProScaleSlots + 2 * kProSegments + 4 + 8 + 3;
    static constexpr int kMiscOff = kBarOff + kBars * 8;
    static constexpr int kBytes = kMiscOff + 16;
    static_assert(kBytes <= 227 * 1024 - 320, "one CTA's shared memory, beside the static variables");
};

// The same with A in tensor memory, fp16
__device__ __forceinline__ void mma_f16_desc(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t b_hi,
                                            uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "mov.b64 b, {%2, %3};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate)
        : "memory");
}

// E4M3 codes of two fp16 pairs (in order), which become what the codes leave
// over (exact: the difference of a value and its rounding to fewer bits)
__device__ __forceinline__ uint32_t take_part_f16(uint32_t &a, uint32_t &b) {
    uint32_t c, x, y;
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "cvt.rn.satfinite.e4m3x2.f16x2 lo, %3;\n\tcvt.rn.satfinite.e4m3x2.f16x2 hi, %4;\n\t"
        "mov.b32 %0, {lo, hi};\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, lo;\n\tcvt.rn.f16x2.e4m3x2 %2, hi;\n\t}"
        : "=r"(c), "=r"(x), "=r"(y)
        : "r"(a), "r"(b));
    const __half2 da = __hsub2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&x));
    const __half2 db = __hsub2(*reinterpret_cast<const __half2 *>(&b), *reinterpret_cast<const __half2 *>(&y));
    a = *reinterpret_cast<const uint32_t *>(&da);
    b = *reinterpret_cast<const uint32_t *>(&db);
    return c;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

__device__ __forceinline__ float max16(const uint32_t *v) {
    float m[5];
#pragma unroll
    for (int i = 0; i < 5; ++i)
        m[i] = max3(__uint_as_float(v[3 * i]), __uint_as_float(v[3 * i + 1]), __uint_as_float(v[3 * i + 2]));
    return max3(max3(m[0], m[1], m[2]), max3(m[3], m[4], __uint_as_float(v[15])), __uint_as_float(v[15]));
}

// A request's rows and keys
struct ProRequest {
    int n, row0, keys, tiles;  // new tokens, first row, keys, row tiles
};

__device__ __forceinline__ ProRequest pro_request(const AttnParams &p, int r) {
    ProRequest d;
    const int a = min(max(p.q_offsets[r], 0), p.tokens), b = min(max(p.q_offsets[r + 1], 0), p.tokens);
    const int64_t cap = static_cast<int64_t>(p.table_width) << p.page_shift;
    const int L = min(max(p.kv_lens[r], 0), INT32_MAX - 255);  // (a tile's last key fits an int)
    d.keys = static_cast<int64_t>(L) < cap ? L : static_cast<int>(cap);
    d.n = max(b - a, 0);
    d.row0 = a;
    // (rows fit 32 bits: tokens * q_heads does)
    d.tiles = (d.n * (p.q_heads / p.kv_heads) + kProRows - 1) / kProRows;
    return d;
}

// The keys [first, last] that row tile j's rows see between them (last < 0:
// none), and its key tiles, one at least: a tile without keys writes zeros.
struct ProKeys {
    int first, last, begin, tiles;
};

__device__ __forceinline__ ProKeys pro_keys(const AttnParams &p, const ProRequest &d, int j) {
    const int group = p.q_heads / p.kv_heads;
    const int lo = j * kProRows;
    const int hi = min(lo + kProRows, d.n * group);
    const int before = d.keys - d.n;
    ProKeys k;
    k.last = before + (hi - 1) / group;
    k.first = p.window > 0 ? max(0, before + lo / group - p.window + 1) : 0;
    k.begin = k.first / kProKeys;
    k.tiles = k.last < 0 ? 1 : k.last / kProKeys - k.begin + 1;
    return k;
}

// A piece of one row tile, as the copy warp hands it to the other roles
// through shared memory (they keep none of it in registers over the tiles)
struct ProSegment {
    int tile, end;         // key tiles of this piece
    int begin, stop;       // of the whole row tile
    int first, last;       // keys seen
    int g, row0;           // kv head, the request's first token row
    int row_first, rows;   // first (token, head) row of the tile, how many
    int before;            // position of the request's first new token
    int done;              // tiles of the CTA's piece before this one; tile == end: no more
    int r, pad[3];
};

struct ProWalk {
    int done, left;  // tiles of the CTA's piece behind and ahead
    int r, g, j, offset;
    __device__ __forceinline__ bool next(const AttnParams &p, ProSegment &s) {
        if (left <= 0) return false;
        ProRequest d = pro_request(p, r);
        while (d.tiles == 0) {
            if (++r >= p.requests) return false;
            d = pro_request(p, r);
        }
        const ProKeys k = pro_keys(p, d, j);
        s.r = r;
        s.g = g;
        s.row0 = d.row0;
        s.row_first = j * kProRows;
        s.rows = min(d.n * (p.q_heads / p.kv_heads) - s.row_first, kProRows);
        s.before = d.keys - d.n;
        s.first = k.first;
        s.last = k.last;
        s.begin = k.begin;
        s.stop = k.begin + k.tiles;
        s.tile = k.begin + offset;
        const int take = min(k.tiles - offset, left);
        s.end = s.tile + take;
        s.done = done;
        done += take;
        left -= take;
        offset += take;
        if (offset == k.tiles) {
            offset = 0;
            if (++j == d.tiles) {
                j = 0;
                if (++g == p.kv_heads) {
                    g = 0;
                    if (++r >= p.requests) left = 0;
                }
            }
        }
        return true;
    }
};

// Key tiles of one kv head of request r, summed by the warp's lanes
__device__ __forceinline__ long long pro_request_work(const AttnParams &p, int r, int lane) {
    const ProRequest d = pro_request(p, r);
    long long n = 0;
    for (int j = lane; j < d.tiles; j += 32) n += pro_keys(p, d, j).tiles;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xFFFFFFFFu, n, o);
    return n;
}

template <int QDT, int DIM>
__global__ void __launch_bounds__(kProThreads, 1) kv_attention_prompt_kernel(const AttnParams p) {
    using Sm = ProSmem<QDT, DIM>;
    extern __shared__ __align__(128) uint8_t pro_smem[];
    __shared__ long long warp_work[kProWarps];
    __shared__ int start_r, start_g, start_j, start_offset, merge_now[2];
    const uint32_t sbase = smem_u32(pro_smem);
    const uint32_t bars = sbase + Sm::kBarOff;
    int next_bar = 0;
    auto take_bars = [&](int n) {
        const uint32_t b = bars + 8u * next_bar;
        next_bar += n;
        return b;
    };
    const uint32_t kfull = take_bars(kProMaxKStages), kempty = take_bars(kProMaxKStages);
    const uint32_t vfull = take_bars(kProMaxVStages), vempty = take_bars(kProMaxVStages);
    const uint32_t scfull = take_bars(kProScaleSlots);
    const uint32_t fcfull = take_bars(kProScaleSlots);
    const uint32_t segfull = take_bars(kProSegments), segfree = take_bars(kProSegments);
    const uint32_t v16full = take_bars(2), v16free = take_bars(2);
    const uint32_t sfull = take_bars(2), wfull = take_bars(4), odone = take_bars(2);
    const uint32_t qfull = take_bars(2), done_bar = take_bars(1);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(pro_smem + Sm::kMiscOff);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < Sm::kKStages; ++s) {
            mbar_init(kfull + 8 * s, 1);
            mbar_init(kempty + 8 * s, 1);
        }
        for (int s = 0; s < kProSegments; ++s) {
            mbar_init(segfull + 8 * s, 1);
            mbar_init(segfree + 8 * s, 256);
        }
        for (int s = 0; s < kProScaleSlots; ++s) {
            mbar_init(scfull + 8 * s, 32);
            mbar_init(fcfull + 8 * s, 8);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(vfull + 8 * s, 1);
            mbar_init(vempty + 8 * s, 128);
            mbar_init(v16full + 8 * s, 128);
            mbar_init(v16free + 8 * s, 1);
            mbar_init(sfull + 8 * s, 1);
            mbar_init(wfull + 16 * s, 128);
            mbar_init(wfull + 16 * s + 8, 128);
            mbar_init(odone + 8 * s, 1);
            mbar_init(qfull + 8 * s, 128);
        }
        mbar_init(done_bar, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == 13) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(tmem_slot)),
                     "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    grid_dependency_sync();

    // the line of tiles (each warp sums a run of requests) and this CTA's piece
    const int per_warp = (p.requests + kProWarps - 1) / kProWarps;
    const int r_begin = min(warp * per_warp, p.requests), r_end = min(r_begin + per_warp, p.requests);
    {
        long long n = 0;
        for (int r = r_begin; r < r_end; ++r) n += pro_request_work(p, r, lane) * p.kv_heads;
        if (lane == 0) warp_work[warp] = n;
    }
    __syncthreads();
    long long total = 0, before = 0;
    for (int w = 0; w < kProWarps; ++w) {
        if (w < warp) before += warp_work[w];
        total += warp_work[w];
    }
    const long long ctas = min(static_cast<long long>(gridDim.x), total);
    const long long cta = static_cast<long long>(blockIdx.x);
    const bool idle = cta >= ctas;
    const long long w0 = idle ? 0 : piece_begin(total, cta, ctas), w1 = idle ? 0 : piece_begin(total, cta + 1, ctas);
    if (!idle && before <= w0 && w0 < before + warp_work[warp]) {
        long long rest = w0 - before;
        for (int r = r_begin; r < r_end; ++r) {
            const long long n = pro_request_work(p, r, lane);
            if (rest >= n * p.kv_heads) {
                rest -= n * p.kv_heads;
                continue;
            }
            const ProRequest d = pro_request(p, r);
            const int g = static_cast<int>(rest / n);
            rest %= n;
            for (int j0 = 0; j0 < d.tiles; j0 += 32) {
                const int j = j0 + lane;
                const long long mine = j < d.tiles ? pro_keys(p, d, j).tiles : 0;
                long long inc = mine;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const long long x = __shfl_up_sync(0xFFFFFFFFu, inc, o);
                    if (lane >= o) inc += x;
                }
                if (rest >= inc - mine && rest < inc) {
                    start_r = r;
                    start_g = g;
                    start_j = j;
                    start_offset = static_cast<int>(rest - (inc - mine));
                }
                const long long chunk = __shfl_sync(0xFFFFFFFFu, inc, 31);
                if (rest < chunk) break;
                rest -= chunk;
            }
            break;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int group = p.q_heads / p.kv_heads;
    ProSegment *segs = reinterpret_cast<ProSegment *>(pro_smem + Sm::kSegOff);
    // piece number n, or nullptr after the last (or a time-out)
    auto segment_at = [&](int n) -> const ProSegment * {
        if (!kv_wait(segfull + 8 * (n & (kProSegments - 1)), (n / kProSegments) & 1u, abort_flag, p.status,
                      p.wait_cycles))
            return nullptr;
        const ProSegment *s = segs + (n & (kProSegments - 1));
        return s->tile < s->end ? s : nullptr;
    };

    if (warp >= 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kProOtherRegs));

      if (warp == 12) {
        // ---------------------------------------------------------- copies
        const int P = 1 << p.page_shift, per_tile = kProKeys >> p.page_shift;
        const int i = lane & 7;
        int kst = 0, vst = 0, count = 0, segment = 0;
        uint32_t kph = 0, vph = 0, kissued = 0, kpar = 0, vissued = 0, vpar = 0;
        bool ok = true;
        ProWalk walk{0, static_cast<int>(w1 - w0), idle ? 0 : start_r, idle ? 0 : start_g, idle ? 0 : start_j,
                     idle ? 0 : start_offset};
        ProSegment s;
        while (ok) {
            const bool more = walk.next(p, s);
            if (!more) s.tile = s.end = 0;
            // (half 1 can fall behind where pieces have no rows for it; the
            // other roles cannot, the stages hold them together)
            ok = __all_sync(0xFFFFFFFFu, kv_wait(segfree + 8 * (segment & (kProSegments - 1)),
                                                  ((segment / kProSegments) & 1u) ^ 1u, abort_flag, p.status,
                                                  p.wait_cycles));
            if (!ok) break;
            if (lane == 0) {
                segs[segment & (kProSegments - 1)] = s;
                mbar_arrive(segfull + 8 * (segment & (kProSegments - 1)));
            }
            __syncwarp();
            ++segment;
            if (!more) break;
            const int32_t *table = p.block_table + static_cast<int64_t>(s.r) * p.table_width;
            auto wanted = [&](int tile) {
                const int64_t b = static_cast<int64_t>(tile) * per_tile + i;
                return lane < 16 && i < per_tile && (b << p.page_shift) <= s.last &&
                       ((b + 1) << p.page_shift) > s.first;
            };
            int page = wanted(s.tile) ? table[s.tile * per_tile + i] : 0;
            for (int tile = s.tile; tile < s.end; ++tile, ++count) {
                const bool mine = wanted(tile);
                const int64_t ph = static_cast<int64_t>(min(max(page, 0), p.num_pages - 1)) * p.kv_heads + s.g;
                if (tile + 1 < s.end) page = wanted(tile + 1) ? table[(tile + 1) * per_tile + i] : 0;
                uint32_t bytes = 0;
                if (mine) {
                    const int in_page = min(s.last + 1 - ((tile * per_tile + i) << p.page_shift), P);
                    bytes = static_cast<uint32_t>((in_page + 7) / 8 * 8 * DIM);
                }
                uint32_t sum = lane < 8 ? bytes : 0u;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
                // keys, and the scales of keys and values
                ok = __all_sync(0xFFFFFFFFu,
                                kv_wait(kempty + 8 * kst, kph ^ 1u, abort_flag, p.status, p.wait_cycles));
                if (!ok) break;
                if (lane == 0) mbar_expect_tx(kfull + 8 * kst, sum);
                __syncwarp();
                if (mine) {
                    if (lane < 8)
                        bulk_copy(sbase + Sm::kKOff + kst * Sm::kTileBytes + i * P * DIM, p.k_cache + ph * P * DIM,
                                  bytes, kfull + 8 * kst);
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(
                                     sbase + Sm::kScaleOff +
                                     static_cast<uint32_t>(((count & (kProScaleSlots - 1)) * 16 + lane) * 4)),
                                 "l"((lane < 8 ? p.k_scale : p.v_scale) + ph)
                                 : "memory");
                }
                asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(
                                 scfull + 8 * (count & (kProScaleSlots - 1)))
                             : "memory");
                kissued |= 1u << kst;
                kpar = (kpar & ~(1u << kst)) | (kph << kst);
                if (++kst == Sm::kKStages) {
                    kst = 0;
                    kph ^= 1u;
                }
                // values
                ok = __all_sync(0xFFFFFFFFu,
                                kv_wait(vempty + 8 * vst, vph ^ 1u, abort_flag, p.status, p.wait_cycles));
                if (!ok) break;
                if (lane == 0) mbar_expect_tx(vfull + 8 * vst, sum);
                __syncwarp();
                if (mine && lane >= 8)
                    bulk_copy(sbase + Sm::kVOff + vst * Sm::kTileBytes + i * P * DIM, p.v_cache + ph * P * DIM, bytes,
                              vfull + 8 * vst);
                vissued |= 1u << vst;
                vpar = (vpar & ~(1u << vst)) | (vph << vst);
                if (++vst == Sm::kVStages) {
                    vst = 0;
                    vph ^= 1u;
                }
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        for (int x = 0; x < Sm::kKStages; ++x)
            if (kissued & (1u << x)) kv_drain(kfull + 8 * x, (kpar >> x) & 1u, p.status);
        for (int x = 0; x < Sm::kVStages; ++x)
            if (vissued & (1u << x)) kv_drain(vfull + 8 * x, (vpar >> x) & 1u, p.status);
      } else if (warp == 13) {
        // ---------------------------------------------------------- MMAs
        {
            const bool leader = elect_one();
            const uint32_t tmem_u = __shfl_sync(0xFFFFFFFFu, tmem, 0);
            const uint32_t idesc_s = (1u << 4) | (static_cast<uint32_t>(kProKeys >> 3) << 17) | (8u << 24);
            const uint32_t idesc_o = (1u << 4) | (1u << 16) | (static_cast<uint32_t>(DIM >> 3) << 17) | (8u << 24);
            auto wait = [&](uint32_t bar, uint32_t parity) {
                return __all_sync(0xFFFFFFFFu, kv_wait(bar, parity & 1u, abort_flag, p.status, p.wait_cycles));
            };
            bool ok = true;
            if (p.stall & kStallMma) ok = wait(done_bar, 0);
            int kst = 0, count = 0, segment = 0;
            uint32_t kph = 0;
            int uses[2] = {0, 0}, segments1 = 0;  // score tiles of each half, pieces of half 1 so far
            const uint32_t q_lo = desc_lo(sbase, 128), k_lo0 = desc_lo(sbase + Sm::kKOff, 128);
            const uint32_t v_lo0 = desc_lo(sbase + Sm::kV16Off, 16 * DIM);
            uint32_t k_lo = k_lo0;
            auto scores = [&](auto half_c) {
                constexpr int half = decltype(half_c)::value;
                if (!leader) return;
#pragma unroll
                for (int part = 0; part < Sm::kParts; ++part) {
#pragma unroll
                    for (int x = 0; x < DIM / 32; ++x) {
                        const uint32_t a = q_lo + ((half * Sm::kParts + part) * Sm::kQPart + 256 * x) / 16;
                        const uint32_t b = k_lo + 256 * x / 16;
                        mma_f8_desc(tmem_u + 128u * half, a, desc_hi(8 * DIM), b, desc_hi(8 * DIM), idesc_s, (part | x) != 0 ? 1u : 0u);
                    }
                }
                mma_commit(sfull + 8 * half);
            };
            // O += W V of tile number `tile` (its V buffer), use u of the half
            auto values = [&](auto half_c, int tile, int u, bool first) {
                constexpr int half = decltype(half_c)::value;
                if (!wait(v16full + 8 * (tile & 1), tile >> 1)) return false;
                const uint32_t v = v_lo0 + ((tile & 1) ? Sm::kV16Bytes / 16 : 0);
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    if (!wait(wfull + 16 * half + 8 * y, u)) return false;
                    tc_fence_after();
                    if (leader) {
#pragma unroll
                        for (int x = y * kProKeys / 32; x < (y + 1) * kProKeys / 32; ++x)
                            mma_f16_desc(tmem_u + 256u + 128u * half, tmem_u + 128u * half + 8u * x, v + 32 * DIM * x / 16,
                                desc_hi(128), idesc_o, x == 0 ? (first ? 0u : 1u) : 1u);
                    }
                }
                if (leader) mma_commit(odone + 8 * half);
                return true;
            };
            using Half0 = std::integral_constant<int, 0>;
            using Half1 = std::integral_constant<int, 1>;
            while (ok) {
                const ProSegment *s = segment_at(segment);
                if (__any_sync(0xFFFFFFFFu, s == nullptr)) break;
                const bool two = s->rows > 128;
                const int tiles = s->end - s->tile;
                bool pending = false;  // half 1 of the tile before
                ok = wait(qfull, segment);
                for (int tile = 0; ok && tile < tiles; ++tile, ++count) {
                    ok = wait(kfull + 8 * kst, kph);
                    if (!ok) break;
                    tc_fence_after();
                    scores(Half0{});
                    if (pending) {
                        ok = values(Half1{}, count - 1, uses[1] - 1, tile == 1);
                        if (!ok) break;
                        if (leader) mma_commit(v16free + 8 * ((count - 1) & 1));
                    }
                    if (two) {
                        if (tile == 0) {
                            ok = wait(qfull + 8, segments1++);
                            if (!ok) break;
                            tc_fence_after();
                        }
                        scores(Half1{});
                        ++uses[1];
                    }
                    if (leader) mma_commit(kempty + 8 * kst);
                    ok = values(Half0{}, count, uses[0], tile == 0);
                    if (!ok) break;
                    ++uses[0];
                    if (leader && !two) mma_commit(v16free + 8 * (count & 1));
                    pending = two;
                    k_lo += Sm::kTileBytes / 16;
                    if (++kst == Sm::kKStages) {
                        kst = 0;
                        kph ^= 1u;
                        k_lo = k_lo0;
                    }
                }
                if (ok && pending) {
                    ok = values(Half1{}, count - 1, uses[1] - 1, tiles == 1);
                    if (ok && leader) mma_commit(v16free + 8 * ((count - 1) & 1));
                }
                ++segment;
            }
            if (leader) mma_commit(done_bar);
        }
        __syncwarp();
      }
    } else if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kProConvertRegs));

        // ------------------------------------- V to fp16, the scales' factors
        const int tid = static_cast<int>(threadIdx.x) - 256;
        int vst = 0, count = 0, segment = 0;
        uint32_t vph = 0;
        bool ok = true;
        while (const ProSegment *sp = segment_at(segment)) {
            const int first = sp->first, last = sp->last, end = sp->end;
            ++segment;
            for (int tile = sp->tile; tile < end; ++tile, ++count) {
                if (tid < 8) {
                    // factors of the 16 keys from 16 tid on: their page's
                    // scales; a page without a seen key was not copied
                    const int slot = count & (kProScaleSlots - 1), pg = (16 * tid) >> p.page_shift;
                    const int key = tile * kProKeys + 16 * tid;
                    ok = ok && kv_wait(scfull + 8 * slot, (count / kProScaleSlots) & 1u, abort_flag, p.status,
                                              p.wait_cycles);
                    const float *sc = reinterpret_cast<const float *>(pro_smem + Sm::kScaleOff) + slot * 16;
                    const bool there = key <= last && key + 15 >= first;
                    const float ks = there ? sc[pg] : 0.0f, vs = there ? value_scale(sc[8 + pg]) : 1.0f;
                    reinterpret_cast<float4 *>(pro_smem + Sm::kFactorOff)[slot * 8 + tid] =
                        make_float4(ks, __log2f(vs), __isnanf(vs) ? 0.0f : __frcp_rn(vs), 0.0f);
                    mbar_arrive(fcfull + 8 * slot);
                }
                constexpr int PIECES = kProKeys * DIM / 16 / 128;  // 16-byte pieces per thread
                ok = ok && kv_wait(vfull + 8 * vst, vph, abort_flag, p.status, p.wait_cycles);
                const uint8_t *src = pro_smem + Sm::kVOff + vst * Sm::kTileBytes;
                uint4 u[PIECES];
#pragma unroll
                for (int k = 0; k < PIECES; ++k) {
                    const int piece = tid + 128 * k;
                    u[k] = *reinterpret_cast<const uint4 *>(src + 16 * piece);
                }
                if (tile * kProKeys < first || tile * kProKeys + kProKeys - 1 > last) {
                    // keys that are not there: whatever the stage holds (NaN
                    // codes too) must not meet their zero weights
#pragma unroll
                    for (int k = 0; k < PIECES; ++k) {
                        const int piece = tid + 128 * k;
                        const int key = tile * kProKeys + piece / (DIM / 2) * 8 + (piece & 7);
                        if (key < first || key > last) u[k] = make_uint4(0u, 0u, 0u, 0u);
                    }
                }
                mbar_arrive(vempty + 8 * vst);
                if (++vst == Sm::kVStages) {
                    vst = 0;
                    vph ^= 1u;
                }
                const int b = count & 1;
                ok = ok && kv_wait(v16free + 8 * b, ((count >> 1) & 1u) ^ 1u, abort_flag, p.status,
                                          p.wait_cycles);
                uint8_t *dst = pro_smem + Sm::kV16Off + b * Sm::kV16Bytes;
#pragma unroll
                for (int k = 0; k < PIECES; ++k) {
                    const int piece = tid + 128 * k;
                    const uint32_t w[4] = {u[k].x, u[k].y, u[k].z, u[k].w};
                    uint32_t h[8];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\t"
                            "cvt.rn.f16x2.e4m3x2 %0, lo;\n\tcvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
                            : "=r"(h[2 * i]), "=r"(h[2 * i + 1])
                            : "r"(w[i]));
                    // [octet][D / 8][8 keys][8 dimensions]
                    uint8_t *at = dst + piece / (DIM / 2) * 16 * DIM + piece % (DIM / 2) / 8 * 256 + (piece & 7) * 16;
                    *reinterpret_cast<uint4 *>(at) = make_uint4(h[0], h[1], h[2], h[3]);
                    *reinterpret_cast<uint4 *>(at + 128) = make_uint4(h[4], h[5], h[6], h[7]);
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                mbar_arrive(v16full + 8 * b);
            }
        }
    } else {

        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kProSoftmaxRegs));
        // ---------------------------------------------------------- softmax
        const int half = warp >> 2, tid = static_cast<int>(threadIdx.x) & 127;
        const uint32_t lane_addr = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t s_tmem = tmem + lane_addr + 128u * half, o_tmem = tmem + lane_addr + 256u + 128u * half;
        float *qf = reinterpret_cast<float *>(pro_smem + Sm::kQfOff) + 128 * half;
        const float4 *factors = reinterpret_cast<const float4 *>(pro_smem + Sm::kFactorOff);
        int count = 0, segment = 0, uses = 0;
        bool ok = true;
        // a piece, with one answer for the half's threads, whose barriers
        // below need all of them (a wait can give up in one thread and not in
        // another)
        auto piece = [&](int n) -> const ProSegment * {
            const ProSegment *s = segment_at(n);
            return group_any(1 + half, s == nullptr) ? nullptr : s;
        };
        // this thread is through with piece n
        auto release = [&](int n) { mbar_arrive(segfree + 8 * (n & (kProSegments - 1))); };
        const ProSegment *s = piece(0);
        while (s != nullptr) {
            const int rows = s->rows - 128 * half;  // valid rows of this half
            const int end = s->end, begin = s->tile;
            if (rows <= 0) {
                count += end - begin;
                release(segment);
                s = piece(++segment);
                continue;
            }
            const bool warp_on = (tid & ~31) < rows;
            const int pos = s->before + (s->row_first + 128 * half + tid) / group;
            // positions of the warp's first and last valid row
            const int pos_lo = __shfl_sync(0xFFFFFFFFu, pos, 0);
            const int pos_hi = __shfl_sync(0xFFFFFFFFu, pos, min(31, max(rows - 1 - (tid & ~31), 0)));
            // The queries as E4M3 parts, and each row's factor.  (The half's
            // earlier score MMAs have retired: it has read their results.)  A
            // warp's 32 rows, eight at a time: lane (r, c) = (lane % 8, lane / 8)
            // holds the 16-dimension chunks c, c + 4 of row r, so that eight
            // lanes store one 128-byte core matrix.
            {
                constexpr int CHUNKS = DIM / 64;
                const int qr = lane & 7, qc = lane >> 3;
                uint4 raw[4][2 * CHUNKS];
                const int first = 128 * half + 32 * (warp & 3) + qr, row_first = s->row_first + first;
                int token = row_first / group, member = row_first % group;
                const int token_step = 8 / group, member_step = 8 % group;
                const uint16_t *q0 = p.q + static_cast<int64_t>(s->row0) * p.q_stride + s->g * group * DIM + 16 * qc;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint16_t *at = q0 + static_cast<int64_t>(token) * p.q_stride + member * DIM;
#pragma unroll
                    for (int x = 0; x < 2 * CHUNKS; ++x) {
                        raw[k][x] = make_uint4(0u, 0u, 0u, 0u);
                        if (first + 8 * k < s->rows)
                            raw[k][x] = *reinterpret_cast<const uint4 *>(at + (x >> 1) * 64 + (x & 1) * 8);
                    }
                    token += token_step;
                    member += member_step;
                    if (member >= group) {
                        member -= group;
                        ++token;
                    }
                }
                uint8_t *dst = pro_smem + half * Sm::kParts * Sm::kQPart + (warp & 3) * 32 * DIM + qc * 128 + qr * 16;
#pragma unroll 1
                for (int b = 0; b < 4; ++b) {
                    uint32_t mag = 0;
#pragma unroll
                    for (int x = 0; x < 2 * CHUNKS; ++x) mag = word_mag_max<QDT>(raw[0][x], mag);
                    mag = fold_mag<QDT>(mag);
                    mag = max(mag, __shfl_xor_sync(0xFFFFFFFFu, mag, 8));
                    mag = max(mag, __shfl_xor_sync(0xFFFFFFFFu, mag, 16));
                    const float most = mag_bits_to_float<QDT>(mag);
                    const int e = part_exponent(most);
                    const uint32_t up = static_cast<uint32_t>(127 + e) << 23;
                    if (qc == 0) qf[32 * (warp & 3) + 8 * b + qr] = part_factor(p.score_scale, most, e);
#pragma unroll
                    for (int x = 0; x < CHUNKS; ++x) {
                        // the scaled row in fp16: exact from 2^-22 of its
                        // largest element on, further than the parts reach
                        uint32_t h[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const uint4 &u = raw[0][2 * x + (i >> 2)];
                            const uint32_t w = (i & 3) == 0 ? u.x : ((i & 3) == 1 ? u.y : ((i & 3) == 2 ? u.z : u.w));
                            const uint64_t x2 = f2_mul(widen16<QDT>(w), f2_pack(up, up));
                            const __half2 y = __floats2half2_rn(__uint_as_float(static_cast<uint32_t>(x2)),
                                                                __uint_as_float(static_cast<uint32_t>(x2 >> 32)));
                            h[i] = *reinterpret_cast<const uint32_t *>(&y);
                        }
#pragma unroll
                        for (int part = 0; part < Sm::kParts; ++part) {
                            uint32_t c[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) c[i] = take_part_f16(h[2 * i], h[2 * i + 1]);
                            *reinterpret_cast<uint4 *>(dst + part * Sm::kQPart + b * 8 * DIM + x * 512) =
                                make_uint4(c[0], c[1], c[2], c[3]);
                        }
                    }
#pragma unroll
                    for (int k = 0; k < 3; ++k)
#pragma unroll
                        for (int x = 0; x < 2 * CHUNKS; ++x) raw[k][x] = raw[k + 1][x];
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                mbar_arrive(qfull + 8 * half);
                __syncwarp();  // the row factors are written
            }
            const float f = qf[tid];
            float m = -INFINITY, l = __isnanf(f) ? f : 0.0f;
            for (int tile = begin; tile < end; ++tile, ++count, ++uses) {
                // (a barrier per slot, not the key stage's, which may be
                // filled again while this half is still in an epilogue)
                ok = ok && kv_wait(fcfull + 8 * (count & (kProScaleSlots - 1)), (count / kProScaleSlots) & 1u,
                                          abort_flag, p.status, p.wait_cycles);
                ok = ok && kv_wait(sfull + 8 * half, uses & 1u, abort_flag, p.status, p.wait_cycles);
                tc_fence_after();
                if (warp_on) {
                    const float4 *fc = factors + (count & (kProScaleSlots - 1)) * 8;
                    const int key0 = tile * kProKeys;
                    // 64 columns at a time, read twice (maximum, weights): a
                    // row of 128 scores does not fit the registers, and the
                    // loops are kept rolled: their code fits the instruction
                    // cache beside the other roles'
                    uint32_t v[2][32];
                    const bool masked =
                        !(key0 + kProKeys - 1 <= pos_lo && (p.window == 0 || key0 > pos_hi - p.window));
                    auto load = [&](int x) {
                        tmem_ld32_nowait(s_tmem + 64 * x, v[0]);
                        tmem_ld32_nowait(s_tmem + 64 * x + 32, v[1]);
                        tmem_wait_ld();
                    };
                    float top = -INFINITY;
#pragma unroll 1
                    for (int x = 0; x < 2; ++x) {
                        load(x);
                        if (masked) {
                            // columns [lo, hi) are seen by this row; 32 that
                            // all rows of the warp see are left alone, the
                            // others go back masked for the second reading
                            const int c0 = key0 + 64 * x;
                            const int lo = p.window > 0 ? pos - p.window + 1 - c0 : 0, hi = pos + 1 - c0;
                            auto below = [](int n) { return n <= 0 ? 0u : (n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u); };
                            const int lo_all = p.window > 0 ? pos_hi - p.window + 1 - c0 : 0, hi_all = pos_lo + 1 - c0;
#pragma unroll
                            for (int y = 0; y < 2; ++y) {
                                if (32 * y >= lo_all && 32 * y + 32 <= hi_all) continue;
                                const uint32_t seen = below(hi - 32 * y) & ~below(lo - 32 * y);
#pragma unroll
                                for (int i = 0; i < 32; ++i)
                                    if (!(seen & (1u << i))) v[y][i] = 0xFF800000u;  // -inf
                                tmem_st32_nowait(s_tmem + 64 * x + 32 * y, v[y]);
                            }
                            tmem_wait_st();
                        }
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            const float raw = max16(v[y / 2] + 16 * (y & 1));
                            const float4 k = fc[4 * x + y];
                            // (-inf where the row sees none of the 16 keys)
                            top = fmaxf(top, raw == -INFINITY ? raw : fmaf(raw, f * k.x, k.y));
                        }
                    }
                    const bool move = top > m + kProMove;
                    if (__any_sync(0xFFFFFFFFu, move)) {
                        const float to = move ? top - kProHead : m;
                        const float keep = to == -INFINITY ? 1.0f : (m == -INFINITY ? 0.0f : ex2(m - to));
                        l *= keep;
                        m = to;
                        if (tile != begin) {
                            ok = ok && kv_wait(odone + 8 * half, (uses - 1) & 1u, abort_flag, p.status,
                                                p.wait_cycles);
                            tc_fence_after();
#pragma unroll 1
                            for (int x = 0; x < DIM / 16; ++x) {
                                uint32_t o[16];
                                tmem_ld16_nowait(o_tmem + 16 * x, o);
                                tmem_wait_ld();
#pragma unroll
                                for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * keep);
                                tmem_st16_nowait(o_tmem + 16 * x, o);
                            }
                        }
                    }
                    const float mu = m == -INFINITY ? 0.0f : m;
#pragma unroll 1
                    for (int x = 0; x < 2; ++x) {
                        load(x);
                        uint32_t w[32];
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            const float4 k = fc[4 * x + y];
                            // (positive, so that -inf stays -inf where the
                            // factor is 0: a page that was not copied)
                            const float a = max_nan(f * k.x, 1e-37f), b = k.y - mu;
                            const uint64_t a2 = f2_pack(__float_as_uint(a), __float_as_uint(a));
                            const uint64_t b2 = f2_pack(__float_as_uint(b), __float_as_uint(b));
                            uint64_t sum[2] = {0, 0};
#pragma unroll
                            for (int i = 0; i < 16; i += 2) {
                                const uint32_t *c = v[y / 2] + 16 * (y & 1) + i;
                                const uint64_t t = f2_fma(f2_pack(c[0], c[1]), a2, b2);
                                const float w0 = ex2(__uint_as_float(static_cast<uint32_t>(t)));
                                const float w1 = ex2(__uint_as_float(static_cast<uint32_t>(t >> 32)));
                                sum[(i >> 1) & 1] =
                                    f2_add(sum[(i >> 1) & 1], f2_pack(__float_as_uint(w0), __float_as_uint(w1)));
                                const __half2 h = __floats2half2_rn(w0, w1);
                                w[8 * y + i / 2] = *reinterpret_cast<const uint32_t *>(&h);
                            }
                            const uint64_t both = f2_add(sum[0], sum[1]);
                            l = fmaf(__uint_as_float(static_cast<uint32_t>(both)) +
                                         __uint_as_float(static_cast<uint32_t>(both >> 32)), k.z, l);
                        }
                        tmem_st32_nowait(s_tmem + 32 * x, w);  // below the columns still to be read
                        // these keys can be multiplied
                        tmem_wait_st();
                        tc_fence_before();
                        mbar_arrive(wfull + 16 * half + 8 * x);
                    }
                } else {
                    tc_fence_before();
                    mbar_arrive(wfull + 16 * half);
                    mbar_arrive(wfull + 16 * half + 8);
                }
            }

            const ProSegment *next = piece(++segment);

            // ------------------------------------------------------ epilogue
            ok = ok && kv_wait(odone + 8 * half, (uses - 1) & 1u, abort_flag, p.status, p.wait_cycles);
            tc_fence_after();
            bool write = begin == s->begin && end == s->stop;
            const bool from_tmem = write;
            constexpr long long kPart = kProRows * (DIM + 2);
            // float4 number c of a row in a partial: rows adjoin, so
            // that a warp's rows are 512 contiguous bytes
            auto quad = [&](float *part, int c) {
                return reinterpret_cast<float4 *>(part) + c * kProRows + 128 * half + tid;
            };
            auto ml_of = [&](float *part) {
                return reinterpret_cast<float2 *>(part + kProRows * DIM) + 128 * half + tid;
            };
            int members = 0, step = 1, node = 0, c0 = 0;
            long long seg0 = 0;
            auto slot_of = [&](int c) { return (c0 + c) * 2 + (c == 0 && seg0 != piece_begin(total, c0, ctas) ? 1 : 0); };
            auto partial = [&](int c) { return p.partials + slot_of(c) * kPart; };
            auto last_of = [&](unsigned *counter, int parts) {
                __threadfence();
                group_sync(1 + half);
                if (tid == 0) {
                    merge_now[half] = atomicInc(counter, static_cast<unsigned>(parts - 1)) ==
                                      static_cast<unsigned>(parts - 1);  // wraps to 0
                    __threadfence();
                }
                group_sync(1 + half);
                const bool last = merge_now[half] != 0;
                group_sync(1 + half);
                return last;
            };
            float top = m, inv = 0.0f;
            // values c .. c + 31 of this thread's columns, added over the
            // members of a node
            auto merge32 = [&](int c, float (&o)[32]) {
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = 0.0f;
#pragma unroll 1
                for (int k = 0; k < members; ++k) {
                    float *part = partial((node + k) * step);
                    const float mk = __ldcg(ml_of(part)).x;
                    float4 x[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[i] = __ldcg(quad(part, c / 4 + i));
                    const float e = mk == -INFINITY ? 0.0f : ex2(mk - top);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        o[4 * i] = fmaf(x[i].x, e, o[4 * i]);
                        o[4 * i + 1] = fmaf(x[i].y, e, o[4 * i + 1]);
                        o[4 * i + 2] = fmaf(x[i].z, e, o[4 * i + 2]);
                        o[4 * i + 3] = fmaf(x[i].w, e, o[4 * i + 3]);
                    }
                }
            };
            auto put32 = [&](float *part, int c, const float (&o)[32]) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    *quad(part, c / 4 + i) = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
            };
            auto from_accumulator = [&](int c, float (&o)[32]) {
                uint32_t v[32];
                tmem_ld32_nowait(o_tmem + c, v);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = __uint_as_float(v[i]);
            };
            if (!write) {
                // the CTAs that share this row tile; a tree of fan-in kProFan
                seg0 = w0 + s->done - (begin - s->begin);
                c0 = piece_of(total, seg0, ctas);
                const int c1 = piece_of(total, seg0 + (s->stop - s->begin) - 1, ctas);
                int n = c1 - c0 + 1, index = static_cast<int>(cta) - c0;
                unsigned *counters = p.counters;
                if (warp_on) {
                    float *part = partial(index);
#pragma unroll 1
                    for (int c = 0; c < DIM; c += 32) {
                        float o[32];
                        from_accumulator(c, o);
                        put32(part, c, o);
                    }
                    *ml_of(part) = make_float2(m, l);
                }
                for (;;) {
                    node = index / kProFan * kProFan;
                    members = min(kProFan, n - node);
                    write = last_of(counters + slot_of(node * step) * 2 + half, members);
                    if (!write) break;
                    top = -INFINITY;
                    l = 0.0f;
                    if (warp_on) {
#pragma unroll 1
                        for (int k = 0; k < members; ++k) top = fmaxf(top, __ldcg(ml_of(partial((node + k) * step))).x);
#pragma unroll 1
                        for (int k = 0; k < members; ++k) {
                            const float2 ml = __ldcg(ml_of(partial((node + k) * step)));
                            // (a part without a reference: 0, or NaN)
                            l = fmaf(ml.y, ml.x == -INFINITY ? 1.0f : ex2(ml.x - top), l);
                        }
                    }
                    m = top;
                    if (n <= kProFan) break;
                    if (warp_on) {
                        float *to = partial(node * step);
#pragma unroll 1
                        for (int c = 0; c < DIM; c += 32) {
                            float o[32];
                            merge32(c, o);
                            put32(to, c, o);
                        }
                    }
                    group_sync(1 + half);  // the members' references have been read
                    if (warp_on) *ml_of(partial(node * step)) = make_float2(m, l);
                    index = node / kProFan;
                    step *= kProFan;
                    n = (n + kProFan - 1) / kProFan;
                    counters += kProMaxCtas * 2 * 2;
                }
            }
            if (write && warp_on) {
                // rows to the output's type in shared memory (the queries' are
                // not needed any more), then out in whole rows: a store per
                // row and thread would touch 32 lines
                inv = 1.0f / l;
                const bool codes = p.out_dtype == FP8L_E4M3;
                const int pieces = codes ? DIM / 16 : DIM / 8;  // 16 bytes each, per row
                uint8_t *stage = pro_smem + half * Sm::kParts * Sm::kQPart + (warp & 3) * 32 * 2 * DIM;
                auto at = [&](int row, int piece) {
                    return reinterpret_cast<uint4 *>(stage + (row * pieces + (piece ^ (row & (pieces - 1)))) * 16);
                };
#pragma unroll 1
                for (int c = 0; c < DIM; c += 32) {
                    float o[32];
                    if (from_tmem)
                        from_accumulator(c, o);
                    else
                        merge32(c, o);
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = l == 0.0f ? 0.0f : o[i] * inv;
                    const int col = c;
                    if (codes) {
                        const Quot d = Quot::make<FP8L_F32>(p.out_scale[0]);
                        uint32_t w[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) w[i] = attn_codes4(&o[4 * i], d);
                        *at(lane, col / 16) = make_uint4(w[0], w[1], w[2], w[3]);
                        *at(lane, col / 16 + 1) = make_uint4(w[4], w[5], w[6], w[7]);
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            *at(lane, col / 8 + i) = make_uint4(pack_out16(o[8 * i], o[8 * i + 1], p.out_dtype),
                                                                pack_out16(o[8 * i + 2], o[8 * i + 3], p.out_dtype),
                                                                pack_out16(o[8 * i + 4], o[8 * i + 5], p.out_dtype),
                                                                pack_out16(o[8 * i + 6], o[8 * i + 7], p.out_dtype));
                    }
                }
                __syncwarp();
                const int at_once = 32 / pieces;  // rows per step of the warp
                const int piece = lane % pieces, row_of = lane / pieces, warp_row = 32 * (warp & 3);
                const int first_row = s->row_first + 128 * half + warp_row + row_of;
                int token = first_row / group, member = first_row % group;
                const int token_step = at_once / group, member_step = at_once % group;
                const int64_t row_bytes = codes ? DIM : 2 * DIM;
                uint8_t *out = static_cast<uint8_t *>(p.out) + 16 * piece;
#pragma unroll 1
                for (int r = row_of; r < 32; r += at_once) {
                    if (warp_row + r < rows)
                        *reinterpret_cast<uint4 *>(out + (static_cast<int64_t>(s->row0 + token) * p.q_heads +
                                                          s->g * group + member) * row_bytes) = *at(r, piece);
                    token += token_step;
                    member += member_step;
                    if (member >= group) {
                        member -= group;
                        ++token;
                    }
                }
                if (p.lse != nullptr && tid < rows) {
                    const int row = s->row_first + 128 * half + tid;
                    attn_store_lse(p, s->row0 + row / group, s->g * group + row % group, m, l);
                }
            }
            tc_fence_before();
            group_sync(1 + half);  // the rows in shared memory have left
            release(segment - 1);
            s = next;
        }
    }

    // MMAs retired.  The two warps without a role wait at the barrier below: here
    // they would wait all the call, and a long one is no time-out.
    if (warp < 14) kv_drain(done_bar, 0, p.status);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    kv_report(abort_flag, p.library_status);
    if (warp == 13)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
}

}  // namespace
}  // namespace fp8l
