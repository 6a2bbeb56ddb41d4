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
// K is multiplied as stored: a 16-bit query row, scaled by a power of two, is
// the sum of two (bf16, exactly: 8 significand bits) or three (fp16) E4M3
// parts, which share the accumulator; two fp8 MMAs take the time of one
// 16-bit one and K is never widened.  The weights need a 16-bit format's
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
// when a score passes it by 15: weights stay below 2^15, fp16 keeps 11 bits
// down to 2^-28 of the row's largest.
//
// Work: the tiles (request, kv head, row tile, key tile) form one line, cut
// into equal pieces for one CTA per SM; row tiles that span pieces are merged
// by the last CTA to arrive, in CTA order, as in the decode kernel.
//
// Roles (448 threads): warps 0-3 and 4-7 softmax of halves 0 and 1 (warp w
// owns tensor-memory lanes 32 (w mod 4) ..), warps 8-11 queries to parts and V
// to fp16, warp 12 copies, warp 13 issues the MMAs.
#pragma once

#include "kv_attention_decode.cuh"

namespace fp8l {
namespace {

constexpr int kProRows = 256;     // query rows per tile, two halves
constexpr int kProKeys = 128;
constexpr int kProThreads = 448;
constexpr int kProWarps = kProThreads / 32;
constexpr int kProMaxKStages = 4;
constexpr int kProMaxVStages = 2;
constexpr int kProScaleSlots = 8;  // tiles whose page scales are held
constexpr int kProMaxCtas = 160;
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
    static constexpr int kQfOff = kScaleOff + kProScaleSlots * 16 * 4;      // [2][256] floats
    static constexpr int kBarOff = kQfOff + 2 * kProRows * 4;
    static constexpr int kBars = 2 * kProMaxKStages + 2 * kProMaxVStages + kProScaleSlots + 4 + 6 + 4;
    static constexpr int kMiscOff = kBarOff + kBars * 8;
    static constexpr int kBytes = kMiscOff + 16;
    static_assert(kBytes <= 227 * 1024 - 256, "one CTA's shared memory, beside the static variables");
};

__device__ __forceinline__ void pro_mma_f16(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc,
                                            uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void tmem_ld32_nowait(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
          "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
          "=r"(r[31])
        : "r"(taddr));
}

__device__ __forceinline__ void tmem_st32_nowait(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
        "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
        "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// E4M3 codes of two values (a in the low byte) and what they leave over
__device__ __forceinline__ uint32_t take_part_unscaled(float &a, float &b) {
    const uint32_t c = take_part(a, b);
    a *= 0.0625f;
    b *= 0.0625f;
    return c;
}

// A request's rows and keys
struct ProRequest {
    int n, row0, keys, tiles;  // new tokens, first row, keys, row tiles
};

__device__ __forceinline__ ProRequest pro_request(const AttnParams &p, int r) {
    ProRequest d;
    const int a = min(max(p.q_offsets[r], 0), p.tokens), b = min(max(p.q_offsets[r + 1], 0), p.tokens);
    const int64_t cap = static_cast<int64_t>(p.table_width) << p.page_shift;
    const int L = max(p.kv_lens[r], 0);
    d.keys = static_cast<int64_t>(L) < cap ? L : static_cast<int>(cap);
    d.n = max(b - a, 0);
    d.row0 = a;
    const int64_t rows = static_cast<int64_t>(d.n) * (p.q_heads / p.kv_heads);
    d.tiles = static_cast<int>((rows + kProRows - 1) / kProRows);
    return d;
}

// The keys [first, last] that row tile j's rows see between them (last < 0:
// none), and its key tiles, one at least: a tile without keys writes zeros.
struct ProKeys {
    int first, last, begin, tiles;
};

__device__ __forceinline__ ProKeys pro_keys(const AttnParams &p, const ProRequest &d, int j) {
    const int group = p.q_heads / p.kv_heads;
    const int64_t lo = static_cast<int64_t>(j) * kProRows;
    const int64_t all = static_cast<int64_t>(d.n) * group;
    const int64_t hi = lo + kProRows < all ? lo + kProRows : all;
    const int before = d.keys - d.n;
    ProKeys k;
    k.last = before + static_cast<int>((hi - 1) / group);
    k.first = p.window > 0 ? max(0, before + static_cast<int>(lo / group) - p.window + 1) : 0;
    k.begin = k.first / kProKeys;
    k.tiles = k.last < 0 ? 1 : k.last / kProKeys - k.begin + 1;
    return k;
}

struct ProSegment {
    int r, g, j;
    ProRequest req;
    ProKeys keys;
    int tile, end;  // key tiles of this piece
    long long at;   // number of `tile` in the line
};

struct ProWalk {
    long long at, left;
    int r, g, j, offset;
    __device__ __forceinline__ bool next(const AttnParams &p, ProSegment &s) {
        if (left <= 0) return false;
        s.req = pro_request(p, r);
        while (s.req.tiles == 0) {
            if (++r >= p.requests) return false;
            s.req = pro_request(p, r);
        }
        s.r = r;
        s.g = g;
        s.j = j;
        s.keys = pro_keys(p, s.req, j);
        s.tile = s.keys.begin + offset;
        const long long take = min(static_cast<long long>(s.keys.tiles - offset), left);
        s.end = s.tile + static_cast<int>(take);
        s.at = at;
        at += take;
        left -= take;
        offset += static_cast<int>(take);
        if (offset == s.keys.tiles) {
            offset = 0;
            if (++j == s.req.tiles) {
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

__device__ __forceinline__ void half_sync(int half) {
    asm volatile("barrier.cta.sync %0, 128;" ::"r"(1 + half) : "memory");
}

// Adds the CTAs' partials of one half of a row tile, in CTA order: a warp
// takes 16 rows at a time, DIM / 32 dimensions per lane.
template <int DIM, typename Partial>
__device__ __forceinline__ void pro_merge(const AttnParams &p, const ProSegment &s, int half, int rows, int group,
                                          int parts, const Partial &partial) {
    constexpr int V = DIM / 32, B = 16;
    const int warp = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31;
    for (int b = warp * 32; b < warp * 32 + 32 && b < rows; b += B) {
        // lanes 0-15 hold the rows' maxima and sums
        const int mine = 128 * half + b + (lane & (B - 1));
        float top = -INFINITY;
        for (int c = 0; c < parts; ++c) top = fmaxf(top, __ldcg(partial(c) + kProRows * DIM + 2 * mine));
        float sum = 0.0f, acc[B][V] = {};
        for (int c = 0; c < parts; ++c) {
            const float *q = partial(c);
            const float2 ml = __ldcg(reinterpret_cast<const float2 *>(q + kProRows * DIM + 2 * mine));
            const float e = ml.x == -INFINITY ? 0.0f : ex2(ml.x - top);
            sum = fmaf(ml.y, e, sum);
#pragma unroll
            for (int i = 0; i < B; ++i) {
                const float ei = __shfl_sync(0xFFFFFFFFu, e, i);
                const float *row = q + (128 * half + b + i) * DIM + V * lane;
                if constexpr (V == 4) {
                    const float4 v = __ldcg(reinterpret_cast<const float4 *>(row));
                    acc[i][0] = fmaf(v.x, ei, acc[i][0]);
                    acc[i][1] = fmaf(v.y, ei, acc[i][1]);
                    acc[i][2] = fmaf(v.z, ei, acc[i][2]);
                    acc[i][3] = fmaf(v.w, ei, acc[i][3]);
                } else {
                    const float2 v = __ldcg(reinterpret_cast<const float2 *>(row));
                    acc[i][0] = fmaf(v.x, ei, acc[i][0]);
                    acc[i][1] = fmaf(v.y, ei, acc[i][1]);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < B; ++i) {
            const float l = __shfl_sync(0xFFFFFFFFu, sum, i);
            if (b + i >= rows) continue;
            const int row = s.j * kProRows + 128 * half + b + i;
#pragma unroll
            for (int k = 0; k < V; ++k) acc[i][k] = l > 0.0f ? acc[i][k] / l : 0.0f;
            attn_store<V>(p, s.req.row0 + row / group, s.g * group + row % group, DIM, V * lane, acc[i]);
        }
        if (lane < B && b + lane < rows && p.lse != nullptr) {
            const int row = s.j * kProRows + 128 * half + b + lane;
            attn_store_lse(p, s.req.row0 + row / group, s.g * group + row % group, top, sum);
        }
    }
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
    const uint32_t v16full = take_bars(2), v16free = take_bars(2);
    const uint32_t sfull = take_bars(2), wfull = take_bars(2), odone = take_bars(2);
    const uint32_t qfull = take_bars(2), qfree = take_bars(1), done_bar = take_bars(1);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(pro_smem + Sm::kMiscOff);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < Sm::kKStages; ++s) {
            mbar_init(kfull + 8 * s, 1);
            mbar_init(kempty + 8 * s, 1);
        }
        for (int s = 0; s < kProScaleSlots; ++s) mbar_init(scfull + 8 * s, 32);
        for (int s = 0; s < 2; ++s) {
            mbar_init(vfull + 8 * s, 1);
            mbar_init(vempty + 8 * s, 128);
            mbar_init(v16full + 8 * s, 128);
            mbar_init(v16free + 8 * s, 1);
            mbar_init(sfull + 8 * s, 1);
            mbar_init(wfull + 8 * s, 128);
            mbar_init(odone + 8 * s, 1);
            mbar_init(qfull + 8 * s, 128);
        }
        mbar_init(qfree, 1);
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
    const long long w0 = idle ? 0 : total * cta / ctas, w1 = idle ? 0 : total * (cta + 1) / ctas;
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
    ProWalk walk{w0, w1 - w0, idle ? 0 : start_r, idle ? 0 : start_g, idle ? 0 : start_j, idle ? 0 : start_offset};
    const int group = p.q_heads / p.kv_heads;
    auto rows_of = [&](const ProSegment &s) {
        const int64_t left = static_cast<int64_t>(s.req.n) * group - static_cast<int64_t>(s.j) * kProRows;
        return static_cast<int>(left < kProRows ? left : kProRows);
    };
    ProSegment s;

    if (warp == 12) {
        // ---------------------------------------------------------- copies
        const int P = 1 << p.page_shift, per_tile = kProKeys >> p.page_shift;
        const int i = lane & 7;
        int kst = 0, vst = 0, count = 0;
        uint32_t kph = 0, vph = 0, kissued = 0, kpar = 0, vissued = 0, vpar = 0;
        bool ok = true;
        while (ok && walk.next(p, s)) {
            const int32_t *table = p.block_table + static_cast<int64_t>(s.r) * p.table_width;
            auto wanted = [&](int tile) {
                const int64_t b = static_cast<int64_t>(tile) * per_tile + i;
                return lane < 16 && i < per_tile && (b << p.page_shift) <= s.keys.last &&
                       ((b + 1) << p.page_shift) > s.keys.first;
            };
            int page = wanted(s.tile) ? table[s.tile * per_tile + i] : 0;
            for (int tile = s.tile; tile < s.end; ++tile, ++count) {
                const bool mine = wanted(tile);
                const int64_t ph = static_cast<int64_t>(min(max(page, 0), p.num_pages - 1)) * p.kv_heads + s.g;
                if (tile + 1 < s.end) page = wanted(tile + 1) ? table[(tile + 1) * per_tile + i] : 0;
                uint32_t bytes = 0;
                if (mine) {
                    const int in_page = min(s.keys.last + 1 - ((tile * per_tile + i) << p.page_shift), P);
                    bytes = static_cast<uint32_t>((in_page + 7) / 8 * 8 * DIM);
                }
                uint32_t sum = lane < 8 ? bytes : 0u;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
                // keys, and the scales of keys and values
                ok = __all_sync(0xFFFFFFFFu,
                                mbar_wait(kempty + 8 * kst, kph ^ 1u, abort_flag, p.status, p.wait_cycles));
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
                                mbar_wait(vempty + 8 * vst, vph ^ 1u, abort_flag, p.status, p.wait_cycles));
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
            if (kissued & (1u << x)) mbar_wait_drain(kfull + 8 * x, (kpar >> x) & 1u, p.status);
        for (int x = 0; x < Sm::kVStages; ++x)
            if (vissued & (1u << x)) mbar_wait_drain(vfull + 8 * x, (vpar >> x) & 1u, p.status);
    } else if (warp == 13) {
        // ---------------------------------------------------------- MMAs
        if (lane == 0) {
            const uint32_t idesc_s = (1u << 4) | (static_cast<uint32_t>(kProKeys >> 3) << 17) | (8u << 24);
            const uint32_t idesc_o = (1u << 4) | (1u << 16) | (static_cast<uint32_t>(DIM >> 3) << 17) | (8u << 24);
            auto wait = [&](uint32_t bar, uint32_t parity) {
                return mbar_wait_fast(bar, parity & 1u, abort_flag, p.status, p.wait_cycles);
            };
            bool ok = true;
            if (p.stall & kStallMma) ok = wait(done_bar, 0);
            int kst = 0, count = 0, segment = 0;
            uint32_t kph = 0;
            int uses[2] = {0, 0};  // score tiles of each half so far
            auto scores = [&](int half) {
                const uint32_t k = sbase + Sm::kKOff + kst * Sm::kTileBytes;
#pragma unroll
                for (int part = 0; part < Sm::kParts; ++part) {
                    const uint32_t q = sbase + (half * Sm::kParts + part) * Sm::kQPart;
#pragma unroll
                    for (int x = 0; x < DIM / 32; ++x)
                        dec_mma(tmem + 128u * half, core_desc(q + 256u * x, 128, 8 * DIM),
                                core_desc(k + 256u * x, 128, 8 * DIM), idesc_s, (part | x) != 0 ? 1u : 0u);
                }
                mma_commit(sfull + 8 * half);
            };
            // O += W V of tile number `tile` (its V buffer), use u of the half
            auto values = [&](int half, int tile, int u, bool first) {
                if (!wait(wfull + 8 * half, u) || !wait(v16full + 8 * (tile & 1), tile >> 1)) return false;
                tc_fence_after();
                const uint32_t v = sbase + Sm::kV16Off + (tile & 1) * Sm::kV16Bytes;
#pragma unroll
                for (int x = 0; x < kProKeys / 16; ++x)
                    pro_mma_f16(tmem + 256u + 128u * half, tmem + 128u * half + 8u * x,
                                core_desc(v + 32u * DIM * x, 16 * DIM, 128), idesc_o, (first && x == 0) ? 0u : 1u);
                mma_commit(odone + 8 * half);
                return true;
            };
            while (ok && walk.next(p, s)) {
                const bool two = rows_of(s) > 128;
                bool pending = false;  // half 1 of the tile before
                ok = wait(qfull + 8 * (segment & 1), segment >> 1);
                for (int tile = s.tile; ok && tile < s.end; ++tile, ++count) {
                    ok = wait(kfull + 8 * kst, kph);
                    if (!ok) break;
                    tc_fence_after();
                    scores(0);
                    if (pending) {
                        ok = values(1, count - 1, uses[1] - 1, tile - 1 == s.tile);
                        if (!ok) break;
                        mma_commit(v16free + 8 * ((count - 1) & 1));
                    }
                    if (two) {
                        scores(1);
                        ++uses[1];
                    }
                    mma_commit(kempty + 8 * kst);
                    if (tile + 1 == s.end) mma_commit(qfree);
                    ok = values(0, count, uses[0], tile == s.tile);
                    if (!ok) break;
                    ++uses[0];
                    if (!two) mma_commit(v16free + 8 * (count & 1));
                    pending = two;
                    if (++kst == Sm::kKStages) {
                        kst = 0;
                        kph ^= 1u;
                    }
                }
                if (ok && pending) {
                    ok = values(1, count - 1, uses[1] - 1, s.end - 1 == s.tile);
                    if (ok) mma_commit(v16free + 8 * ((count - 1) & 1));
                }
                ++segment;
            }
            mma_commit(done_bar);
        }
        __syncwarp();
    } else if (warp >= 8) {
        // ------------------------------------- queries to parts, V to fp16
        const int tid = static_cast<int>(threadIdx.x) - 256;
        float *qf = reinterpret_cast<float *>(pro_smem + Sm::kQfOff);
        int vst = 0, count = 0, segment = 0;
        uint32_t vph = 0;
        bool ok = true;
        while (walk.next(p, s)) {
            const int rows = rows_of(s);
            ok = ok && (segment == 0 ||
                        mbar_wait(qfree, (segment - 1) & 1u, abort_flag, p.status, p.wait_cycles));
            constexpr int LANES = DIM / 8, AT_ONCE = 128 / LANES, BATCH = 8;
            const int l = tid % LANES;
            for (int b = 0; b < rows; b += AT_ONCE * BATCH) {
                uint4 u[BATCH];
#pragma unroll
                for (int k = 0; k < BATCH; ++k) {
                    const int row = b + k * AT_ONCE + tid / LANES;
                    u[k] = make_uint4(0u, 0u, 0u, 0u);
                    if (row < rows) {
                        const int64_t at = static_cast<int64_t>(s.j) * kProRows + row;
                        const int token = s.req.row0 + static_cast<int>(at / group);
                        const int head = s.g * group + static_cast<int>(at % group);
                        u[k] = *reinterpret_cast<const uint4 *>(p.q + static_cast<int64_t>(token) * p.q_stride +
                                                                head * DIM + 8 * l);
                    }
                }
#pragma unroll
                for (int k = 0; k < BATCH; ++k) {
                    const int row = b + k * AT_ONCE + tid / LANES;  // rows past the last are zeros, below 256
                    float x[8];
                    const uint32_t w[4] = {u[k].x, u[k].y, u[k].z, u[k].w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint64_t f = widen16<QDT>(w[i]);
                        x[2 * i] = __uint_as_float(static_cast<uint32_t>(f));
                        x[2 * i + 1] = __uint_as_float(static_cast<uint32_t>(f >> 32));
                    }
                    float m = 0.0f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(x[i]));
#pragma unroll
                    for (int o = LANES / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o, LANES));
                    const int e = m > 0.0f ? min(7 - ilogbf(m), 120) : 0;
                    const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[i] *= up;
                    if (l == 0)
                        qf[(segment & 1) * kProRows + row] =
                            p.score_scale * __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
                    for (int part = 0; part < Sm::kParts; ++part) {
                        uint32_t c[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) c[i] = take_part_unscaled(x[2 * i], x[2 * i + 1]);
                        uint8_t *dst = pro_smem + ((row >> 7) * Sm::kParts + part) * Sm::kQPart +
                                       ((row & 127) >> 3) * 8 * DIM + (l >> 1) * 128 + (row & 7) * 16 + 8 * (l & 1);
                        *reinterpret_cast<uint2 *>(dst) = make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
                    }
                }
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            mbar_arrive(qfull + 8 * (segment & 1));
            ++segment;
            for (int tile = s.tile; tile < s.end; ++tile, ++count) {
                constexpr int PIECES = kProKeys * DIM / 16 / 128;  // 16-byte pieces per thread
                ok = ok && mbar_wait_fast(vfull + 8 * vst, vph, abort_flag, p.status, p.wait_cycles);
                const uint8_t *src = pro_smem + Sm::kVOff + vst * Sm::kTileBytes;
                uint4 u[PIECES];
#pragma unroll
                for (int k = 0; k < PIECES; ++k) {
                    const int piece = tid + 128 * k;
                    const int key = tile * kProKeys + piece / (DIM / 2) * 8 + (piece & 7);
                    u[k] = *reinterpret_cast<const uint4 *>(src + 16 * piece);
                    // keys that are not there: whatever the stage holds (NaN
                    // codes too) must not meet their zero weights
                    if (key < s.keys.first || key > s.keys.last) u[k] = make_uint4(0u, 0u, 0u, 0u);
                }
                mbar_arrive(vempty + 8 * vst);
                if (++vst == Sm::kVStages) {
                    vst = 0;
                    vph ^= 1u;
                }
                const int b = count & 1;
                ok = ok && mbar_wait_fast(v16free + 8 * b, ((count >> 1) & 1u) ^ 1u, abort_flag, p.status,
                                          p.wait_cycles);
                uint8_t *dst = pro_smem + Sm::kV16Off + b * Sm::kV16Bytes;
#pragma unroll
                for (int k = 0; k < PIECES; ++k) {
                    const int piece = tid + 128 * k;
                    const uint32_t w[4] = {u[k].x, u[k].y, u[k].z, u[k].w};
                    uint32_t h[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint32_t two = (i & 1) ? w[i >> 1] >> 16 : w[i >> 1] & 0xFFFFu;
                        asm("{\n\t.reg .b16 c;\n\tcvt.u16.u32 c, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, c;\n\t}"
                            : "=r"(h[i])
                            : "r"(two));
                    }
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
        // ---------------------------------------------------------- softmax
        const int half = warp >> 2, tid = static_cast<int>(threadIdx.x) & 127;
        const uint32_t lane_addr = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t s_tmem = tmem + lane_addr + 128u * half, o_tmem = tmem + lane_addr + 256u + 128u * half;
        const float *qf = reinterpret_cast<const float *>(pro_smem + Sm::kQfOff);
        const float *scales = reinterpret_cast<const float *>(pro_smem + Sm::kScaleOff);
        int count = 0, segment = 0, uses = 0;
        bool ok = true;
        while (walk.next(p, s)) {
            const int rows = rows_of(s) - 128 * half;  // valid rows of this half
            if (rows <= 0) {
                count += s.end - s.tile;
                ++segment;
                continue;
            }
            const bool warp_on = (tid & ~31) < rows;
            const int64_t row = static_cast<int64_t>(s.j) * kProRows + 128 * half + tid;
            const int before = s.req.keys - s.req.n;
            const int pos = before + static_cast<int>(row / group);
            // positions of the warp's first and last valid row
            const int64_t row_lo = row - lane;
            const int64_t row_hi = min(row_lo + 31, static_cast<int64_t>(s.j) * kProRows + 128 * half + rows - 1);
            const int pos_lo = before + static_cast<int>(row_lo / group), pos_hi = before + static_cast<int>(row_hi / group);
            ok = ok && mbar_wait_fast(qfull + 8 * (segment & 1), (segment >> 1) & 1u, abort_flag, p.status,
                                      p.wait_cycles);
            const float f = qf[(segment & 1) * kProRows + 128 * half + tid];
            ++segment;
            float m = -INFINITY, l = 0.0f;
            for (int tile = s.tile; tile < s.end; ++tile, ++count, ++uses) {
                // (a barrier per slot, not the key stage's, which may be
                // filled again while this half is still in an epilogue)
                ok = ok && mbar_wait_fast(scfull + 8 * (count & (kProScaleSlots - 1)), (count / kProScaleSlots) & 1u,
                                          abort_flag, p.status, p.wait_cycles);
                ok = ok && mbar_wait_fast(sfull + 8 * half, uses & 1u, abort_flag, p.status, p.wait_cycles);
                tc_fence_after();
                if (warp_on) {
                    const float *sc = scales + (count & (kProScaleSlots - 1)) * 16;
                    const int key0 = tile * kProKeys;
                    const bool plain = key0 + kProKeys - 1 <= pos_lo && (p.window == 0 || key0 > pos_hi - p.window);
                    // columns [lo, hi) of this row are seen
                    const int lo = p.window > 0 ? pos - p.window + 1 - key0 : 0, hi = pos + 1 - key0;
                    // factors of the 16 columns from 16 x on: the page's
                    // scales; a page without a seen key was not copied
                    auto factors = [&](int x, float &c, float &lv, float &rv) {
                        const int pg = (16 * x) >> p.page_shift;
                        const bool there = key0 + 16 * x <= s.keys.last && key0 + 16 * x + 15 >= s.keys.first;
                        c = there ? f * sc[pg] : 0.0f;
                        const float vs = there ? sc[8 + pg] : 1.0f;
                        lv = __log2f(vs);
                        rv = __frcp_rn(vs);
                    };
                    float top = -INFINITY;
#pragma unroll
                    for (int x = 0; x < kProKeys / 32; ++x) {
                        uint32_t v[32];
                        tmem_ld32_nowait(s_tmem + 32 * x, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            float c, lv, rv;
                            factors(2 * x + y, c, lv, rv);
                            float raw = -INFINITY;
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                const int col = 32 * x + 16 * y + i;
                                const float sv = __uint_as_float(v[16 * y + i]);
                                raw = fmaxf(raw, plain || (col >= lo && col < hi) ? sv : -INFINITY);
                            }
                            if (raw > -INFINITY) top = fmaxf(top, fmaf(raw, c, lv));
                        }
                    }
                    const bool move = top > m + kProMove;
                    if (__any_sync(0xFFFFFFFFu, move)) {
                        const float to = move ? top - kProHead : m;
                        const float keep = to == -INFINITY ? 1.0f : (m == -INFINITY ? 0.0f : ex2(m - to));
                        l *= keep;
                        m = to;
                        if (tile != s.tile) {
                            ok = ok && mbar_wait_fast(odone + 8 * half, (uses - 1) & 1u, abort_flag, p.status,
                                                      p.wait_cycles);
                            tc_fence_after();
#pragma unroll
                            for (int x = 0; x < DIM / 32; ++x) {
                                uint32_t v[32];
                                tmem_ld32_nowait(o_tmem + 32 * x, v);
                                tmem_wait_ld();
#pragma unroll
                                for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * keep);
                                tmem_st32_nowait(o_tmem + 32 * x, v);
                            }
                        }
                    }
                    const float mu = m == -INFINITY ? 0.0f : m;
#pragma unroll
                    for (int x = 0; x < kProKeys / 32; ++x) {
                        uint32_t v[32], w[16];
                        tmem_ld32_nowait(s_tmem + 32 * x, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            float c, lv, rv;
                            factors(2 * x + y, c, lv, rv);
                            const float b = lv - mu;
                            float sum = 0.0f;
#pragma unroll
                            for (int i = 0; i < 16; i += 2) {
                                float a[2];
#pragma unroll
                                for (int k = 0; k < 2; ++k) {
                                    const int col = 32 * x + 16 * y + i + k;
                                    const float t = fmaf(__uint_as_float(v[16 * y + i + k]), c, b);
                                    a[k] = plain || (col >= lo && col < hi) ? ex2(t) : 0.0f;
                                    sum += a[k];
                                }
                                const __half2 h = __floats2half2_rn(a[0], a[1]);
                                w[8 * y + i / 2] = *reinterpret_cast<const uint32_t *>(&h);
                            }
                            l = fmaf(sum, rv, l);
                        }
                        tmem_st_n(s_tmem + 16 * x, w);  // below the columns still to be read
                    }
                    tmem_wait_st();
                }
                tc_fence_before();
                mbar_arrive(wfull + 8 * half);
            }

            // ------------------------------------------------------ epilogue
            ok = ok && mbar_wait_fast(odone + 8 * half, (uses - 1) & 1u, abort_flag, p.status, p.wait_cycles);
            tc_fence_after();
            const bool whole = s.tile == s.keys.begin && s.end == s.keys.begin + s.keys.tiles;
            const bool valid = tid < rows;
            const int token = s.req.row0 + static_cast<int>(row / group), head = s.g * group + static_cast<int>(row % group);
            if (whole) {
                if (warp_on) {
                    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
#pragma unroll
                    for (int x = 0; x < DIM / 32; ++x) {
                        uint32_t v[32];
                        tmem_ld32_nowait(o_tmem + 32 * x, v);
                        tmem_wait_ld();
                        if (valid) {
#pragma unroll
                            for (int y = 0; y < 4; ++y) {
                                float o[8];
#pragma unroll
                                for (int i = 0; i < 8; ++i)
                                    o[i] = l > 0.0f ? __uint_as_float(v[8 * y + i]) * inv : 0.0f;
                                attn_store<8>(p, token, head, DIM, 32 * x + 8 * y, o);
                            }
                        }
                    }
                    if (valid && p.lse != nullptr) attn_store_lse(p, token, head, m, l);
                }
                tc_fence_before();
            } else {
                const long long seg0 = s.at - (s.tile - s.keys.begin), seg1 = seg0 + s.keys.tiles;
                const long long c0 = ((seg0 + 1) * ctas - 1) / total, c1 = (seg1 * ctas - 1) / total;
                constexpr long long kPart = kProRows * (DIM + 2);
                float *part = p.partials + (cta * 2 + (s.tile != s.keys.begin || seg0 == w0 ? 0 : 1)) * kPart;
                if (warp_on) {
#pragma unroll
                    for (int x = 0; x < DIM / 32; ++x) {
                        uint32_t v[32];
                        tmem_ld32_nowait(o_tmem + 32 * x, v);
                        tmem_wait_ld();
                        float *at = part + (128 * half + tid) * DIM + 32 * x;
#pragma unroll
                        for (int i = 0; i < 32; i += 4)
                            *reinterpret_cast<uint4 *>(at + i) = make_uint4(v[i], v[i + 1], v[i + 2], v[i + 3]);
                    }
                    *reinterpret_cast<float2 *>(part + kProRows * DIM + 2 * (128 * half + tid)) = make_float2(m, l);
                }
                tc_fence_before();
                __threadfence();
                half_sync(half);
                if (tid == 0) {
                    const unsigned parts = static_cast<unsigned>(c1 - c0 + 1);
                    merge_now[half] = atomicInc(p.counters + 2 * c0 + half, parts - 1) == parts - 1;  // wraps to 0
                    __threadfence();
                }
                half_sync(half);
                if (merge_now[half]) {
                    pro_merge<DIM>(p, s, half, rows, group, static_cast<int>(c1 - c0 + 1), [&](int c) {
                        const int slot = c == 0 && seg0 != total * c0 / ctas ? 1 : 0;
                        return p.partials + ((c0 + c) * 2 + slot) * kPart;
                    });
                }
                half_sync(half);  // merge_now has been read
            }
        }
    }

    mbar_wait_drain(done_bar, 0, p.status);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 13)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
}

}  // namespace
}  // namespace fp8l
