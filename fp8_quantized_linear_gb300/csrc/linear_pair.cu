// Linear layer on the tcgen05 tensor cores for many tokens: 256 x 256 tiles
// over pairs of SMs (sm_103a).
//
// ("[Kernel][FP8] Initial support with dynamic per-tensor scaling": the W8A8
// product of a prefill batch; "RFC: FP8 Quantization Schema in vLLM": an E4M3
// result through output_scale.)
//
//   z[m, n] = sum_k dec(a[m,k]) dec(w[n,k]) * a_scale(m) w_scale(n) + bias(n)
//   y = the epilogue of epilogue.cuh
//
// A cluster of two CTAs computes a tile of 256 tokens by 256 weight rows with
// tcgen05.mma.cta_group::2 (M = 256, N = 256, K = 32): each CTA stages 128
// rows of a and half of the tile's weight rows per 128-deep k-block (32 KB a
// stage, five stages), the MMA reads the peer's halves from its shared memory,
// and each CTA's TMEM receives its 128 tokens of the accumulator (512
// columns: two accumulators, so the epilogue of one tile runs under the MMAs
// of the next).  With a gate the even CTA stages 128 gate rows and the odd
// one the up rows of the same outputs: the accumulator's left half is the
// gate, its right half the up product, and both sit in the same lane, so the
// epilogue needs no exchange and writes half the columns.
//   warp 0     TMA producer in each CTA; both CTAs' copies complete on the
//              even CTA's full barrier.  With stable weights the first
//              stages' weights are loaded before the wait for the preceding
//              kernel.
//   warp 1     TMEM; in the even CTA one lane issues the MMAs, whose commits
//              arrive on the barriers of both CTAs.
//   warps 2-17 epilogue in each CTA, four warps a TMEM lane quarter (each a
//              quarter of the tile's 32-column chunks; with two, a tile with
//              SiLU and E4M3 output took 0.8 us longer, which a product of one
//              or two rounds shows in full).  One lane waits for the
//              accumulator.  A tile's scales and biases are spread over the
//              threads once and read back from shared memory (any type, any
//              alignment, one load a column).  16-bit results and residuals
//              cross global memory as TMA boxes of 32 rows by 32 columns
//              through a warp's own buffer: a lane has a row, and plain 16-byte
//              accesses of 32 different lines each took the load/store unit
//              from the MMA's operand reads (4096 x 8192 x 28672 with a
//              residual 1007k cycles, with boxes 949k, the plain product's).
// Tail tiles: 256-wide tiles fill whole rounds of the SM pairs; the columns
// left over become narrower tiles when that ends the last round sooner.
// Few tiles: a cluster of two or four pairs shares a tile and splits its
// k-blocks.  Each pair keeps a share of the tile's columns and sends the float
// sums of the others to their pairs' (by then idle) stages through distributed
// shared memory; the owner adds them in pair order, so results are the same
// bits every time (512 x 4096 x 14336: 41.0 us without, 29 with).
// The producer's loop does nothing but wait, arm and load: with its addresses
// computed in the loop the same product took 985k cycles instead of 965k.
// Measured (GB300, replayed graphs): gate/up of 1021 tokens, 28672 x 4096, SiLU
// and E4M3 output, 78.4 to 79.2 us (0.79 of twice the bf16 burst peak; tensor
// pipe 68 % active), down of 4096 tokens, 8192 x 28672 with bias and residual,
// 560 to 568 us cool (0.89; 84 %), 620 to 660 under the power cap; 4096 x 28672
// x 4096 with a residual 303 us (297 for fp8_scaled_mm without one).
// Waits are bounded; a time-out raises both CTAs' abort flags, and all CTAs of
// a cluster meet at its barrier before TMEM is released.
#include <atomic>

#include "linear_launch.cuh"
#include "skinny_device.cuh"
#include "tc_device.cuh"

namespace fp8l {
namespace {

constexpr int LP_BM = 128;  // tokens a CTA; a pair covers 256
constexpr int LP_BN = 256;  // weight rows a tile; each CTA stages half
constexpr int LP_BK = 128;
constexpr int LP_STAGES = 5;  // (six: the same, and no room for the boxes)
constexpr int kLpABytes = LP_BM * LP_BK;
constexpr int kLpBBytes = (LP_BN / 2) * LP_BK;
constexpr int kLpStageBytes = kLpABytes + kLpBBytes;
constexpr int kLpEpiWarps = 16;
constexpr int kLpEpiGroups = kLpEpiWarps / 4;  // warps of a TMEM lane quarter
constexpr int kLpEpiThreads = 32 * kLpEpiWarps;
constexpr int kLpThreads = 64 + kLpEpiThreads;
constexpr int kLpBarriers = 2 * LP_STAGES + 2 + 2 + 1;
constexpr int kLpBoxBytes = 32 * 64;             // 32 rows of 32 16-bit values
constexpr int kLpBoxes = kLpEpiWarps;
constexpr int kLpColBytes = 2 * 2 * LP_BN * 4;  // two tiles' scales and biases
constexpr int kLpBoxOffset = LP_STAGES * kLpStageBytes;  // from the 1024-aligned base
constexpr int kLpColOffset = kLpBoxOffset + kLpBoxes * kLpBoxBytes;
constexpr int kLpBarOffset = kLpColOffset + kLpColBytes;
constexpr size_t kLpSmemBytes = 1024 + kLpBarOffset + (kLpBarriers + kLpBoxes) * 8 + 16;
constexpr uint32_t kLpTmemCols = 2 * LP_BN;

struct PairArgs {
    int M, num_k_blocks;
    int split;  // pairs of a cluster sharing a tile (1: none)
    int tiles_m, main_tiles, n_main, tail_w, tail_n;  // n_main: output columns of the main tiles
    int prefetch;
    const float *a_scale;
    int a_per_token;
    const float *w_scale;
    int w_per_channel;
    Epilogue e;
    unsigned *status;
    long long wait_cycles;
    unsigned stall;
};

// kind::f8f6f4, D f32, A and B E4M3 K-major, N = w, M = 256 (pair)
__host__ __device__ constexpr uint32_t lp_idesc(int w) {
    return (1u << 4) | (static_cast<uint32_t>(w >> 3) << 17) | (static_cast<uint32_t>(256 >> 4) << 24);
}

// TMA load into this CTA's shared memory, completing on an mbarrier of
// either CTA of the pair
__device__ __forceinline__ void lp_tma(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void lp_mma(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                       uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// arrive on the barrier at this offset in both CTAs (a mask of cluster ranks)
// once the MMAs issued so far have retired
__device__ __forceinline__ void lp_commit(uint32_t bar, uint32_t ctas) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
        " [%0], %1;" ::"r"(bar),
        "h"(static_cast<uint16_t>(ctas))
        : "memory");
}

struct LpTile {
    int mt, n0, w;  // 256-token block, first output column, accumulator columns
};

template <bool GATED>
__device__ __forceinline__ LpTile lp_tile(const PairArgs &p, int tile) {
    LpTile t;
    if (tile < p.main_tiles) {
        t.mt = tile % p.tiles_m;
        t.n0 = (tile / p.tiles_m) * (GATED ? LP_BN / 2 : LP_BN);
        t.w = LP_BN;
    } else {
        const int u = tile - p.main_tiles;
        t.mt = u % p.tiles_m;
        t.w = p.tail_w;
        t.n0 = p.n_main + (u / p.tiles_m) * (GATED ? t.w / 2 : t.w);
    }
    return t;
}

// a box between shared memory and a [rows, bytes] matrix (x in bytes)
__device__ __forceinline__ void lp_load_box(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar) {
    mbar_expect_tx(bar, kLpBoxBytes);
    tma_load_2d(dst, map, x, y, bar);
}

__device__ __forceinline__ void lp_store_box(const CUtensorMap *map, int x, int y, uint32_t src) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y), "r"(src)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

__device__ __forceinline__ void lp_tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// until at most N of this thread's stores have still to read shared memory
template <int N>
__device__ __forceinline__ void lp_stores_read() {
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}

// address of 16-byte piece j of lane `row`'s 64 bytes in a box (64-byte
// swizzle: eight rows of a wavefront hit different banks)
__device__ __forceinline__ uint32_t lp_box_piece(uint32_t box, int row, int j) {
    return box + static_cast<uint32_t>(row * 64 + ((j ^ ((row >> 1) & 3)) << 4));
}

__device__ __forceinline__ void lp_st_cluster(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared::cluster.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
                 : "memory");
}

__device__ __forceinline__ uint4 lp_ld_shared(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// z = acc * (sa * scale) + bias of COUNT columns; cols: the tile's scales, then
// its biases LP_BN floats on, in shared memory (all lanes read one address)
template <int COUNT>
__device__ __forceinline__ void lp_scaled(const uint32_t (&r)[COUNT], const float *cols, float sa, bool bias,
                                          float (&v)[COUNT]) {
    const float4 *s4 = reinterpret_cast<const float4 *>(cols);
    const float4 *b4 = reinterpret_cast<const float4 *>(cols + LP_BN);
#pragma unroll
    for (int q = 0; q < COUNT / 4; ++q) {
        const float4 s = s4[q];
        const float4 b = bias ? b4[q] : make_float4(0.f, 0.f, 0.f, 0.f);
        v[4 * q] = fmaf(__uint_as_float(r[4 * q]), sa * s.x, b.x);
        v[4 * q + 1] = fmaf(__uint_as_float(r[4 * q + 1]), sa * s.y, b.y);
        v[4 * q + 2] = fmaf(__uint_as_float(r[4 * q + 2]), sa * s.z, b.z);
        v[4 * q + 3] = fmaf(__uint_as_float(r[4 * q + 3]), sa * s.w, b.w);
    }
}

// The sums of a chunk (32 accumulator columns) that other pairs sent, added to
// this pair's: 16-byte pieces [source][chunk][piece][row] from `part`.
template <int COUNT>
__device__ __forceinline__ void lp_add_parts(uint32_t (&r)[COUNT], uint32_t part, int sources, uint32_t source_bytes) {
    for (int q = 0; q < sources; ++q, part += source_bytes) {
#pragma unroll
        for (int j = 0; j < COUNT / 4; ++j) {
            const uint4 w = lp_ld_shared(part + static_cast<uint32_t>(j * LP_BM * 16));
            r[4 * j] = __float_as_uint(__uint_as_float(r[4 * j]) + __uint_as_float(w.x));
            r[4 * j + 1] = __float_as_uint(__uint_as_float(r[4 * j + 1]) + __uint_as_float(w.y));
            r[4 * j + 2] = __float_as_uint(__uint_as_float(r[4 * j + 2]) + __uint_as_float(w.z));
            r[4 * j + 3] = __float_as_uint(__uint_as_float(r[4 * j + 3]) + __uint_as_float(w.w));
        }
    }
}

template <bool GATED, bool SPLIT>
__global__ void __launch_bounds__(kLpThreads, 1)
linear_pair_kernel(const __grid_constant__ CUtensorMap tmap_a,
                   const __grid_constant__ CUtensorMap tmap_b,
                   const __grid_constant__ CUtensorMap tmap_bt,
                   const __grid_constant__ CUtensorMap tmap_y,
                   const __grid_constant__ CUtensorMap tmap_r, const PairArgs p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t sbase = (raw + 1023u) & ~1023u;
    uint8_t *gbase = smem_raw + (sbase - raw);
    float *cols_sh = reinterpret_cast<float *>(gbase + kLpColOffset);
    const uint32_t bar0 = sbase + kLpBarOffset;
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (LP_STAGES + s); };
    auto tfull_bar = [&](int b) { return bar0 + 8u * (2 * LP_STAGES + b); };
    auto tempty_bar = [&](int b) { return bar0 + 8u * (2 * LP_STAGES + 2 + b); };
    const uint32_t done_bar = bar0 + 8u * (2 * LP_STAGES + 4);
    const uint32_t box_bar0 = done_bar + 8u;  // residual boxes: one an epilogue warp
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(gbase + kLpBarOffset + (kLpBarriers + kLpBoxes) * 8);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t crank = cluster_rank();
    const uint32_t rank = crank & 1u;   // in the pair
    const uint32_t even = crank & ~1u;  // the pair's even CTA
    const uint32_t both = 3u << even;
    const bool leader = rank == 0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < LP_STAGES; ++s) {
            mbar_init(full_bar(s), 1);   // the even CTA's arming arrival (+ both CTAs' bytes)
            mbar_init(empty_bar(s), 1);  // the MMA commit, multicast to both CTAs
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(tfull_bar(b), 1);
            mbar_init(tempty_bar(b), 2 * kLpEpiWarps);  // the pair's epilogue warps
        }
        mbar_init(done_bar, 1);
        for (int b = 0; b < kLpBoxes; ++b) mbar_init(box_bar0 + 8u * b, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(tmem_slot)),
                     "r"(kLpTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();  // both CTAs' barriers exist before either touches the other's
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    const uint32_t peer_abort = map_to_rank(smem_u32(const_cast<int *>(abort_flag)), crank ^ 1u);

    const int num_tiles = p.main_tiles + p.tiles_m * p.tail_n;
    // pairs go round the tiles; or a cluster's one tile, and this pair's share
    // of its k-blocks
    const int pair = SPLIT ? static_cast<int>(blockIdx.x) / (2 * p.split) : static_cast<int>(blockIdx.x) >> 1;
    const int num_pairs = SPLIT ? num_tiles : static_cast<int>(gridDim.x) >> 1;
    const int kpart = SPLIT ? static_cast<int>(crank >> 1) : 0;
    int kb0 = 0, nkb = p.num_k_blocks;
    if constexpr (SPLIT) {
        const int share = p.num_k_blocks / p.split, rem = p.num_k_blocks % p.split;
        kb0 = kpart * share + (kpart < rem ? kpart : rem);
        nkb = share + (kpart < rem ? 1 : 0);
    }

    if (warp == 0) {
        if (lane == 0) {
            asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmap_a)) : "memory");
            asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmap_b)) : "memory");
            if (p.tail_n > 0)
                asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmap_bt)) : "memory");
            uint32_t armed = 0, armed_parity = 0;  // even CTA: stages armed, their parity
            const uint32_t full0 = map_to_rank(full_bar(0), even);  // the even CTA's full barriers
            const int a_row = static_cast<int>(rank) * LP_BM;
            // stable weights: the first tile's first stages before the wait
            int pre = 0;
            if (p.prefetch && pair < num_tiles) {
                const LpTile t = lp_tile<GATED>(p, pair);
                const CUtensorMap *map = t.w != LP_BN ? &tmap_bt : &tmap_b;
                const int w_row = t.n0 + static_cast<int>(rank) * (GATED ? p.e.width : t.w / 2);
                pre = nkb < LP_STAGES ? nkb : LP_STAGES;
                for (int s = 0; s < pre; ++s) {
                    if (leader) {
                        mbar_expect_tx(full_bar(s), 2 * (kLpABytes + static_cast<uint32_t>(t.w / 2) * LP_BK));
                        armed |= 1u << s;
                    }
                    lp_tma(sbase + s * kLpStageBytes + kLpABytes, map, (kb0 + s) * LP_BK, w_row, full0 + 8u * s);
                }
            }
            pdl_wait();
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int tile = pair; ok && tile < num_tiles; tile += num_pairs) {
                const LpTile t = lp_tile<GATED>(p, tile);
                // bytes of a stage in both CTAs: a rows and half of the tile's weight rows
                const uint32_t bytes = 2 * (kLpABytes + static_cast<uint32_t>(t.w / 2) * LP_BK);
                const CUtensorMap *map = t.w != LP_BN ? &tmap_bt : &tmap_b;
                const int x_row = t.mt * 2 * LP_BM + a_row;
                const int w_row = t.n0 + static_cast<int>(rank) * (GATED ? p.e.width : t.w / 2);
                int kb = 0;
                for (; kb < pre; ++kb)  // armed, the weights on their way
                    lp_tma(sbase + kb * kLpStageBytes, &tmap_a, (kb0 + kb) * LP_BK, x_row, full0 + 8u * kb);
                if (kb > 0) {
                    stage = kb == LP_STAGES ? 0 : kb;
                    phase = kb == LP_STAGES ? 1u : 0u;
                    pre = 0;
                }
                for (; kb < nkb; ++kb) {
                    if (!mbar_wait(empty_bar(stage), phase ^ 1u, abort_flag, p.status, p.wait_cycles,
                                   peer_abort)) {
                        ok = false;
                        break;
                    }
                    const uint32_t sa = sbase + stage * kLpStageBytes;
                    const uint32_t fb = full0 + 8u * stage;
                    if (leader) {
                        mbar_expect_tx(full_bar(stage), bytes);
                        armed |= 1u << stage;
                        armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
                    }
                    lp_tma(sa, &tmap_a, (kb0 + kb) * LP_BK, x_row, fb);
                    lp_tma(sa + kLpABytes, map, (kb0 + kb) * LP_BK, w_row, fb);
                    if (++stage == LP_STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            // every armed stage lands before either CTA passes the final
            // cluster barrier
            for (int s = 0; s < LP_STAGES; ++s)
                if (armed & (1u << s)) mbar_wait_drain(full_bar(s), (armed_parity >> s) & 1u, p.status);
        }
        __syncwarp();
        if constexpr (SPLIT) {
            cluster_sync_all();  // every pair's MMAs are through: stages may be written
            cluster_sync_all();  // the sums are with their owners
        }
    } else if (warp == 1) {
        if (lane == 0 && leader) {
            pdl_wait();  // (the waits below are limited, the preceding kernel's time is not)
            int stage = 0;
            uint32_t phase = 0;
            int acc = 0;
            uint32_t acc_phase = 0;
            bool ok = true;
            if (p.stall & kStallMma)
                ok = mbar_wait(done_bar, 0, abort_flag, p.status, p.wait_cycles, peer_abort);
            for (int tile = pair; ok && tile < num_tiles; tile += num_pairs) {
                if (!mbar_wait(tempty_bar(acc), acc_phase ^ 1u, abort_flag, p.status, p.wait_cycles,
                               peer_abort))
                    break;
                tc_fence_after();
                const uint32_t idesc = lp_idesc(tile < p.main_tiles ? LP_BN : p.tail_w);
                const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * LP_BN);
                for (int kb = 0; kb < nkb; ++kb) {
                    if (!mbar_wait_fast(full_bar(stage), phase, abort_flag, p.status, p.wait_cycles,
                                        peer_abort)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t sa = sbase + stage * kLpStageBytes;
                    const uint64_t da = sw128_desc(sa), db = sw128_desc(sa + kLpABytes);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        lp_mma(d_tmem, da + 2 * k, db + 2 * k, idesc, (kb | k) != 0 ? 1u : 0u);
                    lp_commit(empty_bar(stage), both);
                    if (++stage == LP_STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (!ok) break;
                lp_commit(tfull_bar(acc), both);
                acc ^= 1;
                if (acc == 0) acc_phase ^= 1u;
            }
            // every MMA issued has retired
            lp_commit(done_bar, both);
            mbar_wait_drain(done_bar, 0, p.status);
        }
        __syncwarp();
        if constexpr (SPLIT) {
            cluster_sync_all();
            cluster_sync_all();
        }
    } else {
        pdl_wait();
        const int quarter = warp & 3;     // the TMEM lanes this warp may read
        const int grp = (warp - 2) >> 2;  // its quarter of each tile's chunks
        const int et = static_cast<int>(threadIdx.x) - 64;
        const int row = static_cast<int>(rank) * LP_BM + quarter * 32 + lane;
        const float sa0 = epi_ld_f32(p.a_scale);
        const OutScale os = OutScale::make(p.e.out_dtype == FP8L_E4M3 ? epi_ld_f32(p.e.out_scale) : 1.0f);
        const bool bias = p.e.bias != nullptr;
        const uint32_t box = sbase + kLpBoxOffset + static_cast<uint32_t>((warp - 2) * kLpBoxBytes);
        const uint32_t box_bar = box_bar0 + 8u * (warp - 2);
        uint32_t box_phase = 0;  // parity of the box's barrier
        bool loading = false;    // a residual on its way into the box
        int acc = 0;
        uint32_t acc_phase = 0;
        bool ok = true;
        for (int tile = pair; tile < num_tiles; tile += num_pairs) {
            const LpTile t = lp_tile<GATED>(p, tile);
            const int half = t.w / 2;
            const int m = t.mt * 2 * LP_BM + row;
            const bool row_ok = m < p.M;
            // column et's scale and bias (accumulator order) for every thread;
            // the buffer was last read two tiles ago, before the barrier of
            // the tile in between
            float *cols = cols_sh + acc * 2 * LP_BN;
            {
                int n = t.n0 + et;  // weight row of accumulator column et
                bool in = et < t.w && n < p.e.width;
                if constexpr (GATED) {
                    if (et >= half) n = p.e.width + t.n0 + et - half;
                    in = et < t.w && t.n0 + (et >= half ? et - half : et) < p.e.width;
                }
                if (et < LP_BN) {
                    cols[et] = in ? epi_ld_f32(p.w_scale + (p.w_per_channel ? n : 0)) : 0.0f;
                    if (bias) cols[LP_BN + et] = in ? epi_bias(p.e, n) : 0.0f;
                }
            }
            const float sa = p.a_per_token ? (row_ok ? epi_ld_f32(p.a_scale + m) : 0.0f) : sa0;
            const int chunks = GATED ? half / 32 : t.w / 32;
            // this pair's share of the chunks, this warp's quarter of it
            const int own0 = SPLIT ? chunks * kpart / p.split : 0;
            const int own = SPLIT ? chunks * (kpart + 1) / p.split - own0 : chunks;
            const int c_begin = own0 + grp * own / kLpEpiGroups, c_end = own0 + (grp + 1) * own / kLpEpiGroups;
            // (a box partly outside the matrix is cut by TMA; one wholly outside is left out)
            const int box_row = t.mt * 2 * LP_BM + static_cast<int>(rank) * LP_BM + quarter * 32;
            auto box_in = [&](int c) { return box_row < p.M && t.n0 + c * 32 < p.e.width; };
            auto load_res = [&](int c) {
                if (p.e.residual == nullptr || !box_in(c)) return;
                if (lane == 0) {
                    lp_stores_read<0>();  // the last store is through with the box
                    lp_load_box(box, &tmap_r, 2 * (t.n0 + c * 32), box_row, box_bar);
                }
                loading = true;
            };
            if (ok && c_begin < c_end) load_res(c_begin);
            // one lane waits for the accumulator, the others for it at the
            // barrier (polling warps take issue slots from the two that feed
            // the MMAs)
            if (et == 0 && ok) {
                mbar_wait(tfull_bar(acc), acc_phase, abort_flag, p.status, p.wait_cycles, peer_abort);
                tc_fence_before();
            }
            __syncwarp();
            asm volatile("bar.sync 1, %0;" ::"n"(kLpEpiThreads) : "memory");
            ok = __all_sync(0xFFFFFFFFu, ok && !*abort_flag);
            const uint32_t taddr = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) +
                                   static_cast<uint32_t>(acc * LP_BN);
            // split: bytes of the sums one pair sends another, of a chunk's, and
            // where this row's pieces of the ones received begin
            const uint32_t chunk_bytes = 32 * 4 * LP_BM;
            const uint32_t part_bytes = SPLIT ? chunk_bytes * static_cast<uint32_t>((GATED ? 2 : 1) * own) : 0u;
            const uint32_t part0 = sbase + static_cast<uint32_t>((quarter * 32 + lane) * 16);
            if constexpr (SPLIT) {
                tc_fence_after();
                cluster_sync_all();  // every pair's MMAs are through: stages may be written
                for (int q = 1; ok && q < p.split; ++q) {
                    // another pair's chunks, into slot q - 1 .. of that pair: the
                    // sources of an owner in ring order, the same in every run
                    const int to = (kpart + q) % p.split;
                    const int o0 = chunks * to / p.split, o1 = chunks * (to + 1) / p.split;
                    const uint32_t slot = static_cast<uint32_t>(p.split - 1 - q);
                    const uint32_t bytes = chunk_bytes * static_cast<uint32_t>((GATED ? 2 : 1) * (o1 - o0));
                    const uint32_t dst = map_to_rank(part0, 2u * static_cast<uint32_t>(to) + rank) + slot * bytes;
                    const int n = (GATED ? 2 : 1) * (o1 - o0);
                    for (int i = grp; i < n; i += kLpEpiGroups) {
                        // gated: the gate's chunks, then the up's
                        const int col = GATED && i >= o1 - o0 ? half + (o0 + i - (o1 - o0)) * 32 : (o0 + i) * 32;
                        uint32_t r[32];
                        tmem_ld32(taddr + static_cast<uint32_t>(col), r);
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            lp_st_cluster(dst + static_cast<uint32_t>(i) * chunk_bytes +
                                              static_cast<uint32_t>(j * LP_BM * 16),
                                          r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3]);
                    }
                }
                cluster_sync_all();  // the sums are with their owners
            }
            if (!ok) continue;  // the others still meet at the barriers above
            tc_fence_after();
#pragma unroll 1
            for (int c = c_begin; c < c_end; ++c) {
                const int n0 = t.n0 + c * 32;
                float v[32];
                {
                    uint32_t r[32];
                    tmem_ld32(taddr + static_cast<uint32_t>(c * 32), r);
                    if constexpr (SPLIT)
                        lp_add_parts(r, part0 + static_cast<uint32_t>(c - own0) * chunk_bytes, p.split - 1, part_bytes);
                    lp_scaled(r, cols + c * 32, sa, bias, v);
                }
                activate(v, p.e.act);
                if constexpr (GATED) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {  // (sixteen columns at a time: registers)
                        uint32_t r[16];
                        float u[16];
                        lp_tmem_ld16(taddr + static_cast<uint32_t>(half + c * 32 + 16 * h), r);
                        if constexpr (SPLIT)
                            lp_add_parts(r, part0 + static_cast<uint32_t>(own + c - own0) * chunk_bytes +
                                                static_cast<uint32_t>(4 * h * LP_BM * 16),
                                         p.split - 1, part_bytes);
                        lp_scaled(r, cols + half + c * 32 + 16 * h, sa, bias, u);
#pragma unroll
                        for (int j = 0; j < 16; ++j) v[16 * h + j] *= u[j];
                    }
                }
                if (!box_in(c)) continue;
                if (p.e.out_dtype == FP8L_E4M3) {
                    uint32_t w[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) w[i] = os.codes(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                    if (row_ok) {
                        uint4 *dst = reinterpret_cast<uint4 *>(static_cast<uint8_t *>(p.e.y) +
                                                               static_cast<size_t>(m) * p.e.width + n0);
                        dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
                        if (n0 + 32 <= p.e.width) dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
                    }
                    __syncwarp();
                    continue;
                }
                if (p.e.residual != nullptr) {
                    ok = __all_sync(0xFFFFFFFFu, mbar_wait(box_bar, box_phase, abort_flag, p.status,
                                                           p.wait_cycles, peer_abort));
                    if (!ok) break;  // (the lanes decide together: tcgen05.ld needs the whole warp)
                    box_phase ^= 1u;
                    loading = false;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const uint4 w = lp_ld_shared(lp_box_piece(box, lane, q));
                        const uint32_t rw[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float2 f = widen_pair(rw[j], p.e.out_dtype);
                            v[8 * q + 2 * j] += f.x;
                            v[8 * q + 2 * j + 1] += f.y;
                        }
                    }
                } else {
                    if (lane == 0) lp_stores_read<0>();
                    __syncwarp();
                }
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    st_shared_v4(lp_box_piece(box, lane, q), pack_out16(v[8 * q], v[8 * q + 1], p.e.out_dtype),
                                 pack_out16(v[8 * q + 2], v[8 * q + 3], p.e.out_dtype),
                                 pack_out16(v[8 * q + 4], v[8 * q + 5], p.e.out_dtype),
                                 pack_out16(v[8 * q + 6], v[8 * q + 7], p.e.out_dtype));
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) lp_store_box(&tmap_y, 2 * n0, box_row, box);
                if (c + 1 < c_end) load_res(c + 1);
            }
            if (!ok) continue;
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (leader)
                    mbar_arrive(tempty_bar(acc));
                else
                    mbar_arrive_remote(map_to_rank(tempty_bar(acc), even));
            }
            acc ^= 1;
            if (acc == 0) acc_phase ^= 1u;
        }
        // this warp's boxes have landed and left before the CTA exits
        if (lane == 0) {
            if (loading) mbar_wait_drain(box_bar, box_phase, p.status);
            asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        }
        __syncwarp();
    }

    // every copy, MMA and TMEM read of the pair is finished before TMEM is
    // released and before either CTA's shared memory goes away
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    tc_fence_after();
    if (warp == 1) {
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base),
                     "r"(kLpTmemCols)
                     : "memory");
    }
}

// Tile plan: 256-wide tiles, then the columns left over in tiles `tail_w`
// wide (accumulator columns, a multiple of `step`) when the most loaded pair
// then has less to do.  A tile w wide costs max(w, 96) / 256 of a full one
// (its tokens are loaded whatever its width).
struct LpPlan {
    int main_tiles, n_main, tail_w, tail_n;  // n_main in accumulator columns
};

LpPlan lp_plan(int tiles_m, int cols, int pairs, int step) {
    const int nb = (cols + LP_BN - 1) / LP_BN;
    const int64_t total = int64_t(tiles_m) * nb;
    LpPlan best{static_cast<int>(total), nb * LP_BN, 0, 0};
    auto cost = [&](int64_t main_tiles, int64_t tail_tiles, int w) {
        // main tiles go round the pairs, the tail tiles start after the last
        const int64_t mr = main_tiles % pairs, tr = tail_tiles % pairs;
        const int64_t wc = w > 96 ? w : 96;
        int64_t worst = 0;
        for (int q = 0; q < pairs; ++q) {
            const int64_t mc = main_tiles / pairs + (q < mr ? 1 : 0);
            const int64_t d = (q - mr + pairs) % pairs;
            const int64_t c = mc * LP_BN + (tail_tiles / pairs + (d < tr ? 1 : 0)) * wc;
            worst = c > worst ? c : worst;
        }
        return worst;
    };
    if (total % pairs == 0) return best;
    int64_t best_cost = cost(total, 0, LP_BN);
    int64_t c = total / pairs * pairs / tiles_m;  // whole blocks before the tail
    if (c > nb) c = nb;
    const int rem = cols - static_cast<int>(c) * LP_BN;
    if (rem <= 0) return best;
    for (int w = LP_BN - step; w >= step; w -= step) {
        const int tail_n = (rem + w - 1) / w;
        const int64_t cst = cost(c * tiles_m, int64_t(tail_n) * tiles_m, w);
        if (cst < best_cost) {
            best_cost = cst;
            best = LpPlan{static_cast<int>(c) * tiles_m, static_cast<int>(c) * LP_BN, w, tail_n};
        }
    }
    return best;
}

constexpr int kLpMaxDevices = 64;
constexpr int kLpMaxSplit = 4;  // pairs a cluster: eight CTAs, the portable size
std::atomic<int> g_lp_ready[kLpMaxDevices];
std::atomic<int> g_lp_clusters[kLpMaxDevices][kLpMaxSplit + 1];  // of `split` pairs the GPU holds at once

template <bool GATED, bool SPLIT>
bool lp_prepare() {
    return cudaFuncSetAttribute(linear_pair_kernel<GATED, SPLIT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(kLpSmemBytes)) == cudaSuccess;
}

int lp_clusters(int dev, int split) {
    int n = g_lp_clusters[dev][split].load(std::memory_order_relaxed);
    if (n > 0) return n;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(2 * split), 1, 1);
    cfg.blockDim = dim3(kLpThreads, 1, 1);
    cfg.dynamicSmemBytes = kLpSmemBytes;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(2 * split);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, linear_pair_kernel<false, true>, &cfg) != cudaSuccess || n < 1) {
        (void)cudaGetLastError();
        n = 1;
    }
    g_lp_clusters[dev][split].store(n, std::memory_order_relaxed);
    return n;
}

// Pairs that share a tile: the most whose clusters run at once, a power of
// two (the tile's eight chunks are dealt to them), each with four k-blocks or
// more.
int lp_split(int dev, int64_t tiles, int num_k_blocks) {
    int split = kLpMaxSplit;
    while (split > 1 && (tiles > lp_clusters(dev, split) || num_k_blocks < 4 * split)) split /= 2;
    return split;
}

}  // namespace

int launch_linear_pair(const LinearCall &c) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kLpMaxDevices || c.sms < 2) return FP8L_ECUDA;
    if (!g_lp_ready[dev].load(std::memory_order_acquire)) {
        if (!lp_prepare<false, false>() || !lp_prepare<true, false>() || !lp_prepare<false, true>() ||
            !lp_prepare<true, true>())
            return FP8L_ECUDA;
        g_lp_ready[dev].store(1, std::memory_order_release);
    }
    PairArgs p{};
    p.M = c.M;
    p.num_k_blocks = (c.K + LP_BK - 1) / LP_BK;
    p.tiles_m = static_cast<int>((int64_t(c.M) + 2 * LP_BM - 1) / (2 * LP_BM));
    const int pairs = c.sms / 2;
    const int cols = c.gated ? 2 * c.e.width : c.e.width;
    const int64_t whole = int64_t(p.tiles_m) * ((cols + LP_BN - 1) / LP_BN);
    p.split = lp_split(dev, whole, p.num_k_blocks);
    const LpPlan plan = p.split > 1 ? LpPlan{static_cast<int>(whole), (cols + LP_BN - 1) / LP_BN * LP_BN, 0, 0}
                                    : lp_plan(p.tiles_m, cols, pairs, c.gated ? 64 : 32);
    p.main_tiles = plan.main_tiles;
    p.n_main = c.gated ? plan.n_main / 2 : plan.n_main;
    p.tail_w = plan.tail_w;
    p.tail_n = plan.tail_n;
    p.prefetch = c.stable ? 1 : 0;
    p.a_scale = c.a_scale;
    p.a_per_token = c.a_per_token;
    p.w_scale = c.w_scale;
    p.w_per_channel = c.w_per_channel;
    p.e = c.e;
    p.status = c.status;
    const WaitConfig wc = wait_config();
    p.wait_cycles = wc.cycles;
    p.stall = wc.stall;

    CUtensorMap ma, mb, mbt;
    if (make_kmajor_map(&ma, c.x, c.M, c.K, LP_BK, LP_BM) != FP8L_OK ||
        make_kmajor_map(&mb, c.w, c.N, c.K, LP_BK, LP_BN / 2) != FP8L_OK)
        return FP8L_ECUDA;
    mbt = mb;
    if (plan.tail_n > 0 && make_kmajor_map(&mbt, c.w, c.N, c.K, LP_BK, plan.tail_w / 2) != FP8L_OK)
        return FP8L_ECUDA;

    CUtensorMap my = ma, mr = ma;  // (unused ones are any valid map)
    if (c.e.out_dtype != FP8L_E4M3) {
        const uint64_t dims[2] = {static_cast<uint64_t>(c.e.width) * 2, static_cast<uint64_t>(c.M)};
        const uint64_t strides[1] = {static_cast<uint64_t>(c.e.width) * 2};
        const uint32_t box[2] = {64, 32};
        if (make_swizzle64_map(&my, c.e.y, 2, dims, strides, box) != FP8L_OK ||
            (c.e.residual != nullptr &&
             make_swizzle64_map(&mr, c.e.residual, 2, dims, strides, box) != FP8L_OK))
            return FP8L_ECUDA;
    }

    const int64_t tiles = int64_t(plan.main_tiles) + int64_t(p.tiles_m) * plan.tail_n;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(2 * (p.split > 1 ? tiles * p.split : (tiles < pairs ? tiles : pairs))), 1, 1);
    cfg.blockDim = dim3(kLpThreads, 1, 1);
    cfg.dynamicSmemBytes = kLpSmemBytes;
    cfg.stream = c.stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(2 * p.split);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = c.stable ? 2 : 1;
    const auto launch = [&](auto kernel) { return cudaLaunchKernelEx(&cfg, kernel, ma, mb, mbt, my, mr, p); };
    const cudaError_t e = p.split > 1 ? (c.gated ? launch(linear_pair_kernel<true, true>) : launch(linear_pair_kernel<false, true>))
                                      : (c.gated ? launch(linear_pair_kernel<true, false>) : launch(linear_pair_kernel<false, false>));
    if (e != cudaSuccess) return FP8L_ECUDA;
    return launch_status();
}

}  // namespace fp8l
