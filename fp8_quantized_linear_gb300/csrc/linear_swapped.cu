// Linear layer on the tcgen05 tensor cores, operands swapped: weight rows on
// the MMA's M side, tokens on its N side (sm_103a).
//
// ("[Kernel][FP8] Initial support with dynamic per-tensor scaling": the W8A8
// product; "Marlin fp8": decode batches are bound by reading the weights.)
//
//   z[m, n] = sum_k x[m,k] dec(w[n,k]) * scale(m) w_scale(n) + bias(n)
//   y = the epilogue of epilogue.cuh
//
// For a few tokens the product is a weight stream.  A tile is D^T = W X^T of
// 128 weight rows by T tokens (16 <= T <= 128), so no MMA slot is spent on
// padding rows; weights go from HBM by TMA into shared memory and from there
// into the tensor core, and nothing decodes them.  With a gate the 128 rows
// are 64 gate rows and the 64 up rows of the same outputs (two boxes a
// stage), so both meet in one tile whatever the weights' layout.
//
// 16-bit tokens (W8A16) take the same path: a value scaled by a power of two
// per token is a sum of E4M3 parts, each 16 times finer than the one before
// (two for bf16: rounding to 4 significant bits leaves at most 4 of 8; three
// for fp16), and the parts are P T columns of one MMA instead of T.  The
// weights are never widened.  Parts are exact for values near the token's
// largest and stop at E4M3's smallest step: what is left is below 2^-21
// (bf16) or 2^-25 (fp16) of the largest magnitude of the token's row (or of
// 2^-119, where that is more), against 2^-8 and 2^-11 of the result for its own
// rounding.  (Widening the
// weights to 16 bits in tensor memory streamed them at 0.41 to 0.51 of HBM
// whatever the token count; see w8a16 in gemm_swapab.cu.)
//
// Structure (128 threads, one tile a CTA, two CTAs an SM so that one's
// epilogue overlaps the other's stream):
//   warp 0 lane 0  TMA producer into a ring of stages; with stable weights
//                  the kernel is a programmatic dependent of the preceding
//                  one and the first stages' weights are loaded before the
//                  wait for it.
//   warp 1         TMEM; lane 0 issues tcgen05.mma kind::f8f6f4 (M = 128,
//                  N = P T, K = 32), four a k-block.
//   all warps      epilogue: tcgen05.ld, the parts added, into a [T][128]
//                  float tile in the idle ring; then four channels a thread
//                  and token: scales, bias, gate, residual, cast.  A thread
//                  keeps its channels for all its tokens, so scales and
//                  biases are read once, while the stream runs.
// When there are fewer tiles than CTA slots a cluster of `split` CTAs shares
// a tile and splits its k-blocks; the owners add the float tiles through
// distributed shared memory in a fixed order.  Every wait is bounded.
//
// Measured (GB300, replayed graphs over rotating weights; of the copy
// bandwidth): gate/up of 16 tokens, 28672 x 4096 with E4M3 output, 22.6 us, 0.77
// (DRAM reads the weights once), of 128 tokens 28.6 us; 4096 x 14336 of 16
// tokens 14.4 us, 0.60; W8A16 4096 x 11008 of 16 tokens 14.1 us, 0.48 (17.6
// through fp8_w8a16_mm, without the addition), 11008 x 4096 of 47 fp16 tokens
// 17.1 us.  Short
// streams are bound by their ends: launch, first bytes, the cluster's sums.
// Tried (16 tokens of 28672 x 4096 at 22.9 us): 256 threads (27.2: the second
// CTA's start), three CTAs of 75 KB an SM (23.3), one of 112 KB (23.2; 4096 x
// 14336 15.0); at 128 tokens of 28672 x 4096 (33.5 us then), pairs of SMs that
// share the tokens (33.5; a few tokens 5 to 10 % slower), rings of their own for
// weights and tokens (37.6).
#include <atomic>

#include "linear_launch.cuh"
#include "quant_device.cuh"
#include "skinny_device.cuh"
#include "tc_device.cuh"

namespace fp8l {
namespace {

constexpr int LS_BM = 128;            // weight rows a tile = MMA M
constexpr int LS_BK = 128;            // k-block, bytes
constexpr int kLsThreads = 128;
constexpr int kLsWBytes = LS_BM * LS_BK;
constexpr int kLsMaxStages = 16;
constexpr int kLsMaxSplit = 8;        // portable cluster size
constexpr int kLsPitch = LS_BM + 4;   // floats a token row of the float tile
constexpr int kLsBatch = 4;           // epilogue items a thread takes together, where it has so many
// two CTAs per SM: 233472 bytes of shared memory per SM, 1024 reserved per CTA
constexpr size_t kLsSmem = 112 * 1024;

// tokens a tile holds: with one part 128 (an accumulator of 128 columns);
// with parts so many that three stages of weights and parts fit kLsSmem
constexpr int ls_max_tokens(int parts) { return parts == 1 ? 128 : (parts == 2 ? 64 : 48); }

// Tiles that M tokens take, and the tokens of each (a multiple of 16).
int tokens_a_tile(int parts, int64_t M, int *tiles) {
    const int64_t most = ls_max_tokens(parts);
    const int64_t n = (M + most - 1) / most;
    *tiles = static_cast<int>(n);
    return static_cast<int>(((M + n - 1) / n + 15) & ~int64_t(15));
}

struct SwappedArgs {
    int M, K, T;  // T: tokens a tile, a multiple of 16
    int parts;    // MMA N = parts * T
    int stages, stage_bytes;
    int num_k_blocks, split, m_tiles;
    int gated, packed;
    int prefetch;
    const float *token_scale;  // [1], or [M] per token
    int per_token;
    const float *w_scale;
    int w_per_channel;
    Epilogue e;
    unsigned *status;
    long long wait_cycles;
    unsigned stall;
};

__device__ __forceinline__ void ls_mma(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                       uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void ls_tma_4d(uint32_t dst, const CUtensorMap *map, int c0, int c1, int c2,
                                          int c3, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
        : "memory");
}

// Descriptor of a K-major operand in the 64-byte swizzle (packed weights):
// 64-byte rows, 8-row groups 512 bytes apart, swizzle mode 4.
__device__ __forceinline__ uint64_t sw64_desc(uint32_t saddr) {
    return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(1) << 16) |
           (static_cast<uint64_t>(512 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) |
           (static_cast<uint64_t>(4) << 61);
}

__device__ __forceinline__ void ls_tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

__device__ __forceinline__ void tmem_wait_ld() {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void st_shared_float(uint32_t addr, float v) {
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// (no memory clobber: the float tile does not change between the barriers
// around its reads, which may pass the results' stores)
__device__ __forceinline__ float4 ld_shared_float4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr));
    return v;
}

__device__ __forceinline__ uint2 ld_global_uint2(const void *p) {
    uint2 v;
    asm volatile("ld.global.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p) : "memory");
    return v;
}

// Four columns of the float tile for each of B items (from another CTA: for
// the first `valid` of them), the cluster's partials added in rank order.
template <int B>
__device__ __forceinline__ void ls_sums(const uint32_t (&off)[B], int valid, uint32_t shift, int split,
                                        float (&v)[4 * B]) {
#pragma unroll
    for (int u = 0; u < B; ++u) {
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
        if (split == 1) {
            a = ld_shared_float4(off[u] + shift);
        } else if (u < valid) {
            float4 part[kLsMaxSplit];
#pragma unroll
            for (int q = 0; q < kLsMaxSplit; ++q)
                if (q < split) part[q] = ld_cluster_v4(off[u] + shift, static_cast<uint32_t>(q));
#pragma unroll
            for (int q = 0; q < kLsMaxSplit; ++q) {
                if (q < split) {
                    a.x += part[q].x;
                    a.y += part[q].y;
                    a.z += part[q].z;
                    a.w += part[q].w;
                }
            }
        }
        v[4 * u] = a.x;
        v[4 * u + 1] = a.y;
        v[4 * u + 2] = a.z;
        v[4 * u + 3] = a.w;
    }
}

template <int B>  // epilogue items a thread takes together
__global__ void __launch_bounds__(kLsThreads, 2)
linear_swapped_kernel(const __grid_constant__ CUtensorMap tmap_w,
                      const __grid_constant__ CUtensorMap tmap_x, const SwappedArgs p) {
    // every CTA has started: the next kernel on the stream may be scheduled
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t sbase = (raw + 1023u) & ~1023u;  // swizzle atoms
    uint8_t *gbase = smem_raw + (sbase - raw);
    const int S = p.stages;
    const uint32_t sb = static_cast<uint32_t>(p.stage_bytes);
    const uint32_t ring_bytes = static_cast<uint32_t>(S) * sb;
    const uint32_t bar0 = sbase + ring_bytes;
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (S + s); };
    const uint32_t done_bar = bar0 + 8u * (2 * S);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(gbase + ring_bytes + (2 * S + 1) * 8);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    float *sa_sh = reinterpret_cast<float *>(tmem_slot + 2);  // [T]: the tokens' scales
    const int cols = p.parts * p.T;
    const uint32_t tmem_cols = cols <= 32 ? 32u : (cols <= 64 ? 64u : (cols <= 128 ? 128u : 256u));

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int split = p.split;
    const int rank = split > 1 ? static_cast<int>(blockIdx.x) % split : 0;
    const int tile = static_cast<int>(blockIdx.x) / split;
    const int mt = tile % p.m_tiles, nt = tile / p.m_tiles;
    const int base = p.num_k_blocks / split, rem = p.num_k_blocks % split;
    const int kb_begin = rank * base + (rank < rem ? rank : rem);
    const int nkb = base + (rank < rem ? 1 : 0);

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
        }
        mbar_init(done_bar, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(tmem_slot)),
                     "r"(tmem_cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;

    if (warp == 0) {
        if (lane == 0) {
            asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmap_w)) : "memory");
            asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmap_x)) : "memory");
            // the weight boxes of one k-block (with a gate: gate rows, up rows)
            auto load_w = [&](uint32_t st, int kb, uint32_t bar) {
                if (!p.packed) {
                    if (!p.gated) {
                        tma_load_2d(st, &tmap_w, kb * LS_BK, nt * LS_BM, bar);
                    } else {
                        tma_load_2d(st, &tmap_w, kb * LS_BK, nt * (LS_BM / 2), bar);
                        tma_load_2d(st + kLsWBytes / 2, &tmap_w, kb * LS_BK,
                                    p.e.width + nt * (LS_BM / 2), bar);
                    }
                    return;
                }
                // packed: two chunks of 64 k, [groups of 16 rows][16 rows][64 bytes] each
                for (int c = 0; c < 2; ++c) {
                    const uint32_t dst = st + c * (kLsWBytes / 2);
                    if (!p.gated) {
                        ls_tma_4d(dst, &tmap_w, 0, 0, 2 * kb + c, nt * (LS_BM / 16), bar);
                    } else {
                        ls_tma_4d(dst, &tmap_w, 0, 0, 2 * kb + c, nt * (LS_BM / 32), bar);
                        ls_tma_4d(dst + kLsWBytes / 4, &tmap_w, 0, 0, 2 * kb + c,
                                  p.e.width / 16 + nt * (LS_BM / 32), bar);
                    }
                }
            };
            const int x_row = mt * cols;
            const int pre = p.prefetch ? (nkb < S ? nkb : S) : 0;
            for (int i = 0; i < pre; ++i) {
                mbar_expect_tx(full_bar(i), sb);
                load_w(sbase + i * sb, kb_begin + i, full_bar(i));
            }
            asm volatile("griddepcontrol.wait;" ::: "memory");
            for (int i = 0; i < pre; ++i)
                tma_load_2d(sbase + i * sb + kLsWBytes, &tmap_x, (kb_begin + i) * LS_BK, x_row, full_bar(i));
            uint32_t issued = (1u << pre) - 1u;  // stages with a load in flight (parity 0 so far)
            uint32_t issued_parity = 0;
            int stage = pre == S ? 0 : pre;
            uint32_t phase = pre == S ? 1u : 0u;
            for (int i = pre; i < nkb; ++i) {
                if (!mbar_wait(empty_bar(stage), phase ^ 1u, abort_flag, p.status, p.wait_cycles)) break;
                const uint32_t st = sbase + stage * sb;
                mbar_expect_tx(full_bar(stage), sb);
                load_w(st, kb_begin + i, full_bar(stage));
                tma_load_2d(st + kLsWBytes, &tmap_x, (kb_begin + i) * LS_BK, x_row, full_bar(stage));
                issued |= 1u << stage;
                issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
                if (++stage == S) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            // every load this thread issued lands before the CTA exits
            for (int s = 0; s < S; ++s)
                if (issued & (1u << s)) mbar_wait_drain(full_bar(s), (issued_parity >> s) & 1u, p.status);
        }
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0) {
            // (the waits below are limited, the preceding kernel's time is not)
            asm volatile("griddepcontrol.wait;" ::: "memory");
            // kind::f8f6f4, D f32, A and B E4M3 K-major, N = parts * T, M = 128
            const uint32_t idesc = (1u << 4) | (static_cast<uint32_t>(cols >> 3) << 17) |
                                   (static_cast<uint32_t>(LS_BM >> 4) << 24);
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            if (p.stall & kStallMma) ok = mbar_wait(done_bar, 0, abort_flag, p.status, p.wait_cycles);
            for (int i = 0; ok && i < nkb; ++i) {
                if (!mbar_wait_fast(full_bar(stage), phase, abort_flag, p.status, p.wait_cycles)) break;
                tc_fence_after();
                const uint32_t st = sbase + stage * sb;
                const uint64_t dx = sw128_desc(st + kLsWBytes);
                if (p.packed) {
                    const uint64_t d0 = sw64_desc(st), d1 = sw64_desc(st + kLsWBytes / 2);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        ls_mma(tmem_base, (k < 2 ? d0 : d1) + 2 * (k & 1), dx + 2 * k, idesc,
                               (i | k) != 0 ? 1u : 0u);
                } else {
                    const uint64_t dw = sw128_desc(st);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        ls_mma(tmem_base, dw + 2 * k, dx + 2 * k, idesc, (i | k) != 0 ? 1u : 0u);
                }
                mma_commit(empty_bar(stage));
                if (++stage == S) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            // the accumulator is complete (or abandoned) once these retire; the
            // other warps meet this one at a barrier instead of polling for it
            // (polling warps take issue slots from the two that feed the MMAs)
            mma_commit(done_bar);
            if (!mbar_wait(done_bar, 0, abort_flag, p.status, p.wait_cycles))
                mbar_wait_drain(done_bar, 0, p.status);  // none in flight when the CTA exits
            tc_fence_before();
        }
        __syncwarp();
    }

    // ---- epilogue: every thread
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // items of this tile: (token, four output channels), dealt to the
    // cluster's CTAs; a thread's channels are the same for all its items
    const int groups = p.gated ? LS_BM / 8 : LS_BM / 4;  // of four channels, a power of two
    const int gshift = p.gated ? 4 : 5;
    const int m0 = mt * p.T;
    const int rows = p.M - m0 < p.T ? p.M - m0 : p.T;
    const int items = rows * groups;
    const int i0 = static_cast<int>((static_cast<long long>(items) * rank) / split);
    const int i1 = static_cast<int>((static_cast<long long>(items) * (rank + 1)) / split);
    const int first = i0 + static_cast<int>(threadIdx.x);
    const int c4 = (first & (groups - 1)) * 4;
    const int n = nt * (p.gated ? LS_BM / 2 : LS_BM) + c4;
    const bool in = n < p.e.width;  // width % 16 == 0: four channels are in or out together
    float sw[4], bias[4], sw_up[4], bias_up[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        sw[j] = in ? epi_ld_f32(p.w_scale + (p.w_per_channel ? n + j : 0)) : 0.0f;
        bias[j] = in ? epi_bias(p.e, n + j) : 0.0f;
        sw_up[j] = bias_up[j] = 0.0f;
        if (p.gated && in) {
            sw_up[j] = epi_ld_f32(p.w_scale + (p.w_per_channel ? p.e.width + n + j : 0));
            bias_up[j] = epi_bias(p.e, p.e.width + n + j);
        }
    }
    const OutScale os = OutScale::make(p.e.out_dtype == FP8L_E4M3 ? epi_ld_f32(p.e.out_scale) : 1.0f);
    for (int t = threadIdx.x; t < rows; t += kLsThreads)
        sa_sh[t] = epi_ld_f32(p.token_scale + (p.per_token ? m0 + t : 0));
    // from one of a thread's items to the next: tokens, bytes of y
    const int t0 = first >> gshift, t_step = kLsThreads >> gshift;
    const int es = p.e.out_dtype == FP8L_E4M3 ? 1 : 2;
    const size_t y_step = static_cast<size_t>(t_step) * p.e.width * es;
    const size_t y0 = (static_cast<size_t>(m0 + t0) * p.e.width + n) * es;
    // residuals of a batch of items, loaded two batches ahead
    struct Batch {
        uint2 res[B];
    };
    const uint8_t *r_next = static_cast<const uint8_t *>(p.e.residual) + y0;  // (16-bit output)
    auto load_batch = [&](int i) {
        Batch b;
#pragma unroll
        for (int u = 0; u < B; ++u) {
            b.res[u] = make_uint2(0, 0);
            if (in && i + u * kLsThreads < i1) b.res[u] = ld_global_uint2(r_next);
            r_next += y_step;
        }
        return b;
    };
    constexpr int kStep = B * kLsThreads;
    Batch next{}, after{};
    if (p.e.residual != nullptr) {
        next = load_batch(first);
        after = load_batch(first + kStep);
    }

    __syncthreads();
    tc_fence_after();
    // (a warp's lanes decide together: tcgen05.ld needs the whole warp)
    bool ok = __all_sync(0xFFFFFFFFu, !*abort_flag);
    // accumulator row (weight row) 32 warp + lane, token columns 0 .. T-1 (the
    // parts' columns added), into part[t][row] at the start of the ring
    if (ok) {
        const int row = warp * 32 + lane;
        const uint32_t taddr = tmem_base + (static_cast<uint32_t>(warp * 32) << 16);
        for (int c = 0; c < p.T; c += 16) {
            uint32_t r[16];
            float v[16];
            ls_tmem_ld16(taddr + static_cast<uint32_t>(c), r);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] = __uint_as_float(r[j]);
            float f = 0.0625f;
            for (int q = 1; q < p.parts; ++q, f *= 0.0625f) {
                ls_tmem_ld16(taddr + static_cast<uint32_t>(q * p.T + c), r);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 16; ++j) v[j] = fmaf(__uint_as_float(r[j]), f, v[j]);
            }
#pragma unroll
            for (int j = 0; j < 16; ++j)
                st_shared_float(sbase + static_cast<uint32_t>(((c + j) * kLsPitch + row) * 4), v[j]);
        }
    }
    tc_fence_before();
    if (split > 1)
        cluster_sync_all();
    else
        __syncthreads();
    ok = !*abort_flag;

    // a batch's items (i, i + kLsThreads, ...) in stages, so that the branches
    // on what the epilogue does are taken once for all of them: one item after
    // the other took 500 cycles each (128 tokens of 28672 x 128 12.7 us, 7.2 in
    // fours; of 28672 x 4096 33.4 and 30.5)
    uint32_t at = sbase + static_cast<uint32_t>((t0 * kLsPitch + c4) * 4);
    const uint32_t at_step = static_cast<uint32_t>(t_step * kLsPitch * 4);
    const float *scale = sa_sh + t0;
    uint8_t *y = static_cast<uint8_t *>(p.e.y) + y0;
    for (int i = first; ok && in && i < i1; i += kStep) {
        const Batch cur = next;
        next = after;
        if (p.e.residual != nullptr) after = load_batch(i + 2 * kStep);
        uint32_t off[B];
        float pre[B], sa[B], v[4 * B];
#pragma unroll
        for (int u = 0; u < B; ++u) {
            const bool valid = i + u * kLsThreads < i1;  // (else the first once more)
            off[u] = valid ? at + u * at_step : at;
            // a token's own scale (of its parts, a power of two) goes to the
            // sums: times a channel's it may leave the normal range
            const float s = scale[valid ? u * t_step : 0];
            pre[u] = p.parts > 1 ? s : 1.0f;
            sa[u] = p.parts > 1 ? 1.0f : s;
        }
        at += B * at_step;
        scale += B * t_step;
        const int valid = (i1 - i + kLsThreads - 1) / kLsThreads;
        ls_sums(off, valid, 0, split, v);
#pragma unroll
        for (int j = 0; j < 4 * B; ++j) v[j] = fmaf(v[j] * pre[j / 4], sa[j / 4] * sw[j % 4], bias[j % 4]);
        activate(v, p.e.act);
        if (p.gated) {
            float up[4 * B];
            ls_sums(off, valid, LS_BM / 2 * 4, split, up);
#pragma unroll
            for (int j = 0; j < 4 * B; ++j)
                v[j] *= fmaf(up[j] * pre[j / 4], sa[j / 4] * sw_up[j % 4], bias_up[j % 4]);
        }
        if (p.e.out_dtype == FP8L_E4M3) {
#pragma unroll
            for (int u = 0; u < B; ++u) {
                const uint32_t c = os.codes(v[4 * u], v[4 * u + 1], v[4 * u + 2], v[4 * u + 3]);
                if (i + u * kLsThreads < i1) *reinterpret_cast<uint32_t *>(y) = c;
                y += y_step;
            }
        } else {
            if (p.e.residual != nullptr) {
#pragma unroll
                for (int u = 0; u < B; ++u) {
                    const float2 a = widen_pair(cur.res[u].x, p.e.out_dtype), b = widen_pair(cur.res[u].y, p.e.out_dtype);
                    v[4 * u] += a.x;
                    v[4 * u + 1] += a.y;
                    v[4 * u + 2] += b.x;
                    v[4 * u + 3] += b.y;
                }
            }
            uint2 w[B];
#pragma unroll
            for (int u = 0; u < B; ++u)
                w[u] = make_uint2(pack_out16(v[4 * u], v[4 * u + 1], p.e.out_dtype),
                                  pack_out16(v[4 * u + 2], v[4 * u + 3], p.e.out_dtype));
#pragma unroll
            for (int u = 0; u < B; ++u) {
                if (i + u * kLsThreads < i1) *reinterpret_cast<uint2 *>(y) = w[u];
                y += y_step;
            }
        }
    }
    if (split > 1) cluster_sync_all();  // peers may still be reading this CTA's partials

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) {
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base),
                     "r"(tmem_cols)
                     : "memory");
    }
}

// Stand-in for the kernel in occupancy queries: the same block and shared
// memory without TMEM (for a kernel with tcgen05.alloc the query answers one
// CTA per SM whatever its shared memory).
__global__ void __launch_bounds__(kLsThreads, 2) linear_swapped_twin() {}

constexpr int kLsMaxDevices = 64;
std::atomic<int> g_ls_smem_per_sm[kLsMaxDevices];  // 0: attributes not set yet
std::atomic<int> g_ls_reserved[kLsMaxDevices];
// clusters of `split` CTAs the GPU holds at once, by KB of shared memory
std::atomic<int> g_ls_clusters[kLsMaxDevices][kLsSmem / 1024 + 1][kLsMaxSplit + 1];

int ls_prepare(int dev) {
    if (g_ls_smem_per_sm[dev].load(std::memory_order_acquire) > 0) return FP8L_OK;
    int per_sm = 0, reserved = 0;
    for (const auto kernel : {linear_swapped_kernel<1>, linear_swapped_kernel<kLsBatch>})
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kLsSmem)) !=
                cudaSuccess ||
            cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                                 cudaSharedmemCarveoutMaxShared) != cudaSuccess)
            return FP8L_ECUDA;
    if (cudaFuncSetAttribute(linear_swapped_twin, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(kLsSmem)) != cudaSuccess ||
        cudaFuncSetAttribute(linear_swapped_twin, cudaFuncAttributePreferredSharedMemoryCarveout,
                             cudaSharedmemCarveoutMaxShared) != cudaSuccess ||
        cudaDeviceGetAttribute(&per_sm, cudaDevAttrMaxSharedMemoryPerMultiprocessor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&reserved, cudaDevAttrReservedSharedMemoryPerBlock, dev) != cudaSuccess)
        return FP8L_ECUDA;
    g_ls_reserved[dev].store(reserved, std::memory_order_relaxed);
    g_ls_smem_per_sm[dev].store(per_sm, std::memory_order_release);
    return FP8L_OK;
}

int ls_clusters(int dev, size_t smem, int split) {
    std::atomic<int> &slot = g_ls_clusters[dev][smem / 1024][split];
    int n = slot.load(std::memory_order_relaxed);
    if (n > 0) return n;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(split), 1, 1);
    cfg.blockDim = dim3(kLsThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(split);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, linear_swapped_twin, &cfg) != cudaSuccess || n < 1) {
        (void)cudaGetLastError();
        n = 1;
    }
    slot.store(n, std::memory_order_relaxed);
    return n;
}

}  // namespace

int launch_linear_swapped(const LinearCall &c, int parts, const float *token_scale) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kLsMaxDevices) return FP8L_ECUDA;
    if (ls_prepare(dev) != FP8L_OK) return FP8L_ECUDA;
    SwappedArgs p{};
    p.M = c.M;
    p.K = c.K;
    p.parts = parts;
    p.T = tokens_a_tile(parts, c.M, &p.m_tiles);
    const int cols = parts * p.T;
    if (int64_t(p.m_tiles) * cols > 0x7FFFFFFF) return FP8L_ESHAPE;  // token rows of all tiles
    p.stage_bytes = kLsWBytes + cols * LS_BK;
    // the most stages that fit; the float tile reuses the ring
    int stages = static_cast<int>((kLsSmem - 1024 - 24 - 4 * p.T) / (p.stage_bytes + 16));
    if (stages > kLsMaxStages) stages = kLsMaxStages;
    p.stages = stages;
    const size_t smem = 1024 + size_t(stages) * p.stage_bytes + size_t(2 * stages + 1) * 8 + 16 + 4 * size_t(p.T);
    if (stages < 2 || smem > kLsSmem || size_t(p.T) * kLsPitch * 4 > size_t(stages) * p.stage_bytes)
        return FP8L_ESHAPE;
    p.num_k_blocks = (c.K + LS_BK - 1) / LS_BK;
    p.gated = c.gated;
    p.packed = c.packed;
    p.prefetch = c.stable ? 1 : 0;
    p.token_scale = token_scale;
    p.per_token = parts > 1 ? 1 : c.a_per_token;
    p.w_scale = c.w_scale;
    p.w_per_channel = c.w_per_channel;
    p.e = c.e;
    p.status = c.status;
    const WaitConfig wc = wait_config();
    p.wait_cycles = wc.cycles;
    p.stall = wc.stall;

    // split: the largest cluster whose launch runs in one wave (clusters sit
    // in one GPC, so fewer of s CTAs fit than slots / s)
    const int span = c.gated ? LS_BM / 2 : LS_BM;
    const int64_t tiles = int64_t((c.e.width + span - 1) / span) * p.m_tiles;
    const int slots = g_ls_smem_per_sm[dev].load(std::memory_order_relaxed) /
                      static_cast<int>(smem + g_ls_reserved[dev].load(std::memory_order_relaxed));
    int split = kLsMaxSplit < p.num_k_blocks ? kLsMaxSplit : p.num_k_blocks;
    while (split > 1 && (tiles * split > int64_t(c.sms) * slots || tiles > ls_clusters(dev, smem, split)))
        --split;
    p.split = split;
    if (tiles * split > 0x7FFFFFFF) return FP8L_ESHAPE;

    CUtensorMap mw, mx;
    if (c.packed) {
        const uint64_t C = static_cast<uint64_t>((c.K + 63) / 64);
        const uint64_t dims[4] = {64, 16, C, static_cast<uint64_t>(c.N / 16)};
        const uint64_t strides[3] = {64, 1024, C * 1024};
        const uint32_t box[4] = {64, 16, 1, static_cast<uint32_t>(span / 16)};
        if (make_swizzle64_map(&mw, c.w, 4, dims, strides, box) != FP8L_OK) return FP8L_ECUDA;
    } else if (make_kmajor_map(&mw, c.w, c.N, c.K, LS_BK, span) != FP8L_OK) {
        return FP8L_ECUDA;
    }
    const int64_t x_rows = parts > 1 ? int64_t(p.m_tiles) * cols : c.M;
    if (make_kmajor_map(&mx, c.x, x_rows, c.K, LS_BK, cols) != FP8L_OK) return FP8L_ECUDA;

    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(tiles * split), 1, 1);
    cfg.blockDim = dim3(kLsThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = c.stream;
    cudaLaunchAttribute attr[2];
    int nattr = 0;
    if (split > 1) {
        attr[nattr].id = cudaLaunchAttributeClusterDimension;
        attr[nattr].val.clusterDim.x = static_cast<unsigned>(split);
        attr[nattr].val.clusterDim.y = 1;
        attr[nattr].val.clusterDim.z = 1;
        ++nattr;
    }
    if (c.stable) {
        attr[nattr].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[nattr].val.programmaticStreamSerializationAllowed = 1;
        ++nattr;
    }
    cfg.attrs = attr;
    cfg.numAttrs = nattr;
    // items a CTA of a full tile (see the kernel) has: taken in fours where a
    // thread has more than two, else one by one (4096 x 4096 of one token, split
    // eight ways, 7.4 us, 7.8 in fours)
    const int items = (c.M < p.T ? c.M : p.T) * (span / 4) / split;
    const auto kernel = items > 2 * kLsThreads ? linear_swapped_kernel<kLsBatch> : linear_swapped_kernel<1>;
    if (cudaLaunchKernelEx(&cfg, kernel, mw, mx, p) != cudaSuccess) return FP8L_ECUDA;
    return launch_status();
}

// ---------------------------------------------------------------- tokens in parts

namespace {

constexpr int kSplitThreads = 256;
constexpr int kSplitSlice = 8 * kSplitThreads;  // values a block converts

// Row m of x as P rows of E4M3 codes: x 2^e = p0 + p1 / 16 (+ p2 / 256), 2^e
// bringing the row's largest magnitude to [128, 256), where a rounding's
// remainder times 16 stays below E4M3's largest.  Token m of tile i = m / T
// goes to rows i P T + q T + m % T; its scale 2^-e to scale[m].  Every block
// of a row takes the row's maximum itself (a few KB from L2); blocks of slice
// 0 write the scale.
template <int DT, int P>
__global__ void __launch_bounds__(kSplitThreads)
split_tokens_kernel(const uint4 *x, int K, int T, uint8_t *codes, float *scale) {
    __shared__ uint32_t red[33];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    pdl_wait();
    const int m = blockIdx.x, words = K / 8;
    const uint4 *row = x + static_cast<size_t>(m) * words;
    const int mine = blockIdx.y * kSplitThreads + threadIdx.x;
    const uint4 own = mine < words ? ld_act16(row + mine) : make_uint4(0, 0, 0, 0);
    uint32_t mag = word_mag_max<DT>(own, 0);
    for (int w0 = threadIdx.x; w0 < words; w0 += 8 * kSplitThreads) {
        uint4 v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int w = w0 + u * kSplitThreads;
            v[u] = w < words ? ld_act16(row + w) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) mag = word_mag_max<DT>(v[u], mag);
    }
    const float amax = mag_bits_to_float<DT>(block_max_u32(fold_mag<DT>(mag), red));
    // exponent that brings amax to [128, 256), kept where 2^e and 2^-e are normal
    int e = amax > 0.0f ? 7 - ilogbf(amax) : 0;
    e = e > 126 ? 126 : (e < -126 ? -126 : e);
    const float up = __int_as_float((e + 127) << 23);
    // (codes are finite: a row with a value that is not has NaN as its scale)
    if (blockIdx.y == 0 && threadIdx.x == 0)
        scale[m] = amax <= 3.4e38f ? __int_as_float((127 - e) << 23) : __int_as_float(0x7FC00000);
    if (mine >= words) return;
    const uint32_t w4[4] = {own.x, own.y, own.z, own.w};
    float f[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint64_t two = widen16<DT>(w4[j]);
        f[2 * j] = __uint_as_float(static_cast<uint32_t>(two)) * up;
        f[2 * j + 1] = __uint_as_float(static_cast<uint32_t>(two >> 32)) * up;
    }
    uint8_t *out = codes + (static_cast<size_t>(m / T) * P * T + m % T) * K + 8 * static_cast<size_t>(mine);
#pragma unroll
    for (int q = 0; q < P; ++q) {
        uint32_t c[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            c[j] = e4m3x2(f[2 * j], f[2 * j + 1]);
            const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(c[j]), __NV_E4M3);
            const float2 d = __half22float2(__half2(h));
            f[2 * j] = (f[2 * j] - d.x) * 16.0f;  // (exact)
            f[2 * j + 1] = (f[2 * j + 1] - d.y) * 16.0f;
        }
        *reinterpret_cast<uint2 *>(out + static_cast<size_t>(q) * T * K) =
            make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
    }
}

}  // namespace

int linear_parts(int x_dtype) { return x_dtype == FP8L_BF16 ? 2 : 3; }

bool linear_parts_fit(int x_dtype, int64_t M, int64_t N) {
    const int parts = linear_parts(x_dtype);
    int tiles = 0;
    const int T = tokens_a_tile(parts, M, &tiles);
    // rows of the parts, and CTAs (of 128 weight rows, gated or not)
    return int64_t(tiles) * parts * T <= 0x7FFFFFFF && tiles * ((N + LS_BM - 1) / LS_BM) <= 0x7FFFFFFF;
}

size_t linear_parts_bytes(int x_dtype, int64_t M, int64_t K) {
    const int parts = linear_parts(x_dtype);
    int tiles = 0;
    const int T = tokens_a_tile(parts, M, &tiles);
    return size_t(tiles) * parts * T * size_t(K) + ((size_t(M) * 4 + 15) & ~size_t(15));
}

int linear_split_tokens(const LinearCall &c, void *scratch, const float **token_scale) {
    int tiles = 0;
    const int parts = linear_parts(c.x_dtype);
    const int T = tokens_a_tile(parts, c.M, &tiles);
    uint8_t *codes = static_cast<uint8_t *>(scratch);
    float *scale = reinterpret_cast<float *>(codes + size_t(tiles) * parts * T * c.K);
    *token_scale = scale;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(c.M, (c.K + kSplitSlice - 1) / kSplitSlice, 1);
    cfg.blockDim = dim3(kSplitThreads, 1, 1);
    cfg.stream = c.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const uint4 *x = static_cast<const uint4 *>(c.x);
    const cudaError_t e = c.x_dtype == FP8L_BF16
                              ? cudaLaunchKernelEx(&cfg, split_tokens_kernel<FP8L_BF16, 2>, x, c.K, T, codes, scale)
                              : cudaLaunchKernelEx(&cfg, split_tokens_kernel<FP8L_F16, 3>, x, c.K, T, codes, scale);
    if (e != cudaSuccess) return FP8L_ECUDA;
    return launch_status();
}

}  // namespace fp8l
