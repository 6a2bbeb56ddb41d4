// Linear layer of a few tokens: weights streamed through registers (sm_103a).
//
// ("Marlin fp8": weight-only decode, bound by reading the weights; "[Kernel]
// [FP8] Initial support ...", the M = 1..16 rows of the microbenchmark.)
//
//   z[m, n] = sum_k x[m,k] dec(w[n,k]) * scale(m) w_scale(n) + bias(n)
//   y = the epilogue of epilogue.cuh
//
// The weights are read once and are all that counts.  A CTA owns 16 weight
// rows and a group of up to 8 (two tiles: 16) tokens; its 16 warps split K in
// 64-element chunks and add their partial tiles in shared memory.  Lane (g, t)
// reads 16 contiguous bytes of rows g and g + 8 of a chunk with one streaming
// load each, which are its own fragments of mma.sync (weights the 16-row A
// operand, tokens the 8-column B operand; the k order inside a chunk is the
// same permutation for both).  Nothing is staged, so the first bytes reach the
// tensor cores one round trip after the launch: that start is where this form
// beats the swapped tcgen05 kernel (4096 x 4096 of one token 5.1 against 7.4
// us, 16.8 MB at 0.48 of HBM), which takes over where a product is long enough to hide its own.
//
// With a gate rows g are gate rows and rows g + 8 the up rows of the same
// eight outputs: an accumulator holds both, and whole 512-byte halves of the
// packed layout's blocks are read (8 rows each) wherever the two lie.
//
// E4M3 tokens use the E4M3 form of the MMA; 16-bit tokens have the weights
// decoded by the hardware conversion (exact; for bf16 widened once more).
// Epilogue: one output a thread; its scale, bias and residual are loaded
// while the slower warps still stream.
#include <cuda_fp8.h>

#include "linear_launch.cuh"
#include "skinny_device.cuh"

namespace fp8l {
namespace {

constexpr int kStWarps = 16;
constexpr int kStBlock = 1024;  // bytes of a packed block: 16 rows x 64 k

struct StreamArgs {
    const uint8_t *w;
    const void *x;
    int M, N, K;
    const float *a_scale;  // E4M3 tokens only
    int a_per_token;
    const float *w_scale;
    int w_per_channel;
    Epilogue e;
};

// both byte pairs of a word as f16x2: bytes (0, 1) -> lo, (2, 3) -> hi
__device__ __forceinline__ void st_decode(uint32_t w, uint32_t &lo, uint32_t &hi) {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}

__device__ __forceinline__ uint32_t st_to_bf16(uint32_t h) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
    const __nv_bfloat162 b = __floats2bfloat162_rn(f.x, f.y);
    return *reinterpret_cast<const uint32_t *>(&b);
}

template <int XDT>
__device__ __forceinline__ void st_mma16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    if constexpr (XDT == FP8L_BF16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
            "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
            "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <int XDT, int NT, int UNROLL, bool PACKED, bool GATED>
__global__ void __launch_bounds__(kStWarps * 32, 2) linear_stream_kernel(const StreamArgs p) {
    constexpr int kXWords = XDT == FP8L_E4M3 ? 4 : 8;  // 32-bit words a lane, token and chunk
    constexpr int kXBytes = XDT == FP8L_E4M3 ? 1 : 2;
    __shared__ float red[kStWarps][NT][4][32];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    const int lane = threadIdx.x & 31;
    const int warp = threadIdx.x >> 5;
    const int g = lane >> 2;
    const int t4 = lane & 3;
    const int m0 = blockIdx.y * 16;
    const int K = p.K, M = p.M;
    const int nchunks = (K + 63) >> 6;
    // first weight row of the fragment's upper and lower eight
    const int row_a = GATED ? blockIdx.x * 8 : blockIdx.x * 16;
    const int row_b = GATED ? p.e.width + blockIdx.x * 8 : row_a + 8;
    auto offset = [&](int row) -> size_t {  // of the row's first byte; eight rows of a packed block
        if constexpr (PACKED)
            return (static_cast<size_t>(row >> 4) * nchunks * 2 + ((row >> 3) & 1)) * (kStBlock / 2);
        else
            return static_cast<size_t>(row) * K;
    };
    const uint8_t *w_a = p.w + offset(row_a) + (PACKED ? 16 * lane : static_cast<size_t>(g) * K + 16 * t4);
    // (one pointer a lane and a uniform distance: a second pointer spills)
    const size_t apart = PACKED && !GATED ? kStBlock / 2 : offset(row_b) - offset(row_a);
    constexpr int kStep = PACKED ? kStBlock : 64;  // bytes to the next chunk
    const char *xbase = static_cast<const char *>(p.x);

    float acc[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[nt][r] = 0.0f;

    for (int c0 = warp; c0 < nchunks; c0 += kStWarps * UNROLL) {
        uint4 wa[UNROLL], wb[UNROLL];
        uint32_t xw[UNROLL][NT][kXWords];
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            const int c = c0 + u * kStWarps;
            const int kk = c * 64 + 16 * t4;  // first k of this lane's 16
            const bool kin = (c < nchunks) && (kk < K);
            wa[u] = kin ? ld_stream16(w_a + static_cast<size_t>(c) * kStep) : make_uint4(0, 0, 0, 0);
            wb[u] = kin ? ld_stream16(w_a + apart + static_cast<size_t>(c) * kStep) : make_uint4(0, 0, 0, 0);
            // everything but the weights may come from the preceding kernel
            if (u == 0 && c0 == warp) pdl_wait();
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int m = m0 + g + 8 * nt;
                const bool in = kin && (m < M);
                const uint4 *xp = reinterpret_cast<const uint4 *>(
                    xbase + (static_cast<size_t>(m) * K + kk) * kXBytes);
#pragma unroll
                for (int v = 0; v < kXWords / 4; ++v) {
                    const uint4 t = in ? ld_act16(xp + v) : make_uint4(0, 0, 0, 0);
                    xw[u][nt][4 * v + 0] = t.x;
                    xw[u][nt][4 * v + 1] = t.y;
                    xw[u][nt][4 * v + 2] = t.z;
                    xw[u][nt][4 * v + 3] = t.w;
                }
            }
        }
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            const uint32_t ra[4] = {wa[u].x, wa[u].y, wa[u].z, wa[u].w};
            const uint32_t rb[4] = {wb[u].x, wb[u].y, wb[u].z, wb[u].w};
            if constexpr (XDT == FP8L_E4M3) {
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        mma_e4m3(acc[nt], ra[2 * j], rb[2 * j], ra[2 * j + 1], rb[2 * j + 1],
                                 xw[u][nt][2 * j], xw[u][nt][2 * j + 1]);
            } else {
                // step j: bytes 4j, 4j+1 are the low-k slots, 4j+2, 4j+3 the high-k ones
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t a0, a1, a2, a3;
                    st_decode(ra[j], a0, a2);
                    st_decode(rb[j], a1, a3);
                    if constexpr (XDT == FP8L_BF16) {
                        a0 = st_to_bf16(a0);
                        a1 = st_to_bf16(a1);
                        a2 = st_to_bf16(a2);
                        a3 = st_to_bf16(a3);
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        st_mma16<XDT>(acc[nt], a0, a1, a2, a3, xw[u][nt][2 * j], xw[u][nt][2 * j + 1]);
                }
            }
        }
    }

    pdl_wait();  // (warps that had no chunk)
    // one output a thread: (token, channel), channel fastest
    constexpr int kCh = GATED ? 8 : 16;
    static_assert(kCh * 8 * NT <= kStWarps * 32, "an output a thread");
    const int ch = threadIdx.x % kCh, tk = threadIdx.x / kCh;
    const int m = m0 + tk;
    const bool mine = threadIdx.x < kCh * 8 * NT && m < M;
    const int n = blockIdx.x * kCh + ch;
    const size_t yi = static_cast<size_t>(m) * p.e.width + n;
    float sc = 0.0f, bias = 0.0f, sc_up = 0.0f, bias_up = 0.0f, res = 0.0f;
    if (mine) {
        const float sa = XDT == FP8L_E4M3 ? ld_act_f32(p.a_scale + (p.a_per_token ? m : 0)) : 1.0f;
        sc = sa * epi_ld_f32(p.w_scale + (p.w_per_channel ? n : 0));
        bias = epi_bias(p.e, n);
        if constexpr (GATED) {
            sc_up = sa * epi_ld_f32(p.w_scale + (p.w_per_channel ? p.e.width + n : 0));
            bias_up = epi_bias(p.e, p.e.width + n);
        }
        if (p.e.residual != nullptr) res = epi_ld_16(p.e.residual, yi, p.e.out_dtype);
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int r = 0; r < 4; ++r) red[warp][nt][r][lane] = acc[nt][r];
    __syncthreads();
    if (!mine) return;
    const int nt = tk >> 3, col = tk & 7;
    const int lane_src = ((ch & 7) << 2) | (col >> 1);
    auto sum_of = [&](int upper) {
        const int r = (upper << 1) | (col & 1);
        float sum = 0.0f;
#pragma unroll
        for (int wi = 0; wi < kStWarps; ++wi) sum += red[wi][nt][r][lane_src];
        return sum;
    };
    float v[1] = {fmaf(sum_of(GATED ? 0 : ch >> 3), sc, bias)};
    activate(v, p.e.act);
    if constexpr (GATED) v[0] *= fmaf(sum_of(1), sc_up, bias_up);
    v[0] += res;
    if (p.e.out_dtype == FP8L_F16)
        static_cast<__half *>(p.e.y)[yi] = __float2half_rn(v[0]);
    else if (p.e.out_dtype == FP8L_BF16)
        static_cast<__nv_bfloat16 *>(p.e.y)[yi] = __float2bfloat16_rn(v[0]);
    else
        static_cast<uint8_t *>(p.e.y)[yi] = static_cast<uint8_t>(
            __nv_cvt_float_to_fp8(__fdiv_rn(v[0], ld_act_f32(p.e.out_scale)), __NV_SATFINITE, __NV_E4M3));
}

// Chunks a warp loads before it computes: four where 64 registers hold them
// (one token tile of codes, or of packed weights without a gate), else two
// (four spilled with a gate: 22016 x 4096 28.1 us, three 23.6,
// against 19.0).
template <int XDT, int NT, bool PACKED, bool GATED>
int launch_stream(const StreamArgs &p, bool stable, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.N / 16), static_cast<unsigned>((p.M + 15) / 16), 1);
    cfg.blockDim = dim3(kStWarps * 32, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = stable ? 1 : 0;
    constexpr int unroll = NT == 1 && ((PACKED && !GATED) || XDT == FP8L_E4M3) ? 4 : 2;
    if (cudaLaunchKernelEx(&cfg, linear_stream_kernel<XDT, NT, unroll, PACKED, GATED>, p) != cudaSuccess)
        return FP8L_ECUDA;
    return launch_status();
}

template <int XDT, bool PACKED>
int dispatch_stream(const StreamArgs &p, const LinearCall &c) {
    const bool two = c.M > 8;
    if (c.gated)
        return two ? launch_stream<XDT, 2, PACKED, true>(p, c.stable, c.stream)
                   : launch_stream<XDT, 1, PACKED, true>(p, c.stable, c.stream);
    return two ? launch_stream<XDT, 2, PACKED, false>(p, c.stable, c.stream)
               : launch_stream<XDT, 1, PACKED, false>(p, c.stable, c.stream);
}

}  // namespace

int launch_linear_stream(const LinearCall &c) {
    if (c.M > kLinearStreamTokens) return FP8L_ESHAPE;
    const StreamArgs p{c.w, c.x, c.M, c.N, c.K, c.a_scale, c.a_per_token, c.w_scale, c.w_per_channel, c.e};
    if (c.x_dtype == FP8L_E4M3) return dispatch_stream<FP8L_E4M3, false>(p, c);
    if (c.x_dtype == FP8L_BF16)
        return c.packed ? dispatch_stream<FP8L_BF16, true>(p, c) : dispatch_stream<FP8L_BF16, false>(p, c);
    return c.packed ? dispatch_stream<FP8L_F16, true>(p, c) : dispatch_stream<FP8L_F16, false>(p, c);
}

}  // namespace fp8l
