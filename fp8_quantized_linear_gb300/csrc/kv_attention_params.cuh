// What the attention kernels share: arguments, bounded waits, barriers,
// tensor-memory moves, MMA issue, output steps.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kv_device.cuh"
#include "quant_device.cuh"
#include "tc_device.cuh"

namespace fp8l {

struct AttnParams {
    const uint16_t *q;
    int tokens;
    int64_t q_stride;
    int q_heads, kv_heads;
    const uint8_t *k_cache, *v_cache;
    const float *k_scale, *v_scale;
    int num_pages, page_shift;
    const int32_t *block_table;
    int table_width;
    const int32_t *q_offsets, *kv_lens;
    int requests;
    float score_scale;  // sm_scale * log2(e)
    int window;
    const float *out_scale;
    void *out;
    int out_dtype;
    float *lse;
    int stages;
    float *partials;
    unsigned *counters, *status;
    unsigned *library_status;  // a call that gave up is recorded here too
    long long wait_cycles;
    unsigned stall;
};

namespace {

// ---------------------------------------------------------------- waits, barriers, tensor memory, MMAs

// A wait for the phase of parity `parity` without a call (a register split
// between warpgroups does not allow one).  Warps that wait share issue slots
// with the ones that work, so a failed try sleeps before the next.
template <int SLEEP = 20>
__device__ __forceinline__ bool kv_wait(uint32_t bar, uint32_t parity, volatile int *abort_flag, unsigned *status,
                                        long long limit) {
    if (mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
#pragma unroll 1
    while (!mbar_try_wait(bar, parity)) {
        if (*abort_flag) return false;
        if (clock64() - t0 > limit) {
            *abort_flag = 1;
            atomicOr(status, kStatusTimeout);
            return false;
        }
        if (SLEEP > 0) __nanosleep(SLEEP);
    }
    return true;
}

// A wait that ignores the abort flag, while tearing down
__device__ __forceinline__ void kv_drain(uint32_t bar, uint32_t parity, unsigned *status) {
    const long long t0 = clock64();
#pragma unroll 1
    while (!mbar_try_wait(bar, parity)) {
        if (clock64() - t0 > kDefaultWaitCycles) {
            atomicOr(status, kStatusTimeout);
            return;
        }
    }
}

// At the end of a block: a wait that gave up in it also goes to the library's
// word.  The workspace of a captured call belongs to its graph, where no
// status read looks and every replay clears it.
__device__ __forceinline__ void kv_report(const volatile int *abort_flag, unsigned *library_status) {
    if (threadIdx.x == 0 && *abort_flag) atomicOr(library_status, kStatusTimeout);
}

// One lane of the (converged) warp, always the same
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xFFFFFFFF;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r));
    return r != 0u;
}

// Barrier `id` over `threads` threads of the block
__device__ __forceinline__ void wide_sync(int id, int threads) {
    asm volatile("barrier.cta.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// The same, with whether any of them says so
__device__ __forceinline__ bool wide_any(int id, int threads, bool x) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, %2, %3, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(x ? 1u : 0u), "r"(id), "r"(threads)
        : "memory");
    return r != 0u;
}

// Those of a group of four warps
__device__ __forceinline__ void group_sync(int id) { wide_sync(id, 128); }
__device__ __forceinline__ bool group_any(int id, bool x) { return wide_any(id, 128, x); }

__device__ __forceinline__ void bulk_copy(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
        "l"(src), "r"(bytes), "r"(bar)
        : "memory");
}

// Operand descriptors as two words: the address moves only in the low one,
// so a step along an operand is one addition (a single thread issues every
// MMA, and its instructions are the critical path).
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lbo) {
    return ((addr & 0x3FFFFu) >> 4) | ((lbo >> 4) << 16);
}
constexpr uint32_t desc_hi(uint32_t sbo) { return (sbo >> 4) | (1u << 14); }

// D (tensor memory) = or += A B^T, both operands in shared memory, fp8
__device__ __forceinline__ void mma_f8_desc(uint32_t d_tmem, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo,
                                            uint32_t b_hi, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "mov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %4};\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %5, p;\n\t}" ::"r"(d_tmem),
        "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
        : "r"(taddr));
}

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
        : "memory");
}

__device__ __forceinline__ void tmem_ld16_nowait(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

__device__ __forceinline__ void tmem_st16_nowait(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
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

__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A block's scale of values as the softmax takes it, by its logarithm and its
// reciprocal: a smaller one (0 too, of a block of zeros not written here)
// counts as the smallest.  (__log2f is within 3 units in the last place, 2^-20
// for scales around 0.01 and 2^-16 for the smallest: so much do a page's weights
// and the log-sum-exp stray.)
__device__ __forceinline__ float value_scale(float s) { return s < kKvMinScale ? kKvMinScale : s; }

// Exponent e with 2^7 <= m 2^e < 2^8, at most 120 (rows below 2^-113 lose
// their last bits) so that 2^-e stays a normal float32; m >= 0
__device__ __forceinline__ int part_exponent(float m) {
    return min(134 - static_cast<int>(__float_as_uint(m) >> 23), 120);
}

// The factor of a row's scores, score_scale 2^-e; NaN when an element is not
// finite (the parts of an infinity would be numbers)
__device__ __forceinline__ float part_factor(float score_scale, float m, int e) {
    return m < INFINITY ? score_scale * __uint_as_float(static_cast<uint32_t>(127 - e) << 23) : NAN;
}

// ---------------------------------------------------------------- the line of tiles

// A line of `total` tiles cut into `pieces` (below 2^15): piece c begins at
// floor(total c / pieces), without a 64-bit product.
__device__ __forceinline__ long long piece_begin(long long total, long long c, long long pieces) {
    const long long each = total / pieces;
    const unsigned rest = static_cast<unsigned>(total - each * pieces);
    return each * c + rest * static_cast<unsigned>(c) / static_cast<unsigned>(pieces);
}

// The piece that tile `at` is in
__device__ __forceinline__ int piece_of(long long total, long long at, long long pieces) {
    return static_cast<int>(((at + 1) * pieces - 1) / total);
}

// ---------------------------------------------------------------- outputs

constexpr float kLn2 = 0.693147180559945309f;

// A row's sum l is 0 only when it sees no key (out 0, lse -inf); a NaN that it
// met stays in l, and the row comes out as NaN, not as a row without keys.

// E4M3 codes of four outputs; the code of a NaN is NaN (the saturating
// quotient would clamp it to a number)
__device__ __forceinline__ uint32_t attn_codes4(const float *o, const Quot &d) {
    uint32_t c = codes_of_word<FP8L_F32, true>(make_uint4(__float_as_uint(o[0]), __float_as_uint(o[1]),
                                                         __float_as_uint(o[2]), __float_as_uint(o[3])), d).x;
    if (__isnanf(o[0]) || __isnanf(o[1]) || __isnanf(o[2]) || __isnanf(o[3])) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (__isnanf(o[i])) c |= 0x7Fu << (8 * i);
    }
    return c;
}

// VALS (4 or 8) consecutive outputs of a row from dimension d on
template <int VALS>
__device__ __forceinline__ void attn_store(const AttnParams &p, int token, int head, int dim, int d,
                                           const float (&o)[VALS]) {
    static_assert(VALS == 4 || VALS == 8, "whole words of codes, at most one 16-byte store");
    const int64_t at = (static_cast<int64_t>(token) * p.q_heads + head) * dim + d;
    if (p.out_dtype == FP8L_E4M3) {
        const Quot s = Quot::make<FP8L_F32>(p.out_scale[0]);
        uint8_t *y = static_cast<uint8_t *>(p.out) + at;
#pragma unroll
        for (int i = 0; i < VALS; i += 4) *reinterpret_cast<uint32_t *>(y + i) = attn_codes4(&o[i], s);
    } else {
        uint16_t *y = static_cast<uint16_t *>(p.out) + at;
        uint32_t w[VALS / 2];
#pragma unroll
        for (int i = 0; i < VALS / 2; ++i) w[i] = pack_out16(o[2 * i], o[2 * i + 1], p.out_dtype);
        if constexpr (VALS == 4)
            *reinterpret_cast<uint2 *>(y) = make_uint2(w[0], w[1]);
        else
            *reinterpret_cast<uint4 *>(y) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// lse from the reference m (base 2) and the sum l = sum 2^(s - m)
__device__ __forceinline__ void attn_store_lse(const AttnParams &p, int token, int head, float m, float l) {
    p.lse[static_cast<int64_t>(token) * p.q_heads + head] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
}

}  // namespace
}  // namespace fp8l
