// Block table and slot map of a step, built on the GPU from the requests'
// lengths (fp8_kv_plan).
//
// Per request r with kv cached and q new tokens, P tokens a page:
//   off_r  = sum of q before r (cut at the step's T rows), q' = q within T
//   old    = ceil(kv / P),  need = max(0, min(ceil((kv + q') / P), W) - old)
//   base_r = sum of need before r;  got = clamp(F - base_r, 0, need)
// and a token's page is block_table[r][b] for an old block b, or
// free_pages[base_r + b - old] for a new one, so no token waits for another
// block's table entry.
//
// The work is a few kilobytes: what bounds it is the chain launch -> lengths
// -> two prefix sums -> search -> store.  So every block forms both prefix
// sums itself (two block scans of 512 requests a round, in shared memory)
// instead of meeting the others at a grid barrier or in a second launch, and
// takes its share of the rows and of the new table entries, each found in
// the prefix sums by bisection in shared memory.
//
// Measured (GB300, replayed from a graph): 3.0-3.3 us for 64 requests of one new
// token, 7.7 us for 1021 requests with 25085 (two rounds of scans, 13 blocks);
// an empty launch takes 2 us.
#include "kv_device.cuh"

namespace fp8l {
namespace {

constexpr int kPlanThreads = 512;
constexpr int kPlanRowsPerBlock = 4 * kPlanThreads;

struct PlanParams {
    const int32_t *q_lens, *kv_lens;
    int requests, tokens, page_shift;
    int32_t *block_table;
    int table_width;
    const int32_t *free_pages;
    int num_free;
    int32_t *q_offsets, *kv_lens_out, *positions, *slots, *used;
};

// Blocks of n tokens (n + P - 1 may not fit an int)
__device__ __forceinline__ int blocks_of(int n, int page_shift) {
    return (n >> page_shift) + ((n & ((1 << page_shift) - 1)) != 0 ? 1 : 0);
}

// Exclusive prefix sum over the block of one value per thread, plus `carry`;
// carry grows by the block's total.
__device__ __forceinline__ int block_scan(int v, int &carry, int *red) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int n = __shfl_up_sync(0xFFFFFFFFu, inc, o);
        if (lane >= o) inc += n;
    }
    if (lane == 31) red[warp] = inc;
    __syncthreads();
    int before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kPlanThreads / 32; ++w) {
        const int n = red[w];
        if (w < warp) before += n;
        total += n;
    }
    __syncthreads();
    const int out = carry + before + inc - v;
    carry += total;
    return out;
}

// Largest r in [0, n) with start[r] <= x (start non-decreasing, start[0] <= x)
__device__ __forceinline__ int last_not_above(const int *start, int n, int x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (start[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kPlanThreads) kv_plan_kernel(const PlanParams p) {
    extern __shared__ int plan_smem[];
    __shared__ int red[kPlanThreads / 32];
    int *off = plan_smem;                        // [requests] first row
    int *base = plan_smem + p.requests;          // [requests] new blocks before
    int *cached = plan_smem + 2 * p.requests;    // [requests] tokens before the step
    const int P = 1 << p.page_shift, R = p.requests, T = p.tokens;
    grid_dependency_sync();

    int rows = 0, blocks = 0, lost = 0;
    for (int r0 = 0; r0 < R; r0 += kPlanThreads) {
        const int r = r0 + static_cast<int>(threadIdx.x);
        const bool mine = r < R;
        const int kv = mine ? max(p.kv_lens[r], 0) : 0;
        const int q = mine ? max(p.q_lens[r], 0) : 0;
        const int at = min(block_scan(q, rows, red), T);
        const int total = kv + min(q, T - at);
        const int old = blocks_of(kv, p.page_shift);
        const int need = max(min(blocks_of(total, p.page_shift), p.table_width) - old, 0);
        const int b = block_scan(need, blocks, red);
        if (mine) {
            off[r] = at;
            base[r] = b;
            cached[r] = kv;
            const int got = min(max(p.num_free - b, 0), need);
            const int after = static_cast<int>(
                min(static_cast<int64_t>(total), static_cast<int64_t>(old + got) << p.page_shift));
            lost += total - after;
            if (blockIdx.x == 0) {
                p.q_offsets[r] = at;
                p.kv_lens_out[r] = after;
            }
        }
    }
    rows = min(rows, T);
    if (blockIdx.x == 0) {
        int all = 0;
        block_scan(lost, all, red);
        if (threadIdx.x == 0) {
            p.q_offsets[R] = rows;
            p.used[0] = min(blocks, p.num_free);
            p.used[1] = all;
        }
    }
    __syncthreads();

    const int stride = static_cast<int>(gridDim.x) * kPlanThreads;
    const int first = static_cast<int>(blockIdx.x) * kPlanThreads + static_cast<int>(threadIdx.x);
    for (int k = first; k < blocks; k += stride) {
        const int r = last_not_above(base, R, k);
        const int old = blocks_of(cached[r], p.page_shift);
        p.block_table[static_cast<int64_t>(r) * p.table_width + old + (k - base[r])] =
            k < p.num_free ? p.free_pages[k] : -1;
    }
    for (int64_t t64 = first; t64 < T; t64 += stride) {
        const int t = static_cast<int>(t64);
        int pos = 0, slot = -1;
        if (t < rows) {
            const int r = last_not_above(off, R, t);
            const int kv = cached[r];
            pos = kv + t - off[r];
            const int b = pos >> p.page_shift, old = blocks_of(kv, p.page_shift);
            int page = -1;
            if (b < p.table_width) {
                if (b < old) {
                    page = p.block_table[static_cast<int64_t>(r) * p.table_width + b];
                } else {
                    const int k = base[r] + b - old;
                    if (k < p.num_free) page = p.free_pages[k];
                }
            }
            if (page >= 0) slot = (page << p.page_shift) + (pos & (P - 1));
        }
        p.positions[t] = pos;
        p.slots[t] = slot;
    }
}

// An int32 array of the call
struct Span {
    const int32_t *at;
    int64_t n;
    bool meets(const Span &o) const {
        const uintptr_t a = reinterpret_cast<uintptr_t>(at), b = reinterpret_cast<uintptr_t>(o.at);
        return n > 0 && o.n > 0 && a < b + 4 * static_cast<uintptr_t>(o.n) && b < a + 4 * static_cast<uintptr_t>(n);
    }
};

}  // namespace
}  // namespace fp8l

extern "C" int fp8_kv_plan(const int32_t *q_lens, const int32_t *kv_lens, int64_t requests, int64_t tokens,
                           int64_t page_size, int32_t *block_table, int64_t table_width,
                           const int32_t *free_pages, int64_t num_free, int32_t *q_offsets,
                           int32_t *kv_lens_out, int32_t *positions, int32_t *slots, int32_t *used,
                           void *stream) {
    using namespace fp8l;
    if (requests < 1 || requests > kKvMaxRequests || tokens < 0 || tokens > INT32_MAX ||
        !kv_page_size_ok(page_size) || table_width < 1 || table_width > INT32_MAX || num_free < 0 ||
        num_free > INT32_MAX / page_size)
        return FP8L_ESHAPE;
    if (!q_lens || !kv_lens || !block_table || (!free_pages && num_free > 0) || !q_offsets || !kv_lens_out ||
        ((!positions || !slots) && tokens > 0) || !used)
        return FP8L_EINVAL;
    for (const void *ptr : {static_cast<const void *>(q_lens), static_cast<const void *>(kv_lens),
                            static_cast<const void *>(block_table), static_cast<const void *>(free_pages),
                            static_cast<const void *>(q_offsets), static_cast<const void *>(kv_lens_out),
                            static_cast<const void *>(positions), static_cast<const void *>(slots),
                            static_cast<const void *>(used)})
        if (!aligned4(ptr)) return FP8L_EALIGN;
    // Every block reads all inputs while others write outputs, so none may
    // share memory; only the lengths may be updated in place (below).
    const bool in_place = kv_lens_out == kv_lens;
    const Span inputs[3] = {{q_lens, requests}, {free_pages, num_free}, {kv_lens, requests}};
    const Span outputs[6] = {{block_table, requests * table_width}, {q_offsets, requests + 1}, {positions, tokens},
                             {slots, tokens}, {used, 2}, {kv_lens_out, requests}};
    for (int i = 0; i < 6; ++i) {
        for (int j = 0; j < 3; ++j)
            if (!(in_place && i == 5 && j == 2) && outputs[i].meets(inputs[j])) return FP8L_EINVAL;
        for (int j = 0; j < i; ++j)
            if (outputs[i].meets(outputs[j])) return FP8L_EINVAL;
    }
    int sms = 0;
    if (int st = check_device(&sms); st != FP8L_OK) return st;
    PlanParams p;
    p.q_lens = q_lens;
    p.kv_lens = kv_lens;
    p.requests = static_cast<int>(requests);
    p.tokens = static_cast<int>(tokens);
    p.page_shift = __builtin_ctzll(static_cast<unsigned long long>(page_size));
    p.block_table = block_table;
    p.table_width = static_cast<int>(table_width);
    p.free_pages = free_pages;
    p.num_free = static_cast<int>(num_free);
    p.q_offsets = q_offsets;
    p.kv_lens_out = kv_lens_out;
    p.positions = positions;
    p.slots = slots;
    p.used = used;
    // up to 96 KB of prefix sums (8192 requests)
    const size_t smem = 3 * sizeof(int) * static_cast<size_t>(requests);
    static std::atomic<unsigned long long> ready{0};
    if (smem > 47 * 1024)
        if (int st = allow_smem(kv_plan_kernel, 3 * sizeof(int) * kKvMaxRequests, ready, false); st != FP8L_OK)
            return st;
    // In place, one block: each thread reads a request's length before it writes
    // it, and nobody else reads it.  Measured (us, apart / in place): 64 decoding
    // 3.0 / 3.0, 12 requests with 19927 rows 4.2 / 16.9, 1021 with 24699 7.6 / 47
    const int64_t want = in_place ? 1 : (tokens + kPlanRowsPerBlock - 1) / kPlanRowsPerBlock;
    const unsigned grid = static_cast<unsigned>(want < 1 ? 1 : (want > sms ? sms : want));
    return launch_dependent(kv_plan_kernel, dim3(grid), kPlanThreads, smem, as_stream(stream), p);
}
