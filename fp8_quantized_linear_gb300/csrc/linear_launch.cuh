// What the linear products' launchers share (linear.cu and the kernels'
// translation units).
#pragma once

#include "epilogue.cuh"

namespace fp8l {

// One product with its epilogue; every pointer checked.
struct LinearCall {
    const void *x;  // [M, K] E4M3 codes, or 16-bit activations (x_dtype)
    int x_dtype;
    const uint8_t *w;  // [N, K] codes, or their packed layout
    int packed;
    int M, N, K;
    int gated;
    const float *a_scale;  // E4M3 x: [1], or [M] per token
    int a_per_token;
    const float *w_scale;  // [1] or [N]
    int w_per_channel;
    Epilogue e;
    unsigned *status;
    int sms;
    bool stable;
    cudaStream_t stream;
};

// 2-D or higher TMA map over bytes with the 64-byte swizzle (api.cu).
int make_swizzle64_map(CUtensorMap *map, const void *ptr, int rank, const uint64_t *dims,
                       const uint64_t *strides, const uint32_t *box);

// Swapped operands: weight rows on the MMA's M side, tokens on its N side.
// parts: E4M3 numbers a token value is held in (1: the codes themselves).
int launch_linear_swapped(const LinearCall &c, int parts, const float *token_scale);

// Weights streamed through registers, up to 16 tokens a CTA: as many tokens as
// the grid's second dimension holds.
constexpr int64_t kLinearStreamTokens = 65535 * 16;
int launch_linear_stream(const LinearCall &c);

// 256-token by 256-row tiles over pairs of SMs (E4M3 tokens, row-major weights).
int launch_linear_pair(const LinearCall &c);

// 16-bit tokens as sums of E4M3 parts: bytes of the scratch that
// linear_split_tokens fills and launch_linear_swapped reads.
int linear_parts(int x_dtype);
bool linear_parts_fit(int x_dtype, int64_t M, int64_t N);  // tensor map and grid count that many
size_t linear_parts_bytes(int x_dtype, int64_t M, int64_t K);
int linear_split_tokens(const LinearCall &c, void *scratch, const float **token_scale);

}  // namespace fp8l
