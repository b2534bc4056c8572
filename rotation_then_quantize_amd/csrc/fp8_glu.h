// fp8_glu.h -- what the kernels of the gated feed-forward's product share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "block_internal.h"
#include "fp8_act.h"
#include "fp8_tile.h"

namespace rtq {
namespace fp8 {

// The outputs of one or more channels' sums.
struct GluOut {
    int act;
    void* h_codes;   // [T][2 N], or nullptr
    void* h_scale;
    void* y;         // [T][N], or nullptr
    bool y_bf16;
    void* y_codes;   // [T][N], or nullptr
    void* y_scale;
};

// Kernel arguments of the product and its outputs.
struct GluParams {
    const uint8_t* x;        // [T][K]
    const void* x_scale;     // [blocks of K][T]
    const uint8_t* w;        // [2 N][K]
    const void* w_scale;     // [2 N / 128][blocks of K]
    int64_t T;
    int N, K;
    int tiles_t, tiles_n;    // of tokens and of channels
    GluOut out;
};

// f(integral_constant) for the activation, which is one of three.
template <typename F>
__device__ __forceinline__ void for_act(int act, F f) {
    if (act == RTQ_ACT_SILU)
        f(std::integral_constant<int, RTQ_ACT_SILU>{});
    else if (act == RTQ_ACT_GELU)
        f(std::integral_constant<int, RTQ_ACT_GELU>{});
    else
        f(std::integral_constant<int, RTQ_ACT_GELU_TANH>{});
}

// A group's scale exponent as a byte that orders like it, 0 for a group of zeros: the largest of several parts' bytes
// is the whole group's.
__device__ __forceinline__ uint32_t exponent_byte(uint32_t amax) { return amax == 0u ? 0u : static_cast<uint32_t>(scale_exponent<false>(amax) + 121); }
__device__ __forceinline__ int byte_exponent(uint32_t b) { return b == 0u ? 0 : static_cast<int>(b) - 121; }
// 2^-e of a byte's exponent; for zeros, whose codes do not depend on it, 2^121.
__device__ __forceinline__ float byte_inverse(uint32_t b) { return __uint_as_float((248u - b) << 23); }
// The largest of the four bytes of a word.
__device__ __forceinline__ uint32_t max_byte(uint32_t w) {
    return max(max(w & 0xffu, w >> 8 & 0xffu), max(w >> 16 & 0xffu, w >> 24));
}

// Bits of the largest magnitude of m and v: one instruction, whose median with infinity is the larger of two numbers, and
// where one of them is no number the other one.
__device__ __forceinline__ float magnitude(float m, float v) {
    return __builtin_amdgcn_fmed3f(m, __builtin_fabsf(v), __builtin_inff());
}

// m[i]'s maximum over the four 16-lane rows of a wave, in row i: two swaps of halves for four numbers, then one of rows.
__device__ __forceinline__ uint32_t max_rows(const uint32_t (&m)[4]) {
    const auto a = __builtin_amdgcn_permlane32_swap(m[0], m[2], false, false);
    const auto b = __builtin_amdgcn_permlane32_swap(m[1], m[3], false, false);
    const auto c = __builtin_amdgcn_permlane16_swap(max(a[0], a[1]), max(b[0], b[1]), false, false);
    return max(c[0], c[1]);
}

}  // namespace fp8

fp8::GluParams glu_params(const GluArgs& a);
// 256 tokens by 128 channels per workgroup; reductions of at least two blocks.
hipError_t launch_glu_large(const fp8::GluParams& p, bool e8m0, hipStream_t stream);

}  // namespace rtq
