// fp8_glu.h -- what the kernels of the gated feed-forward's product share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "block_internal.h"
#include "fp8_act.h"
#include "fp8_internal.h"
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

constexpr int kGluStage = 2048;                                    // LDS that a wave's outputs go through
constexpr int glu_bytes(int tokens) { return 3 * tokens * 4; }     // exponents [y, g, u][token][wave]

// The outputs of kR row tiles from kI0 on, kR * 16 tokens of a wave: acc[i][j], j < 2, are the sums of 16 channels' gates
// (lane: token l % 16, channels 4 (l / 16) .. +4), j + 2 those of their partners.  The tile's first token and channel are m0
// and n0 (N and n0 multiples of 128); the wave's tokens begin at `row` of the tile, its 32 channels at 32 wn: four waves make
// a group, and all waves of the workgroup come here.  Codes take the largest magnitudes of 32 channels each, whose exponents
// the four waves exchange as bytes (the scale's exponent is monotone in the magnitude).  stage: the wave's kGluStage bytes of
// LDS, so that stores write runs of 32 bytes of a token's codes (of 128 with the other waves'); bytes: glu_bytes of LDS.
template <int kR, int kI0, bool kE8M0, int TM>
__device__ __forceinline__ void glu_outputs(const GluParams& p, const v4f (&acc)[TM][4], int64_t m0, int row, int n0, int wn, int tid,
                                            uint8_t* stage, uint8_t* bytes, int tokens) {
    static_assert(kR == 2 || kR == 4, "row tiles");
    const int lane = tid & 63, g = lane >> 4, l15 = lane & 15;
    const GluOut& o = p.out;
    const int64_t cm0 = m0 + row + kI0 * 16;
    const int cn0 = n0 + wn * 32;
    float y[kR][8];
    for_act(o.act, [&](auto act) {
#pragma unroll
        for (int i = 0; i < kR; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) y[i][e] = act_value<decltype(act)::value>(acc[kI0 + i][e / 4][e % 4]) * acc[kI0 + i][2 + e / 4][e % 4];
    });
    if (o.y != nullptr) {
        if (o.y_bf16) {   // two row tiles at a time, 64 bytes a token; chunk c of row r at c ^ (r & 3)
#pragma unroll
            for (int h = 0; h < kR / 2; ++h) {
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float* v = y[2 * h + i] + 4 * j;
                        *reinterpret_cast<uint2*>(stage + (16 * i + l15) * 64 + (((2 * j + (g >> 1)) ^ (l15 & 3)) << 4) + (g & 1) * 8) =
                            uint2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
                    }
                lds_done();
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const int at = 16 * q + (lane >> 2), c = lane & 3;
                    const v4i x = *reinterpret_cast<const v4i*>(stage + at * 64 + ((c ^ (at & 3)) << 4));
                    const int64_t m = cm0 + 32 * h + at;
                    if (m < p.T) __builtin_nontemporal_store(x, reinterpret_cast<v4i*>(static_cast<uint16_t*>(o.y) + m * p.N + cn0 + 8 * c));
                }
                lds_done();
            }
        } else {
#pragma unroll
            for (int i = 0; i < kR; ++i) {
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    *reinterpret_cast<v4f*>(stage + l15 * 128 + (((4 * j + g) ^ (l15 & 7)) << 4)) = v4f{y[i][4 * j], y[i][4 * j + 1], y[i][4 * j + 2], y[i][4 * j + 3]};
                lds_done();
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const int at = 8 * q + (lane >> 3), c = lane & 7;
                    const v4f x = *reinterpret_cast<const v4f*>(stage + at * 128 + ((c ^ (at & 7)) << 4));
                    const int64_t m = cm0 + 16 * i + at;
                    if (m < p.T) __builtin_nontemporal_store(x, reinterpret_cast<v4f*>(static_cast<float*>(o.y) + m * p.N + cn0 + 4 * c));
                }
                lds_done();
            }
        }
    }
    const bool codes = o.y_codes != nullptr, keep = o.h_codes != nullptr;
    if (!codes && !keep) return;
    // exponents: of this wave's 32 channels, then of the group's 128
    const int row0 = row + kI0 * 16 + l15;
    auto value = [&](int kind, int i, int e) { return kind == 0 ? y[i][e] : acc[kI0 + i][(kind - 1) * 2 + e / 4][e % 4]; };
    auto put_byte = [&](auto kindc) {
        constexpr int kind = decltype(kindc)::value;
        float m[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < kR; ++i) {
#pragma unroll
            for (int e = 0; e < 8; ++e) m[i] = magnitude(m[i], value(kind, i, e));
        }
        if (max(max(m[0], m[1]), max(m[2], m[3])) == __builtin_inff()) {   // one branch for all: with one each their latencies add up
#pragma unroll
            for (int i = 0; i < kR; ++i) {
                m[i] = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float v = __builtin_fabsf(value(kind, i, e));
                    m[i] = v < __builtin_inff() ? max(m[i], v) : m[i];
                }
            }
        }
        const uint32_t mine = max_rows({__float_as_uint(m[0]), __float_as_uint(m[1]), __float_as_uint(m[2]), __float_as_uint(m[3])});
        if (g < kR) bytes[(kind * tokens + row0 + 16 * g) * 4 + wn] = static_cast<uint8_t>(exponent_byte(mine));
    };
    auto put_codes = [&](auto kindc, void* out, int64_t stride, int column, void* scale, int group) {
        constexpr int kind = decltype(kindc)::value;
#pragma unroll
        for (int i = 0; i < kR; ++i) {
            const uint32_t b = max_byte(reinterpret_cast<const uint32_t*>(bytes)[kind * tokens + row0 + 16 * i]);
            const float inv = byte_inverse(b);
#pragma unroll
            for (int j = 0; j < 2; ++j)
                *reinterpret_cast<uint32_t*>(stage + (16 * i + l15) * 32 + 16 * j + 4 * g) =
                    encode4<false>(value(kind, i, 4 * j) * inv, value(kind, i, 4 * j + 1) * inv, value(kind, i, 4 * j + 2) * inv, value(kind, i, 4 * j + 3) * inv);
            const int64_t m = cm0 + 16 * i + l15;
            if (wn == kind && g == i && m < p.T) store_scale(scale, kE8M0, group * p.T + m, byte_exponent(b));
        }
        lds_done();
#pragma unroll
        for (int q = 0; q < kR / 2; ++q) {
            const int at = 32 * q + (lane >> 1);
            const v4i x = *reinterpret_cast<const v4i*>(stage + at * 32 + (lane & 1) * 16);
            const int64_t m = cm0 + at;
            if (m < p.T) *reinterpret_cast<v4i*>(static_cast<uint8_t*>(out) + m * stride + column + (lane & 1) * 16) = x;
        }
        lds_done();
    };
    constexpr auto kY = std::integral_constant<int, 0>{};
    constexpr auto kG = std::integral_constant<int, 1>{};
    constexpr auto kU = std::integral_constant<int, 2>{};
    if (codes) put_byte(kY);
    if (keep) {
        put_byte(kG);
        put_byte(kU);
    }
    lds_done();
    barrier();
    if (codes) put_codes(kY, o.y_codes, p.N, cn0, o.y_scale, n0 / kFp8Block);
    if (keep) {
        put_codes(kG, o.h_codes, 2 * static_cast<int64_t>(p.N), cn0, o.h_scale, n0 / kFp8Block);
        put_codes(kU, o.h_codes, 2 * static_cast<int64_t>(p.N), p.N + cn0, o.h_scale, (p.N + n0) / kFp8Block);
    }
}

}  // namespace fp8

fp8::GluParams glu_params(const GluArgs& a);
// 256 tokens by 128 channels per workgroup; reductions of at least two blocks.
hipError_t launch_glu_large(const fp8::GluParams& p, bool e8m0, hipStream_t stream);
// At most 16 tokens.  sums: [T][2 N] fp32 receives [g u], or nullptr: y is written.
hipError_t launch_glu_small(fp8::GluParams p, bool e8m0, float* sums, hipStream_t stream);
// `tokens` (64 or 128) by 128 channels per workgroup.
hipError_t launch_glu_tile(const fp8::GluParams& p, bool e8m0, int tokens, hipStream_t stream);

}  // namespace rtq
