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

// A group's scale as the bits of a float, which order like it: 2^-121 for a group of zeros, whose codes do not depend on it (it
// is 1).  The largest of several parts' bits is the whole group's.
constexpr uint32_t kZeros = 6u << 23;
__device__ __forceinline__ uint32_t scale_bits(uint32_t amax) { return amax == 0u ? kZeros : static_cast<uint32_t>(scale_exponent<false>(amax) + 127) << 23; }
__device__ __forceinline__ int bits_exponent(uint32_t b) { return b == kZeros ? 0 : static_cast<int>(b >> 23) - 127; }

// The largest magnitude of m, a and b in one instruction; of numbers that are none, the others'.  (From fmaxf the compiler makes
// it with an instruction more for each number.)  a and b must not come straight from a matrix instruction, for whose results
// the compiler does not wait here.
__device__ __forceinline__ float magnitude(float m, float a, float b) {
    float r;
    asm("v_max3_f32 %0, %1, |%2|, |%3|" : "=v"(r) : "v"(m), "v"(a), "v"(b));
    return r;
}

// m[i]'s maximum over the four 16-lane rows of a wave, in row i: two swaps of halves for four numbers, then one of rows.
__device__ __forceinline__ uint32_t max_rows(float m0, float m1, float m2, float m3) {
    const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(m0), __float_as_uint(m2), false, false);
    const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(m1), __float_as_uint(m3), false, false);
    const auto c = __builtin_amdgcn_permlane16_swap(max(a[0], a[1]), max(b[0], b[1]), false, false);
    return max(c[0], c[1]);
}

// Codes of four values by 2^e, as encode4 of the values times 2^-e.
typedef short v2s __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t encode4_by(const float* v, float scale) {
    v2s w = __builtin_bit_cast(v2s, v[0]);   // both halves are written: any register serves, without an instruction for it
    w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, v[0], v[1], scale, false);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, v[2], v[3], scale, true);
    return __builtin_bit_cast(uint32_t, w);
}

constexpr int kGluStep = 8192, kGluStage = 3 * kGluStep;           // LDS that outputs go through, in three buffers
constexpr int kGluSet = 3 * 64, kGluScales = 2 * kGluSet * 4;      // and the scales of two steps

struct GluLds {
    uint8_t* stage;     // [kGluStage]
    uint32_t* scales;   // [2][kGluSet], zeros at first
    int turn = 0;       // the buffer of the next values
    int set = 0;        // the scales of the next step
};

// The outputs of kR row tiles from kI0 on, kR * 16 tokens of a wave: acc[i][j], j < 2, are the sums of 16 channels' gates (lane:
// token l % 16, channels 4 (l / 16) .. +4), j + 2 those of their partners.  All 8 waves of the workgroup come here: wave (wm,
// wn) has kWaveRows tokens from kWaveRows wm on of the tile and 32 channels from 32 wn on of its 128, a group; m0 and n0 are the
// tile's first token and channel.  kKeep: with the checkpoint.
//
// Codes: the four waves of a group join the scales of their 32 channels in LDS (a scale is monotone in the magnitude), and the
// codes go through LDS to whole lines of a token's 128.  Two barriers for all kinds of codes; kR is as large as the LDS for them
// allows (4608 x 4096, 16384 channels with the checkpoint, fp32 scales outside the instruction: 593 us; the three kinds one
// after the other, of four row tiles, 611, half of the outputs' time then waits for LDS and barriers).
template <int kR, bool kKeep, int kI0, int kWaveRows, bool kE8M0, int TM>
__device__ __forceinline__ void glu_outputs(const GluParams& p, const v4f (&acc)[TM][4], int64_t m0, int n0, int wm, int wn, int tid,
                                            GluLds& lds) {
    constexpr int kTokens = 2 * kWaveRows, kKinds = kKeep ? 3 : 1, kStep = 32 * kR, kBuffer = kStep * kFp8Block;
    static_assert(kR == 1 || kR == 2 || kR == 4, "row tiles");
    static_assert(kKinds * kBuffer <= kGluStage && kKinds * kStep <= kGluSet, "a buffer and scales for each kind of codes");
    const int lane = tid & 63, g = lane >> 4, l15 = lane & 15;
    const GluOut& o = p.out;
    const int rows = static_cast<int>(min<int64_t>(kTokens, p.T - m0));   // of the tile: what a lane adds to its first is below 2^32
    float v[kKinds][kR][8];   // y, and g, u
#pragma unroll
    for (int i = 0; i < kR; ++i)
#pragma unroll
        for (int e = 0; kKeep && e < 8; ++e) {
            v[kKinds - 2][i][e] = acc[kI0 + i][e / 4][e % 4];
            v[kKinds - 1][i][e] = acc[kI0 + i][2 + e / 4][e % 4];
        }
    for_act(o.act, [&](auto act) {
#pragma unroll
        for (int i = 0; i < kR; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) v[0][i][e] = act_value<decltype(act)::value>(acc[kI0 + i][e / 4][e % 4]) * acc[kI0 + i][2 + e / 4][e % 4];
    });
    __builtin_amdgcn_sched_barrier(0);   // all sums have been read here, as magnitude() wants it
    // Values.  A step's rows in LDS: those of wave-row 0, then of 1; chunk c (16 bytes) of row r is at c ^ (r & 7).
    auto buffer = [&]() { return lds.stage + lds.turn * kGluStep; };
    auto next = [&]() { lds.turn = lds.turn == 2 ? 0 : lds.turn + 1; };
    auto handed = [&]() {   // what the waves wrote is in LDS, for every wave
        lds_done();
        barrier();
    };
    if (o.y != nullptr && o.y_bf16) {   // a row tile a step: 32 rows of 256 bytes
#pragma unroll
        for (int i = 0; i < kR; ++i) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float* y = v[0][i] + 4 * j;
                *reinterpret_cast<uint2*>(buffer() + (16 * wm + l15) * 256 + (((4 * wn + 2 * j + (g >> 1)) ^ (l15 & 7)) << 4) + (g & 1) * 8) =
                    uint2{pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3])};
            }
            handed();
            const int r = tid >> 4, c = tid & 15, line = (r >> 4) * kWaveRows + (kI0 + i) * 16 + (r & 15);
            const v4i x = *reinterpret_cast<const v4i*>(buffer() + r * 256 + ((c ^ (r & 7)) << 4));
            const uint32_t far = static_cast<uint32_t>(line) * static_cast<uint32_t>(p.N) + static_cast<uint32_t>(8 * c);
            if (line < rows) __builtin_nontemporal_store(x, reinterpret_cast<v4i*>(static_cast<uint16_t*>(o.y) + m0 * p.N + n0 + far));
            next();
        }
    } else if (o.y != nullptr) {   // half a row tile's rows of each wave-row a step: 16 rows of 512 bytes
#pragma unroll
        for (int i = 0; i < kR; ++i)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                if (l15 >> 3 == q) {
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        *reinterpret_cast<v4f*>(buffer() + (8 * wm + (l15 & 7)) * 512 + (((8 * wn + 4 * j + g) ^ (l15 & 7)) << 4)) =
                            v4f{v[0][i][4 * j], v[0][i][4 * j + 1], v[0][i][4 * j + 2], v[0][i][4 * j + 3]};
                }
                handed();
                const int r = tid >> 5, c = tid & 31, line = (r >> 3) * kWaveRows + (kI0 + i) * 16 + 8 * q + (r & 7);
                const v4f x = *reinterpret_cast<const v4f*>(buffer() + r * 512 + ((c ^ (r & 7)) << 4));
                const uint32_t far = static_cast<uint32_t>(line) * static_cast<uint32_t>(p.N) + static_cast<uint32_t>(4 * c);
                if (line < rows) __builtin_nontemporal_store(x, reinterpret_cast<v4f*>(static_cast<float*>(o.y) + m0 * p.N + n0 + far));
                next();
            }
    }
    const bool codes = o.y_codes != nullptr;
    if (!codes && !kKeep) return;
    // Scales of this wave's 32 channels, of four parts (a kind's row tile) at a time: lane row k has part k's.  Words: [kind][token of
    // the step].
    const int row0 = kWaveRows * wm + kI0 * 16 + l15;
    uint32_t* scales = lds.scales + lds.set * kGluSet;
    lds.set ^= 1;
    const int word0 = 16 * kR * wm + l15;
    auto largest = [&](const float* x) {
        float m = 0.f;
#pragma unroll
        for (int e = 0; e < 8; e += 2) m = magnitude(m, x[e], x[e + 1]);
        return m;
    };
    auto finite = [&](const float* x) {
        float m = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) m = __builtin_fabsf(x[e]) < __builtin_inff() ? max(m, __builtin_fabsf(x[e])) : m;
        return m;
    };
    auto put_scales = [&](const float* x0, const float* x1, const float* x2, const float* x3, int kind, bool some) {
        float m0 = largest(x0), m1 = largest(x1), m2 = largest(x2), m3 = largest(x3);
        if (max(max(m0, m1), max(m2, m3)) == __builtin_inff()) m0 = finite(x0), m1 = finite(x1), m2 = finite(x2), m3 = finite(x3);
        const uint32_t mine = max_rows(m0, m1, m2, m3);
        if (some) __hip_atomic_fetch_max(scales + (kind + g / kR) * kStep + word0 + 16 * (g % kR), scale_bits(mine), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
    };
    if constexpr (kR == 1) {
        put_scales(v[0][0], v[kKeep ? 1 : 0][0], v[kKinds - 1][0], v[0][0], 0, g < kKinds && (g > 0 || codes));
    } else {
        if (codes) put_scales(v[0][0], v[0][1], v[0][kR - 2], v[0][kR - 1], 0, g < kR);
        if constexpr (kKeep) put_scales(v[1][0], v[1][1], v[2][0], v[2][1], 1, true);
    }
    handed();
    // Codes: a buffer for each kind, 32 kR rows of 128 bytes.  All scales are read first: behind a write to LDS the compiler
    // would hold the next read back until it has been done.
    uint32_t top[kKinds][kR];
#pragma unroll
    for (int kind = 0; kind < kKinds; ++kind)
#pragma unroll
        for (int i = 0; i < kR; ++i) top[kind][i] = scales[kind * kStep + word0 + 16 * i];
    uint8_t* mine = lds.stage + word0 * 128 + 4 * g;
    const int place[2] = {(2 * wn ^ (l15 & 7)) << 4, ((2 * wn + 1) ^ (l15 & 7)) << 4};
    auto put_codes = [&](auto kindc, void* scale, int group) {
        constexpr int kind = decltype(kindc)::value;
        uint32_t of_mine = 0u;   // lane row i's
#pragma unroll
        for (int i = 0; i < kR; ++i) {
            of_mine = g == i ? top[kind][i] : of_mine;
#pragma unroll
            for (int j = 0; j < 2; ++j)
                *reinterpret_cast<uint32_t*>(mine + kind * kBuffer + 16 * i * 128 + place[j]) = encode4_by(v[kind][i] + 4 * j, __uint_as_float(top[kind][i]));
        }
        if (wn == kind && g < kR && row0 + 16 * g < rows)
            store_scale(scale, kE8M0, group * p.T + m0 + row0 + 16 * g, bits_exponent(of_mine));
    };
    if (codes) put_codes(std::integral_constant<int, 0>{}, o.y_scale, n0 / kFp8Block);
    if constexpr (kKeep) {
        put_codes(std::integral_constant<int, kKinds - 2>{}, o.h_scale, n0 / kFp8Block);
        put_codes(std::integral_constant<int, kKinds - 1>{}, o.h_scale, (p.N + n0) / kFp8Block);
    }
    handed();
    if (tid < kKinds * kStep) scales[tid] = 0u;   // for the step after the next one, two barriers from here
#pragma unroll
    for (int q = 0; q < (kR + 1) / 2; ++q) {
        const int r = 64 * q + (tid >> 3), c = tid & 7, line = r / (16 * kR) * kWaveRows + kI0 * 16 + r % (16 * kR);   // of the tile
        const uint8_t* at = lds.stage + r * 128 + ((c ^ (r & 7)) << 4);
        v4i x[kKinds];
#pragma unroll
        for (int kind = 0; kind < kKinds; ++kind) x[kind] = *reinterpret_cast<const v4i*>(at + kind * kBuffer);
        // a tile's lines are at most 2^28 bytes apart
        const uint32_t far = static_cast<uint32_t>(line) * static_cast<uint32_t>(p.N) + static_cast<uint32_t>(16 * c);
        if (line < rows && (kR > 1 || r < kStep)) {
            if (codes) *reinterpret_cast<v4i*>(static_cast<uint8_t*>(o.y_codes) + m0 * p.N + n0 + far) = x[0];
            if constexpr (kKeep) {
                uint8_t* out = static_cast<uint8_t*>(o.h_codes) + m0 * 2 * p.N + n0;
                const uint32_t twice = 2 * far - static_cast<uint32_t>(16 * c);
                // past the caches, for the backward pass; y's codes are read next (this product with the checkpoint and the next one,
                // 4608 x 4096, 16384 channels: 863 us, h through the caches 893; without the checkpoint 831, y's past them 842)
                __builtin_nontemporal_store(x[kKinds - 2], reinterpret_cast<v4i*>(out + twice));
                __builtin_nontemporal_store(x[kKinds - 1], reinterpret_cast<v4i*>(out + p.N + twice));
            }
        }
    }
    lds_done();   // read before the next barrier, behind which codes are written again ...
    if (o.y != nullptr) barrier();   // ... and values at once
}

// All outputs of a tile.
template <int kWaveRows, bool kE8M0, int TM>
__device__ __forceinline__ void glu_tile_outputs(const GluParams& p, const v4f (&acc)[TM][4], int64_t m0, int n0, int wm, int wn, int tid,
                                                 GluLds& lds) {
    if constexpr (TM == 1) {
        if (p.out.h_codes != nullptr)
            glu_outputs<1, true, 0, kWaveRows, kE8M0>(p, acc, m0, n0, wm, wn, tid, lds);
        else
            glu_outputs<1, false, 0, kWaveRows, kE8M0>(p, acc, m0, n0, wm, wn, tid, lds);
    } else if (p.out.h_codes != nullptr) {
        glu_outputs<2, true, 0, kWaveRows, kE8M0>(p, acc, m0, n0, wm, wn, tid, lds);
        if constexpr (TM >= 4) glu_outputs<2, true, 2, kWaveRows, kE8M0>(p, acc, m0, n0, wm, wn, tid, lds);
        if constexpr (TM == 8) {
            glu_outputs<2, true, 4, kWaveRows, kE8M0>(p, acc, m0, n0, wm, wn, tid, lds);
            glu_outputs<2, true, 6, kWaveRows, kE8M0>(p, acc, m0, n0, wm, wn, tid, lds);
        }
    } else {
        glu_outputs<TM == 2 ? 2 : 4, false, 0, kWaveRows, kE8M0>(p, acc, m0, n0, wm, wn, tid, lds);
        if constexpr (TM == 8) glu_outputs<4, false, 4, kWaveRows, kE8M0>(p, acc, m0, n0, wm, wn, tid, lds);
    }
}

}  // namespace fp8

fp8::GluParams glu_params(const GluArgs& a);
// 256 tokens by 128 channels per workgroup; reductions of at least two blocks.
hipError_t launch_glu_large(const fp8::GluParams& p, bool e8m0, hipStream_t stream);
// At most 32 tokens.  sums: [T][2 N] fp32 receives [g u], or nullptr: y is written.
hipError_t launch_glu_small(fp8::GluParams p, bool e8m0, float* sums, hipStream_t stream);
// `tokens` (32, 64 or 128) by 128 channels per workgroup.
hipError_t launch_glu_tile(const fp8::GluParams& p, bool e8m0, int tokens, hipStream_t stream);

}  // namespace rtq
