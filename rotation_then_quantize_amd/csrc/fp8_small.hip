// fp8_small.hip -- the 8-bit product for a few tokens (at most 16): the weights stream through once.
//
// The time is the weight bytes over HBM's rate, so nothing else may take longer.  A workgroup takes 16 kRT
// weight rows and the whole reduction, its 8 waves the blocks of 128 in turn; each wave loads its weight
// fragments straight into registers (a block's 16 rows are 16 runs of 128 bytes, in two 16-byte loads a
// lane) several blocks ahead, multiplies each with the block of the activations (16 x 16 x 128, the tokens
// padded to 16) and scales the sums in fp32.  The waves' sums meet in LDS, in a fixed order.  More rows per
// workgroup and few units in flight stream best (16384 x 4096 weights: 16.3 us with 64 rows and one unit of 8
// KB a wave beside the one in use, 17.9 us with two; 25 us with 32 rows, 29.6 us with 16).
//
// kX quantises the activations on the way: a lane holds 32 elements of its token's block, the four lanes
// of a token share the maximum, and the codes are the matrix instruction's operand as they stand.  Every
// workgroup does so again (T K elements, against its 16 kRT K weight bytes), which saves a launch.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp8_internal.h"
#include "fp8_tile.h"
#include "rtq_internal.h"

namespace rtq {
namespace {

using namespace fp8;

constexpr int kWaves = 8;
constexpr int kTokens = 16;

enum SmallX : int { kCodes = 0, kBF16 = 1, kF32 = 2 };

// Descriptor over [base, base + bytes), for loads into registers.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t resource(const void* base, int64_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, static_cast<int>(bytes), kBufferWord3);
}
// Scale i as stored: E8M0 or fp32 (0 past the end).
template <bool kE8M0>
__device__ __forceinline__ uint32_t load_raw(__amdgpu_buffer_rsrc_t r, uint32_t i) {
    if constexpr (kE8M0) return __builtin_amdgcn_raw_buffer_load_b8(r, i, 0, 0);
    return __builtin_amdgcn_raw_buffer_load_b32(r, 4 * i, 0, 0);
}
template <bool kE8M0>
__device__ __forceinline__ float raw_value(uint32_t r) {
    return kE8M0 ? e8m0_value(r) : __uint_as_float(r);
}

struct SmallParams {
    Fp8GemmParams g;
    const void* x;     // kX: activations [M][R] in place of codes and scales
};

// What a wave loads for one block of the reduction.  All of it goes through descriptors that end with the
// arrays: weight rows past N, tokens past M and elements past the reduction's end read as zeros.
template <int kRT, int kX>
struct Unit {
    v4i lo[kRT], hi[kRT];                    // weight chunks g and g + 4
    v4i x[kX == kCodes ? 2 : (kX == kBF16 ? 4 : 8)];   // the token's chunks g and g + 4: codes or elements
    uint32_t sa, sw;                         // scales as stored
};

// The unit's activations as codes, and their scale.
template <int kX, bool kE8M0, typename U>
__device__ __forceinline__ v8i activations(const U& u, float* scale) {
    if constexpr (kX == kCodes) {
        *scale = raw_value<kE8M0>(u.sa);
        return v8i{u.x[0].x, u.x[0].y, u.x[0].z, u.x[0].w, u.x[1].x, u.x[1].y, u.x[1].z, u.x[1].w};
    } else {
        float v[32];
        if constexpr (kX == kBF16) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t w = static_cast<uint32_t>(u.x[q][e]);
                    v[8 * q + 2 * e] = bf16_lo(w);
                    v[8 * q + 2 * e + 1] = bf16_hi(w);
                }
        } else {
#pragma unroll
            for (int q = 0; q < 8; ++q)
#pragma unroll
                for (int e = 0; e < 4; ++e) v[4 * q + e] = __uint_as_float(static_cast<uint32_t>(u.x[q][e]));
        }
        uint32_t m = 0u;
#pragma unroll
        for (int e = 0; e < 4; ++e) m = max(m, amax8(v + 8 * e));
        m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 16)));
        m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 32)));
        const int e = scale_exponent<false>(m);
        const float inv = pow2(-e);
        v8i c;
#pragma unroll
        for (int w = 0; w < 8; ++w)
            c[w] = static_cast<int>(encode4<false>(v[4 * w] * inv, v[4 * w + 1] * inv, v[4 * w + 2] * inv, v[4 * w + 3] * inv));
        *scale = pow2(e);
        return c;
    }
}

template <int kRT, int kX, bool kE5M2, bool kE8M0>
__global__ void __launch_bounds__(64 * kWaves)
fp8_small_kernel(SmallParams sp) {
    const Fp8GemmParams& p = sp.g;
    __shared__ __attribute__((aligned(16))) v4f s_sum[kWaves][kRT][64];
    constexpr int kAhead = kRT == 4 ? 1 : 2;   // units in flight beside the one in use
    constexpr int kScaleSize = kE8M0 ? 1 : 4;
    constexpr int kElem = kX == kCodes ? 1 : (kX == kBF16 ? 2 : 4);
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g = lane >> 4, l15 = lane & 15;
    const int R = p.R, blocks = (R + BK - 1) / BK;
    const int M = static_cast<int>(p.M), N = static_cast<int>(p.N);
    const int n0 = static_cast<int>(blockIdx.x) * 16 * kRT;
    const bool token = l15 < M;

    const __amdgpu_buffer_rsrc_t rw = resource(p.w + static_cast<int64_t>(n0) * R, static_cast<int64_t>(min(16 * kRT, N - n0)) * R);
    const __amdgpu_buffer_rsrc_t rx = resource(kX == kCodes ? static_cast<const void*>(p.a) : sp.x, static_cast<int64_t>(M) * R * kElem);
    const __amdgpu_buffer_rsrc_t rsa = resource(p.a_scale, static_cast<int64_t>(blocks) * M * kScaleSize);
    const __amdgpu_buffer_rsrc_t rsw = resource(static_cast<const uint8_t*>(p.w_scale) + n0 / BK * p.w_out_stride * kScaleSize,
                                                static_cast<int64_t>(blocks) * kScaleSize);
    const uint32_t woff = static_cast<uint32_t>(l15 * R + 16 * g), xoff = static_cast<uint32_t>((l15 * R + 16 * g) * kElem);
    auto load = [&](Unit<kRT, kX>& u, int kb) {
        const int k = kb * BK + 16 * g;
        const uint32_t o0 = k < R ? static_cast<uint32_t>(kb * BK) : kOob, o1 = k + 64 < R ? static_cast<uint32_t>(kb * BK + 64) : kOob;
#pragma unroll
        for (int i = 0; i < kRT; ++i) {
            u.lo[i] = __builtin_amdgcn_raw_buffer_load_b128(rw, woff + static_cast<uint32_t>(16 * i * R) + o0, 0, 0);
            u.hi[i] = __builtin_amdgcn_raw_buffer_load_b128(rw, woff + static_cast<uint32_t>(16 * i * R) + o1, 0, 0);
        }
        const uint32_t x0 = o0 == kOob ? kOob : xoff + o0 * kElem, x1 = o1 == kOob ? kOob : xoff + o1 * kElem;
#pragma unroll
        for (int e = 0; e < kElem; ++e) {
            u.x[e] = __builtin_amdgcn_raw_buffer_load_b128(rx, x0 + 16 * e, 0, 0);
            u.x[kElem + e] = __builtin_amdgcn_raw_buffer_load_b128(rx, x1 + 16 * e, 0, 0);
        }
        if constexpr (kX == kCodes) u.sa = load_raw<kE8M0>(rsa, token && kb < blocks ? static_cast<uint32_t>(kb * M + l15) : kOob / 4);
        u.sw = load_raw<kE8M0>(rsw, static_cast<uint32_t>(kb));
    };
    v4f acc[kRT];
#pragma unroll
    for (int i = 0; i < kRT; ++i) acc[i] = v4f{0.f, 0.f, 0.f, 0.f};
    auto multiply = [&](const Unit<kRT, kX>& u) {
        float s;
        const v8i a = activations<kX, kE8M0>(u, &s);
        s *= raw_value<kE8M0>(u.sw);
#pragma unroll
        for (int i = 0; i < kRT; ++i) {
            const v8i w{u.lo[i].x, u.lo[i].y, u.lo[i].z, u.lo[i].w, u.hi[i].x, u.hi[i].y, u.hi[i].z, u.hi[i].w};
            const v4f d = mfma<kE5M2>(w, a, v4f{0.f, 0.f, 0.f, 0.f});
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[i][r] = __builtin_fmaf(d[r], s, acc[i][r]);
        }
    };
    // The wave's blocks: wave + 8 j, j over turns from a place of the workgroup's own (rows a power of two
    // apart share memory channels: workgroups at the same place of their rows would crowd them).  Past the
    // last turn a unit is all zeros.  (Workgroup b runs on XCD b % 8, so b / 8 differs within an XCD.)
    const int turns = (blocks + kWaves - 1) / kWaves, start = static_cast<int>(blockIdx.x / 8) % turns;
    auto block = [&](int t) {
        const int j = t + start;
        return t < turns ? wave + kWaves * (j < turns ? j : j - turns) : blocks;
    };
    Unit<kRT, kX> u[kAhead];
#pragma unroll
    for (int q = 0; q < kAhead; ++q) load(u[q], block(q));
    for (int t = 0; t < turns; t += kAhead) {
#pragma unroll
        for (int q = 0; q < kAhead; ++q) {
            multiply(u[q]);
            load(u[q], block(t + q + kAhead));
        }
    }
#pragma unroll
    for (int i = 0; i < kRT; ++i) s_sum[wave][i][lane] = acc[i];
    __syncthreads();
    if (tid < 64 * kRT) {
        const int i = tid >> 6;
        v4f s = s_sum[0][i][lane];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) s += s_sum[w][i][lane];
        if (token) {
            const int n = n0 + 16 * i + 4 * g;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                if (n + r < N) {
                    const int64_t at = static_cast<int64_t>(l15) * N + n + r;
                    if (p.y_bf16)
                        static_cast<uint16_t*>(p.y)[at] = static_cast<uint16_t>(pack_bf16x2(s[r], 0.0f));
                    else
                        static_cast<float*>(p.y)[at] = s[r];
                }
            }
        }
    }
}

template <int kX, bool kE5M2, bool kE8M0>
hipError_t launch_rows(const SmallParams& p, hipStream_t stream) {
    // Rows per workgroup: as many as leave a workgroup for each CU (each repeats the activations' part).
    const int64_t tiles = (p.g.N + 15) / 16;
    const int cus = device_cu_count();
    if (tiles >= 4 * cus)
        fp8_small_kernel<4, kX, kE5M2, kE8M0><<<static_cast<unsigned>((tiles + 3) / 4), 64 * kWaves, 0, stream>>>(p);
    else if (tiles >= 2 * cus)
        fp8_small_kernel<2, kX, kE5M2, kE8M0><<<static_cast<unsigned>((tiles + 1) / 2), 64 * kWaves, 0, stream>>>(p);
    else
        fp8_small_kernel<1, kX, kE5M2, kE8M0><<<static_cast<unsigned>(tiles), 64 * kWaves, 0, stream>>>(p);
    return hipGetLastError();
}

template <int kX, bool kE5M2>
hipError_t launch(const SmallParams& p, hipStream_t stream) {
    return p.g.e8m0 ? launch_rows<kX, kE5M2, true>(p, stream) : launch_rows<kX, kE5M2, false>(p, stream);
}

}  // namespace

bool fp8_small_takes(int64_t M) { return M <= kTokens; }
// Every workgroup quantises all M R elements again: beyond about 2^16 of them that takes longer than a
// launch of its own (13 x 16384, 4096 rows: 25.8 us so, 23 us with the quantiser's launch; 16 x 4096, 16384
// rows: 19.0 and 20 us).
bool fp8_small_linear_takes(int64_t M, int R) { return M <= kTokens && M * R <= 65536; }

hipError_t launch_fp8_small(const fp8::Fp8GemmParams& g, bool e5m2, hipStream_t stream) {
    const SmallParams p{g, nullptr};
    return e5m2 ? launch<kCodes, true>(p, stream) : launch<kCodes, false>(p, stream);
}

hipError_t launch_fp8_small_linear(const Fp8GemmArgs& g, const void* x, bool x_bf16, hipStream_t stream) {
    SmallParams p{};
    p.g = fp8_gemm_params(g);
    p.x = x;
    return x_bf16 ? launch<kBF16, false>(p, stream) : launch<kF32, false>(p, stream);
}

}  // namespace rtq
