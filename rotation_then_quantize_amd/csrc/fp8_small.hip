// fp8_small.hip -- the 8-bit products for a few tokens, and for outputs of few tiles: no staging of shared
// tiles, no barrier until the end.
//
// A workgroup takes 16 kTT rows (tokens) by 16 kRT columns of the output and the whole reduction, its 8
// waves the blocks of 128 in turn.  Each wave loads its operands straight into the matrix instruction's
// registers (a block of 16 rows is 16 runs of 128 bytes, in two 16-byte loads a lane), multiplies block
// by block (16 x 16 x 128) and scales the sums in fp32.  The waves' sums meet in LDS, in a fixed order.
// Transposed weights ([reduction][columns]) go through LDS, each wave's through a part of its own, for the
// transposing read.
//
// kX quantises the activations on the way: a lane holds 32 elements of its token's block, the four lanes
// of a token share the maximum, and the codes are the matrix instruction's operand as they stand.  Every
// workgroup of a row of tiles does so again, which saves a launch; the first of them stores the codes and
// scales where they are kept.
//
// A few tokens (kTT = 1) are bound by the weights' bytes.  More columns per workgroup and few units a wave
// stream best (16384 x 4096 weights: 15.0 us, 4.5 TB/s, with 64 columns and one unit of 8 KB a wave, loaded again
// as soon as it has been multiplied, the other waves' loads being in flight meanwhile; when all XCDs began at the
// same place of their rows 16.3 so, 17.9 with two units, 25 with 32 columns, 29.6 with 16).  Small outputs are bound by latency: one
// launch, one chain of loads, products and sums.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp8_internal.h"
#include "fp8_tile.h"
#include "rtq_internal.h"

namespace rtq {
namespace {

using namespace fp8;

constexpr int kWaves = 8;
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
    void* keep;        // kX: their codes [M][R] and scales [blocks][M], or nullptr
    void* keep_scale;
};

// One token tile of a unit: chunks g and g + 4 of the lane's token (codes or elements), and its scale.
template <int kX>
struct Tokens {
    v4i x[kX == kCodes ? 2 : (kX == kBF16 ? 4 : 8)];
    uint32_t scale;
};
// What a wave loads for one block of the reduction.  All of it goes through descriptors that end with the
// arrays: rows past M or N and elements past the reduction's end read as zeros.
template <int kTT, int kRT, int kX, bool kTrans>
struct Unit {
    Tokens<kX> t[kTT];
    v4i lo[kTrans ? 1 : kRT], hi[kTrans ? 1 : kRT];   // weight chunks g and g + 4 (transposed: in LDS)
    uint32_t sw;
};

// The tile's activations as codes, and their scale.
template <int kX, bool kE5M2, bool kE8M0>
__device__ __forceinline__ v8i activations(const Tokens<kX>& u, float* scale) {
    if constexpr (kX == kCodes) {
        *scale = raw_value<kE8M0>(u.scale);
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
        const int e = scale_exponent<kE5M2>(m);
        const float inv = pow2(-e);
        v8i c;
#pragma unroll
        for (int w = 0; w < 8; ++w)
            c[w] = static_cast<int>(encode4<kE5M2>(v[4 * w] * inv, v[4 * w + 1] * inv, v[4 * w + 2] * inv, v[4 * w + 3] * inv));
        *scale = pow2(e);
        return c;
    }
}

template <int kTT, int kRT, bool kTrans>
constexpr int small_lds() {
    constexpr int sums = kWaves * kTT * kRT * 64 * 16, staged = kTrans ? kWaves * 2 * BK * 16 * kRT : 0;
    return sums > staged ? sums : staged;
}

template <int kTT, int kRT, int kX, bool kE5M2, bool kE8M0, bool kTrans>
__global__ void __launch_bounds__(64 * kWaves)
fp8_small_kernel(SmallParams sp) {
    const Fp8GemmParams& p = sp.g;
    extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
    constexpr int kUnits = kTrans ? 2 : (kTT == 1 && kRT == 4 ? 1 : 2);   // units a wave holds, the one in use among them
    constexpr int kScaleSize = kE8M0 ? 1 : 4;
    constexpr int kElem = kX == kCodes ? 1 : (kX == kBF16 ? 2 : 4);
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g = lane >> 4, l15 = lane & 15;
    const int R = p.R, blocks = (R + BK - 1) / BK;
    const int N = static_cast<int>(p.N);

    // Tiles in 8 contiguous ranges, one per XCD (workgroup b runs on XCD b % 8), the row tiles of a column
    // tile next to each other: they read the same weights.
    const int total = p.tiles_m * p.tiles_n, per = (total + 7) / 8;
    const int local = static_cast<int>(blockIdx.x) / 8, lin = static_cast<int>(blockIdx.x) % 8 * per + local;
    if (local >= per || lin >= total) return;
    const int64_t m0 = static_cast<int64_t>(lin % p.tiles_m) * 16 * kTT;
    const int n0 = lin / p.tiles_m * 16 * kRT;
    const int rows = static_cast<int>(min<int64_t>(16 * kTT, p.M - m0));

    const __amdgpu_buffer_rsrc_t rw = resource(p.w + (kTrans ? 0 : static_cast<int64_t>(n0) * R),
                                               kTrans ? 0 : static_cast<int64_t>(min(16 * kRT, N - n0)) * R);
    const __amdgpu_buffer_rsrc_t rx = resource((kX == kCodes ? static_cast<const uint8_t*>(p.a) : static_cast<const uint8_t*>(sp.x)) + m0 * R * kElem,
                                               static_cast<int64_t>(rows) * R * kElem);
    const uint32_t woff = static_cast<uint32_t>(l15 * R + 16 * g), xoff = static_cast<uint32_t>((l15 * R + 16 * g) * kElem);
    constexpr int kPitch = 16 * kRT, kDma = BK * kPitch / 1024;
    const uint32_t my_lds = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(lds)) + static_cast<uint32_t>(wave * 2 * BK * kPitch);
    const int w_row = lane / kRT;
    const uint32_t tr0 = my_lds + static_cast<uint32_t>((16 * g + (l15 >> 1)) * kPitch + (tr_swizzle<kPitch>(16 * g + (l15 >> 1)) << 4) + (lane & 1) * 8);

    auto load = [&](Unit<kTT, kRT, kX, kTrans>& u, int kb, int slot) {
        const int k = kb * BK + 16 * g;
        const uint32_t o0 = k < R ? static_cast<uint32_t>(kb * BK) : kOob, o1 = k + 64 < R ? static_cast<uint32_t>(kb * BK + 64) : kOob;
        if constexpr (!kTrans) {
#pragma unroll
            for (int i = 0; i < kRT; ++i) {
                u.lo[i] = __builtin_amdgcn_raw_buffer_load_b128(rw, woff + static_cast<uint32_t>(16 * i * R) + o0, 0, 0);
                u.hi[i] = __builtin_amdgcn_raw_buffer_load_b128(rw, woff + static_cast<uint32_t>(16 * i * R) + o1, 0, 0);
            }
        }
        const uint32_t x0 = o0 == kOob ? kOob : xoff + o0 * kElem, x1 = o1 == kOob ? kOob : xoff + o1 * kElem;
        const int kc = min(kb, blocks - 1), some = kb < blocks ? kScaleSize : 0;   // past the end all reads as zeros
        const __amdgpu_buffer_rsrc_t rsa = resource(static_cast<const uint8_t*>(p.a_scale) + (static_cast<int64_t>(kc) * p.M + m0) * kScaleSize,
                                                    rows * some);
        const __amdgpu_buffer_rsrc_t rsw = resource(static_cast<const uint8_t*>(p.w_scale) +
                                                        (n0 / BK * p.w_out_stride + kc * p.w_red_stride) * kScaleSize, some);
#pragma unroll
        for (int t = 0; t < kTT; ++t) {
            const uint32_t row = static_cast<uint32_t>(16 * t) * static_cast<uint32_t>(R * kElem);
#pragma unroll
            for (int e = 0; e < kElem; ++e) {
                u.t[t].x[e] = __builtin_amdgcn_raw_buffer_load_b128(rx, x0 + row + 16 * e, 0, 0);
                u.t[t].x[kElem + e] = __builtin_amdgcn_raw_buffer_load_b128(rx, x1 + row + 16 * e, 0, 0);
            }
            if constexpr (kX == kCodes) u.t[t].scale = load_raw<kE8M0>(rsa, static_cast<uint32_t>(16 * t + l15));
        }
        u.sw = load_raw<kE8M0>(rsw, 0u);
        if constexpr (kTrans) {   // last: the wait below counts on it
            const int64_t n_rows = max(0, min(BK, R - kb * BK));
            const int64_t bytes = n_rows * N - n0;
            const v4i rt = make_rsrc(p.w + static_cast<int64_t>(kc) * BK * N + n0, bytes > 0 ? static_cast<uint32_t>(bytes) : 0u);
#pragma unroll
            for (int q = 0; q < kDma; ++q) {
                const int row = q * (64 / kRT) + w_row;
                load_to_lds(rt, static_cast<uint32_t>(row) * static_cast<uint32_t>(N) + static_cast<uint32_t>(((lane % kRT) ^ tr_swizzle<kPitch>(row)) << 4),
                            my_lds + static_cast<uint32_t>(slot * BK * kPitch + q * 1024));
            }
        }
    };
    v4f acc[kTT][kRT];
#pragma unroll
    for (int t = 0; t < kTT; ++t)
#pragma unroll
        for (int i = 0; i < kRT; ++i) acc[t][i] = v4f{0.f, 0.f, 0.f, 0.f};
    const bool keep = kX != kCodes && sp.keep != nullptr && n0 == 0;
    auto multiply = [&](const Unit<kTT, kRT, kX, kTrans>& u, int kb, int slot) {
        v8i w[kRT];
        if constexpr (kTrans) {
            wait_vmcnt<kDma>();   // all but the next unit's loads to LDS, the last ones issued, have landed
#pragma unroll
            for (int i = 0; i < kRT; ++i) {
                const uint32_t at = (tr0 + static_cast<uint32_t>(slot * BK * kPitch)) ^ static_cast<uint32_t>(i << 4);
                const v2i r[4] = {read_tr8(at), read_tr8(at + 8 * kPitch), read_tr8(at + 64 * kPitch), read_tr8(at + 72 * kPitch)};
                w[i] = v8i{r[0].x, r[0].y, r[1].x, r[1].y, r[2].x, r[2].y, r[3].x, r[3].y};
            }
        } else {
#pragma unroll
            for (int i = 0; i < kRT; ++i)
                w[i] = v8i{u.lo[i].x, u.lo[i].y, u.lo[i].z, u.lo[i].w, u.hi[i].x, u.hi[i].y, u.hi[i].z, u.hi[i].w};
        }
        const float sw = raw_value<kE8M0>(u.sw);
#pragma unroll
        for (int t = 0; t < kTT; ++t) {
            float s;
            const v8i a = activations<kX, kE5M2, kE8M0>(u.t[t], &s);
            if (keep) {
                const int row = 16 * t + l15, k = kb * BK + 16 * g;
                uint8_t* at = static_cast<uint8_t*>(sp.keep) + (m0 + row) * R + k;
                if (row < rows && k < R) *reinterpret_cast<v4i*>(at) = v4i{a[0], a[1], a[2], a[3]};
                if (row < rows && k + 64 < R) *reinterpret_cast<v4i*>(at + 64) = v4i{a[4], a[5], a[6], a[7]};
                if (row < rows && g == 0 && kb < blocks)
                    store_scale(sp.keep_scale, kE8M0, static_cast<int64_t>(kb) * p.M + m0 + row,
                                static_cast<int>(__float_as_uint(s) >> 23) - 127);
            }
            s *= sw;
#pragma unroll
            for (int i = 0; i < kRT; ++i) {
                const v4f d = mfma<kE5M2>(w[i], a, v4f{0.f, 0.f, 0.f, 0.f});
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[t][i][r] = __builtin_fmaf(d[r], s, acc[t][i][r]);
            }
        }
        if constexpr (kTrans) lds_done();   // the weights are in registers before the slot is filled again
    };
    // The wave's blocks: wave + 8 j, j over turns from a place of the workgroup's own: rows a power of two
    // apart share memory channels, and workgroups at the same place of their rows would crowd them (13 x 16384,
    // 4096 columns, product alone: 16.5 us; 22 with the same place in all XCDs).  Past the last turn a unit is
    // all zeros.
    const int turns = (blocks + kWaves - 1) / kWaves, start = static_cast<int>(blockIdx.x) % turns;
    auto block = [&](int t) {
        const int j = t + start;
        return t < turns ? wave + kWaves * (j < turns ? j : j - turns) : blocks;
    };
    Unit<kTT, kRT, kX, kTrans> u[kUnits];
#pragma unroll
    for (int q = 0; q < kUnits; ++q) load(u[q], block(q), q);
    for (int t = 0; t < turns; t += kUnits) {
#pragma unroll
        for (int q = 0; q < kUnits; ++q) {
            multiply(u[q], block(t + q), q);
            load(u[q], block(t + q + kUnits), q);
        }
    }
    if constexpr (kTrans) {
        wait_vmcnt<0>();   // nothing is still writing the LDS that the sums go to
        __syncthreads();
    }
    v4f* sums = reinterpret_cast<v4f*>(lds);   // [wave][token tile][column tile][lane]
    constexpr int kSums = kTT * kRT * 64;
#pragma unroll
    for (int t = 0; t < kTT; ++t)
#pragma unroll
        for (int i = 0; i < kRT; ++i) sums[(wave * kTT * kRT + t * kRT + i) * 64 + lane] = acc[t][i];
    __syncthreads();
    for (int e = tid; e < kSums; e += 64 * kWaves) {
        v4f s = sums[e];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) s += sums[w * kSums + e];
        const int t = e / (64 * kRT), i = e / 64 % kRT, l = e % 64;
        store4(p.y, p.y_bf16, p.M, p.N, m0 + 16 * t + (l & 15), n0 + 16 * i + 4 * (l >> 4), s);
    }
}

template <int kTT, int kRT, int kX, bool kE5M2, bool kE8M0, bool kTrans>
hipError_t launch_tile(SmallParams p, hipStream_t stream) {
    auto kernel = fp8_small_kernel<kTT, kRT, kX, kE5M2, kE8M0, kTrans>;
    constexpr int lds = small_lds<kTT, kRT, kTrans>();
    if constexpr (lds > 65536) {
        int per_cu = 0;
        const hipError_t e = kernel_blocks_per_cu(reinterpret_cast<const void*>(kernel), 64 * kWaves, lds, &per_cu);
        if (e != hipSuccess) return e;
    }
    p.g.tiles_m = static_cast<int>((p.g.M + 16 * kTT - 1) / (16 * kTT));
    p.g.tiles_n = static_cast<int>((p.g.N + 16 * kRT - 1) / (16 * kRT));
    const int total = p.g.tiles_m * p.g.tiles_n;
    kernel<<<static_cast<unsigned>((total + 7) / 8 * 8), 64 * kWaves, lds, stream>>>(p);
    return hipGetLastError();
}

template <int kX, bool kE5M2, bool kE8M0, bool kTrans>
hipError_t launch_form(const SmallParams& p, hipStream_t stream) {
    const int64_t tiles = (p.g.N + 15) / 16;
    const int cus = device_cu_count();
    if (p.g.M > 16) {
        // 32 tokens by 64 columns, or by 32 where that leaves CUs idle (layers, us with 64 and with 32: 32 x 1024, 1024
        // columns, 16 tiles of 64: 10.0, 8.5; 200 x 2048, 1024, 112 tiles: 12.8, 10.5; 200 x 1024, 2048, 224 tiles: 10.2,
        // 15.7; 256 x 2048, 2048, 256 tiles: 13.0, 19.7)
        if ((p.g.M + 31) / 32 * ((p.g.N + 63) / 64) >= cus / 2) return launch_tile<2, 4, kX, kE5M2, kE8M0, kTrans>(p, stream);
        return launch_tile<2, 2, kX, kE5M2, kE8M0, kTrans>(p, stream);
    }
    // Columns per workgroup: as few as leave no CU with two (each repeats the activations' part, and a CU with two
    // takes twice as long as the others: layers of one token, 4096 long, 4608 columns 8.5 us with 32, 10.5 with
    // 16; 9216 columns 11.6 with 64, 14.8 with 32).
    if (tiles > 2 * cus) return launch_tile<1, 4, kX, kE5M2, kE8M0, kTrans>(p, stream);
    if (tiles > cus) return launch_tile<1, 2, kX, kE5M2, kE8M0, kTrans>(p, stream);
    return launch_tile<1, 1, kX, kE5M2, kE8M0, kTrans>(p, stream);
}

template <int kX, bool kE5M2, bool kTrans>
hipError_t launch(const SmallParams& p, hipStream_t stream) {
    return p.g.e8m0 ? launch_form<kX, kE5M2, true, kTrans>(p, stream) : launch_form<kX, kE5M2, false, kTrans>(p, stream);
}

template <bool kE5M2, bool kTrans>
hipError_t launch_x(const SmallParams& p, bool x_bf16, hipStream_t stream) {
    return x_bf16 ? launch<kBF16, kE5M2, kTrans>(p, stream) : launch<kF32, kE5M2, kTrans>(p, stream);
}

// More than 16 rows: an output whose workgroups all run at once, and at most two turns of the waves through
// the reduction.  (Layer, 391 x 1936, 1001 columns: 11.6 us, 14.0 through the quantiser and shared tiles; 200
// x 2048, 1024: 10.9 and 12.6; but 300 x 1024, 2048, 320 workgroups: 18.7 and 10.3; 40 x 4096, 2048: 16.3 and
// 14.3.)
bool fits(int64_t M, int64_t N, int R) {
    return R <= 2048 && (M + 31) / 32 * ((N + 63) / 64) <= device_cu_count();
}

}  // namespace

// At most 16 rows: always, but transposed weights, whose rows of 16 to 64 bytes a workgroup stream badly, only up to 16
// M of them (16 tokens, reduction x columns, us here and with 64 x 64 tiles: 2048 x 4096 6.5, 9.4; 4096 x 4096 9.0, 9.9;
// 8192 x 4096 16.0, 12.0; 16384 x 4096 34.0, 18.0; but 4096 x 8192 10.8, 12.0; 4096 x 16384 15.5, 15.8).
bool fp8_small_takes(int64_t M, int64_t N, int R, bool trans) {
    if (M <= 16) return !trans || N * R <= int64_t{16} << 20;
    return fits(M, N, R);
}
// Every workgroup quantises its rows again: of few tokens, along a long reduction that takes longer than a launch
// of its own, the sooner the fewer columns a workgroup has (4096 columns, 1 x 4096: 7.2 us so, 9.2 with the
// quantiser's launch, 16 x 6144: 12.2 and 11.0, 1 x 8192: 11.2 and 10.0, 2 x 32768: 41.0 and 33.2; 64 columns a
// workgroup, 16384 columns, 2 x 6144: 22.2 and 24.1, 28672 columns, 1 x 8192: 45.1 and 46.1).
bool fp8_small_linear_takes(int64_t M, int64_t N, int R, bool trans) {
    return fp8_small_takes(M, N, R, trans) && (M > 16 || R <= ((N + 15) / 16 > 2 * device_cu_count() ? 8192 : 4096));
}

hipError_t launch_fp8_small(const fp8::Fp8GemmParams& g, bool trans, bool e5m2, hipStream_t stream) {
    const SmallParams p{g, nullptr, nullptr, nullptr};
    if (trans) return e5m2 ? launch<kCodes, true, true>(p, stream) : launch<kCodes, false, true>(p, stream);
    return e5m2 ? launch<kCodes, true, false>(p, stream) : launch<kCodes, false, false>(p, stream);
}

hipError_t launch_fp8_small_linear(const Fp8GemmArgs& g, const void* x, bool x_bf16, void* keep, void* keep_scale,
                                   hipStream_t stream) {
    const SmallParams p{fp8_gemm_params(g), x, keep, keep_scale};
    if (g.trans) return g.a_e5m2 ? launch_x<true, true>(p, x_bf16, stream) : launch_x<false, true>(p, x_bf16, stream);
    return launch_x<false, false>(p, x_bf16, stream);
}

}  // namespace rtq
