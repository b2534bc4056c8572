// fp8_gemm.hip -- products of 8-bit floating point codes with one scale for each block of 128, on the
// gfx950 matrix cores:
//
//   y[t][n]  = sum_kb sa[kb][t] sw[n / 128][kb]  sum_{k in kb} qa[t][k] qw[n][k]
//   dx[t][k] = sum_nb sg[nb][t] sw[nb][k / 128]  sum_{n in nb} qg[t][n] qw[n][k]
//
// A block of 128 along the reduction is one v_mfma_f32_16x16x128_f8f6f4, so a block's sum is one
// instruction from a zero accumulator, and its scale enters as one fp32 multiply-add into the running
// sum.  The matrix core aligns an instruction's products to about 2^-14 of the largest before it adds
// them (measured: 1.8e-5 relative error of one 128-long sum in the 2-norm, whichever fp8 instruction
// computes it); everything from there on is fp32.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "fp8_internal.h"
#include "fp8_tile.h"
#include "rtq_internal.h"

namespace rtq {
namespace {

using namespace fp8;

// Four consecutive outputs of row m from column n.
__device__ __forceinline__ void store4(void* y, bool bf16, int64_t M, int64_t N, int64_t m, int64_t n, const v4f& v) {
    if (m >= M || n >= N) return;
    const int64_t at = m * N + n;
    if (n + 4 <= N && N % 4 == 0) {
        if (bf16)
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(y) + at) = uint2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
        else
            *reinterpret_cast<v4f*>(static_cast<float*>(y) + at) = v;
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (n + i < N) {
            if (bf16)
                static_cast<uint16_t*>(y)[at + i] = static_cast<uint16_t>(pack_bf16x2(v[i], 0.0f));
            else
                static_cast<float*>(y)[at + i] = v[i];
        }
    }
}

template <int BM, int BN, int kWavesM, int kWavesN, int kSlots, bool kTrans, bool kE5M2, bool kE8M0>
__global__ void __launch_bounds__(64 * kWavesM * kWavesN)
fp8_gemm_kernel(Fp8GemmParams p) {
    constexpr int kWaves = kWavesM * kWavesN;
    constexpr int WM = BM / kWavesM, WN = BN / kWavesN;
    constexpr int TM = WM / 16, TN = WN / 16;
    constexpr int kABytes = BM * BK, kWBytes = BN * BK, kStage = kABytes + kWBytes;
    constexpr int kALoads = BM / 8 / kWaves, kWLoads = BN / 8 / kWaves;   // 1 KB loads per wave
    constexpr int kChunks = BN / 16;                                      // kTrans: 16-byte chunks per LDS row
    static_assert(BM % (8 * kWaves) == 0 && BN % (8 * kWaves) == 0, "whole loads per wave");
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const uint32_t lds_base = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(lds));

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / kWavesN, wn = wave % kWavesN;
    const int g = lane >> 4, l15 = lane & 15;

    const int tile = static_cast<int>(blockIdx.x) / p.split, part = static_cast<int>(blockIdx.x) % p.split;
    const int64_t m0 = static_cast<int64_t>(tile % p.tiles_m) * BM, n0 = static_cast<int64_t>(tile / p.tiles_m) * BN;
    const int blocks = (p.R + BK - 1) / BK;
    const int kb0 = static_cast<int>(static_cast<int64_t>(blocks) * part / p.split);
    const int kb1 = static_cast<int>(static_cast<int64_t>(blocks) * (part + 1) / p.split);

    const int rows_a = static_cast<int>(min<int64_t>(BM, p.M - m0));
    const int rows_w = static_cast<int>(min<int64_t>(BN, p.N - n0));
    const v4i rsa = make_rsrc(p.a + m0 * p.R, static_cast<uint32_t>(rows_a) * static_cast<uint32_t>(p.R));
    v4i rsw = make_rsrc(p.w + (kTrans ? 0 : n0 * p.R), static_cast<uint32_t>(rows_w) * static_cast<uint32_t>(p.R));

    // LDS rows of 128 bytes, chunk c (16 bytes) of row r at chunk c ^ ((r >> 1) & 7); lane group g holds
    // chunks g and g + 4 of its row, which makes the 16-byte reads free of bank conflicts (see the large
    // kernel).  Transposed weights: rows of BN bytes (one n), chunk c of row r at c ^ row_swizzle(r): 8 rows
    // of one chunk touch all banks once.
    auto row_swizzle = [](int row) { return (row * BN / 256) & (kChunks - 1); };
    auto issue = [&](int kb) {
        const uint32_t slot = lds_base + static_cast<uint32_t>(((kb - kb0) % kSlots) * kStage);
#pragma unroll
        for (int q = 0; q < kALoads; ++q) {
            const int row = 8 * (q * kWaves + wave) + (lane >> 3);
            const int col = kb * BK + (((lane & 7) ^ ((row >> 1) & 7)) << 4);
            load_to_lds(rsa, col < p.R ? static_cast<uint32_t>(row * p.R + col) : kOob,
                        slot + static_cast<uint32_t>((q * kWaves + wave) * 1024));
        }
        if constexpr (kTrans) {
            const int rows = min(BK, p.R - kb * BK);
            rsw = make_rsrc(p.w + static_cast<int64_t>(kb) * BK * p.N + n0,
                            static_cast<uint32_t>(rows * p.N - n0));
        }
#pragma unroll
        for (int q = 0; q < kWLoads; ++q) {
            uint32_t off;
            if constexpr (kTrans) {
                const int row = (64 / kChunks) * (q * kWaves + wave) + lane / kChunks;
                off = static_cast<uint32_t>(row * static_cast<int>(p.N) + (((lane % kChunks) ^ row_swizzle(row)) << 4));
            } else {
                const int row = 8 * (q * kWaves + wave) + (lane >> 3);
                const int col = kb * BK + (((lane & 7) ^ ((row >> 1) & 7)) << 4);
                off = col < p.R ? static_cast<uint32_t>(row * p.R + col) : kOob;
            }
            load_to_lds(rsw, off, slot + static_cast<uint32_t>(kABytes + (q * kWaves + wave) * 1024));
        }
    };
    const uint32_t f0 = static_cast<uint32_t>(l15 * BK + ((g ^ (l15 >> 1)) << 4));
    const uint32_t f1 = static_cast<uint32_t>(l15 * BK + (((g + 4) ^ (l15 >> 1)) << 4));
    auto read_frag = [&](const uint8_t* base) {
        const v4i x = *reinterpret_cast<const v4i*>(base + f0), y = *reinterpret_cast<const v4i*>(base + f1);
        return v8i{x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
    };
    auto read_frag_tr = [&](uint32_t base, int chunk) {
        v2i r[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int row = 64 * (q >> 1) + 16 * g + 8 * (q & 1) + (l15 >> 1);
            r[q] = read_tr8(base + static_cast<uint32_t>(row * BN + ((chunk ^ row_swizzle(row)) << 4) + (lane & 1) * 8));
        }
        return v8i{r[0].x, r[0].y, r[1].x, r[1].y, r[2].x, r[2].y, r[3].x, r[3].y};
    };

    v4f acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};

    int64_t mi[TM];   // the lane's row of each row tile, kept inside the array
#pragma unroll
    for (int i = 0; i < TM; ++i) mi[i] = min<int64_t>(m0 + wm * WM + i * 16 + l15, p.M - 1);
    const int64_t wblock = min<int64_t>((n0 + wn * WN) / kFp8Block, (p.N - 1) / kFp8Block);

#pragma unroll
    for (int s = 0; s < kSlots - 1; ++s)
        if (kb0 + s < kb1) issue(kb0 + s);
    constexpr int kLoads = kALoads + kWLoads;
    for (int kb = kb0; kb < kb1; ++kb) {
        const float sw = load_scale<kE8M0>(p.w_scale, wblock * p.w_out_stride + kb * p.w_red_stride);
        float s[TM];
#pragma unroll
        for (int i = 0; i < TM; ++i) s[i] = load_scale<kE8M0>(p.a_scale, kb * p.M + mi[i]) * sw;
        // block kb has landed (later blocks may be in flight), in every wave; block kb - 1 is read
        if (kSlots > 2 && kb + kSlots - 2 < kb1)
            wait_vmcnt<(kSlots - 2) * kLoads>();
        else
            wait_vmcnt<0>();
        barrier();
        if (kb + kSlots - 1 < kb1) issue(kb + kSlots - 1);
        const int slot = ((kb - kb0) % kSlots) * kStage;
        v8i fa[TM], fw[TN];
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            if constexpr (kTrans)
                fw[j] = read_frag_tr(lds_base + static_cast<uint32_t>(slot + kABytes), (wn * WN + j * 16) / 16);
            else
                fw[j] = read_frag(lds + slot + kABytes + (wn * WN + j * 16) * BK);
        }
#pragma unroll
        for (int i = 0; i < TM; ++i) fa[i] = read_frag(lds + slot + (wm * WM + i * 16) * BK);
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                const v4f d = mfma<kE5M2>(fw[j], fa[i], v4f{0.f, 0.f, 0.f, 0.f});
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[i][j][r] = __builtin_fmaf(d[r], s[i], acc[i][j][r]);
            }
        lds_done();   // the fragments are in registers before the barrier that lets the slot be refilled
    }
    void* y = p.y;
    if (p.split > 1) y = static_cast<float*>(p.y) + static_cast<int64_t>(part) * p.M * p.N;
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
            store4(y, p.split == 1 && p.y_bf16, p.M, p.N, m0 + wm * WM + i * 16 + l15, n0 + wn * WN + j * 16 + 4 * g,
                   acc[i][j]);
}

// y = the sum of the split partials, in order (the result does not depend on which finished first).
__global__ void __launch_bounds__(256)
fp8_reduce_kernel(const float* __restrict__ part, int split, int64_t n, void* __restrict__ y, bool y_bf16) {
    const int64_t i = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 4;
    if (i >= n) return;
    if (i + 4 <= n && n % 4 == 0) {
        v4f s = *reinterpret_cast<const v4f*>(part + i);
        for (int k = 1; k < split; ++k) s += *reinterpret_cast<const v4f*>(part + k * n + i);
        if (y_bf16)
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(y) + i) = uint2{pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3])};
        else
            *reinterpret_cast<v4f*>(static_cast<float*>(y) + i) = s;
        return;
    }
    for (int64_t e = i; e < min(i + 4, n); ++e) {
        float s = part[e];
        for (int k = 1; k < split; ++k) s += part[k * n + e];
        if (y_bf16)
            static_cast<uint16_t*>(y)[e] = static_cast<uint16_t>(pack_bf16x2(s, 0.0f));
        else
            static_cast<float*>(y)[e] = s;
    }
}

constexpr int kTile = 64;   // the small tile's rows and columns
constexpr int kMaxSplit = 16;

// Ranges of the reduction per tile: enough workgroups for two per CU, each at least four blocks long.
int choose_split(int64_t tiles, int blocks) {
    const int64_t want = 2 * 256;
    if (tiles >= want) return 1;
    const int64_t s = std::min<int64_t>(want / tiles, blocks / 4);
    return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(s, kMaxSplit)));
}

// (the large kernel's loads run two stages ahead, so it takes reductions of at least two blocks)
bool use_large(int64_t M, int64_t N, int R) { return R > BK && ((M + 255) / 256) * ((N + 255) / 256) >= 96; }

template <bool kTrans, bool kE5M2>
hipError_t launch(const Fp8GemmArgs& g, hipStream_t stream) {
    constexpr int kSlots = 4;
    constexpr size_t lds = static_cast<size_t>(kSlots) * 2 * kTile * BK;
    auto kernel = g.e8m0 ? fp8_gemm_kernel<kTile, kTile, 2, 2, kSlots, kTrans, kE5M2, true>
                         : fp8_gemm_kernel<kTile, kTile, 2, 2, kSlots, kTrans, kE5M2, false>;
    int per_cu = 0;
    hipError_t e = kernel_blocks_per_cu(reinterpret_cast<const void*>(kernel), 256, lds, &per_cu);
    if (e != hipSuccess) return e;
    Fp8GemmParams p = fp8_gemm_params(g);
    if (!kTrans && fp8_small_takes(g.M)) return launch_fp8_small(p, kE5M2, stream);
    if (use_large(g.M, g.N, g.R)) {
        return launch_fp8_gemm_large(p, kTrans, kE5M2, stream);
    }
    p.tiles_m = static_cast<int>((g.M + kTile - 1) / kTile);
    p.tiles_n = static_cast<int>((g.N + kTile - 1) / kTile);
    const int64_t tiles = static_cast<int64_t>(p.tiles_m) * p.tiles_n;
    p.split = choose_split(tiles, static_cast<int>(fp8_groups(g.R)));
    if (g.workspace == nullptr || g.ws_bytes < static_cast<size_t>(p.split) * g.M * g.N * sizeof(float)) p.split = 1;
    p.y = p.split > 1 ? g.workspace : g.y;
    kernel<<<static_cast<unsigned>(tiles * p.split), 256, lds, stream>>>(p);
    e = hipGetLastError();
    if (e != hipSuccess || p.split == 1) return e;
    const int64_t n = g.M * g.N;
    fp8_reduce_kernel<<<static_cast<unsigned>((n + 1023) / 1024), 256, 0, stream>>>(static_cast<const float*>(g.workspace),
                                                                                    p.split, n, g.y, g.y_bf16);
    return hipGetLastError();
}

}  // namespace

fp8::Fp8GemmParams fp8_gemm_params(const Fp8GemmArgs& g) {
    fp8::Fp8GemmParams p{};
    p.a = static_cast<const uint8_t*>(g.a);
    p.a_scale = g.a_scale;
    p.w = static_cast<const uint8_t*>(g.w);
    p.w_scale = g.w_scale;
    p.e8m0 = g.e8m0;
    p.M = g.M;
    p.N = g.N;
    p.R = g.R;
    p.w_out_stride = g.trans ? 1 : fp8_groups(g.R);
    p.w_red_stride = g.trans ? fp8_groups(g.N) : 1;
    p.split = 1;
    p.y = g.y;
    p.y_bf16 = g.y_bf16;
    return p;
}

size_t fp8_gemm_workspace_bytes(int64_t M, int64_t N, int R, bool trans) {
    if ((!trans && fp8_small_takes(M)) || use_large(M, N, R)) return 0;
    const int64_t tiles = ((M + kTile - 1) / kTile) * ((N + kTile - 1) / kTile);
    const int split = choose_split(tiles, static_cast<int>(fp8_groups(R)));
    return split > 1 ? static_cast<size_t>(split) * M * N * sizeof(float) : 0;
}

hipError_t launch_fp8_gemm(const Fp8GemmArgs& g, hipStream_t stream) {
    if (g.trans) return g.a_e5m2 ? launch<true, true>(g, stream) : launch<true, false>(g, stream);
    return g.a_e5m2 ? launch<false, true>(g, stream) : launch<false, false>(g, stream);
}

}  // namespace rtq
