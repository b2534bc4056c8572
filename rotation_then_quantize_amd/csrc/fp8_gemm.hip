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
// computes it); everything from there on is fp32, but for E8M0 scales in the large kernel, see there.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "fp8_internal.h"
#include "fp8_tile.h"
#include "rtq_internal.h"

namespace rtq {
namespace {

using namespace fp8;

constexpr int kTable = 32;   // blocks whose scales are in LDS (an even number)

template <int BM, int BN, int kSlots>
constexpr int tile_lds() { return kSlots * (BM + BN) * BK + kTable * BM * static_cast<int>(sizeof(float)); }

// A tile of BM x BN outputs, a ring of kSlots LDS stages of one block of the reduction each, loaded kSlots
// stages ahead (tiles this small are bound by the loads' latency, not by their products); a block's fragments
// are read while the block before it is multiplied (with branches in that stage, which made the compiler wait
// for the reads first, 512 x 4096 x 4096 took 20.8 us instead of 18.4).  The rows' scales times the weight's,
// of kTable blocks at a time, are put into LDS beforehand: loads of scales among the stages' would make every
// wait for one a wait for the stages behind it.
template <int BM, int BN, int kWavesM, int kWavesN, int kSlots, bool kTrans, bool kE5M2, bool kE8M0>
__global__ void __launch_bounds__(64 * kWavesM * kWavesN)
fp8_gemm_kernel(Fp8GemmParams p) {
    constexpr int kWaves = kWavesM * kWavesN;
    constexpr int WM = BM / kWavesM, WN = BN / kWavesN;
    constexpr int TM = WM / 16, TN = WN / 16;
    constexpr int kABytes = BM * BK, kWBytes = BN * BK, kStage = kABytes + kWBytes;
    constexpr int kALoads = BM / 8 / kWaves, kWLoads = BN / 8 / kWaves;   // 1 KB loads per wave
    static_assert(BM % (8 * kWaves) == 0 && BN % (8 * kWaves) == 0 && BN <= kFp8Block, "whole loads per wave, one weight scale");
    extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
    const uint32_t lds_base = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(lds));
    float* table = reinterpret_cast<float*>(lds + kSlots * kStage);

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / kWavesN, wn = wave % kWavesN;
    const int g = lane >> 4, l15 = lane & 15;

    // 8 contiguous ranges of tiles and their parts, one per XCD (workgroup b runs on XCD b % 8)
    const int total = p.tiles_m * p.tiles_n * p.split, per = (total + 7) / 8;
    const int b = static_cast<int>(block_index()), local = b / 8, lin = b % 8 * per + local;
    if (local >= per || lin >= total) return;
    const int tile = lin / p.split, part = lin % p.split;
    const int64_t m0 = static_cast<int64_t>(tile % p.tiles_m) * BM, n0 = static_cast<int64_t>(tile / p.tiles_m) * BN;
    const int blocks = (p.R + BK - 1) / BK;
    const int kb0 = static_cast<int>(static_cast<int64_t>(blocks) * part / p.split);
    const int kb1 = static_cast<int>(static_cast<int64_t>(blocks) * (part + 1) / p.split);

    const int rows_a = static_cast<int>(min<int64_t>(BM, p.M - m0));
    const int rows_w = static_cast<int>(min<int64_t>(BN, p.N - n0));
    const int end = min(p.R, kb1 * BK);   // of this part of the reduction: loads past it give zeros
    const v4i rsa = make_rsrc(p.a + m0 * p.R, static_cast<uint32_t>(rows_a) * static_cast<uint32_t>(p.R));
    v4i rsw = make_rsrc(p.w + (kTrans ? 0 : n0 * p.R), static_cast<uint32_t>(rows_w) * static_cast<uint32_t>(p.R));

    // LDS rows of 128 bytes, chunk c (16 bytes) of row r at chunk c ^ ((r >> 1) & 7); lane group g holds
    // chunks g and g + 4 of its row, which makes the 16-byte reads free of bank conflicts (see the large
    // kernel).  Transposed weights: rows of BN bytes.
    auto issue = [&](int kb) {
        const uint32_t slot = lds_base + static_cast<uint32_t>(((kb - kb0) % kSlots) * kStage);
#pragma unroll
        for (int q = 0; q < kALoads; ++q) {
            const int row = 8 * (q * kWaves + wave) + (lane >> 3);
            const int col = kb * BK + (((lane & 7) ^ ((row >> 1) & 7)) << 4);
            load_to_lds(rsa, col < end ? static_cast<uint32_t>(row * p.R + col) : kOob,
                        slot + static_cast<uint32_t>((q * kWaves + wave) * 1024));
        }
        if constexpr (kTrans) {
            const int rows = min(BK, end - kb * BK);
            rsw = make_rsrc(p.w + static_cast<int64_t>(kb) * BK * p.N + n0,
                            rows > 0 ? static_cast<uint32_t>(rows * p.N - n0) : 0u);
        }
#pragma unroll
        for (int q = 0; q < kWLoads; ++q) {
            uint32_t off;
            if constexpr (kTrans) {
                constexpr int kChunks = BN / 16;   // 16-byte chunks of an LDS row
                const int row = (64 / kChunks) * (q * kWaves + wave) + lane / kChunks;
                off = static_cast<uint32_t>(row * static_cast<int>(p.N) + (((lane % kChunks) ^ tr_swizzle<BN>(row)) << 4));
            } else {
                const int row = 8 * (q * kWaves + wave) + (lane >> 3);
                const int col = kb * BK + (((lane & 7) ^ ((row >> 1) & 7)) << 4);
                off = col < end ? static_cast<uint32_t>(row * p.R + col) : kOob;
            }
            load_to_lds(rsw, off, slot + static_cast<uint32_t>(kABytes + (q * kWaves + wave) * 1024));
        }
    };
    const int64_t wblock = n0 / kFp8Block;
    auto fill = [&](int c0) {   // the table of blocks c0 ..; row r of wave-row wm at [block][wm][r % 16][r / 16]
#pragma unroll 4
        for (int e = tid; e < kTable * BM; e += 64 * kWaves) {
            const int kb = min(c0 + e / BM, blocks - 1), r = e % BM;
            const int64_t m = min<int64_t>(m0 + r, p.M - 1);
            table[e / BM * BM + (r / WM * 16 + (r & 15)) * TM + (r % WM >> 4)] =
                load_scale<kE8M0>(p.a_scale, kb * p.M + m) * load_scale<kE8M0>(p.w_scale, wblock * p.w_out_stride + kb * p.w_red_stride);
        }
    };
    const uint32_t f0 = static_cast<uint32_t>(l15 * BK + ((g ^ (l15 >> 1)) << 4));
    const uint32_t f1 = static_cast<uint32_t>(l15 * BK + (((g + 4) ^ (l15 >> 1)) << 4));
    auto read_frag = [&](const uint8_t* base) {
        const v4i x = *reinterpret_cast<const v4i*>(base + f0), y = *reinterpret_cast<const v4i*>(base + f1);
        return v8i{x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
    };
    const int tr_row = 16 * g + (l15 >> 1);
    const uint32_t tr0 = static_cast<uint32_t>(tr_row * BN + (lane & 1) * 8);
    auto read_frag_tr = [&](uint32_t base, int chunk) {
        const uint32_t at = base + tr0 + static_cast<uint32_t>((chunk ^ tr_swizzle<BN>(tr_row)) << 4);
        const v2i r[4] = {read_tr8(at), read_tr8(at + 8 * BN), read_tr8(at + 64 * BN), read_tr8(at + 72 * BN)};
        return v8i{r[0].x, r[0].y, r[1].x, r[1].y, r[2].x, r[2].y, r[3].x, r[3].y};
    };

    v4f acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};

    constexpr int kLoads = kALoads + kWLoads;
    v8i fa[2][TM], fw[2][TN];
    float sc[2][TM];
    auto read_scales = [&](auto set, int kb) {
        constexpr int P = decltype(set)::value;
#pragma unroll
        for (int i = 0; i < TM; ++i) sc[P][i] = table[(kb - kb0) % kTable * BM + (wm * 16 + l15) * TM + i];
    };
    auto read = [&](auto set, int kb) {
        constexpr int P = decltype(set)::value;
        const int slot = ((kb - kb0) % kSlots) * kStage;
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            if constexpr (kTrans)
                fw[P][j] = read_frag_tr(lds_base + static_cast<uint32_t>(slot + kABytes), (wn * WN + j * 16) / 16);
            else
                fw[P][j] = read_frag(lds + slot + kABytes + (wn * WN + j * 16) * BK);
        }
#pragma unroll
        for (int i = 0; i < TM; ++i) fa[P][i] = read_frag(lds + slot + (wm * WM + i * 16) * BK);
        read_scales(set, kb);
    };
    // Block kb from the fragments and scales of set P, while those of block kb + 1 are read into the other.
    // Nothing here is conditional: with a branch the compiler would wait for all of the reads before the
    // products.  Past the last block zeros are loaded, and what is read is not used.
    auto block = [&](auto set, int kb) {
        constexpr int P = decltype(set)::value;
        lds_done();                            // this wave's fragments of block kb are in registers
        wait_vmcnt<(kSlots - 2) * kLoads>();   // block kb + 1 has landed (later ones may be in flight) ...
        barrier();                             // ... in every wave; block kb's slot is free
        issue(kb + kSlots);
        read(std::integral_constant<int, 1 - P>{}, kb + 1);
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                const v4f d = mfma<kE5M2>(fw[P][j], fa[P][i], v4f{0.f, 0.f, 0.f, 0.f});
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[i][j][r] = __builtin_fmaf(d[r], sc[P][i], acc[i][j][r]);
            }
    };
    constexpr auto P0 = std::integral_constant<int, 0>{};
    constexpr auto P1 = std::integral_constant<int, 1>{};
#pragma unroll
    for (int s = 0; s < kSlots; ++s) issue(kb0 + s);
    fill(kb0);
    wait_vmcnt<(kSlots - 1) * kLoads>();
    lds_done();
    barrier();
    read(P0, kb0);
    for (int c0 = kb0; c0 < kb1; c0 += kTable) {
        if (c0 != kb0) {   // the next blocks' scales, once every wave has read the last of the old ones
            lds_done();
            barrier();
            fill(c0);
            lds_done();
            barrier();
            read_scales(P0, c0);
        }
        const int c1 = min(c0 + kTable, kb1);
        int kb = c0;
        for (; kb + 1 < c1; kb += 2) {
            block(P0, kb);
            block(P1, kb + 1);
        }
        if (kb < c1) block(P0, kb);
    }
    wait_vmcnt<0>();   // nothing is still writing this workgroup's LDS when another one gets it
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
    const int64_t first = static_cast<int64_t>(blockIdx.x) * 1024;
    if (n % 4 == 0) {
        const int64_t i = first + threadIdx.x * 4;
        if (i >= n) return;
        const v4f s = sum_parts<v4f>(part + i, split, n);
        if (y_bf16)
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(y) + i) = uint2{pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3])};
        else
            *reinterpret_cast<v4f*>(static_cast<float*>(y) + i) = s;
        return;
    }
    for (int64_t i = first + threadIdx.x; i < min(first + 1024, n); i += 256) {
        const float s = sum_parts<float>(part + i, split, n);
        if (y_bf16)
            static_cast<uint16_t*>(y)[i] = static_cast<uint16_t>(pack_bf16x2(s, 0.0f));
        else
            static_cast<float*>(y)[i] = s;
    }
}

// How a product runs.
enum Form : int { kSmall, kTile64, kTile128, kLarge };
struct Plan {
    Form form;
    int split;   // ranges of the reduction per tile, summed by a second kernel
};

// Measured at a reduction of 4096 (M x 4096 outputs, us):
//              M = 64      128      256      512      768      1000     1500     2048
//   64 x 64    13.0        13.4     14.0     17.8     29.0     34.7     51.9     75.6
//   128 x 128  19.9        21.1     21.4     22.2     23.2     24.3     42.9     49.3
//   256 x 256  32.5        33.1     33.1     33.4     33.5     33.4     34.8     38.9
// A tile costs its chain of stages as long as each CU has one (128: one workgroup per CU, 64: two), so the
// smallest tile whose workgroups fit at once is taken, and where none fits the largest.  Splitting the reduction shortens the chain of the 64
// x 64 tiles: in as many parts as give each CU one workgroup (64 x 1024 outputs, 4096 long: 12.3 us whole, 10.1
// in two parts, 8.0 in five; M = 128: 13.4 and 12.4 in two), or two where the parts stay long (M = 128,
// reduction of 16384: 45.0, in two 28.2, in four 22.9; of 4096: 12.4, 12.7).  The second kernel loads four
// parts beside the first at once, so five of them cost little more than two (8656 long, 23 x 697: 11.7 in five
// parts, 12.9 in eleven; 2064 long, 64 x 512: 8.5 whole, 9.4 in two).
Plan plan(int64_t M, int64_t N, int R, bool trans) {
    if (fp8_small_takes(M, N, R, trans)) return {kSmall, 1};
    auto tiles = [&](int64_t t) { return (M + t - 1) / t * ((N + t - 1) / t); };
    const int blocks = static_cast<int>(fp8_groups(R));
    const int64_t cus = device_cu_count();
    if (tiles(64) > 2 * cus) {
        if (tiles(128) <= cus) return {kTile128, 1};
        if (blocks > 1) return {kLarge, 1};   // (its loads run two stages ahead)
    }
    const int parts = blocks >= 30 ? std::max(5, blocks / 12) : blocks / 12;
    const int64_t one = std::min<int64_t>(cus / tiles(64), parts), two = std::min<int64_t>(2 * cus / tiles(64), blocks / 32);
    return {kTile64, static_cast<int>(std::clamp<int64_t>(std::max(one, two), 1, 16))};
}

template <int BT, int kWavesM, int kWavesN, int kSlots, bool kTrans, bool kE5M2>
hipError_t launch_tiles(Fp8GemmParams p, const Fp8GemmArgs& g, int split, hipStream_t stream) {
    auto kernel = g.e8m0 ? fp8_gemm_kernel<BT, BT, kWavesM, kWavesN, kSlots, kTrans, kE5M2, true>
                         : fp8_gemm_kernel<BT, BT, kWavesM, kWavesN, kSlots, kTrans, kE5M2, false>;
    constexpr int threads = 64 * kWavesM * kWavesN, lds = tile_lds<BT, BT, kSlots>();
    int per_cu = 0;
    hipError_t e = kernel_blocks_per_cu(reinterpret_cast<const void*>(kernel), threads, lds, &per_cu);
    if (e != hipSuccess) return e;
    p.tiles_m = static_cast<int>((g.M + BT - 1) / BT);
    p.tiles_n = static_cast<int>((g.N + BT - 1) / BT);
    p.split = split;
    if (g.workspace == nullptr || g.ws_bytes < static_cast<size_t>(split) * g.M * g.N * sizeof(float)) p.split = 1;
    if (p.split > 1) p.y = g.workspace;
    const int64_t total = static_cast<int64_t>(p.tiles_m) * p.tiles_n * p.split;
    kernel<<<grid_of((total + 7) / 8 * 8), threads, lds, stream>>>(p);
    e = hipGetLastError();
    if (g.parts != nullptr) *g.parts = p.split;
    if (e != hipSuccess || p.split == 1 || g.parts != nullptr) return e;
    const int64_t n = g.M * g.N;
    fp8_reduce_kernel<<<static_cast<unsigned>((n + 1023) / 1024), 256, 0, stream>>>(static_cast<const float*>(g.workspace),
                                                                                    p.split, n, g.y, g.y_bf16);
    return hipGetLastError();
}

template <bool kTrans, bool kE5M2>
hipError_t launch(const Fp8GemmArgs& g, hipStream_t stream) {
    const Fp8GemmParams p = fp8_gemm_params(g);
    const Plan how = plan(g.M, g.N, g.R, kTrans);
    if (g.parts != nullptr) *g.parts = 1;
    switch (how.form) {
        case kSmall: return launch_fp8_small(p, kTrans, kE5M2, stream);
        case kLarge: return launch_fp8_gemm_large(p, kTrans, kE5M2, stream);
        case kTile128: return launch_tiles<128, 2, 4, 4, kTrans, kE5M2>(p, g, how.split, stream);
        default: return launch_tiles<64, 2, 2, 4, kTrans, kE5M2>(p, g, how.split, stream);
    }
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
    if (M == 0) return 0;
    const int split = plan(M, N, R, trans).split;
    return split > 1 ? static_cast<size_t>(split) * M * N * sizeof(float) : 0;
}

hipError_t launch_fp8_gemm(const Fp8GemmArgs& g, hipStream_t stream) {
    if (g.trans) return g.a_e5m2 ? launch<true, true>(g, stream) : launch<true, false>(g, stream);
    return g.a_e5m2 ? launch<false, true>(g, stream) : launch<false, false>(g, stream);
}

}  // namespace rtq
