// fp8_glu_large.hip -- the gated feed-forward's product for many tokens and channels: y = f(g) u, [g u] = x W^T, with 256
// tokens by 128 channels per workgroup, their codes and scales made from the sums in registers.
//
// The product is the large one's (fp8_gemm_large.hip): 8 waves, each 128 x 64 sums in 8 x 4 tiles of
// v_mfma_f32_16x16x128_f8f6f4, one block of 128 of the reduction a stage, two stages in LDS, loaded straight into it two
// stages ahead over the ends of tiles, persistent workgroups.  What differs:
//
//   - The 256 weight rows of a stage are 128 of the gate and the same 128 channels' of the other projection, laid so that
//     a wave's column tiles 0 and 1 are 32 channels' gates and 2 and 3 their partners: g and u of a channel and token meet
//     in one lane.
//   - A wave needs two weight scales a stage.  E8M0, applied inside the instruction: four rows' bytes a register, the two weights'
//     bytes in one, chosen by the instruction.  fp32, applied outside: the row's scale and the two factors are read apart
//     and multiplied when used (two multiplies a row tile; tables of both products would take eight more registers, and
//     there are none).  4608 x 4096, 16384 channels: to codes 506 us with E8M0 scales, 562 with fp32; with the checkpoint 533
//     and 593.  fp32 scales that happen to be powers of two stay outside all the same: the instruction cuts up to 2^-20 of the
//     running sum off with each block that it adds, and an output's bits would go by its neighbours' scales.
//   - The outputs (glu_outputs), two or four row tiles at a time: f(g) u fits beside the sums, and the LDS that is left holds
//     their codes.
//
// Without the fusion [g u] would be written and read again in fp32: 4608 x 4096 -> 2 x 16384, 1.2 GB.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "fp8_glu.h"
#include "fp8_internal.h"
#include "rtq_internal.h"

namespace rtq {
namespace {

using namespace fp8;

constexpr int kXcds = 8;
constexpr int kTileM = 256, kChannels = 128, BN = 2 * kChannels;
constexpr int kWavesM = 2, kWavesN = 4, kWaves = kWavesM * kWavesN, kThreads = 64 * kWaves;
constexpr int kRing = 2 * (kTileM + BN) * BK;
constexpr int kSlotScales = kTileM + 2 * 64;                                       // tokens', then 64 copies of the two weights'
constexpr int kScaleBytes = 2 * kSlotScales * static_cast<int>(sizeof(float));
constexpr int kLds = kRing + kScaleBytes + kGluStage + kGluScales;

// Tile index within the XCD-ordered sequence -> (tile_m, tile_n), in bands of 8 N-tiles.
__device__ __forceinline__ void tile_of(int lin, int tiles_m, int tiles_n, int* tm, int* tn) {
    constexpr int kBand = 8;
    const int band = lin / (kBand * tiles_m);
    const int in_band = lin % (kBand * tiles_m);
    const int band_w = min(kBand, tiles_n - band * kBand);
    *tm = in_band / band_w;
    *tn = band * kBand + in_band % band_w;
}

template <bool kE8M0>
__device__ __forceinline__ uint32_t load_raw(const void* s, int64_t i) {
    return kE8M0 ? static_cast<const uint8_t*>(s)[i] : static_cast<const uint32_t*>(s)[i];
}
// The same value, computed again where it is used, so that the K loop keeps no register for it.
__device__ __forceinline__ int again(int v) {
    asm volatile("" : "+v"(v));
    return v;
}

struct LargeParams {
    GluParams g;
    int full;      // tiles [0, full) are taken whole; the rest as two halves of their tokens
};

// Tiles of BM tokens: kTileM, or half of that.
template <int BM, bool kE8M0>
__device__ __forceinline__ void large_tiles(const LargeParams& lp, uint8_t* lds, int first, int end, int stride) {
    constexpr int WM = BM / kWavesM, TM = WM / 16, TN = 4;
    constexpr int kABytes = BM * BK, kStage = kABytes + BN * BK;
    constexpr int kALoads = BM / 8 / kWaves, kWLoads = BN / 8 / kWaves;   // 1 KB loads per wave
    constexpr int kHalves = kTileM / BM;                                  // tiles of BM tokens per whole tile
    static_assert(TM == 4 || TM == 8, "row tiles");
    const GluParams& p = lp.g;
    const uint32_t lds_base = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(lds));
    using Scale = std::conditional_t<kE8M0, uint8_t, float>;
    Scale* s_scale = reinterpret_cast<Scale*>(lds + kRing);               // [slot][kSlotScales]

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / kWavesN, wn = wave % kWavesN;
    const int g = lane >> 4, l15 = lane & 15;
    const int nk = (p.K + BK - 1) / BK;

    if (first >= end) return;
    auto place = [&](int lin, int64_t* m0, int* n0) {
        int tm, tn;
        tile_of(lin / kHalves, p.tiles_t, p.tiles_n, &tm, &tn);
        *m0 = static_cast<int64_t>(tm) * kTileM + (lin % kHalves) * BM;
        *n0 = tn * kChannels;
    };
    // The loads run two stages ahead of the products, over the ends of tiles: their own tile and block.  Past the last
    // tile the descriptors are empty, and loads give zeros that nothing uses.
    int c_kb = 0, c_n0 = 0;
    int64_t c_m0 = 0;
    v4i rsa, rsw;
    const int second = wave >= kWaves / 2 ? 1 : 0;   // this wave loads the other projection's rows
    auto set_cursor = [&](int lin) {
        const bool any = lin < end;
        if (any) place(lin, &c_m0, &c_n0);
        c_kb = 0;
        const int rows_a = any ? static_cast<int>(max<int64_t>(0, min<int64_t>(BM, p.T - c_m0))) : 0;
        const int rows_w = any ? kChannels : 0;
        rsa = make_rsrc(p.x + c_m0 * p.K, static_cast<uint32_t>(rows_a) * static_cast<uint32_t>(p.K));
        rsw = make_rsrc(p.w + (static_cast<int64_t>(second) * p.N + c_n0) * p.K, static_cast<uint32_t>(rows_w) * static_cast<uint32_t>(p.K));
    };

    // Load geometry as in the large product: instruction q of wave w fills LDS rows 8 (8 q + w) .. +8 of an operand, lane L
    // the 16 bytes at 16 L; chunk c of row r sits at c ^ ((r >> 1) & 7).  LDS weight row 64 q + 16 j + l is channel
    // 32 q + 16 (j % 2) + l of the gate (j < 2) or of its partner.
    const int kcol = ((lane & 7) ^ ((4 * wave + (lane >> 4)) & 7)) << 4;
    const uint32_t a_off = static_cast<uint32_t>((8 * wave + (lane >> 3)) * p.K + kcol);
    const uint32_t w_off = static_cast<uint32_t>((8 * (wave % (kWaves / 2)) + (lane >> 3)) * p.K + kcol);
    const uint32_t a_step = static_cast<uint32_t>(8 * kWaves * p.K), w_step = a_step / 2;   // rows q -> q + 1
    const uint32_t wave_lds = static_cast<uint32_t>(wave * 1024);

    // The stage's scales, written to LDS a stage ahead: thread t's are those of token t % BM, where a lane reads its row
    // tiles' in one run, and of the gate's block (t < 256) or its partner's, next to each other.  (Several threads write the
    // same value to the same place: without a branch.)
    const int s_row = tid % WM;
    const int s_at = (tid % BM / WM * 16 + (s_row & 15)) * TM + (s_row >> 4);
    const int s_wat = kTileM + tid % 64 * 2 + tid / 256;
    constexpr int kScaleSize = kE8M0 ? 1 : 4;
    uint32_t r_a = 0u, r_w = 0u;   // as loaded: converting them here would wait for the loads just issued
    auto load_scales = [&]() {
        const int m = static_cast<int>(min<int64_t>(c_m0 + tid % BM, p.T - 1));
        const uint8_t* sa = static_cast<const uint8_t*>(p.x_scale) + static_cast<int64_t>(c_kb) * p.T * kScaleSize;
        const uint8_t* sw = static_cast<const uint8_t*>(p.w_scale) +
                            (static_cast<int64_t>((second * p.N + c_n0) / kFp8Block) * nk + c_kb) * kScaleSize;
        r_a = load_raw<kE8M0>(sa, m);
        r_w = load_raw<kE8M0>(sw, 0);
    };
    auto write_scales = [&](int slot) {
        if constexpr (kE8M0) {
            s_scale[slot * kSlotScales + s_at] = static_cast<uint8_t>(r_a);
            s_scale[slot * kSlotScales + s_wat] = static_cast<uint8_t>(r_w);
        } else {
            s_scale[slot * kSlotScales + s_at] = __uint_as_float(r_a);
            s_scale[slot * kSlotScales + s_wat] = __uint_as_float(r_w);
        }
    };
    auto issue = [&](int slot) {   // the cursor's stage, and the cursor moves on
        const int kb = c_kb;
        const uint32_t base = lds_base + static_cast<uint32_t>(slot * kStage) + wave_lds;
        // past the row's end: an offset that every descriptor refuses (loads then give zeros)
        const uint32_t k0 = kb * BK + kcol < p.K ? static_cast<uint32_t>(kb * BK) : kOob;
#pragma unroll
        for (int q = 0; q < kALoads; ++q) load_to_lds(rsa, a_off + q * a_step + k0, base + q * kWaves * 1024);
#pragma unroll
        for (int q = 0; q < kWLoads; ++q) load_to_lds(rsw, w_off + q * w_step + k0, base + kABytes + q * kWaves * 1024);
        load_scales();
        ++c_kb;
    };

    const uint32_t f0 = static_cast<uint32_t>(l15 * BK + ((g ^ (l15 >> 1)) << 4));
    const uint32_t f1 = static_cast<uint32_t>(l15 * BK + (((g + 4) ^ (l15 >> 1)) << 4));
    auto read_rows = [&](const uint8_t* base) {
        const v4i x = *reinterpret_cast<const v4i*>(base + f0), y = *reinterpret_cast<const v4i*>(base + f1);
        return v8i{x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
    };
    auto read_a = [&](int slot, int i) { return read_rows(lds + slot * kStage + (wm * WM + i * 16) * BK); };
    auto read_w = [&](int slot, int j) { return read_rows(lds + slot * kStage + kABytes + (wn * 64 + j * 16) * BK); };

    v4f acc[TM][TN];
    v8i fw[TN], fa[2];
    // Scales outside: the sums of the row tile multiplied last, the tokens' scales, the two weights', and the products
    // carried over the stage's end.  Inside: four row tiles' bytes a word, this stage's and the next's.
    v4f d[TN];
    float sc[TM], sw[2], last[2] = {0.f, 0.f};
    uint32_t eb[TM / 4], eb_next[TM / 4], ew = 0u, ew_next = 0u;
    auto read_scales = [&](int slot) {
        const Scale* q = s_scale + slot * kSlotScales;
        if constexpr (kE8M0) {
#pragma unroll
            for (int i = 0; i < TM / 4; ++i) eb_next[i] = reinterpret_cast<const uint32_t*>(q + (wm * 16 + l15) * TM)[i];
            ew_next = *reinterpret_cast<const uint16_t*>(q + kTileM);
        } else {
#pragma unroll
            for (int i = 0; i < TM / 4; ++i) {
                const v4f x = reinterpret_cast<const v4f*>(q + (wm * 16 + l15) * TM)[i];
                sc[4 * i] = x[0];
                sc[4 * i + 1] = x[1];
                sc[4 * i + 2] = x[2];
                sc[4 * i + 3] = x[3];
            }
            sw[0] = q[kTileM];
            sw[1] = q[kTileM + 1];
        }
    };
    auto add = [&](v4f& a, const v4f& x, float s) {
#pragma unroll
        for (int r = 0; r < 4; ++r) a[r] = __builtin_fmaf(x[r], s, a[r]);
    };
    // E8M0: the scaled product of row tile i and column tile j
    auto scaled = [&](auto ic, auto jc) {
        constexpr int i = decltype(ic)::value, j = decltype(jc)::value;
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fw[j], fa[i & 1], acc[i][j], 0, 0, j / 2, static_cast<int>(ew),
                                                                     i % 4, static_cast<int>(eb[i / 4]));
    };

    // One stage, from `slot`.  What it reads ahead is the next stage of this tile or of the next one; behind the last
    // stage of all that is whatever the other slot holds, and is not used.
    auto stage = [&](int slot) {
        if constexpr (kE8M0) {
#pragma unroll
            for (int i = 0; i < TM / 4; ++i) eb[i] = eb_next[i];
            ew = ew_next;
        }
        auto row = [&](auto ic) {
            constexpr int i = decltype(ic)::value;
            float s[2] = {0.f, 0.f};
            if constexpr (!kE8M0) {
                s[0] = i == 0 ? last[0] : sc[i == 0 ? 0 : i - 1] * sw[0];
                s[1] = i == 0 ? last[1] : sc[i == 0 ? 0 : i - 1] * sw[1];
            }
            auto column = [&](auto jc) {
                constexpr int j = decltype(jc)::value;
                if constexpr (kE8M0) {
                    scaled(ic, jc);
                } else {
                    // the sums of the row tile before this one, four instructions old
                    add(acc[i == 0 ? TM - 1 : i - 1][j], d[j], s[j / 2]);
                    d[j] = mfma<false>(fw[j], fa[i & 1], v4f{0.f, 0.f, 0.f, 0.f});
                }
                if constexpr (i == TM - 1) fw[j] = read_w(1 - slot, j);
            };
            column(std::integral_constant<int, 0>{});
            column(std::integral_constant<int, 1>{});
            column(std::integral_constant<int, 2>{});
            column(std::integral_constant<int, 3>{});
            if constexpr (i == 0 && !kE8M0) read_scales(slot);
            if constexpr (i + 2 < TM) fa[i & 1] = read_a(slot, i + 2);
            if constexpr (i == TM - 2) {
                lds_done();          // this wave's last fragments of the stage are in registers
                wait_vmcnt<0>();     // its part of the next stage, and that stage's scales, have landed
                write_scales(1 - slot);
                lds_done();
                barrier();
                issue(slot);
                fa[0] = read_a(1 - slot, 0);
                if constexpr (kE8M0) read_scales(1 - slot);
            }
            if constexpr (i == TM - 1) fa[1] = read_a(1 - slot, 1);
            __builtin_amdgcn_sched_barrier(0);
        };
        row(std::integral_constant<int, 0>{});
        row(std::integral_constant<int, 1>{});
        row(std::integral_constant<int, 2>{});
        row(std::integral_constant<int, 3>{});
        if constexpr (TM == 8) {
            row(std::integral_constant<int, TM - 4>{});
            row(std::integral_constant<int, TM - 3>{});
            row(std::integral_constant<int, TM - 2>{});
            row(std::integral_constant<int, TM - 1>{});
        }
        if constexpr (!kE8M0) {
            last[0] = sc[TM - 1] * sw[0];
            last[1] = sc[TM - 1] * sw[1];
        }
    };

    GluLds out_lds{lds + kRing + kScaleBytes, reinterpret_cast<uint32_t*>(lds + kRing + kScaleBytes + kGluStage)};
    if (tid < 2 * kGluSet) out_lds.scales[tid] = 0u;
    set_cursor(first);
    issue(0);
    wait_vmcnt<0>();
    write_scales(0);
    issue(1);
    lds_done();
    barrier();
#pragma unroll
    for (int j = 0; j < TN; ++j) fw[j] = read_w(0, j);
    fa[0] = read_a(0, 0);
    fa[1] = read_a(0, 1);
    if constexpr (kE8M0) read_scales(0);
    int slot = 0;
    for (int lin = first; lin < end; lin += stride) {
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            d[j] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < TM; ++i) acc[i][j] = d[j];
        }
        last[0] = last[1] = 0.f;
        // nk - 2 stages that load this tile's, then two that load the next tile's (the stage stays one basic block)
        for (int half = 0; half < 2; ++half) {
            for (int s = half == 0 ? nk - 2 : 2; s > 0; --s) {
                stage(slot);
                slot = 1 - slot;
            }
            if (half == 0) set_cursor(lin + stride);
        }
        if constexpr (!kE8M0) {
#pragma unroll
            for (int j = 0; j < TN; ++j) add(acc[TM - 1][j], d[j], last[j / 2]);
        }
        int64_t m0;
        int n0;
        place(lin, &m0, &n0);
        glu_tile_outputs<WM, kE8M0>(p, acc, m0, n0, wm, wn, again(tid), out_lds);
    }
    wait_vmcnt<0>();   // nothing is still writing LDS when the workgroup's next tiles, or another workgroup, use it
}

template <bool kE8M0>
__global__ void __launch_bounds__(kThreads, 1)
glu_large_kernel(LargeParams p) {
    extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
    // Tiles are split into 8 contiguous ranges, one per XCD (block b runs on XCD b % 8); the blocks of an XCD walk their
    // range together, in bands of 8 N-tiles, and share operand panels in that L2.
    const int xcd = blockIdx.x % kXcds, local = blockIdx.x / kXcds, stride = gridDim.x / kXcds;
    const int per = (p.full + kXcds - 1) / kXcds;
    const int first = xcd * per + local, end = min((xcd + 1) * per, p.full);
    const int rest = 2 * (p.g.tiles_t * p.g.tiles_n - p.full), rper = (rest + kXcds - 1) / kXcds, r0 = 2 * p.full;
    const int rfirst = r0 + xcd * rper + local, rend = r0 + min((xcd + 1) * rper, rest);
    large_tiles<kTileM, kE8M0>(p, lds, first, end, stride);
    if (rest > 0) {
        __syncthreads();
        large_tiles<kTileM / 2, kE8M0>(p, lds, rfirst, rend, stride);
    }
}

}  // namespace

hipError_t launch_glu_large(const GluParams& g, bool e8m0, hipStream_t stream) {
    auto kernel = e8m0 ? glu_large_kernel<true> : glu_large_kernel<false>;
    int per_cu = 0;
    hipError_t e = kernel_blocks_per_cu(reinterpret_cast<const void*>(kernel), kThreads, kLds, &per_cu);
    if (e != hipSuccess) return e;
    LargeParams p{};
    p.g = g;
    p.g.tiles_t = static_cast<int>((g.T + kTileM - 1) / kTileM);
    p.g.tiles_n = g.N / kChannels;
    const int cus = std::max(kXcds, device_cu_count() / kXcds * kXcds);
    // whole rounds of whole tiles; a remainder that fills at most half a round goes as halves of 128 tokens
    const int total = p.g.tiles_t * p.g.tiles_n, rest = total % cus;
    p.full = rest > 0 && rest <= cus / 2 ? total - rest : total;
    kernel<<<cus, kThreads, kLds, stream>>>(p);
    return hipGetLastError();
}

}  // namespace rtq
