// fp8_gemm_large.hip -- the 8-bit product for outputs of many tiles: 256 x 256 outputs per
// workgroup.
//
// A workgroup of 8 waves (two per SIMD) owns 256 x 256 outputs, each wave 128 x 64 of them as 8 x 4
// tiles of v_mfma_f32_16x16x128_f8f6f4.  One LDS stage is one block of 128 along the reduction: 256
// rows x 128 bytes of each operand (64 KB), two stages.  An instruction from a zero accumulator gives a
// tile's sum over the block; its four values per lane are multiplied into the running sum by the
// block's scale four instructions later, so the vector unit works in the matrix unit's shadow (4 fp32
// multiply-adds, 16 clocks, per 32-clock instruction).  E8M0 scales go into the instruction itself
// (one byte per row of each operand), which then adds into the running sum, as if sixteen products at a time with each
// result cut off to fp32: a block may lose 2^-20 of the running sum (128 products of 2^-7 vanish beside 2^21, not 2^20).
//
// Pipeline.  Stage s + 2 is loaded into stage s's slot as soon as every wave has read its last fragments
// of stage s, which is two row tiles before that stage's end; the barrier that says so also says that
// stage s + 1 has landed, so the fragments of its first tiles are read while the last tiles of stage s
// are multiplied.  One barrier per stage.  Loads write LDS directly (no staging registers).
//
// Scales.  Each stage's 256 row scales, times the weight's two block scales, go through LDS (written by
// one thread per row a stage ahead), arranged so that a lane reads the scales of its 8 row tiles as two
// 16-byte words.
//
// Persistent: one workgroup per CU walks its tiles.  The stages of all its tiles are one stream: the last
// stages of a tile load the first ones of the next, and its epilogue runs with those in LDS.
//
// 4608 x 4096, 16384 columns: fp32 scales 284 us (2180 TFLOP/s), E8M0 250-263 us (2350-2470 TFLOP/s).  The
// matrix instructions are busy 53-58% of the time, at 1.7-1.9 GHz: the card's power sets the clock, and fewer
// clocks in the same kernel (no bank conflicts, 3% fewer) did not shorten it.
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

constexpr int kXcds = 8;
constexpr int kTileM = 256, BN = 256;
constexpr int kWavesM = 2, kWavesN = 4, kWaves = kWavesM * kWavesN, kThreads = 64 * kWaves;
constexpr int kBlocks = BN / BK;                                                            // weight scales across
constexpr int kRing = 2 * (kTileM + BN) * BK;
constexpr int kScaleBytes = 2 * kBlocks * kTileM * static_cast<int>(sizeof(float));         // [slot][column block][row]
constexpr int kStageOut = kWaves * 16 * 128;                                                // epilogue: 16 rows x 128 bytes a wave
constexpr int kLds = kRing + kScaleBytes + kStageOut;

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
// The same value, computed again where it is used: what a tile's ends derive from it is then not kept in
// registers through the K loop, which has none to spare.
__device__ __forceinline__ int again(int v) {
    asm volatile("" : "+v"(v));
    return v;
}

struct LargeParams {
    Fp8GemmParams g;
    int full;      // tiles [0, full) are taken whole; the rest as two halves of their rows
};

// Tiles of BM rows: kTileM, or half of that.
template <int BM, bool kTrans, bool kE5M2, bool kE8M0>
__device__ __forceinline__ void large_tiles(const LargeParams& lp, uint8_t* lds, int first, int end, int stride) {
    constexpr int WM = BM / kWavesM, TM = WM / 16, WN = BN / kWavesN, TN = WN / 16;
    static_assert(TN == 4, "the transposing read's addresses");
    constexpr int kABytes = BM * BK, kStage = kABytes + BN * BK;
    constexpr int kALoads = BM / 8 / kWaves, kWLoads = BN / 8 / kWaves;   // 1 KB loads per wave
    constexpr int kHalves = kTileM / BM;                                  // tiles of BM rows per whole tile
    static_assert(TM % 2 == 0 && TM >= 4, "row tiles");
    const Fp8GemmParams& p = lp.g;
    const uint32_t lds_base = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(lds));
    float* s_scale = reinterpret_cast<float*>(lds + kRing);

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / kWavesN, wn = wave % kWavesN;
    const int g = lane >> 4, l15 = lane & 15;
    const int nk = (p.R + BK - 1) / BK;

    if (first >= end) return;
    auto place = [&](int lin, int64_t* m0, int64_t* n0) {
        int tm, tn;
        tile_of(lin / kHalves, p.tiles_m, p.tiles_n, &tm, &tn);
        *m0 = static_cast<int64_t>(tm) * kTileM + (lin % kHalves) * BM;
        *n0 = static_cast<int64_t>(tn) * BN;
    };
    // The loads run two stages ahead of the products, over the ends of tiles: their own tile and block.
    // Past the last tile the descriptors are empty, and loads give zeros that nothing uses.
    int c_kb = 0;
    int64_t c_m0 = 0, c_n0 = 0;
    uint32_t c_mask = 0u;
    v4i rsa, rsw;
    auto set_cursor = [&](int lin) {
        const bool any = lin < end;
        if (any) place(lin, &c_m0, &c_n0);
        c_kb = 0;
        c_mask = any ? ~0u : 0u;
        const int rows_a = any ? static_cast<int>(max<int64_t>(0, min<int64_t>(BM, p.M - c_m0))) : 0;
        const int rows_w = any ? static_cast<int>(min<int64_t>(BN, p.N - c_n0)) : 0;
        rsa = make_rsrc(p.a + c_m0 * p.R, static_cast<uint32_t>(rows_a) * static_cast<uint32_t>(p.R));
        rsw = make_rsrc(p.w + (kTrans ? c_n0 : c_n0 * p.R), static_cast<uint32_t>(rows_w) * static_cast<uint32_t>(p.R));
    };

    // Load geometry.  Instruction q of wave w fills LDS rows 8 (8 q + w) .. +8 of an operand (128 bytes
    // each), lane L the 16 bytes at 16 L; chunk c of row r sits at c ^ ((r >> 1) & 7).  Lane group g holds
    // chunks g and g + 4 of its row (any order serves, if both operands have it).  A 16-byte LDS read
    // takes 16 lanes at a time, 8 of them from one lane group and 8 of the next (0-3, 12-15 and 20-27 are
    // the first 16): with chunks g and g + 1 their rows' places fall on all 64 banks once.
    // Transposed weights: rows of BN bytes (one n), chunk c of row r at c ^ tr_swizzle(r).
    const int kcol = ((lane & 7) ^ ((4 * wave + (lane >> 4)) & 7)) << 4;
    const uint32_t a_off = static_cast<uint32_t>((8 * wave + (lane >> 3)) * p.R + kcol);
    constexpr int kTrRows = 1024 / BN;   // LDS rows of a load of transposed weights
    const int tr_row = kTrRows * wave + lane * 16 / BN;
    const uint32_t w_off = kTrans ? static_cast<uint32_t>(tr_row * static_cast<int>(p.N) +
                                                          (((lane % (BN / 16)) ^ tr_swizzle<BN>(tr_row)) << 4))
                                  : a_off;
    const uint32_t a_step = static_cast<uint32_t>(8 * kWaves * p.R);                                // rows q -> q + 1
    const uint32_t w_step = kTrans ? static_cast<uint32_t>(kTrRows * kWaves) * static_cast<uint32_t>(p.N) : a_step;
    static_assert(kTrRows * kWaves % 32 == 0, "a lane's rows differ by what the swizzle does not see");
    const uint32_t wave_lds = static_cast<uint32_t>(wave * 1024);

    // The stage's scales: thread t holds row t % BM's scale and, for its wave's column block, the
    // weight's, until they are written to LDS (with 128 rows, threads 256.. write the same again).
    const int s_row = tid % WM, s_cb = tid / BM % kBlocks;
    const int s_at = s_cb * kTileM + ((tid % BM / WM) * 16 + (s_row & 15)) * TM + (s_row >> 4);
    constexpr int kScaleSize = kE8M0 ? 1 : 4;
    uint32_t r_a = 0u, r_w = 0u;   // as loaded: converting them here would wait for the loads just issued
    auto load_scales = [&]() {
        const int m = static_cast<int>(min<int64_t>(c_m0 + tid % BM, p.M - 1));
        const int c = static_cast<int>(min<int64_t>(c_n0 / BK + s_cb, (p.N - 1) / BK));
        const uint8_t* sa = static_cast<const uint8_t*>(p.a_scale) + static_cast<int64_t>(c_kb) * p.M * kScaleSize;
        const uint8_t* sw = static_cast<const uint8_t*>(p.w_scale) + (c * p.w_out_stride + c_kb * p.w_red_stride) * kScaleSize;
        r_a = load_raw<kE8M0>(sa, m);
        r_w = load_raw<kE8M0>(sw, 0);
    };
    auto write_scales = [&](int slot) {
        if constexpr (kE8M0)   // both bytes, for the matrix instruction
            reinterpret_cast<uint16_t*>(s_scale)[slot * kBlocks * kTileM + s_at] = static_cast<uint16_t>(r_a | r_w << 8);
        else
            s_scale[slot * kBlocks * kTileM + s_at] = __uint_as_float(r_a) * __uint_as_float(r_w);
    };
    auto issue = [&](int slot) {   // the cursor's stage, and the cursor moves on
        const int kb = c_kb;
        const uint32_t base = lds_base + static_cast<uint32_t>(slot * kStage) + wave_lds;
        // past the row's end: an offset that every descriptor refuses (loads then give zeros)
        const uint32_t k0 = kb * BK + kcol < p.R ? static_cast<uint32_t>(kb * BK) : kOob;
#pragma unroll
        for (int q = 0; q < kALoads; ++q) load_to_lds(rsa, a_off + q * a_step + k0, base + q * kWaves * 1024);
        if constexpr (kTrans) {
            // the block's rows from column c_n0 on; an empty descriptor stays empty
            const int rows = min(BK, p.R - kb * BK);
            rsw = make_rsrc(p.w + static_cast<int64_t>(kb) * BK * p.N + c_n0,
                            (static_cast<uint32_t>(rows) * static_cast<uint32_t>(p.N) - static_cast<uint32_t>(c_n0)) & c_mask);
        }
#pragma unroll
        for (int q = 0; q < kWLoads; ++q)
            load_to_lds(rsw, w_off + q * w_step + (kTrans ? 0u : k0), base + kABytes + q * kWaves * 1024);
        load_scales();
        ++c_kb;
    };

    const uint32_t f0 = static_cast<uint32_t>(l15 * BK + ((g ^ (l15 >> 1)) << 4));
    const uint32_t f1 = static_cast<uint32_t>(l15 * BK + (((g + 4) ^ (l15 >> 1)) << 4));
    const uint32_t tr0 = lds_base + static_cast<uint32_t>(kABytes + (16 * g + (l15 >> 1)) * BN +
                                                          (((4 * wn) ^ tr_swizzle<BN>(16 * g + (l15 >> 1))) << 4) + (lane & 1) * 8);
    auto read_rows = [&](const uint8_t* base) {
        const v4i x = *reinterpret_cast<const v4i*>(base + f0), y = *reinterpret_cast<const v4i*>(base + f1);
        return v8i{x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
    };
    auto read_a = [&](int slot, int i) { return read_rows(lds + slot * kStage + (wm * WM + i * 16) * BK); };
    auto read_w = [&](int slot, int j) {
        if constexpr (kTrans) {
            // rows 16 g + r, + 8, + 64, + 72 (r = l15 / 2), chunk (4 wn + j) ^ tr_swizzle: the rows' swizzle is
            // one and j two bits of the first address, so one register serves all of them
            const uint32_t base = (tr0 + static_cast<uint32_t>(slot * kStage)) ^ static_cast<uint32_t>(j << 4);
            const v2i r[4] = {read_tr8(base), read_tr8(base + 8 * BN), read_tr8(base + 64 * BN), read_tr8(base + 72 * BN)};
            return v8i{r[0].x, r[0].y, r[1].x, r[1].y, r[2].x, r[2].y, r[3].x, r[3].y};
        } else {
            return read_rows(lds + slot * kStage + kABytes + (wn * WN + j * 16) * BK);
        }
    };

    v4f acc[TM][TN];
    v8i fw[TN], fa[2];
    // fp32 scales: the sums of the row tile multiplied last, its scales, and the one carried over the
    // stage's end.  E8M0: the bytes of two row tiles and the weight a word, this stage's and the next's.
    v4f d[TN];
    float sc[TM], s_last = 0.f;
    uint32_t eb[TM / 2], eb_next[TM / 2];
    const int s_mine = (wn / 2) * kTileM + (wm * 16 + l15) * TM;
    auto read_scales = [&](int slot) {
        if constexpr (kE8M0) {
            const uint32_t* q = reinterpret_cast<const uint32_t*>(reinterpret_cast<const uint16_t*>(s_scale) + slot * kBlocks * kTileM + s_mine);
#pragma unroll
            for (int i = 0; i < TM / 2; ++i) eb_next[i] = q[i];
        } else {
            const v4f* q = reinterpret_cast<const v4f*>(s_scale + slot * kBlocks * kTileM + s_mine);
#pragma unroll
            for (int i = 0; i < TM / 4; ++i) {
                const v4f x = q[i];
                sc[4 * i] = x[0];
                sc[4 * i + 1] = x[1];
                sc[4 * i + 2] = x[2];
                sc[4 * i + 3] = x[3];
            }
        }
    };
    auto add = [&](v4f& a, const v4f& x, float s) {
#pragma unroll
        for (int r = 0; r < 4; ++r) a[r] = __builtin_fmaf(x[r], s, a[r]);
    };

    // One stage, from `slot`.  What it reads ahead is the next stage of this tile or of the next one; behind
    // the last stage of all that is whatever the other slot holds, and is not used.
    auto stage = [&](int slot) {
        if constexpr (kE8M0) {
#pragma unroll
            for (int i = 0; i < TM / 2; ++i) eb[i] = eb_next[i];
        }
#pragma unroll
        for (int i = 0; i < TM; ++i) {
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                if constexpr (kE8M0) {
                    const int e = static_cast<int>(eb[i / 2]);
                    acc[i][j] = i % 2 == 0 ? mfma_scaled<kE5M2, 0>(fw[j], fa[0], acc[i][j], e)
                                           : mfma_scaled<kE5M2, 2>(fw[j], fa[1], acc[i][j], e);
                } else {
                    // the sums of the row tile before this one, four instructions old
                    if (i == 0)
                        add(acc[TM - 1][j], d[j], s_last);
                    else
                        add(acc[i - 1][j], d[j], sc[i - 1]);
                    d[j] = mfma<kE5M2>(fw[j], fa[i & 1], v4f{0.f, 0.f, 0.f, 0.f});
                }
                if (i == TM - 1) fw[j] = read_w(1 - slot, j);
            }
            if (i == 0 && !kE8M0) read_scales(slot);
            if (i + 2 < TM) fa[i & 1] = read_a(slot, i + 2);
            if (i == TM - 2) {
                lds_done();          // this wave's last fragments of the stage are in registers
                wait_vmcnt<0>();     // its part of the next stage, and that stage's scales, have landed
                write_scales(1 - slot);
                lds_done();
                barrier();
                issue(slot);
                fa[0] = read_a(1 - slot, 0);
                if constexpr (kE8M0) read_scales(1 - slot);
            }
            if (i == TM - 1) fa[1] = read_a(1 - slot, 1);
            __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (!kE8M0) s_last = sc[TM - 1];
    };

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
        s_last = 0.f;
        // nk - 2 stages that load this tile's, then two that load the next tile's (the compiler keeps the
        // stage one basic block, whose registers just suffice, if nothing in it branches)
        for (int half = 0; half < 2; ++half) {
            for (int s = half == 0 ? nk - 2 : 2; s > 0; --s) {
                stage(slot);
                slot = 1 - slot;
            }
            if (half == 0) set_cursor(lin + stride);
        }
        if constexpr (!kE8M0) {
#pragma unroll
            for (int j = 0; j < TN; ++j) add(acc[TM - 1][j], d[j], s_last);
        }
        int64_t m0, n0;
        place(lin, &m0, &n0);
        const int64_t cm0 = m0 + wm * WM, cn0 = n0 + wn * WN;
        // Epilogue: 16 rows at a time through the wave's 2 KB of LDS (128 bytes a row, chunk c of row r at
        // c ^ (r & 7)), so that the streaming stores write whole runs of 128 bytes.
        const int lane_e = again(tid) & 63, g = lane_e >> 4, l15 = lane_e & 15;
        uint8_t* stg = lds + kRing + kScaleBytes + wave * 2048;
        const int rr = lane_e >> 3, rc = lane_e & 7;
        const bool vec = p.N % (p.y_bf16 ? 8 : 4) == 0;
        if (p.y_bf16) {
#pragma unroll
            for (int i = 0; i < TM; ++i) {
#pragma unroll
                for (int j = 0; j < TN; ++j)
                    *reinterpret_cast<uint2*>(stg + l15 * 128 + (((2 * j + (g >> 1)) ^ (l15 & 7)) << 4) + (g & 1) * 8) =
                        uint2{pack_bf16x2(acc[i][j][0], acc[i][j][1]), pack_bf16x2(acc[i][j][2], acc[i][j][3])};
                lds_done();
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int row = rr + 8 * h;
                    const uint8_t* q = stg + row * 128 + ((rc ^ (row & 7)) << 4);
                    const v4i x = *reinterpret_cast<const v4i*>(q);
                    const int64_t m = cm0 + i * 16 + row, n = cn0 + rc * 8;
                    if (m < p.M && n < p.N) {
                        uint16_t* y = static_cast<uint16_t*>(p.y) + m * p.N + n;
                        if (vec) {
                            __builtin_nontemporal_store(x, reinterpret_cast<v4i*>(y));
                        } else {
#pragma unroll 1
                            for (int e = 0; e < 8 && n + e < p.N; ++e) y[e] = reinterpret_cast<const uint16_t*>(q)[e];
                        }
                    }
                }
                lds_done();
            }
        } else {
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int hj = 0; hj < TN / 2; ++hj) {
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        *reinterpret_cast<v4f*>(stg + l15 * 128 + (((4 * j + g) ^ (l15 & 7)) << 4)) = acc[i][2 * hj + j];
                    lds_done();
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int row = rr + 8 * h;
                        const uint8_t* q = stg + row * 128 + ((rc ^ (row & 7)) << 4);
                        const v4f x = *reinterpret_cast<const v4f*>(q);
                        const int64_t m = cm0 + i * 16 + row, n = cn0 + hj * 32 + rc * 4;
                        if (m < p.M && n < p.N) {
                            float* y = static_cast<float*>(p.y) + m * p.N + n;
                            if (vec) {
                                __builtin_nontemporal_store(x, reinterpret_cast<v4f*>(y));
                            } else {
#pragma unroll 1
                                for (int e = 0; e < 4 && n + e < p.N; ++e) y[e] = reinterpret_cast<const float*>(q)[e];
                            }
                        }
                    }
                    lds_done();
                }
        }
    }
    wait_vmcnt<0>();   // nothing is still writing LDS when the workgroup's next tiles, or another workgroup, use it
}

template <bool kTrans, bool kE5M2, bool kE8M0>
__global__ void __launch_bounds__(kThreads, 1)
fp8_gemm_large_kernel(LargeParams p) {
    extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
    // Tiles are split into 8 contiguous ranges, one per XCD (block b runs on XCD b % 8); the blocks of an
    // XCD walk their range together, in bands of 8 N-tiles, and share operand panels in that L2.
    const int xcd = blockIdx.x % kXcds, local = blockIdx.x / kXcds, stride = gridDim.x / kXcds;
    const int per = (p.full + kXcds - 1) / kXcds;
    large_tiles<kTileM, kTrans, kE5M2, kE8M0>(p, lds, xcd * per + local, min((xcd + 1) * per, p.full), stride);
    const int rest = 2 * (p.g.tiles_m * p.g.tiles_n - p.full), rper = (rest + kXcds - 1) / kXcds;
    if (rest > 0) {
        __syncthreads();
        const int r0 = 2 * p.full;
        large_tiles<kTileM / 2, kTrans, kE5M2, kE8M0>(p, lds, r0 + xcd * rper + local, r0 + min((xcd + 1) * rper, rest), stride);
    }
}

template <bool kTrans, bool kE5M2, bool kE8M0>
hipError_t launch(const Fp8GemmParams& g, hipStream_t stream) {
    auto kernel = fp8_gemm_large_kernel<kTrans, kE5M2, kE8M0>;
    int per_cu = 0;
    hipError_t e = kernel_blocks_per_cu(reinterpret_cast<const void*>(kernel), kThreads, kLds, &per_cu);
    if (e != hipSuccess) return e;
    LargeParams p{};
    p.g = g;
    p.g.tiles_m = static_cast<int>((g.M + kTileM - 1) / kTileM);
    p.g.tiles_n = static_cast<int>((g.N + BN - 1) / BN);
    const int cus = std::max(kXcds, device_cu_count() / kXcds * kXcds);
    // whole rounds of whole tiles; a remainder that fills at most half a round goes as halves of 128 rows (4608 x
    // 4096 x 4096, a round and an eighth: 90 us, 105 without)
    const int total = p.g.tiles_m * p.g.tiles_n, rest = total % cus;
    p.full = rest > 0 && rest <= cus / 2 ? total - rest : total;
    kernel<<<cus, kThreads, kLds, stream>>>(p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_fp8_gemm_large(const Fp8GemmParams& g, bool trans, bool e5m2, hipStream_t stream) {
    auto pick = [&](auto t, auto f) {
        constexpr bool kT = decltype(t)::value, kF = decltype(f)::value;
        return g.e8m0 ? launch<kT, kF, true>(g, stream) : launch<kT, kF, false>(g, stream);
    };
    constexpr auto yes = std::true_type{};
    constexpr auto no = std::false_type{};
    if (trans) return e5m2 ? pick(yes, yes) : pick(yes, no);
    return e5m2 ? pick(no, yes) : pick(no, no);
}

}  // namespace rtq
