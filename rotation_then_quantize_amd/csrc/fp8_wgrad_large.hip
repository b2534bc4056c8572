// fp8_wgrad_large.hip -- the weight gradient from the 8-bit checkpoint for outputs of many tiles: 256 x 256
// of dw per workgroup.
//
// A workgroup of 8 waves (two per SIMD) owns 256 rows n and 256 columns k, each wave 128 x 64 of them as
// 8 x 4 tiles of v_mfma_f32_16x16x32_bf16.  One LDS stage is 64 tokens: 64 rows of 256 bf16 of dy and of
// the decoded input (64 KB), two stages.  dy is loaded into LDS directly; the codes go through registers,
// where a thread decodes 16 codes of each of two tokens (one scale per token and 128 codes) and writes them
// as bf16.  Both operands have the reduction (t) as their row: the transposing LDS read gives each lane four
// consecutive t of one column.
//
// Pipeline and schedule are those of the large product: the next stage's loads are issued as soon as every
// wave has read its last fragments of the stage whose slot they take, one barrier per stage, and the
// stages of all of a workgroup's tiles are one stream.  The codes of stage s + 1 are decoded behind the
// products of stage s.  The codes' loads stand in loops over distinct descriptors, one turn each: the compiler holds
// the descriptors' sizes in vector registers and cannot see that they are the same in all lanes.
//
// 4608 tokens, 12288 x 4096 outputs: 380-407 us, 1140-1220 TFLOP/s, its matrix instructions busy 55% of the time
// at the clock that the card's power allows.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "fp8_internal.h"
#include "fp8_tile.h"
#include "fp8_wgrad.h"
#include "rtq_internal.h"

namespace rtq {
namespace {

using namespace fp8;

constexpr int BT = 64;                          // tokens per stage
constexpr int BK2 = 256;                        // columns k per tile
constexpr int kWavesN = 2, kWavesK = 4, kWaves = kWavesN * kWavesK;
constexpr int kThreads = 64 * kWaves;
constexpr int WK = BK2 / kWavesK, TK = WK / 16;
constexpr int kXcds = 8;
constexpr int kMaxN = 256;
constexpr int kRow = 512;                       // LDS bytes of a token's 256 bf16
constexpr int kOp = BT * kRow, kStage = 2 * kOp;
constexpr int kRing = 2 * kStage;
constexpr int kLds = kRing + kWaves * 16 * 128;   // and the epilogue's 16 rows x 128 bytes a wave

// Tile index within the XCD-ordered sequence -> (tile_n, tile_k), in bands of 8 k-tiles.
__device__ __forceinline__ void tile_of(int lin, int tiles_n, int tiles_k, int* tn, int* tk) {
    constexpr int kBand = 8;
    const int band = lin / (kBand * tiles_n);
    const int in_band = lin % (kBand * tiles_n);
    const int band_w = min(kBand, tiles_k - band * kBand);
    *tn = in_band / band_w;
    *tk = band * kBand + in_band % band_w;
}

__device__ __forceinline__ int again(int v) {   // see the large product: not kept over the loop
    asm volatile("" : "+v"(v));
    return v;
}

// Rows n of a tile: 256, or 128 (a half).
template <int BN, bool kE8M0>
__device__ __forceinline__ void large_tiles(const WgradParams& p, uint8_t* lds, int first, int end, int stride) {
    constexpr int WN = BN / kWavesN, TN = WN / 16;
    constexpr int kHalves = kMaxN / BN;
    constexpr int kDyLoads = BT * BN * 2 / 1024 / kWaves;   // 1 KB loads per wave
    constexpr int kDyRow = BN * 2;                          // LDS bytes of a token's dy
    constexpr int kRowsPerLoad = 1024 / kDyRow;
    const uint32_t lds_base = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(lds));
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wn = wave / kWavesK, wk = wave % kWavesK;
    const int g = lane >> 4, l15 = lane & 15;
    const int nt = static_cast<int>((p.T + BT - 1) / BT);

    if (first >= end) return;
    auto place = [&](int lin, int* n0, int* k0) {
        int tn, tk;
        tile_of(lin / kHalves, p.tiles_n, p.tiles_k, &tn, &tk);
        *n0 = tn * kMaxN + (lin % kHalves) * BN;
        *k0 = tk * BK2;
    };
    // the loads' own tile and stage; past the last tile they load nothing
    int c_n0 = 0, c_k0 = 0, c_t = 0;
    uint32_t c_mask = 0u;
    auto set_cursor = [&](int lin) {
        const bool any = lin < end;
        if (any) place(lin, &c_n0, &c_k0);
        c_t = 0;
        c_mask = any && c_n0 < p.N ? ~0u : 0u;
    };

    // dy: instruction q of wave w fills LDS rows kRowsPerLoad (8 q + w) .. of dy, lane L the 16 bytes at 16 L.
    // The 32-byte unit u (16 columns) of row t sits at u ^ (t & 7): a transposing read takes 4 rows of one
    // unit for each of two lane groups, 8 rows in all, whose places fall on all banks once.
    const int d_row = kRowsPerLoad * wave + lane * 16 / kDyRow;
    const int d_chunk = (lane % (kDyRow / 16)) ^ ((d_row & 7) << 1);
    const uint32_t d_off = static_cast<uint32_t>(d_row) * static_cast<uint32_t>(p.N) * 2u + static_cast<uint32_t>(d_chunk * 16);
    const uint32_t d_step = static_cast<uint32_t>(kRowsPerLoad * kWaves) * static_cast<uint32_t>(p.N) * 2u;
    static_assert(kRowsPerLoad * kWaves % 8 == 0, "a lane's rows differ by multiples of 8");
    // codes: thread's tokens tid / 16 and + 32, 16 codes from 16 (tid % 16): one unit of bf16 each
    const int x_row = tid >> 4;
    const uint32_t x_off = static_cast<uint32_t>(x_row) * static_cast<uint32_t>(p.K) + static_cast<uint32_t>((tid & 15) * 16);
    const uint32_t x_put = static_cast<uint32_t>(kOp + x_row * kRow + (((tid & 15) ^ (x_row & 7)) << 5));
    v4i x_codes[2];
    uint32_t x_scale[2];
    int x_rows = 0;   // tokens that there are among the stage's: past them the scale is taken as 0 (the last token's may be
                      // infinite, and times the zeros there would be none)
    auto issue = [&](int slot) {   // the cursor's stage, and the cursor moves on
        const int64_t t0 = static_cast<int64_t>(c_t) * BT;
        const int rows = static_cast<int>(min<int64_t>(BT, p.T - t0));
        x_rows = rows;
        const uint32_t dy_bytes = (static_cast<uint32_t>(rows) * static_cast<uint32_t>(p.N) - static_cast<uint32_t>(c_n0)) * 2u;
        const uint32_t x_bytes = static_cast<uint32_t>(rows) * static_cast<uint32_t>(p.K) - static_cast<uint32_t>(c_k0);
        const __amdgpu_buffer_rsrc_t rx = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<uint8_t*>(p.x) + t0 * p.K + c_k0, (short)0, static_cast<int>(x_bytes & c_mask), kBufferWord3);
        const int kb = min(c_k0 + (tid & 15) * 16, p.K - 1) / kFp8Block;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            x_codes[h] = __builtin_amdgcn_raw_buffer_load_b128(rx, x_off + static_cast<uint32_t>(32 * h) * static_cast<uint32_t>(p.K), 0, 0);
            const int64_t at = static_cast<int64_t>(kb) * p.T + min<int64_t>(t0 + x_row + 32 * h, p.T - 1);
            if constexpr (kE8M0)
                x_scale[h] = static_cast<const uint8_t*>(p.x_scale)[at];
            else
                x_scale[h] = static_cast<const uint32_t*>(p.x_scale)[at];
        }
        const v4i rsd = make_rsrc(p.dy + t0 * p.N + c_n0, dy_bytes & c_mask);
        const uint32_t base = lds_base + static_cast<uint32_t>(slot * kStage + wave * 1024);
#pragma unroll
        for (int q = 0; q < kDyLoads; ++q) load_to_lds(rsd, d_off + q * d_step, base + q * kWaves * 1024);
        ++c_t;
    };
    auto decode = [&](int slot) {   // the codes that issue loaded last
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float raw = kE8M0 ? e8m0_value(x_scale[h]) : __uint_as_float(x_scale[h]);
            const float s = x_row + 32 * h < x_rows ? raw : 0.0f;
            uint32_t w[8];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float v[4];
                decode4<false>(static_cast<uint32_t>(x_codes[h][q]), v);
                w[2 * q] = pack_bf16x2(v[0] * s, v[1] * s);
                w[2 * q + 1] = pack_bf16x2(v[2] * s, v[3] * s);
            }
            uint8_t* at = lds + slot * kStage + x_put + 32 * h * kRow;
            *reinterpret_cast<uint4*>(at) = uint4{w[0], w[1], w[2], w[3]};
            *reinterpret_cast<uint4*>(at + 16) = uint4{w[4], w[5], w[6], w[7]};
        }
    };

    // Fragments: lane group g holds tokens 16 q + 4 g + (0..3), q = 0..3, of its column (any order serves, if
    // both operands have it); column unit u at u ^ (t & 7).
    const int r4 = l15 >> 2, swz = 4 * (g & 1) + r4;
    const uint32_t a0 = lds_base + static_cast<uint32_t>((4 * g + r4) * kDyRow + (((WN / 16 * wn) ^ swz) << 5) + (l15 & 3) * 8);
    const uint32_t w0 = lds_base + static_cast<uint32_t>(kOp + (4 * g + r4) * kRow + (((TK * wk) ^ swz) << 5) + (l15 & 3) * 8);
    auto frag = [&](uint32_t base, int pitch) {
        const v2i r[4] = {read_tr16(base), read_tr16(base + 16 * pitch), read_tr16(base + 32 * pitch), read_tr16(base + 48 * pitch)};
        return v8i{r[0].x, r[0].y, r[1].x, r[1].y, r[2].x, r[2].y, r[3].x, r[3].y};
    };
    auto read_dy = [&](int slot, int i) { return frag((a0 + static_cast<uint32_t>(slot * kStage)) ^ static_cast<uint32_t>(i << 5), kDyRow); };
    auto read_x = [&](int slot, int j) { return frag((w0 + static_cast<uint32_t>(slot * kStage)) ^ static_cast<uint32_t>(j << 5), kRow); };

    v4f acc[TN][TK];
    v8i fx[TK], fd[2];
    auto stage = [&](int slot) {
#pragma unroll
        for (int i = 0; i < TN; ++i) {
#pragma unroll
            for (int j = 0; j < TK; ++j) {
                acc[i][j] = mfma_bf16(fx[j], fd[i & 1], acc[i][j]);
                if (i == TN - 1) fx[j] = read_x(1 - slot, j);
            }
            if (i + 2 < TN) fd[i & 1] = read_dy(slot, i + 2);
            if (i == TN - 3) decode(1 - slot);
            if (i == TN - 2) {
                lds_done();          // this wave's last fragments of the stage are in registers
                wait_vmcnt<0>();     // its part of the next stage has landed
                barrier();
                issue(slot);
                fd[0] = read_dy(1 - slot, 0);
            }
            if (i == TN - 1) fd[1] = read_dy(1 - slot, 1);
            __builtin_amdgcn_sched_barrier(0);
        }
    };

    set_cursor(first);
    issue(0);
    wait_vmcnt<0>();
    decode(0);
    issue(1);
    lds_done();
    barrier();
#pragma unroll
    for (int j = 0; j < TK; ++j) fx[j] = read_x(0, j);
    fd[0] = read_dy(0, 0);
    fd[1] = read_dy(0, 1);
    int slot = 0;
    for (int lin = first; lin < end; lin += stride) {
#pragma unroll
        for (int i = 0; i < TN; ++i)
#pragma unroll
            for (int j = 0; j < TK; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
        for (int half = 0; half < 2; ++half) {   // nt - 2 stages that load this tile's, two that load the next's
            for (int s = half == 0 ? nt - 2 : 2; s > 0; --s) {
                stage(slot);
                slot = 1 - slot;
            }
            if (half == 0) set_cursor(lin + stride);
        }
        int n0, k0;
        place(lin, &n0, &k0);
        // Epilogue: 16 rows n at a time through the wave's 2 KB of LDS (128 bytes a row, chunk c of row r at
        // c ^ (r & 7)).  A lane holds row l15, columns 16 j + 4 g .. +4.
        const int lane_e = again(tid) & 63, ge = lane_e >> 4, le = lane_e & 15;
        uint8_t* stg = lds + kRing + wave * 2048;
        const int rr = lane_e >> 3, rc = lane_e & 7;
        const int cn = n0 + wn * WN, ck = k0 + wk * WK;
        const bool wide = p.dw_bf16 && !p.accumulate;   // staged as bf16, 64 columns a row
#pragma unroll
        for (int i = 0; i < TN; ++i) {
            if (wide) {
#pragma unroll
                for (int j = 0; j < TK; ++j)
                    *reinterpret_cast<uint2*>(stg + le * 128 + (((2 * j + (ge >> 1)) ^ (le & 7)) << 4) + (ge & 1) * 8) =
                        uint2{pack_bf16x2(acc[i][j][0], acc[i][j][1]), pack_bf16x2(acc[i][j][2], acc[i][j][3])};
                lds_done();
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int row = rr + 8 * h, n = cn + i * 16 + row, k = ck + rc * 8;
                    const v4i x = *reinterpret_cast<const v4i*>(stg + row * 128 + ((rc ^ (row & 7)) << 4));
                    if (n < p.N && k < p.K)   // K is a multiple of 16
                        __builtin_nontemporal_store(
                            x, reinterpret_cast<v4i*>(static_cast<uint16_t*>(p.dw) + static_cast<int64_t>(n) * p.K + k));
                }
                lds_done();
            } else {
#pragma unroll
                for (int hj = 0; hj < TK / 2; ++hj) {
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        *reinterpret_cast<v4f*>(stg + le * 128 + (((4 * j + ge) ^ (le & 7)) << 4)) = acc[i][2 * hj + j];
                    lds_done();
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int row = rr + 8 * h, n = cn + i * 16 + row, k = ck + hj * 32 + rc * 4;
                        const v4f x = *reinterpret_cast<const v4f*>(stg + row * 128 + ((rc ^ (row & 7)) << 4));
                        if (n < p.N && k < p.K) {
                            const int64_t at = static_cast<int64_t>(n) * p.K + k;
                            if (!p.dw_bf16 && !p.accumulate)
                                __builtin_nontemporal_store(x, reinterpret_cast<v4f*>(static_cast<float*>(p.dw) + at));
                            else
                                wgrad_put4(p.dw, p.dw_bf16, p.accumulate, at, x);
                        }
                    }
                    lds_done();
                }
            }
        }
    }
    wait_vmcnt<0>();   // nothing is still writing LDS when the workgroup's next tiles, or another workgroup, use it
}

template <bool kE8M0>
__global__ void __launch_bounds__(kThreads, 1)
fp8_wgrad_large_kernel(WgradParams p, int full) {
    extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
    const int xcd = blockIdx.x % kXcds, local = blockIdx.x / kXcds, stride = gridDim.x / kXcds;
    const int per = (full + kXcds - 1) / kXcds;
    large_tiles<256, kE8M0>(p, lds, xcd * per + local, min((xcd + 1) * per, full), stride);
    const int rest = 2 * (p.tiles_n * p.tiles_k - full), rper = (rest + kXcds - 1) / kXcds;
    if (rest > 0) {
        __syncthreads();
        large_tiles<128, kE8M0>(p, lds, 2 * full + xcd * rper + local, 2 * full + min((xcd + 1) * rper, rest), stride);
    }
}

}  // namespace

// Where the small kernel's 128 x 128 tiles do not all run at once (4608 tokens, 2560 x 2048 outputs: 81 us,
// 108 there; 4096 x 2048: 89 and 110; 130 tokens, 4096 x 4096: 20 and 31; but 4608 tokens, 2048 x 2048, which is
// 256 of them: 83 and 63).
bool wgrad_large_takes(int64_t T, int N, int K) {
    return T > BT && static_cast<int64_t>((N + 127) / 128) * ((K + 127) / 128) > device_cu_count();
}

hipError_t launch_wgrad_large(const WgradParams& g, bool e8m0, hipStream_t stream) {
    auto kernel = e8m0 ? fp8_wgrad_large_kernel<true> : fp8_wgrad_large_kernel<false>;
    int per_cu = 0;
    hipError_t e = kernel_blocks_per_cu(reinterpret_cast<const void*>(kernel), kThreads, kLds, &per_cu);
    if (e != hipSuccess) return e;
    WgradParams p = g;
    p.tiles_n = (g.N + 255) / 256;
    p.tiles_k = (g.K + 255) / 256;
    const int cus = std::max(kXcds, device_cu_count() / kXcds * kXcds);
    const int total = p.tiles_n * p.tiles_k, rest = total % cus;
    // whole rounds of 256-row tiles; a remainder that fills at most half a round goes as 128-row halves (4608
    // tokens, 4608 x 4096 outputs: 202 us, 236 without)
    const int full = rest > 0 && rest <= cus / 2 ? total - rest : total;
    kernel<<<cus, kThreads, kLds, stream>>>(p, full);
    return hipGetLastError();
}

}  // namespace rtq
