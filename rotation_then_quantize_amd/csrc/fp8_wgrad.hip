// fp8_wgrad.hip -- weight gradient of the 8-bit layer from its 8-bit checkpoint on the gfx950 bf16
// matrix cores:
//
//   dw[n][k] = sum_t dy[t][n] * x^[t][k],   x^[t][k] = sx[k / 128][t] qx[t][k]
//
// The scale varies along the reduction (t), so it cannot be taken out of the sum: the codes are decoded
// to bf16 in LDS (exact for power-of-two scales, as rtq_fp8_quantize writes them: a code has at most 4
// significant bits; one rounding to bf16 for general scales) and multiplied with dy as it is, summed in
// fp32.  Both operands have the reduction as their row index; the transposing LDS read gives each lane
// consecutive t of one column.
//
// This file: 128 x 128 tiles, one per workgroup, for outputs of few tiles, which are bound by the latency of
// each workgroup's chain of stages.  Outputs of many tiles: fp8_wgrad_large.hip.
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

constexpr int kTile = 128;        // rows n and columns k: one scale a token
constexpr int BT = 64;            // tokens per LDS stage
constexpr int kWavesN = 2, kWavesK = 4, kWaves = kWavesN * kWavesK, kThreads = 64 * kWaves;
constexpr int WN = kTile / kWavesN, WK = kTile / kWavesK, TN = WN / 16, TK = WK / 16;
constexpr int kSlots = 4;         // stages of dy and of codes in LDS
constexpr int kRow = kTile * 2;   // LDS bytes of a token's dy, or of its decoded input
constexpr int kDy = BT * kRow, kRaw = BT * kTile, kStage = kDy + kRaw;
constexpr int kTable = 1024;      // tokens whose scales are in LDS, and those of two stages more
constexpr int kLds = kSlots * kStage + 2 * BT * kRow + (kTable + 2 * BT) * static_cast<int>(sizeof(float));

// The stages of dy and of the codes are loaded kSlots stages ahead, straight into LDS; while stage s is
// multiplied, the codes of stage s + 2 are decoded into a bf16 copy (two of them in turn) and the fragments of
// stage s + 1 are read.
template <bool kE8M0>
__global__ void __launch_bounds__(kThreads)
fp8_wgrad_kernel(WgradParams p) {
    extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
    const uint32_t lds_base = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(lds));
    constexpr int kDecoded = kSlots * kStage;
    float* table = reinterpret_cast<float*>(lds + kDecoded + 2 * BT * kRow);
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wn = wave / kWavesK, wk = wave % kWavesK;
    const int g = lane >> 4, l15 = lane & 15;

    // 8 contiguous ranges of tiles and their parts, one per XCD (workgroup b runs on XCD b % 8)
    const int total = p.tiles_n * p.tiles_k * p.split, per = (total + 7) / 8;
    const int local = static_cast<int>(blockIdx.x) / 8, lin = static_cast<int>(blockIdx.x) % 8 * per + local;
    if (local >= per || lin >= total) return;
    const int tile = lin / p.split, part = lin % p.split;
    const int n0 = tile / p.tiles_k * kTile, k0 = tile % p.tiles_k * kTile;
    const int64_t stages = (p.T + BT - 1) / BT;
    const int64_t s0 = stages * part / p.split;
    const int nt = static_cast<int>(stages * (part + 1) / p.split - s0);

    const int64_t end = min<int64_t>(p.T, (s0 + nt) * BT);   // loads past this part's tokens give zeros
    // dy: 4 rows of 256 bytes a load; the 32-byte unit u (16 columns) of row t at u ^ (t & 7).  Codes: 8 rows
    // of 128 bytes a load.
    const int d_row = 4 * wave + (lane >> 4);
    const uint32_t d_off = static_cast<uint32_t>(d_row) * static_cast<uint32_t>(p.N) * 2u +
                           static_cast<uint32_t>(((lane & 15) ^ ((d_row & 7) << 1)) << 4);
    const uint32_t x_off = static_cast<uint32_t>(8 * wave + (lane >> 3)) * static_cast<uint32_t>(p.K) + static_cast<uint32_t>((lane & 7) * 16);
    auto issue = [&](int s) {
        const int64_t t0 = (s0 + s) * BT;
        const int rows = static_cast<int>(max<int64_t>(0, min<int64_t>(BT, end - t0)));
        const uint32_t mask = rows > 0 ? ~0u : 0u;
        const v4i rd = make_rsrc(p.dy + t0 * p.N + n0, ((static_cast<uint32_t>(rows) * static_cast<uint32_t>(p.N) - static_cast<uint32_t>(n0)) * 2u) & mask);
        const v4i rx = make_rsrc(p.x + t0 * p.K + k0, (static_cast<uint32_t>(rows) * static_cast<uint32_t>(p.K) - static_cast<uint32_t>(k0)) & mask);
        const uint32_t slot = lds_base + static_cast<uint32_t>(s % kSlots * kStage + wave * 1024);
        load_to_lds(rd, d_off, slot);
        load_to_lds(rd, d_off + 64u * static_cast<uint32_t>(p.N), slot + kWaves * 1024);
        load_to_lds(rx, x_off, slot + kDy);
    };
    constexpr int kLoads = 3;
    const int64_t xs = static_cast<int64_t>(k0 / kFp8Block) * p.T;
    auto fill = [&](int s) {   // the scales of the stages s .., zeros past the last token (an infinite one times the
                               // zeros there would be none)
#pragma unroll
        for (int e = tid; e < kTable + 2 * BT; e += kThreads) {
            const int64_t t = (s0 + s) * BT + e;
            const float v = load_scale<kE8M0>(p.x_scale, xs + min<int64_t>(t, p.T - 1));
            table[e] = t < p.T ? v : 0.0f;
        }
    };
    const int x_row = tid >> 3;
    v4i q;      // 16 codes a thread
    float sc;   // and their token's scale; the table begins with stage `first`
    auto read_codes = [&](int s, int first) {
        q = *reinterpret_cast<const v4i*>(lds + s % kSlots * kStage + kDy + tid * 16);
        sc = table[(s - first) * BT + x_row];
    };
    auto decode = [&](int s) {
        uint32_t w[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float v[4];
            decode4<false>(static_cast<uint32_t>(q[e]), v);
            w[2 * e] = pack_bf16x2(v[0] * sc, v[1] * sc);
            w[2 * e + 1] = pack_bf16x2(v[2] * sc, v[3] * sc);
        }
        uint8_t* at = lds + kDecoded + (s & 1) * BT * kRow + x_row * kRow + (((tid & 7) ^ (x_row & 7)) << 5);
        *reinterpret_cast<uint4*>(at) = uint4{w[0], w[1], w[2], w[3]};
        *reinterpret_cast<uint4*>(at + 16) = uint4{w[4], w[5], w[6], w[7]};
    };
    // Fragments: lane group g holds tokens 16 q + 4 g + (0..3), q = 0..3, of its column.
    const int r4 = l15 >> 2, swz = 4 * (g & 1) + r4;
    const uint32_t d0 = lds_base + static_cast<uint32_t>((4 * g + r4) * kRow + (((TN * wn) ^ swz) << 5) + (l15 & 3) * 8);
    const uint32_t x0 = lds_base + static_cast<uint32_t>(kDecoded + (4 * g + r4) * kRow + (((TK * wk) ^ swz) << 5) + (l15 & 3) * 8);
    auto frag = [&](uint32_t at) {
        const v2i r[4] = {read_tr16(at), read_tr16(at + 16 * kRow), read_tr16(at + 32 * kRow), read_tr16(at + 48 * kRow)};
        return v8i{r[0].x, r[0].y, r[1].x, r[1].y, r[2].x, r[2].y, r[3].x, r[3].y};
    };

    v4f acc[TK][TN];
#pragma unroll
    for (int j = 0; j < TK; ++j)
#pragma unroll
        for (int i = 0; i < TN; ++i) acc[j][i] = v4f{0.f, 0.f, 0.f, 0.f};
    v8i fx[2][TK], fd[2][TN];
    auto read = [&](auto set, int s) {
        constexpr int P = decltype(set)::value;
        const uint32_t dy = d0 + static_cast<uint32_t>(s % kSlots * kStage), x = x0 + static_cast<uint32_t>((s & 1) * BT * kRow);
#pragma unroll
        for (int j = 0; j < TK; ++j) fx[P][j] = frag(x ^ static_cast<uint32_t>(j << 5));
#pragma unroll
        for (int i = 0; i < TN; ++i) fd[P][i] = frag(dy ^ static_cast<uint32_t>(i << 5));
    };
    // Stage s from the fragments of set P, while those of stage s + 1 are read and stage s + 2 is decoded.
    // Nothing here is conditional (see the products); past the last stage zeros are loaded and decoded.
    auto stage = [&](auto set, int s, int first) {
        constexpr int P = decltype(set)::value;
        lds_done();              // this wave's part of the decoded stage s + 1 is written, its fragments of stage s are read
        wait_vmcnt<kLoads>();    // stage s + 2 has landed (the next one may be in flight) ...
        barrier();               // ... in every wave; stage s's slot and decoded copy are free
        issue(s + kSlots);
        read_codes(s + 2, first);   // before the fragments: it is needed first
        read(std::integral_constant<int, 1 - P>{}, s + 1);
#pragma unroll
        for (int j = 0; j < TK; ++j)
#pragma unroll
            for (int i = 0; i < TN; ++i) acc[j][i] = mfma_bf16(fx[P][j], fd[P][i], acc[j][i]);
        decode(s + 2);
    };
    constexpr auto P0 = std::integral_constant<int, 0>{};
    constexpr auto P1 = std::integral_constant<int, 1>{};
    if (nt > 0) {
#pragma unroll
        for (int s = 0; s < kSlots; ++s) issue(s);
        fill(0);
        wait_vmcnt<(kSlots - 2) * kLoads>();
        lds_done();
        barrier();   // stages 0 and 1 and the scales, in every wave
        read_codes(0, 0);
        decode(0);
        read_codes(1, 0);
        decode(1);
        lds_done();
        barrier();
        read(P0, 0);
        // The table holds the scales of kTable / BT stages; stage s decodes stage s + 2.
        constexpr int kPer = kTable / BT;
        for (int c = 0; c < nt; c += kPer) {
            if (c > 0) {   // once every wave has decoded the last of the old ones
                lds_done();
                barrier();
                fill(c);
                lds_done();
                barrier();
            }
            const int c1 = min(c + kPer, nt);
            int s = c;
            for (; s + 1 < c1; s += 2) {
                stage(P0, s, c);
                stage(P1, s + 1, c);
            }
            if (s < c1) stage(P0, s, c);
        }
        wait_vmcnt<0>();   // nothing is still writing this workgroup's LDS when another one gets it
    }
    void* dw = p.dw;
    if (p.split > 1) dw = static_cast<float*>(p.dw) + static_cast<int64_t>(part) * p.N * p.K;
#pragma unroll
    for (int j = 0; j < TK; ++j)
#pragma unroll
        for (int i = 0; i < TN; ++i) {
            // K is a multiple of 16: four columns are all in or all out
            const int n = n0 + wn * WN + i * 16 + l15, k = k0 + wk * WK + j * 16 + 4 * g;
            if (n < p.N && k < p.K)
                wgrad_put4(dw, p.split == 1 && p.dw_bf16, p.split == 1 && p.accumulate, static_cast<int64_t>(n) * p.K + k,
                           acc[j][i]);
        }
}

// dw (+)= the sum of the split partials, in order.
__global__ void __launch_bounds__(256)
wgrad_reduce_kernel(const float* __restrict__ part, int split, int64_t n, void* __restrict__ dw, bool bf16, bool accumulate) {
    const int64_t i = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 4;
    if (i >= n) return;   // n is a multiple of 16
    wgrad_put4(dw, bf16, accumulate, i, sum_parts<v4f>(part + i, split, n));
}

int64_t tiles_of(int N, int K) { return static_cast<int64_t>((N + kTile - 1) / kTile) * ((K + kTile - 1) / kTile); }

// Parts of the tokens: as many as fill the CUs, of at least 8 stages (the second kernel costs what shorter chains
// save: 512 tokens, 2048 x 1024 outputs 11.8 us whole, 16.0 in two parts; 4608 tokens, 512 x 512 outputs 16.6 us
// in nine parts, 21.4 in four; 1024 tokens, 512 x 512: 13.4 in two, 15.0 whole).
int choose_split(int64_t tiles, int64_t T) {
    return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({device_cu_count() / tiles, (T + BT - 1) / BT / 8, 16})));
}

}  // namespace

size_t fp8_wgrad_workspace_bytes(int64_t T, int N, int K) {
    if (wgrad_large_takes(T, N, K)) return 0;
    const int split = choose_split(tiles_of(N, K), T);
    return split > 1 ? static_cast<size_t>(split) * N * K * sizeof(float) : 0;
}

hipError_t launch_fp8_wgrad(const Fp8WgradArgs& g, hipStream_t stream) {
    WgradParams p{};
    p.dy = static_cast<const uint16_t*>(g.dy);
    p.x = static_cast<const uint8_t*>(g.x_codes);
    p.x_scale = g.x_scale;
    p.T = g.T;
    p.N = g.N;
    p.K = g.K;
    p.split = 1;
    p.dw = g.dw;
    p.dw_bf16 = g.dw_bf16;
    p.accumulate = g.accumulate;
    if (wgrad_large_takes(g.T, g.N, g.K)) return launch_wgrad_large(p, g.e8m0, stream);
    auto kernel = g.e8m0 ? fp8_wgrad_kernel<true> : fp8_wgrad_kernel<false>;
    int per_cu = 0;
    hipError_t e = kernel_blocks_per_cu(reinterpret_cast<const void*>(kernel), kThreads, kLds, &per_cu);
    if (e != hipSuccess) return e;
    p.tiles_n = (g.N + kTile - 1) / kTile;
    p.tiles_k = (g.K + kTile - 1) / kTile;
    p.split = choose_split(tiles_of(g.N, g.K), g.T);
    const int64_t n = static_cast<int64_t>(g.N) * g.K;
    if (g.workspace == nullptr || g.ws_bytes < static_cast<size_t>(p.split) * n * sizeof(float)) p.split = 1;
    if (p.split > 1) p.dw = g.workspace;
    const int64_t total = tiles_of(g.N, g.K) * p.split;
    kernel<<<static_cast<unsigned>((total + 7) / 8 * 8), kThreads, kLds, stream>>>(p);
    e = hipGetLastError();
    if (e != hipSuccess || p.split == 1) return e;
    wgrad_reduce_kernel<<<static_cast<unsigned>((n / 4 + 255) / 256), 256, 0, stream>>>(
        static_cast<const float*>(g.workspace), p.split, n, g.dw, g.dw_bf16, g.accumulate);
    return hipGetLastError();
}

}  // namespace rtq
