// fp8_wgrad.hip -- weight gradient of the 8-bit layer from its 8-bit checkpoint on the gfx950 bf16
// matrix cores:
//
//   dw[n][k] = sum_t dy[t][n] * x^[t][k],   x^[t][k] = sx[k / 128][t] qx[t][k]
//
// The scale varies along the reduction (t), so it cannot be taken out of the sum: the codes are decoded
// to bf16 on their way into LDS (exact for power-of-two scales, as rtq_fp8_quantize writes them: a code
// has at most 4 significant bits; one rounding to bf16 for general scales) and multiplied with dy as it
// is, summed in fp32.  Both operands have the reduction as their row index; the transposing LDS read
// gives each lane consecutive t of one column.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "fp8_internal.h"
#include "fp8_tile.h"
#include "fp8_wgrad.h"
#include "rtq_internal.h"

namespace rtq {
namespace {

using namespace fp8;

constexpr int kTile = 64;
constexpr int BT = 32;        // tokens per LDS stage: one 16 x 16 x 32 matrix instruction
constexpr int kRow = kTile * 2;   // bytes of an LDS row (bf16)

template <bool kE8M0>
__global__ void __launch_bounds__(256)
fp8_wgrad_kernel(WgradParams p) {
    __shared__ __attribute__((aligned(16))) uint8_t s_dy[BT * kRow];
    __shared__ __attribute__((aligned(16))) uint8_t s_x[BT * kRow];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int g = lane >> 4, l15 = lane & 15;
    const int wk = wave >> 1, wn = wave & 1;   // 32 columns of k and 32 rows of n per wave
    const int tile = static_cast<int>(blockIdx.x) / p.split, part = static_cast<int>(blockIdx.x) % p.split;
    const int n0 = tile / p.tiles_k * kTile, k0 = tile % p.tiles_k * kTile;
    const int64_t stages = (p.T + BT - 1) / BT;
    const int64_t s0 = stages * part / p.split, s1 = stages * (part + 1) / p.split;

    // thread: row tid / 8 of the stage, 8 columns from 8 (tid % 8); chunk c (16 bytes) of row r sits at
    // c ^ (2 (r & 3)), so that the 4 rows x 32 bytes of a transposing read touch different banks
    const int row = tid >> 3, col = (tid & 7) * 8;
    const uint32_t put = static_cast<uint32_t>(row * kRow + (((tid & 7) ^ ((row & 3) << 1)) << 4));
    const int64_t xs_row = static_cast<int64_t>(min(k0 + col, p.K - 1) / kFp8Block) * p.T;
    const uint32_t base_dy = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(s_dy));
    const uint32_t base_x = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(s_x));

    v4f acc[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};

    auto read = [&](uint32_t base, int c0) {   // 8 t of column c0 + l15: t = 8 g .. 8 g + 7
        v2i f[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = 8 * g + 4 * h + (l15 >> 2);
            const int chunk = (c0 / 8 + ((lane & 3) >> 1)) ^ ((r & 3) << 1);
            f[h] = read_tr16(base + static_cast<uint32_t>(r * kRow + (chunk << 4) + (lane & 1) * 8));
        }
        return __builtin_bit_cast(v8bf, v4i{f[0].x, f[0].y, f[1].x, f[1].y});
    };
    for (int64_t s = s0; s < s1; ++s) {
        const int64_t t = s * BT + row;
        uint4 d{0u, 0u, 0u, 0u};
        uint2 q{0u, 0u};
        float sc = 0.0f;
        if (t < p.T) {
            if (n0 + col < p.N) d = *reinterpret_cast<const uint4*>(p.dy + t * p.N + n0 + col);
            if (k0 + col < p.K) q = *reinterpret_cast<const uint2*>(p.x + t * p.K + k0 + col);
            sc = load_scale<kE8M0>(p.x_scale, xs_row + t);
        }
        float v[8];
        decode4<false>(q.x, v);
        decode4<false>(q.y, v + 4);
        uint4 x{pack_bf16x2(v[0] * sc, v[1] * sc), pack_bf16x2(v[2] * sc, v[3] * sc),
                pack_bf16x2(v[4] * sc, v[5] * sc), pack_bf16x2(v[6] * sc, v[7] * sc)};
        __syncthreads();
        *reinterpret_cast<uint4*>(s_dy + put) = d;
        *reinterpret_cast<uint4*>(s_x + put) = x;
        __syncthreads();
        v8bf fx[2], fd[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            fx[i] = read(base_x, wk * 32 + i * 16);
            fd[i] = read(base_dy, wn * 32 + i * 16);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fx[i], fd[j], acc[i][j], 0, 0, 0);
    }
    void* dw = p.dw;
    if (p.split > 1) dw = static_cast<float*>(p.dw) + static_cast<int64_t>(part) * p.N * p.K;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            // K is a multiple of 16: four columns are all in or all out
            const int n = n0 + wn * 32 + j * 16 + l15, k = k0 + wk * 32 + i * 16 + 4 * g;
            if (n < p.N && k < p.K)
                wgrad_put4(dw, p.split == 1 && p.dw_bf16, p.split == 1 && p.accumulate, static_cast<int64_t>(n) * p.K + k,
                     acc[i][j]);
        }
}

// dw (+)= the sum of the split partials, in order.
__global__ void __launch_bounds__(256)
wgrad_reduce_kernel(const float* __restrict__ part, int split, int64_t n, void* __restrict__ dw, bool bf16, bool accumulate) {
    const int64_t i = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 4;
    if (i >= n) return;   // n is a multiple of 16
    v4f s = *reinterpret_cast<const v4f*>(part + i);
    for (int k = 1; k < split; ++k) s += *reinterpret_cast<const v4f*>(part + k * n + i);
    wgrad_put4(dw, bf16, accumulate, i, s);
}

int choose_split(int64_t tiles, int64_t stages) {
    const int64_t want = 2 * 256;
    if (tiles >= want) return 1;
    return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({want / tiles, stages / 4, 16})));
}

int64_t tiles_of(int N, int K) { return static_cast<int64_t>((N + kTile - 1) / kTile) * ((K + kTile - 1) / kTile); }

}  // namespace

size_t fp8_wgrad_workspace_bytes(int64_t T, int N, int K) {
    if (wgrad_large_takes(T, N, K)) return 0;
    const int split = choose_split(tiles_of(N, K), (T + BT - 1) / BT);
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
    p.dw = g.dw;
    p.dw_bf16 = g.dw_bf16;
    p.accumulate = g.accumulate;
    if (wgrad_large_takes(g.T, g.N, g.K)) return launch_wgrad_large(p, g.e8m0, stream);
    p.tiles_n = (g.N + kTile - 1) / kTile;
    p.tiles_k = (g.K + kTile - 1) / kTile;
    const int64_t tiles = tiles_of(g.N, g.K);
    p.split = choose_split(tiles, (g.T + BT - 1) / BT);
    const int64_t n = static_cast<int64_t>(g.N) * g.K;
    if (g.workspace == nullptr || g.ws_bytes < static_cast<size_t>(p.split) * n * sizeof(float)) p.split = 1;
    if (p.split > 1) p.dw = g.workspace;
    if (g.e8m0)
        fp8_wgrad_kernel<true><<<static_cast<unsigned>(tiles * p.split), 256, 0, stream>>>(p);
    else
        fp8_wgrad_kernel<false><<<static_cast<unsigned>(tiles * p.split), 256, 0, stream>>>(p);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.split == 1) return e;
    wgrad_reduce_kernel<<<static_cast<unsigned>((n / 4 + 255) / 256), 256, 0, stream>>>(
        static_cast<const float*>(g.workspace), p.split, n, g.dw, g.dw_bf16, g.accumulate);
    return hipGetLastError();
}

}  // namespace rtq
