// fp8_glu_small.hip -- the gated feed-forward's product for at most 32 tokens: bound by the weights' bytes.
//
// A workgroup takes 16 kC channels, as many rows of the gate and their partners, and the whole reduction, its 8 waves the
// blocks of 128 in turn.  Each wave loads its operands into registers, 16 rows of its next block as soon as it has decoded those
// before.  They are multiplied as bf16, which has every code's value: its products are added in fp32 (1e-7 of the sums' 2-norm;
// the 8-bit instruction aligns them first, 2e-5), and their time goes beside the loads' (1 x 4096, 16384 channels: 24.1 us; with
// the rows' loads behind the products 26.0, the 8-bit instruction so 25.2).  The waves' sums meet in LDS, in a fixed order, and y = f(g) u is written
// from there; where codes are wanted, whose scales go over the channels of several workgroups, the sums are written
// (glu_finish_kernel makes the codes).  A workgroup for the 128 channels of a scale, which needs no second launch, reads at
// most 32 GB/s on its CU: 1 x 4096, 16384 channels in 39 us, 4096 channels in 33 (24 and 8 so).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "fp8_glu.h"
#include "fp8_internal.h"
#include "rtq_internal.h"

namespace rtq {
namespace {

using namespace fp8;

constexpr int kWaves = 8, kThreads = 64 * kWaves;

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

// The values of eight e4m3 codes.
__device__ __forceinline__ v8bf values(int lo, int hi) {
    const auto a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(static_cast<uint32_t>(lo), 1.f, false);
    const auto b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(static_cast<uint32_t>(lo), 1.f, true);
    const auto c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(static_cast<uint32_t>(hi), 1.f, false);
    const auto d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(static_cast<uint32_t>(hi), 1.f, true);
    return v8bf{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}
__device__ __forceinline__ v4f products(const v8bf& w, const v8bf& a, const v4f& c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, a, c, 0, 0, 0); }

// kTT tiles of 16 tokens.  sums: [T][2 N] fp32, or nullptr: y is written
template <int kC, int kTT, bool kE8M0>
__global__ void __launch_bounds__(kThreads)
glu_small_kernel(GluParams p, float* sums) {
    constexpr int kTiles = 2 * kC, kSums = kTiles * 64;
    __shared__ __attribute__((aligned(16))) v4f s_sums[kWaves * kSums];   // [wave][tile][lane]
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g = lane >> 4, l15 = lane & 15;
    const int K = p.K, blocks = (K + BK - 1) / BK, T = static_cast<int>(p.T);

    // 8 contiguous ranges of channels, one per XCD (workgroup b runs on XCD b % 8); an XCD's workgroups begin at the same
    // place of their rows, see below (1 x 4096, 16384 channels: 24.1 us, neighbours on different XCDs 32.1)
    const int total = p.tiles_n, per = (total + 7) / 8;
    const int b = static_cast<int>(blockIdx.x), local = b / 8, lin = b % 8 * per + local;
    if (local >= per || lin >= total) return;
    const int n0 = lin * 16 * kC, channels = min(16 * kC, p.N - n0);

    auto resource = [](const void* base, int64_t bytes) {   // loads past its end give zeros
        return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, static_cast<int>(bytes), kBufferWord3);
    };
    const __amdgpu_buffer_rsrc_t rw[2] = {resource(p.w + static_cast<int64_t>(n0) * K, static_cast<int64_t>(channels) * K),
                                          resource(p.w + static_cast<int64_t>(p.N + n0) * K, static_cast<int64_t>(channels) * K)};
    const __amdgpu_buffer_rsrc_t rx = resource(p.x, static_cast<int64_t>(T) * K);
    const uint32_t off = static_cast<uint32_t>(l15 * K + 16 * g), tile = static_cast<uint32_t>(16 * K);

    v4i lo[kTiles], hi[kTiles];   // chunks g and g + 4 of 16 rows each: the gate's kC tiles, then their partners
    v4i x0[kTT], x1[kTT];
    float sx[kTT], sw[kTiles];
    // Block of scales of tile i (48 channels may lie in two).  fp32: each tile's scale is loaded by itself, into a scalar
    // register.  Bytes have no scalar load: lane i loads tile i's.
    auto w_row = [&](int i) { return static_cast<int64_t>((i / kC * p.N + min(n0 + i % kC * 16, p.N - 16)) / kFp8Block) * blocks; };
    const int64_t w_mine = w_row(lane % kTiles);
    const float* w_tile[kTiles];
#pragma unroll
    for (int i = 0; i < kTiles; ++i) w_tile[i] = static_cast<const float*>(p.w_scale) + w_row(i);
    uint32_t o0, o1;
    auto begin = [&](int kb) {    // the block's offsets; past the last block all reads as zeros
        const int k = kb * BK + 16 * g;
        o0 = k < K ? off + static_cast<uint32_t>(kb * BK) : kOob;
        o1 = k + 64 < K ? off + static_cast<uint32_t>(kb * BK + 64) : kOob;
    };
    auto load_tile = [&](int i) {
        const uint32_t row = static_cast<uint32_t>(i % kC) * tile;
        lo[i] = __builtin_amdgcn_raw_buffer_load_b128(rw[i / kC], o0 + row, 0, 0);
        hi[i] = __builtin_amdgcn_raw_buffer_load_b128(rw[i / kC], o1 + row, 0, 0);
    };
    auto load_tokens = [&](int kb) {
        const int kc = min(kb, blocks - 1);
#pragma unroll
        for (int t = 0; t < kTT; ++t) {
            x0[t] = __builtin_amdgcn_raw_buffer_load_b128(rx, o0 + t * tile, 0, 0);
            x1[t] = __builtin_amdgcn_raw_buffer_load_b128(rx, o1 + t * tile, 0, 0);
            const float a = load_scale<kE8M0>(p.x_scale, kc * p.T + min(16 * t + l15, T - 1));
            sx[t] = kb < blocks ? a : 0.f;   // past the last block no infinity meets the zeros
        }
        if constexpr (kE8M0) {
            const float w = load_scale<true>(p.w_scale, w_mine + kc);
            sw[0] = kb < blocks ? w : 0.f;
        } else {
#pragma unroll
            for (int i = 0; i < kTiles; ++i) {
                const float w = kC == 3 || i % kC == 0 ? w_tile[i][kc] : sw[i - 1];
                sw[i] = kb < blocks ? w : 0.f;
            }
        }
    };
    v4f acc[kTiles][kTT];
#pragma unroll
    for (int i = 0; i < kTiles; ++i)
#pragma unroll
        for (int t = 0; t < kTT; ++t) acc[i][t] = v4f{0.f, 0.f, 0.f, 0.f};
    // The wave's blocks: wave + 8 j, j over turns from a place of the XCD's own: rows a power of two apart share memory
    // channels, and workgroups at the same place of their rows would crowd them (33.6 us).
    const int turns = (blocks + kWaves - 1) / kWaves, start = b % turns;
    auto block = [&](int t) {
        const int j = t + start;
        return t < turns ? wave + kWaves * (j < turns ? j : j - turns) : blocks;
    };
    begin(block(0));
    load_tokens(block(0));
#pragma unroll
    for (int i = 0; i < kTiles; ++i) load_tile(i);
    for (int turn = 0; turn < turns; ++turn) {
        v8bf a[kTT][4];
        float s[kTT], now[kTiles];
#pragma unroll
        for (int t = 0; t < kTT; ++t) {
            a[t][0] = values(x0[t].x, x0[t].y);
            a[t][1] = values(x0[t].z, x0[t].w);
            a[t][2] = values(x1[t].x, x1[t].y);
            a[t][3] = values(x1[t].z, x1[t].w);
            s[t] = sx[t];
        }
#pragma unroll
        for (int i = 0; i < kTiles; ++i) now[i] = kE8M0 ? __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(sw[0]), i)) : sw[i];
        const int next = block(turn + 1);
        begin(next);
        load_tokens(next);
#pragma unroll
        for (int i = 0; i < kTiles; ++i) {
            const v8bf w[4] = {values(lo[i].x, lo[i].y), values(lo[i].z, lo[i].w), values(hi[i].x, hi[i].y), values(hi[i].z, hi[i].w)};
            load_tile(i);
            constexpr v4f zero = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int t = 0; t < kTT; ++t) {
                const v4f d = products(w[2], a[t][2], products(w[0], a[t][0], zero)) + products(w[3], a[t][3], products(w[1], a[t][1], zero));
                const float by = s[t] * now[i];
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[i][t][r] = __builtin_fmaf(d[r], by, acc[i][t][r]);
            }
            __builtin_amdgcn_sched_barrier(0);   // the loads stay before the products
        }
    }
#pragma unroll
    for (int t = 0; t < kTT; ++t) {
        if (t > 0) __syncthreads();
#pragma unroll
        for (int i = 0; i < kTiles; ++i) s_sums[wave * kSums + i * 64 + lane] = acc[i][t];
        __syncthreads();
        auto sum = [&](int e) {
            v4f v = s_sums[e];
#pragma unroll
            for (int w = 1; w < kWaves; ++w) v += s_sums[w * kSums + e];
            return v;
        };
        // a wave takes 16 rows: lane l token l % 16, channels 4 (l / 16) .. +4
        const int token = 16 * t + l15;
        if (sums != nullptr) {
            const int c = n0 + wave % kC * 16 + 4 * g;
            if (wave < kTiles) {
                const v4f v = sum(tid);
                if (token < T && c < p.N) *reinterpret_cast<v4f*>(sums + (static_cast<int64_t>(token) * 2 + wave / kC) * p.N + c) = v;
            }
        } else if (wave < kC) {
            const v4f gate = sum(tid), up = sum(tid + 64 * kC);
            v4f y;
            for_act(p.out.act, [&](auto act) {
#pragma unroll
                for (int r = 0; r < 4; ++r) y[r] = act_value<decltype(act)::value>(gate[r]) * up[r];
            });
            store4(p.out.y, p.out.y_bf16, T, p.N, token, n0 + wave * 16 + 4 * g, y);
        }
    }
}

}  // namespace

// Tiles of 16 channels per workgroup: as few bytes on the fullest CU as can be, a tile's two projections and the tokens once a
// workgroup, and of equals the most (13 x 4096, 10880 channels, 680 tiles: three a workgroup, one workgroup on each of 227 CUs,
// 17.0 us; with two, 84 CUs have two workgroups, 23.3; 16 x 4096, 14336: four 23.1, two 25.2; 32 x 4096, 16384: four 28.3, two
// 32.5).  For up to 16 tokens two, where they fill all CUs alike: within 3% of the best (a CU's second workgroup
// can load while the first joins its sums; two, three, four; 1 x 4096, 16384 channels: 24.2, 32.9, 25.2; 24576: 36.7, 37.6, 42.4;
// 32768: 44.7, 50.9, 47.4; 49152: 65.6, 70.5, 68.9; 65536: 85.4, 98.0, 89.9; 1 x 8192, 16384: 45.0, 59.3, 47.0; 1 x 2048, 32768:
// 26.1, 30.7, 26.8; 16 x 4096, 16384: 25.2, 34.8, 25.7; 32768: 46.7, 54.1, 48.5; 49152: 71.1, 74.1, 71.0).
hipError_t launch_glu_small(GluParams p, bool e8m0, float* sums, hipStream_t stream) {
    const int tiles = p.N / 16, cus = device_cu_count(), token_tiles = p.T <= 16 ? 1 : 2;
    auto cost = [&](int c) { return ((tiles + c - 1) / c + cus - 1) / cus * (2 * c + token_tiles); };
    int most = 1;
    for (int c = 2; c <= 4; ++c)
        if (cost(c) <= cost(most)) most = c;
    if (token_tiles == 1 && tiles % (2 * cus) == 0) most = 2;
    auto go = [&](auto channels, auto tokens) {
        constexpr int kC = decltype(channels)::value, kTT = decltype(tokens)::value;
        auto kernel = e8m0 ? glu_small_kernel<kC, kTT, true> : glu_small_kernel<kC, kTT, false>;
        p.tiles_n = (tiles + kC - 1) / kC;
        kernel<<<static_cast<unsigned>((p.tiles_n + 7) / 8 * 8), kThreads, 0, stream>>>(p, sums);
        return hipGetLastError();
    };
    auto by_channels = [&](auto tokens) {
        switch (most) {
            case 1: return go(std::integral_constant<int, 1>{}, tokens);
            case 2: return go(std::integral_constant<int, 2>{}, tokens);
            case 3: return go(std::integral_constant<int, 3>{}, tokens);
            default: return go(std::integral_constant<int, 4>{}, tokens);
        }
    };
    return token_tiles == 1 ? by_channels(std::integral_constant<int, 1>{}) : by_channels(std::integral_constant<int, 2>{});
}

}  // namespace rtq
