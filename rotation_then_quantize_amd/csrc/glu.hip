// glu.hip -- the gated feed-forward's first half on gfx950, y = f(g) u with [g u] = x W^T from 8-bit codes, and its
// backward pass from the 8-bit checkpoint of [g u]:
//
//   dg = dy u^ f'(g^),  du = dy f(g^)
//
// The backward pass is one pass over HBM: 4 bytes read and 6 written for each channel and token.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "block_internal.h"
#include "fp8_act.h"
#include "fp8_device.h"
#include "fp8_glu.h"
#include "fp8_internal.h"
#include "fp8_tile.h"
#include "rtq_internal.h"

namespace rtq {
namespace {

using namespace fp8;

constexpr int kThreads = 256;
constexpr int kWaveCols = 512;   // a wave's channels: four groups of 16 lanes, 8 channels a lane

// y = f(g) u from the sums [parts][T][2 N], codes and scales on the way.  A wave takes 512 channels of a token.
struct FinishParams {
    const float* h;
    int parts;
    int64_t T;
    int N;
    int col_waves;
    void* h_codes;
    void* h_scale;
    void* y;
    bool y_bf16;
    void* y_codes;
    void* y_scale;
    bool e8m0;
};

template <int kAct>
__global__ void __launch_bounds__(kThreads)
glu_finish_kernel(FinishParams p) {
    const int lane = threadIdx.x & 63;
    const int64_t wave = block_index() * (kThreads / 64) + (threadIdx.x >> 6);
    const int64_t t = wave / p.col_waves;
    const int c = static_cast<int>(wave % p.col_waves) * kWaveCols + lane * 8;
    if (t >= p.T) return;
    const bool in = c < p.N;   // N is a multiple of 128: a group's lanes are all in or all out
    const int64_t at = t * 2 * p.N + c;
    float g[8], u[8];
    auto load = [&](float* v, int64_t i) {
        v4f s[2] = {v4f{0.f, 0.f, 0.f, 0.f}, v4f{0.f, 0.f, 0.f, 0.f}};
        if (in) {
#pragma unroll
            for (int q = 0; q < 2; ++q) s[q] = sum_parts<v4f>(p.h + i + 4 * q, p.parts, p.T * 2 * p.N);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = s[e / 4][e % 4];
    };
    load(g, at);
    load(u, at + p.N);
    uint2 q;
    auto put_scale = [&](void* s, int64_t group, int e) {
        if (in && (lane & 15) == 0) store_scale(s, p.e8m0, group * p.T + t, e);
    };
    if (p.h_codes != nullptr) {
        uint8_t* codes = static_cast<uint8_t*>(p.h_codes) + at;
        int e = quantise8<false>(g, &q);
        if (in) *reinterpret_cast<uint2*>(codes) = q;
        put_scale(p.h_scale, c / kFp8Block, e);
        e = quantise8<false>(u, &q);
        if (in) *reinterpret_cast<uint2*>(codes + p.N) = q;
        put_scale(p.h_scale, (p.N + c) / kFp8Block, e);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] = act_value<kAct>(g[i]) * u[i];
    const int64_t out = t * p.N + c;
    if (p.y != nullptr) {
        if (in && p.y_bf16) store8<true>(p.y, out, g);
        if (in && !p.y_bf16) store8<false>(p.y, out, g);
    } else {
        const int e = quantise8<false>(g, &q);
        if (in) *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.y_codes) + out) = q;
        put_scale(p.y_scale, c / kFp8Block, e);
    }
}

template <typename F>
hipError_t with_act(int act, F f) {
    switch (act) {
        case RTQ_ACT_GELU_TANH: return f(std::integral_constant<int, RTQ_ACT_GELU_TANH>{});
        case RTQ_ACT_GELU: return f(std::integral_constant<int, RTQ_ACT_GELU>{});
        case RTQ_ACT_SILU: return f(std::integral_constant<int, RTQ_ACT_SILU>{});
        default: return hipErrorInvalidValue;
    }
}

size_t sums_bytes(int64_t T, int N) { return static_cast<size_t>(T) * 2 * N * sizeof(float); }

// The outputs from the sums in the workspace.
hipError_t launch_finish(const GluArgs& a, int parts, hipStream_t stream) {
    const int col_waves = (a.N + kWaveCols - 1) / kWaveCols;
    const int64_t waves = a.T * col_waves;
    const FinishParams p{static_cast<const float*>(a.workspace), parts, a.T, a.N, col_waves, a.h_codes, a.h_scale, a.y, a.y_bf16,
                         a.y_codes, a.y_scale, a.e8m0};
    return with_act(a.act, [&](auto act) {
        glu_finish_kernel<decltype(act)::value><<<grid_of((waves + kThreads / 64 - 1) / (kThreads / 64)), kThreads, 0, stream>>>(p);
        return hipGetLastError();
    });
}

// The products' sums to the workspace, and the outputs from there.
hipError_t launch_sums(const GluArgs& a, hipStream_t stream) {
    int parts = 1;
    Fp8GemmArgs g{};
    g.a = a.x;
    g.a_scale = a.x_scale;
    g.w = a.w;
    g.w_scale = a.w_scale;
    g.e8m0 = a.e8m0;
    g.M = a.T;
    g.N = 2 * a.N;
    g.R = a.K;
    g.y = a.workspace;
    g.workspace = a.workspace;
    g.ws_bytes = a.ws_bytes;
    g.parts = &parts;
    const hipError_t e = launch_fp8_gemm(g, stream);
    return e != hipSuccess ? e : launch_finish(a, parts, stream);
}

hipError_t launch_small(const GluArgs& a, hipStream_t stream) {
    if (a.y_codes == nullptr && a.h_codes == nullptr) return launch_glu_small(glu_params(a), a.e8m0, nullptr, stream);
    const hipError_t e = launch_glu_small(glu_params(a), a.e8m0, static_cast<float*>(a.workspace), stream);
    return e != hipSuccess ? e : launch_finish(a, 1, stream);
}

// How a product runs.
enum Form : int { kSmall, kSums, kTile32, kTile64, kTile128, kLarge };
// Measured with codes (us; T x K, N channels; fp32 scales, E8M0 ones within 2% but for the last column's long reductions of many
// tiles: 1024 and 2048 x 4096, 4096 in 35.2 and 56.9):
//                        sums    32     64     128    256 tokens a tile
//   64 x 512, 1152        8.1    5.5    6.4    8.2    9.3
//   64 x 1024, 4096      11.1    7.2    8.2   11.4   12.9
//   391 x 1936, 1152     14.1   14.3   16.0   21.3   24.1
//   391 x 2048, 1152     13.8   11.0   12.9   18.8   20.7
//   100 x 2048, 4096     13.3   11.0   12.8   18.7   20.5
//   300 x 2560, 1152     14.5   14.1   16.7   23.5   25.6
//   506 x 3136, 768      16.6   17.4   20.5   29.1   31.3
//   64 x 4096, 4096      14.3   18.4   21.6   31.8   34.7
//   64 x 4096, 10880     26.3   24.7   27.5   34.2   38.8
//   64 x 4096, 16384     37.5   35.9   38.2   40.7   46.8
//   256 x 4096, 4096     22.6   19.0   21.5   32.5   35.3
//   512 x 4096, 4096     29.8   35.9   23.4   32.9   35.5
//   1024 x 4096, 4096    46.8   71.0   45.5   35.8   37.9
//   2048 x 4096, 4096    79.9  140     92.9   72.7   62.3
//   48 x 8192, 8192      37.5   51.9   56.4   66.0   77.9
//   128 x 8192, 8192     52.2   51.7   57.1   71.2   78.6
//   256 x 16384, 4096    83.1   85.1   97.5  130     154
// A tile costs its chain of blocks as long as each CU has one (0.5, 0.6, 0.95 and 1.1 us a block where the weights are in the
// caches; where they come from HBM and fill the CUs, 64 x 4096, 16384, 1.1 to 1.4, for which LDS does not account), so the
// smallest whose workgroups fit at once is taken, and where none fits the largest.  The product that leaves its sums in the
// workspace splits the reduction over idle CUs and costs a launch: it is better where the reduction is long, with tiles for
// more than half of the CUs where it is very long.  Rows that begin inside a line of 128 bytes are slower to load, and more so
// in tiles, so that the sums are level with them sooner (sums and tiles of 32; whole lines, blocks 16, 20, 22, 26: 391 tokens,
// 1152 channels 13.6 11.1, 15.1 14.3, 15.6 14.1, 17.0 15.7; 64, 4096: 13.1 11.1, 14.1 14.2, 14.6 14.0, 13.6 15.8; 100, 2048:
// 13.1 10.6, 13.8 13.6, 14.4 13.9, 13.4 15.6; others, blocks 11, 14, 16, 19: 391, 1152: 12.2 10.9, 13.3 12.8, 14.0 14.4, 15.2
// 16.6; 64, 4096: 10.5 10.7, 11.1 12.8, 11.3 14.3, 14.2 16.6; 100, 2048: 9.9 8.4, 10.4 9.7, 10.7 12.0, 13.7 15.2).
// Few tokens: as the weights stream (fp8_glu_small.hip), but where workgroups are fewer than CUs and the reduction long (y
// alone, with codes, and either from sums: 1 x 16384, 1024 channels 18.7, 20.5, 13.9; 1 x 8192, 1152: 10.8, 12.8, 9.6; 4 x 4096,
// 1152: 7.1, 9.1, 7.7; 4 x 2048, 1152: 4.9, 7.0, 7.7).  17 to 32 of them so where they are wide and the reduction is not short
// (y alone, with codes, either from sums, either by tiles of 64: 32 x 2048, 4096: 7.5, 9.8, 12.5, 12.4; 32 x 4096, 4096: 11.0,
// 12.9, 13.6, 20.9; 32 x 4096, 16384: 28.3, 31.1, 35.6, 37.0; 32 x 4096, 28672: 51.9, 55.3, 65.8, 54.8; but 32 x 2048, 16384:
// 15.0, 17.6, 16.6, 14.0; 32 x 512, 4096: 4.9, 7.7, 9.3, 6.1; 32 x 4096, 2048: 10.9, 13.1, 11.6, 20.9); with 64 tokens their
// loads from the caches are as long as the weights' (4096 x 16384 44.8, 47.0, 37.6, 38.2).  Which outputs are asked for does not
// choose: y is the same bits with the checkpoint and without.
Form plan(int64_t T, int N, int K) {
    const int64_t cus = device_cu_count();
    const int blocks = static_cast<int>(fp8_groups(K));
    auto tiles = [&](int tokens) { return (T + tokens - 1) / tokens * (N / 128); };
    if (T <= 16) return N / 16 < cus && blocks >= 32 ? kSums : kSmall;
    if (T <= 32 && N / 16 >= cus && (blocks > 16 || (2 * tiles(64) < cus && blocks > 8))) return kSmall;
    if (tiles(32) <= cus) return blocks <= (K % kFp8Block == 0 ? 20 : 14) || (2 * tiles(32) > cus && blocks <= 48) ? kTile32 : kSums;
    if (tiles(64) <= cus) return kTile64;
    if (tiles(128) <= cus || blocks == 1) return kTile128;   // (the large form's loads run two blocks ahead)
    return kLarge;
}

// A wave takes 512 channels of a token: their gradients' two parts, 512 channels of the gate and of the other.
template <bool kBF16, bool kE8M0, bool kE5M2, int kAct>
__global__ void __launch_bounds__(kThreads)
glu_backward_kernel(const void* dy, const uint8_t* __restrict__ h_codes, const void* __restrict__ h_scale, int64_t T, int N,
                    int col_waves, void* dh, void* dh_codes, void* dh_scale) {
    const int lane = threadIdx.x & 63;
    const int64_t wave = block_index() * (kThreads / 64) + (threadIdx.x >> 6);
    const int64_t t = wave / col_waves;
    const int c = static_cast<int>(wave % col_waves) * kWaveCols + lane * 8;
    if (t >= T) return;
    const bool in = c < N;
    const int64_t at = t * 2 * N + c;
    uint2 qg = {0u, 0u}, qu = {0u, 0u};
    Row8<kBF16> d;
    d.zero();
    float sg = 1.f, su = 1.f;
    if (in) {
        qg = *reinterpret_cast<const uint2*>(h_codes + at);
        qu = *reinterpret_cast<const uint2*>(h_codes + at + N);
        d.load(dy, t * N + c);
        sg = load_scale<kE8M0>(h_scale, static_cast<int64_t>(c / kFp8Block) * T + t);
        su = load_scale<kE8M0>(h_scale, static_cast<int64_t>((N + c) / kFp8Block) * T + t);
    }
    float g[8], u[8], v[8];
    decode4<false>(qg.x, g);
    decode4<false>(qg.y, g + 4);
    decode4<false>(qu.x, u);
    decode4<false>(qu.y, u + 4);
    d.get(v);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float x = g[i] * sg;
        g[i] = v[i] * (u[i] * su) * act_slope<kAct>(x);
        u[i] = v[i] * act_value<kAct>(x);
    }
    if (dh != nullptr && in) {
        store8<kBF16>(dh, at, g);
        store8<kBF16>(dh, at + N, u);
    }
    if (dh_codes != nullptr) {
        uint2 q;
        uint8_t* codes = static_cast<uint8_t*>(dh_codes) + at;
        const int eg = quantise8<kE5M2>(g, &q);
        if (in) *reinterpret_cast<uint2*>(codes) = q;
        const int eu = quantise8<kE5M2>(u, &q);
        if (in) *reinterpret_cast<uint2*>(codes + N) = q;
        if (in && (lane & 15) == 0) {
            store_scale(dh_scale, kE8M0, static_cast<int64_t>(c / kFp8Block) * T + t, eg);
            store_scale(dh_scale, kE8M0, static_cast<int64_t>((N + c) / kFp8Block) * T + t, eu);
        }
    }
}

template <bool kBF16, bool kE8M0, bool kE5M2>
hipError_t backward(const GluBackwardArgs& a, hipStream_t stream) {
    const int col_waves = (a.N + kWaveCols - 1) / kWaveCols;
    const int64_t waves = a.T * col_waves;
    return with_act(a.act, [&](auto act) {
        glu_backward_kernel<kBF16, kE8M0, kE5M2, decltype(act)::value>
            <<<grid_of((waves + kThreads / 64 - 1) / (kThreads / 64)), kThreads, 0, stream>>>(
                a.dy, static_cast<const uint8_t*>(a.h_codes), a.h_scale, a.T, a.N, col_waves, a.dh, a.dh_codes, a.dh_scale);
        return hipGetLastError();
    });
}

}  // namespace

fp8::GluParams glu_params(const GluArgs& a) {
    fp8::GluParams p{};
    p.x = static_cast<const uint8_t*>(a.x);
    p.x_scale = a.x_scale;
    p.w = static_cast<const uint8_t*>(a.w);
    p.w_scale = a.w_scale;
    p.T = a.T;
    p.N = a.N;
    p.K = a.K;
    p.out = fp8::GluOut{a.act, a.h_codes, a.h_scale, a.y, a.y_bf16, a.y_codes, a.y_scale};
    return p;
}

size_t fp8_glu_workspace_bytes(int64_t T, int N, int K) {
    if (T == 0) return 0;
    switch (plan(T, N, K)) {
        case kSums: return std::max(sums_bytes(T, N), fp8_gemm_workspace_bytes(T, 2 * N, K, false));
        case kSmall: return sums_bytes(T, N);
        default: return 0;
    }
}

hipError_t launch_fp8_glu(const GluArgs& a, hipStream_t stream) {
    switch (plan(a.T, a.N, a.K)) {
        case kSmall: return launch_small(a, stream);
        case kTile32: return launch_glu_tile(glu_params(a), a.e8m0, 32, stream);
        case kTile64: return launch_glu_tile(glu_params(a), a.e8m0, 64, stream);
        case kTile128: return launch_glu_tile(glu_params(a), a.e8m0, 128, stream);
        case kLarge: return launch_glu_large(glu_params(a), a.e8m0, stream);
        default: return launch_sums(a, stream);
    }
}

hipError_t launch_glu_backward(const GluBackwardArgs& a, hipStream_t stream) {
    auto pick = [&](auto bf16, auto e8m0) {
        constexpr bool kB = decltype(bf16)::value, k8 = decltype(e8m0)::value;
        return a.e5m2 ? backward<kB, k8, true>(a, stream) : backward<kB, k8, false>(a, stream);
    };
    constexpr auto yes = std::true_type{};
    constexpr auto no = std::false_type{};
    if (a.bf16) return a.e8m0 ? pick(yes, yes) : pick(yes, no);
    return a.e8m0 ? pick(no, yes) : pick(no, no);
}

}  // namespace rtq
