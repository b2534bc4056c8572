// rmsnorm.hip -- root-mean-square norm over rows on gfx950, with the residual's addition before it and an 8-bit
// output with scales for groups of 128 behind it, and its backward pass:
//
//   h = round(x + r),  rho = 1 / sqrt(mean h^2 + eps),  n = h rho gamma
//   dh = dr + rho gamma dn - h rho^3 mean(gamma dn h),  dgamma = sum over rows of dn h rho
//
// Both are one pass over HBM: a row stays in registers between its sum and what is computed from it.  Sums of
// squares are held in fp64 (products of fp32 values neither overflow nor round there, and fp64 adds run at the
// fp32 rate), so rho is good to its rounding to fp32.
//
// h and dh are stored past the caches: the residual stream is read again a sublayer later, the codes at once (4608 x 4096: 23.9
// us, 26.9 with plain stores, backward 30.3 and 33.3; 132 and 151 MB, 5.5 and 5.0 TB/s.  Non-temporal loads of x and r bring as
// much where they come from HBM and cost 20% where a kernel before has left them in the cache).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "block_internal.h"
#include "fp8_device.h"
#include "fp8_internal.h"
#include "rtq_internal.h"

namespace rtq {
namespace {

using namespace fp8;

constexpr int kLaneCols = 8;                     // consecutive elements of a lane's chunk
constexpr int kWaveCols = 64 * kLaneCols;
constexpr int kChunks = 2;                       // chunks a lane holds of a row
constexpr int kMostTeam = 16;                    // waves that share a row

// 1 / sqrt(v) of a positive v: the hardware's approximation and one Newton step (0 for an infinite v).
__device__ __forceinline__ double rsqrt64(double v) {
    const double r = __builtin_amdgcn_rsq(v);
    const double s = r * (1.5 - 0.5 * v * r * r);
    return r == 0.0 ? 0.0 : s;
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) v += __shfl_xor(v, m);
    return v;
}

// Sums over the kTeam waves of a team, in each of them.  `slots`: kN * kTeam places of the team's own, not used
// again before every wave has passed another barrier.
template <int kTeam, int kN>
__device__ __forceinline__ void team_sum(double (&v)[kN], double* slots, int wave) {
#pragma unroll
    for (int i = 0; i < kN; ++i) v[i] = wave_sum(v[i]);
    if constexpr (kTeam > 1) {
        if ((threadIdx.x & 63) == 0) {
#pragma unroll
            for (int i = 0; i < kN; ++i) slots[i * kTeam + wave] = v[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            v[i] = 0.0;
#pragma unroll
            for (int w = 0; w < kTeam; ++w) v[i] += slots[i * kTeam + w];
        }
    }
}

struct RmsForwardParams {
    const void* x;
    const void* residual;
    int64_t rows;
    int d;
    double inv_d, eps;
    const void* gamma;
    void* h;
    void* y;
    void* codes;
    void* scale;
    bool e8m0;
};

// The residual stream's 8 values: x + r rounded to r's type.
template <bool kX16, bool kRes, bool kR16>
__device__ __forceinline__ void add_residual(const Row8<kX16>& x, const Row8<kR16>& r, float* v) {
    x.get(v);
    if constexpr (kRes) {
        float w[8];
        r.get(w);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += w[i];
        if constexpr (kR16) {
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                const uint32_t p = pack_bf16x2(v[i], v[i + 1]);
                v[i] = bf16_lo(p);
                v[i + 1] = bf16_hi(p);
            }
        }
    }
}

// n = h rho gamma of a chunk -> y, codes and scales.  All lanes come here; `put`: this lane's chunk exists.
template <bool kX16, bool kG16>
__device__ __forceinline__ void put_chunk(const RmsForwardParams& p, const float* h, const Row8<kG16>& gamma, float rho, bool put,
                                          int64_t row, int c) {
    float g[8], n[8];
    gamma.get(g);
#pragma unroll
    for (int i = 0; i < 8; ++i) n[i] = h[i] * rho * g[i];
    const int64_t at = row * p.d + c;
    if (p.y != nullptr && put) store8<kX16>(p.y, at, n);
    if (p.codes != nullptr) {
        uint2 q;
        const int e = quantise8<false>(n, &q);
        if (put) {
            *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.codes) + at) = q;
            if ((threadIdx.x & 15) == 0) store_scale(p.scale, p.e8m0, static_cast<int64_t>(c / kFp8Block) * p.rows + row, e);
        }
    }
}

constexpr int forward_waves(int team) { return team < 4 ? 4 : team; }

// A team of kTeam waves takes a row of at most kTeam * kChunks * 512 elements.
template <bool kX16, bool kRes, bool kR16, bool kG16, int kTeam>
__global__ void __launch_bounds__(64 * forward_waves(kTeam))
rmsnorm_forward_kernel(RmsForwardParams p) {
    constexpr int kTeams = forward_waves(kTeam) / kTeam;
    __shared__ double slots[kTeams * kTeam];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, team = wave / kTeam, mine = wave % kTeam;
    const int64_t row = block_index() * kTeams + team;
    if (row - team >= p.rows) return;
    const bool any = row < p.rows;
    Row8<kX16> x[kChunks];
    Row8<kR16> r[kChunks];
    Row8<kG16> g[kChunks];
    int c[kChunks];
    bool put[kChunks];
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
        c[i] = (i * kTeam + mine) * kWaveCols + lane * kLaneCols;
        put[i] = any && c[i] < p.d;
        x[i].zero();
        if (put[i]) x[i].load(p.x, row * p.d + c[i]);
        if constexpr (kRes) {
            r[i].zero();
            if (put[i]) r[i].load(p.residual, row * p.d + c[i]);
        }
        g[i].zero();
        if (put[i]) g[i].load(p.gamma, c[i]);
    }
    float h[kChunks][8];
    double sum[1] = {0.0};
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
        add_residual<kX16, kRes, kR16>(x[i], r[i], h[i]);
        if constexpr (kRes) {
            if (put[i]) stream8<kR16>(p.h, row * p.d + c[i], h[i]);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[0] = __builtin_fma(static_cast<double>(h[i][e]), static_cast<double>(h[i][e]), sum[0]);
    }
    team_sum<kTeam, 1>(sum, slots + team * kTeam, mine);
    const float rho = static_cast<float>(rsqrt64(__builtin_fma(sum[0], p.inv_d, p.eps)));
#pragma unroll
    for (int i = 0; i < kChunks; ++i) put_chunk<kX16, kG16>(p, h[i], g[i], rho, put[i], row, c[i]);
}

// Rows of any length: a workgroup a row, which is read again for the outputs (each element by the thread that read
// and wrote it before).
template <bool kX16, bool kRes, bool kR16, bool kG16>
__global__ void __launch_bounds__(64 * kMostTeam)
rmsnorm_forward_long_kernel(RmsForwardParams p) {
    __shared__ double slots[kMostTeam];
    const int64_t row = block_index();
    if (row >= p.rows) return;
    constexpr int kStep = kMostTeam * kWaveCols;
    const int c0 = static_cast<int>(threadIdx.x) * kLaneCols;
    double sum[1] = {0.0};
    float h[8];
    for (int c = c0; c < p.d; c += kStep) {
        Row8<kX16> x;
        Row8<kR16> r;
        x.load(p.x, row * p.d + c);
        if constexpr (kRes) r.load(p.residual, row * p.d + c);
        add_residual<kX16, kRes, kR16>(x, r, h);
        if constexpr (kRes) store8<kR16>(p.h, row * p.d + c, h);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[0] = __builtin_fma(static_cast<double>(h[e]), static_cast<double>(h[e]), sum[0]);
    }
    team_sum<kMostTeam, 1>(sum, slots, static_cast<int>(threadIdx.x >> 6));
    const float rho = static_cast<float>(rsqrt64(__builtin_fma(sum[0], p.inv_d, p.eps)));
    for (int c = c0; c - c0 < p.d; c += kStep) {   // all lanes together: they share groups
        const bool put = c < p.d;
        Row8<kRes ? kR16 : kX16> x;
        Row8<kG16> g;
        x.zero();
        g.zero();
        if (put) {
            x.load(kRes ? p.h : p.x, row * p.d + c);
            g.load(p.gamma, c);
        }
        x.get(h);
        put_chunk<kX16, kG16>(p, h, g, rho, put, row, c);
    }
}

// Waves that share a row of d elements (0: none of them holds it).
int team_of(int d) {
    int t = 1;
    while (t <= kMostTeam && d > t * kChunks * kWaveCols) t *= 2;
    return t <= kMostTeam ? t : 0;
}

template <typename F>
hipError_t with_team(int team, F f) {
    switch (team) {
        case 1: return f(std::integral_constant<int, 1>{});
        case 2: return f(std::integral_constant<int, 2>{});
        case 4: return f(std::integral_constant<int, 4>{});
        case 8: return f(std::integral_constant<int, 8>{});
        default: return f(std::integral_constant<int, 16>{});
    }
}

template <bool kX16, bool kRes, bool kR16, bool kG16>
hipError_t forward(const RmsForwardArgs& a, hipStream_t stream) {
    const RmsForwardParams p{a.x, a.residual, a.rows, a.d, 1.0 / a.d, a.eps, a.gamma, a.h, a.y, a.codes, a.scale, a.e8m0};
    const int team = team_of(a.d);
    if (team == 0) {
        rmsnorm_forward_long_kernel<kX16, kRes, kR16, kG16><<<grid_of(a.rows, 1 << 21), 64 * kMostTeam, 0, stream>>>(p);
        return hipGetLastError();
    }
    return with_team(team, [&](auto t) {
        constexpr int kTeam = decltype(t)::value, kWaves = forward_waves(kTeam), kTeams = kWaves / kTeam;
        const int64_t blocks = (a.rows + kTeams - 1) / kTeams;
        rmsnorm_forward_kernel<kX16, kRes, kR16, kG16, kTeam><<<grid_of(blocks, 1 << 21), 64 * kWaves, 0, stream>>>(p);
        return hipGetLastError();
    });
}

template <bool kX16, bool kG16>
hipError_t forward_types(const RmsForwardArgs& a, hipStream_t stream) {
    if (a.residual == nullptr) return forward<kX16, false, kX16, kG16>(a, stream);
    return a.r_bf16 ? forward<kX16, true, true, kG16>(a, stream) : forward<kX16, true, false, kG16>(a, stream);
}

// ---- backward

struct RmsBackwardParams {
    const void* dn;
    const void* h;
    const void* dresidual;   // or nullptr
    int64_t rows;
    int d;
    double inv_d, eps;
    const void* gamma;
    void* dh;
    float* part;             // [workgroups][d] sums of dgamma, or nullptr
};

// A chunk of a row: dr becomes dh = dr + rho (a - h k), a = gamma dn, k = rho^2 mean(a h), and sum, dgamma's, takes dn (h rho).
// Rows far from 1 keep their bits: k is about as large as dh itself and h rho about 1, where rho^3 mean(a h) and dn rho would
// leave fp32's range with h rho^3 mean(a h) and dn h rho still ordinary numbers.
__device__ __forceinline__ void row_gradient(float* dr, float* sum, const float* dn, const float* gamma, const float* h, float rho, float k) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        sum[i] = __builtin_fmaf(dn[i], h[i] * rho, sum[i]);
        dr[i] = __builtin_fmaf(rho, __builtin_fmaf(-h[i], k, dn[i] * gamma[i]), dr[i]);
    }
}

constexpr int backward_waves(int team) { return team < 8 ? 8 : team; }

// Workgroups of teams of kTeam waves walk the rows, the next row's loads in flight behind each (but for the longest
// rows, whose 16 waves leave 128 registers a thread, of which 3 to 11 spill as it is: 2304 x 16384 66.5 us, 4608 x 8192
// 57.2); a lane keeps the sums of dgamma of its columns, the teams' meet in LDS at the end.
template <bool kN16, bool kH16, bool kG16, int kTeam>
__global__ void __launch_bounds__(64 * backward_waves(kTeam))
rmsnorm_backward_kernel(RmsBackwardParams p) {
    constexpr int kWaves = backward_waves(kTeam), kTeams = kWaves / kTeam, kHalf = kWaves * kChunks * kWaveCols / 2;
    constexpr bool kAhead = kTeam < kMostTeam;
    __shared__ double slots[2][2 * kWaves];
    __shared__ float sums[kTeams > 1 ? kHalf : 1];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, team = wave / kTeam, mine = wave % kTeam;
    int c[kChunks];
    Row8<kG16> g[kChunks];
    float acc[kChunks][8];
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
        c[i] = (i * kTeam + mine) * kWaveCols + lane * kLaneCols;
        g[i].zero();
        if (c[i] < p.d) g[i].load(p.gamma, c[i]);
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[i][e] = 0.f;
    }
    struct Loaded {
        Row8<kN16> dn[kChunks];
        Row8<kH16> h[kChunks], dr[kChunks];
    };
    auto load = [&](Loaded& l, int64_t row) {
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
            l.dn[i].zero();
            l.h[i].zero();
            l.dr[i].zero();
            if (row < p.rows && c[i] < p.d) {
                l.dn[i].load(p.dn, row * p.d + c[i]);
                l.h[i].load(p.h, row * p.d + c[i]);
                if (p.dresidual != nullptr) l.dr[i].load(p.dresidual, row * p.d + c[i]);
            }
        }
    };
    const int64_t stride = static_cast<int64_t>(gridDim.x) * kTeams;
    Loaded l;
    if constexpr (kAhead) load(l, static_cast<int64_t>(blockIdx.x) * kTeams + team);
    int turn = 0;
    for (int64_t first = static_cast<int64_t>(blockIdx.x) * kTeams; first < p.rows; first += stride) {   // every team takes each turn
        const int64_t row = first + team;
        Loaded now;
        if constexpr (kAhead) {
            now = l;
            load(l, row + stride);
        } else {
            load(now, row);
        }
        double s[2] = {0.0, 0.0};
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
            float h[8], a[8], w[8];
            now.h[i].get(h);
            now.dn[i].get(a);
            g[i].get(w);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                s[0] = __builtin_fma(static_cast<double>(h[e]), static_cast<double>(h[e]), s[0]);
                s[1] = __builtin_fma(static_cast<double>(a[e] * w[e]), static_cast<double>(h[e]), s[1]);
            }
        }
        team_sum<kTeam, 2>(s, slots[turn] + team * 2 * kTeam, mine);
        turn ^= 1;
        const double r64 = rsqrt64(__builtin_fma(s[0], p.inv_d, p.eps));
        const float rho = static_cast<float>(r64), k = static_cast<float>(r64 * r64 * (s[1] * p.inv_d));
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
            float h[8], a[8], w[8], v[8];
            now.h[i].get(h);
            now.dn[i].get(a);
            now.dr[i].get(v);
            g[i].get(w);
            row_gradient(v, acc[i], a, w, h, rho, k);
            if (row < p.rows && c[i] < p.d) stream8<kH16>(p.dh, row * p.d + c[i], v);
        }
    }
    if (p.part == nullptr) return;
    if constexpr (kTeams > 1) {
#pragma unroll
        for (int half = kTeams / 2; half > 0; half /= 2) {
            __syncthreads();
            float* at = sums + (team % half) * kTeam * kChunks * kWaveCols;
            if (team >= half && team < 2 * half) {
#pragma unroll
                for (int i = 0; i < kChunks; ++i) store8<false>(at, c[i], acc[i]);
            }
            __syncthreads();
            if (team < half) {
#pragma unroll
                for (int i = 0; i < kChunks; ++i) {
                    Row8<false> o;
                    float v[8];
                    o.load(at, c[i]);
                    o.get(v);
#pragma unroll
                    for (int e = 0; e < 8; ++e) acc[i][e] += v[e];
                }
            }
        }
    }
    if (team == 0) {
#pragma unroll
        for (int i = 0; i < kChunks; ++i)
            if (c[i] < p.d) store8<false>(p.part, static_cast<int64_t>(blockIdx.x) * p.d + c[i], acc[i]);
    }
}

// Rows of any length: a workgroup walks rows, each read twice; the sums of dgamma are in its part of the workspace.
template <bool kN16, bool kH16, bool kG16>
__global__ void __launch_bounds__(64 * kMostTeam)
rmsnorm_backward_long_kernel(RmsBackwardParams p) {
    __shared__ double slots[2][2 * kMostTeam];
    constexpr int kStep = kMostTeam * kWaveCols;
    const int c0 = static_cast<int>(threadIdx.x) * kLaneCols;
    int turn = 0;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        double s[2] = {0.0, 0.0};
        float h[8], a[8], w[8], v[8];
        auto load = [&](int c) {
            Row8<kN16> x;
            Row8<kH16> y;
            Row8<kG16> z;
            x.load(p.dn, row * p.d + c);
            y.load(p.h, row * p.d + c);
            z.load(p.gamma, c);
            x.get(a);
            y.get(h);
            z.get(w);
        };
        for (int c = c0; c < p.d; c += kStep) {
            load(c);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                s[0] = __builtin_fma(static_cast<double>(h[e]), static_cast<double>(h[e]), s[0]);
                s[1] = __builtin_fma(static_cast<double>(a[e] * w[e]), static_cast<double>(h[e]), s[1]);
            }
        }
        team_sum<kMostTeam, 2>(s, slots[turn], static_cast<int>(threadIdx.x >> 6));
        turn ^= 1;
        const double r64 = rsqrt64(__builtin_fma(s[0], p.inv_d, p.eps));
        const float rho = static_cast<float>(r64), k = static_cast<float>(r64 * r64 * (s[1] * p.inv_d));
        for (int c = c0; c < p.d; c += kStep) {
            load(c);
            Row8<kH16> o;
            o.zero();
            if (p.dresidual != nullptr) o.load(p.dresidual, row * p.d + c);
            o.get(v);
            Row8<false> old;
            float sum[8];
            old.zero();
            const int64_t at = static_cast<int64_t>(blockIdx.x) * p.d + c;
            if (p.part != nullptr && row != blockIdx.x) old.load(p.part, at);
            old.get(sum);
            row_gradient(v, sum, a, w, h, rho, k);
            if (p.part != nullptr) store8<false>(p.part, at, sum);
            store8<kH16>(p.dh, row * p.d + c, v);
        }
    }
}

// dgamma = (dgamma +) the parts' sum, in an order that their number alone decides: 32 columns a workgroup, thread t
// parts t / 32, + 32, ..
template <bool kG16>
__global__ void __launch_bounds__(1024)
dgamma_kernel(const float* __restrict__ part, int parts, int d, void* dgamma, bool accumulate) {
    __shared__ float sums[32][33];
    const int lane = static_cast<int>(threadIdx.x & 31), slice = static_cast<int>(threadIdx.x >> 5);
    const int c = static_cast<int>(blockIdx.x) * 32 + lane;
    float s = 0.f;
    if (c < d) {
#pragma unroll 8
        for (int q = slice; q < parts; q += 32) s += part[static_cast<int64_t>(q) * d + c];
    }
    sums[slice][lane] = s;
    __syncthreads();
    if (slice != 0 || c >= d) return;
#pragma unroll
    for (int q = 1; q < 32; ++q) s += sums[q][lane];
    if constexpr (kG16) {
        uint16_t* out = static_cast<uint16_t*>(dgamma) + c;
        if (accumulate) s += bf16_lo(*out);
        *out = static_cast<uint16_t>(pack_bf16x2(s, 0.f));
    } else {
        float* out = static_cast<float*>(dgamma) + c;
        *out = accumulate ? s + *out : s;
    }
}

// Workgroups of the backward pass: one a CU.
int backward_parts(int64_t rows, int d) {
    const int team = team_of(d), teams = team == 0 ? 1 : backward_waves(team) / team;
    return static_cast<int>(std::min<int64_t>(device_cu_count(), (rows + teams - 1) / teams));
}

template <bool kN16, bool kH16, bool kG16>
hipError_t backward(const RmsBackwardArgs& a, hipStream_t stream) {
    const RmsBackwardParams p{a.dn, a.h, a.dresidual, a.rows, a.d, 1.0 / a.d, a.eps, a.gamma, a.dh,
                              a.dgamma != nullptr ? static_cast<float*>(a.workspace) : nullptr};
    const int parts = backward_parts(a.rows, a.d);
    if (parts > 0) {
        const int team = team_of(a.d);
        hipError_t e;
        if (team == 0) {
            rmsnorm_backward_long_kernel<kN16, kH16, kG16><<<parts, 64 * kMostTeam, 0, stream>>>(p);
            e = hipGetLastError();
        } else {
            e = with_team(team, [&](auto t) {
                constexpr int kTeam = decltype(t)::value;
                rmsnorm_backward_kernel<kN16, kH16, kG16, kTeam><<<parts, 64 * backward_waves(kTeam), 0, stream>>>(p);
                return hipGetLastError();
            });
        }
        if (e != hipSuccess || a.dgamma == nullptr) return e;
    }
    if (a.dgamma == nullptr || (parts == 0 && a.accumulate)) return hipSuccess;
    auto kernel = a.dg_bf16 ? dgamma_kernel<true> : dgamma_kernel<false>;
    kernel<<<(a.d + 31) / 32, 1024, 0, stream>>>(static_cast<const float*>(a.workspace), parts, a.d, a.dgamma, a.accumulate);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_rmsnorm_forward(const RmsForwardArgs& a, hipStream_t stream) {
    if (a.x_bf16) return a.g_bf16 ? forward_types<true, true>(a, stream) : forward_types<true, false>(a, stream);
    return a.g_bf16 ? forward_types<false, true>(a, stream) : forward_types<false, false>(a, stream);
}

size_t rmsnorm_backward_workspace_bytes(int64_t rows, int d) {
    return static_cast<size_t>(backward_parts(rows, d)) * static_cast<size_t>(d) * sizeof(float);
}

hipError_t launch_rmsnorm_backward(const RmsBackwardArgs& a, hipStream_t stream) {
    auto pick = [&](auto n, auto h) {
        constexpr bool kN = decltype(n)::value, kH = decltype(h)::value;
        return a.g_bf16 ? backward<kN, kH, true>(a, stream) : backward<kN, kH, false>(a, stream);
    };
    constexpr auto yes = std::true_type{};
    constexpr auto no = std::false_type{};
    if (a.dn_bf16) return a.h_bf16 ? pick(yes, yes) : pick(yes, no);
    return a.h_bf16 ? pick(no, yes) : pick(no, no);
}

}  // namespace rtq
