// fp8_rows.hip -- the passes over rows of the 8-bit floating point layer on gfx950: quantise (groups
// of 128 along a row, or 128 x 128 blocks of a weight), read back, and an activation function with
// its input kept in 8 bits, forward and backward.
//
// A block's scale is the power of two 2^e with amax in (top / 2, top] * 2^e, so x / 2^e is exact and
// the only rounding is the code's own.  A power of two costs no precision against amax / top (the
// codes are floating point; only values that reach the subnormal codes, 2^-14 below amax, have one
// bit less), lets the matrix cores apply the scale, and makes the decoded value exact in bf16.
//
// All of it is bound by HBM: a bf16 element is read once (2 bytes) and its code (1 byte) and, per
// group, its scale written once.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "../../include/rtq.h"
#include "fp8_act.h"
#include "fp8_device.h"
#include "fp8_internal.h"

namespace rtq {
namespace {

using namespace fp8;

constexpr int kThreads = 256;
constexpr int kWaveCols = 512;   // a wave's columns: four groups of 16 lanes, 8 elements a lane

// What a row pass writes beside the codes of its input.
enum RowY : int { kNoY = 0, kYRows = 1, kYCodes = 2 };

struct RowsOut {
    void* codes;
    void* scale;
    void* y;
    void* y_codes;
    void* y_scale;
    bool e8m0;
};

// A wave takes kRows rows of 512 columns: 16 lanes a group, 8 elements a lane.  All the rows' loads are
// issued first.  Lane 16 g + r keeps the exponent of group g in row r, so that the wave stores each
// group's scales as one run of the group-major array.
template <bool kBF16, bool kE5M2, int kAct, int kY, int kRows>
__global__ void __launch_bounds__(kThreads)
fp8_rows_kernel(const void* __restrict__ x, int64_t rows, int d, int col_waves, RowsOut o) {
    const int lane = threadIdx.x & 63;
    const int64_t wave = block_index() * (kThreads / 64) + (threadIdx.x >> 6);
    const int64_t r0 = wave / col_waves * kRows;
    const int c = static_cast<int>(wave % col_waves) * kWaveCols + lane * 8;
    if (r0 >= rows) return;
    const bool in = c < d;   // d is a multiple of 16: a lane's 8 elements are all in or all out
    Row8<kBF16> in8[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        in8[r].zero();
        if (in && r0 + r < rows) in8[r].load(x, (r0 + r) * d + c);
    }
    int keep = 0, keep_y = 0;
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        float v[8];
        in8[r].get(v);
        uint2 q;
        const int e = quantise8<kE5M2>(v, &q);
        if ((lane & 15) == r) keep = e;
        const bool put = in && r0 + r < rows;
        const int64_t at = (r0 + r) * d + c;
        if (put) *reinterpret_cast<uint2*>(static_cast<uint8_t*>(o.codes) + at) = q;
        if constexpr (kY != kNoY) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = act_value<kAct>(v[i]);
        }
        if constexpr (kY == kYRows) {
            if (put) store8<kBF16>(o.y, at, v);
        }
        if constexpr (kY == kYCodes) {
            const int ey = quantise8<false>(v, &q);
            if ((lane & 15) == r) keep_y = ey;
            if (put) *reinterpret_cast<uint2*>(static_cast<uint8_t*>(o.y_codes) + at) = q;
        }
    }
    // the wave's group g = lane / 16 begins at column c - 8 (lane % 16)
    const int c0 = c - 8 * (lane & 15);
    const int r = lane & 15;
    if (r < kRows && r0 + r < rows && c0 < d) {
        const int64_t at = static_cast<int64_t>(c0 / kFp8Block) * rows + r0 + r;
        store_scale(o.scale, o.e8m0, at, keep);
        if constexpr (kY == kYCodes) store_scale(o.y_scale, o.e8m0, at, keep_y);
    }
}

// Rows per wave: two loads in flight for each lane, and many waves (4608 rows, us:
//                            1        2        4        8        16
//   quantise 4096 columns   14.2     13.3     13.4     14.2     16.4
//   quantise 16384          45.1     40.9     41.9     45.2     47.2
//   GELU (tanh) 16384       69.1     68.2     69.8     77.5     84.5
// at 40.9 and 68.2 us 5.5 TB/s: more rows fill a cache line of scales, but even out worse over the CUs).  One
// where there are fewer waves than the card has SIMDs for twice over (2048), so that no SIMD idles: there a pass takes
// a launch's time either way (64 to 256 rows x 4096: 5.1-5.5 us with one and with two).
template <bool kBF16, bool kE5M2, int kAct, int kY>
hipError_t launch_rows(const void* x, int64_t rows, int d, const RowsOut& o, hipStream_t stream) {
    const int col_waves = (d + kWaveCols - 1) / kWaveCols;
    auto go = [&](auto per) {
        constexpr int kRows = decltype(per)::value;
        const int64_t waves = (rows + kRows - 1) / kRows * col_waves;
        fp8_rows_kernel<kBF16, kE5M2, kAct, kY, kRows>
            <<<grid_of((waves + kThreads / 64 - 1) / (kThreads / 64)), kThreads, 0, stream>>>(x, rows, d, col_waves, o);
        return hipGetLastError();
    };
    return rows * col_waves >= 2048 ? go(std::integral_constant<int, 2>{}) : go(std::integral_constant<int, 1>{});
}

// A workgroup takes one 128 x 128 block of a weight: 16 lanes a row, 8 elements a lane, 16 rows a pass.
template <bool kBF16, bool kE5M2>
__global__ void __launch_bounds__(kThreads)
fp8_blocks_kernel(const void* __restrict__ x, int64_t rows, int d, void* __restrict__ codes, void* __restrict__ scale,
                  bool e8m0) {
    constexpr int kPass = kThreads / 16;
    __shared__ uint32_t s_max[kThreads / 64];
    const int groups = (d + kFp8Block - 1) / kFp8Block;
    const int64_t br = block_index() / groups;
    const int bc = static_cast<int>(block_index() % groups);
    if (br * kFp8Block >= rows) return;
    const int64_t r0 = br * kFp8Block + threadIdx.x / 16;
    const int c = bc * kFp8Block + (threadIdx.x % 16) * 8;
    Row8<kBF16> in8[kFp8Block / kPass];
#pragma unroll
    for (int p = 0; p < kFp8Block / kPass; ++p) {
        in8[p].zero();
        if (c < d && r0 + p * kPass < rows) in8[p].load(x, (r0 + p * kPass) * d + c);
    }
    uint32_t m = 0u;
#pragma unroll
    for (int p = 0; p < kFp8Block / kPass; ++p) {
        float v[8];
        in8[p].get(v);
        m = max(m, amax8(v));
    }
    m = max16(m);
    m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 16)));
    m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 32)));
    if ((threadIdx.x & 63) == 0) s_max[threadIdx.x >> 6] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 64; ++w) m = max(m, s_max[w]);
    const int e = scale_exponent<kE5M2>(m);
    const float inv = pow2(-e);
#pragma unroll
    for (int p = 0; p < kFp8Block / kPass; ++p) {
        if (c < d && r0 + p * kPass < rows) {
            float v[8];
            in8[p].get(v);
            uint2 q;
            q.x = encode4<kE5M2>(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
            q.y = encode4<kE5M2>(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv);
            *reinterpret_cast<uint2*>(static_cast<uint8_t*>(codes) + (r0 + p * kPass) * d + c) = q;
        }
    }
    if (threadIdx.x == 0) store_scale(scale, e8m0, br * groups + bc, e);
}

// Elementwise passes over codes: a thread takes 8 elements of kElemRows rows (the gradient of GELU at 2304 x 4096:
// 11.1 us with one, 12.4 with two, 13.5 with four; at 4608 x 16384 73.3, 71.6, 73.5).
constexpr int kElemRows = 2;

template <bool kE5M2, bool kBF16, bool kE8M0>
__global__ void __launch_bounds__(kThreads)
fp8_dequant_kernel(const uint8_t* __restrict__ codes, const void* __restrict__ scale, bool blocks,
                   int64_t rows, int d, int64_t units, void* __restrict__ y) {
    const int64_t u = block_index() * kThreads + threadIdx.x;
    if (u >= units) return;
    const int per_row = d / 8;
    const int c = static_cast<int>(u % per_row) * 8;
    const int64_t r0 = u / per_row * kElemRows;
    const int64_t groups = (d + kFp8Block - 1) / kFp8Block;
    uint2 q[kElemRows];
    float s[kElemRows];
#pragma unroll
    for (int r = 0; r < kElemRows; ++r) {
        if (r0 + r < rows) {
            q[r] = *reinterpret_cast<const uint2*>(codes + (r0 + r) * d + c);
            s[r] = load_scale<kE8M0>(scale, blocks ? (r0 + r) / kFp8Block * groups + c / kFp8Block : c / kFp8Block * rows + r0 + r);
        }
    }
#pragma unroll
    for (int r = 0; r < kElemRows; ++r) {
        if (r0 + r < rows) {
            float v[8];
            decode4<kE5M2>(q[r].x, v);
            decode4<kE5M2>(q[r].y, v + 4);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] *= s[r];
            store8<kBF16>(y, (r0 + r) * d + c, v);
        }
    }
}

template <bool kBF16, int kAct, bool kE8M0>
__global__ void __launch_bounds__(kThreads)
act_backward_kernel(const void* dy, const uint8_t* __restrict__ codes, const void* __restrict__ scale,
                    int64_t rows, int d, int64_t units, void* dh) {   // dh may be dy
    const int64_t u = block_index() * kThreads + threadIdx.x;
    if (u >= units) return;
    const int per_row = d / 8;
    const int c = static_cast<int>(u % per_row) * 8;
    const int64_t r0 = u / per_row * kElemRows;
    uint2 q[kElemRows];
    float s[kElemRows];
    Row8<kBF16> g[kElemRows];
#pragma unroll
    for (int r = 0; r < kElemRows; ++r) {
        if (r0 + r < rows) {
            q[r] = *reinterpret_cast<const uint2*>(codes + (r0 + r) * d + c);
            g[r].load(dy, (r0 + r) * d + c);
            s[r] = load_scale<kE8M0>(scale, c / kFp8Block * rows + r0 + r);
        }
    }
#pragma unroll
    for (int r = 0; r < kElemRows; ++r) {
        if (r0 + r < rows) {
            float v[8], w[8];
            decode4<false>(q[r].x, v);
            decode4<false>(q[r].y, v + 4);
            g[r].get(w);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = w[i] * act_slope<kAct>(v[i] * s[r]);
            store8<kBF16>(dh, (r0 + r) * d + c, v);
        }
    }
}

int64_t elem_units(int64_t rows, int d) { return (rows + kElemRows - 1) / kElemRows * (d / 8); }
dim3 elem_blocks(int64_t units) { return grid_of((units + kThreads - 1) / kThreads); }

template <bool kBF16, int kAct>
hipError_t act_forward(const ActForwardArgs& a, hipStream_t stream) {
    const RowsOut o{a.h_codes, a.h_scale, a.y, a.y_codes, a.y_scale, a.e8m0};
    if (a.y_codes != nullptr) return launch_rows<kBF16, false, kAct, kYCodes>(a.h, a.rows, a.d, o, stream);
    return launch_rows<kBF16, false, kAct, kYRows>(a.h, a.rows, a.d, o, stream);
}

template <bool kBF16, int kAct>
hipError_t act_backward(const ActBackwardArgs& a, hipStream_t stream) {
    const int64_t units = elem_units(a.rows, a.d);
    auto go = [&](auto kernel) {
        kernel<<<elem_blocks(units), kThreads, 0, stream>>>(a.dy, static_cast<const uint8_t*>(a.h_codes), a.h_scale, a.rows,
                                                            a.d, units, a.dh);
        return hipGetLastError();
    };
    return a.e8m0 ? go(act_backward_kernel<kBF16, kAct, true>) : go(act_backward_kernel<kBF16, kAct, false>);
}

}  // namespace

hipError_t launch_fp8_quantize_rows(const Fp8QuantArgs& a, hipStream_t stream) {
    const RowsOut o{a.codes, a.scale, nullptr, nullptr, nullptr, a.e8m0};
    if (a.x_bf16)
        return a.e5m2 ? launch_rows<true, true, 0, kNoY>(a.x, a.rows, a.d, o, stream)
                      : launch_rows<true, false, 0, kNoY>(a.x, a.rows, a.d, o, stream);
    return a.e5m2 ? launch_rows<false, true, 0, kNoY>(a.x, a.rows, a.d, o, stream)
                  : launch_rows<false, false, 0, kNoY>(a.x, a.rows, a.d, o, stream);
}

hipError_t launch_fp8_quantize_blocks(const Fp8QuantArgs& a, hipStream_t stream) {
    const dim3 grid = grid_of(fp8_groups(a.rows) * fp8_groups(a.d));
    auto go = [&](auto kernel) {
        kernel<<<grid, kThreads, 0, stream>>>(a.x, a.rows, a.d, a.codes, a.scale, a.e8m0);
        return hipGetLastError();
    };
    if (a.x_bf16) return a.e5m2 ? go(fp8_blocks_kernel<true, true>) : go(fp8_blocks_kernel<true, false>);
    return a.e5m2 ? go(fp8_blocks_kernel<false, true>) : go(fp8_blocks_kernel<false, false>);
}

hipError_t launch_fp8_dequantize(const Fp8DequantArgs& a, hipStream_t stream) {
    const int64_t units = elem_units(a.rows, a.d);
    auto go = [&](auto kernel) {
        kernel<<<elem_blocks(units), kThreads, 0, stream>>>(static_cast<const uint8_t*>(a.codes), a.scale, a.blocks, a.rows,
                                                            a.d, units, a.y);
        return hipGetLastError();
    };
    auto pick = [&](auto e8m0) {
        constexpr bool k8 = decltype(e8m0)::value;
        if (a.y_bf16) return a.e5m2 ? go(fp8_dequant_kernel<true, true, k8>) : go(fp8_dequant_kernel<false, true, k8>);
        return a.e5m2 ? go(fp8_dequant_kernel<true, false, k8>) : go(fp8_dequant_kernel<false, false, k8>);
    };
    return a.e8m0 ? pick(std::true_type{}) : pick(std::false_type{});
}

hipError_t launch_act_fp8_forward(const ActForwardArgs& a, hipStream_t stream) {
    switch (a.act) {
        case RTQ_ACT_GELU_TANH:
            return a.bf16 ? act_forward<true, RTQ_ACT_GELU_TANH>(a, stream) : act_forward<false, RTQ_ACT_GELU_TANH>(a, stream);
        case RTQ_ACT_GELU:
            return a.bf16 ? act_forward<true, RTQ_ACT_GELU>(a, stream) : act_forward<false, RTQ_ACT_GELU>(a, stream);
        case RTQ_ACT_SILU:
            return a.bf16 ? act_forward<true, RTQ_ACT_SILU>(a, stream) : act_forward<false, RTQ_ACT_SILU>(a, stream);
        default:
            return hipErrorInvalidValue;
    }
}

hipError_t launch_act_fp8_backward(const ActBackwardArgs& a, hipStream_t stream) {
    switch (a.act) {
        case RTQ_ACT_GELU_TANH:
            return a.bf16 ? act_backward<true, RTQ_ACT_GELU_TANH>(a, stream) : act_backward<false, RTQ_ACT_GELU_TANH>(a, stream);
        case RTQ_ACT_GELU:
            return a.bf16 ? act_backward<true, RTQ_ACT_GELU>(a, stream) : act_backward<false, RTQ_ACT_GELU>(a, stream);
        case RTQ_ACT_SILU:
            return a.bf16 ? act_backward<true, RTQ_ACT_SILU>(a, stream) : act_backward<false, RTQ_ACT_SILU>(a, stream);
        default:
            return hipErrorInvalidValue;
    }
}

}  // namespace rtq
