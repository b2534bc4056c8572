// grads.hip -- the 2-norm of many tensors together and their scaling to at most a given norm, on gfx950:
//
//   norm = sqrt(sum over tensors and elements of g^2),  out = g min(1, most / (norm + 1e-6))
//
// Bound by HBM: each element is read for the norm, and read and written for the scaling.  Sums are held in fp64: no
// square of an fp32 value overflows there, and with sums of fixed ranges added in a fixed order equal calls give equal
// bits.  Tensors go to the kernel as its argument, kMost a launch, cut into pieces of equal size; a workgroup takes one.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "block_internal.h"
#include "fp8_device.h"

namespace rtq {
namespace {

using namespace fp8;

constexpr int kThreads = 256;
constexpr int kMost = 96;                        // tensors of a launch: their table fits the 4 KB of arguments
constexpr int kPass = kThreads * 8;              // elements a workgroup takes at a time
constexpr int64_t kScalePiece = 2 * kPass;       // elements of a piece that is scaled, or more

struct Table {
    const void* data[kMost];
    void* out[kMost];
    int64_t n[kMost];
    uint32_t first[kMost + 1];                   // piece that each tensor begins with, and their number
    uint32_t bf16[kMost / 32];
    int64_t piece;                               // elements a workgroup takes
    int count;
};
static_assert(sizeof(Table) + 64 <= 4096, "kernel arguments");

struct Place {
    int tensor;
    int64_t begin, end;                          // elements of the piece
    bool bf16;
};

// The piece of this workgroup: of the last tensor that begins at or before it, which all lanes look for at once (arguments are
// read from host memory: a search in steps takes as many of its round trips).
__device__ __forceinline__ Place place(const Table& t, uint32_t piece) {
    static_assert(kMost <= 128, "two tensors a lane");
    const int lane = static_cast<int>(threadIdx.x & 63);
    const uint32_t* first = t.first;
    const uint32_t a = first[min(lane, t.count)], b = first[min(lane + 64, t.count)];
    const int before = __popcll(__ballot(lane < t.count && a <= piece)) + __popcll(__ballot(lane + 64 < t.count && b <= piece));
    const int lo = __builtin_amdgcn_readfirstlane(before) - 1;
    const int64_t begin = static_cast<int64_t>(piece - t.first[lo]) * t.piece;
    return {lo, begin, min(begin + t.piece, t.n[lo]), (t.bf16[lo / 32] >> (lo % 32) & 1u) != 0u};
}

__device__ __forceinline__ double block_sum(double v, double* slots) {
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) v += __shfl_xor(v, m);
    if ((threadIdx.x & 63) == 0) slots[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0;
#pragma unroll 1
    for (unsigned w = 0; w < blockDim.x / 64; ++w) v += slots[w];
    return v;
}

template <bool kBF16>
__device__ __forceinline__ double squares(const void* data, int64_t begin, int64_t end) {
    double s = 0.0;
    int64_t i = begin + threadIdx.x * 8;
#pragma unroll 4
    for (; i + 8 <= end; i += kThreads * 8) {
        Row8<kBF16> r;
        float v[8];
        r.load(data, i);
        r.get(v);
#pragma unroll
        for (int e = 0; e < 8; ++e) s = __builtin_fma(static_cast<double>(v[e]), static_cast<double>(v[e]), s);
    }
    for (; i < end; ++i) {   // one thread's, less than 8
        const float v = kBF16 ? bf16_lo(static_cast<const uint16_t*>(data)[i]) : static_cast<const float*>(data)[i];
        s = __builtin_fma(static_cast<double>(v), static_cast<double>(v), s);
    }
    return s;
}

__global__ void __launch_bounds__(kThreads)
grad_squares_kernel(Table t, double* __restrict__ part) {
    __shared__ double slots[kThreads / 64];
    const Place w = place(t, blockIdx.x);
    const double s = block_sum(w.bf16 ? squares<true>(t.data[w.tensor], w.begin, w.end)
                                      : squares<false>(t.data[w.tensor], w.begin, w.end), slots);
    if (threadIdx.x == 0) part[blockIdx.x] = s;
}

__global__ void __launch_bounds__(1024)
grad_root_kernel(const double* __restrict__ part, int64_t n, float* norm) {
    __shared__ double slots[1024 / 64];
    double s = 0.0;
    for (int64_t i = threadIdx.x; i < n; i += 4 * 1024) {   // four loads at once
        double v[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = part[min<int64_t>(i + 1024 * q, n - 1)];
#pragma unroll
        for (int q = 0; q < 4; ++q) s += i + 1024 * q < n ? v[q] : 0.0;
    }
    s = block_sum(s, slots);
    if (threadIdx.x == 0) *norm = static_cast<float>(sqrt(s));
}

template <bool kBF16>
__device__ __forceinline__ void scale(const void* data, void* out, int64_t begin, int64_t end, float c) {
    int64_t i = begin + threadIdx.x * 8;
#pragma unroll 4
    for (; i + 8 <= end; i += kThreads * 8) {
        Row8<kBF16> r;
        float v[8];
        r.load(data, i);
        r.get(v);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= c;
        stream8<kBF16>(out, i, v);
    }
    for (; i < end; ++i) {
        if constexpr (kBF16)
            static_cast<uint16_t*>(out)[i] = static_cast<uint16_t>(pack_bf16x2(bf16_lo(static_cast<const uint16_t*>(data)[i]) * c, 0.f));
        else
            static_cast<float*>(out)[i] = static_cast<const float*>(data)[i] * c;
    }
}

__global__ void __launch_bounds__(kThreads)
grad_scale_kernel(Table t, const float* __restrict__ norm, float most) {
    const float c0 = most / (*norm + 1e-6f);
    const float c = c0 > 1.f ? 1.f : c0;         // a NaN stays
    const Place w = place(t, gridDim.x - 1 - blockIdx.x);   // the other way round: the norm's pass has left the last pieces in the cache
    const void* data = t.data[w.tensor];
    void* out = t.out[w.tensor];
    if (c == 1.f && data == out) return;         // nothing to change
    if (w.bf16)
        scale<true>(data, out, w.begin, w.end, c);
    else
        scale<false>(data, out, w.begin, w.end, c);
}

// Elements of a piece whose squares are summed: about 2048 pieces in all, 8 a CU (805 MB of bf16: 139 us, with pieces of 16384
// 158; their sums are two loads a thread).  What is scaled goes in pieces of 4096 (norm and scaling of 805 MB 400 us, with
// 2048 elements 404, 8192 409, 16384 415, 32768 425; with stores through the cache, which push out what the norm's pass has
// left there, 454).
// Beyond 2^34 elements pieces are larger, so that a launch has fewer than 2^32 work-items.
int64_t piece_of(const TensorSpan* t, int count, int64_t least, int64_t pieces) {
    int64_t total = 0;
    for (int i = 0; i < count; ++i) total += t[i].n;
    return std::max(least / kPass, (total + pieces * kPass - 1) / (pieces * kPass)) * kPass;
}
int64_t norm_piece(const TensorSpan* t, int count) { return piece_of(t, count, 4 * kPass, 2048); }

// f(table, its pieces) for as many tables as the tensors need.
template <typename F>
hipError_t each_table(const TensorSpan* t, int count, int64_t piece, F f) {
    Table table{};
    table.piece = piece;
    int64_t at = 0;
    auto flush = [&]() {
        table.first[table.count] = static_cast<uint32_t>(at);
        const hipError_t e = table.count > 0 ? f(table, at) : hipSuccess;
        table = Table{};
        table.piece = piece;
        at = 0;
        return e;
    };
    for (int i = 0; i < count; ++i) {
        if (t[i].n == 0) continue;
        if (table.count == kMost) {
            const hipError_t e = flush();
            if (e != hipSuccess) return e;
        }
        const int k = table.count++;
        table.data[k] = t[i].data;
        table.out[k] = t[i].out;
        table.n[k] = t[i].n;
        table.first[k] = static_cast<uint32_t>(at);
        if (t[i].bf16) table.bf16[k / 32] |= 1u << (k % 32);
        at += (t[i].n + piece - 1) / piece;
    }
    return flush();
}

}  // namespace

size_t grad_norm_workspace_bytes(const TensorSpan* t, int count) {
    const int64_t piece = norm_piece(t, count);
    int64_t pieces = 0;
    for (int i = 0; i < count; ++i) pieces += (t[i].n + piece - 1) / piece;
    return static_cast<size_t>(pieces) * sizeof(double);
}

hipError_t launch_grad_norm(const TensorSpan* t, int count, float* norm, void* workspace, hipStream_t stream) {
    double* part = static_cast<double*>(workspace);
    int64_t done = 0;
    const hipError_t e = each_table(t, count, norm_piece(t, count), [&](const Table& table, int64_t n) {
        grad_squares_kernel<<<static_cast<unsigned>(n), kThreads, 0, stream>>>(table, part + done);
        done += n;
        return hipGetLastError();
    });
    if (e != hipSuccess) return e;
    grad_root_kernel<<<1, 1024, 0, stream>>>(part, done, norm);
    return hipGetLastError();
}

hipError_t launch_grad_clip(const TensorSpan* t, int count, const float* norm, float most, hipStream_t stream) {
    return each_table(t, count, piece_of(t, count, kScalePiece, 1 << 22), [&](const Table& table, int64_t n) {
        grad_scale_kernel<<<static_cast<unsigned>(n), kThreads, 0, stream>>>(table, norm, most);
        return hipGetLastError();
    });
}

}  // namespace rtq
