// fp8_tile.h -- what the 8-bit products' tile kernels share: buffer loads into LDS, waits, and the
// matrix instruction.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp8_device.h"

// The LDS-writing loads set M0 in inline assembly; M0 is otherwise unused by these kernels.
#pragma clang diagnostic ignored "-Winline-asm"

namespace rtq {
namespace fp8 {

constexpr int BK = 128;                      // reduction bytes per LDS stage: one block of scales
constexpr int kBufferWord3 = 0x00020000;     // gfx9 buffer descriptor word 3 (raw, 32-bit dwords)
constexpr uint32_t kOob = 0x80000000u;       // an offset past every descriptor used here: loads give 0

// Raw buffer descriptor over [base, base + bytes): loads at offsets >= bytes return zero.
__device__ __forceinline__ v4i make_rsrc(const void* base, uint32_t bytes) {
    const uint64_t b = reinterpret_cast<uint64_t>(base);
    v4i r;
    r.x = __builtin_amdgcn_readfirstlane(static_cast<int>(static_cast<uint32_t>(b)));
    r.y = __builtin_amdgcn_readfirstlane(static_cast<int>(static_cast<uint32_t>(b >> 32) & 0xffffu));
    r.z = __builtin_amdgcn_readfirstlane(static_cast<int>(bytes));
    r.w = kBufferWord3;
    return r;
}

// 16 bytes per lane from buffer offset voff to LDS address lds_addr + 16 * lane.
// Wait states, which the hardware does not check and the compiler inserts for its own loads only: one between the
// write of M0 and the load, and five between a vector instruction that wrote the descriptor (make_rsrc's
// v_readfirstlane) and the load.
__device__ __forceinline__ void load_to_lds(v4i rsrc, uint32_t voff, uint32_t lds_addr) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 :
                 : "s"(__builtin_amdgcn_readfirstlane(static_cast<int>(lds_addr))), "v"(voff), "s"(rsrc)
                 : "memory", "m0");
}

__device__ __forceinline__ void barrier() { asm volatile("s_barrier" ::: "memory"); }
// orders a wave's own LDS accesses against the barrier that hands their memory on
__device__ __forceinline__ void lds_done() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }
// Wait until at most n vector-memory operations of this wave are outstanding.
template <int n>
__device__ __forceinline__ void wait_vmcnt() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(n) : "memory");
}

typedef __attribute__((address_space(3))) v2i* lds_v2i;
// 8 x 16 bytes transposed: the 16 lanes of a group give the addresses of 8 bytes each, two lanes to a
// row; lane i of the group gets byte i of the rows, first row first.
__device__ __forceinline__ v2i read_tr8(uint32_t lds_addr) {
    return __builtin_amdgcn_ds_read_tr8_b64_v2i32(reinterpret_cast<lds_v2i>(lds_addr));
}

typedef short v4s __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4s* lds_v4s;
// 4 x 16 16-bit elements transposed: the 16 lanes of a group give the addresses of 4 elements each, four
// lanes to a row; lane i of the group gets element i of the rows, first row first.
__device__ __forceinline__ v2i read_tr16(uint32_t lds_addr) {
    return __builtin_bit_cast(v2i, __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<lds_v4s>(lds_addr)));
}

// Two 16 x 16 x 32 bf16 products, 16 elements of the reduction a lane; layout as below.
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
__device__ __forceinline__ v4f mfma_bf16(const v8i& x, const v8i& y, v4f c) {
    c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, v4i{x[0], x[1], x[2], x[3]}),
                                                __builtin_bit_cast(v8bf, v4i{y[0], y[1], y[2], y[3]}), c, 0, 0, 0);
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, v4i{x[4], x[5], x[6], x[7]}),
                                                   __builtin_bit_cast(v8bf, v4i{y[4], y[5], y[6], y[7]}), c, 0, 0, 0);
}

// Where transposed weights sit in LDS rows of kBytes (one n of the block): chunk c (16 bytes) of row r at
// c ^ tr_swizzle(r), so that a transposing read's 8 rows of one chunk, and those of the next lane group 16
// rows further on, touch all banks once.
template <int kBytes>
__device__ __forceinline__ int tr_swizzle(int row) {
    static_assert(kBytes == 16 || kBytes == 32 || kBytes == 64 || kBytes == 128 || kBytes == 256, "row bytes");
    if constexpr (kBytes == 256) return (row & 7) | ((row >> 4) & 1) << 3;
    if constexpr (kBytes == 128) return ((row >> 1) & 3) | ((row >> 4) & 1) << 2;
    if constexpr (kBytes == 64) return ((row >> 2) & 1) | ((row >> 4) & 1) << 1;
    if constexpr (kBytes == 32) return (row >> 4) & 1;
    return 0;
}

// 16 x 16 x 128 product of e4m3 (first operand: weights) and e4m3 or e5m2 codes, 32 codes of one row a
// lane.  Lane l of the result holds column l % 16 (second operand's row), rows 4 (l / 16) .. +4.
template <bool kE5M2>
__device__ __forceinline__ v4f mfma(const v8i& w, const v8i& a, v4f c) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, a, c, 0, kE5M2 ? 1 : 0, 0, 0, 0, 0);
}

// The same with E8M0 scales, added to c: byte kByte of `scales` is that of the second operand's row (the
// lane's), the byte above it the weight block's.
template <bool kE5M2, int kByte>
__device__ __forceinline__ v4f mfma_scaled(const v8i& w, const v8i& a, v4f c, int scales) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, a, c, 0, kE5M2 ? 1 : 0, kByte + 1, scales, kByte, scales);
}

// part[0] + part[n] + part[2 n] + .., in order, `split` terms; four are loaded at a time (one at a time, each load's
// latency would be paid in turn: 64 x 1024 outputs in ten parts, product and sum 12.9 us, 11.7 so).
template <typename T>
__device__ __forceinline__ T sum_parts(const float* part, int split, int64_t n) {
    T s = *reinterpret_cast<const T*>(part);
    for (int k = 1; k < split; k += 4) {
        T x[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) x[q] = *reinterpret_cast<const T*>(part + min(k + q, split - 1) * n);
#pragma unroll
        for (int q = 0; q < 4; ++q) s = k + q < split ? s + x[q] : s;
    }
    return s;
}

// Four consecutive outputs of row m from column n.
__device__ __forceinline__ void store4(void* y, bool bf16, int64_t M, int64_t N, int64_t m, int64_t n, const v4f& v) {
    if (m >= M || n >= N) return;
    const int64_t at = m * N + n;
    if (n + 4 <= N && N % 4 == 0) {
        if (bf16)
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(y) + at) = uint2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
        else
            *reinterpret_cast<v4f*>(static_cast<float*>(y) + at) = v;
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (n + i < N) {
            if (bf16)
                static_cast<uint16_t*>(y)[at + i] = static_cast<uint16_t>(pack_bf16x2(v[i], 0.0f));
            else
                static_cast<float*>(y)[at + i] = v[i];
        }
    }
}

// Kernel arguments of a product: out[m][n] = sum over the reduction r of a[m][r] w[n][r] (or w[r][n]).
struct Fp8GemmParams {
    const uint8_t* a;                     // [M][R]
    const void* a_scale;                  // [blocks of R][M]
    const uint8_t* w;                     // [N][R], or transposed [R][N]
    const void* w_scale;
    int64_t M, N;
    int R;
    int tiles_m, tiles_n;
    int64_t w_out_stride, w_red_stride;   // weight scale of (output block, reduction block)
    int split;                            // equal ranges of the reduction per tile
    void* y;                              // output (split 1), or fp32 partials [split][M][N]
    bool y_bf16, e8m0;
};

}  // namespace fp8

struct Fp8GemmArgs;
fp8::Fp8GemmParams fp8_gemm_params(const Fp8GemmArgs& g);
// The product for a few rows or a small output (fp8_small.hip), from codes.
bool fp8_small_takes(int64_t M, int64_t N, int R, bool trans);
hipError_t launch_fp8_small(const fp8::Fp8GemmParams& g, bool trans, bool e5m2, hipStream_t stream);
// Tiles of 256 x 256; reductions of at least two blocks.
hipError_t launch_fp8_gemm_large(const fp8::Fp8GemmParams& g, bool trans, bool e5m2, hipStream_t stream);

}  // namespace rtq
