// fp8_device.h -- device helpers of the 8-bit floating point kernels: scales of blocks of 128,
// conversions, and loads.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace rtq {
namespace fp8 {

// A launch of more work-items than a grid's first dimension holds (2^32) goes over two; each kernel returns in
// the workgroups past its last.  The first dimension is a multiple of 8, the number of XCDs.
inline dim3 grid_of(int64_t blocks, int64_t most = 1 << 22) {   // most: times the workgroup's threads, below 2^32
    return blocks <= most ? dim3(static_cast<unsigned>(blocks))
                          : dim3(static_cast<unsigned>(most), static_cast<unsigned>((blocks + most - 1) / most));
}
__device__ __forceinline__ int64_t block_index() { return static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x; }


typedef int v2i __attribute__((ext_vector_type(2)));
typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v2f __attribute__((ext_vector_type(2)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

constexpr uint32_t kInfBits = 0x7f800000u;

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Two fp32 values -> a bf16 pair (the first in the low half), to nearest even.
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
    const v2f v = {lo, hi};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, v2bf));
}

// The exponent e of a block's scale 2^e: the smallest with amax <= top * 2^e, top = 1.75 * 2^8 (e4m3)
// or 1.75 * 2^15 (e5m2), so it follows from amax's exponent and whether its mantissa exceeds 1.75.
// It is at least -120 (both 2^e and 2^-e are then normal fp32 numbers; at most 120 holds by itself)
// and 0 for a block of zeros.  m: the bits of amax, finite.
template <bool kE5M2>
__device__ __forceinline__ int scale_exponent(uint32_t m) {
    constexpr int kTop = kE5M2 ? 15 : 8;
    const int e = static_cast<int>(m >> 23) - 127 - kTop + ((m & 0x7fffffu) > 0x600000u ? 1 : 0);
    return m == 0u ? 0 : max(e, -120);
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// E8M0 byte -> fp32 (0 is 2^-127, a subnormal; 255 is NaN)
__device__ __forceinline__ float e8m0_value(uint32_t b) {
    const uint32_t u = b == 0u ? 0x00400000u : (b == 255u ? 0x7fc00000u : b << 23);
    return __uint_as_float(u);
}
// The scale type is a template parameter wherever scales are loaded: with a run-time flag the compiler may
// turn the choice into lane masks and let the other type's scalar load run, past the end of the array.
template <bool kE8M0>
__device__ __forceinline__ float load_scale(const void* s, int64_t i) {
    if constexpr (kE8M0) return e8m0_value(static_cast<const uint8_t*>(s)[i]);
    return static_cast<const float*>(s)[i];
}
__device__ __forceinline__ void store_scale(void* s, bool e8m0, int64_t i, int e) {
    if (e8m0)
        static_cast<uint8_t*>(s)[i] = static_cast<uint8_t>(e + 127);
    else
        static_cast<float*>(s)[i] = pow2(e);
}

// Four fp32 values -> four codes, each to nearest even (NaN stays NaN, an infinity becomes NaN in
// e4m3, which has none, and stays one in e5m2).
template <bool kE5M2>
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
    int w = 0;
    if constexpr (kE5M2) {
        w = __builtin_amdgcn_cvt_pk_bf8_f32(a, b, w, false);
        w = __builtin_amdgcn_cvt_pk_bf8_f32(c, d, w, true);
    } else {
        w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, w, false);
        w = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
    }
    return static_cast<uint32_t>(w);
}
template <bool kE5M2>
__device__ __forceinline__ void decode4(uint32_t w, float* v) {
    v2f lo, hi;
    if constexpr (kE5M2) {
        lo = __builtin_amdgcn_cvt_pk_f32_bf8(static_cast<int>(w), false);
        hi = __builtin_amdgcn_cvt_pk_f32_bf8(static_cast<int>(w), true);
    } else {
        lo = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w), false);
        hi = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w), true);
    }
    v[0] = lo.x;
    v[1] = lo.y;
    v[2] = hi.x;
    v[3] = hi.y;
}

// Maximum over the 16 lanes of a DPP row, in all of them (rotations by 8, 4, 2 and 1).
__device__ __forceinline__ uint32_t max16(uint32_t m) {
    m = max(m, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(m), 0x128, 0xf, 0xf, true)));
    m = max(m, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(m), 0x124, 0xf, 0xf, true)));
    m = max(m, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(m), 0x122, 0xf, 0xf, true)));
    m = max(m, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(m), 0x121, 0xf, 0xf, true)));
    return m;
}

// Bits of the largest finite magnitude of eight values.  Magnitudes order as their bits, with NaN
// and infinity above every finite one: only where one shows up are they sorted out.
__device__ __forceinline__ uint32_t amax8(const float* v) {
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
    if (m >= kInfBits) {
        m = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t b = __float_as_uint(v[i]) & 0x7fffffffu;
            m = max(m, b < kInfBits ? b : 0u);
        }
    }
    return m;
}

// Eight values of a row from [rows][d] of bf16 or fp32
template <bool kBF16>
struct Row8;
template <>
struct Row8<true> {
    uint4 r;
    __device__ __forceinline__ void load(const void* x, int64_t i) {
        r = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + i);
    }
    __device__ __forceinline__ void zero() { r = uint4{0u, 0u, 0u, 0u}; }
    __device__ __forceinline__ void get(float* v) const {
        v[0] = bf16_lo(r.x); v[1] = bf16_hi(r.x); v[2] = bf16_lo(r.y); v[3] = bf16_hi(r.y);
        v[4] = bf16_lo(r.z); v[5] = bf16_hi(r.z); v[6] = bf16_lo(r.w); v[7] = bf16_hi(r.w);
    }
};
template <>
struct Row8<false> {
    float4 r, s;
    __device__ __forceinline__ void load(const void* x, int64_t i) {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(x) + i);
        r = p[0];
        s = p[1];
    }
    __device__ __forceinline__ void zero() { r = float4{0.f, 0.f, 0.f, 0.f}; s = r; }
    __device__ __forceinline__ void get(float* v) const {
        v[0] = r.x; v[1] = r.y; v[2] = r.z; v[3] = r.w;
        v[4] = s.x; v[5] = s.y; v[6] = s.z; v[7] = s.w;
    }
};
template <bool kBF16>
__device__ __forceinline__ void store8(void* y, int64_t i, const float* v) {
    if constexpr (kBF16) {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(y) + i) =
            uint4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
    } else {
        float4* p = reinterpret_cast<float4*>(static_cast<float*>(y) + i);
        p[0] = float4{v[0], v[1], v[2], v[3]};
        p[1] = float4{v[4], v[5], v[6], v[7]};
    }
}


// The same past the caches, for what is not read again soon.
template <bool kBF16>
__device__ __forceinline__ void stream8(void* y, int64_t i, const float* v) {
    if constexpr (kBF16) {
        const v4i p = {static_cast<int>(pack_bf16x2(v[0], v[1])), static_cast<int>(pack_bf16x2(v[2], v[3])),
                       static_cast<int>(pack_bf16x2(v[4], v[5])), static_cast<int>(pack_bf16x2(v[6], v[7]))};
        __builtin_nontemporal_store(p, reinterpret_cast<v4i*>(static_cast<uint16_t*>(y) + i));
    } else {
        v4f* p = reinterpret_cast<v4f*>(static_cast<float*>(y) + i);
        __builtin_nontemporal_store(v4f{v[0], v[1], v[2], v[3]}, p);
        __builtin_nontemporal_store(v4f{v[4], v[5], v[6], v[7]}, p + 1);
    }
}

// One row's 8 elements of a lane -> 8 codes; returns the group's exponent (the same in its 16 lanes).
template <bool kE5M2>
__device__ __forceinline__ int quantise8(const float* v, uint2* codes) {
    const int e = scale_exponent<kE5M2>(max16(amax8(v)));
    const float inv = pow2(-e);
    codes->x = encode4<kE5M2>(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
    codes->y = encode4<kE5M2>(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv);
    return e;
}

}  // namespace fp8
}  // namespace rtq
