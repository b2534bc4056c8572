// fp8_wgrad.h -- what the weight-gradient kernels share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp8_device.h"

namespace rtq {

struct WgradParams {
    const uint16_t* dy;      // [T][N] bf16
    const uint8_t* x;        // [T][K] e4m3
    const void* x_scale;     // [blocks of K][T]
    int64_t T;
    int N, K;
    int tiles_n, tiles_k;
    int split;               // equal ranges of the tokens per tile
    void* dw;                // output (split 1), or fp32 partials [split][N][K]
    bool dw_bf16, accumulate;
};

// Four consecutive values at element `at` of dw.
__device__ __forceinline__ void wgrad_put4(void* dw, bool bf16, bool accumulate, int64_t at, fp8::v4f v) {
    using namespace fp8;
    if (bf16) {
        uint2* q = reinterpret_cast<uint2*>(static_cast<uint16_t*>(dw) + at);
        if (accumulate) {
            const uint2 o = *q;
            v += v4f{bf16_lo(o.x), bf16_hi(o.x), bf16_lo(o.y), bf16_hi(o.y)};
        }
        *q = uint2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    } else {
        v4f* q = reinterpret_cast<v4f*>(static_cast<float*>(dw) + at);
        if (accumulate) v += *q;
        *q = v;
    }
}

// Outputs of many 256 x 256 tiles (fp8_wgrad_large.hip); its loads run two stages of 64 tokens ahead.
bool wgrad_large_takes(int64_t T, int N, int K);
hipError_t launch_wgrad_large(const WgradParams& g, bool e8m0, hipStream_t stream);

}  // namespace rtq
