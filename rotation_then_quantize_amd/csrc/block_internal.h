// block_internal.h -- launchers of what stands around the 8-bit linear layers of an MLP block (norm, gated
// feed-forward, gradient norm and clipping), shared between the C-ABI layer and the HIP translation units.  Not
// part of the public interface.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace rtq {

struct RmsForwardArgs {
    const void* x;          // [rows][d]
    bool x_bf16;            // type of x and y
    const void* residual;   // [rows][d], or nullptr
    bool r_bf16;            // type of residual and h
    int64_t rows;
    int d;
    const void* gamma;      // [d]
    bool g_bf16;
    float eps;
    void* h;                // [rows][d] (with residual)
    void* y;                // or nullptr
    void* codes;            // or nullptr
    void* scale;
    bool e8m0;
};
hipError_t launch_rmsnorm_forward(const RmsForwardArgs& a, hipStream_t stream);

struct RmsBackwardArgs {
    const void* dn;         // [rows][d]
    bool dn_bf16;
    const void* h;          // [rows][d]
    bool h_bf16;            // type of h, dresidual and dh
    const void* dresidual;  // or nullptr
    int64_t rows;
    int d;
    const void* gamma;
    bool g_bf16;
    float eps;
    void* dh;
    void* dgamma;           // [d], or nullptr
    bool dg_bf16;
    bool accumulate;
    void* workspace;        // rmsnorm_backward_workspace_bytes, if dgamma is given
};
hipError_t launch_rmsnorm_backward(const RmsBackwardArgs& a, hipStream_t stream);
size_t rmsnorm_backward_workspace_bytes(int64_t rows, int d);

// y = act(g) u, [g u] = x W^T, W [2 N][K] (the gate's rows first), N a multiple of 128.
struct GluArgs {
    const void* x;          // [T][K] e4m3
    const void* x_scale;    // [groups of K][T]
    const void* w;          // [2 N][K] e4m3
    const void* w_scale;    // [2 N / 128][groups of K]
    bool e8m0;              // type of all scales
    int64_t T;
    int N, K;
    int act;                // rtq_act
    void* h_codes;          // [T][2 N] e4m3, or nullptr
    void* h_scale;          // [2 N / 128][T]
    void* y;                // [T][N], or nullptr
    bool y_bf16;
    void* y_codes;          // [T][N] e4m3, or nullptr (then y is set)
    void* y_scale;          // [N / 128][T]
    void* workspace;
    size_t ws_bytes;
};
hipError_t launch_fp8_glu(const GluArgs& a, hipStream_t stream);
size_t fp8_glu_workspace_bytes(int64_t T, int N, int K);

struct GluBackwardArgs {
    const void* dy;         // [T][N]
    bool bf16;              // type of dy and dh
    const void* h_codes;    // [T][2 N] e4m3
    const void* h_scale;
    bool e8m0;              // type of both scales
    int64_t T;
    int N;
    int act;
    void* dh;               // [T][2 N], or nullptr
    void* dh_codes;         // [T][2 N], or nullptr
    bool e5m2;
    void* dh_scale;
};
hipError_t launch_glu_backward(const GluBackwardArgs& a, hipStream_t stream);

struct TensorSpan {
    const void* data;
    void* out;
    int64_t n;
    bool bf16;
};
// Sum of squares of all tensors, its root to *norm.
hipError_t launch_grad_norm(const TensorSpan* t, int count, float* norm, void* workspace, hipStream_t stream);
size_t grad_norm_workspace_bytes(const TensorSpan* t, int count);
// out = data * min(1, most / (*norm + 1e-6))
hipError_t launch_grad_clip(const TensorSpan* t, int count, const float* norm, float most, hipStream_t stream);

}  // namespace rtq
