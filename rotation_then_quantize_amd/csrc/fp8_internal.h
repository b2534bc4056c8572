// fp8_internal.h -- launchers of the 8-bit floating point kernels (blocks of 128), shared between
// the C-ABI layer and the HIP translation units.  Not part of the public interface.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace rtq {

constexpr int kFp8Block = 128;   // elements per scale along a row, and rows per scale of a weight
constexpr int64_t fp8_groups(int64_t d) { return (d + kFp8Block - 1) / kFp8Block; }

// Scales are fp32 or E8M0 bytes (2^(b - 127)).  Row groups: [ceil(d / 128)][rows], group-major (the
// products read a tile's 64-256 row scales of one group as one run).  Blocks: [ceil(rows / 128)]
// [ceil(d / 128)].
struct Fp8QuantArgs {
    const void* x;       // [rows][d] fp32 or bf16
    bool x_bf16;
    int64_t rows;
    int d;
    bool e5m2;
    void* codes;         // [rows][d]
    void* scale;
    bool e8m0;
};
hipError_t launch_fp8_quantize_rows(const Fp8QuantArgs& a, hipStream_t stream);
hipError_t launch_fp8_quantize_blocks(const Fp8QuantArgs& a, hipStream_t stream);

struct Fp8DequantArgs {
    const void* codes;
    bool e5m2;
    const void* scale;
    bool e8m0;
    bool blocks;
    int64_t rows;
    int d;
    void* y;             // [rows][d] fp32 or bf16
    bool y_bf16;
};
hipError_t launch_fp8_dequantize(const Fp8DequantArgs& a, hipStream_t stream);

struct ActForwardArgs {
    const void* h;       // [rows][d] fp32 or bf16
    bool bf16;           // type of h and of y
    int64_t rows;
    int d;
    int act;             // rtq_act
    void* h_codes;       // e4m3
    void* h_scale;
    void* y;             // or nullptr
    void* y_codes;       // or nullptr (then y is set)
    void* y_scale;
    bool e8m0;
};
hipError_t launch_act_fp8_forward(const ActForwardArgs& a, hipStream_t stream);

struct ActBackwardArgs {
    const void* dy;      // [rows][d] fp32 or bf16
    bool bf16;           // type of dy and dh
    const void* h_codes;
    const void* h_scale;
    bool e8m0;
    int64_t rows;
    int d;
    int act;
    void* dh;
};
hipError_t launch_act_fp8_backward(const ActBackwardArgs& a, hipStream_t stream);

// out[m][n] = sum over the reduction of a * w with block scales.
//   !trans: out[t][n] = sum_k a[t][k] w[n][k]   (M = T, N_out = N, R = K)
//    trans: out[t][k] = sum_n a[t][n] w[n][k]   (M = T, N_out = K, R = N)
struct Fp8GemmArgs {
    const void* a;        // [M][R] codes
    bool a_e5m2;
    const void* a_scale;  // [ceil(R / 128)][M]
    const void* w;        // e4m3 codes, [N_out][R] or (trans) [R][N_out]
    const void* w_scale;  // the weight's block scales, row-major as stored
    bool e8m0;            // type of both scales
    int64_t M, N;         // rows and columns of the output
    int R;                // reduction length
    bool trans;
    void* y;
    bool y_bf16;
    void* workspace;      // optional: partial sums of a split reduction
    size_t ws_bytes;
    int* parts = nullptr; // if given (y fp32 and workspace the same place): the partial sums [*parts][M][N] are left there, and not added
};
hipError_t launch_fp8_gemm(const Fp8GemmArgs& g, hipStream_t stream);
// The layer for a few rows or a small output in one launch: x [M][R] (fp32 or bf16) is quantised on the way
// to row groups of g's format (g.a and g.a_scale are not used), which go to keep and keep_scale if those
// are given.  Takes what fp8_small_linear_takes says.
bool fp8_small_linear_takes(int64_t M, int64_t N, int R, bool trans);
hipError_t launch_fp8_small_linear(const Fp8GemmArgs& g, const void* x, bool x_bf16, void* keep, void* keep_scale,
                                   hipStream_t stream);
// Workspace bytes launch_fp8_gemm can use for these sizes (0: none).
size_t fp8_gemm_workspace_bytes(int64_t M, int64_t N, int R, bool trans);

struct Fp8WgradArgs {
    const void* dy;       // [T][N] bf16
    const void* x_codes;  // [T][K] e4m3
    const void* x_scale;  // [ceil(K / 128)][T]
    bool e8m0;
    int64_t T;
    int N, K;
    void* dw;             // [N][K]
    bool dw_bf16;
    bool accumulate;
    void* workspace;
    size_t ws_bytes;
};
hipError_t launch_fp8_wgrad(const Fp8WgradArgs& g, hipStream_t stream);
size_t fp8_wgrad_workspace_bytes(int64_t T, int N, int K);

}  // namespace rtq
