// fp8_api.cpp -- the C ABI of the 8-bit floating point layer (scales for blocks of 128): argument
// checks and dispatch, with the conventions of rtq_api.cpp.  Every check runs on the host before
// anything is enqueued.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/rtq.h"
#include "fp8_internal.h"
#include "rtq_status.h"

namespace {

using rtq::check_ptr;
using rtq::fail;
using rtq::fp8_groups;
using rtq::hip_status;
using rtq::ok;

constexpr int64_t kMaxDim = 1 << 20;   // row length: a 256-row panel's offsets stay in 31 bits
constexpr int64_t kMaxRows = (int64_t{1} << 31) - 1;

// No C++ exception leaves a C entry point.
template <typename F>
rtq_status guarded(F f) {
    try {
        return f();
    } catch (...) {
        return RTQ_ERR_HIP;
    }
}

rtq_status check_rows(int64_t rows, const char* name) {
    if (rows < 0) return fail(RTQ_ERR_INVALID_ARG, "%s must be >= 0", name);
    if (rows > kMaxRows) return fail(RTQ_ERR_UNSUPPORTED, "%s too large (max %lld)", name, static_cast<long long>(kMaxRows));
    return RTQ_OK;
}

// A row length that codes are stored with.
rtq_status check_len(int64_t d, const char* name, int multiple = 16) {
    if (d <= 0) return fail(RTQ_ERR_INVALID_ARG, "%s must be positive (got %lld)", name, static_cast<long long>(d));
    if (d % multiple != 0)
        return fail(RTQ_ERR_UNSUPPORTED, "%s must be a multiple of %d (got %lld)", name, multiple, static_cast<long long>(d));
    if (d > kMaxDim)
        return fail(RTQ_ERR_UNSUPPORTED, "%s too large (max %lld)", name, static_cast<long long>(kMaxDim));
    return RTQ_OK;
}

rtq_status check_float(rtq_dtype t, const char* name) {
    if (t != RTQ_F32 && t != RTQ_BF16) return fail(RTQ_ERR_UNSUPPORTED, "%s must be RTQ_F32 or RTQ_BF16", name);
    return RTQ_OK;
}
rtq_status check_code(rtq_dtype t, const char* name) {
    if (t != RTQ_E4M3 && t != RTQ_E5M2) return fail(RTQ_ERR_UNSUPPORTED, "%s must be RTQ_E4M3 or RTQ_E5M2", name);
    return RTQ_OK;
}
rtq_status check_scale(rtq_dtype t) {
    if (t != RTQ_F32 && t != RTQ_E8M0) return fail(RTQ_ERR_UNSUPPORTED, "st must be RTQ_F32 or RTQ_E8M0");
    return RTQ_OK;
}
rtq_status check_layout(rtq_fp8_layout l) {
    if (l != RTQ_FP8_ROWS && l != RTQ_FP8_BLOCKS) return fail(RTQ_ERR_INVALID_ARG, "unknown layout %d", static_cast<int>(l));
    return RTQ_OK;
}
rtq_status check_act(rtq_act a) {
    if (a != RTQ_ACT_GELU_TANH && a != RTQ_ACT_GELU && a != RTQ_ACT_SILU)
        return fail(RTQ_ERR_INVALID_ARG, "unknown activation %d", static_cast<int>(a));
    return RTQ_OK;
}
rtq_status check_workspace(const void* ws) {
    if (reinterpret_cast<uintptr_t>(ws) % 16 != 0) return fail(RTQ_ERR_MISALIGNED, "workspace is not 16-byte aligned");
    return RTQ_OK;
}

// An array of `rows` rows: it may be NULL where it is empty.
rtq_status check_row_ptr(const void* p, const char* name, int64_t rows) {
    return rows == 0 && p == nullptr ? RTQ_OK : check_ptr(p, name);
}

size_t align256(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }
// Bytes of the codes and (fp32) scales of row groups in a workspace.
size_t code_part(int64_t rows, int64_t d) { return align256(static_cast<size_t>(rows) * static_cast<size_t>(d)); }
size_t scale_part(int64_t rows, int64_t d) { return align256(static_cast<size_t>(rows) * fp8_groups(d) * sizeof(float)); }

bool sizes_ok(int64_t T, int64_t N, int64_t K) {
    return T >= 0 && T <= kMaxRows && N > 0 && N <= kMaxDim && K > 0 && K <= kMaxDim;
}

rtq_status plan_quantize(const void* x, rtq_dtype xt, int64_t rows, int32_t d, void* codes, rtq_dtype ct, void* scale,
                         rtq_dtype st, rtq::Fp8QuantArgs* q) {
    RTQ_TRY(check_rows(rows, "rows"));
    RTQ_TRY(check_len(d, "d"));
    RTQ_TRY(check_float(xt, "xt"));
    RTQ_TRY(check_code(ct, "ct"));
    RTQ_TRY(check_scale(st));
    RTQ_TRY(check_row_ptr(x, "x", rows));
    RTQ_TRY(check_row_ptr(codes, "codes", rows));
    RTQ_TRY(check_row_ptr(scale, "scale", rows));
    *q = rtq::Fp8QuantArgs{x, xt == RTQ_BF16, rows, d, ct == RTQ_E5M2, codes, scale, st == RTQ_E8M0};
    return RTQ_OK;
}

// The product's arguments, trans: dx = g W, else y = a W^T.  (M, out, R): rows and columns of the
// output and the reduction.
rtq_status plan_gemm(const void* a, rtq_dtype at, const void* a_scale, int64_t T, const void* w, const void* w_scale,
                     rtq_dtype st, int64_t N, int32_t K, bool trans, void* y, rtq_dtype yt, rtq::Fp8GemmArgs* g) {
    RTQ_TRY(check_rows(T, "T"));
    RTQ_TRY(check_len(K, "K"));
    RTQ_TRY(check_len(N, "N", trans ? 16 : 1));
    RTQ_TRY(check_code(at, trans ? "gt" : "at"));
    RTQ_TRY(check_scale(st));
    RTQ_TRY(check_float(yt, trans ? "dxt" : "yt"));
    RTQ_TRY(check_row_ptr(a, trans ? "g_codes" : "a_codes", T));
    RTQ_TRY(check_row_ptr(a_scale, trans ? "g_scale" : "a_scale", T));
    RTQ_TRY(check_ptr(w, "w_codes"));
    RTQ_TRY(check_ptr(w_scale, "w_scale"));
    RTQ_TRY(check_row_ptr(y, trans ? "dx" : "y", T));
    rtq::Fp8GemmArgs p{};
    p.a = a;
    p.a_e5m2 = at == RTQ_E5M2;
    p.a_scale = a_scale;
    p.w = w;
    p.w_scale = w_scale;
    p.e8m0 = st == RTQ_E8M0;
    p.M = T;
    p.N = trans ? K : N;
    p.R = static_cast<int>(trans ? N : K);
    p.trans = trans;
    p.y = y;
    p.y_bf16 = yt == RTQ_BF16;
    // one workgroup per 64 x 64 outputs at least, each split at most 16 ways
    if ((p.M + 63) / 64 * ((p.N + 63) / 64) > kMaxRows / 16)
        return fail(RTQ_ERR_UNSUPPORTED, "output too large (%lld x %lld)", static_cast<long long>(p.M),
                    static_cast<long long>(p.N));
    *g = p;
    return RTQ_OK;
}

// Quantise rows into (codes, scale), then the product on the same stream.
rtq_status quantize_then_gemm(const rtq::Fp8QuantArgs& q, const rtq::Fp8GemmArgs& g, hipStream_t s) {
    RTQ_TRY(hip_status(rtq::launch_fp8_quantize_rows(q, s), "fp8 quantise launch"));
    return hip_status(rtq::launch_fp8_gemm(g, s), "fp8 product launch");
}

}  // namespace

extern "C" {

rtq_status rtq_fp8_quantize(const void* x, rtq_dtype xt, int64_t rows, int32_t d, rtq_fp8_layout layout, void* codes,
                            rtq_dtype ct, void* scale, rtq_dtype st, void* stream) {
    return guarded([&]() -> rtq_status {
        rtq::Fp8QuantArgs q{};
        RTQ_TRY(check_layout(layout));
        RTQ_TRY(plan_quantize(x, xt, rows, d, codes, ct, scale, st, &q));
        if (rows == 0) return ok();
        hipStream_t s = static_cast<hipStream_t>(stream);
        return hip_status(layout == RTQ_FP8_ROWS ? rtq::launch_fp8_quantize_rows(q, s) : rtq::launch_fp8_quantize_blocks(q, s),
                          "fp8 quantise launch");
    });
}

rtq_status rtq_fp8_dequantize(const void* codes, rtq_dtype ct, const void* scale, rtq_dtype st, int64_t rows, int32_t d,
                              rtq_fp8_layout layout, void* y, rtq_dtype yt, void* stream) {
    return guarded([&]() -> rtq_status {
        RTQ_TRY(check_layout(layout));
        RTQ_TRY(check_rows(rows, "rows"));
        RTQ_TRY(check_len(d, "d"));
        RTQ_TRY(check_code(ct, "ct"));
        RTQ_TRY(check_scale(st));
        RTQ_TRY(check_float(yt, "yt"));
        RTQ_TRY(check_row_ptr(codes, "codes", rows));
        RTQ_TRY(check_row_ptr(scale, "scale", rows));
        RTQ_TRY(check_row_ptr(y, "y", rows));
        if (rows == 0) return ok();
        const rtq::Fp8DequantArgs a{codes, ct == RTQ_E5M2, scale, st == RTQ_E8M0, layout == RTQ_FP8_BLOCKS,
                                    rows, d, y, yt == RTQ_BF16};
        return hip_status(rtq::launch_fp8_dequantize(a, static_cast<hipStream_t>(stream)), "fp8 dequantise launch");
    });
}

size_t rtq_fp8_qgemm_workspace(int64_t T, int64_t N, int32_t K) {
    return sizes_ok(T, N, K) ? rtq::fp8_gemm_workspace_bytes(T, N, K, false) : 0;
}

rtq_status rtq_fp8_qgemm(const void* a_codes, rtq_dtype at, const void* a_scale, int64_t T, const void* w_codes,
                         const void* w_scale, rtq_dtype st, int64_t N, int32_t K, void* y, rtq_dtype yt, void* workspace,
                         size_t ws_bytes, void* stream) {
    return guarded([&]() -> rtq_status {
        rtq::Fp8GemmArgs g{};
        RTQ_TRY(plan_gemm(a_codes, at, a_scale, T, w_codes, w_scale, st, N, K, false, y, yt, &g));
        RTQ_TRY(check_workspace(workspace));
        if (T == 0) return ok();
        g.workspace = workspace;
        g.ws_bytes = workspace != nullptr ? ws_bytes : 0;
        return hip_status(rtq::launch_fp8_gemm(g, static_cast<hipStream_t>(stream)), "fp8 product launch");
    });
}

size_t rtq_fp8_dgrad_workspace(int64_t T, int32_t N, int32_t K) {
    return sizes_ok(T, N, K) ? rtq::fp8_gemm_workspace_bytes(T, K, N, true) : 0;
}

rtq_status rtq_fp8_dgrad(const void* g_codes, rtq_dtype gt, const void* g_scale, int64_t T, const void* w_codes,
                         const void* w_scale, rtq_dtype st, int32_t N, int32_t K, void* dx, rtq_dtype dxt, void* workspace,
                         size_t ws_bytes, void* stream) {
    return guarded([&]() -> rtq_status {
        rtq::Fp8GemmArgs g{};
        RTQ_TRY(plan_gemm(g_codes, gt, g_scale, T, w_codes, w_scale, st, N, K, true, dx, dxt, &g));
        RTQ_TRY(check_workspace(workspace));
        if (T == 0) return ok();
        g.workspace = workspace;
        g.ws_bytes = workspace != nullptr ? ws_bytes : 0;
        return hip_status(rtq::launch_fp8_gemm(g, static_cast<hipStream_t>(stream)), "fp8 dgrad launch");
    });
}

size_t rtq_fp8_linear_workspace(int64_t T, int64_t N, int32_t K) {
    return sizes_ok(T, N, K) ? code_part(T, K) + scale_part(T, K) + rtq::fp8_gemm_workspace_bytes(T, N, K, false) : 0;
}

rtq_status rtq_fp8_linear(const void* x, rtq_dtype xt, int64_t T, const void* w_codes, const void* w_scale, rtq_dtype st,
                          int64_t N, int32_t K, void* x_codes, void* x_scale, void* y, rtq_dtype yt, void* workspace,
                          size_t ws_bytes, void* stream) {
    return guarded([&]() -> rtq_status {
        RTQ_TRY(check_rows(T, "T"));
        RTQ_TRY(check_len(K, "K"));
        if (T > 0 && (x_codes == nullptr) != (x_scale == nullptr))
            return fail(RTQ_ERR_INVALID_ARG, "x_codes and x_scale are given together or not at all");
        RTQ_TRY(check_workspace(workspace));
        unsigned char* ws = static_cast<unsigned char*>(workspace);
        size_t left = workspace != nullptr ? ws_bytes : 0;
        const bool keep = x_codes != nullptr;
        if (T > 0 && !keep) {
            const size_t need = code_part(T, K) + scale_part(T, K);
            if (workspace == nullptr) return fail(RTQ_ERR_INVALID_ARG, "workspace is NULL");
            if (left < need) return fail(RTQ_ERR_INVALID_ARG, "workspace too small: %zu < %zu bytes", left, need);
            x_codes = ws;
            x_scale = ws + code_part(T, K);
            ws += need;
            left -= need;
        }
        rtq::Fp8QuantArgs q{};
        rtq::Fp8GemmArgs g{};
        RTQ_TRY(plan_quantize(x, xt, T, K, x_codes, RTQ_E4M3, x_scale, st, &q));
        RTQ_TRY(plan_gemm(x_codes, RTQ_E4M3, x_scale, T, w_codes, w_scale, st, N, K, false, y, yt, &g));
        if (T == 0) return ok();
        g.workspace = left > 0 ? ws : nullptr;
        g.ws_bytes = left;
        hipStream_t s = static_cast<hipStream_t>(stream);
        if (rtq::fp8_small_linear_takes(T, N, K, false))
            return hip_status(rtq::launch_fp8_small_linear(g, x, xt == RTQ_BF16, keep ? x_codes : nullptr,
                                                           keep ? x_scale : nullptr, s), "fp8 product launch");
        return quantize_then_gemm(q, g, s);
    });
}

size_t rtq_fp8_linear_dgrad_workspace(int64_t T, int32_t N, int32_t K) {
    return sizes_ok(T, N, K) ? code_part(T, N) + scale_part(T, N) + rtq::fp8_gemm_workspace_bytes(T, K, N, true) : 0;
}

rtq_status rtq_fp8_linear_dgrad(const void* dy, rtq_dtype dyt, rtq_dtype gt, int64_t T, const void* w_codes,
                                const void* w_scale, rtq_dtype st, int32_t N, int32_t K, void* dx, rtq_dtype dxt,
                                void* workspace, size_t ws_bytes, void* stream) {
    return guarded([&]() -> rtq_status {
        RTQ_TRY(check_rows(T, "T"));
        RTQ_TRY(check_len(N, "N"));
        if (T > 0 && workspace == nullptr) return fail(RTQ_ERR_INVALID_ARG, "workspace is NULL");
        RTQ_TRY(check_workspace(workspace));
        const size_t need = code_part(T, N) + scale_part(T, N);
        if (T > 0 && ws_bytes < need) return fail(RTQ_ERR_INVALID_ARG, "workspace too small: %zu < %zu bytes", ws_bytes, need);
        unsigned char* ws = static_cast<unsigned char*>(workspace);
        void* codes = ws;
        void* scale = ws + code_part(T, N);
        rtq::Fp8QuantArgs q{};
        rtq::Fp8GemmArgs g{};
        RTQ_TRY(check_row_ptr(dy, "dy", T));
        RTQ_TRY(check_float(dyt, "dyt"));
        RTQ_TRY(check_code(gt, "gt"));
        RTQ_TRY(plan_quantize(dy, dyt, T, N, codes, gt, scale, st, &q));
        RTQ_TRY(plan_gemm(codes, gt, scale, T, w_codes, w_scale, st, N, K, true, dx, dxt, &g));
        if (T == 0) return ok();
        g.workspace = ws_bytes > need ? ws + need : nullptr;
        g.ws_bytes = ws_bytes - need;
        hipStream_t s = static_cast<hipStream_t>(stream);
        if (rtq::fp8_small_linear_takes(T, K, N, true))
            return hip_status(rtq::launch_fp8_small_linear(g, dy, dyt == RTQ_BF16, nullptr, nullptr, s), "fp8 dgrad launch");
        return quantize_then_gemm(q, g, s);
    });
}

size_t rtq_fp8_wgrad_workspace(int64_t T, int32_t N, int32_t K) {
    return sizes_ok(T, N, K) ? rtq::fp8_wgrad_workspace_bytes(T, N, K) : 0;
}

rtq_status rtq_fp8_wgrad(const void* dy, int64_t T, const void* x_codes, const void* x_scale, rtq_dtype st, int32_t N,
                         int32_t K, void* dw, rtq_dtype dwt, int32_t accumulate, void* workspace, size_t ws_bytes,
                         void* stream) {
    return guarded([&]() -> rtq_status {
        RTQ_TRY(check_rows(T, "T"));
        RTQ_TRY(check_len(N, "N", 8));
        RTQ_TRY(check_len(K, "K"));
        RTQ_TRY(check_scale(st));
        RTQ_TRY(check_float(dwt, "dwt"));
        if (accumulate != 0 && accumulate != 1) return fail(RTQ_ERR_INVALID_ARG, "accumulate must be 0 or 1");
        RTQ_TRY(check_row_ptr(dy, "dy", T));
        RTQ_TRY(check_row_ptr(x_codes, "x_codes", T));
        RTQ_TRY(check_row_ptr(x_scale, "x_scale", T));
        RTQ_TRY(check_ptr(dw, "dw"));
        RTQ_TRY(check_workspace(workspace));
        if (T == 0 && accumulate) return ok();
        const rtq::Fp8WgradArgs g{dy, x_codes, x_scale, st == RTQ_E8M0, T, N, K, dw, dwt == RTQ_BF16, accumulate != 0,
                                  workspace, workspace != nullptr ? ws_bytes : 0};
        return hip_status(rtq::launch_fp8_wgrad(g, static_cast<hipStream_t>(stream)), "fp8 wgrad launch");
    });
}

rtq_status rtq_act_fp8_forward(const void* h, rtq_dtype ht, int64_t rows, int32_t d, rtq_act act, void* h_codes,
                               void* h_scale, void* y, void* y_codes, void* y_scale, rtq_dtype st, void* stream) {
    return guarded([&]() -> rtq_status {
        RTQ_TRY(check_rows(rows, "rows"));
        RTQ_TRY(check_len(d, "d"));
        RTQ_TRY(check_act(act));
        RTQ_TRY(check_float(ht, "ht"));
        RTQ_TRY(check_scale(st));
        RTQ_TRY(check_row_ptr(h, "h", rows));
        RTQ_TRY(check_row_ptr(h_codes, "h_codes", rows));
        RTQ_TRY(check_row_ptr(h_scale, "h_scale", rows));
        if (rows == 0) return ok();
        if ((y_codes == nullptr) != (y_scale == nullptr))
            return fail(RTQ_ERR_INVALID_ARG, "y_codes and y_scale are given together or not at all");
        if ((y == nullptr) == (y_codes == nullptr))
            return fail(RTQ_ERR_INVALID_ARG, "give either y, or y_codes and y_scale");
        if (y != nullptr) {
            RTQ_TRY(check_row_ptr(y, "y", rows));
        } else {
            RTQ_TRY(check_row_ptr(y_codes, "y_codes", rows));
            RTQ_TRY(check_row_ptr(y_scale, "y_scale", rows));
        }
        const rtq::ActForwardArgs a{h, ht == RTQ_BF16, rows, d, act, h_codes, h_scale, y, y_codes, y_scale, st == RTQ_E8M0};
        return hip_status(rtq::launch_act_fp8_forward(a, static_cast<hipStream_t>(stream)), "act forward launch");
    });
}

rtq_status rtq_act_fp8_backward(const void* dy, rtq_dtype dyt, const void* h_codes, const void* h_scale, rtq_dtype st,
                                int64_t rows, int32_t d, rtq_act act, void* dh, void* stream) {
    return guarded([&]() -> rtq_status {
        RTQ_TRY(check_rows(rows, "rows"));
        RTQ_TRY(check_len(d, "d"));
        RTQ_TRY(check_act(act));
        RTQ_TRY(check_float(dyt, "dyt"));
        RTQ_TRY(check_scale(st));
        RTQ_TRY(check_row_ptr(dy, "dy", rows));
        RTQ_TRY(check_row_ptr(h_codes, "h_codes", rows));
        RTQ_TRY(check_row_ptr(h_scale, "h_scale", rows));
        RTQ_TRY(check_row_ptr(dh, "dh", rows));
        if (rows == 0) return ok();
        const rtq::ActBackwardArgs a{dy, dyt == RTQ_BF16, h_codes, h_scale, st == RTQ_E8M0, rows, d, act, dh};
        return hip_status(rtq::launch_act_fp8_backward(a, static_cast<hipStream_t>(stream)), "act backward launch");
    });
}

}  // extern "C"
