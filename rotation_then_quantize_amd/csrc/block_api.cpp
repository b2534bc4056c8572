// block_api.cpp -- the C ABI of what stands around the 8-bit linear layers of an MLP block: norm, gated feed-forward,
// gradient norm and clipping.  Argument checks and dispatch, with the conventions of fp8_api.cpp.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <initializer_list>
#include <vector>

#include "../../include/rtq.h"
#include "block_internal.h"
#include "fp8_checks.h"
#include "rtq_status.h"

namespace {

using namespace rtq;

constexpr int64_t kMostElements = int64_t{1} << 37;   // of a tensor
constexpr int32_t kMostTensors = 1 << 20;

rtq_status check_eps(float eps) {
    if (!(eps > 0.f) || !std::isfinite(eps)) return fail(RTQ_ERR_INVALID_ARG, "eps must be positive and finite");
    return RTQ_OK;
}

// codes and scale: both or none.
rtq_status check_pair(const void* codes, const void* scale, const char* what) {
    if ((codes == nullptr) != (scale == nullptr))
        return fail(RTQ_ERR_INVALID_ARG, "%s_codes and %s_scale are given together or not at all", what, what);
    return RTQ_OK;
}
rtq_status check_optional(const void* p, const char* name) { return p == nullptr ? RTQ_OK : check_ptr(p, name); }

rtq_status check_channels(int64_t N) {
    RTQ_TRY(check_len(N, "N", 128));
    if (2 * N > kMaxDim) return fail(RTQ_ERR_UNSUPPORTED, "N too large (max %lld)", static_cast<long long>(kMaxDim / 2));
    return RTQ_OK;
}

bool glu_sizes_ok(int64_t T, int64_t N, int64_t K) { return sizes_ok(T, 2 * N, K) && N % 128 == 0 && K % 16 == 0; }

// An array of a call: what it reads, or writes.  `place`: it goes element by element, each read by the thread that then writes
// there, so that an output may lie exactly on an input of the same size.
struct Array {
    const char* name;
    const void* data;
    size_t bytes;
    bool out;
    bool place;
};
Array input(const char* name, const void* p, size_t bytes, bool place = false) { return {name, p, bytes, false, place}; }
Array output(const char* name, const void* p, size_t bytes, bool place = false) { return {name, p, bytes, true, place}; }

// No output overlaps another array (a workgroup would write over what another has yet to read), but for those `place`s.
rtq_status check_apart(std::initializer_list<Array> arrays) {
    for (const Array* o = arrays.begin(); o != arrays.end(); ++o) {
        if (!o->out || o->data == nullptr || o->bytes == 0) continue;
        const uintptr_t begin = reinterpret_cast<uintptr_t>(o->data);
        for (const Array* a = arrays.begin(); a != arrays.end(); ++a) {
            if (a == o || a->data == nullptr || a->bytes == 0) continue;
            const uintptr_t other = reinterpret_cast<uintptr_t>(a->data);
            if (begin + o->bytes <= other || other + a->bytes <= begin) continue;
            if (!a->out && o->place && a->place && begin == other && o->bytes == a->bytes) continue;
            return fail(RTQ_ERR_INVALID_ARG, "%s overlaps %s", o->name, a->name);
        }
    }
    return RTQ_OK;
}

size_t elements(int64_t rows, int64_t d, size_t size) { return static_cast<size_t>(rows) * static_cast<size_t>(d) * size; }
size_t float_size(rtq_dtype t) { return t == RTQ_BF16 ? 2 : 4; }
size_t scale_size(rtq_dtype t) { return t == RTQ_E8M0 ? 1 : 4; }
// Scales of row groups.
size_t row_scales(int64_t rows, int64_t d, rtq_dtype st) { return elements(rows, fp8_groups(d), scale_size(st)); }

rtq_status spans_of(const rtq_tensor* tensors, void* const* outs, int32_t count, std::vector<TensorSpan>* spans) {
    if (count < 0 || count > kMostTensors) return fail(RTQ_ERR_INVALID_ARG, "count must be 0..%d (got %d)", kMostTensors, count);
    if (count > 0 && tensors == nullptr) return fail(RTQ_ERR_INVALID_ARG, "tensors is NULL");
    spans->reserve(static_cast<size_t>(count));
    for (int32_t i = 0; i < count; ++i) {
        const rtq_tensor& t = tensors[i];
        if (t.n < 0) return fail(RTQ_ERR_INVALID_ARG, "tensor %d: n must be >= 0", i);
        if (t.n > kMostElements) return fail(RTQ_ERR_UNSUPPORTED, "tensor %d too large (max %lld elements)", i, static_cast<long long>(kMostElements));
        RTQ_TRY(check_float(t.type, "tensor type"));
        void* out = outs != nullptr ? outs[i] : t.data;
        if (t.n > 0) {
            RTQ_TRY(check_ptr(t.data, "tensor"));
            RTQ_TRY(check_ptr(out, "out"));
        }
        spans->push_back(TensorSpan{t.data, out, t.n, t.type == RTQ_BF16});
    }
    return RTQ_OK;
}

}  // namespace

extern "C" {

rtq_status rtq_rmsnorm_forward(const void* x, rtq_dtype xt, const void* residual, rtq_dtype rt, int64_t rows, int32_t d,
                               const void* gamma, rtq_dtype gt, float eps, void* h, void* y, void* codes, void* scale,
                               rtq_dtype st, void* stream) {
    return guarded([&]() -> rtq_status {
        RTQ_TRY(check_rows(rows, "rows"));
        RTQ_TRY(check_len(d, "d"));
        RTQ_TRY(check_float(xt, "xt"));
        RTQ_TRY(check_float(rt, "rt"));
        RTQ_TRY(check_float(gt, "gt"));
        RTQ_TRY(check_scale(st));
        RTQ_TRY(check_eps(eps));
        RTQ_TRY(check_ptr(gamma, "gamma"));
        RTQ_TRY(check_row_ptr(x, "x", rows));
        if (rows == 0) return ok();
        if ((residual == nullptr) != (h == nullptr))
            return fail(RTQ_ERR_INVALID_ARG, "residual and h are given together or not at all");
        RTQ_TRY(check_optional(residual, "residual"));
        RTQ_TRY(check_optional(h, "h"));
        if ((codes == nullptr) != (scale == nullptr))
            return fail(RTQ_ERR_INVALID_ARG, "codes and scale are given together or not at all");
        if (y == nullptr && codes == nullptr) return fail(RTQ_ERR_INVALID_ARG, "give y, or codes and scale, or all of them");
        RTQ_TRY(check_optional(y, "y"));
        RTQ_TRY(check_optional(codes, "codes"));
        RTQ_TRY(check_optional(scale, "scale"));
        if (h != nullptr && (y == h || (h == x && rt != xt)))
            return fail(RTQ_ERR_INVALID_ARG, "h must not be y, nor x of another type");
        const size_t nx = elements(rows, d, float_size(xt)), nr = elements(rows, d, float_size(rt));
        RTQ_TRY(check_apart({input("x", x, nx, true), input("residual", residual, nr, true), input("gamma", gamma, elements(1, d, float_size(gt))),
                             output("h", h, nr, true), output("y", y, nx, true), output("codes", codes, elements(rows, d, 1)),
                             output("scale", scale, row_scales(rows, d, st))}));
        const RmsForwardArgs a{x, xt == RTQ_BF16, residual, rt == RTQ_BF16, rows, d, gamma, gt == RTQ_BF16, eps,
                               h, y, codes, scale, st == RTQ_E8M0};
        return hip_status(launch_rmsnorm_forward(a, static_cast<hipStream_t>(stream)), "rmsnorm forward launch");
    });
}

size_t rtq_rmsnorm_backward_workspace(int64_t rows, int32_t d) {
    return rows >= 0 && rows <= kMaxRows && d > 0 && d <= kMaxDim ? rmsnorm_backward_workspace_bytes(rows, d) : 0;
}

rtq_status rtq_rmsnorm_backward(const void* dn, rtq_dtype dnt, const void* h, rtq_dtype ht, const void* dresidual,
                                int64_t rows, int32_t d, const void* gamma, rtq_dtype gt, float eps, void* dh,
                                void* dgamma, rtq_dtype dgt, int32_t accumulate, void* workspace, size_t ws_bytes,
                                void* stream) {
    return guarded([&]() -> rtq_status {
        RTQ_TRY(check_rows(rows, "rows"));
        RTQ_TRY(check_len(d, "d"));
        RTQ_TRY(check_float(dnt, "dnt"));
        RTQ_TRY(check_float(ht, "ht"));
        RTQ_TRY(check_float(gt, "gt"));
        RTQ_TRY(check_float(dgt, "dgt"));
        RTQ_TRY(check_eps(eps));
        if (accumulate != 0 && accumulate != 1) return fail(RTQ_ERR_INVALID_ARG, "accumulate must be 0 or 1");
        RTQ_TRY(check_ptr(gamma, "gamma"));
        RTQ_TRY(check_row_ptr(dn, "dn", rows));
        RTQ_TRY(check_row_ptr(h, "h", rows));
        RTQ_TRY(check_row_ptr(dh, "dh", rows));
        RTQ_TRY(check_optional(dresidual, "dresidual"));
        RTQ_TRY(check_optional(dgamma, "dgamma"));
        RTQ_TRY(check_workspace(workspace));
        if (rows > 0 && (dh == h || (dh == dn && dnt != ht)))
            return fail(RTQ_ERR_INVALID_ARG, "dh must not be h, nor dn of another type");
        if (rows > 0 && dgamma != nullptr) {
            const size_t need = rmsnorm_backward_workspace_bytes(rows, d);
            if (workspace == nullptr) return fail(RTQ_ERR_INVALID_ARG, "workspace is NULL");
            if (ws_bytes < need) return fail(RTQ_ERR_INVALID_ARG, "workspace too small: %zu < %zu bytes", ws_bytes, need);
        }
        if (rows > 0) {
            const size_t nh = elements(rows, d, float_size(ht));
            RTQ_TRY(check_apart({input("dn", dn, elements(rows, d, float_size(dnt)), true), input("h", h, nh),
                                 input("dresidual", dresidual, nh, true), input("gamma", gamma, elements(1, d, float_size(gt))),
                                 output("dh", dh, nh, true), output("dgamma", dgamma, elements(1, d, float_size(dgt))),
                                 output("workspace", workspace, dgamma != nullptr ? rmsnorm_backward_workspace_bytes(rows, d) : 0)}));
        }
        const RmsBackwardArgs a{dn, dnt == RTQ_BF16, h, ht == RTQ_BF16, dresidual, rows, d, gamma, gt == RTQ_BF16, eps,
                                dh, dgamma, dgt == RTQ_BF16, accumulate != 0, workspace};
        return hip_status(launch_rmsnorm_backward(a, static_cast<hipStream_t>(stream)), "rmsnorm backward launch");
    });
}

size_t rtq_fp8_glu_workspace(int64_t T, int32_t N, int32_t K) {
    return glu_sizes_ok(T, N, K) ? fp8_glu_workspace_bytes(T, N, K) : 0;
}

rtq_status rtq_fp8_glu(const void* x_codes, const void* x_scale, int64_t T, const void* w_codes, const void* w_scale,
                       rtq_dtype st, int32_t N, int32_t K, rtq_act act, void* h_codes, void* h_scale, void* y, rtq_dtype yt,
                       void* y_codes, void* y_scale, void* workspace, size_t ws_bytes, void* stream) {
    return guarded([&]() -> rtq_status {
        RTQ_TRY(check_rows(T, "T"));
        RTQ_TRY(check_len(K, "K"));
        RTQ_TRY(check_channels(N));
        RTQ_TRY(check_act(act));
        RTQ_TRY(check_scale(st));
        RTQ_TRY(check_float(yt, "yt"));
        RTQ_TRY(check_row_ptr(x_codes, "x_codes", T));
        RTQ_TRY(check_row_ptr(x_scale, "x_scale", T));
        RTQ_TRY(check_ptr(w_codes, "w_codes"));
        RTQ_TRY(check_ptr(w_scale, "w_scale"));
        RTQ_TRY(check_workspace(workspace));
        if (T == 0) return ok();
        if ((T + 63) / 64 * (2 * static_cast<int64_t>(N) / 64) > kMaxRows / 16)
            return fail(RTQ_ERR_UNSUPPORTED, "output too large (%lld x %d)", static_cast<long long>(T), N);
        RTQ_TRY(check_pair(h_codes, h_scale, "h"));
        RTQ_TRY(check_pair(y_codes, y_scale, "y"));
        if ((y == nullptr) == (y_codes == nullptr)) return fail(RTQ_ERR_INVALID_ARG, "give either y, or y_codes and y_scale");
        RTQ_TRY(check_optional(h_codes, "h_codes"));
        RTQ_TRY(check_optional(h_scale, "h_scale"));
        RTQ_TRY(check_optional(y, "y"));
        RTQ_TRY(check_optional(y_codes, "y_codes"));
        RTQ_TRY(check_optional(y_scale, "y_scale"));
        const size_t need = fp8_glu_workspace_bytes(T, N, K);
        if (need > 0 && workspace == nullptr) return fail(RTQ_ERR_INVALID_ARG, "workspace is NULL");
        if (need > 0 && ws_bytes < need) return fail(RTQ_ERR_INVALID_ARG, "workspace too small: %zu < %zu bytes", ws_bytes, need);
        RTQ_TRY(check_apart({input("x_codes", x_codes, elements(T, K, 1)), input("x_scale", x_scale, row_scales(T, K, st)),
                             input("w_codes", w_codes, elements(2 * static_cast<int64_t>(N), K, 1)),
                             input("w_scale", w_scale, row_scales(fp8_groups(2 * static_cast<int64_t>(N)), K, st)),
                             output("h_codes", h_codes, elements(T, 2 * static_cast<int64_t>(N), 1)),
                             output("h_scale", h_scale, row_scales(T, 2 * static_cast<int64_t>(N), st)),
                             output("y", y, elements(T, N, float_size(yt))), output("y_codes", y_codes, elements(T, N, 1)),
                             output("y_scale", y_scale, row_scales(T, N, st)), output("workspace", workspace, need)}));
        const GluArgs a{x_codes, x_scale, w_codes, w_scale, st == RTQ_E8M0, T, N, K, act, h_codes, h_scale, y, yt == RTQ_BF16,
                        y_codes, y_scale, workspace, ws_bytes};
        return hip_status(launch_fp8_glu(a, static_cast<hipStream_t>(stream)), "fp8 glu launch");
    });
}

rtq_status rtq_glu_fp8_backward(const void* dy, rtq_dtype dyt, const void* h_codes, const void* h_scale, rtq_dtype st,
                                int64_t T, int32_t N, rtq_act act, void* dh, void* dh_codes, rtq_dtype gt, void* dh_scale,
                                void* stream) {
    return guarded([&]() -> rtq_status {
        RTQ_TRY(check_rows(T, "T"));
        RTQ_TRY(check_channels(N));
        RTQ_TRY(check_act(act));
        RTQ_TRY(check_float(dyt, "dyt"));
        RTQ_TRY(check_scale(st));
        RTQ_TRY(check_code(gt, "gt"));
        RTQ_TRY(check_row_ptr(dy, "dy", T));
        RTQ_TRY(check_row_ptr(h_codes, "h_codes", T));
        RTQ_TRY(check_row_ptr(h_scale, "h_scale", T));
        if (T == 0) return ok();
        RTQ_TRY(check_pair(dh_codes, dh_scale, "dh"));
        if (dh == nullptr && dh_codes == nullptr) return fail(RTQ_ERR_INVALID_ARG, "give dh, or dh_codes and dh_scale, or all of them");
        RTQ_TRY(check_optional(dh, "dh"));
        RTQ_TRY(check_optional(dh_codes, "dh_codes"));
        RTQ_TRY(check_optional(dh_scale, "dh_scale"));
        const int64_t both = 2 * static_cast<int64_t>(N);
        RTQ_TRY(check_apart({input("dy", dy, elements(T, N, float_size(dyt))), input("h_codes", h_codes, elements(T, both, 1)),
                             input("h_scale", h_scale, row_scales(T, both, st)), output("dh", dh, elements(T, both, float_size(dyt))),
                             output("dh_codes", dh_codes, elements(T, both, 1)), output("dh_scale", dh_scale, row_scales(T, both, st))}));
        const GluBackwardArgs a{dy, dyt == RTQ_BF16, h_codes, h_scale, st == RTQ_E8M0, T, N, act, dh, dh_codes, gt == RTQ_E5M2, dh_scale};
        return hip_status(launch_glu_backward(a, static_cast<hipStream_t>(stream)), "glu backward launch");
    });
}

size_t rtq_grad_norm_workspace(const rtq_tensor* tensors, int32_t count) {
    size_t need = 0;
    guarded([&]() -> rtq_status {
        std::vector<TensorSpan> spans;
        RTQ_TRY(spans_of(tensors, nullptr, count, &spans));
        need = grad_norm_workspace_bytes(spans.data(), count);
        return RTQ_OK;
    });
    return need;
}

rtq_status rtq_grad_norm(const rtq_tensor* tensors, int32_t count, float* norm, void* workspace, size_t ws_bytes, void* stream) {
    return guarded([&]() -> rtq_status {
        std::vector<TensorSpan> spans;
        RTQ_TRY(spans_of(tensors, nullptr, count, &spans));
        RTQ_TRY(check_ptr(norm, "norm"));
        RTQ_TRY(check_workspace(workspace));
        const size_t need = grad_norm_workspace_bytes(spans.data(), count);
        if (need > 0 && workspace == nullptr) return fail(RTQ_ERR_INVALID_ARG, "workspace is NULL");
        if (ws_bytes < need) return fail(RTQ_ERR_INVALID_ARG, "workspace too small: %zu < %zu bytes", ws_bytes, need);
        return hip_status(launch_grad_norm(spans.data(), count, norm, workspace, static_cast<hipStream_t>(stream)), "grad norm launch");
    });
}

rtq_status rtq_grad_clip(const rtq_tensor* tensors, void* const* outs, int32_t count, const float* norm, float most, void* stream) {
    return guarded([&]() -> rtq_status {
        std::vector<TensorSpan> spans;
        RTQ_TRY(spans_of(tensors, outs, count, &spans));
        RTQ_TRY(check_ptr(norm, "norm"));
        if (!(most >= 0.f) || !std::isfinite(most)) return fail(RTQ_ERR_INVALID_ARG, "most must be finite and not negative");
        return hip_status(launch_grad_clip(spans.data(), count, norm, most, static_cast<hipStream_t>(stream)), "grad clip launch");
    });
}

}  // extern "C"
