// fp8_checks.h -- argument checks that the C-ABI calls of the 8-bit floating point layers share.
#pragma once

#include <cstdint>

#include "../../include/rtq.h"
#include "fp8_internal.h"
#include "rtq_status.h"

namespace rtq {

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

inline rtq_status check_rows(int64_t rows, const char* name) {
    if (rows < 0) return fail(RTQ_ERR_INVALID_ARG, "%s must be >= 0", name);
    if (rows > kMaxRows) return fail(RTQ_ERR_UNSUPPORTED, "%s too large (max %lld)", name, static_cast<long long>(kMaxRows));
    return RTQ_OK;
}

// A row length that codes are stored with.
inline rtq_status check_len(int64_t d, const char* name, int multiple = 16) {
    if (d <= 0) return fail(RTQ_ERR_INVALID_ARG, "%s must be positive (got %lld)", name, static_cast<long long>(d));
    if (d % multiple != 0)
        return fail(RTQ_ERR_UNSUPPORTED, "%s must be a multiple of %d (got %lld)", name, multiple, static_cast<long long>(d));
    if (d > kMaxDim)
        return fail(RTQ_ERR_UNSUPPORTED, "%s too large (max %lld)", name, static_cast<long long>(kMaxDim));
    return RTQ_OK;
}

inline rtq_status check_float(rtq_dtype t, const char* name) {
    if (t != RTQ_F32 && t != RTQ_BF16) return fail(RTQ_ERR_UNSUPPORTED, "%s must be RTQ_F32 or RTQ_BF16", name);
    return RTQ_OK;
}
inline rtq_status check_code(rtq_dtype t, const char* name) {
    if (t != RTQ_E4M3 && t != RTQ_E5M2) return fail(RTQ_ERR_UNSUPPORTED, "%s must be RTQ_E4M3 or RTQ_E5M2", name);
    return RTQ_OK;
}
inline rtq_status check_scale(rtq_dtype t) {
    if (t != RTQ_F32 && t != RTQ_E8M0) return fail(RTQ_ERR_UNSUPPORTED, "st must be RTQ_F32 or RTQ_E8M0");
    return RTQ_OK;
}
inline rtq_status check_layout(rtq_fp8_layout l) {
    if (l != RTQ_FP8_ROWS && l != RTQ_FP8_BLOCKS) return fail(RTQ_ERR_INVALID_ARG, "unknown layout %d", static_cast<int>(l));
    return RTQ_OK;
}
inline rtq_status check_act(rtq_act a) {
    if (a != RTQ_ACT_GELU_TANH && a != RTQ_ACT_GELU && a != RTQ_ACT_SILU)
        return fail(RTQ_ERR_INVALID_ARG, "unknown activation %d", static_cast<int>(a));
    return RTQ_OK;
}
inline rtq_status check_workspace(const void* ws) {
    if (reinterpret_cast<uintptr_t>(ws) % 16 != 0) return fail(RTQ_ERR_MISALIGNED, "workspace is not 16-byte aligned");
    return RTQ_OK;
}

// An array of `rows` rows: it may be NULL where it is empty.
inline rtq_status check_row_ptr(const void* p, const char* name, int64_t rows) {
    return rows == 0 && p == nullptr ? RTQ_OK : check_ptr(p, name);
}

inline size_t align256(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }
// Bytes of the codes and (fp32) scales of row groups in a workspace.
inline size_t code_part(int64_t rows, int64_t d) { return align256(static_cast<size_t>(rows) * static_cast<size_t>(d)); }
inline size_t scale_part(int64_t rows, int64_t d) { return align256(static_cast<size_t>(rows) * fp8_groups(d) * sizeof(float)); }

inline bool sizes_ok(int64_t T, int64_t N, int64_t K) {
    return T >= 0 && T <= kMaxRows && N > 0 && N <= kMaxDim && K > 0 && K <= kMaxDim;
}

}  // namespace rtq
