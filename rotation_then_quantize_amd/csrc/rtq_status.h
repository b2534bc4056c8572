// rtq_status.h -- error reporting and argument checks shared by the C-ABI translation units.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/rtq.h"

namespace rtq {

// Record the message rtq_last_error() returns on this thread and give the status back.
rtq_status fail(rtq_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
rtq_status ok();
rtq_status hip_status(hipError_t e, const char* what);
// Device pointers: not NULL, 16-byte aligned.
rtq_status check_ptr(const void* p, const char* name);

}  // namespace rtq

#define RTQ_TRY(expr)                     \
    do {                                  \
        rtq_status _s = (expr);           \
        if (_s != RTQ_OK) return _s;      \
    } while (0)
