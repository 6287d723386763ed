// host.h -- error reporting and argument checks shared by the C entry points (api.cpp, train.cpp).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>

#include "moe_int4.h"

namespace moe {

// Records the calling thread's error text (moe_last_error) and returns `status`.
int fail(int status, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
int hip_fail(hipError_t e, const char* what);
void clear_error();

bool aligned(const void* p, size_t a);
int check_ptr(const void* p, const char* name, size_t align = 16);

// MOE_OK when the current device is a gfx950
int device_ok();

}  // namespace moe

#define CHECK(expr)                   \
    do {                              \
        int rc_ = (expr);             \
        if (rc_ != MOE_OK) return rc_; \
    } while (0)

#define HIP_CHECK(expr, what)                    \
    do {                                         \
        hipError_t e_ = (expr);                  \
        if (e_ != hipSuccess) return ::moe::hip_fail(e_, what); \
    } while (0)
