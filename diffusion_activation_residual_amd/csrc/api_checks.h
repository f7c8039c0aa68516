// api_checks.h -- what the argument checks of the newer ABI files share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>

#include "cfz.h"

namespace cfz {

// A status with its text for cfz_last_error (cfz_api.hip).
cfz_status report(cfz_status st, const char *text);

static cfz_status fail(cfz_status st, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
static cfz_status fail(cfz_status st, const char *fmt, ...)
{
    char text[256];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(text, sizeof text, fmt, ap);
    va_end(ap);
    return report(st, text);
}

static inline cfz_status hip_status(hipError_t e, const char *what)
{
    if (e == hipSuccess)
        return CFZ_OK;
    return fail(CFZ_ERR_HIP, "%s: %s (%d)", what, hipGetErrorString(e), (int)e);
}

static inline bool aligned(const void *p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

}  // namespace cfz

#define CFZ_TRY(x)                                                                                 \
    do {                                                                                           \
        const cfz_status cfz_st_ = (x);                                                            \
        if (cfz_st_ != CFZ_OK)                                                                     \
            return cfz_st_;                                                                        \
    } while (0)
