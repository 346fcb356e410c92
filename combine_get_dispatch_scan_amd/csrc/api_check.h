// Error reporting and argument checks shared by the C entry points (host only).
#pragma once

#include <stdarg.h>
#include <stddef.h>
#include <stdint.h>
#include <stdio.h>

#include <string>

#include "moe_ep.h"

namespace moe_ep {

// Message of the last error on this thread (ep_last_error).
inline thread_local std::string g_err;

inline int fail(int code, const char* fmt, ...)
{
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    g_err = buf;
    return code;
}

inline int hip_fail(hipError_t e, const char* what)
{
    return fail(EP_EHIP, "%s: %s", what, hipGetErrorString(e));
}

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

}  // namespace moe_ep
