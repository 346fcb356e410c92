// Argument checks shared by the C entry points on rows, groups and weights (host only).
#pragma once

#include "api_check.h"

#define EP_TRY(call)          \
    do {                      \
        const int rc_ = call; \
        if (rc_)              \
            return rc_;       \
    } while (0)

namespace moe_ep {

inline bool width_ok(int w) { return w >= 128 && w <= EP_MAX_HIDDEN && w % 128 == 0; }

inline int check_width(const char* name, int w)
{
    if (width_ok(w))
        return EP_OK;
    return fail(EP_EINVAL, "%s=%d must be a multiple of 128 in [128, %d]", name, w, EP_MAX_HIDDEN);
}

inline int check_groups(const int32_t* off, int G, int stride, int rows, bool optional = false)
{
    if (rows < 0 || rows > 0x7FFFFF00)
        return fail(EP_EINVAL, "num_rows=%d must be in [0, 2^31 - 256]", rows);
    if (optional && !off) {
        if (G != 0 || stride != 0)
            return fail(EP_EINVAL, "num_groups and group_stride must be 0 without group_offsets");
        return EP_OK;
    }
    if (G < 1 || G > EP_MAX_EXPERTS)
        return fail(EP_EINVAL, "num_groups=%d must be in [1, %d]", G, EP_MAX_EXPERTS);
    if (stride < 0)
        return fail(EP_EINVAL, "group_stride=%d must be >= 0", stride);
    if (!off || !aligned(off, 4))
        return fail(EP_EINVAL, "group_offsets must be a non-NULL 4-byte aligned device pointer");
    return EP_OK;
}

inline int check_ptr(const char* name, const void* p, size_t a)
{
    if (p && aligned(p, a))
        return EP_OK;
    return fail(EP_EINVAL, "%s must be a non-NULL %zu-byte aligned device pointer", name, a);
}

inline int check_scale_ld(int ld, int rows)
{
    if (ld == 0 || (ld >= rows && ld % 4 == 0))
        return EP_OK;
    return fail(EP_EINVAL, "scale_ld=%d must be 0, or >= num_rows=%d and a multiple of 4", ld, rows);
}

}  // namespace moe_ep
