// lm_checks.h -- checks of arguments that the entry points of the language-model
// operators share (lm_api.cpp, attn_api.cpp).  Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <initializer_list>

#include "../../include/msscan.h"
#include "msscan_internal.h"

namespace msscan {
namespace {

inline ms_status fail(ms_status s, const char* fmt, ...) {
    char text[400];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(text, sizeof text, fmt, ap);
    va_end(ap);
    return report(s, text);
}

constexpr int64_t kMax31 = 0x7fffffffLL;

inline ms_status check_aligned(std::initializer_list<const void*> ptrs) {
    for (const void* p : ptrs)
        if (reinterpret_cast<uintptr_t>(p) & 15u)
            return fail(MS_ERR_ALIGN, "pointer %p is not 16-byte aligned", p);
    return MS_OK;
}

// What is read element by element, or in vectors that assume no more.
inline ms_status check_element_aligned(size_t size, std::initializer_list<const void*> ptrs) {
    for (const void* p : ptrs)
        if (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(size - 1))
            return fail(MS_ERR_ALIGN, "pointer %p is not aligned to its element", p);
    return MS_OK;
}

inline size_t io_size(int32_t io) { return io == MS_BF16 ? 2 : 4; }

inline ms_status check_io(int32_t io, const char* name = "io") {
    if (io != MS_F32 && io != MS_BF16)
        return fail(MS_ERR_DTYPE, "%s=%d is not MS_F32 (0) or MS_BF16 (1)", name, io);
    return MS_OK;
}

inline ms_status check_id_bits(int32_t bits) {
    if (bits != 32 && bits != 64) return fail(MS_ERR_DTYPE, "id_bits=%d is not 32 or 64", bits);
    return MS_OK;
}

inline ms_status check_workspace(size_t need, const void* workspace, size_t given) {
    if (need && (!workspace || given < need))
        return fail(MS_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need,
                    workspace ? given : (size_t)0);
    return MS_OK;
}

inline ms_status launched(hipError_t e) {
    return e == hipSuccess ? MS_OK : fail(MS_ERR_HIP, "launch failed: %s", hipGetErrorString(e));
}

inline ms_status check_scale(float scale, bool positive) {
    if (!std::isfinite(scale) || (positive && !(scale > 0.f)))
        return fail(MS_ERR_SHAPE, "scale=%g must be finite%s", (double)scale,
                    positive ? " and > 0" : "");
    return MS_OK;
}

}  // namespace
}  // namespace msscan
