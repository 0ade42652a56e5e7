// Host-side argument checks shared by the C ABI's entry points.
#pragma once

#include <initializer_list>

#include "gdr_device.h"

namespace gdr {

inline bool aligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline bool dtype_ok(gdr_dtype_t d) { return d == GDR_F32 || d == GDR_BF16; }

inline gdr_status_t from_hip(hipError_t e) { return e == hipSuccess ? GDR_OK : GDR_ERR_DEVICE; }

// Every listed pointer must be non-NULL and 16-byte aligned.
inline bool ptrs_ok(std::initializer_list<const void*> ps) {
    for (const void* p : ps)
        if (!p || !aligned(p)) return false;
    return true;
}

inline bool opt_ok(const void* p) { return !p || aligned(p); }

// Element-aligned pointer (scalar gates and outputs are accessed per element).
inline bool elem_ok(const void* p, size_t bytes) {
    return p && (reinterpret_cast<uintptr_t>(p) % bytes) == 0;
}

// Largest element count of any tensor must fit the kernels' 64-bit offsets.
inline bool sizes_ok(int64_t a, int64_t b, int64_t c) {
    if (a < 0 || b < 0 || c < 0) return false;
    const double n = (double)a * (double)b * (double)c;
    return n < 4.0e18;
}

}  // namespace gdr
