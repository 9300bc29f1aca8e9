// Argument checks that the C ABI's files share.
#pragma once
#include <hip/hip_runtime.h>

#include "host.h"

namespace sq {

inline sq_status fail_hip(hipError_t e, const char* what) {
    set_error("%s: %s", what, hipGetErrorString(e));
    return SQ_ERR_HIP;
}

inline bool dtype_ok(int32_t dt) { return dt == SQ_DTYPE_F32 || dt == SQ_DTYPE_BF16 || dt == SQ_DTYPE_F16; }
inline int64_t esize(int32_t dt) { return dt == SQ_DTYPE_F32 ? 4 : 2; }
inline bool aligned(const void* p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }

inline sq_status check_f32(const float* a, const char* name, uintptr_t to) {
    if (!a) { set_error("%s is NULL", name); return SQ_ERR_ARG; }
    if (!aligned(a, to)) { set_error("%s must be aligned to %u bytes", name, unsigned(to)); return SQ_ERR_ARG; }
    return SQ_OK;
}

inline sq_status check_work(const void* work, size_t bytes, size_t need) {
    if (bytes < need) { set_error("workspace of %zu bytes, the call needs %zu", bytes, need); return SQ_ERR_SHAPE; }
    if (need && (!work || !aligned(work, 256))) { set_error("workspace NULL or not 256-byte aligned"); return SQ_ERR_ARG; }
    return SQ_OK;
}

}  // namespace sq

#define SQ_TRY(x) do { const sq_status st_ = (x); if (st_ != SQ_OK) return st_; } while (0)
