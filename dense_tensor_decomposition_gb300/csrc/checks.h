// Checks of arguments that the files of entry points share.
#pragma once

#include <cstddef>
#include <cstdint>

#include "api.h"
#include "mttkrp.h"

namespace mk {

inline size_t type_bytes(int type) { return type == MTTKRP_F32 ? 4 : 2; }
inline bool type_ok(int type) { return type == MTTKRP_F32 || type == MTTKRP_BF16 || type == MTTKRP_F16; }
// a: a power of two
inline bool aligned_to(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// bytes from the first to behind the last element of rows x width, rows `stride` apart
inline size_t span_bytes(int64_t rows, int64_t width, int64_t stride, size_t elem) {
    return rows == 0 ? 0 : ((size_t)(rows - 1) * stride + width) * elem;
}

inline bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return na != 0 && nb != 0 && x < y + nb && y < x + na;
}

inline int check_workspace(const void* ws, size_t bytes, size_t need) {
    if (need == 0) return MTTKRP_OK;
    if (ws == nullptr || bytes < need)
        return fail(MTTKRP_ERR_WORKSPACE, "workspace of %zu bytes, %zu are needed", ws ? bytes : (size_t)0, need);
    if (!aligned_to(ws, 256)) return fail(MTTKRP_ERR_WORKSPACE, "workspace must be 256-byte aligned");
    return MTTKRP_OK;
}

}  // namespace mk
