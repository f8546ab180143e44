// Host helpers shared by the C-ABI files: alignment, argument checks, workspace addressing.
#pragma once

#include "../../include/ssm_scan.h"

#include <stddef.h>
#include <stdint.h>

namespace ssm_api {

constexpr size_t kStatusBytes = 256;

inline size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

// A pointer may be null only when the array it describes is empty.
inline bool ptr_ok(const void* ptr, size_t count) { return count == 0 || ptr != nullptr; }

inline int check_arrays(const void* const* ptrs, const size_t* counts, int n) {
    for (int i = 0; i < n; ++i) {
        if (!ptr_ok(ptrs[i], counts[i])) return SSM_ERR_INVALID_ARG;
        if (counts[i] && !aligned16(ptrs[i])) return SSM_ERR_MISALIGNED;
    }
    return SSM_OK;
}

template <typename T>
T* at(void* ws, size_t off) {
    return reinterpret_cast<T*>(static_cast<char*>(ws) + off);
}

}  // namespace ssm_api
