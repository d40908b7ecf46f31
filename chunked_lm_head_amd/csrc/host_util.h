// host_util.h — small host helpers shared by the C ABI's translation units.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace lmhead {

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t round_up(int64_t a, int64_t b) { return cdiv(a, b) * b; }
inline bool aligned(const void* ptr, uintptr_t a) { return ((uintptr_t)ptr % a) == 0; }

inline int grid_1d(int64_t items, int per_block, int cap) {
    int64_t g = cdiv(items, per_block);
    if (g < 1) g = 1;
    return (int)(g < cap ? g : cap);
}

// LMHEAD_OK when the current device is a gfx950 (lmhead_api.hip)
int check_device();
// LMHEAD_OK, or LMHEAD_ERR_HIP when a launch since the last call failed
int launched();

}  // namespace lmhead
