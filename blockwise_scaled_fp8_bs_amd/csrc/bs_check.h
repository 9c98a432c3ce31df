// Host-side argument checks shared by the C entry points (bs_api.hip,
// bs_block_api.hip): the status and message of a failed check.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/bs.h"

namespace bs {

// Leading dimensions (elements) stay below 2^22 so that the kernels' lane
// and in-tile offsets (up to 256 rows of a tile) fit in 32 bits.
constexpr int64_t kMaxLd = (int64_t)1 << 22;

// Sets the calling thread's message and returns st.
bs_status fail(bs_status st, const char* fn, const char* fmt, ...) __attribute__((format(printf, 3, 4)));

// Clears the calling thread's message and returns BS_OK.
bs_status ok();

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline bs_status hip_status(hipError_t e, const char* fn) {
    if (e == hipSuccess) return ok();
    return fail(BS_ERR_HIP, fn, "kernel launch failed: %s", hipGetErrorString(e));
}

}  // namespace bs

// Returns from the calling entry point (which names itself in `fn`) unless cond holds.
#define REQUIRE(cond, code, ...)                               \
    do {                                                       \
        if (!(cond)) return ::bs::fail(code, fn, __VA_ARGS__); \
    } while (0)
