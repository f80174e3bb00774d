// Argument checks and error text shared by the files that implement the C ABI.
#pragma once

#include "../../include/sam.h"

namespace sam {

inline bool ranges_overlap(const void* a, unsigned long long abytes, const void* b, unsigned long long bbytes)
{
    if (!a || !b || abytes == 0 || bbytes == 0) return false;
    const unsigned long long x = (unsigned long long)a, y = (unsigned long long)b;
    return x < y + bbytes && y < x + abytes;
}

inline bool aligned16(const void* p) { return ((unsigned long long)p & 15ull) == 0; }
inline bool aligned4(const void* p) { return ((unsigned long long)p & 3ull) == 0; }

inline unsigned long long align256(unsigned long long x) { return (x + 255ull) & ~255ull; }

// Sets this thread's error text and returns `s`.
sam_status api_fail(sam_status s, const char* fmt, ...);
// Clears it and returns SAM_OK.
sam_status api_ok();
// The current device is a gfx950 GPU on which the kernels load.
sam_status api_device_check();

}  // namespace sam
