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

// A device buffer of a call. 0 bytes: may be null.
struct Buf {
    const void* p;
    unsigned long long bytes;
    const char* name;
    int align;
    bool written;
};

// Null, alignment and overlap: nothing that is written may overlap anything else.
inline sam_status check_buffers(const Buf* b, int n)
{
    for (int i = 0; i < n; ++i) {
        if (b[i].bytes && !b[i].p) return api_fail(SAM_ERR_INVALID_ARG, "%s is null", b[i].name);
        if (b[i].bytes && (unsigned long long)b[i].p % (unsigned)b[i].align)
            return api_fail(SAM_ERR_MISALIGNED, "%s must be %d-byte aligned", b[i].name, b[i].align);
    }
    for (int i = 0; i < n; ++i)
        for (int j = 0; j < n; ++j)
            if (i != j && b[i].written && ranges_overlap(b[i].p, b[i].bytes, b[j].p, b[j].bytes))
                return api_fail(SAM_ERR_INVALID_ARG, "%s overlaps %s", b[i].name, b[j].name);
    return SAM_OK;
}

// Bytes from the first value of `rows` rows of `cols` values to the last, row stride ld.
inline unsigned long long span(long long rows, long long ld, long long cols, int es)
{
    return rows > 0 ? ((unsigned long long)(rows - 1) * ld + cols) * es : 0;
}

}  // namespace sam
