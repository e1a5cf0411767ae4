// What the C-ABI entry points share: the thread's error text (kept in
// api.hip) and the checks of alignment and overlap.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gdn.h"

#define GDN_EXPORT extern "C" __attribute__((visibility("default")))

namespace gdn {

// records the message of the calling thread's failed call; returns `code`
int fail(int code, const char *fmt, ...);
// records success; returns GDN_OK
int ok();

inline bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

// byte range of a strided row buffer [rows][stride] whose rows use `cols`
// elements of `elem` bytes
struct Span {
    uintptr_t lo, hi;
};
inline Span row_span(const void *p, int64_t rows, int64_t stride, int64_t cols, int64_t elem) {
    const uintptr_t lo = (uintptr_t)p;
    if (rows <= 0 || cols <= 0) return {lo, lo};
    return {lo, lo + (uintptr_t)(((rows - 1) * stride + cols) * elem)};
}
// empty ranges overlap nothing
inline bool overlap(Span a, Span b) { return a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi; }

inline int hip_status(hipError_t e, const char *what) {
    if (e != hipSuccess) return fail(GDN_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
    return ok();
}

}  // namespace gdn
