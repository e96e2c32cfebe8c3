// ranges.h -- argument checks that the C ABI's entry points share.
#pragma once

#include <initializer_list>

#include "calls.h"
#include "skinny_experts.h"

namespace skinny {

inline int el_bytes(int dtype) { return dtype == SKINNY_BF16 ? 2 : 4; }
inline bool dtype_ok(int d) { return d == SKINNY_BF16 || d == SKINNY_F32; }
inline uintptr_t addr(const void *p) { return reinterpret_cast<uintptr_t>(p); }
inline bool aligned(const void *p, int bytes) { return addr(p) % (uintptr_t)bytes == 0; }

// The bytes [lo, hi) that a matrix of `rows` rows of `cols` elements occupies.
struct Range {
    uintptr_t lo, hi;
};
inline Range span(const void *p, int64_t rows, int64_t cols, int64_t ld, int el) {
    if (!p || rows <= 0 || cols <= 0) return {0, 0};
    return {addr(p), addr(p) + (uintptr_t)(((rows - 1) * ld + cols) * el)};
}
// Whether a range that is written meets one of the others.
inline bool meets(const Range &w, std::initializer_list<Range> others) {
    for (const Range &o : others)
        if (w.lo < w.hi && o.lo < o.hi && ranges_overlap(w.lo, w.hi, o.lo, o.hi)) return true;
    return false;
}
inline skinny_status_t launched(cudaError_t e) { return e == cudaSuccess ? SKINNY_OK : SKINNY_ERR_LAUNCH; }

}  // namespace skinny
