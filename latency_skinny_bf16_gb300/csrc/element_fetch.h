// element_fetch.h -- what a copy of one bf16 element to shared memory reads.
#pragma once

#include <cstdint>

namespace skinny {

// cp.async moves aligned four-byte words.  An element comes with the neighbour that its word holds, which lies between
// the tensor's first and last elements unless it is one of those two itself: that one is loaded by itself.  (A copy of
// two bytes and zeros for every element of an even place: 8192 tokens, 32 + 8 heads of 61 70 us, so 51.)
struct ElementFetch {
    uintptr_t from;
    int bytes;
};
constexpr ElementFetch element_fetch(uintptr_t at, uintptr_t first, uintptr_t last) {
    const uintptr_t word = at & ~(uintptr_t)3;
    if (word < first || word + 2 > last) return {at, 2};
    return {word, 4};
}

}  // namespace skinny
