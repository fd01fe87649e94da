// kda_check.h -- argument checks shared by the entry points of the C ABI
// (kda_api.cpp, kda_tree_api.cpp).  Host only, no HIP call.
#pragma once

#include <stdint.h>

#include <initializer_list>

#include "kda.h"

namespace kda {
namespace check {

struct Span {
    uintptr_t lo = 0, hi = 0;  // [lo, hi); empty spans overlap nothing
};

inline Span span(const void* p, uint64_t bytes) {
    Span s;
    if (p && bytes) {
        s.lo = reinterpret_cast<uintptr_t>(p);
        s.hi = s.lo + bytes;
    }
    return s;
}

inline bool overlaps(const Span& a, const Span& b) {
    return a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi;
}

inline bool overlaps_any(const Span& a, std::initializer_list<Span> others) {
    for (const Span& b : others)
        if (overlaps(a, b)) return true;
    return false;
}

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline bool valid_dtype(kda_dtype dt) { return dt == KDA_F32 || dt == KDA_BF16; }

inline uint64_t esize(kda_dtype dt) { return dt == KDA_F32 ? 4u : 2u; }

// Largest element count a single tensor may have (keeps byte sizes in range).
constexpr uint64_t kMaxElems = (uint64_t)1 << 56;

}  // namespace check
}  // namespace kda
