// Whether two arrays of rows share a byte.
#pragma once

#include <algorithm>
#include <cstdint>
#include <utility>

namespace moe {

struct Span {
    const void* at;                // nullptr: not there
    int64_t rows, width, pitch;    // bytes of a row, and from row to row (at least the width)
};

// Exact, so that rows side by side in one buffer (columns of it) are told from rows on one another.
inline bool overlap(Span a, Span b) {
    if (!a.at || !b.at || a.rows < 1 || b.rows < 1 || a.width < 1 || b.width < 1) return false;
    if (reinterpret_cast<uintptr_t>(b.at) < reinterpret_cast<uintptr_t>(a.at)) std::swap(a, b);
    const int64_t by = (int64_t)(reinterpret_cast<uintptr_t>(b.at) - reinterpret_cast<uintptr_t>(a.at));   // b begins here in a
    for (Span* s : {&a, &b})
        if (s->rows == 1 || s->pitch == s->width) {   // one run
            s->width += (s->rows - 1) * s->pitch;
            s->pitch = s->width;
            s->rows = 1;
        }
    if (by >= (a.rows - 1) * a.pitch + a.width) return false;
    auto meets = [&](int64_t from) {   // a row of b, and the last of a's that begins before its end
        const int64_t i = std::min((from + b.width - 1) / a.pitch, a.rows - 1);
        return i * a.pitch + a.width > from;
    };
    // rows of one pitch lie alike, the first tells; otherwise one by one while they are within a
    const int64_t rows = a.pitch == b.pitch ? 1 : b.rows, end = (a.rows - 1) * a.pitch + a.width;
    for (int64_t j = 0; j < rows && by + j * b.pitch < end; ++j)
        if (meets(by + j * b.pitch)) return true;
    return false;
}

}  // namespace moe
