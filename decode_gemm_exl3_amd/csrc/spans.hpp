// spans.hpp - whether the results of a call are apart from its arguments (host).
#pragma once
#include <stdint.h>

#include <initializer_list>

namespace exl3 {

// Memory that a call reads or writes: `rows` pieces of `bytes` bytes, `pitch` bytes
// from one to the next (at least `bytes`).  A null pointer or no bytes: none.
struct Span {
    const void* at;
    int64_t bytes;
    int64_t rows = 1, pitch = 0;
};

// Does any byte of the one piece `a` belong to `b`?  Bytes between b's rows do not.
inline bool overlap(const Span& a, const Span& b) {
    if (!a.at || !b.at || a.bytes <= 0 || b.bytes <= 0 || b.rows <= 0) return false;
    const __int128 from = (__int128)(uintptr_t)a.at - (uintptr_t)b.at, end = from + a.bytes;  // a, from b's first byte on
    if (end <= 0 || from >= (__int128)(b.rows - 1) * b.pitch + b.bytes) return false;
    if (b.rows == 1 || from < 0) return true;
    const __int128 in_row = from % b.pitch;
    return in_row < b.bytes || in_row + a.bytes > b.pitch;
}

// Are the results (one piece each) apart from the arguments and from each other?
inline bool apart(std::initializer_list<Span> results, std::initializer_list<Span> arguments) {
    for (const Span* r = results.begin(); r != results.end(); ++r) {
        for (const Span& a : arguments)
            if (overlap(*r, a)) return false;
        for (const Span* s = results.begin(); s != r; ++s)
            if (overlap(*r, *s)) return false;
    }
    return true;
}

}  // namespace exl3
