// Which buffers of a call share memory (host; api_tokens.cpp, api_policy.cpp).
#pragma once

#include <stdint.h>

#include <initializer_list>

namespace mx {

// A buffer: `rows` rows of `bytes` bytes, `step` bytes apart.
struct Span {
    uintptr_t at;
    int64_t rows, bytes, step;
    Span(const void *p, int64_t n) : at((uintptr_t)p), rows(1), bytes(n), step(n) {}
    Span(const void *p, int64_t rows_, int64_t n, int64_t step_) : at((uintptr_t)p), rows(rows_), bytes(n), step(step_) {}
    bool empty() const { return !at || rows <= 0 || bytes <= 0; }
    uintptr_t end() const { return at + (rows - 1) * step + bytes; }
};

// Whether rows of a and b, both step bytes apart, share a byte: b's row j meets
// a's row i if j - i lies between two bounds that follow from the distance.
inline bool rows_meet(const Span &a, const Span &b, int64_t step) {
    const int64_t d = (int64_t)(a.at - b.at);
    const int64_t above = d - b.bytes, below = d + a.bytes;          // above < (j - i) * step < below
    const int64_t lo = above >= 0 ? above / step + 1 : -((-above - 1) / step);
    const int64_t hi = below > 0 ? (below - 1) / step : -(-below / step) - 1;
    return (lo > 1 - a.rows ? lo : 1 - a.rows) <= (hi < b.rows - 1 ? hi : b.rows - 1);
}
inline bool meet(const Span &a, const Span &b) {
    if (a.empty() || b.empty() || a.end() <= b.at || b.end() <= a.at) return false;
    if (a.rows == 1 || a.step == b.step) return rows_meet(a, b, b.step);
    if (b.rows == 1) return rows_meet(b, a, a.step);
    if (a.rows > b.rows) return meet(b, a);
    for (int64_t i = 0; i < a.rows; ++i)
        if (rows_meet(Span(reinterpret_cast<const void *>(a.at + i * a.step), a.bytes), b, b.step)) return true;
    return false;
}

// Whether an output shares a byte with an input or with another output.
inline bool overlap(std::initializer_list<Span> outputs, std::initializer_list<Span> inputs) {
    for (const Span *o = outputs.begin(); o != outputs.end(); ++o) {
        for (const Span &i : inputs)
            if (meet(*o, i)) return true;
        for (const Span *q = o + 1; q != outputs.end(); ++q)
            if (meet(*o, *q)) return true;
    }
    return false;
}

}  // namespace mx
