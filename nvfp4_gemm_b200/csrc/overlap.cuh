// overlap.cuh -- host checks that the outputs of a call share no memory with what else it
// reads or writes.
#pragma once
#include <algorithm>
#include <cstdint>
#include <memory>
#include <new>
#include <numeric>

#include "common.cuh"

namespace pact {

struct Rows {   // `rows` rows of `width` bytes, `ld` bytes from one to the next
    uintptr_t p;
    int64_t ld, width, rows;
};
inline Rows matrix(const pact_bf16 *p, int64_t ld, int64_t cols, int64_t rows) {
    return {(uintptr_t)p, 2 * ld, 2 * cols, rows};
}
inline Rows memory(const void *p, int64_t bytes) { return {(uintptr_t)p, bytes, bytes, 1}; }

// Whether two sets of rows share a byte (columns of one buffer may lie side by side).  Each row of the later
// one that starts between the ends of the earlier one is looked up there; they come to lie at
// columns that repeat, from earlier rows on, after ld / gcd of the two strides.
inline bool overlap(Rows a, Rows b) {
    if (a.p > b.p) std::swap(a, b);
    const int64_t extent = (a.rows - 1) * a.ld + a.width, d = (int64_t)(b.p - a.p);
    if (d >= extent) return false;
    const int64_t rows = std::min(b.rows, a.ld / std::gcd(a.ld, b.ld));
    for (int64_t j = 0, at = d; j < rows && at < extent; ++j, at += b.ld) {
        const int64_t row = at / a.ld, col = at % a.ld;
        if (col < a.width || (col + b.width > a.ld && row + 1 < a.rows)) return true;
    }
    return false;
}

// Whether any of the first `outs` of `n` overlaps another one of the n.
inline bool overlap_any(const Rows *m, int outs, int n) {
    for (int i = 0; i < outs; ++i)
        for (int j = i + 1; j < n; ++j)
            if (overlap(m[i], m[j])) return true;
    return false;
}

// Byte ranges that a call writes or only reads, collected one by one, then compared all at once.
struct Ranges {
    struct Range {
        uintptr_t begin, end;
        bool written;
    };
    std::unique_ptr<Range[]> r;   // not a vector: nothing may be thrown through a C entry
    int64_t n = 0;
    explicit Ranges(int64_t most) : r(new (std::nothrow) Range[most]) {}
    void add(const void *p, int64_t bytes, bool written) {
        if (r && p) r[n++] = {(uintptr_t)p, (uintptr_t)p + bytes, written};
    }
    // Whether no written range overlaps another one (ranges that are only read may).  Sorts them; false
    // without host memory for the list, too.
    bool disjoint() {
        if (!r) return false;
        std::sort(&r[0], &r[0] + n, [](const Range &a, const Range &b) { return a.begin < b.begin; });
        uintptr_t written = 0, any = 0;   // ends of the ranges before
        for (int64_t i = 0; i < n; ++i) {
            if (r[i].begin < (r[i].written ? any : written)) return false;
            any = std::max(any, r[i].end);
            if (r[i].written) written = std::max(written, r[i].end);
        }
        return true;
    }
};

}  // namespace pact
