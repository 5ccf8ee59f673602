// overlap.cuh -- host checks that the outputs of a call share no memory with what else it
// reads or writes.
#pragma once
#include <algorithm>
#include <cstdint>
#include <memory>
#include <new>

#include "common.cuh"

namespace pact {

struct Rows {   // a matrix of `rows` rows of the call, in BF16
    const pact_bf16 *p;
    int64_t ld, cols;
};

// Whether the later matrix's first row lies in the earlier one's rows: the answer for matrices of one row
// stride (columns of one buffer may lie side by side), and a lower bound of it for others.
inline bool overlap(Rows a, Rows b, int64_t rows) {
    if ((uintptr_t)a.p > (uintptr_t)b.p) std::swap(a, b);
    const int64_t d = (int64_t)(((uintptr_t)b.p - (uintptr_t)a.p) / sizeof(pact_bf16));
    if (d >= (rows - 1) * a.ld + a.cols) return false;
    return d % a.ld < a.cols || (d % a.ld + b.cols > a.ld && d / a.ld + 1 < rows);
}

// Whether any of the first `outs` of `n` matrices overlaps another one of the n.
inline bool overlap_any(const Rows *m, int outs, int n, int64_t rows) {
    for (int i = 0; i < outs; ++i)
        for (int j = i + 1; j < n; ++j)
            if (overlap(m[i], m[j], rows)) return true;
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
