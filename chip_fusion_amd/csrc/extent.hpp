// Which elements of memory a tensor of rows or pages takes, and whether two
// tensors share any: outputs that lie between inputs' rows (slices of one
// projection, keys and values of a page side by side) are told from outputs
// that lie over them.  Host code, no device.
#pragma once
#include <algorithm>
#include <cstdint>
#include <initializer_list>
#include <utility>

namespace b2b {

// Elements at .. at + run - 1, repeated by up to three (count, stride) levels,
// the outermost first; counted in elements of 2 bytes.
struct Extent {
    struct Level {
        int64_t n, stride;
    };
    int64_t at, run, size;      // size: from the first element to behind the last
    Level by[3];
    int levels;

    Extent(const void* p, int64_t dim, std::initializer_list<Level> dims) : at((int64_t)((uintptr_t)p / 2)), run(dim), levels(0) {
        for (const Level& d : dims)
            if (d.n > 1 && d.stride > 0) by[levels++] = d;
        std::sort(by, by + levels, [](const Level& a, const Level& b) { return a.stride > b.stride; });
        // steps that leave no gap make one run
        while (levels && by[levels - 1].stride <= run) {
            --levels;
            run += (by[levels].n - 1) * by[levels].stride;
        }
        size = run;
        for (int i = 0; i < levels; ++i) size += (by[i].n - 1) * by[i].stride;
    }
    // one step of the outermost level
    Extent inner(int64_t i) const {
        Extent e = *this;
        e.at += i * by[0].stride;
        e.size -= (by[0].n - 1) * by[0].stride;
        --e.levels;
        std::copy(by + 1, by + levels, e.by);
        return e;
    }
    // whether an element lies in [from, to)
    bool meets(int64_t from, int64_t to) const {
        if (to <= at || from >= at + size) return false;
        if (!levels) return true;
        const Level& d = by[0];
        // the first step that begins in the range or behind it
        const int64_t k = from <= at ? 0 : (from - at + d.stride - 1) / d.stride;
        if (k < d.n && at + k * d.stride < to) return true;
        // those before it that reach into it (one, but for steps that lie in each other)
        const Extent first = inner(0);
        for (int64_t i = std::min(k, d.n) - 1; i >= 0 && at + i * d.stride + first.size > from; --i)
            if (inner(i).meets(from, to)) return true;
        return false;
    }
};

inline bool overlap(const Extent& a, const Extent& b) {
    if (a.at + a.size <= b.at || b.at + b.size <= a.at) return false;
    if (!a.levels) return b.meets(a.at, a.at + a.size);
    if (!b.levels) return a.meets(b.at, b.at + b.size);
    const int64_t step = a.by[0].stride;
    const Extent x = a.inner(0), y = b.inner(0);
    if (step == b.by[0].stride && x.size <= step && y.size <= step) {
        // b's step i lies between a's steps i + k and i + k + 1
        const int64_t far = y.at - x.at, k = far >= 0 ? far / step : -((step - 1 - far) / step);
        for (int64_t j : {k, k + 1}) {
            if (j >= a.by[0].n || j <= -b.by[0].n) continue;
            Extent z = y;
            z.at -= j * step;
            if (overlap(x, z)) return true;
        }
        return false;
    }
    // steps of different lengths in each other's ranges: one after another
    const bool fewer = a.by[0].n <= b.by[0].n;
    const Extent &one = fewer ? a : b, &other = fewer ? b : a;
    for (int64_t i = 0; i < one.by[0].n; ++i)
        if (overlap(one.inner(i), other)) return true;
    return false;
}

}  // namespace b2b
