// Extents and their overlaps against sets of elements, one by one: tensors of all
// layouts and many that no caller has.  Prints the number of cases and of overlaps.
#include <cstdio>
#include <cstdlib>
#include <random>
#include <set>
#include <vector>

#include "extent.hpp"

using b2b::Extent;

struct Tensor {
    int64_t at, dim;
    std::vector<Extent::Level> by;
    Extent extent() const {
        const void* p = (const void*)(uintptr_t)(2 * at);
        if (by.size() == 1) return Extent(p, dim, {by[0]});
        if (by.size() == 2) return Extent(p, dim, {by[0], by[1]});
        return Extent(p, dim, {by[0], by[1], by[2]});
    }
    std::set<int64_t> elements() const {
        std::set<int64_t> out = {at};
        for (const auto& d : by) {
            std::set<int64_t> more;
            for (int64_t x : out)
                for (int64_t i = 0; i < d.n; ++i) more.insert(x + i * d.stride);
            out.swap(more);
        }
        std::set<int64_t> all;
        for (int64_t x : out)
            for (int64_t i = 0; i < dim; ++i) all.insert(x + i);
        return all;
    }
};

int main() {
    std::mt19937 rng(1);
    auto pick = [&](int lo, int hi) { return (int64_t)(lo + (int)(rng() % (unsigned)(hi - lo + 1))); };
    const int64_t dims[] = {1, 2, 3, 4}, strides[] = {0, 1, 2, 3, 4, 6, 8, 9, 12, 16, 24, 40, 48};
    int cases = 0, overlaps = 0, wrong = 0;
    auto tensor = [&](int levels) {
        Tensor t{pick(100, 260), dims[pick(0, 3)], {}};
        for (int i = 0; i < levels; ++i) t.by.push_back({pick(1, 5), strides[pick(0, 12)]});
        return t;
    };
    auto check = [&](const Tensor& a, const Tensor& b) {
        const auto x = a.elements(), y = b.elements();
        bool want = false;
        for (int64_t e : x) want = want || y.count(e);
        const Extent p = a.extent(), q = b.extent();
        const bool got = overlap(p, q), back = overlap(q, p);
        const int64_t size = *x.rbegin() - *x.begin() + 1;
        ++cases;
        overlaps += want;
        if (got != want || back != want || p.size != size) {
            if (++wrong < 5) std::printf("case %d: %d %d, %d expected, size %ld of %ld\n", cases, got, back, want, (long)p.size, (long)size);
        }
    };
    for (int i = 0; i < 60000; ++i) {
        const Tensor a = tensor((int)pick(1, 3));
        Tensor b = tensor((int)pick(1, 3));
        if (i % 2) {                    // of the same strides, as slices of one tensor are
            b.by = a.by;
            for (auto& d : b.by) d.n = pick(1, 5);
        }
        check(a, b);
    }
    // slices of a projection of T rows: queries in the place of queries, keys one row on, keys between
    for (int64_t T : {1, 2, 5})
        for (int64_t off = -40; off <= 40; ++off)
            check(Tensor{200, 4, {{T, 16}, {2, 4}}}, Tensor{200 + off, 4, {{T, 16}, {1, 4}}});
    std::printf("%d cases, %d overlaps, %d wrong\n", cases, overlaps, wrong);
    return wrong != 0;
}
