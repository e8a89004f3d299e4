// Whether the device memory of a call's arguments overlaps where it must not
// (host code of rr_optim.cu).
#pragma once

#include <algorithm>
#include <cstddef>
#include <cstdint>
#include <vector>

namespace rr {

// A span of device memory of one argument; written ones may touch nothing.
struct Span {
    uintptr_t lo, hi;
    bool written;
};
struct Spans {
    std::vector<Span> all, spare;
    std::vector<size_t> cuts;
    void add(const void *p, int64_t bytes, bool written)
    {
        const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
        if (p && bytes > 0) all.push_back(Span{lo, lo + (uintptr_t)bytes, written});
    }
    // Looks at neighbours in the order of addresses.  Lists over flat buffers are
    // ascending stretches that keep apart as wholes, and need no sorting.
    bool touch()
    {
        auto before = [](const Span &x, const Span &y) { return x.lo < y.lo; };
        cut_up();
        std::vector<Span> &hulls = spare;
        hulls.clear();
        for (size_t k = 0; k + 1 < cuts.size(); ++k) {
            Span hull = all[cuts[k]];
            for (size_t i = cuts[k]; i < cuts[k + 1]; ++i) hull.hi = std::max(hull.hi, all[i].hi);
            hull.written = true;
            hulls.push_back(hull);
        }
        if (cuts.size() <= 64) {
            std::sort(hulls.begin(), hulls.end(), before);
            if (!neighbours_touch(hulls.data(), hulls.size())) {
                for (size_t k = 0; k + 1 < cuts.size(); ++k)
                    if (neighbours_touch(&all[cuts[k]], cuts[k + 1] - cuts[k])) return true;
                return false;
            }
        }
        for (; cuts.size() > 2; cut_up()) {  // join ascending stretches two by two
            spare.resize(all.size());
            for (size_t k = 0; k + 1 < cuts.size(); k += 2) {
                const size_t mid = cuts[k + 1], end = k + 2 < cuts.size() ? cuts[k + 2] : mid;
                std::merge(all.begin() + cuts[k], all.begin() + mid, all.begin() + mid, all.begin() + end,
                           spare.begin() + cuts[k], before);
            }
            all.swap(spare);
        }
        return neighbours_touch(all.data(), all.size());
    }

private:
    // cuts: where ascending stretches begin, and the end.
    void cut_up()
    {
        cuts.clear();
        if (!all.empty()) cuts.push_back(0);
        for (size_t i = 1; i < all.size(); ++i)
            if (all[i].lo < all[i - 1].lo) cuts.push_back(i);
        cuts.push_back(all.size());
    }
    static bool neighbours_touch(const Span *s, size_t n)
    {
        uintptr_t any = 0, written = 0;
        for (size_t i = 0; i < n; ++i) {
            if (s[i].lo < written || (s[i].written && s[i].lo < any)) return true;
            any = std::max(any, s[i].hi);
            if (s[i].written) written = std::max(written, s[i].hi);
        }
        return false;
    }
};

}  // namespace rr
