// rr_spans.h against a comparison of every pair, on random lists: flat buffers'
// views, scattered tensors, empty ones, many lists and few.
#include <cstdio>
#include <random>

#include "rr_spans.h"

int main()
{
    std::mt19937 r(11);
    auto below = [&](int n) { return (int)(r() % (unsigned)n); };
    int seen[2] = {0, 0};
    rr::Spans spans;
    for (int trial = 0; trial < 20000; ++trial) {
        const int lists = 1 + below(8), n = trial % 50 == 0 ? 200 : 1 + below(12);
        const int room = n * (trial % 3 == 0 ? 40 : trial % 3 == 1 ? 4000 : 40000);
        std::vector<rr::Span> plain;
        spans.all.clear();
        for (int l = 0; l < lists; ++l) {
            const bool written = below(3) > 0, flat = below(3) > 0;
            uintptr_t at = 4096 + (uintptr_t)below(room);
            for (int i = 0; i < n; ++i) {
                const int size = below(10) == 0 ? 0 : 1 + below(30);
                if (!flat) at = 4096 + (uintptr_t)below(room);
                spans.add(reinterpret_cast<const void *>(at), size, written);
                if (size) plain.push_back(rr::Span{at, at + size, written});
                at += size + (below(40) ? 0 : 5) - (below(200) ? 0 : 1);
            }
        }
        bool bad = false;
        for (size_t i = 0; i < plain.size(); ++i)
            for (size_t j = 0; j < i; ++j)
                bad |= plain[i].lo < plain[j].hi && plain[j].lo < plain[i].hi && (plain[i].written || plain[j].written);
        ++seen[bad];
        if (spans.touch() != bad) {
            std::printf("trial %d: %s\n", trial, bad ? "an overlap was missed" : "an overlap was seen where none is");
            return 1;
        }
    }
    std::printf("ok: %d apart, %d overlapping\n", seen[0], seen[1]);
    return seen[0] > 1000 && seen[1] > 1000 ? 0 : 1;
}
