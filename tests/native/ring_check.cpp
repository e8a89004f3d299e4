// Plays the two accumulators of a product and one warp that adds them up
// (rr_ring.h): the products stop for good after some number of stages, and every
// tile that the warp calls good must have been made of its own stages, each once.
#include <cstdio>
#include <vector>

#include "rr_ring.h"

namespace {

// A barrier whose phases complete one by one; a test of parity p is true when the
// last completed phase has it (or, on a fresh barrier, for parity 1).
struct Barrier {
    int completed = 0;
    bool test(int parity) const { return (completed & 1) != parity; }
};

struct Products {
    std::vector<int> all;  // numbers of the stages in order
    int stop, issued = 0;
    Barrier done[2], free[2];
    int holds[2] = {-1, -1};
    rr::Turn<2> turn{1};
    Products(int stages, int stop) : stop(stop)
    {
        for (int i = 0; i < stages; ++i) all.push_back(i);
    }
    void run()  // as far as they can
    {
        while (issued < (int)all.size() && issued < stop && free[turn.at].test(turn.phase)) {
            holds[turn.at] = all[issued++];
            ++done[turn.at].completed;
            turn.next();
        }
    }
};

int play(const std::vector<int> &depths, int stop)
{
    int stages = 0, bad = 0;
    for (int d : depths) stages += d;
    Products p(stages, stop);
    rr::Turn<2> turn(0);
    bool ok = true, failed = false;
    int stage = 0, released = 0;
    for (int d : depths) {
        std::vector<int> got;
        ok = rr::take_turns(
            ok, turn, d,
            [&](const rr::Turn<2> &t) {  // the limit: nothing moves any more
                p.run();
                return p.done[t.at].test(t.phase);
            },
            [&](const rr::Turn<2> &t) { got.push_back(p.holds[t.at]); },
            [&](const rr::Turn<2> &t) {
                ++p.free[t.at].completed;
                ++released;
            });
        bool right = (int)got.size() == d;
        for (int k = 0; k < d && right; ++k) right = got[k] == stage + k;
        if (ok && !right) ++bad;           // a tile called good that is not made of its stages
        if (ok && failed) ++bad;           // good again after a wait that ran out
        if (!ok && stage + d <= stop) ++bad;  // called bad though all of it came
        failed = failed || !ok;
        stage += d;
    }
    if (released > p.issued) ++bad;        // let go what was never there
    return bad;
}

}  // namespace

int main()
{
    const std::vector<std::vector<int>> lists = {{1, 1, 1, 1, 1, 1, 1}, {2, 2, 2, 2, 2, 2}, {2, 1, 2, 1, 1, 2}, {3, 3, 3, 3}, {4, 4, 4},
                                                 {1, 5, 2, 7, 1, 1, 8}, {56, 2, 56}, {16, 16, 2, 2, 1}};
    for (size_t i = 0; i < lists.size(); ++i) {
        int stages = 0;
        for (int d : lists[i]) stages += d;
        for (int stop = 0; stop <= stages; ++stop)
            if (int bad = play(lists[i], stop)) {
                std::printf("list %zu, products stop after %d of %d stages: %d wrong\n", i, stop, stages, bad);
                return 1;
            }
    }
    std::puts("ok");
    return 0;
}
