// Turns of a ring of barriers, and how a warp takes what comes around in one
// (rr_muon.cu; host code too, for the tests).  Not part of the public ABI.
#pragma once

#if defined(__CUDACC__)
#define RR_HD __host__ __device__ __forceinline__
#else
#define RR_HD inline
#endif

namespace rr {

// A place in a ring, and the parity of the barrier phase that belongs to it.
template <int N>
struct Turn {
    int at = 0, phase;
    RR_HD explicit Turn(int first) : phase(first) {}
    RR_HD void next()
    {
        if (++at == N) {
            at = 0;
            phase ^= 1;
        }
    }
};

// Waits for `depth` turns one after the other, takes each and lets it go again.
// `ok` is what became of a thread's turns before: once a wait has run out, nothing
// later counts, in this stretch or in one after it.  A barrier's parity tells a phase
// from the next one only, so one that stands still would look complete again two
// phases on; and what a thread was too late for it does not let go, or others would
// lose what lies there.  It takes all turns, as the threads of its warp take them
// together (what it takes then is no use, and ok says so).
template <int N, class Wait, class Take, class Release>
RR_HD bool take_turns(bool ok, Turn<N> &turn, int depth, Wait wait, Take take, Release release)
{
    for (; depth > 0; --depth, turn.next()) {
        ok = ok && wait(turn);
        take(turn);
        if (ok) release(turn);
    }
    return ok;
}

}  // namespace rr
