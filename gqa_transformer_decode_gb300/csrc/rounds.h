// rounds.h -- loops whose end is not to depend on what they find: rounds of work that several warps
// begin together, each of which may give up in any of them, and walks along a line.  Plain C++, so
// that the way they end can be tested without a GPU.
#pragma once

#ifdef __CUDACC__
#define EMBER_ROUNDS __device__ __forceinline__
#else
#define EMBER_ROUNDS inline
#endif

namespace ember {

// Every worker calls this with the same n.  Before each round it says whether it is ready, and
// all(ok) answers them all with whether every one was: a barrier that each must come to.  A
// worker that gave up, in a round's work or waiting for it, still comes to the next vote, so that
// nobody waits there for good; after a vote that fails none of them comes again.
// True: all rounds were done.
template <class Ready, class All, class Work>
EMBER_ROUNDS bool rounds_together(int n, Ready ready, All all, Work work) {
    bool ok = true;
    for (int i = 0; i < n; ++i) {
        ok = ok && ready(i);
        if (!all(ok)) return false;
        ok = work(i);
    }
    return ok;
}

// From place `at` of a line on by `step`; false at the line's end, and where there is no step, so
// that a walk ends even if what it reads changes under it.
EMBER_ROUNDS bool walk_on(unsigned& at, int step, unsigned end) {
    if (step <= 0 || (unsigned)step >= end - at) return false;
    at += (unsigned)step;
    return true;
}

}  // namespace ember
