// When a wait inside a kernel is recorded and when it is given up.  No device calls, so that a host
// program can run it.
#pragma once

#ifdef __CUDACC__
#define SK_HD __host__ __device__ __forceinline__
#else
#define SK_HD inline
#endif

namespace sk {

// One wait: `test` (does not block) and `poll` (blocks for some time) say whether the phase has
// completed.  `limit` is how many polls pass before `late` is called, once a poll; after `most` more the
// wait is given up by `stop`, after which `stopped` holds and `limit` is not positive for every wait of the
// CTA that begins: such a wait looks once and returns without a poll.  (A wait that had begun ends within
// its own limits.)  So a CTA ends within the time of one more wait and what its roles take without waiting.
// Returns whether the phase completed.
template <class Ops>
SK_HD bool wait_by_rule(Ops &&ops, int most)
{
    if (ops.test()) return true;
    int left = ops.limit();
    do {
        if (--left < 0) {
            ops.late();
            if (left < -most) ops.stop();
            if (ops.stopped()) return false;
        }
    } while (!ops.poll());
    return true;
}

}  // namespace sk
