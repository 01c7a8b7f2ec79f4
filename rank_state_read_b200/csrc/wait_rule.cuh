// When a wait inside a kernel is recorded and when it is given up, and which copies are under way then.
// No device calls, so that a host program can run it.
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

// Phases of a ring of up to 16 stages that one copy after another fills: which parity the next wait on a
// stage takes, and which stages have a copy under way.  A wait that was lost leaves both as they are,
// so that a later one still asks for that copy.
struct RingPhases {
    unsigned parity_bits = 0, under_way = 0;

    SK_HD void issued(int stage) { under_way |= 1u << stage; }
    SK_HD unsigned parity(int stage) const { return parity_bits >> stage & 1; }
    SK_HD bool pending(int stage) const { return under_way >> stage & 1; }
    SK_HD void landed(int stage)
    {
        parity_bits ^= 1u << stage;
        under_way &= ~(1u << stage);
    }
};

}  // namespace sk
