// ring_end.h -- how a TMA ring's copies land after a wait of its CTAs has run out (on the device and, as a
// template over the barriers, on the host).
//
// Slice i of a ring goes into stage i % stages; its copies complete the phase i / stages of the stage's barrier. A
// CTA that ends while copies are under way leaves them to write into shared memory that is another's by then.
//
// A ring of two CTAs (a pair) has its barriers in the first one: its producer says for each slice how many bytes both
// CTAs' copies bring. Where the producers gave up after different slices, a barrier waits for bytes that nobody sends, or has
// got bytes that nobody announced; either is made good first. (A producer is at most a ring ahead of the other, since a
// stage is free again only when both its copies have been used.)
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define FDPP_RING_FN __device__ inline
#else
#define FDPP_RING_FN inline
#endif

namespace fdpp {

// The first slice of the ring's last turn.
FDPP_RING_FN uint32_t ring_last_turn(uint32_t issued, uint32_t stages) { return issued > stages ? issued - stages : 0u; }

// Waits for the copies of a ring whose producer issued `own` slices and, in a pair, the other CTA's `other` (the
// same number for a ring of one CTA). Neither issues any more.
//   ring.announce(stage)         arrives at the stage's barrier and announces one CTA's bytes
//   ring.excuse(stage)           takes one CTA's announced bytes back
//   ring.landed(stage, parity)   waits (bounded) for the phase
template <typename Ring>
FDPP_RING_FN void land_ring(Ring& ring, uint32_t own, uint32_t other, uint32_t stages)
{
    const uint32_t end = own > other ? own : other;
    for (uint32_t i = ring_last_turn(end, stages); i < end; ++i) {
        const uint32_t stage = i % stages;
        if (i >= own) ring.announce(stage);
        else if (i >= other) ring.excuse(stage);
        ring.landed(stage, (i / stages) & 1u);
    }
}

}  // namespace fdpp
