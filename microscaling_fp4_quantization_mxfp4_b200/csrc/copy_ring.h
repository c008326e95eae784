// Bookkeeping of a ring of shared-memory slots that asynchronous copies fill, each slot behind an mbarrier: when
// the next copy may be asked for, and which copies may still be in flight once a wait has run out.  Plain integers,
// so that it compiles for the host too, where a model of the barriers tests it.
//
// Copy n goes to slot n % slots and completes phase n / slots of the slot's barrier.  It is asked for only when copy
// n - slots has landed and been read, so that at most one phase of a barrier is open.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define FP4_RING_FN __host__ __device__ __forceinline__
#else
#define FP4_RING_FN inline
#endif

namespace fp4ring {

// A reader whose wait ran out (`late`) asks for no more: the slot's phase may still be open, and a second arrival
// in it is undefined.
FP4_RING_FN bool may_ask(bool late, uint32_t asked, uint32_t count) { return !late && asked < count; }

// Of `asked` copies, those from this one on may be in flight.
FP4_RING_FN uint32_t first_open(uint32_t asked, uint32_t slots) { return asked > slots ? asked - slots : 0u; }
FP4_RING_FN uint32_t slot_of(uint32_t n, uint32_t slots) { return n % slots; }
FP4_RING_FN uint32_t parity_of(uint32_t n, uint32_t slots) { return (n / slots) & 1u; }

// A ring over an SM pair: copy n is two shares, one asked for by each CTA, and the leader announces the bytes of both
// on its barrier when it asks for its own.  Once both CTAs have stopped, after the leader has asked `mine` times
// and its peer `peers` times, the copies in flight are waited for; those of which only one share comes are
// made to count that share alone.  barriers: announce_one(slot), arrival with one share's bytes; forgo_one(slot), one
// announced share will not land; wait(slot, parity), false when it runs out.
template <class Barriers>
FP4_RING_FN bool settle_pair(uint32_t mine, uint32_t peers, uint32_t slots, Barriers& barriers) {
  const uint32_t most = mine > peers ? mine : peers;
  for (uint32_t n = first_open(most, slots); n < most; ++n) {
    const uint32_t slot = slot_of(n, slots);
    if (n >= mine) barriers.announce_one(slot);
    else if (n >= peers) barriers.forgo_one(slot);
    if (!barriers.wait(slot, parity_of(n, slots))) return false;
  }
  return true;
}

}  // namespace fp4ring
