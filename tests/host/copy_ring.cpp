// Model of mbarriers and of copies that land late, driven by the kernels' own ring bookkeeping (csrc/copy_ring.h).
#include <stdint.h>

#include <vector>

#include "copy_ring.h"

namespace {

// One arrival a phase; the phase completes when it has arrived and as many bytes have landed as were announced.
struct Bar {
  uint32_t phase = 0;
  int pending = 1, tx = 0, bad = 0;
  void settle() {
    if (pending == 0 && tx == 0) {
      ++phase;
      pending = 1;
    }
  }
  void announce(int bytes) {
    if (pending == 0) ++bad;              // a second arrival in one phase
    --pending;
    tx += bytes;
    settle();
  }
  void land(int bytes) {
    tx -= bytes;
    settle();
  }
  bool done(uint32_t parity) const { return (phase & 1u) != parity; }
};

struct Copy {
  uint32_t slot;
  bool landed;
};

}  // namespace

extern "C" {

// `count` copies through a ring read R at a time, as a block of the norm's backward pass reads its rows.  Copy
// `stuck` and those behind it land only after the reader's wait for `stuck` has run out: each `lag` steps of R
// later, or while the block waits at its end.  ask_late: the reader goes on asking.  Returns the number of faults: second
// arrivals, copies asked for into a slot with one in flight, copies in flight when the block has gone.
int ring_faults(uint32_t slots, uint32_t count, uint32_t R, uint32_t stuck, uint32_t lag, int ask_late) {
  std::vector<Bar> bar(slots);
  std::vector<Copy> copies;
  int faults = 0;
  uint32_t steps_late = 0;
  bool late = false;
  auto ask = [&] {
    const uint32_t n = (uint32_t)copies.size(), s = fp4ring::slot_of(n, slots);
    for (const Copy& c : copies)
      if (c.slot == s && !c.landed) ++faults;
    bar[s].announce(64);
    copies.push_back({s, false});
    if (n < stuck) {
      copies.back().landed = true;
      bar[s].land(64);
    }
  };
  auto land_oldest = [&] {
    for (Copy& c : copies)
      if (!c.landed) {
        c.landed = true;
        bar[c.slot].land(64);
        return;
      }
  };
  while (copies.size() < slots && fp4ring::may_ask(false, (uint32_t)copies.size(), count)) ask();
  for (uint32_t n0 = 0; n0 < count; n0 += R) {
    for (uint32_t r = 0; r < R && n0 + r < count; ++r) {
      const uint32_t n = n0 + r;
      if (!late && !bar[fp4ring::slot_of(n, slots)].done(fp4ring::parity_of(n, slots))) late = true;
    }
    if (n0 > 0)
      for (uint32_t r = 0; r < R && fp4ring::may_ask(late && !ask_late, (uint32_t)copies.size(), count); ++r) ask();
    if (late && ++steps_late % lag == 0) land_oldest();
  }
  if (late) {
    const uint32_t asked = (uint32_t)copies.size();
    for (uint32_t n = fp4ring::first_open(asked, slots); n < asked; ++n) {
      const uint32_t s = fp4ring::slot_of(n, slots);
      for (Copy& c : copies)                 // the copy lands while it is waited for
        if (c.slot == s && !c.landed && !bar[s].done(fp4ring::parity_of(n, slots))) {
          c.landed = true;
          bar[s].land(64);
        }
      if (!bar[s].done(fp4ring::parity_of(n, slots))) ++faults;
    }
  }
  for (const Copy& c : copies) faults += c.landed ? 0 : 1;
  for (const Bar& b : bar) faults += b.bad;
  return faults;
}


// An SM pair that stopped after `done` copies through the ring had landed and been read, `mine` asked for by the
// leader and `peers` by its peer.  Bit n of own_late / peer_late: that CTA's share of copy done + n lands only while the
// pair waits for it at the end.  Returns the faults, as above, and waits that run out.
int pair_faults(uint32_t slots, uint32_t done, uint32_t mine, uint32_t peers, uint32_t own_late, uint32_t peer_late) {
  struct Ring {
    std::vector<Bar> bar;
    struct Share {
      uint32_t n;
      bool landed;
    };
    std::vector<Share> shares;
    uint32_t slots;
    int faults = 0;
    void announce_one(uint32_t slot) { bar[slot].announce(64); }
    void forgo_one(uint32_t slot) { bar[slot].land(64); }
    bool wait(uint32_t slot, uint32_t parity) {
      for (Share& s : shares)
        if (s.n % slots == slot && !s.landed) {
          if (bar[slot].done(parity)) ++faults;           // the phase is over, a share of it still flies
          s.landed = true;
          bar[slot].land(64);
        }
      if (!bar[slot].done(parity)) ++faults;
      return true;
    }
  } ring;
  ring.bar.resize(slots);
  ring.slots = slots;
  for (uint32_t n = 0; n < (mine > peers ? mine : peers); ++n) {
    const uint32_t slot = fp4ring::slot_of(n, slots);
    if (n < mine) ring.bar[slot].announce(128);
    for (int who = 0; who < 2; ++who) {
      if (n >= (who ? peers : mine)) continue;
      const bool late = n >= done && ((who ? peer_late : own_late) >> (n - done) & 1u);
      ring.shares.push_back({n, !late});
      if (!late) ring.bar[slot].land(64);
    }
  }
  fp4ring::settle_pair(mine, peers, slots, ring);
  for (const auto& s : ring.shares) ring.faults += s.landed ? 0 : 1;
  for (const Bar& b : ring.bar) ring.faults += b.bad;
  return ring.faults;
}


// A producer asked for `asked` copies, all but the last `slots` of which have landed, and waits at its end for those that
// `counted` says may be in flight.  Returns those that still fly when it has gone.
int copies_missed(uint32_t slots, uint32_t asked, uint32_t counted) {
  std::vector<Bar> bar(slots);
  std::vector<bool> flies(slots, false);
  for (uint32_t n = 0; n < asked; ++n) {
    const uint32_t s = fp4ring::slot_of(n, slots);
    bar[s].announce(64);
    if (n + slots < asked) bar[s].land(64);
    else flies[s] = true;
  }
  for (uint32_t n = fp4ring::first_open(counted, slots); n < counted; ++n) {
    const uint32_t s = fp4ring::slot_of(n, slots);
    if (!bar[s].done(fp4ring::parity_of(n, slots)) && flies[s]) {         // it lands while it is waited for
      flies[s] = false;
      bar[s].land(64);
    }
  }
  int missed = 0;
  for (bool f : flies) missed += f;
  return missed;
}

}
