// Work along an axis of steps in even pieces, and where the parts of a unit's result lie.
#pragma once

#include "sm103.cuh"

namespace fa {

// `total` steps (below 2^31) dealt to at most `most` workers in contiguous pieces that
// differ by one step at most; the longer pieces come first.
struct Split {
  unsigned total, base, longer;
  int workers;
  FA_DEV Split(unsigned steps, unsigned most) : total(steps) {
    workers = (int)min(steps, most);
    base = workers > 0 ? steps / (unsigned)workers : 0u;
    longer = steps - base * (unsigned)workers;
  }
  FA_DEV unsigned start(int w) const { return (unsigned)w * base + min((unsigned)w, longer); }
  // The worker whose piece holds step x (0 <= x < total).
  FA_DEV int owner(unsigned x) const {
    const unsigned in_longer = longer * (base + 1);
    return (int)(x < in_longer ? x / (base + 1) : longer + (x - in_longer) / base);
  }
  // The slot of a unit's part number `part` of `parts` (its first worker is `first`):
  // unit's own slot, or the worker's slot for the unit that starts in its piece and goes
  // on (odd) or came from the piece before (even).
  FA_DEV static unsigned slot(unsigned unit, unsigned units, int parts, int first, int part) {
    return parts == 1 ? unit : units + 2u * (unsigned)(first + part) + (part == 0 ? 1u : 0u);
  }
};

}  // namespace fa
