// w8_turns.h -- slots of the grouped products' rings in turn, and the barriers that tell
// that a slot of A is used.  Plain C++, so that the rules are also tested on the host.
#pragma once

#include <stdint.h>

#include "w8_layout.h"

namespace w8 {

// Slots of a ring in turn, and the parity of their use.
struct Turn {
    int n = 0, k = 0;    // uses so far, the next slot
    uint32_t parity = 0;
    W8_HD void step(int slots)
    {
        ++n;
        if (++k == slots) {
            k = 0;
            parity ^= 1u;
        }
    }
};

// Two groups of warps take the stages of A by turns, and before its stage a group waits
// until the stage that had the slot before is used.  A wait names a phase by its parity,
// so it is sound only on a barrier each of whose phases the group waits for: it may
// neither skip one (an arrival that is still on its way would let it take the phase
// before for the next) nor come so late that the next one has ended, too.  With an even
// number of slots a slot is always the same group's and has one barrier; with an odd one
// the groups have it by turns, and the uses go round twice as many barriers.
W8_HD constexpr int used_bars(int slots) { return slots % 2 ? 2 * slots : slots; }

} // namespace w8
