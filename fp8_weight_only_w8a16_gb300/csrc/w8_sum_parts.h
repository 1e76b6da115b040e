// w8_sum_parts.h -- which of the two parts of the sums in tensor memory an item of
// the grouped products has, and which barriers its roles wait for.  Plain C++, so
// that the protocol is also tested on the host.
#pragma once

#include <stdint.h>

#include "w8_layout.h"

namespace w8 {

// The issuer and the warps that store count alike.  A wait names a phase by its
// parity, so a role that skips a phase takes the one before it for the next: an item
// of both parts fills and waits for both barriers, though one commit follows the
// other at once.
struct Parts {
    uint32_t used = 0, parity = 0; // a bit a part: whether it has been used, whether an odd number of times
    uint32_t mask = 0, next = 1;   // the item's parts, the next small item's
    W8_HD void take(int n, int cols)
    {
        mask = n > cols ? 3u : next;
        next = n > cols ? next : next ^ 3u;
    }
    W8_HD uint32_t first() const { return mask == 2 ? 1u : 0u; }
    // Part i's sums: the issuer commits to the barrier, the storing warps wait for it
    // (for its phase of this parity) before they read any of them.
    W8_HD bool fills(int i) const { return mask >> i & 1u; }
    W8_HD uint32_t fill_parity(int i) const { return parity >> i & 1u; }
    // Part i was read before: the issuer waits for that, its last use, which has the
    // other parity.
    W8_HD bool frees(int i) const { return (mask & used) >> i & 1u; }
    W8_HD uint32_t free_parity(int i) const { return (parity >> i & 1u) ^ 1u; }
    W8_HD void done()
    {
        used |= mask;
        parity ^= mask;
    }
};

} // namespace w8
