// w8_copies.h -- which copies of a CTA may still be in flight.  A copying lane
// that is done, or that gave up, waits for them before the CTA leaves: its shared
// memory belongs to another kernel afterwards.  Plain C++, so that the bookkeeping
// is tested on the host.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define W8_HD __host__ __device__ __forceinline__
#else
#define W8_HD inline
#endif

namespace w8 {

// A ring of S slots that one lane fills in turn.  Use i of the ring is use
// i / S of slot i % S, counted by a barrier phase of its own.
template <int S>
struct Ring {
    int used = 0;        // slots filled so far: a slot counts once its copies are issued
    int k = 0;           // the next one,
    uint32_t parity = 0; // and the parity of its use

    // Whether the next slot may be filled: the first time round at once, else when
    // wait(slot, parity) says that what it held before has been read.
    template <typename Wait>
    W8_HD bool take(const Wait &wait) const
    {
        return used < S || wait(k, parity ^ 1u);
    }
    W8_HD void filled()
    {
        ++used;
        if (++k == S) {
            k = 0;
            parity ^= 1u;
        }
    }
    // wait(slot, parity) for each use whose copies may not have landed: the last
    // of every slot.  (That a slot was filled again says that its copies before had.)
    template <typename Wait>
    W8_HD void drain(const Wait &wait) const
    {
        for (int i = used > S ? used - S : 0; i < used; ++i)
            wait(i % S, uint32_t(i / S) & 1u);
    }
};

} // namespace w8
