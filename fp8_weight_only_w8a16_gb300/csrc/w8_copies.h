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

// What one CTA of a pair has issued.  Keys, values and queries of both CTAs count
// on barriers of the first, which expects both CTAs' bytes; the values of an item's
// last tile count on a barrier of their own CTA.  After a wait that gave up the two
// may differ, by one use of a barrier at most: a barrier is used again only once
// the products that read both CTAs' copies are done.  `full` and `last`: the parity
// of how often each slot has been used so, a bit a slot.
struct PairIssued {
    uint32_t full;
    uint32_t values;  // whether a slot's last use of `full` was for values, not keys
    uint32_t last;
    uint32_t used;    // slots filled
    uint32_t queries; // items whose queries were copied
    uint32_t expects; // answers of the grid that this CTA expects,
    uint32_t asks;    // that the first CTA has asked for
};

// Waits for every copy that may still be on its way into a CTA of a pair, `mine`
// and `peer` being what the two CTAs have issued.  Where only one of them issued
// its part of a phase, the first CTA makes up for the other's: it expects what it
// had not (expect_*), or counts what never comes as come (forgo_*).  The first CTA
// waits for both CTAs' copies, so neither leaves before it is through.
template <typename Bars>
W8_HD void pair_drain(const PairIssued &mine, const PairIssued &peer, bool first, int slots, Bars &bars)
{
    for (int s = 0; s < slots; ++s) {
        bars.wait_last(s, (mine.last >> s & 1u) ^ 1u); // (never used: the phase before the first, ended)
        if (!first)
            continue;
        uint32_t uses = mine.full >> s & 1u;
        if (uses != (peer.full >> s & 1u)) {
            if (mine.used < peer.used) {
                bars.expect_full(s, peer.values >> s & 1u);
                uses ^= 1u;
            } else {
                bars.forgo_full(s, mine.values >> s & 1u);
            }
        }
        bars.wait_full(s, uses ^ 1u);
    }
    if (first) {
        uint32_t uses = mine.queries;
        if (mine.queries < peer.queries) {
            bars.expect_queries();
            uses = peer.queries;
        } else if (mine.queries > peer.queries) {
            bars.forgo_queries();
        }
        bars.wait_queries((uses & 1u) ^ 1u);
    }
    // the grid's answers, in two places in turn, come to both CTAs
    const uint32_t asks = first ? mine.asks : peer.asks;
    for (uint32_t i = asks > 2 ? asks - 2 : 0; i < asks; ++i) {
        if (i >= mine.expects)
            bars.expect_answer(i & 1u);
        bars.wait_answer(i & 1u, i >> 1 & 1u);
    }
}

} // namespace w8
