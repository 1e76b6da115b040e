"""Host-side tests of the attention kernels' copy bookkeeping (csrc/w8_copies.h):
whatever the point at which a wait gives up, every copy that was issued has been
waited for when the CTA leaves.  Compiled for the host against a model of the
barriers: a phase ends with its arrivals and bytes, a wait for a phase that can
never end is an error."""
from __future__ import annotations

import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "fp8_weight_only_w8a16_gb300", "csrc")

RING = r"""
#include <cassert>
#include <cstdio>
#include <vector>
#include "w8_copies.h"

// One CTA copies `uses` slots' worth; its reader has read `read` of them and stops.
template <int S> void run(int uses, int read)
{
    w8::Ring<S> ring;
    std::vector<int> issued;
    for (int i = 0; i < uses; ++i) {
        // slot k's use of the parity before is read
        if (!ring.take([&](int k, uint32_t parity) {
                assert(k == i % S && parity == (uint32_t(i / S - 1) & 1u));
                return i - S < read;
            }))
            break;
        issued.push_back(i);
        ring.filled();
    }
    assert(int(issued.size()) == (uses < read + S ? uses : read + S));
    // the last phase of that parity of slot k that has begun
    std::vector<bool> waited(uses, false);
    ring.drain([&](int k, uint32_t parity) {
        int use = -1;
        for (int i : issued)
            if (i % S == k)
                use = i;
        assert(use >= 0); // else nothing ends the phase
        assert((uint32_t(use / S) & 1u) == parity);
        waited[use] = true;
    });
    for (int i : issued)
        assert(waited[i] || i < read); // what has been read has landed
}
template <int S> void all()
{
    for (int uses = 0; uses < 4 * S + 2; ++uses)
        for (int read = 0; read <= uses; ++read)
            run<S>(uses, read);
}
int main()
{
    all<2>();
    all<3>();
    all<4>();
    all<5>();
    all<12>();
    puts("ok");
}
"""


def run(tmp_path, text):
    src, exe = tmp_path / "t.cc", tmp_path / "t"
    src.write_text(text)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout == "ok\n"


def test_ring_is_drained_wherever_its_reader_stops(tmp_path):
    run(tmp_path, RING)


@pytest.mark.parametrize("kernel,rings", [("w8_latent_paged.cu", 2), ("w8_latent_expanded.cu", 1), ("w8_latent_pair.cu", 1)])
def test_kernels_drain_their_rings(kernel, rings):
    """Every ring of a copying lane is drained, whether or not the lane itself gave up.  (In a pair the second
    CTA's lane waits so for the products that read it: their arrivals are the last to reach the CTA.)"""
    text = open(os.path.join(CSRC, kernel)).read()
    assert text.count("Ring<") == rings and text.count(".drain(") == rings
    for part in text.split(".drain(")[:-1]:
        line = part.splitlines()[-2].strip()  # the line before: no condition
        assert not line.startswith(("if", "else"))


PAIR = r"""
#include <cassert>
#include <cstdio>
#include <cstdlib>
#include <map>
#include <string>
#include <vector>
#include "w8_copies.h"

// One barrier of one arrival a phase: bytes that the phase still waits for, and
// the copies that count on it and have not landed.
struct Bar {
    int phase = 0, pending = 1, bytes = 0;
    std::vector<int *> copies; // their bytes, 0 once landed
    void step()
    {
        while (pending == 0 && bytes == 0) {
            ++phase;
            pending = 1;
        }
    }
    void expect(int n)
    {
        assert(pending == 1); // not twice in a phase
        pending = 0;
        bytes += n;
        step();
    }
    void forgo(int n)
    {
        bytes -= n;
        step();
    }
    void land(int *c)
    {
        bytes -= *c;
        *c = 0;
        step();
    }
    void land_all()
    {
        for (int *c : copies)
            if (*c)
                land(c);
    }
    // What the hardware's wait does with a parity, everything that can land having landed.
    void wait(uint32_t parity, bool &ended)
    {
        land_all();
        ended = (uint32_t(phase) & 1u) != parity;
    }
};

constexpr int kK = 7, kV = 5, kQ = 3, kAnswer = 16;
enum Kind { Keys, Values, Last };

struct Cta {
    std::vector<Bar> full, v_last;
    Bar q, next[2];
    w8::PairIssued did{};
    std::vector<int *> into; // copies on their way into this CTA
    explicit Cta(int slots) : full(slots), v_last(slots) {}
};

struct Bars {
    Cta &c;
    bool all = true;
    void ended(Bar &b, uint32_t parity)
    {
        bool e;
        b.wait(parity, e);
        all = all && e;
    }
    void wait_last(int s, uint32_t p) { ended(c.v_last[s], p); }
    void wait_full(int s, uint32_t p) { ended(c.full[s], p); }
    void expect_full(int s, bool v) { c.full[s].expect(v ? kV : kK); }
    void forgo_full(int s, bool v) { c.full[s].forgo(v ? kV : kK); }
    void wait_queries(uint32_t p) { ended(c.q, p); }
    void expect_queries() { c.q.expect(kQ); }
    void forgo_queries() { c.q.forgo(kQ); }
    void wait_answer(int k, uint32_t p) { ended(c.next[k], p); }
    void expect_answer(int k) { c.next[k].expect(kAnswer); }
};

int *copy(Cta &into, Bar &bar, int bytes)
{
    int *c = new int(bytes);
    into.into.push_back(c);
    bar.copies.push_back(c);
    return c;
}

// A pair with the given items; the products have read `read` slots, with what
// belongs to them; each CTA gives up after `stop[r]` of its steps (a step: the
// queries of an item, a slot, an answer expected).
void run(int slots, const std::vector<int> &items, int read, const int (&stop)[2])
{
    Cta cta[2] = {Cta(slots), Cta(slots)};
    // the sequence of both CTAs' steps
    struct Step { int what; int slot, use; Kind kind; };
    std::vector<Step> steps;
    int use = 0, work = 0, item = 0;
    std::vector<int> first_use, begin; // of each item with keys; each item's first step
    for (int tiles : items) {
        begin.push_back(int(steps.size()));
        steps.push_back({2, item & 1, item, Keys}); // an answer
        ++item;
        if (tiles > 0) {
            first_use.push_back(use);
            steps.push_back({1, 0, work++, Keys}); // queries
            for (int i = 0; i <= tiles; ++i) {
                if (i < tiles)
                    steps.push_back({0, use % slots, use, Keys}), ++use;
                if (i > 0)
                    steps.push_back({0, use % slots, use, i == tiles ? Last : Values}), ++use;
            }
        }
    }
    first_use.push_back(use);
    // Steps in the order in which time runs, CTA by CTA as far as the reads allow.
    int at[2] = {0, 0};
    bool moved = true;
    std::map<int, std::vector<std::pair<Bar *, int *>>> of_use;
    std::map<int, std::vector<std::pair<Bar *, int *>>> of_queries;
    auto reads = [&](int upto) { // slots up to here have been read
        for (auto &u : of_use)
            if (u.first < upto)
                for (auto &c : u.second)
                    if (*c.second)
                        c.first->land(c.second);
        for (auto &u : of_queries)
            if (first_use[u.first] < upto)
                for (auto &c : u.second)
                    if (*c.second)
                        c.first->land(c.second);
    };
    int done = 0; // slots that are read so far: `read` at most, and only what both CTAs have copied
    std::vector<int> copied(use, 0);
    while (moved) {
        moved = false;
        for (int r = 0; r < 2; ++r) {
            Cta &c = cta[r];
            while (at[r] < int(steps.size()) && at[r] < stop[r]) {
                const Step &s = steps[at[r]];
                if (s.what == 0 && s.use - slots >= done)
                    break; // its slot has not been read
                if (s.what == 1 && s.use > 0 && first_use[s.use] - 1 > done) // the last item's scores (all but its last values)
                    break;
                // the answer before has come; asking also takes both CTAs' word on the one before that
                if (s.what == 2 && s.use >= 1 && int(cta[0].did.asks) < s.use)
                    break;
                if (s.what == 2 && s.use >= 2 && r == 0 && at[1] < begin[s.use - 1])
                    break;
                if (s.what == 2) {
                    if (s.use >= 1)
                        c.next[s.slot ^ 1].land_all();
                    c.next[s.slot].expect(kAnswer);
                    ++c.did.expects;
                    if (r == 0) {
                        ++c.did.asks;
                        for (auto &o : cta) {
                            o.next[s.slot].land_all(); // what was there before has been read
                            copy(o, o.next[s.slot], kAnswer);
                        }
                    }
                } else if (s.what == 1) {
                    if (r == 0)
                        c.q.expect(2 * kQ);
                    of_queries[s.use].push_back({&cta[0].q, copy(c, cta[0].q, kQ)});
                    ++c.did.queries;
                } else {
                    const int n = s.kind == Keys ? kK : kV;
                    if (s.kind == Last) {
                        c.v_last[s.slot].expect(kV);
                        of_use[s.use].push_back({&c.v_last[s.slot], copy(c, c.v_last[s.slot], kV)});
                        c.did.last ^= 1u << s.slot;
                    } else {
                        if (r == 0)
                            c.full[s.slot].expect(2 * n);
                        of_use[s.use].push_back({&cta[0].full[s.slot], copy(c, cta[0].full[s.slot], n)});
                        c.did.full ^= 1u << s.slot;
                        c.did.values = s.kind == Values ? c.did.values | 1u << s.slot : c.did.values & ~(1u << s.slot);
                    }
                    ++copied[s.use];
                    c.did.used = uint32_t(s.use + 1);
                }
                ++at[r];
                moved = true;
            }
        }
        while (done < read && done < use && copied[done] == 2)
            ++done, moved = true;
        reads(done);
    }
    for (int r = 0; r < 2; ++r) {
        Bars bars{cta[r]};
        w8::pair_drain(cta[r].did, cta[r ^ 1].did, r == 0, slots, bars);
        assert(bars.all); // no phase is waited for that never ends
    }
    for (auto &c : cta)
        for (int *p : c.into) {
            assert(*p == 0); // landed, and waited for
            delete p;
        }
}

int main()
{
    const std::vector<std::vector<int>> lists = {{1}, {3}, {0, 2, 1}, {1, 1, 1, 1, 1}, {5, 2}, {2, 0, 0, 0, 4, 1}, {9}};
    for (int slots : {4, 5, 8})
        for (const auto &items : lists) {
            int steps = 0, uses = 0;
            for (int t : items)
                steps += 1 + (t > 0 ? 2 * t + 1 : 0), uses += 2 * t;
            for (int read = 0; read <= uses; ++read)
                for (int a = 0; a <= steps; ++a)
                    for (int b = 0; b <= steps; ++b) {
                        const int stop[2] = {a, b};
                        run(slots, items, read, stop);
                    }
        }
    puts("ok");
}
"""


def test_pair_is_drained_wherever_either_cta_stops(tmp_path):
    """Every copy into either CTA of a pair is waited for, and no phase that never ends, whatever the two
    had issued when they gave up."""
    run(tmp_path, PAIR)


def test_pair_kernel_waits_instead_of_sleeping():
    assert "nanosleep" not in open(os.path.join(CSRC, "w8_latent_pair.cu")).read()
