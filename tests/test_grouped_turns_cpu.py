"""Host-side test of the widening warps' waits in the grouped products (csrc/w8_turns.h):
however late an arrival lands, and whichever barrier's lands first, a slot of A is
written again only once its use has ended, no wait is for a phase that has passed, and
nothing is on its way when the last waits have ended.  Barriers are modelled as the
hardware has them: a wait names a phase by its parity, and passes while the phase of
the other parity runs."""
from __future__ import annotations

import os
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp8_weight_only_w8a16_gb300", "csrc")

MODEL = r"""
#include <cassert>
#include <cstdio>
#include <random>
#include "w8_turns.h"
using namespace w8;

struct Bar {
    int phase = 0, late = 0; // late: arrivals on their way (one arrival ends a phase)
    bool passes(uint32_t parity) const { return uint32_t(phase & 1) != parity; }
};

int main()
{
    std::mt19937 rng(1);
    for (int round = 0; round < 30000; ++round) {
        const int slots = 2 + int(rng() % 6), stages = int(rng() % 40);
        const int slow[3] = {1 + int(rng() % 6), 1 + int(rng() % 6), 1 + int(rng() % 6)}; // groups and landings that lag
        Bar used[16];
        const int bars = used_bars(slots);
        bool placed[64] = {};
        int issued = 0, done = 0;
        Turn use[2]; // each group's: the use of the stage `slots` before its next
        int next[2] = {0, 1}, commit = 0;
        int end = stages > slots ? stages - slots : 0; // the last waits
        for (int step = 0; end < stages || done < stages; ++step) {
            assert(step < 200000); // every wait ends
            const int who = int(rng() % 5);
            if (who < 2 && next[who] < stages) {
                const int n = next[who];
                Turn &tu = use[who];
                if (rng() % unsigned(slow[who]))
                    continue;
                if (n >= slots) {
                    assert(tu.n == n - slots);
                    if (bars == slots)
                        assert(tu.k == n % slots && tu.parity == uint32_t((n / slots & 1) ^ 1));
                    if (!used[tu.k].passes(tu.parity))
                        continue;
                    assert(n - slots < done); // its use is over
                }
                placed[n] = true;
                for (int i = n; i < n + 2; ++i)
                    if (i >= slots)
                        tu.step(bars);
                next[who] = n + 2;
            } else if (who == 2 && issued < stages && placed[issued]) {
                ++issued;
            } else if (who == 3 && done < issued) { // a stage's steps end: its arrival is on its way
                ++used[commit].late;
                commit = commit + 1 == bars ? 0 : commit + 1;
                ++done;
            } else if (who == 4) {
                Bar &b = used[rng() % 16u];
                if (b.late && rng() % unsigned(slow[2]) == 0) {
                    --b.late;
                    ++b.phase;
                }
            }
            if (done == stages && end < stages) { // all steps are seen to be done
                if (used[end % bars].passes(uint32_t(end / bars) & 1u))
                    ++end;
            }
        }
        for (const Bar &b : used)
            assert(b.late == 0);
    }
    puts("ok");
}
"""


def test_slots_are_written_again_only_once_they_are_used(tmp_path):
    src, exe = tmp_path / "t.cc", tmp_path / "t"
    src.write_text(MODEL)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-O1", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout == "ok\n"


def test_the_kernel_waits_so():
    text = open(os.path.join(CSRC, "w8_grouped.cu")).read()
    assert "constexpr int kUsed = used_bars(cfg.a);" in text
    # (as many barriers as slots: the slot's own, the phase of the lap before)
    assert "constexpr bool kSlots = kUsed == cfg.a;" in text and "const int use = kSlots ? ta.k : ku," in text
    assert ("pair_commit(&sh.used[use]);\n                        if constexpr (!kSlots)\n                            "
            "ku = ku + 1 == kUsed ? 0 : ku + 1;") in text
    assert "ok = kSlots ? wait(&sh.used[ta.k], ta.parity ^ 1u) : wait(&sh.used[tu.k], tu.parity);" in text
    assert ("if constexpr (!kSlots)\n                    if (ta.n >= cfg.a)\n                        tu.step(kUsed);\n"
            "                ta.step(cfg.a);") in text
    assert "wait_last(sh.used, cfg.a, to.n, kUsed)" in text
    assert text.count("sh.used") == 6  # the four above, and the two that set them up
