"""Host-side test of how the grouped products' roles pass the two parts of the sums
(csrc/w8_sum_parts.h): whenever arrivals come, however late one barrier's are behind
the other's, sums are read only once they are made and made again only once they are
read.  Barriers are modelled as the hardware has them: a wait names a phase by its
parity, and passes while the phase of the other parity runs."""
from __future__ import annotations

import os
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp8_weight_only_w8a16_gb300", "csrc")

MODEL = r"""
#include <cassert>
#include <cstdio>
#include <random>
#include <vector>
#include "w8_sum_parts.h"
using w8::Parts;

constexpr int kCols = 128, kReaders = 3;
struct Bar {
    int count, arrived = 0, phase = 0;
    std::vector<int> late; // the items of the arrivals on their way, the next to land first
    bool passes(uint32_t parity) const { return uint32_t(phase & 1) != parity; }
    int land()
    {
        const int item = late.front();
        late.erase(late.begin());
        if (++arrived == count) {
            arrived = 0;
            ++phase;
        }
        return item;
    }
};
int main()
{
    std::mt19937 rng(1);
    for (int round = 0; round < 20000; ++round) {
        const int items = 2 + int(rng() % 9);
        std::vector<int> n(items);
        for (int &v : n)
            v = 32 * (1 + int(rng() % (rng() % 2 ? 8 : 4)));
        Bar sums[2] = {{1}, {1}}, read[2] = {{kReaders}, {kReaders}};
        std::vector<bool> made(items);            // a commit behind the item's steps has landed
        int holds[2] = {-1, -1}, left[2] = {0, 0}; // a part's item, readers that are not through with it
        Parts issue, reader[kReaders];
        int at = 0, pos[kReaders] = {};
        bool begun = false;
        for (int step = 0; at < items || pos[0] < items || pos[1] < items || pos[2] < items; ++step) {
            assert(step < 100000); // every wait ends
            const int who = int(rng() % 8);
            if (who == 0 && at < items) { // the issuer
                if (!begun) {
                    issue.take(n[at], kCols);
                    begun = true;
                }
                bool ok = true;
                for (int i = 0; i < 2; ++i)
                    ok = ok && (!issue.frees(i) || read[i].passes(issue.free_parity(i)));
                if (!ok)
                    continue;
                for (int i = 0; i < 2; ++i)
                    if (issue.mask >> i & 1) {
                        assert(left[i] == 0); // the part's sums are made again: all have read them
                        holds[i] = at;
                        left[i] = kReaders;
                    }
                for (int i = 0; i < 2; ++i)
                    if (issue.fills(i))
                        sums[i].late.push_back(at);
                issue.done();
                begun = false;
                ++at;
            } else if (who <= kReaders && who > 0 && pos[who - 1] < items) {
                Parts &p = reader[who - 1];
                const Parts before = p;
                p.take(n[pos[who - 1]], kCols);
                bool ok = true;
                for (int i = 0; i < 2; ++i)
                    ok = ok && (!p.fills(i) || sums[i].passes(p.fill_parity(i)));
                if (!ok) {
                    p = before;
                    continue;
                }
                for (int i = 0; i < 2; ++i)
                    if (p.mask >> i & 1) {
                        assert(holds[i] == pos[who - 1] && made[pos[who - 1]]); // this item's sums, their steps done
                        --left[i];
                        read[i].late.push_back(pos[who - 1]);
                    }
                p.done();
                ++pos[who - 1];
            } else if (who >= 6) { // an arrival lands, on any barrier that has one
                Bar *const all[4] = {&sums[0], &sums[1], &read[0], &read[1]};
                const int b = int(rng() % 4);
                if (!all[b]->late.empty()) {
                    const int item = all[b]->land();
                    if (b < 2)
                        made[item] = true;
                }
            }
        }
    }
    puts("ok");
}
"""


def test_sums_are_read_when_made_and_made_when_read(tmp_path):
    src, exe = tmp_path / "t.cc", tmp_path / "t"
    src.write_text(MODEL)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-O1", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout == "ok\n"


def test_the_kernel_waits_as_modelled():
    """Each of the four questions is asked in the kernel, for both parts."""
    text = open(os.path.join(CSRC, "w8_grouped.cu")).read()
    assert text.count("if (parts.frees(i))") == 1 and "bar_wait(&sh.sums_read[i], parts.free_parity(i))" in text
    assert "if (ok && parts.fills(i))\n                            pair_commit(&sh.sums[i]);" in text
    assert "if (parts.fills(i))\n                    ok = ok && warp_wait(&sh.sums[i], parts.fill_parity(i));" in text
    assert "parts.mask" not in text and "parts.parity" not in text
