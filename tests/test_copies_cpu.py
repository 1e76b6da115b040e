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


@pytest.mark.parametrize("kernel,rings", [("w8_latent_paged.cu", 2), ("w8_latent_expanded.cu", 1)])
def test_kernels_drain_their_rings(kernel, rings):
    """Every ring of a copying lane is drained, whether or not the lane itself gave up."""
    text = open(os.path.join(CSRC, kernel)).read()
    assert text.count("Ring<") == rings and text.count(".drain(") == rings
    for part in text.split(".drain(")[:-1]:
        line = part.splitlines()[-2].strip()  # the line before: no condition
        assert not line.startswith(("if", "else"))
