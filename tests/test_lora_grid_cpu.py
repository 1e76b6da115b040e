"""Host-side test of the adapters' launch shape (csrc/w8_layout.h): one to eight steps a
CTA at every size that the call takes."""
from __future__ import annotations

import os
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp8_weight_only_w8a16_gb300", "csrc")

TEXT = r"""
#include <cassert>
#include <cstdio>
#include <initializer_list>
#include "w8_layout.h"
int main()
{
    using w8::expand_steps;
    for (int sms : {1, 132, 148, 152})
        for (int64_t tiles = 1; tiles <= (1 << 26) + 1024; tiles = tiles * 3 / 2 + 1)
            for (int64_t blocks = 1; blocks <= 1 << 15; blocks = blocks * 3 / 2 + 1) {
                const int per = expand_steps(tiles, blocks, sms);
                const int64_t steps = tiles * blocks, wave = 4 * sms;
                assert(per >= 1 && per <= 8);
                assert(per == 8 || per * wave >= steps);
                assert(per == 1 || (per - 1) * wave < steps);
            }
    assert(expand_steps((1 << 26) + 1024, 1 << 15, 152) == 8); // 2^41 steps
    puts("ok");
}
"""


def test_steps_of_a_cta(tmp_path):
    src, exe = tmp_path / "t.cc", tmp_path / "t"
    src.write_text(TEXT)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout == "ok\n"
