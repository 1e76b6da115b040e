"""Host-side test of what an operator's first call prepares: the shared-memory limits
of all of its kernels, so that a capture after one call of any size sets none."""
from __future__ import annotations

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp8_weight_only_w8a16_gb300", "csrc")


@pytest.mark.parametrize("name,entry", [("w8_grouped.cu", "launch_grouped"), ("w8_lora.cu", "launch_lora"),
                                        ("w8_group_rows.cu", "launch_group_rows")])
def test_one_place_raises_all_limits_before_any_launch(name, entry):
    text = open(os.path.join(CSRC, name)).read()
    assert text.count("raise_smem(") == 1 and text.count("std::atomic<uint64_t>") == 1
    body = text[text.index(f"cudaError_t {entry}("):]
    first = body[:body.index("\n}\n")]
    at = re.search(r"raise_all\(|raise_smem\(", first)
    assert at and at.start() < re.search(r"launch_dependent|launch_sized|lora<", first).start()


def test_the_adapters_list_names_every_kernel_past_the_default():
    text = open(os.path.join(CSRC, "w8_lora.cu")).read()
    raised = text[text.index("cudaError_t raise_all()"):]
    raised = raised[:raised.index("\n}\n")]
    for kernel in ("shrink_kernel<8>", "shrink_tc_kernel<64>", "shrink_tc_kernel<128>", "expand_tc_kernel<64>", "expand_tc_kernel<128>"):
        assert f"&{kernel})" in raised
