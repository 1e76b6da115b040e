"""GPU tests of the first capture: in a fresh process one small call of an operator on
the device is enough, whatever sizes, ranks and types a capture then asks for.  Each
runs in a process of its own, where nothing else has loaded or prepared the kernels."""
from __future__ import annotations

import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

COMMON = r"""
import torch
from fp8_weight_only_w8a16_gb300 import grouped, w8
from tests.grouped_util import BF, Planes, check, cuda_gen, groups_of, i32, product_bound, silu64, silu_bound

def captured(call):
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    graph.replay()
    torch.cuda.synchronize()
"""

GROUPED = COMMON + r"""
n, k = 96, 160
half = n // 2
first = Planes(2, n, k, False, seed=1)
y = torch.zeros(3, n, dtype=BF, device="cuda")
grouped.grouped_gemv(first.build, 0, i32([0, 1, 3]), torch.ones(3, k, dtype=BF, device="cuda"), y)
torch.cuda.synchronize()
for bf16 in (False, True):
    p = Planes(3, n, k, bf16, gated=True, seed=2)
    for counts in ([3, 0, 20], [50, 45, 64], [200, 30, 140]):
        x = (torch.randn(sum(counts), k, generator=cuda_gen(3), device="cuda") * 0.5).to(BF)
        offsets = groups_of(counts)
        want, mag = p.products(offsets, x)
        y = torch.zeros(sum(counts), n, dtype=BF, device="cuda")
        h = torch.zeros(sum(counts), half, dtype=BF, device="cuda")
        captured(lambda: grouped.grouped_gemv(p.build, 0, offsets, x, y))
        check(y, want, product_bound(want, mag, k))
        captured(lambda: grouped.grouped_gemv(p.build, 0, offsets, x, h, silu_mul=True))
        check(h, silu64(want[:, :half]) * want[:, half:], silu_bound(want[:, :half], want[:, half:], mag[:, :half], mag[:, half:], k))
assert grouped.device_status() == 0
print("ok")
"""

ADAPTERS = COMMON + r"""
from tests.test_gpu_lora import buffer, lora64
g = cuda_gen(1)

def call(toks, k, n, rank, adapters, pad):
    x, y, out = buffer((toks, k), 0, g), buffer((toks, n), pad, g), buffer((toks, n), pad, g)
    a, b = buffer((adapters, rank, k), 0, g, 0.1), buffer((adapters, n, rank), 0, g, 0.3)
    order = torch.randperm(toks, generator=g, device="cuda").to(torch.int32)
    offsets = groups_of([toks // adapters] * (adapters - 1) + [toks - toks // adapters * (adapters - 1)])
    ws = grouped.new_lora_workspace(toks, k, rank, adapters)
    torch.cuda.synchronize()
    return (lambda: grouped.lora_add(x, a, b, order, offsets, y, out, ws)), (x, a, b, order, offsets, y, None, None), out

call(2, 64, 64, 8, 1, 0)[0]()
torch.cuda.synchronize()
for toks, k, n, rank, adapters, pad in ((5, 64, 40, 16, 2, 0), (5, 64, 40, 128, 2, 8), (40, 128, 40, 64, 4, 1), (300, 4096, 264, 64, 2, 0),
                                        (300, 512, 264, 64, 2, 0), (300, 2048, 264, 128, 2, 0), (1100, 8192, 264, 32, 2, 0),
                                        (1100, 512, 264, 16, 2, 0)):
    run, args, out = call(toks, k, n, rank, adapters, pad)
    captured(run)
    want, bound = lora64(*args)
    check(out, want, bound)
assert grouped.device_status() == 0
print("ok")
"""

OTHERS = COMMON + r"""
g = cuda_gen(1)
ids, w = torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.zeros(1, 1, device="cuda")
grouped.expert_route(torch.ones(1, 4, device="cuda"), None, ids, w)
order, offsets = torch.zeros(1, dtype=torch.int32, device="cuda"), i32([0, 0])
grouped.group_rows(ids, 1, order, None, offsets)
out = torch.zeros(1, 8, dtype=BF, device="cuda")
grouped.expert_sum(torch.ones(1, 8, dtype=BF, device="cuda"), ids, w, out)
torch.cuda.synchronize()
for experts, dtype in ((64, BF), (100, torch.float32), (256, BF), (300, torch.float32), (1024, BF)):
    x = torch.randn(2000, experts, generator=g, device="cuda").to(dtype)
    ids, w = torch.zeros(2000, 6, dtype=torch.int32, device="cuda"), torch.zeros(2000, 6, device="cuda")
    order, rows, offsets = torch.zeros(12000, dtype=torch.int32, device="cuda"), torch.zeros(12000, dtype=torch.int32, device="cuda"), i32([0] * (experts + 1))
    ws = grouped.new_group_workspace(12000, experts)
    y, out = torch.randn(12000, 41, generator=g, device="cuda").to(BF), torch.zeros(2000, 41, dtype=BF, device="cuda")

    def step():
        grouped.expert_route(x, None, ids, w)
        grouped.group_rows(ids, 6, order, rows, offsets, ws)
        grouped.expert_sum(y, ids, w, out)

    captured(step)
    assert torch.equal(ids.long(), torch.sort(x.double(), dim=1, descending=True, stable=True).indices[:, :6])
    assert torch.equal(order.long(), torch.argsort(ids.reshape(-1), stable=True)) and torch.equal(rows, order // 6)
    want = (y.view(2000, 6, 41).double() * w.double()[:, :, None]).sum(1)
    assert ((out.double() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-5).all()
print("ok")
"""


@pytest.mark.parametrize("name", ["GROUPED", "ADAPTERS", "OTHERS"])
def test_one_small_call_prepares_every_capture(name):
    got = subprocess.run([sys.executable, "-c", globals()[name]], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert got.returncode == 0 and got.stdout.endswith("ok\n"), got.stderr[-2000:]
