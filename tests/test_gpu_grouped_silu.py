"""GPU tests of SiLU-and-multiply in the grouped products: how exact it is, and gates
far from 0.

A bf16 plane of two columns and rows of ones make the sums g and u from two bf16
values each, exactly, so the output is the function's alone.  Its error is counted in
the rounding itself: with the function within 2^-19.5 of its value (expf within two
units of 2^-23, twice; 1 + e^-|g| and its reciprocal; five roundings to fp32: below
2^-19.7), the output is one of the bf16 values between those that the definition's
value, less and more that much, rounds to."""
from __future__ import annotations

import pytest
import torch

from .grouped_util import BF, cuda_gen, groups_of, silu64

pytestmark = pytest.mark.gpu
REL = 2.0 ** -19.5
TINY = 2.0 ** -149  # a unit of the smallest fp32 values


@pytest.fixture(scope="module")
def grouped():
    from fp8_weight_only_w8a16_gb300 import grouped
    yield grouped
    assert grouped.device_status() == 0


def parts(v):
    """fp32 values of 16 bits as two bf16 values: v, and what they are."""
    v = (v.float().contiguous().view(torch.int32) & ~0xFF).view(torch.float32).double()
    hi = v.to(BF)
    lo = (v - hi.double()).to(BF)
    assert torch.equal(hi.double() + lo.double(), v)
    return hi, lo, v


def run(grouped, g, u, counts):
    """silu(g) u for [planes, inner] gates and ups, every row of a group alike."""
    from fp8_weight_only_w8a16_gb300 import w8
    groups, inner = g.shape
    w = torch.zeros(groups, 2 * inner, 32, dtype=BF, device="cuda")
    w[:, :inner, 0], w[:, :inner, 1], g = parts(g)
    w[:, inner:, 0], w[:, inner:, 1], u = parts(u)
    build = w8.bind([w8.Plane.from_tensor(w[e], layout=w8.SRC_GATE_UP) for e in range(groups)])
    pos = sum(counts)
    x = torch.zeros(pos, 32, dtype=BF, device="cuda")
    x[:, :2] = 1.0
    h = torch.zeros(pos, inner, dtype=BF, device="cuda")
    grouped.grouped_gemv(build, 0, groups_of(counts), x, h, silu_mul=True)
    rows = torch.repeat_interleave(torch.arange(groups, device="cuda"), torch.tensor(counts, device="cuda"))
    return h, g[rows], u[rows]


def check(h, want):
    slack = REL * want.abs() + TINY
    low, high = ((want - slack).float().to(BF), (want + slack).float().to(BF))
    bad = ~((h >= low) & (h <= high))
    assert not bad.any(), (int(bad.sum()), h[bad][:4], want[bad][:4])


COUNTS = [[3, 1, 20, 16], [50, 45, 64, 40], [100, 97, 128, 110]]  # items of each size


@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("spread", [0.25, 2.0, 20.0, 60.0])
def test_within_the_functions_error(grouped, counts, spread):
    g = cuda_gen(int(4 * spread))
    gate = torch.randn(len(counts), 4096, generator=g, device="cuda") * spread
    up = torch.randn(len(counts), 4096, generator=g, device="cuda")
    h, gv, uv = run(grouped, gate.clamp(-85, 85), up, counts)
    check(h, silu64(gv) * uv)


@pytest.mark.parametrize("counts", COUNTS)
def test_gates_far_from_zero(grouped, counts):
    """Where e^-g is past fp32, the product with a large u is not; and very large ones."""
    g = cuda_gen(9)
    n = 2048
    gate = -80 - 94 * torch.rand(len(counts), n, generator=g, device="cuda")  # (e^-87 is a normal fp32 value still)
    up = torch.randn(len(counts), n, generator=g, device="cuda").sign() * 2.0 ** (127 * torch.rand(len(counts), n, generator=g, device="cuda"))
    gate[:, :64] = 1.0 + 3 * torch.rand(len(counts), 64, generator=g, device="cuda")  # g u past fp32, silu(g) u not always
    up[:, :64] = 1.9 * 2.0 ** 127 / gate[:, :64]
    gate[:, 64:128] = 2.0 ** (100 * torch.rand(len(counts), 64, generator=g, device="cuda"))
    up[:, 64:128] = 1.0 / gate[:, 64:128]
    h, gv, uv = run(grouped, gate, up, counts)
    want = gv * torch.exp(gv.clamp(max=0.0)) / (1 + torch.exp(-gv.abs())) * uv
    check(h, want)
