"""GPU tests of the grouped products with rows that are not finite: at every item size,
rows in turn and rows by number, plain and with SiLU."""
from __future__ import annotations

import pytest
import torch

from .grouped_util import BF, Planes, cuda_gen, groups_of, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def grouped():
    from fp8_weight_only_w8a16_gb300 import grouped
    yield grouped
    assert grouped.device_status() == 0


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("sizes", [[19, 21, 0, 7], [50, 60, 0, 55], [200, 0, 140, 257]])
@pytest.mark.parametrize("k", [128, 1000])
def test_rows_stay_apart(grouped, bf16, silu, sizes, k):
    """NaN and infinities in a row of x reach the outputs of its positions only, and a
    position whose row is outside is zero, whatever row 0 (or any other) holds."""
    n = 80
    p = Planes(len(sizes), n, k, bf16, gated=True, whole=True, seed=8)
    g = cuda_gen(k)
    pos = sum(sizes)
    x = torch.randint(1, 9, (pos, k), generator=g, device="cuda").to(BF)
    offsets = groups_of(sizes)
    bad = x.clone()
    bad[0, 5], bad[pos // 2, k - 1], bad[pos - 1, 0] = float("nan"), float("inf"), -float("inf")
    wrong = torch.zeros(pos + 1, dtype=torch.bool, device="cuda")
    wrong[[0, pos // 2, pos - 1]] = True
    by_number = torch.randint(0, pos, (pos,), generator=g, device="cuda").to(torch.int32)
    by_number[[3, pos - 2]] = i32([0, 0])
    outside = by_number.clone()
    outside[::5] = -1
    outside[1::7] = pos
    for rows in (None, by_number, outside):
        shape = (pos, n // 2 if silu else n)
        clean, y = torch.full(shape, 7.0, dtype=BF, device="cuda"), torch.full(shape, 7.0, dtype=BF, device="cuda")
        grouped.grouped_gemv(p.build, 0, offsets, x, clean, x_rows=rows, silu_mul=silu)
        grouped.grouped_gemv(p.build, 0, offsets, bad, y, x_rows=rows, silu_mul=silu)
        names = torch.arange(pos, device="cuda") if rows is None else rows.long()
        out = (names < 0) | (names >= pos)
        reached = wrong[torch.where(out, pos, names)]
        assert reached.any() and torch.equal(y[~reached], clean[~reached])
        assert (y[out] == 0).all() and torch.isfinite(clean.float()).all()
        nan = reached & (names == 0)
        assert nan.any() and torch.isnan(y[nan]).all()
        if not silu:
            assert not torch.isfinite(y[reached]).any()


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("sizes", [[19, 21], [50, 60], [200, 140]])
def test_outputs_without_values_in_between(grouped, bf16, sizes):
    """The same at items of every size: what stale places held (NaN of the call before)
    reaches no sum."""
    p = Planes(2, 272, 320, bf16, whole=True, seed=3)
    pos = sum(sizes)
    x = torch.randint(-8, 9, (pos, 320), generator=cuda_gen(1), device="cuda").to(BF)
    nothing = torch.full_like(x, float("nan"))
    rows = torch.arange(pos - 1, -1, -1, device="cuda").to(torch.int32)
    for by in (None, rows):
        full, few = groups_of(sizes), groups_of([s - 15 for s in sizes])
        for offsets in (full, few):
            y = torch.zeros(pos, 272, dtype=BF, device="cuda")
            grouped.grouped_gemv(p.build, 0, full, nothing, y, x_rows=by)
            assert torch.isnan(y).all()
            y.fill_(7.0)
            grouped.grouped_gemv(p.build, 0, offsets, x, y, x_rows=by)
            held = int(offsets[-1])
            assert torch.equal(y[:held], p.products(offsets, x, by)[0].to(BF)) and (y[held:] == 7).all()
