"""GPU tests of the router's weights at the error that its own operations add up to,
and of infinite scores.

u = 2^-24.  expf is within 2 units of 2^-23 (4 u); an argument x - max is off by
|x - max| u; a sigmoid, 1 / (1 + e), by 4 u of e's share, one of the sum and one of the
quotient: 6 u.  The chosen ones' sum is a tree over 32 lanes: 5 additions; over all
experts each lane adds its own first (2 to 32 of them).  The sum's terms are off as the
weight itself, each by its share; the quotient and the scale add one u each."""
from __future__ import annotations

import pytest
import torch

from .grouped_util import BF, U, check, cuda_gen
from .test_gpu_route import INF, route64, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def grouped():
    from fp8_weight_only_w8a16_gb300 import grouped
    return grouped


def weight_bound(x, ids, want, sigmoid, normalize):
    x, held = x.double(), ids >= 0
    v = torch.where(held, x.gather(1, ids.clamp(min=0).long()), -INF)
    m = v.amax(1, keepdim=True)
    share = torch.where(held, want / want.sum(1, keepdim=True), 0.0)
    d = torch.where(held, m - v, 0.0)  # of the chosen ones
    if sigmoid:
        far = normalize & (m < -30)
        own = torch.where(far, d + 4 + 2.0 ** -19, 6.0)  # (e^-30 is 2^-43: 2^-19 u)
        units = own + (share * own).sum(1, keepdim=True) + 5 + 2 if normalize else own + 1
    elif normalize:
        own = d + 4
        units = own + (share * own).sum(1, keepdim=True) + 5 + 2
    else:
        per = next(p for p in (2, 4, 8, 16, 32) if x.shape[1] <= 32 * p)
        p = torch.softmax(x, 1)
        units = d + 4 + (p * (m - x + 4)).sum(1, keepdim=True) + per + 5 + 2
    return want.abs() * units * U * (1 + 2.0 ** -16) + 1e-43


@pytest.mark.parametrize("experts,top", [(1, 1), (7, 3), (60, 6), (128, 6), (256, 8), (257, 9), (500, 4), (1024, 32)])
@pytest.mark.parametrize("sigmoid,bias", [(False, False), (True, False), (True, True)])
@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("spread,shift", [(0.5, 0.0), (2.0, 0.0), (6.0, 0.0), (3.0, -45.0)])
def test_weights_to_a_few_units(grouped, experts, top, sigmoid, bias, dtype, spread, shift):
    g = cuda_gen(experts + top)
    x = (torch.randn(400, experts, generator=g, device="cuda") * spread + shift).to(dtype)
    b = torch.randn(experts, generator=g, device="cuda") * 0.2 if bias else None
    for normalize, scale in ((True, 2.5), (False, 1.0)):
        ids, w = run(grouped, x, b, top, sigmoid, normalize, scale)
        want_ids, want = route64(x, b, top, sigmoid, normalize, scale)
        assert torch.equal(ids, want_ids)
        check(w, want, weight_bound(x, ids, want, sigmoid, normalize))


@pytest.mark.parametrize("experts", [60, 300, 1024])
@pytest.mark.parametrize("many", [1, 3, 40])
@pytest.mark.parametrize("top", [1, 2, 8])
@pytest.mark.parametrize("dtype", [BF, torch.float32])
def test_infinite_biases(grouped, experts, many, top, dtype):
    """Experts with a bias of +inf come first, the lowest number first; their weights are their sigmoids."""
    g = cuda_gen(experts + many)
    x = torch.randn(300, experts, generator=g, device="cuda").to(dtype)
    b = torch.randn(experts, generator=g, device="cuda") * 0.1
    b[torch.randperm(experts, generator=g, device="cuda")[:many]] = INF
    for normalize in (True, False):
        ids, w = run(grouped, x, b, top, True, normalize)
        want_ids, want = route64(x, b, top, True, normalize, 1.0)
        assert torch.equal(ids, want_ids)
        check(w, want, weight_bound(x, ids, want, True, normalize))


@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("experts", [60, 256])
def test_infinite_logits(grouped, dtype, normalize, experts):
    """+inf: first of all; with softmax the token's weights are NaN, with sigmoids 1 before they are normalised."""
    g = cuda_gen(3)
    x = torch.randn(40, experts, generator=g, device="cuda").to(dtype)
    x[:20, 11] = INF
    x[5:9, 7] = INF
    ids, w = run(grouped, x, None, 4, False, normalize)
    assert torch.equal(ids, route64(x, None, 4, False, normalize, 1.0)[0])
    assert torch.isnan(w[:20]).all() and torch.isfinite(w[20:]).all()
    for b in (None, torch.randn(experts, generator=g, device="cuda") * 0.1):
        ids, w = run(grouped, x, b, 4, True, normalize)
        want_ids, want = route64(x, b, 4, True, normalize, 1.0)
        assert torch.equal(ids, want_ids)
        finite = x.clamp(max=1e4)  # (a sigmoid of 1 either way)
        check(w, want, weight_bound(finite, ids, want, True, normalize))
