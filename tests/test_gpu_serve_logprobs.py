"""GPU tests of token_logprobs against a 64-bit plain form.

Bounds: with u = 2^-24, the sum of exponentials carries a factor of at most
2^-20 (the exponential, its argument's rounding weighted by the term, joins)
plus n u over the longest chain of additions (a thread's run, 40 joins), here
n <= 2048; a log probability adds 3 roundings of its own size and of the
distance to the maximum; the entropy is a quotient of two such sums, its terms
up to ln V.  Top tokens are compared exactly: a logit's order is not rounded."""
from __future__ import annotations

import pytest
import torch

from tests.serve_util import NEG, U, logprobs64

pytestmark = pytest.mark.gpu
REL = 2.0 ** -20 + 2048 * U


@pytest.fixture(scope="module")
def serve():
    from fp8_weight_only_w8a16_gb300 import serve
    return serve


def run(serve, x, tokens, top, ws=None, entropy=True):
    rows = x.shape[0]
    nan = float("nan")
    lp = torch.full((rows,), nan, device="cuda")
    ent = torch.full((rows,), nan, device="cuda") if entropy else None
    ids = torch.full((rows, top), -1, dtype=torch.int32, device="cuda") if top else None
    tlp = torch.full((rows, top), nan, device="cuda") if top else None
    ws = serve.new_logprobs_workspace(rows, x.shape[1], top) if ws is None else ws
    serve.token_logprobs(x, tokens, lp, ent, ids, tlp, ws)
    torch.cuda.synchronize()
    return lp, ent, ids, tlp


def check(serve, x, tokens, top, ws=None):
    lp, ent, ids, tlp = run(serve, x, tokens, top, ws)
    wlp, went, wids, wtlp, lse = logprobs64(x, tokens, top)
    span = x.double().masked_fill(torch.isinf(x), 0).abs().amax(1)

    def near(got, want, bound):
        fin = torch.isfinite(want)
        assert torch.equal(torch.isfinite(got), fin) and torch.equal(got[~fin].double(), want[~fin])
        err = torch.where(fin, (got.double() - want).abs(), 0.0)
        assert (err <= bound).all(), float((err - bound).max())

    bound = REL + 4 * U * (span + wlp.abs().nan_to_num(posinf=0))
    near(lp, wlp, bound)
    near(ent, went, (REL * (2 + went) + 2 * REL * 12 + 8 * U * 12))
    if top:
        assert torch.equal(ids.long(), wids)
        near(tlp, wtlp, (REL + 4 * U * (span + 60))[:, None] + 4 * U * wtlp.abs().nan_to_num(posinf=0))


def logits(rows, vocab, dtype, seed, ld=None, offset=0, std=3.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    ld = vocab if ld is None else ld
    store = torch.full((rows * ld + offset,), float("nan"), device="cuda", dtype=dtype)
    x = store[offset:].view(rows, ld)[:, :vocab]
    x.copy_(torch.randn(rows, vocab, generator=g, device="cuda") * std)
    tok = torch.randint(0, vocab, (rows,), generator=g, device="cuda").to(torch.int32)
    return x, tok


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,vocab,top,ld,offset", [
    (1, 154880, 5, None, 0), (1, 154880, 0, None, 0), (3, 32003, 32, None, 0), (5, 1025, 20, 1031, 1),
    (2, 1, 1, None, 0), (4, 7, 7, 9, 3), (17, 129283, 3, None, 0), (40, 4096, 1, 5000, 0),
    (700, 3001, 2, 3001, 5), (1, 40, 32, None, 7)])
def test_random_rows(serve, dtype, rows, vocab, top, ld, offset):
    x, tok = logits(rows, vocab, dtype, rows * 7 + vocab, ld, offset)
    check(serve, x, tok, top)


def test_more_rows_than_counters(serve):
    x, tok = logits(9000, 2051, torch.bfloat16, 1)
    check(serve, x, tok, 4)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,vocab,top,ld,offset", [
    (1, 154880, 0, None, 0), (1, 154880, 5, None, 3), (48, 129283, 0, 129290, 1), (3, 32003, 20, None, 7), (700, 4097, 1, None, 1),
    (5, 9, 0, 11, 2), (2, 154880, 0, None, 1)])
def test_every_logit_counts_once(serve, dtype, rows, vocab, top, ld, offset):
    """Equal logits: the terms are 1 and their sum a whole number below 2^24, both exact, so that only the
    logarithm's rounding is left (2 units): a vector that is lost or taken twice is 4 / 154880 of the sum at
    least.  Then larger logits in the row's first and last places, where vectors stick out of it: their terms
    add 2^-20 of the sum."""
    x, _ = logits(rows, vocab, dtype, 1, ld, offset)
    tok = torch.arange(rows, device="cuda").to(torch.int32) % vocab
    x.fill_(2.5)
    lp, ent, _, _ = run(serve, x, tok, top)
    want = torch.log(torch.tensor(float(vocab), dtype=torch.float64, device="cuda"))
    bound = 2 * U * 16 + 4 * U * 2.5
    assert ((lp.double() + want).abs() <= bound).all() and ((ent.double() - want).abs() <= bound).all()
    x[:, :7], x[:, -7:] = 5.0, 5.5
    lp, ent, _, _ = run(serve, x, tok, top)
    wlp, went, _, _, _ = logprobs64(x, tok, top)
    assert ((lp.double() - wlp).abs() <= bound + 2.0 ** -20).all()
    assert ((ent.double() - went).abs() <= bound + 2.0 ** -18).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("order", ["ascending", "descending", "equal", "pairs"])
def test_order_of_the_logits(serve, dtype, order):
    """Every logit beats the ones before it; or all are equal (the lowest token first)."""
    v = 20011
    x = {"ascending": torch.linspace(-20, 20, v), "descending": torch.linspace(20, -20, v),
         "equal": torch.full((v,), 1.5), "pairs": torch.randn(v).round()}[order]
    x = x.to("cuda", dtype)[None].repeat(3, 1)
    check(serve, x, torch.tensor([0, 7, v - 1], dtype=torch.int32, device="cuda"), 32)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("value", ["inf", "lowest"])
@pytest.mark.parametrize("kept", [1, 3, 5000])
def test_banned_tokens(serve, dtype, value, kept):
    x, _ = logits(4, 20011, dtype, kept)
    fill = float("-inf") if value == "inf" else torch.finfo(dtype).min
    g = torch.Generator().manual_seed(kept)
    keep = torch.stack([torch.randperm(20011, generator=g)[:kept] for _ in range(4)]).cuda()
    y = torch.full_like(x, fill).scatter(1, keep, x.gather(1, keep))
    tok = keep[:, 0].to(torch.int32)
    tok[1] = 0 if 0 not in keep[1] else 1
    check(serve, y, tok, 6) if value == "inf" else check_lowest(serve, y, tok)


def check_lowest(serve, y, tok):
    lp, ent, ids, _ = run(serve, y, tok, 3)
    wlp, went, wids, _, _ = logprobs64(y, tok, 3)
    assert torch.equal(ids.long(), wids)
    assert torch.allclose(lp.double(), wlp, rtol=2.0 ** -19, atol=2e-4)
    assert torch.allclose(ent.double(), went, rtol=0, atol=2e-3)


@pytest.mark.parametrize("top", [1, 20, 32])
@pytest.mark.parametrize("kept", [0, 5, 400])
def test_masks_in_every_place(serve, kept, top):
    """Few tokens above a value that the rest share -- -inf, the lowest, or any other --
    and the shared value's own lowest tokens behind them."""
    g = torch.Generator().manual_seed(kept + top)
    for fill in (NEG, -3.0e38, -1.0, 2.0):
        x = torch.full((3, 60013), fill)
        for r in range(3):
            at = torch.randperm(60013, generator=g)[:kept]
            x[r, at] = torch.rand(kept, generator=g) * 3 + 2.5
        x[1, :30000] = min(fill, -2.0) * 1.1 if fill > NEG else NEG  # the shared value starts late
        x = x.cuda()
        order = torch.sort(x.double(), dim=1, descending=True, stable=True).indices[:, :top]
        _, _, ids, _ = run(serve, x, torch.zeros(3, dtype=torch.int32, device="cuda"), top)
        assert torch.equal(ids.long(), order), fill


def test_lowest_value_everywhere(serve):
    """A row of the type's lowest value is a flat distribution, not an empty one."""
    for dtype in (torch.bfloat16, torch.float32):
        x = torch.full((2, 5003), torch.finfo(dtype).min, dtype=dtype, device="cuda")
        lp, ent, ids, tlp = run(serve, x, torch.zeros(2, dtype=torch.int32, device="cuda"), 4)
        flat = torch.log(torch.tensor(5003.0, dtype=torch.float64))
        assert torch.allclose(lp.double().cpu(), -flat.expand(2), atol=2e-5)
        assert torch.allclose(ent.double().cpu(), flat.expand(2), atol=2e-5)
        assert ids.tolist() == [[0, 1, 2, 3]] * 2


def test_rows_without_a_distribution(serve):
    """All -inf, +inf or NaN somewhere: NaN, and the rows beside are not touched."""
    x, tok = logits(5, 30011, torch.float32, 9)
    clean = run(serve, x.clone(), tok, 3)
    x[1] = float("-inf")
    x[2, 29000] = float("nan")
    x[3, 17] = float("inf")
    lp, ent, ids, tlp = run(serve, x, tok, 3)
    bad = torch.tensor([False, True, True, True, False], device="cuda")
    assert torch.equal(torch.isnan(lp), bad) and torch.equal(torch.isnan(ent), bad)
    assert ids[1].tolist() == [0, 1, 2]
    assert ((ids >= 0) & (ids < 30011)).all()
    for got, want in zip((lp, ent, ids, tlp), clean):
        assert torch.equal(got[~bad], want[~bad])


def test_tokens_outside_the_vocabulary(serve):
    x, _ = logits(4, 1000, torch.bfloat16, 3)
    tok = torch.tensor([-1, 1000, 2 ** 31 - 1, 5], dtype=torch.int32, device="cuda")
    lp, ent, _, _ = run(serve, x, tok, 0)
    assert torch.isnan(lp[:3]).all() and torch.isfinite(lp[3]) and torch.isfinite(ent).all()


def test_one_workspace_for_many_shapes(serve):
    """The counters stay where they are whatever the shape, and are left at zero."""
    ws = serve.new_logprobs_workspace(64, 154880, 32)
    for rows, vocab, top in ((1, 154880, 32), (64, 154880, 5), (3, 20011, 0), (64, 20011, 32), (1, 154880, 1)):
        x, tok = logits(rows, vocab, torch.bfloat16, rows + vocab)
        check(serve, x, tok, top, ws)


@pytest.mark.parametrize("most", [305, 700, 9000])
def test_a_workspace_for_many_rows_serves_fewer(serve, most):
    ws = serve.new_logprobs_workspace(most, 40000, 8)
    for rows in (1, 2, 150, 304, most):
        x, tok = logits(rows, 40000, torch.bfloat16, rows)
        check(serve, x, tok, 8, ws)


def test_same_answer_every_time_and_in_a_graph(serve):
    x, tok = logits(6, 154880, torch.bfloat16, 77)
    first = run(serve, x, tok, 20)
    for _ in range(3):
        for a, b in zip(run(serve, x, tok, 20), first):
            assert torch.equal(a, b)
    lp, ent = torch.zeros(6, device="cuda"), torch.zeros(6, device="cuda")
    ids, tlp = torch.zeros(6, 20, dtype=torch.int32, device="cuda"), torch.zeros(6, 20, device="cuda")
    ws = serve.new_logprobs_workspace(6, 154880, 20)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        serve.token_logprobs(x, tok, lp, ent, ids, tlp, ws)
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    for a, b in zip((lp, ent, ids, tlp), first):
        assert torch.equal(a, b)


def test_without_entropy(serve):
    x, tok = logits(3, 5000, torch.float32, 4)
    lp, _, _, _ = run(serve, x, tok, 0, entropy=False)
    assert torch.equal(lp, run(serve, x, tok, 2)[0])
