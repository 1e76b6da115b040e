"""GPU tests of what a query does not see inside its own request: later tokens
that hold NaN or infinities reach the queries that see them, as the definition
in 64 bits says, and leave the others' outputs within their bounds."""
from __future__ import annotations

import pytest
import torch

from tests.serve_util import attend64, lse_bound, out_bound
from tests.test_gpu_serve_attention import Expanded, Paged, pairs

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
BAD = [float("nan"), float("inf"), float("-inf")]


@pytest.fixture(scope="module")
def serve():
    from fp8_weight_only_w8a16_gb300 import serve
    serve.device_status(reset=True)
    yield serve
    assert serve.device_status() == 0, "a bounded wait gave up"


def check_rows(out, lse, q, k, v, scale, cols):
    """Rows [a, ..] that all see the keys k, v: NaN where the definition's sum is, else within the bounds
    (their magnitudes without the tokens that are not finite: they have no weight in a sum that is)."""
    see = torch.ones(q.shape[0], k.shape[0], dtype=torch.bool, device=q.device)
    o, l, _, _ = attend64(q, k, v, scale, see)
    held = torch.isfinite(k).all(1) & torch.isfinite(v).all(1)
    _, _, a, x = attend64(q, k[held], v[held], scale, see[:, held])
    assert torch.equal(torch.isnan(out), torch.isnan(o)) and not torch.isinf(out).any()
    assert torch.equal(torch.isnan(lse), torch.isnan(l)) and torch.equal(torch.isinf(lse), torch.isinf(l))
    fin = torch.isfinite(o)
    err, bound = (out.double() - o).abs(), out_bound(o, a, x, cols, k.shape[0])
    assert (err[fin] <= bound[fin]).all(), float((err / bound)[fin].max())
    fin = torch.isfinite(l)
    assert ((lse.double() - l).abs()[fin] <= lse_bound(l, x, cols, k.shape[0])[fin]).all()
    return int(torch.isnan(o).any(1).sum()), int((~torch.isnan(o)).all(1).sum())


@pytest.mark.parametrize("heads", [1, 3, 16, 20, 64, 100])
@pytest.mark.parametrize("lens,q_lens,page", [
    ([70, 259, 64, 130], [5, 8, 4, 2], 16), ([66, 33], [66, 33], 32), ([8111, 300, 4000], [4, 1, 7], 64),
    ([129, 200], [70, 3], 128)])
def test_paged_later_tokens_reach_no_earlier_query(serve, heads, lens, q_lens, page):
    c = Paged(lens, q_lens, heads, page, seed=heads + len(lens))
    g = torch.Generator().manual_seed(heads)
    for r, (n, q) in enumerate(zip(lens, q_lens)):
        # one of the last tokens each round: a value of the latent, at the tile halves' edges too, or of the rope key
        for back in sorted({0, q // 2, q - 1, min(q, n - 1)}):
            j = n - 1 - back
            col = [0, 255, 256, 511, 300, 540][int(torch.randint(0, 6, (1,), generator=g))]
            at = (c.table[r, j // page].long(), j % page, col)
            kept = c.cache[at].clone()
            c.cache[at] = BAD[int(torch.randint(0, 3, (1,), generator=g))]
            out, lse = c.run(serve)
            bad = fine = 0
            for s, (n2, q2) in enumerate(zip(lens, q_lens)):
                ids = c.table[s, :-(-n2 // page)].long()
                k = c.cache[ids].reshape(-1, 576)[:n2]
                for i in range(q2):
                    t, m = c.cu[s] + i, n2 - q2 + i + 1
                    rows = torch.cat([c.q_lat[t], c.q_rope[t]], 1)
                    b, f = check_rows(out[t], lse[t], rows, k[:m], k[:m, :512], c.scale, 576)
                    assert s == r and m > j or b == 0  # nobody else's row
                    bad, fine = bad + b, fine + f
            assert fine > 0 or len(lens) == 1
            c.cache[at] = kept


def test_paged_all_later_tokens_bad(serve):
    """Every draft token but the first holds nothing but NaN: the first one's output is as without them."""
    c = Paged([1000, 77], [4, 3], 16, 16, seed=5)
    want, wl = c.run(serve)
    for r, (n, q) in enumerate(zip(c.lens, [4, 3])):
        for j in range(n - q + 1, n):
            c.cache[c.table[r, j // 16].long(), j % 16] = float("nan")
    out, lse = c.run(serve)
    for t in (0, 4):
        assert torch.equal(out[t], want[t]) and torch.equal(lse[t], wl[t])
    for t in (1, 2, 3, 5, 6):
        assert torch.isnan(out[t]).all() and torch.isnan(lse[t]).all()


# ---------------------------------------------------------------------------
# expanded form
# ---------------------------------------------------------------------------

def check_head(out, lse, q, k, v, see, scale):
    """One head's rows by the definition: a value that is not finite counts for the rows that see it alone, a
    key that is not finite gives them a score of -inf (no weight) or a sum that is NaN."""
    whole = torch.isfinite(k).all(1)
    x = (q.double() @ k.double().T * scale).masked_fill(~see, float("-inf"))
    lse64 = torch.logsumexp(torch.where(see, x, float("-inf")), 1)
    nan = torch.isnan(x).any(1) | (x == float("inf")).any(1)
    lse64 = torch.where(nan, float("nan"), lse64)
    empty = torch.isneginf(lse64)
    o, l, a, big = attend64(q, torch.where(whole[:, None], k, 0.0), torch.where(torch.isfinite(v), v, 0.0), scale,
                            see & whole[None, :])
    w = torch.exp(x - torch.where(empty, 0.0, lse64)[:, None])
    for j in (~torch.isfinite(v).all(1)).nonzero()[:, 0].tolist():
        o += torch.where(see[:, j, None], w[:, j, None] * torch.where(torch.isfinite(v[j]), 0.0, v[j].double()), 0.0)
    o = torch.where(nan[:, None], float("nan"), o)
    assert torch.equal(torch.isnan(lse), nan) and torch.equal(torch.isneginf(lse), empty)
    ok = ~nan & ~empty
    assert ((lse.double() - l).abs() <= lse_bound(l, big, q.shape[1], k.shape[0]))[ok].all()
    fin = torch.isfinite(o)
    assert torch.equal(torch.isnan(out), torch.isnan(o))
    assert torch.equal(out[~fin & ~torch.isnan(o)].double(), o[~fin & ~torch.isnan(o)])
    err, bound = (out.double() - o).abs(), out_bound(o, a, big, q.shape[1], k.shape[0])
    assert (err <= bound)[fin].all(), float((err / bound)[fin].max())
    return int((~fin).any(1).sum())


EXPANDED = [([300, 65], [300, 80], 3), ([5, 129, 64], [5, 500, 64], 3), ([200, 7], [30, 0], 2),
            ([1600], [1600], 64), ([520, 1111], [520, 1400], 64)]


@pytest.mark.parametrize("nope,cols", [(192, 256), (128, 128)])
@pytest.mark.parametrize("q,k,heads", EXPANDED)
def test_expanded_later_keys_reach_no_earlier_query(serve, nope, cols, q, k, heads):
    c = Expanded(q, k, heads, nope, cols, seed=sum(q), std=0.5)
    assert pairs(serve, c) == (heads == 64)
    clean, cl = c.run(serve)
    g = torch.Generator().manual_seed(nope + heads)

    def pick(n):
        return int(torch.randint(0, n, (1,), generator=g))

    reached = 0
    for r, (n, keys) in enumerate(zip(q, k)):
        if keys == 0:
            continue
        for what in ("v", "v", "v", "k_nope", "k_rope"):
            # the request's last key, its first, any
            j = c.cu_k[r] + [keys - 1, pick(keys), pick(keys), pick(keys)][pick(4)]
            head = pick(heads)
            x = getattr(c, what)
            at = (j, pick(64)) if what == "k_rope" else (j, head, [0, x.shape[2] - 1, pick(x.shape[2])][pick(3)])
            kept = x[at].clone()
            x[at] = BAD[pick(3)]
            out, lse = c.run(serve)
            a, b, d, e = c.cu_q[r], c.cu_q[r + 1], c.cu_k[r], c.cu_k[r + 1]
            see = torch.arange(keys, device="cuda")[None, :] <= keys - n + torch.arange(n, device="cuda")[:, None]
            for h in range(heads):
                if what == "k_rope" and h % 16 in (0, 15) or h == head:
                    reached += check_head(out[a:b, h], lse[a:b, h], torch.cat([c.q_nope[a:b, h], c.q_rope[a:b, h]], 1),
                                          torch.cat([c.k_nope[d:e, h], c.k_rope[d:e]], 1), c.v[d:e, h], see, c.scale)
            others = [h for h in range(heads) if h != head] if what != "k_rope" else []
            assert torch.equal(out[:, others], clean[:, others]) and torch.equal(lse[:, others], cl[:, others])
            assert torch.equal(out[:a], clean[:a]) and torch.equal(out[b:], clean[b:])
            x[at] = kept
    assert reached > 0
    out, lse = c.run(serve)
    assert torch.equal(out, clean) and torch.equal(lse, cl)


@pytest.mark.parametrize("nope,cols", [(192, 256), (128, 128)])
@pytest.mark.parametrize("n,heads", [(300, 3), (1600, 64)])
def test_expanded_all_later_keys_bad(serve, nope, cols, n, heads):
    """Every key from one on holds nothing but NaN: the queries before it get what they get of the keys before it."""
    c = Expanded([n], [n], heads, nope, cols, seed=n)
    want, wl = c.run(serve)
    at = n // 2 + 3
    c.k_nope[at:], c.k_rope[at:], c.v[at:] = float("nan"), float("nan"), float("nan")
    out, lse = c.run(serve)
    assert torch.isnan(out[at:]).all() and torch.isnan(lse[at:]).all()
    assert torch.equal(lse[:at], wl[:at]) and torch.isfinite(out[:at]).all()
    for h in (0, heads - 1):
        q = torch.cat([c.q_nope[:at, h], c.q_rope[:at, h]], 1)
        k = torch.cat([c.k_nope[:at, h], c.k_rope[:at]], 1)
        see = torch.ones(at, at, dtype=torch.bool, device="cuda").tril()
        assert check_head(out[:at, h], lse[:at, h], q, k, c.v[:at, h], see, c.scale) == 0
