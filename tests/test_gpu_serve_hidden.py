"""GPU tests of what a query does not see inside its own request: later tokens
that hold NaN or infinities reach the queries that see them, as the definition
in 64 bits says, and leave the others' outputs within their bounds."""
from __future__ import annotations

import pytest
import torch

from tests.serve_util import attend64, lse_bound, out_bound
from tests.test_gpu_serve_attention import Paged

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
