"""GPU tests of what the serving operators refuse when they are called as a user
calls them: a W8Error before anything is enqueued, and the outputs untouched; and of calls that
look odd and are not refused."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def serve():
    from fp8_weight_only_w8a16_gb300 import serve
    return serve


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("rows", [lambda t: t[:1].expand(8, -1), lambda t: t.as_strided((8, 10), (4, 1))])
def test_tables_whose_rows_share_storage(serve, rows):
    table = rows(torch.full((8, 10), 3, dtype=torch.int32, device="cuda"))
    out = torch.full((8, 2, 512), 7.0, dtype=BF, device="cuda")
    with pytest.raises(serve.W8Error):
        serve.latent_attn_paged(torch.zeros(8, 2, 512, dtype=BF, device="cuda"), torch.zeros(8, 2, 64, dtype=BF, device="cuda"),
                                torch.zeros(4, 16, 576, dtype=BF, device="cuda"), table, i32([160] * 8), i32(range(9)), 0.1,
                                out, None, serve.new_latent_paged_workspace(8, 2, 8))
    seq, cu, pos, slots = i32([-9] * 8), i32([-9] * 9), i32([-9] * 8), torch.full((8,), -9, device="cuda")
    head, status = i32([-9]), i32([-9])
    with pytest.raises(serve.W8Error):
        serve.block_tables(i32([0] * 8), i32([1] * 8), 16, i32(range(20)), i32([0]), table, seq, cu, slots, pos, head, status)
    torch.cuda.synchronize()
    assert (out == 7).all() and (table == 3).all()
    for t in (seq, cu, pos, slots, head, status):
        assert (t == -9).all()


def test_one_token_at_an_odd_place(serve):
    """A single token, whose axis has an odd stride, gets the answer of its copy."""
    g = torch.Generator(device="cuda").manual_seed(3)

    def odd(*shape):
        x = torch.randn(shape, generator=g, device="cuda").to(BF)
        y = torch.empty(x.numel() + 13, dtype=BF, device="cuda").as_strided(shape, (x.numel() + 13,) + x.stride()[1:])
        return x, y.copy_(x)

    lat, rope, cache = odd(1, 3, 512), odd(1, 3, 64), odd(1, 16, 576)
    q, qr, k, v, kr = odd(1, 3, 128), odd(1, 3, 64), odd(1, 3, 128), odd(1, 3, 128), odd(1, 64)
    got = []
    for i in range(2):
        out, lse = odd(1, 3, 512)[i], torch.zeros(1, 3, device="cuda")
        serve.latent_attn_paged(lat[i], rope[i], cache[i], i32([[0]]), i32([7]), i32([0, 1]), 0.1, out, lse,
                                serve.new_latent_paged_workspace(1, 3, 1))
        o2, l2 = odd(1, 3, 128)[i], torch.zeros(1, 3, device="cuda")
        serve.latent_attn_expanded(q[i], qr[i], k[i], kr[i], v[i], i32([0, 1]), i32([0, 1]), 0.1, True, o2, l2)
        got.append((out, lse, o2, l2))
    torch.cuda.synchronize()
    for a, b in zip(*got):
        assert torch.equal(a, b)
    assert torch.equal(got[0][2], v[0])  # the only key's value
