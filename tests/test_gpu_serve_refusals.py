"""GPU tests of what the serving operators refuse when they are called as a user
calls them: a W8Error before anything is enqueued, and the outputs untouched; of calls that
look odd and are not refused; and of what the status call waits for."""
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


def test_lengths_are_not_advanced_in_place(serve):
    """Every CTA reads all lengths while the first writes the new ones."""
    n = 3000
    ctx, new, free = i32([5] * n), i32([1] * n), i32(range(9))
    table, seq, cu = torch.full((n, 2), 3, dtype=torch.int32, device="cuda"), i32([0] * n), i32([0] * (n + 1))
    slots, pos, head = torch.zeros(n, dtype=torch.int64, device="cuda"), i32([0] * n), i32([0])
    for kw in (dict(seq_lens=ctx), dict(seq_lens=new), dict(positions=ctx)):
        with pytest.raises(serve.W8Error):
            serve.block_tables(ctx, new, 16, free, head, table, **{**dict(seq_lens=seq, positions=pos), **kw}, cu_new=cu,
                               slots=slots, free_head_out=i32([0]), status=i32([0]))
    torch.cuda.synchronize()
    assert (ctx == 5).all() and (new == 1).all() and (table == 3).all()


def test_tables_buffers_side_by_side(serve):
    """Inputs and outputs cut from one buffer, none on another, also between the table's rows."""
    n, width, ld = 300, 3, 8
    lens = torch.zeros(6 * n + 20, dtype=torch.int32, device="cuda")
    at = 0

    def cut(k):
        nonlocal at
        at += k
        return lens[at - k:at]

    ctx, seq, new, cu, free, head, out, status = (cut(k) for k in (n, n, n, n + 1, n, 1, 1, 1))
    ctx.fill_(16)
    new.fill_(1)
    free.copy_(torch.arange(n))
    pos, slots = i32([0] * n), torch.zeros(n, dtype=torch.int64, device="cuda")
    table = torch.full((n, ld), -7, dtype=torch.int32, device="cuda")
    serve.block_tables(ctx, new, 16, free, head, table[:, :width], seq, cu, slots, pos, out, status)
    assert int(status) == 0 and int(out) == n and (seq == 17).all() and torch.equal(cu, torch.arange(n + 1, device="cuda").int())
    assert torch.equal(table[:, 1], torch.arange(n, device="cuda").int()) and (table[:, 2:] == -7).all()
    assert torch.equal(slots, torch.arange(n, device="cuda") * 16)
    # one request's length in the gap behind its table row
    row = torch.tensor([[-7, -7, -7, 16, -7]], dtype=torch.int32, device="cuda")
    serve.block_tables(row[0, 3:4], new[:1], 16, free, head, row[:, :3], seq[:1], cu[:2], slots[:1], pos[:1], out, status)
    assert row.tolist() == [[-7, 0, -7, 16, -7]] and int(status) == 0


@pytest.mark.parametrize("reset", [False, True])
@pytest.mark.parametrize("module", ["serve", "w8"])
def test_device_status_waits_for_every_stream(serve, module, reset):
    """A wait that gives up sets the word when its launch runs: the call waits for launches of streams that
    do not block, as torch's own do not."""
    torch.cuda.synchronize()
    done, side = torch.cuda.Event(), torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)  # some 50 ms
        done.record()
    assert not done.query()
    assert (serve if module == "serve" else serve.w8).device_status(reset=reset) == 0
    assert done.query()
