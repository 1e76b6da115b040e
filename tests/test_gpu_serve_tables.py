"""GPU tests of the paged bookkeeping and the latent-cache write against plain
Python and torch indexing: every value is a whole number or a copy, so all
comparisons are exact."""
from __future__ import annotations

import random

import pytest
import torch

from tests.serve_util import tables_plain

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def serve():
    from fp8_weight_only_w8a16_gb300 import serve
    return serve


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def run_tables(serve, ctx, new, page, free, head, table, toks, ld_extra=0):
    n, width = len(ctx), len(table[0])
    full = torch.full((n, width + ld_extra), -7, dtype=torch.int32, device="cuda")
    full[:, :width] = i32(table)
    t = full[:, :width]
    o = dict(seq=i32([-9] * n), cu=i32([-9] * (n + 1)), pos=i32([-9] * (toks + 1)),
             slots=torch.full((toks + 1,), -9, dtype=torch.int64, device="cuda"),
             out=i32([-9]), status=i32([-9]))
    serve.block_tables(i32(ctx), i32(new), page, i32(free), i32([head]), t, o["seq"], o["cu"],
                       o["slots"][:toks], o["pos"][:toks], o["out"], o["status"])
    torch.cuda.synchronize()
    assert int(o["slots"][toks]) == -9 and int(o["pos"][toks]) == -9
    assert (full[:, width:] == -7).all()
    return (t.tolist(), o["seq"].tolist(), o["cu"].tolist(), o["slots"][:toks].tolist(),
            o["pos"][:toks].tolist(), int(o["out"]), int(o["status"]))


def make(rng, n, page, ctx_hi, new_hi, width=None, spare=9):
    ctx = [rng.randint(0, ctx_hi) for _ in range(n)]
    new = [rng.randint(0, new_hi) for _ in range(n)]
    if width is None:
        width = max(-(-(c + k) // page) for c, k in zip(ctx, new)) + 1
    ids = list(range(100000))
    rng.shuffle(ids)
    table = [[ids.pop() if p < -(-c // page) else -5 for p in range(width)] for c in ctx]
    need = sum(-(-(c + k) // page) - -(-c // page) for c, k in zip(ctx, new))
    return ctx, new, table, [ids.pop() for _ in range(need + spare)]


@pytest.mark.parametrize("n,page,ctx_hi,new_hi", [
    (1, 16, 0, 1), (1, 64, 500, 40), (3, 1, 9, 5), (33, 48, 700, 3), (64, 64, 4000, 1),
    (200, 16, 900, 90), (1025, 32, 300, 2), (2500, 7, 60, 4)])
def test_tables_against_plain(serve, n, page, ctx_hi, new_hi):
    rng = random.Random(n * 131 + page)
    ctx, new, table, free = make(rng, n, page, ctx_hi, new_hi)
    toks = sum(new) + 3
    want = tables_plain(ctx, new, page, free, 4, table, toks)
    assert run_tables(serve, ctx, new, page, free, 4, table, toks, ld_extra=3) == want
    assert want[-1] == 0


def test_tables_most_requests(serve):
    n = serve.MAX_REQUESTS
    rng = random.Random(5)
    ctx, new = [rng.randint(0, 40) for _ in range(n)], [rng.randint(0, 2) for _ in range(n)]
    table = [[r * 3 + p for p in range(3)] for r in range(n)]
    free = [60000 + i for i in range(n)]
    want = tables_plain(ctx, new, 16, free, 0, table, sum(new))
    assert run_tables(serve, ctx, new, 16, free, 0, table, sum(new)) == want


@pytest.mark.parametrize("new", [[0, 0, 0], [0, 5, 0], [1, 0, 0]])
def test_tables_empty_requests(serve, new):
    table = [[-5] * 4 for _ in range(3)]
    want = tables_plain([0, 0, 0], new, 4, [9, 8, 7], 0, table, 6)
    assert run_tables(serve, [0, 0, 0], new, 4, [9, 8, 7], 0, table, 6) == want


def test_tables_free_list_runs_out(serve):
    table = [[-5] * 8 for _ in range(4)]
    args = ([0, 3, 0, 4], [9, 9, 2, 30], 4, [50, 51, 52, 53, 54, 55], 2, table, 50)
    args[5][1][0] = 40
    args[5][3][0] = 41
    want = tables_plain(*args)
    assert want[-1] == 3 and -1 in want[0][3]  # the last request outgrows its row too
    assert run_tables(serve, *args) == want


def test_tables_row_outgrown_takes_no_page(serve):
    table = [[-5] * 2, [-5] * 2, [3, 4]]
    args = ([0, 0, 12], [20, 3, 5], 4, [10, 11, 12, 13, 14], 0, table, 28)
    want = tables_plain(*args)
    assert want[-1] == 2 and want[5] == 3
    assert run_tables(serve, *args) == want


def test_tables_bad_lengths_are_flagged(serve):
    table = [[-5] * 4 for _ in range(3)]
    args = ([-3, 2, 0], [2, -8, 3], 4, [10, 11, 12], 0, table, 2)
    args[5][1][0] = 6
    want = tables_plain(*args)
    assert want[-1] == 4
    assert run_tables(serve, *args) == want
    # a sequence at the end of the number range: cut there, nothing wraps
    ctx, page = 2 ** 31 - 3, 1 << 20
    table = [[-5] * 4]
    got = run_tables(serve, [ctx], [10], page, [1, 2], 0, table, 4)
    assert got[1] == [2 ** 31 - 1] and got[-1] == 6 and got[3] == [-1] * 4 and got[5] == 0


@pytest.mark.parametrize("at", [0, 1, 3])
def test_tables_behind_a_sum_that_is_cut(serve, at):
    """A length that takes the sum of tokens past the number range: the requests behind it still get their
    pages written, each page that is taken off the list."""
    page, width = 1 << 20, 3
    ctx, new = [0, 5, page, page - 1, 2 * page], [3, 4, 2, page, 7]
    new[at] = 2 ** 31 - 1 - ctx[at]
    new[4] = 2 ** 31 - 1 - ctx[4] if at == 3 else new[4]
    table = [[40 + 3 * r + p if p < -(-c // page) else -5 for p in range(width)] for r, c in enumerate(ctx)]
    args = (ctx, new, page, list(range(100, 120)), 2, table, 9)
    want = list(tables_plain(*args))
    want[2] = [min(c, 2 ** 31 - 1) for c in want[2]]
    assert run_tables(serve, *args) == tuple(want)
    assert want[-1] == 6 and not any(-5 in row for r, row in enumerate(want[0]) if r == at)


def test_tables_slots_pass_32_bits(serve):
    page = 1 << 20
    got = run_tables(serve, [5], [3], page, [1], 0, [[2 ** 31 - 1, -5]], 3)
    assert got[3] == [(2 ** 31 - 1) * page + 5 + i for i in range(3)]


def test_tables_no_tokens_and_no_free_pages(serve):
    got = run_tables(serve, [4], [0], 4, [], 0, [[7, -5]], 0)
    assert got == ([[7, -5]], [4], [0, 0], [], [], 0, 0)


def test_tables_in_a_graph_and_on_a_stream(serve):
    rng = random.Random(3)
    ctx, new, table, free = make(rng, 40, 16, 300, 3)
    toks = sum(new)
    want = tables_plain(ctx, new, 16, free, 0, table, toks)
    t, c, n = i32(table), i32(ctx), i32(new)
    f, h = i32(free), i32([0])
    seq, cu, pos = i32([0] * 40), i32([0] * 41), i32([0] * toks)
    slots, out, status = torch.zeros(toks, dtype=torch.int64, device="cuda"), i32([0]), i32([9])
    side = torch.cuda.Stream()
    call = lambda: serve.block_tables(c, n, 16, f, h, t, seq, cu, slots, pos, out, status)  # noqa: E731
    with torch.cuda.stream(side):
        side.wait_stream(torch.cuda.default_stream())
        call()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            call()
        slots.zero_()
        g.replay()
    side.synchronize()
    assert slots.tolist() == want[3] and t.tolist() == want[0] and int(status) == 0


# ---------------------------------------------------------------------------
# latent-cache write
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("toks,page,row,tok_pad,page_pad", [
    (1, 16, 576, 0, 0), (7, 64, 2624, 0, 0), (129, 16, 640, 8, 64), (1000, 48, 2624, 64, 0),
    (4099, 1, 576, 0, 8)])
def test_cache_write(serve, toks, page, row, tok_pad, page_pad):
    g = torch.Generator().manual_seed(toks)
    pages = -(-toks // page) + 2
    rows = torch.randn(toks, row, generator=g).to(torch.bfloat16).cuda()
    store = torch.randn(pages, page * (576 + tok_pad) + page_pad, generator=g).to(torch.bfloat16).cuda()
    before = store.clone()
    cache = store.as_strided((pages, page, 576), (store.stride(0), 576 + tok_pad, 1))
    slots = torch.randperm(pages * page, generator=g)[:toks]
    if toks > 5:
        slots[1], slots[3], slots[5] = -1, pages * page, 1 << 40  # none of them a slot
    lat, rope = rows[:, row - 576:row - 64], rows[:, row - 64:]
    serve.latent_cache_write(lat, rope, slots.cuda(), cache)
    want = before.clone()
    view = want.as_strided(cache.shape, cache.stride())
    ok = (slots >= 0) & (slots < pages * page)
    view[slots[ok] // page, slots[ok] % page] = torch.cat([lat, rope], 1)[ok.cuda()]
    assert torch.equal(store.view(torch.int16), want.view(torch.int16))


def test_cache_write_passes_32_bits(serve):
    pages, page = 60000, 64  # 2.2e9 elements
    cache = torch.empty(pages, page, 576, dtype=torch.bfloat16, device="cuda")
    slots = torch.tensor([pages * page - 1, 0, 3750000], device="cuda")
    rows = torch.randn(3, 576, device="cuda").to(torch.bfloat16)
    serve.latent_cache_write(rows[:, :512], rows[:, 512:], slots, cache)
    assert torch.equal(cache.view(-1, 576)[slots], rows)


def test_cache_write_nothing(serve):
    cache = torch.zeros(1, 16, 576, dtype=torch.bfloat16, device="cuda")
    rows = torch.ones(4, 576, dtype=torch.bfloat16, device="cuda")
    serve.latent_cache_write(rows[:, :512], rows[:, 512:], torch.zeros(0, dtype=torch.int64, device="cuda"), cache)
    assert not cache.any()
