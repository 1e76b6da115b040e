"""GPU tests of the adapters where they have rows enough for tiles of 128 positions: a
NaN in a row, rows and offsets out of range, offsets that change under replay (and with
them the tiles and the ranges of k), the same bits every time.  Both first products: by
tiles of 128 where rank x k is large, by tiles of 16 where it is small."""
from __future__ import annotations

import pytest
import torch

from .grouped_util import BF, check, cuda_gen, groups_of, i32
from .test_gpu_lora import buffer, lora64

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")

# rank, k: rank x k (the rank up to 64 or 128) from 131072 takes the first product by tiles of 128
ROUTES = [(64, 4096), (64, 512), (104, 2048), (128, 520), (40, 4100)]


@pytest.fixture(scope="module")
def grouped():
    from fp8_weight_only_w8a16_gb300 import grouped
    yield grouped
    assert grouped.device_status() == 0


class Call:
    def __init__(self, grouped, rank, k, toks=600, n=264, adapters=4, seed=1):
        g = cuda_gen(seed)
        self.grouped, self.gen, self.toks = grouped, g, toks
        self.x, self.y = buffer((toks, k), -k % 8, g), buffer((toks, n), 8, g)
        self.a, self.b = buffer((adapters, rank, k), -k % 8, g, 0.1), buffer((adapters, n, rank), -rank % 8, g, 0.3)
        self.order = torch.randperm(toks, generator=g, device="cuda").to(torch.int32)
        self.scales = torch.randn(adapters, generator=g, device="cuda")
        self.ws = grouped.new_lora_workspace(toks, k, rank, adapters)
        self.ws.fill_(0xFF)  # NaN

    def run(self, offsets, x=None, order=None, out=None):
        out = torch.full_like(self.y, 7.0) if out is None else out
        return self.grouped.lora_add(self.x if x is None else x, self.a, self.b, self.order if order is None else order, offsets, self.y, out,
                                     self.ws, scales=self.scales)

    def compare(self, out, offsets, order=None):
        """Named rows within their bounds, the others as they were."""
        order = self.order if order is None else order
        want, bound = lora64(self.x, self.a, self.b, order, offsets, self.y, None, self.scales)
        at = offsets.tolist()
        named = order[at[0]:at[-1]].long()
        named = named[(named >= 0) & (named < self.toks)]
        check(out[named], want[named], bound[named])
        rest = torch.ones(self.toks, dtype=torch.bool, device="cuda")
        rest[named] = False
        assert (out[rest] == 7).all()


@pytest.mark.parametrize("rank,k", ROUTES)
def test_a_row_that_is_not_finite_stays_alone(grouped, rank, k):
    c = Call(grouped, rank, k)
    offsets = groups_of([300, 0, 170, 130])
    clean = c.run(offsets)
    c.compare(clean, offsets)
    rows = [9, 200, 599]
    bad = torch.empty_strided(c.x.shape, c.x.stride(), dtype=BF, device="cuda").copy_(c.x)
    bad[9, 100], bad[200, k - 1], bad[599, 0] = NAN, INF, -INF
    keep = torch.ones(c.toks, dtype=torch.bool, device="cuda")
    keep[rows] = False
    for _ in range(3):
        out = c.run(offsets, x=bad)
        assert torch.equal(out[keep], clean[keep])
        assert torch.isnan(out[9]).all() and not torch.isfinite(out[rows]).any()
    # what the tiles' places held before reaches nothing: the next calls are clean again
    assert torch.equal(c.run(offsets), clean)
    order = c.order.clone()
    order[::3] = -1
    out = c.run(offsets, order=order)
    left = order[order >= 0].long()
    assert torch.equal(out[left], clean[left])


@pytest.mark.parametrize("rank,k", ROUTES)
def test_rows_and_offsets_out_of_range(grouped, rank, k):
    c = Call(grouped, rank, k)
    order = c.order.clone()
    order[[0, 5, 127, 128, 299, 300, 599]] = i32([-1, c.toks, 2 ** 31 - 1, -2 ** 31, -7, c.toks + 3, -1])
    offsets = groups_of([300, 0, 170, 130])
    c.compare(c.run(offsets, order=order), offsets, order)
    for wild in ([-5, 200, 100, 450, 10000], [40, 40, 600, 3, -1], [600, 0, 5, 7, 600], [0, 0, 0, 0, 0], [100, 2 ** 31 - 1, 0, -2 ** 31, 9]):
        cut = [min(max(v, 0), c.toks) for v in wild]
        for i in range(1, 5):
            cut[i] = max(cut[i], cut[i - 1])
        c.compare(c.run(i32(wild), order=order), i32(cut), order)


@pytest.mark.parametrize("rank,k", ROUTES)
def test_offsets_that_change_under_replay(grouped, rank, k):
    c = Call(grouped, rank, k)
    offsets, out = groups_of([300, 0, 170, 130]), torch.full_like(c.y, 7.0)
    c.run(offsets)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(offsets, out=out)
        c.run(offsets, out=out)  # one after the other on one workspace
    for counts in ([600, 0, 0, 0], [1, 1, 1, 1], [0, 0, 0, 0], [129, 127, 128, 216], [0, 0, 0, 600], [150, 150, 150, 150], [0, 5, 0, 0]):
        offsets.copy_(groups_of(counts))
        c.x.copy_(torch.randn(c.x.shape, generator=c.gen, device="cuda"))
        c.order.copy_(torch.randperm(c.toks, generator=c.gen, device="cuda"))
        out.fill_(7.0)
        graph.replay()
        c.compare(out, groups_of(counts))
        again = out.clone()
        graph.replay()
        assert torch.equal(out, again)


@pytest.mark.parametrize("rank,k", ROUTES)
def test_many_times_the_same_bits(grouped, rank, k):
    c = Call(grouped, rank, k, toks=1500, n=1000, adapters=6, seed=3)
    offsets = groups_of([300, 0, 470, 130, 599, 1])
    first = c.run(offsets)
    c.compare(first, offsets)
    for _ in range(25):
        assert torch.equal(c.run(offsets), first)


@pytest.mark.parametrize("rank,k,toks", [(64, 4096, 600), (64, 512, 600), (128, 520, 600), (64, 512, 40), (16, 512, 600)])
def test_weights_that_are_not_finite_stay_in_their_places(grouped, rank, k, toks):
    """A NaN or an infinity in a row of B reaches that column of its adapter's rows, one in A all of the adapter's columns."""
    c = Call(grouped, rank, k, toks=toks)
    offsets = groups_of([toks // 2, 0, toks // 4, toks - toks // 2 - toks // 4])
    clean = c.run(offsets)
    c.compare(clean, offsets)
    mine = c.order[toks // 2:toks // 2 + toks // 4].long()
    others = torch.ones(toks, dtype=torch.bool, device="cuda")
    others[mine] = False
    columns = torch.ones(264, dtype=torch.bool, device="cuda")
    columns[[17, 263]] = False
    old = c.b[2, [17, 263], 3].clone()
    c.b[2, 17, 3], c.b[2, 263, 3] = INF, NAN
    out = c.run(offsets)
    assert torch.equal(out[others], clean[others]) and torch.equal(out[mine][:, columns], clean[mine][:, columns])
    assert not torch.isfinite(out[mine][:, ~columns]).any()
    c.b[2, [17, 263], 3] = old
    c.a[2, 5, k - 1] = NAN
    out = c.run(offsets)
    assert torch.equal(out[others], clean[others]) and torch.isnan(out[mine]).all()
