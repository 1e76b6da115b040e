"""GPU tests of latent attention, both forms, against 64-bit plain forms; the
bounds are derived in serve_util.py from the arithmetic that the header
states."""
from __future__ import annotations

import pytest
import torch

from tests.serve_util import NEG, check_attention, expanded64, paged64

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def serve():
    from fp8_weight_only_w8a16_gb300 import serve
    serve.device_status(reset=True)
    yield serve
    assert serve.device_status() == 0, "a bounded wait gave up"


def cu_of(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------------------
# absorbed form over the paged cache
# ---------------------------------------------------------------------------

class Paged:
    def __init__(self, lens, q_lens, heads, page, seed=0, spare=3, tok_pad=0, page_pad=0, q_pad=0, dirty=True):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.lens, self.cu, self.heads, self.page = lens, cu_of(q_lens), heads, page
        t, n = self.cu[-1], len(lens)
        counts = [-(-x // page) for x in lens]
        pages = sum(counts) + spare
        width = max(1, max(counts))
        perm = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).tolist()
        self.table = torch.full((n, width), 10 ** 6, dtype=torch.int32)  # unused entries are no page
        for r, c in enumerate(counts):
            self.table[r, :c] = torch.tensor([perm.pop() for _ in range(c)], dtype=torch.int32)
        store = torch.randn(pages, page * (576 + tok_pad) + page_pad, generator=g, device="cuda").to(BF)
        self.cache = store.as_strided((pages, page, 576), (store.stride(0), 576 + tok_pad, 1))
        if dirty:  # rows that no request holds: whatever was there before
            used = torch.zeros(pages, page, dtype=torch.bool)
            for r, x in enumerate(lens):
                for p in range(counts[r]):
                    used[self.table[r, p], :min(page, x - p * page)] = True
            bad = torch.tensor([float("nan"), float("inf"), NEG], device="cuda").to(BF)
            self.cache[~used.cuda()] = bad.repeat(192)[None]
        self.table = self.table.cuda()
        self.q_lat = torch.randn(max(t, 1), heads, 512 + q_pad, generator=g, device="cuda").to(BF)[:t, :, :512]
        self.q_rope = torch.randn(max(t, 1), heads, 256 + q_pad, generator=g, device="cuda").to(BF)[:t, :, 192:256]
        self.scale = 1.0 / 16

    def run(self, serve, ws=None, lse=True):
        t = self.cu[-1]
        out = torch.full((t, self.heads, 512), 7.0, dtype=BF, device="cuda")
        l = torch.full((t, self.heads), 7.0, device="cuda") if lse else None
        ws = serve.new_latent_paged_workspace(t, self.heads, len(self.lens)) if ws is None else ws
        serve.latent_attn_paged(self.q_lat, self.q_rope, self.cache, self.table, i32(self.lens), i32(self.cu),
                                self.scale, out, l, ws)
        torch.cuda.synchronize()
        return out, l

    def check(self, serve, **kw):
        out, lse = self.run(serve, **kw)
        clean = torch.where(torch.isfinite(self.cache), self.cache, 0.0)
        want = paged64(self.q_lat, self.q_rope, clean, self.table.clamp(0, self.cache.shape[0] - 1), self.lens,
                       self.cu, self.scale)
        check_attention(out, lse, want, 576, max(self.lens + [1]))
        return out, lse


@pytest.mark.parametrize("heads", [1, 8, 16, 20, 64, 100, 128])
@pytest.mark.parametrize("page", [16, 64, 128])
def test_paged_ragged(serve, heads, page):
    lens = [1, 0, 63, 64, 65, 127, 128, 129, 300, 1000, 2, 16, 17]
    Paged(lens, [1] * 13, heads, page, seed=heads + page).check(serve)


@pytest.mark.parametrize("q_lens", [[1, 2, 3, 4], [0, 5, 0, 8], [33, 1, 0, 7], [4, 4, 4, 4]])
@pytest.mark.parametrize("heads", [3, 16, 64])
def test_paged_several_tokens(serve, q_lens, heads):
    lens = [max(q, n) for q, n in zip(q_lens, [70, 259, 1, 64])]
    Paged(lens, q_lens, heads, 32, seed=heads).check(serve)


def test_paged_queries_before_the_first_key(serve):
    """More query tokens than cached ones: the first see nothing."""
    c = Paged([3, 0, 66], [5, 4, 70], 16, 16, seed=2)
    out, lse = c.check(serve)
    assert not out[:2].any() and torch.isneginf(lse[:2]).all()
    assert not out[5:9].any() and torch.isneginf(lse[5:9]).all()


@pytest.mark.parametrize("lens", [[1], [31], [5000], [20011], [40000, 7], [9000, 1, 12000]])
@pytest.mark.parametrize("heads", [16, 64])
def test_paged_long_contexts_are_split(serve, lens, heads):
    Paged(lens, [1] * len(lens), heads, 64, seed=len(lens)).check(serve)


@pytest.mark.parametrize("lens,q_lens", [
    ([40000], [1]), ([20011, 7], [1, 1]), ([9000, 1, 12000], [1, 1, 1]), ([64 * 152 + 1], [1]), ([30011, 640], [2, 3]),
    ([1 + 997 * i % 5000 for i in range(150)], [1] * 150)])
@pytest.mark.parametrize("heads", [16, 20, 64])
def test_paged_every_token_counts_once(serve, lens, q_lens, heads):
    """Queries of zeros weigh every token alike, and a token's value says which tile it lies in: the weights
    (1), their sums (whole numbers below 2^24) and so O and z are exact.  Left are the logarithm and its
    product, 2^-21 + 2^-22 of the log-sum, and the quotient's rounding to bf16, 2^-8 of it: a token that is
    lost or taken twice is 1 / 40000 of z, a tile the whole of its column."""
    c = Paged(lens, q_lens, heads, 64, seed=len(lens))
    c.q_lat, c.q_rope = torch.zeros_like(c.q_lat), torch.zeros_like(c.q_rope)
    for r, n in enumerate(lens):
        j = torch.arange(n, device="cuda")
        rows = torch.zeros(n, 576, dtype=BF, device="cuda")
        rows[j, j // 64 % 512] = 1
        c.cache[c.table[r, j // 64].long(), j % 64] = rows
    out, lse = c.run(serve)
    for r, (n, q) in enumerate(zip(lens, q_lens)):
        for i in range(q):
            t, m = c.cu[r] + i, n - q + i + 1
            want = torch.log(torch.tensor(float(m), dtype=torch.float64))
            assert (lse[t].double().cpu() - want).abs().max() <= 2.0 ** -21 + 2.0 ** -22 * want
            share = torch.bincount(torch.arange(m, device="cuda") // 64 % 512, minlength=512).double() / m
            assert ((out[t].double() - share).abs() <= 2.0 ** -8 * (1 + 2.0 ** -7) * share).all()


def test_paged_many_requests(serve):
    g = torch.Generator().manual_seed(1)
    lens = torch.randint(0, 200, (700,), generator=g).tolist()
    Paged(lens, [1] * 700, 8, 16, seed=5).check(serve)


@pytest.mark.parametrize("n", [1, 2, 3, 37, 75, 76, 77, 151, 152, 153, 305])
@pytest.mark.parametrize("heads", [16, 64])
def test_paged_cuts_of_the_work(serve, n, heads):
    """One-tile requests from fewer than there are SMs to more, with and without a long one among
    them: cuts fall on a request's begin, beside it and inside it, and some SMs have no work."""
    for long in (None, 0, n // 2, n - 1):
        lens = [1 + (17 * i) % 64 for i in range(n)]
        if long is not None:
            lens[long] = 2500
        q_lens = [1 + (i % 5 == 4) for i in range(n)]
        Paged([max(a, b) for a, b in zip(lens, q_lens)], q_lens, heads, 16, seed=n).check(serve)


@pytest.mark.parametrize("page", [16, 256, 1024])
def test_paged_strides(serve, page):
    Paged([200, 77, 1030], [1, 2, 1], 20, page, seed=page, tok_pad=64, page_pad=8 * 13, q_pad=8).check(serve)


def test_paged_strided_outputs_and_no_lse(serve):
    c = Paged([100, 300], [1, 1], 6, 16, seed=4)
    want, _ = c.run(serve)
    store = torch.full((2, 6, 520), 3.0, dtype=BF, device="cuda")
    ws = serve.new_latent_paged_workspace(2, 6, 2)
    serve.latent_attn_paged(c.q_lat, c.q_rope, c.cache, c.table, i32(c.lens), i32(c.cu), c.scale,
                            store[:, :, 4:516], None, ws)
    assert torch.equal(store[:, :, 4:516], want)
    assert (store[:, :, :4] == 3).all() and (store[:, :, 516:] == 3).all()


def test_paged_tokens_that_no_request_holds(serve):
    c = Paged([40, 90], [2, 1], 4, 16, seed=6)
    want, wl = c.run(serve)
    t = 6
    ql = torch.zeros(t, 4, 512, dtype=BF, device="cuda")
    qr = torch.zeros(t, 4, 64, dtype=BF, device="cuda")
    ql[1:4], qr[1:4] = c.q_lat, c.q_rope
    out, lse = torch.full((t, 4, 512), 7.0, dtype=BF, device="cuda"), torch.full((t, 4), 7.0, device="cuda")
    ws = serve.new_latent_paged_workspace(t, 4, 2)
    serve.latent_attn_paged(ql, qr, c.cache, c.table, i32(c.lens), i32([1, 3, 4]), c.scale, out, lse, ws)
    assert torch.equal(out[1:4], want) and torch.equal(lse[1:4], wl)
    assert (out[0] == 7).all() and (out[4:] == 7).all() and (lse[0] == 7).all() and (lse[4:] == 7).all()


def test_paged_lengths_are_cut_to_the_table(serve):
    """A length past the table's width, a negative one and offsets past the tokens stay inside the buffers."""
    c = Paged([64, 48], [1, 1], 4, 16, seed=7, dirty=False)
    want, wl = c.run(serve)
    out, lse = torch.zeros(2, 4, 512, dtype=BF, device="cuda"), torch.zeros(2, 4, device="cuda")
    ws = serve.new_latent_paged_workspace(2, 4, 2)
    serve.latent_attn_paged(c.q_lat, c.q_rope, c.cache, c.table, i32([2 ** 31 - 1, -5]), i32([0, 1, 2 ** 31 - 1]),
                            c.scale, out, lse, ws)
    assert torch.equal(out[0], want[0]) and torch.equal(lse[0], wl[0])
    assert not out[1].any() and torch.isneginf(lse[1]).all()


def test_paged_a_page_outside_the_cache_reads_as_zeros(serve):
    c = Paged([40], [1], 4, 16, seed=8, dirty=False)
    for bad in (-1, c.cache.shape[0], 2 ** 31 - 1, -2 ** 31):
        c.table[0, 1] = bad
        out, lse = c.run(serve)
        k = c.cache.clone()
        k[c.table[0, 0].item()], ids = k[c.table[0, 0].item()], c.table.clone()
        zero = torch.cat([c.cache, torch.zeros_like(c.cache[:1])])
        ids[0, 1] = zero.shape[0] - 1
        check_attention(out, lse, paged64(c.q_lat, c.q_rope, zero, ids, c.lens, c.cu, c.scale), 576, 40)


@pytest.mark.parametrize("scale,std", [(1.0, 1.0), (1e-4, 1.0), (0.0625, 30.0)])
def test_paged_peaked_and_flat_weights(serve, scale, std):
    """Scores that spread over thousands, and scores that are all but equal."""
    c = Paged([1500, 333], [1, 2], 16, 64, seed=9)
    c.scale = scale
    c.q_lat = (c.q_lat * std).to(BF)
    c.check(serve)


def test_paged_rising_scores(serve):
    """Every tile's maximum is above the last one's: the running maximum is raised all along."""
    c = Paged([3000], [1], 16, 64, seed=10)
    j = torch.arange(3000, device="cuda")
    c.cache[c.table[0, (j // 64).long()].long(), j % 64, 0] = (j.float() / 8).to(BF)
    c.q_lat[:, :, 0] = 4.0
    c.check(serve)
    c.cache[c.table[0, (j // 64).long()].long(), j % 64, 0] = ((3000 - j).float() / 8).to(BF)
    c.check(serve)


def test_paged_visible_nan_reaches_its_request_only(serve):
    c = Paged([100, 100, 100], [1, 1, 1], 8, 16, seed=11)
    want, wl = c.run(serve)
    c.cache[c.table[1, 2].long(), 3, 5] = float("nan")
    out, lse = c.run(serve)
    assert torch.isnan(out[1]).any() and torch.isnan(lse[1]).all()
    for i in (0, 2):
        assert torch.equal(out[i], want[i]) and torch.equal(lse[i], wl[i])


def test_paged_offsets_pass_32_bits(serve):
    pages, page = 60000, 64  # 2.2e9 elements, 4.4e9 bytes
    c = Paged([130, 64], [1, 1], 16, page, seed=12, dirty=False)
    big = torch.empty(pages, page, 576, dtype=BF, device="cuda")
    far = torch.tensor([59999, 58000, 3, 0, 59998, 41, 7], device="cuda")[:c.cache.shape[0]]
    big[far] = c.cache
    want, wl = c.run(serve)
    c.cache, c.table = big, torch.where(c.table < 100, far[c.table.long().clamp(0, far.numel() - 1)].int(), c.table)
    out, lse = c.run(serve)
    assert torch.equal(out, want) and torch.equal(lse, wl)


def test_paged_same_answer_every_time(serve):
    """Also with one workspace for other shapes in between, and from a graph on another stream."""
    c = Paged([7000, 130, 0, 2500], [1, 3, 1, 2], 64, 64, seed=13)
    ws = serve.new_latent_paged_workspace(16, 128, 16)
    first, fl = c.check(serve, ws=ws)
    other = Paged([5000, 6000, 900], [1, 1, 4], 16, 16, seed=14)
    for _ in range(3):
        other.check(serve, ws=ws)
        out, lse = c.run(serve, ws=ws)
        assert torch.equal(out, first) and torch.equal(lse, fl)
    out, lse = torch.zeros_like(first), torch.zeros_like(fl)
    lens, cu, side = i32(c.lens), i32(c.cu), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        serve.latent_attn_paged(c.q_lat, c.q_rope, c.cache, c.table, lens, cu, c.scale, out, lse, ws)
    for _ in range(2):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first) and torch.equal(lse, fl)


def test_paged_lengths_that_change_between_replays(serve):
    """A captured step reads the lengths of the replay, not of the capture."""
    c = Paged([4000, 900], [1, 1], 16, 64, seed=15, dirty=False)
    out, lse = torch.zeros(2, 16, 512, dtype=BF, device="cuda"), torch.zeros(2, 16, device="cuda")
    ws, lens, cu = serve.new_latent_paged_workspace(2, 16, 2), i32(c.lens), i32(c.cu)
    c.run(serve)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        serve.latent_attn_paged(c.q_lat, c.q_rope, c.cache, c.table, lens, cu, c.scale, out, lse, ws)
    for new in ([4000, 900], [17, 899], [0, 1], [3999, 64]):
        lens.copy_(i32(new))
        g.replay()
        torch.cuda.synchronize()
        check_attention(out, lse, paged64(c.q_lat, c.q_rope, c.cache, c.table, new, c.cu, c.scale), 576, 4000)


# ---------------------------------------------------------------------------
# expanded form
# ---------------------------------------------------------------------------

class Expanded:
    def __init__(self, q_lens, k_lens, heads, nope, v, seed=0, causal=True, extra=0, std=1.0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.cu_q, self.cu_k, self.causal, self.heads = cu_of(q_lens), cu_of(k_lens), causal, heads
        self.nope, self.v_cols, self.scale = nope, v, 1.5 / (nope + 64) ** 0.5
        tq, tk = self.cu_q[-1], self.cu_k[-1]

        def normal(*shape):
            return (torch.randn(*shape, generator=g, device="cuda") * std).to(BF)

        q = normal(max(tq, 1), heads, nope + 64 + extra)[:tq]
        kv = normal(max(tk, 1), heads, nope + v + extra)[:tk]
        self.q_nope, self.q_rope = q[:, :, :nope], q[:, :, nope:nope + 64]
        self.k_nope, self.v = kv[:, :, :nope], kv[:, :, nope:nope + v]
        self.k_rope = normal(max(tk, 1), 64 + extra)[:tk, :64]

    def run(self, serve, lse=True, cu_q=None, cu_k=None):
        t = self.q_nope.shape[0]
        out = torch.full((t, self.heads, self.v_cols), 7.0, dtype=BF, device="cuda")
        l = torch.full((t, self.heads), 7.0, device="cuda") if lse else None
        serve.latent_attn_expanded(self.q_nope, self.q_rope, self.k_nope, self.k_rope, self.v,
                                   i32(cu_q or self.cu_q), i32(cu_k or self.cu_k), self.scale, self.causal, out, l)
        torch.cuda.synchronize()
        return out, l

    def check(self, serve):
        out, lse = self.run(serve)
        want = expanded64(self.q_nope, self.q_rope, self.k_nope, self.k_rope, self.v, self.cu_q, self.cu_k,
                          self.scale, self.causal)
        longest = max([b - a for a, b in zip(self.cu_k, self.cu_k[1:])] + [1])
        check_attention(out, lse, want, self.nope + 64, longest)
        return out, lse


DIMS = [(192, 256), (128, 128)]


@pytest.mark.parametrize("nope,v", DIMS)
@pytest.mark.parametrize("n", [1, 2, 63, 64, 65, 127, 128, 129, 255, 257, 400])
def test_expanded_one_prompt(serve, nope, v, n):
    Expanded([n], [n], 3, nope, v, seed=n).check(serve)


@pytest.mark.parametrize("nope,v", DIMS)
@pytest.mark.parametrize("causal", [True, False])
def test_expanded_ragged(serve, nope, v, causal):
    q = [5, 0, 130, 1, 64, 200, 33]
    k = [5, 9, 131, 300, 64, 517, 33]
    Expanded(q, k, 5, nope, v, seed=3, causal=causal, extra=8).check(serve)


@pytest.mark.parametrize("nope,v", DIMS)
def test_expanded_queries_that_see_nothing(serve, nope, v):
    """Fewer keys than queries, and no keys at all."""
    c = Expanded([200, 7, 140], [30, 0, 139], 2, nope, v, seed=4)
    out, lse = c.check(serve)
    assert not out[:170].any() and torch.isneginf(lse[:170]).all()
    assert not out[200:207].any() and torch.isneginf(lse[200:207]).all()
    c = Expanded([9], [0], 2, nope, v, seed=5)
    out, lse = c.run(serve)
    assert not out.any() and torch.isneginf(lse).all()


@pytest.mark.parametrize("nope,v", DIMS)
def test_expanded_chunk_of_a_longer_prompt(serve, nope, v):
    Expanded([129, 40], [1700, 1064], 4, nope, v, seed=6).check(serve)


def pairs(serve, c):
    """Whether the case is long enough for the kernel of CTA pairs."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    n_q, n_req = c.cu_q[-1], len(c.cu_q) - 1
    return n_q * c.heads >= 5 * 128 * sms and n_q // n_req >= 512


@pytest.mark.parametrize("nope,v", DIMS)
@pytest.mark.parametrize("q,k,causal", [
    ([1600], [1600], True), ([1537], [1700], True), ([520, 1111], [520, 1400], True),
    ([1, 1900, 0], [200, 1900, 64], True), ([1543], [130], True), ([1550], [1551], False)])
def test_expanded_long_prompts(serve, nope, v, q, k, causal):
    """The kernel of CTA pairs: several items a pair, ragged ends, queries that see nothing."""
    c = Expanded(q, k, 64, nope, v, seed=sum(q), causal=causal)
    assert pairs(serve, c)
    first, fl = c.check(serve)
    for _ in range(3):
        out, lse = c.run(serve)
        assert torch.equal(out, first) and torch.equal(lse, fl)


@pytest.mark.parametrize("nope,v", DIMS)
def test_expanded_long_prompts_beside_anything(serve, nope, v):
    """Other requests' keys may hold anything, rows past a request's queries are not touched, peaks rise all along."""
    c = Expanded([1100, 530], [1100, 530], 64, nope, v, seed=21, extra=8)
    assert pairs(serve, c)
    c.k_rope[:, 0] = torch.arange(1630, device="cuda") / 8
    c.q_rope[:, :, 0] = 4.0
    want, wl = c.check(serve)
    bad = torch.tensor([float("nan"), float("inf"), NEG], device="cuda").to(BF)
    c.k_nope[1100:], c.v[1100:] = bad.repeat(nope)[:nope], bad.repeat(v)[:v]
    out, lse = c.run(serve)
    assert torch.equal(out[:1100], want[:1100]) and torch.equal(lse[:1100], wl[:1100])
    assert torch.isnan(out[1100:]).any()
    c = Expanded([1630], [1630], 64, nope, v, seed=22)
    want, wl = c.run(serve)
    store = torch.full((1630, 64, v + 24), 3.0, dtype=BF, device="cuda")
    serve.latent_attn_expanded(c.q_nope, c.q_rope, c.k_nope, c.k_rope, c.v, i32(c.cu_q), i32(c.cu_k), c.scale, True,
                               store[:, :, 8:8 + v], None)
    assert torch.equal(store[:, :, 8:8 + v], want)
    assert (store[:, :, :8] == 3).all() and (store[:, :, 8 + v:] == 3).all()
    # a graph replayed behind other work of the stream
    out, lse = torch.zeros_like(want), torch.zeros_like(wl)
    cq, ck = i32(c.cu_q), i32(c.cu_k)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(3):
            serve.latent_attn_expanded(c.q_nope, c.q_rope, c.k_nope, c.k_rope, c.v, cq, ck, c.scale, True, out, lse)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, wl)


@pytest.mark.parametrize("nope,v", DIMS)
def test_expanded_many_heads(serve, nope, v):
    Expanded([300, 65], [300, 80], 64, nope, v, seed=7).check(serve)


def test_expanded_many_requests(serve):
    g = torch.Generator().manual_seed(2)
    q = torch.randint(0, 9, (300,), generator=g).tolist()
    k = [a + b for a, b in zip(q, torch.randint(0, 90, (300,), generator=g).tolist())]
    Expanded(q, k, 2, 128, 128, seed=8).check(serve)


@pytest.mark.parametrize("nope,v", DIMS)
@pytest.mark.parametrize("std", [0.01, 6.0])
def test_expanded_peaked_and_flat_weights(serve, nope, v, std):
    Expanded([333], [333], 4, nope, v, seed=9, std=std).check(serve)


@pytest.mark.parametrize("nope,v", DIMS)
def test_expanded_rising_scores(serve, nope, v):
    c = Expanded([700], [700], 2, nope, v, seed=10)
    c.k_rope[:, 0] = torch.arange(700, device="cuda") / 4
    c.q_rope[:, :, 0] = 8.0
    c.check(serve)


@pytest.mark.parametrize("nope,v", DIMS)
def test_expanded_other_requests_may_hold_anything(serve, nope, v):
    c = Expanded([100, 50, 30], [100, 70, 30], 3, nope, v, seed=11)
    want, wl = c.run(serve)
    a, b = c.cu_k[1:3]
    bad = torch.tensor([float("nan"), float("inf"), NEG], device="cuda").to(BF)
    c.k_nope[a:b] = bad.repeat(nope)[:nope]
    c.v[a:b] = bad.repeat(v)[:v]
    c.k_rope[a:b] = bad.repeat(64)[:64]
    out, lse = c.run(serve)
    for lo, hi in ((0, 100), (150, 180)):
        assert torch.equal(out[lo:hi], want[lo:hi]) and torch.equal(lse[lo:hi], wl[lo:hi])
    assert torch.isnan(out[100:150]).any()


@pytest.mark.parametrize("nope,v", DIMS)
def test_expanded_strided_output(serve, nope, v):
    c = Expanded([140, 3], [150, 3], 3, nope, v, seed=12)
    want, wl = c.run(serve)
    store = torch.full((143, 3, v + 24), 3.0, dtype=BF, device="cuda")
    serve.latent_attn_expanded(c.q_nope, c.q_rope, c.k_nope, c.k_rope, c.v, i32(c.cu_q), i32(c.cu_k), c.scale, True,
                               store[:, :, 8:8 + v], None)
    assert torch.equal(store[:, :, 8:8 + v], want)
    assert (store[:, :, :8] == 3).all() and (store[:, :, 8 + v:] == 3).all()


@pytest.mark.parametrize("nope,v", DIMS)
def test_expanded_offsets_are_cut(serve, nope, v):
    """Offsets past the tokens stay inside the buffers; tokens that no request holds are not written."""
    c = Expanded([60, 70], [60, 70], 2, nope, v, seed=13)
    want, wl = c.run(serve)
    out, lse = c.run(serve, cu_q=[0, 60, 2 ** 31 - 1], cu_k=[0, 60, 2 ** 31 - 1])
    assert torch.equal(out, want) and torch.equal(lse, wl)
    out, lse = c.run(serve, cu_q=[60, 130], cu_k=[60, 130])
    assert torch.equal(out[60:], want[60:]) and torch.equal(lse[60:], wl[60:])
    assert (out[:60] == 7).all() and (lse[:60] == 7).all()


@pytest.mark.parametrize("nope,v", DIMS)
def test_expanded_same_answer_every_time(serve, nope, v):
    c = Expanded([500, 129], [700, 129], 8, nope, v, seed=14)
    first, fl = c.run(serve)
    for _ in range(5):
        out, lse = c.run(serve)
        assert torch.equal(out, first) and torch.equal(lse, fl)
    out, lse, cq, ck = torch.zeros_like(first), torch.zeros_like(fl), i32(c.cu_q), i32(c.cu_k)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        serve.latent_attn_expanded(c.q_nope, c.q_rope, c.k_nope, c.k_rope, c.v, cq, ck, c.scale, True, out, lse)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first) and torch.equal(lse, fl)


# ---------------------------------------------------------------------------
# the two forms are one function
# ---------------------------------------------------------------------------

def test_both_forms_agree(serve):
    """Queries carried into the latent space by the expansion's own weights see
    the same scores: softmax weights, and so the log-sums, agree; the outputs
    agree once the latent one is expanded.  Weights of one nonzero a row (a
    power of two) make both carryings exact in bf16, so the bounds are those of
    the two attention forms alone."""
    heads, n = 4, 200
    g = torch.Generator(device="cuda").manual_seed(15)
    lat = torch.randn(n, 512, generator=g, device="cuda").to(BF)
    rope = torch.randn(n, 64, generator=g, device="cuda").to(BF)
    pick = torch.stack([torch.randperm(512, generator=g, device="cuda")[:448] for _ in range(heads)])  # [h, 448]
    kv = lat[:, pick.flatten()].view(n, heads, 448)
    q = torch.randn(n, heads, 256, generator=g, device="cuda").to(BF)
    q_lat = torch.zeros(n, heads, 512, dtype=BF, device="cuda")
    q_lat.scatter_(2, pick[:, :192].expand(n, -1, -1), q[:, :, :192])
    out, lse = torch.zeros(n, heads, 256, dtype=BF, device="cuda"), torch.zeros(n, heads, device="cuda")
    serve.latent_attn_expanded(q[:, :, :192], q[:, :, 192:], kv[:, :, :192], rope, kv[:, :, 192:], i32([0, n]),
                               i32([0, n]), 1.0 / 16, True, out, lse)
    cache = torch.zeros(13, 16, 576, dtype=BF, device="cuda")
    table = torch.randperm(13, generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()[None]
    slots = table[0].long().repeat_interleave(16)[:n] * 16 + torch.arange(n, device="cuda") % 16
    serve.latent_cache_write(lat, rope, slots, cache)
    o2, l2 = torch.zeros(n, heads, 512, dtype=BF, device="cuda"), torch.zeros(n, heads, device="cuda")
    ws = serve.new_latent_paged_workspace(n, heads, 1)
    serve.latent_attn_paged(q_lat, q[:, :, 192:], cache, table, i32([n]), i32([0, n]), 1.0 / 16, o2, l2, ws)
    want = expanded64(q[:, :, :192], q[:, :, 192:], kv[:, :, :192], rope, kv[:, :, 192:], [0, n], [0, n], 1.0 / 16, True)
    check_attention(out, lse, want, 256, n)
    check_attention(torch.gather(o2, 2, pick[:, 192:].expand(n, -1, -1)), l2, want, 576, n)
