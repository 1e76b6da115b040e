"""GPU test of the serving step that runs the operators together: tokens that a
request decodes one after another (absorbed form, paged cache) get the attention
output that the same tokens get as one prompt (expanded form).

The two differ by roundings to bf16 alone: on the absorbed side of the carried
query, the latent output and its expansion, on the expanded side of the keys and
values.  Each is 2^-9 of its value in the root mean square at most; a score of
standard deviation 1 moves by two of them, a weight by as much, the output by
that and two more: 5 x 2^-9 = 0.01 of its norm, twice that is allowed."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu


def test_decoded_tokens_match_the_prompt():
    from fp8_weight_only_w8a16_gb300 import latent_step, serve, w8
    args = dict(heads=16, hidden=512, q_rank=256, vocab=1000, requests=2, pages=40, page=16, seed=3)
    g = torch.Generator(device="cuda").manual_seed(4)
    lens = [150, 71]
    q_c = [torch.randn(n, 256, generator=g, device="cuda").to(torch.bfloat16) for n in lens]
    kv_a = [torch.randn(n, 576, generator=g, device="cuda").to(torch.bfloat16) for n in lens]

    def i32(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    whole = latent_step.LatentLayer(**args)
    want = whole.attention(torch.cat(q_c), torch.cat(kv_a), i32(lens), True).float()
    want = [want[:150], want[150:]]
    # the same in parts: a prompt, then several tokens at once, one by one, none
    parts = latent_step.LatentLayer(**args)
    at = [0, 0]
    for new in ([130, 60], [4, 1], [1, 1], [0, 3], [15, 6]):
        rows = [slice(a, a + n) for a, n in zip(at, new)]
        out = parts.attention(torch.cat([x[r] for x, r in zip(q_c, rows)]), torch.cat([x[r] for x, r in zip(kv_a, rows)]),
                              i32(new), at == [0, 0]).float()
        for r in range(2):
            got = out[:new[0]] if r == 0 else out[new[0]:]
            ref = want[r][rows[r]]
            if new[r]:
                assert float((got - ref).norm() / ref.norm()) < 0.02
        at = [a + n for a, n in zip(at, new)]
    assert at == lens and parts.seq_lens.tolist() == lens and int(parts.status) == 0
    tokens, logprob, entropy, ids, tops = parts.step(q_c[0][:2], kv_a[0][:2], i32([1, 1]), False)
    assert torch.equal(ids[:, 0], tokens) and torch.equal(tops[:, 0], logprob)
    assert (logprob < 0).all() and (entropy > 0).all() and (tops[:, :-1] >= tops[:, 1:]).all()
    assert serve.device_status() == 0 and w8.device_status() == 0


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def small_layer(**kw):
    from fp8_weight_only_w8a16_gb300 import latent_step
    return latent_step.LatentLayer(**{**dict(heads=16, hidden=512, q_rank=256, vocab=1000, requests=4, pages=40, page=16, seed=3), **kw})


def activations(toks, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(toks, 256, generator=g, device="cuda").to(torch.bfloat16),
            torch.randn(toks, 576, generator=g, device="cuda").to(torch.bfloat16))


@pytest.mark.parametrize("new", [[0, 2, 1, 3], [1, 0, 0, 2], [2, 1, 0, 0], [0, 0, 0, 1], [0, 0, 0, 0], [1, 2, 1, 1]])
def test_requests_that_append_nothing(new):
    """Each request's tokens come from its own last row of the attention output, whichever requests are idle:
    bit for bit what the projections and the log probabilities give for those rows.  An idle request gets
    -1 and NaN."""
    from fp8_weight_only_w8a16_gb300 import serve, w8
    layer = small_layer()
    layer.step(*activations(90, 5), i32([20, 30, 7, 33]), True)
    q_c, kv_a = activations(sum(new), 6)
    attention, seen = layer.attention, []
    layer.attention = lambda *args: seen.append(attention(*args)) or seen[0]
    tokens, logprob, entropy, ids, tops = layer.step(q_c, kv_a, i32(new), False)
    live = [r for r in range(4) if new[r]]
    idle = [r for r in range(4) if not new[r]]
    assert (tokens[idle] == -1).all() and (ids[idle] == -1).all()
    for values in (logprob, entropy, tops):
        assert torch.isnan(values[idle]).all() and torch.isfinite(values[live]).all()
    if live:
        hidden = layer.project(2, seen[0], layer.hidden)
        ends = [max(sum(new[:r + 1]) - 1, 0) for r in range(4)]
        logits = torch.empty(4, 1000, dtype=torch.bfloat16, device="cuda")
        w8.bf16_gemv(layer.head, 0, hidden[ends], logits, layer.head_ws)
        want = logits.argmax(1).to(torch.int32)
        lp, ent = torch.empty(4, device="cuda"), torch.empty(4, device="cuda")
        top, top_lp = torch.empty(4, 5, dtype=torch.int32, device="cuda"), torch.empty(4, 5, device="cuda")
        serve.token_logprobs(logits, want, lp, ent, top, top_lp, serve.new_logprobs_workspace(4, 1000, 5))
        for got, ref in ((tokens, want), (logprob, lp), (entropy, ent), (ids, top), (tops, top_lp)):
            assert torch.equal(got[live], ref[live])
    assert serve.device_status() == 0 and w8.device_status() == 0


@pytest.mark.parametrize("layer,first,new,toks", [
    (dict(pages=5), [20, 16, 0, 1], [0, 0, 17, 0], 17),       # no page left
    (dict(pages=40), [20, 16, 0, 1], [1, 1, 1, 1], 3),        # more tokens than rows,
    (dict(pages=40), [20, 16, 0, 1], [1, 1, 1, 1], 5),        # fewer,
    (dict(pages=40), [20, 16, 0, 1], [1, -1, 1, 1], 3),       # a length below zero
    (dict(pages=4), [20, 0, 0, 0], [50, 0, 0, 0], 50)])       # a table row outgrown
def test_a_step_that_does_not_fit_is_refused(layer, first, new, toks):
    """... and leaves the layer as it was: the next step that fits gives what it gives without it."""
    from fp8_weight_only_w8a16_gb300 import serve, w8
    layers = [small_layer(**layer) for _ in range(2)]
    for l in layers:
        l.step(*activations(sum(first), 7), i32(first), True)
    for _ in range(2):
        with pytest.raises(ValueError):
            layers[0].step(*activations(toks, 8), i32(new), False)
    assert layers[0].ctx.tolist() == first
    got = [l.step(*activations(3, 9), i32([2, 0, 0, 1]), False) for l in layers]
    for a, b in zip(*got):
        assert torch.equal(a[[0, 3]], b[[0, 3]])
    assert torch.equal(layers[0].ctx, layers[1].ctx) and torch.equal(layers[0].free_head, layers[1].free_head)
    assert serve.device_status() == 0 and w8.device_status() == 0


def test_rows_and_requests_are_counted():
    layer = small_layer()
    q_c, kv_a = activations(4, 10)
    with pytest.raises(ValueError):
        layer.step(q_c, kv_a[:3], i32([1, 1, 1, 1]), True)
    with pytest.raises(ValueError):
        layer.step(q_c, kv_a, i32([1, 1, 2]), True)


def test_a_prompt_has_nothing_cached():
    """The expanded form sees the step's own tokens only: a request that has more is not a prompt's."""
    layer = small_layer()
    layer.step(*activations(30, 11), i32([20, 10, 0, 0]), True)
    with pytest.raises(ValueError):
        layer.step(*activations(3, 12), i32([0, 2, 0, 1]), True)
    assert layer.ctx.tolist() == [20, 10, 0, 0]
    # requests that start beside idle ones are
    tokens = layer.step(*activations(3, 12), i32([0, 0, 2, 1]), True)[0]
    assert layer.ctx.tolist() == [20, 10, 2, 1] and (tokens[:2] == -1).all() and (tokens[2:] >= 0).all()
