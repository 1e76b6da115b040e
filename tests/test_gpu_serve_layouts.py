"""GPU tests of operand layouts other than token by token: heads outermost (as a
batched product over the heads writes them) and operands cut out of wider ones.
An operand's place changes nothing: the outputs are those of its copy, bit for bit."""
from __future__ import annotations

import pytest
import torch

from tests.test_gpu_serve_attention import Expanded, Paged, cu_of, i32, pairs

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def serve():
    from fp8_weight_only_w8a16_gb300 import serve
    serve.device_status(reset=True)
    yield serve
    assert serve.device_status() == 0, "a bounded wait gave up"


def heads_first(x):
    """The same values [T, H, d], stored [H][T][d]."""
    return x.transpose(0, 1).contiguous().transpose(0, 1)


def far_apart(x):
    """The same values, token rows 2^16 elements and heads 1032 apart or more."""
    t, h, d = x.shape
    store = torch.full((t, max(h, 63), 1032 + 8), float("nan"), dtype=BF, device="cuda")
    store[:, :h, 8:8 + d] = x
    return store[:, :h, 8:8 + d]


LAYOUTS = [heads_first, far_apart]


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("lens,q_lens,heads", [([300, 77, 1000], [1, 3, 1], 20), ([513], [1], 64), ([40, 9], [1, 1], 1)])
def test_paged_layouts(serve, layout, lens, q_lens, heads):
    c = Paged(lens, q_lens, heads, 16, seed=heads)
    want, wl = c.run(serve)
    t = cu_of(q_lens)[-1]
    out, lse = layout(torch.zeros(t, heads, 512, dtype=BF, device="cuda")), torch.zeros(t, heads, device="cuda")
    serve.latent_attn_paged(layout(c.q_lat), layout(c.q_rope), c.cache, c.table, i32(c.lens), i32(c.cu), c.scale, out, lse,
                            serve.new_latent_paged_workspace(t, heads, len(lens)))
    assert torch.equal(out, want) and torch.equal(lse, wl)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("nope,v", [(192, 256), (128, 128)])
@pytest.mark.parametrize("q,k,heads", [([140, 3], [150, 3], 3), ([1], [1], 5), ([70], [70], 1), ([1630], [1700], 64)])
def test_expanded_layouts(serve, layout, nope, v, q, k, heads):
    c = Expanded(q, k, heads, nope, v, seed=sum(q))
    assert pairs(serve, c) == (heads == 64)
    want, wl = c.run(serve)
    t = sum(q)
    out, lse = layout(torch.zeros(t, heads, v, dtype=BF, device="cuda")), torch.zeros(t, heads, device="cuda")
    serve.latent_attn_expanded(layout(c.q_nope), layout(c.q_rope), layout(c.k_nope), c.k_rope, layout(c.v), i32(c.cu_q), i32(c.cu_k),
                               c.scale, True, out, lse)
    assert torch.equal(out, want) and torch.equal(lse, wl)
