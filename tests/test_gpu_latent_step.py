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
