"""One attention layer of a serving step, from the projections' inputs to the log
probabilities of the sampled tokens: the w8a16 projections (``w8``) with the
serving operators (``serve``) between and after them.

    python -m fp8_weight_only_w8a16_gb300.latent_step

runs two prompts and a few decode steps on random weights.  A step is

    block_tables -> latent_cache_write -> q_b projection
      prompt (nothing cached before):  kv_b projection -> latent_attn_expanded
      otherwise (decode, draft rows):  queries times W_UK -> latent_attn_paged -> times W_UV
    -> o_proj projection -> lm_head projection of the last tokens -> token_logprobs

kv_b's rows of a head are its 192 key rows W_UK and its 256 value rows W_UV: a
prompt expands the latents with them once, a decode step carries its few queries
into the latent space instead and reads the cache as it is.  The norms of the
model and the other layers are left out; activations come from the caller.
"""
from __future__ import annotations

import torch

from . import serve, w8

NOPE, ROPE, V, LATENT = 192, 64, 256, 512
MAX_TOKENS = 256  # of a projection call


def rotate(x: torch.Tensor, positions: torch.Tensor) -> torch.Tensor:
    """Rotary embedding of the last axis (64 columns, halves paired)."""
    half = x.shape[-1] // 2
    angle = positions.float()[:, None] * 10000.0 ** (-torch.arange(half, device=x.device) / half)
    shape = (x.shape[0],) + (1,) * (x.dim() - 2) + (half,)
    c, s = angle.cos().view(shape), angle.sin().view(shape)
    a, b = x.float().split(half, -1)
    return torch.cat([a * c - b * s, a * s + b * c], -1).to(torch.bfloat16)


def quantized(w: torch.Tensor):
    """E4M3 codes and row scales of w [n, k]."""
    scale = w.abs().amax(1) / 448.0
    return (w / scale[:, None]).to(torch.float8_e4m3fn).view(torch.uint8), scale


class LatentLayer:
    """Weights, cache, free list and tables of one layer on one GPU."""

    def __init__(self, heads: int = 64, hidden: int = 6144, q_rank: int = 2048, vocab: int = 4096,
                 requests: int = 2, pages: int = 64, page: int = 64, seed: int = 0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def weight(n, k):
            return torch.randn(n, k, generator=g, device="cuda") * k ** -0.5

        q_b, kv_b = quantized(weight(heads * (NOPE + ROPE), q_rank)), quantized(weight(heads * (NOPE + V), LATENT))
        o_proj = quantized(weight(hidden, heads * V))
        self.heads, self.hidden, self.vocab, self.page = heads, hidden, vocab, page
        self.build = w8.bind([w8.Plane.from_tensor(*p) for p in (q_b, kv_b, o_proj)])
        self.head = w8.bind([w8.Plane.from_tensor(weight(vocab, hidden).to(torch.bfloat16))])
        self.gemv_ws, self.head_ws = self.build.new_workspace(), self.head.new_workspace()
        # W_UK and W_UV as they are: the codes times their row's scale
        kv = (kv_b[0].view(torch.float8_e4m3fn).float() * kv_b[1][:, None]).to(torch.bfloat16).view(heads, NOPE + V, LATENT)
        self.w_uk, self.w_uv = kv[:, :NOPE], kv[:, NOPE:]
        self.scale = (NOPE + ROPE) ** -0.5
        ints = dict(dtype=torch.int32, device="cuda")
        self.cache = torch.zeros(pages, page, LATENT + ROPE, dtype=torch.bfloat16, device="cuda")
        self.free = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).to(**ints)
        self.free_head, self.next_head = torch.zeros(1, **ints), torch.zeros(1, **ints)
        self.table = torch.full((requests, pages), -1, **ints)
        self.ctx, self.seq_lens = torch.zeros(requests, **ints), torch.zeros(requests, **ints)
        self.cu, self.status = torch.zeros(requests + 1, **ints), torch.zeros(1, **ints)
        self.attn_ws = serve.new_latent_paged_workspace(MAX_TOKENS, heads, requests)
        self.logprob_ws = serve.new_logprobs_workspace(requests, vocab, 5)

    def project(self, plane: int, x: torch.Tensor, n: int) -> torch.Tensor:
        y = torch.empty(x.shape[0], n, dtype=torch.bfloat16, device="cuda")
        for i in range(0, x.shape[0], MAX_TOKENS):
            w8.w8_gemv(self.build, plane, x[i:i + MAX_TOKENS], y[i:i + MAX_TOKENS], self.gemv_ws)
        return y

    def attention(self, q_c: torch.Tensor, kv_a: torch.Tensor, new_lens: torch.Tensor, prompt: bool):
        """The attention output [T, heads * 256] of the step's tokens: q_c [T, q_rank],
        kv_a [T, 576] (the latent and the key to be rotated), new_lens tokens a request;
        prompt: the step is its requests' first, and they attend to its own tokens alone.
        A step that does not fit -- pages, table rows, or other than T tokens in all -- is
        refused and leaves the layer as it was; to know, it waits for the lengths."""
        toks, heads = q_c.shape[0], self.heads
        if kv_a.shape[0] != toks or new_lens.numel() != self.ctx.numel():
            raise ValueError("kv_a has a row a token, new_lens an entry a request")
        slots = torch.empty(toks, dtype=torch.int64, device="cuda")
        positions = torch.empty(toks, dtype=torch.int32, device="cuda")
        serve.block_tables(self.ctx, new_lens, self.page, self.free, self.free_head, self.table, self.seq_lens,
                           self.cu, slots, positions, self.next_head, self.status)
        cached = ((self.ctx > 0) & (new_lens > 0)).any().to(torch.int32)[None]
        status, total, cached = torch.cat([self.status, self.cu[-1:], cached]).tolist()
        if prompt and cached:
            raise ValueError("a prompt's requests have nothing cached")
        if status or total != toks:
            raise ValueError(f"{total} new tokens for {toks} rows" if total != toks else
                             "a length below zero" if status & 4 else
                             "no free page is left" if status & 1 else "a request outgrows its table row")
        self.free_head, self.next_head = self.next_head, self.free_head
        self.ctx.copy_(self.seq_lens)
        latent, k_rope = kv_a[:, :LATENT], rotate(kv_a[:, LATENT:], positions)
        serve.latent_cache_write(latent, k_rope, slots, self.cache)
        q = self.project(0, q_c, heads * (NOPE + ROPE)).view(toks, heads, NOPE + ROPE)
        q_nope, q_rope = q[:, :, :NOPE], rotate(q[:, :, NOPE:], positions)
        if prompt:
            kv = self.project(1, latent.contiguous(), heads * (NOPE + V)).view(toks, heads, NOPE + V)
            out = torch.empty(toks, heads, V, dtype=torch.bfloat16, device="cuda")
            serve.latent_attn_expanded(q_nope, q_rope, kv[:, :, :NOPE], k_rope, kv[:, :, NOPE:], self.cu, self.cu,
                                       self.scale, True, out)
        else:
            q_lat = torch.bmm(q_nope.transpose(0, 1), self.w_uk).transpose(0, 1)
            o_lat = torch.empty(toks, heads, LATENT, dtype=torch.bfloat16, device="cuda")
            serve.latent_attn_paged(q_lat, q_rope, self.cache, self.table, self.seq_lens, self.cu, self.scale, o_lat, None,
                                    self.attn_ws)
            out = torch.bmm(o_lat.transpose(0, 1), self.w_uv.transpose(1, 2)).transpose(0, 1).contiguous()
        return out.view(toks, heads * V)

    def step(self, q_c: torch.Tensor, kv_a: torch.Tensor, new_lens: torch.Tensor, prompt: bool):
        """The greedy next token of every request, its log probability, the entropy and
        the five likeliest tokens with theirs.  A request that appends nothing has no
        next token: -1, and NaN for the values."""
        rows, idle = new_lens.numel(), new_lens <= 0
        hidden = self.project(2, self.attention(q_c, kv_a, new_lens, prompt), self.hidden)
        logits = torch.zeros(rows, self.vocab, dtype=torch.bfloat16, device="cuda")
        if hidden.shape[0] > 0:
            # each request's last token (an idle one's place holds another's, or lies before the first)
            w8.bf16_gemv(self.head, 0, hidden[(self.cu[1:].long() - 1).clamp(min=0)], logits, self.head_ws)
        tokens = logits.argmax(1).to(torch.int32).masked_fill_(idle, -1)
        logprob, entropy = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
        ids = torch.empty(rows, 5, dtype=torch.int32, device="cuda")
        tops = torch.empty(rows, 5, device="cuda")
        serve.token_logprobs(logits, tokens, logprob, entropy, ids, tops, self.logprob_ws)
        nan = float("nan")
        return (tokens, logprob, entropy.masked_fill_(idle, nan), ids.masked_fill_(idle[:, None], -1),
                tops.masked_fill_(idle[:, None], nan))


def main():
    layer = LatentLayer()
    g = torch.Generator(device="cuda").manual_seed(1)

    def activations(toks):
        return (torch.randn(toks, 2048, generator=g, device="cuda").to(torch.bfloat16),
                torch.randn(toks, LATENT + ROPE, generator=g, device="cuda").to(torch.bfloat16))

    for lens, prompt in (([150, 77], True), ([1, 1], False), ([3, 1], False)):
        new = torch.tensor(lens, dtype=torch.int32, device="cuda")
        tokens, logprob, entropy, ids, tops = layer.step(*activations(sum(lens)), new, prompt)
        print(f"{'prompt' if prompt else 'decode'} {lens}: tokens {tokens.tolist()} "
              f"log p {[round(v, 3) for v in logprob.tolist()]} entropy {[round(v, 3) for v in entropy.tolist()]} "
              f"top {ids[:, :3].tolist()}")
    assert serve.device_status() == 0 and w8.device_status() == 0


if __name__ == "__main__":
    main()
