"""The serving operators around the projections, as they are measured: paged
bookkeeping (block tables, slot map), the latent-cache write, latent attention
in its absorbed form over the paged cache and in its expanded form over a
prompt, and the log probabilities of given tokens over the vocabulary.

``run`` computes one pass: with ``own`` false from elementary torch operations
in fp32, with ``own`` true through the framework's calls.  Sizes are those of
the repository's decode workloads (64 heads of 192 + 64 query / 256 value
columns, a latent of 512 + 64, a vocabulary of 154880) and, beside them, the
generic 128 + 64 / 128 head.
"""
from __future__ import annotations

import math

import torch

own = False  # set by the measuring program

LATENT, ROPE = 512, 64
VOCAB = 154880
NEG = float("-inf")


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one decode step of a mid-sized batch: every request appends one token
        {"name": "tables_decode", "op": "tables", "reqs": 64, "new_lo": 1, "new_hi": 1,
         "ctx_hi": 8192, "page": 64},
        # a scheduler step that admits prompts beside running requests: ragged, many tokens
        {"name": "tables_prompts", "op": "tables", "reqs": 1021, "new_lo": 0, "new_hi": 257,
         "ctx_hi": 30000, "page": 16},
        # the cache rows of one decode step, taken from the merged qkv_a output
        {"name": "write_decode", "op": "write", "toks": 8, "page": 64, "row": 2624},
        # the cache rows of a large prompt chunk, small pages
        {"name": "write_chunk", "op": "write", "toks": 16391, "page": 16, "row": 2624},
        # one request, one token, a short context: latency
        {"name": "paged_single", "op": "paged", "reqs": 1, "q_lo": 1, "q_hi": 1, "heads": 64,
         "len_lo": 1531, "len_hi": 1531, "page": 64},
        # speculative decoding: a verify step of 1 to 4 draft rows a request, ragged contexts
        {"name": "paged_draft", "op": "paged", "reqs": 24, "q_lo": 1, "q_hi": 4, "heads": 64,
         "len_lo": 900, "len_hi": 8111, "page": 16},
        # a large decode batch over long ragged contexts: the bandwidth case
        {"name": "paged_batch", "op": "paged", "reqs": 128, "q_lo": 1, "q_hi": 1, "heads": 64,
         "len_lo": 1, "len_hi": 16384, "page": 64},
        # a few short prompts of odd lengths, prefix already cached, generic head
        {"name": "expanded_ragged", "op": "expanded", "reqs": 3, "q_lo": 37, "q_hi": 611,
         "prefix_hi": 333, "heads": 16, "nope": 128, "v": 128},
        # one long prompt at the model's own head
        {"name": "expanded_prompt", "op": "expanded", "reqs": 1, "q_lo": 4096, "q_hi": 4096,
         "prefix_hi": 0, "heads": 64, "nope": 192, "v": 256},
        # the sampled token of one decode step, bf16 logits as the head projection writes them
        {"name": "logprobs_single", "op": "logprobs", "rows": 1, "vocab": VOCAB, "top": 5,
         "bf16": True, "banned": 0.0},
        # a batch with fp32 logits (after penalties), banned tokens, the most alternatives
        {"name": "logprobs_batch", "op": "logprobs", "rows": 48, "vocab": VOCAB, "top": 20,
         "bf16": False, "banned": 0.25},
        # scoring a prompt: a row a prompt token
        {"name": "logprobs_prompt", "op": "logprobs", "rows": 1024, "vocab": VOCAB, "top": 1,
         "bf16": True, "banned": 0.0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "write", "paged", "paged", "expanded", "expanded", "logprobs",
                     "logprobs"])
    if op == "tables":
        hi = rng.choice([1, 1, 4, 257])
        return {"op": op, "reqs": _log(rng, 1, 1024), "new_lo": rng.choice([0, 1]), "new_hi": hi,
                "ctx_hi": _log(rng, 1, 30000), "page": rng.choice([16, 32, 64, 128, 48])}
    if op == "write":
        return {"op": op, "toks": _log(rng, 1, 16000), "page": rng.choice([16, 32, 64, 128]),
                "row": rng.choice([576, 640, 2624])}
    if op == "paged":
        heads = rng.choice([8, 16, 20, 32, 64, 64, 128])
        reqs = _log(rng, 1, 128)
        budget = (1 << 20) // max(1, heads // 64)  # cached tokens: no more than the largest listed case
        hi = _log(rng, 1, min(16384, budget // reqs))
        return {"op": op, "reqs": reqs, "q_lo": rng.choice([0, 1, 1]),
                "q_hi": rng.choice([1, 1, 2, 5, 8]) if reqs * hi <= 1 << 17 else 1,
                "heads": heads, "len_lo": rng.choice([0, hi // 2, hi]), "len_hi": hi,
                "page": rng.choice([16, 32, 64, 128])}
    if op == "expanded":
        nope, v = rng.choice([(192, 256), (128, 128)])
        heads = rng.choice([8, 16, 40, 64])
        reqs = rng.choice([1, 1, 2, 5, 9])
        hi = _log(rng, 1, 3500 // max(1, reqs // 2))
        return {"op": op, "reqs": reqs, "q_lo": rng.choice([0, hi // 3, hi]), "q_hi": hi,
                "prefix_hi": rng.choice([0, 0, 129, 500]), "heads": heads, "nope": nope, "v": v}
    rows = _log(rng, 1, 900)
    bf16 = rng.random() < 0.6
    vocab = rng.choice([VOCAB, VOCAB, 32003, 129283, 1025])
    return {"op": op, "rows": rows if bf16 else max(1, rows // 2), "vocab": vocab,
            "top": rng.choice([0, 1, 5, 20, 32]), "bf16": bf16,
            "banned": rng.choice([0.0, 0.0, 0.3, 0.999])}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _ints(case, seed):
    """The integer side of a case (request lengths), made on the host: contexts
    and the order of the requests go by the seed, the number of tokens by the case."""
    g = torch.Generator().manual_seed(int(seed) * 7919 + 11)
    n = case["reqs"]
    fixed = torch.Generator().manual_seed(5)
    order = torch.randperm(n, generator=g)

    def between(lo, hi, n):
        return torch.randint(lo, hi + 1, (n,), generator=g, dtype=torch.int64)

    def appended(lo, hi):
        new = torch.randint(min(lo, hi), hi + 1, (n,), generator=fixed, dtype=torch.int64)
        if int(new.sum()) == 0:
            new[0] = 1
        return new[order]

    if case["op"] == "tables":
        return between(0, case["ctx_hi"], n), appended(case["new_lo"], case["new_hi"]), g
    q = appended(case["q_lo"], case["q_hi"])
    if case["op"] == "paged":
        length = between(case["len_lo"], case["len_hi"], n)
        return q, torch.where(length > 0, torch.maximum(length, q), length), g
    return q, q + between(0, case["prefix_hi"], n), g


def _cu(x):
    return torch.cat([torch.zeros(1, dtype=torch.int64), torch.cumsum(x, 0)]).to(torch.int32)


def prepare(case, seed):
    dev = torch.device("cuda:0")
    op = case["op"]
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    s = {"case": case, "ws": None}

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=gen, device=dev) * std).to(torch.bfloat16)

    if op == "tables":
        ctx, new, g = _ints(case, seed)
        page, n = case["page"], case["reqs"]
        have = (ctx + page - 1) // page
        want = (ctx + new + page - 1) // page
        width = -(-(case["ctx_hi"] + case["new_hi"]) // page) + 1
        perm = torch.randperm(int(want.sum()) + 64, generator=g).to(torch.int32)
        owned = torch.full((n, width), -1, dtype=torch.int32)
        used = int(have.sum())
        owned[torch.arange(width)[None, :] < have[:, None]] = perm[:used]
        toks = int(new.sum())
        s.update(ctx=ctx.to(torch.int32).to(dev), new=new.to(torch.int32).to(dev),
                 table=owned.to(dev), free=perm[used:].contiguous().to(dev),
                 head=torch.full((1,), 3, dtype=torch.int32, device=dev),
                 head_out=torch.zeros(1, dtype=torch.int32, device=dev),
                 seq_lens=torch.zeros(n, dtype=torch.int32, device=dev),
                 cu_new=torch.zeros(n + 1, dtype=torch.int32, device=dev),
                 slots=torch.zeros(toks + 5, dtype=torch.int64, device=dev),
                 positions=torch.zeros(toks + 5, dtype=torch.int32, device=dev),
                 status=torch.zeros(1, dtype=torch.int32, device=dev))
    elif op == "write":
        toks, page = case["toks"], case["page"]
        pages = -(-toks // page) + 3
        g = torch.Generator().manual_seed(int(seed) * 7919 + 11)
        slots = torch.randperm(pages * page, generator=g)[:toks]
        if toks > 4:
            slots[toks // 2] = -1  # a padding row of a captured step
        rows = normal(toks, case["row"])
        s.update(latent=rows[:, case["row"] - 576:case["row"] - 64], rope=rows[:, case["row"] - 64:],
                 slots=slots.to(dev), cache=normal(pages, page, LATENT + ROPE))
    elif op == "paged":
        q, length, g = _ints(case, seed)
        page, n, heads = case["page"], case["reqs"], case["heads"]
        pages = (length + page - 1) // page
        total = int(pages.sum()) + 2
        width = max(1, int(pages.max()))
        perm = torch.randperm(total, generator=g).to(torch.int32)
        table = torch.zeros((n, width), dtype=torch.int32)
        held = torch.arange(width)[None, :] < pages[:, None]
        table[held] = perm[:int(pages.sum())]
        toks = int(q.sum())
        s.update(q_lat=normal(toks, heads, LATENT), q_rope=normal(toks, heads, ROPE),
                 cache=normal(total, page, LATENT + ROPE), table=table.to(dev),
                 seq_lens=length.to(torch.int32).to(dev), cu_q=_cu(q).to(dev),
                 q_max=int(q.max()), scale=1.0 / 16,
                 out=torch.empty(toks, heads, LATENT, dtype=torch.bfloat16, device=dev),
                 lse=torch.empty(toks, heads, dtype=torch.float32, device=dev))
        if own:
            from fp8_weight_only_w8a16_gb300 import serve
            s["ws"] = serve.new_latent_paged_workspace(toks, heads, n, device=dev)
    elif op == "expanded":
        q, k, _ = _ints(case, seed)
        heads, nope, v = case["heads"], case["nope"], case["v"]
        tq, tk = int(q.sum()), int(k.sum())
        queries = normal(tq, heads, nope + ROPE)
        kv = normal(tk, heads, nope + v)  # the kv_b projection's output
        s.update(q_nope=queries[:, :, :nope], q_rope=queries[:, :, nope:], k_nope=kv[:, :, :nope],
                 k_rope=normal(tk, ROPE), v=kv[:, :, nope:], cu_q=_cu(q).to(dev),
                 cu_k=_cu(k).to(dev), q_max=int(q.max()), k_max=max(1, int(k.max())),
                 scale=1.5 / math.sqrt(nope + ROPE),
                 out=torch.empty(tq, heads, v, dtype=torch.bfloat16, device=dev),
                 lse=torch.empty(tq, heads, dtype=torch.float32, device=dev))
    else:
        rows, vocab, top = case["rows"], case["vocab"], case["top"]
        logits = torch.randn(rows, vocab, generator=gen, device=dev) * 2.5
        if case["banned"]:
            logits.masked_fill_(torch.rand(rows, vocab, generator=gen, device=dev) < case["banned"], NEG)
        logits = logits.to(torch.bfloat16) if case["bf16"] else logits
        ids = torch.randint(0, vocab, (rows,), generator=gen, device=dev)
        likely = torch.argmax(logits, 1)
        pick = torch.rand(rows, generator=gen, device=dev) < 0.7
        s.update(logits=logits, tokens=torch.where(pick, likely, ids).to(torch.int32),
                 logprob=torch.empty(rows, dtype=torch.float32, device=dev),
                 entropy=torch.empty(rows, dtype=torch.float32, device=dev),
                 top_ids=torch.empty(rows, top, dtype=torch.int32, device=dev),
                 top_logprobs=torch.empty(rows, top, dtype=torch.float32, device=dev))
        if own:
            from fp8_weight_only_w8a16_gb300 import serve
            s["ws"] = serve.new_logprobs_workspace(rows, vocab, top, device=dev)
    return s


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------

def _run_own(s):
    from fp8_weight_only_w8a16_gb300 import serve
    op = s["case"]["op"]
    if op == "tables":
        serve.block_tables(s["ctx"], s["new"], s["case"]["page"], s["free"], s["head"], s["table"],
                           s["seq_lens"], s["cu_new"], s["slots"], s["positions"], s["head_out"],
                           s["status"])
        return {k: s[k] for k in ("table", "seq_lens", "cu_new", "slots", "positions", "head_out", "status")}
    if op == "write":
        serve.latent_cache_write(s["latent"], s["rope"], s["slots"], s["cache"])
        return {"cache": s["cache"]}
    if op == "paged":
        serve.latent_attn_paged(s["q_lat"], s["q_rope"], s["cache"], s["table"], s["seq_lens"],
                                s["cu_q"], s["scale"], s["out"], s["lse"], s["ws"])
        return {"out": s["out"], "lse": s["lse"]}
    if op == "expanded":
        serve.latent_attn_expanded(s["q_nope"], s["q_rope"], s["k_nope"], s["k_rope"], s["v"],
                                   s["cu_q"], s["cu_k"], s["scale"], True, s["out"], s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    serve.token_logprobs(s["logits"], s["tokens"], s["logprob"], s["entropy"], s["top_ids"],
                         s["top_logprobs"], s["ws"])
    return {k: s[k] for k in ("logprob", "entropy", "top_ids", "top_logprobs")}


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------

def _tables(s):
    page = s["case"]["page"]
    ctx, new, table, free = s["ctx"].long(), s["new"].long(), s["table"], s["free"]
    n, width = table.shape
    have, want = (ctx + page - 1) // page, (ctx + new + page - 1) // page
    need = want.clamp(max=width) - have.clamp(max=width)
    base = s["head"].long() + torch.cumsum(need, 0) - need
    col = torch.arange(width, device=table.device)[None, :]
    at = base[:, None] + col - have[:, None]
    fresh = torch.where(at < free.numel(), free[at.clamp(0, free.numel() - 1)], -1)
    table.copy_(torch.where((col >= have[:, None]) & (col < want[:, None]), fresh, table))
    cu = torch.cat([torch.zeros_like(new[:1]), torch.cumsum(new, 0)])
    t = torch.arange(s["slots"].numel(), device=table.device)
    r = torch.searchsorted(cu, t, right=True) - 1
    live = r < n
    r = r.clamp(max=n - 1)
    pos = ctx[r] + t - cu[r]
    entry = table[r, (pos // page).clamp(0, width - 1)].long()
    held = live & (pos // page < width) & (entry >= 0)
    total = s["head"].long() + need.sum()
    status = (total > free.numel()).int() + 2 * (want > width).any().int() + 4 * (cu[-1] > t.numel()).int()
    return {"table": table, "seq_lens": (ctx + new).to(torch.int32), "cu_new": cu.to(torch.int32),
            "slots": torch.where(held, entry * page + pos % page, -1),
            "positions": torch.where(live, pos, -1).to(torch.int32),
            "head_out": total.clamp(max=free.numel()).to(torch.int32),
            "status": status.reshape(1).to(torch.int32)}


def _write(s):
    cache = s["cache"]
    flat = cache.view(-1, LATENT + ROPE)
    rows = torch.cat([s["latent"], s["rope"]], 1)
    # a padding row (slot -1) writes the first real token's row once more
    ok = s["slots"] >= 0
    first = torch.argmax(ok.int())
    src = torch.where(ok, torch.arange(ok.numel(), device=ok.device), first)
    flat.index_copy_(0, s["slots"][src], rows[src])
    return {"cache": cache}


def _by_request(cu, q_max, toks):
    """Padded query rows [requests, q_max] of a ragged batch, and each token's request and place."""
    cu = cu.long()
    idx = (cu[:-1, None] + torch.arange(q_max, device=cu.device)).clamp(max=toks - 1)
    t = torch.arange(toks, device=cu.device)
    r = torch.searchsorted(cu, t, right=True) - 1
    return idx, r, t - cu[r]


def _softmax_values(x, vis, v, product):
    """softmax over the visible entries of x times v, and its log-sum; rows that see nothing give 0 and -inf."""
    x = torch.where(vis, x, NEG)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == NEG, 0.0, m)
    p = torch.exp(x - m)
    z = p.sum(-1, keepdim=True)
    o = product(p, v) / torch.where(z > 0, z, 1.0)
    return o, (m + torch.log(z)).squeeze(-1)


def _paged(s):
    cu, lens, table = s["cu_q"], s["seq_lens"].long(), s["table"].long()
    toks, heads, _ = s["q_lat"].shape
    n = lens.numel()
    idx, r, i = _by_request(cu, s["q_max"], toks)
    q = torch.cat([s["q_lat"], s["q_rope"]], 2).float()[idx]          # [n, q, h, 576]
    k = s["cache"][table].reshape(n, -1, LATENT + ROPE).float()       # [n, width * page, 576]
    j = torch.arange(k.shape[1], device=k.device)
    k = torch.where((j[None, :] < lens[:, None])[..., None], k, 0.0)
    ql = (cu[1:] - cu[:-1]).long()
    limit = lens[:, None] - ql[:, None] + torch.arange(s["q_max"], device=k.device)  # last visible key
    vis = (j <= limit[..., None])[:, :, None, :] & (j < lens[:, None])[:, None, None, :]
    x = torch.matmul(q.flatten(1, 2), k.transpose(1, 2)).view(n, s["q_max"], heads, -1) * s["scale"]
    o, lse = _softmax_values(x, vis, k[..., :LATENT],
                             lambda p, v: torch.matmul(p.flatten(1, 2), v).view(n, s["q_max"], heads, LATENT))
    return {"out": o[r, i].to(torch.bfloat16), "lse": lse[r, i]}


def _expanded(s):
    toks, heads, _ = s["q_nope"].shape
    idx, r, i = _by_request(s["cu_q"], s["q_max"], toks)
    q = torch.cat([s["q_nope"], s["q_rope"]], 2).float()[idx].transpose(1, 2)         # [n, h, q, d]
    tk = s["k_rope"].shape[0]
    kidx = _by_request(s["cu_k"], s["k_max"], tk)[0]
    k = torch.cat([s["k_nope"], s["k_rope"][:, None, :].expand(-1, heads, -1)], 2).float()[kidx].permute(0, 2, 3, 1)
    v = s["v"].float()[kidx].transpose(1, 2)
    ql, kl = (s["cu_q"][1:] - s["cu_q"][:-1]).long(), (s["cu_k"][1:] - s["cu_k"][:-1]).long()
    j = torch.arange(s["k_max"], device=k.device)
    limit = (kl - ql)[:, None] + torch.arange(s["q_max"], device=k.device)
    vis = ((j <= limit[..., None]) & (j < kl[:, None, None]))[:, None]
    o, lse = _softmax_values(torch.matmul(q, k) * s["scale"], vis, v, torch.matmul)
    return {"out": o[r, :, i].to(torch.bfloat16), "lse": lse[r, :, i]}


def _logprobs(s):
    x = s["logits"].float()
    rows, vocab = x.shape
    top = s["top_ids"].shape[1]
    m = x.amax(1, keepdim=True)
    d = x - m
    e = torch.exp(d)
    z = e.sum(1)
    logz = torch.log(z)
    entropy = logz - torch.where(e > 0, e * d, 0.0).sum(1) / z
    logprob = d.gather(1, s["tokens"].long()[:, None])[:, 0] - logz
    # values in order with the lowest index first among equals: one 64-bit key an entry
    bits = (x + 0.0).view(torch.int32)
    order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long()
    key = order * (1 << 32) + (vocab - 1 - torch.arange(vocab, device=x.device))
    ids = vocab - 1 - torch.topk(key, top, 1).values % (1 << 32)
    return {"logprob": logprob, "entropy": entropy, "top_ids": ids.to(torch.int32),
            "top_logprobs": d.gather(1, ids) - logz[:, None]}


def run(state):
    if own:
        return _run_own(state)
    return {"tables": _tables, "write": _write, "paged": _paged, "expanded": _expanded,
            "logprobs": _logprobs}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op in ("tables", "paged", "expanded"):
        a, b, _ = _ints(case, 0)
    if op == "tables":
        toks = int(b.sum())
        fresh = int(((a + b + case["page"] - 1) // case["page"] - (a + case["page"] - 1) // case["page"]).sum())
        return {"bytes": 16 * case["reqs"] + 8 * fresh + 12 * toks + 20, "flops": 0}
    if op == "write":
        return {"bytes": case["toks"] * (2 * 2 * (LATENT + ROPE) + 8), "flops": 0}
    if op == "paged":
        toks, h = int(a.sum()), case["heads"]
        seen = int((a * b - a * (a - 1) // 2).clamp(min=0).sum())  # (query token, key) pairs
        return {"bytes": 2 * (LATENT + ROPE) * int(b[a > 0].sum()) + toks * h * (2 * (LATENT + ROPE) + 2 * LATENT + 4),
                "flops": 2 * h * seen * (2 * LATENT + ROPE)}
    if op == "expanded":
        h, nope, v = case["heads"], case["nope"], case["v"]
        pairs = int((a * b - a * (a - 1) // 2).sum())
        return {"bytes": int(a.sum()) * h * 2 * (nope + ROPE + v + 2) + int(b.sum()) * 2 * (h * (nope + v) + ROPE),
                "flops": 2 * h * pairs * (nope + ROPE + v)}
    return {"bytes": case["rows"] * (case["vocab"] * (2 if case["bf16"] else 4) + 12 + 8 * case["top"]),
            "flops": 0}


# ---------------------------------------------------------------------------
# the definitions in 64 bits, a request (a head, a row) at a time
# ---------------------------------------------------------------------------

def _attend64(q, k, v, scale, offset):
    """q [a, d], k [b, d], v [b, e]; query i sees keys 0 .. offset + i."""
    x = q @ k.T * scale
    i = torch.arange(q.shape[0], device=q.device)[:, None]
    x = x.masked_fill(torch.arange(k.shape[0], device=q.device)[None, :] > offset + i, NEG)
    lse = torch.logsumexp(x, 1)
    w = torch.exp(x - lse[:, None]).nan_to_num(0.0)
    return w @ v, lse


def exact(case, seed):
    op = case["op"]
    if op == "tables":
        return None  # whole numbers
    s = prepare(case, seed)
    if op == "write":
        cache = s["cache"].double()
        flat = cache.view(-1, LATENT + ROPE)
        for t, slot in enumerate(s["slots"].tolist()):
            if slot >= 0:
                flat[slot, :LATENT] = s["latent"][t]
                flat[slot, LATENT:] = s["rope"][t]
        return {"cache": cache}
    if op == "logprobs":
        if case["rows"] * case["vocab"] > 4e8:
            return None
        x = s["logits"].double()
        lse = torch.logsumexp(x, 1)
        lp = x - lse[:, None]
        p = torch.exp(lp)
        return {"logprob": lp[torch.arange(case["rows"]), s["tokens"].long()],
                "entropy": -torch.special.xlogy(p, p).sum(1), "top_ids": None,
                "top_logprobs": torch.topk(lp, case["top"], 1).values}
    cu_q = s["cu_q"].tolist()
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda:0")
    lse = torch.full(s["lse"].shape, NEG, dtype=torch.float64, device="cuda:0")
    if op == "paged":
        lens = s["seq_lens"].tolist()
        for r, n in enumerate(lens):
            a, b = cu_q[r], cu_q[r + 1]
            if n == 0 or a == b:
                continue
            pages = s["table"][r, :-(-n // case["page"])].long()
            k = s["cache"][pages].reshape(-1, LATENT + ROPE)[:n].double()
            x = torch.einsum("thd,nd->thn", s["q_lat"][a:b].double(), k[:, :LATENT])
            x = (x + torch.einsum("thd,nd->thn", s["q_rope"][a:b].double(), k[:, LATENT:])) * s["scale"]
            place = n - (b - a) + torch.arange(b - a, device=x.device)
            x = x.masked_fill((torch.arange(n, device=x.device) > place[:, None])[:, None, :], NEG)
            w = torch.softmax(x, -1)
            out[a:b] = torch.einsum("thn,nd->thd", w, k[:, :LATENT])
            lse[a:b] = torch.logsumexp(x, -1)
        return {"out": out, "lse": lse}
    cu_k = s["cu_k"].tolist()
    if sum((b - a) * (d - c) for a, b, c, d in zip(cu_q, cu_q[1:], cu_k, cu_k[1:])) * case["heads"] > 2e9:
        return None
    for r in range(case["reqs"]):
        (a, b), (c, d) = cu_q[r:r + 2], cu_k[r:r + 2]
        if a == b or c == d:
            continue
        for h in range(case["heads"]):
            q = torch.cat([s["q_nope"][a:b, h], s["q_rope"][a:b, h]], 1).double()
            k = torch.cat([s["k_nope"][c:d, h], s["k_rope"][c:d]], 1).double()
            out[a:b, h], lse[a:b, h] = _attend64(q, k, s["v"][c:d, h].double(), s["scale"], (d - c) - (b - a))
    return {"out": out, "lse": lse}
