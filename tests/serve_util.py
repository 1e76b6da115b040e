"""64-bit plain forms of the serving operators and the error bounds that the
GPU tests hold them to.

Bounds of the attention outputs, from the arithmetic that w8_serve.h states.
With u = 2^-24 the fp32 unit, O and A = sum_j p_j |v_j| the exact output and
its magnitude, X = max_j scale sum_d |q_d k_jd|, D columns, L keys:
  a score is off by at most g X, g = 2 (D + 2) u (an adder that truncates
  loses up to twice the unit an addition), plus 4 u |x| for the scaled,
  shifted argument of the exponential, so a weight by a factor 1 + e with
  e = 1.1 (g X + 4 u X) + 2^-21 (the exponential itself);
  the quotient of two such sums by at most 2 e and the sums' own 2 L u each;
  a weight's rounding to bf16 (8 significant bits: half a unit is at most 2^-8
  of the value) adds 2^-8 of A, the output's 2^-8 of |O|.
"""
from __future__ import annotations

import torch

U = 2.0 ** -24
NEG = float("-inf")


def attend64(q, k, v, scale, see):
    """q [a, d], k [b, d], v [b, e] (any float type), see [a, b] bool ->
    out, lse, A, X in 64 bits."""
    q, k, v = q.double(), k.double(), v.double()
    k = torch.where(see.any(0)[:, None], k, 0.0)
    v = torch.where(see.any(0)[:, None], v, 0.0)
    x = (q @ k.T * scale).masked_fill(~see, NEG)
    mag = (q.abs() @ k.abs().T * scale).masked_fill(~see, 0.0)
    m = x.amax(1, keepdim=True) if x.shape[1] else x.new_full((x.shape[0], 1), NEG)
    m = torch.where(torch.isneginf(m), 0.0, m)
    p = torch.exp(x - m)
    z = p.sum(1, keepdim=True)
    w = p / torch.where(z > 0, z, 1.0)
    big = mag.amax(1) if x.shape[1] else x.new_zeros(x.shape[0])
    return w @ v, (m + torch.log(z))[:, 0], w @ v.abs(), big


def out_bound(o, a, x, cols, keys):
    e = 1.1 * (2 * (cols + 2) * U * x + 4 * U * x) + 2.0 ** -21
    return 2.0 ** -8 * o.abs() * (1 + 2.0 ** -7) + (2.0 ** -8 + 2 * e[..., None] + 4 * keys * U) * a * (1 + 2.0 ** -7) + 1e-30


def lse_bound(lse, x, cols, keys):
    """The score's error, the sum's, the logarithm's and the final addition's."""
    fin = torch.where(torch.isinf(lse), 0.0, lse)
    return 1.1 * (2 * (cols + 2) * U * x + 4 * U * x) + 2.0 ** -20 + 2 * keys * U + 4 * U * (fin.abs() + x)


def check_attention(out, lse, want, cols, keys, what=""):
    o, l, a, x = want
    err, bound = (out.double() - o).abs(), out_bound(o, a, x, cols, keys)
    assert torch.isfinite(out.float()).all(), what
    assert (err <= bound).all(), (what, float((err / bound).max()))
    if lse is not None:
        same = torch.isneginf(lse) == torch.isneginf(l)
        assert same.all(), what
        d = torch.where(torch.isneginf(l), 0.0, (lse.double() - l).abs())
        assert (d <= lse_bound(l, x, cols, keys)).all(), (what, float(d.max()))


def paged64(q_lat, q_rope, cache, table, lens, cu, scale):
    """out, lse, A, X [T, H, ...] of the absorbed form, a request at a time."""
    t, h, _ = q_lat.shape
    dev = q_lat.device
    out = torch.zeros(t, h, 512, dtype=torch.float64, device=dev)
    a = torch.zeros_like(out)
    lse = torch.full((t, h), NEG, dtype=torch.float64, device=dev)
    x = torch.zeros_like(lse)
    q = torch.cat([q_lat, q_rope], 2)
    page = cache.shape[1]
    for r, n in enumerate(lens):
        c0, c1 = cu[r], cu[r + 1]
        if c1 <= c0:
            continue
        ids = table[r, :-(-n // page)].long()
        k = cache[ids].reshape(-1, 576)[:n] if n else cache.new_zeros(0, 576)
        i = torch.arange(c1 - c0, device=dev)
        see = torch.arange(n, device=dev)[None, :] <= (n - (c1 - c0) + i)[:, None]
        see = see.repeat_interleave(h, 0)
        o, l, aa, xx = attend64(q[c0:c1].reshape(-1, 576), k, k[:, :512], scale, see)
        out[c0:c1], a[c0:c1] = o.view(-1, h, 512), aa.view(-1, h, 512)
        lse[c0:c1], x[c0:c1] = l.view(-1, h), xx.view(-1, h)
    return out, lse, a, x


def expanded64(q_nope, q_rope, k_nope, k_rope, v, cu_q, cu_k, scale, causal):
    t, h, _ = q_nope.shape
    dev = q_nope.device
    out = torch.zeros(t, h, v.shape[2], dtype=torch.float64, device=dev)
    a = torch.zeros_like(out)
    lse = torch.full((t, h), NEG, dtype=torch.float64, device=dev)
    x = torch.zeros_like(lse)
    for r in range(len(cu_q) - 1):
        (a0, a1), (b0, b1) = cu_q[r:r + 2], cu_k[r:r + 2]
        if a1 <= a0:
            continue
        i = torch.arange(a1 - a0, device=dev)[:, None]
        j = torch.arange(b1 - b0, device=dev)[None, :]
        see = (j <= (b1 - b0) - (a1 - a0) + i) if causal else torch.ones_like(i + j, dtype=torch.bool)
        for head in range(h):
            q = torch.cat([q_nope[a0:a1, head], q_rope[a0:a1, head]], 1)
            k = torch.cat([k_nope[b0:b1, head], k_rope[b0:b1]], 1)
            out[a0:a1, head], lse[a0:a1, head], a[a0:a1, head], x[a0:a1, head] = attend64(
                q, k, v[b0:b1, head], scale, see)
    return out, lse, a, x


def tables_plain(ctx, new, page, free, head, table, toks):
    """The step's bookkeeping, a request and a token at a time (Python integers)."""
    table = [list(row) for row in table]
    width, status, nxt = len(table[0]), 0, max(head, 0)
    seq, cu, slots, positions = [], [0], [-1] * toks, [-1] * toks
    for r, (c, n) in enumerate(zip(ctx, new)):
        if c < 0 or n < 0 or c + n > 2 ** 31 - 1:
            status |= 4
        c, n = max(c, 0), max(n, 0)
        n = min(n, 2 ** 31 - 1 - c)
        have, want = -(-c // page), -(-(c + n) // page)
        if want > width:
            status |= 2
        for p in range(have, min(want, width)):
            table[r][p] = free[nxt] if nxt < len(free) else -1
            nxt += 1
        for i in range(n):
            t, pos = cu[-1] + i, c + i
            if t >= toks:
                break
            positions[t] = pos
            if pos // page < width and table[r][pos // page] >= 0:
                slots[t] = table[r][pos // page] * page + pos % page
        seq.append(c + n)
        cu.append(cu[-1] + n)
    status |= (1 if nxt > len(free) else 0) | (4 if cu[-1] > toks else 0)
    return table, seq, cu, slots, positions, min(nxt, len(free)), status


def logprobs64(x, tokens, top):
    """logprob, entropy, ids, their log probabilities, by a stable sort in 64 bits."""
    x = x.double()
    lse = torch.logsumexp(x, 1, keepdim=True)
    lp = x - lse
    p = torch.exp(lp)
    ent = -torch.where(p > 0, p * lp, 0.0).sum(1)
    got = lp.gather(1, tokens.long().clamp(0, x.shape[1] - 1)[:, None])[:, 0]
    order = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :top]
    return got, ent, order, lp.gather(1, order), lse[:, 0]
