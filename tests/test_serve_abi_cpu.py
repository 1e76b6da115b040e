"""Host-side tests of the serving operators' C ABI (no GPU): every function of
w8_serve.h is exported, the packed argument structs have the header's layout,
and every refusal is made before any CUDA call."""
from __future__ import annotations

import os
import re
import subprocess

import pytest

from fp8_weight_only_w8a16_gb300 import serve

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "w8_serve.h")
P = 0x100000  # an aligned address; a refused call never reads it


def test_every_declared_function_is_exported():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"^[A-Za-z_][\w \*]*?\b(w8_\w+)\s*\([^;{]*\)\s*;", text, flags=re.M))
    assert names == set(serve.EXPORTS)
    for name in names:
        assert hasattr(serve.lib, name)
    assert serve.lib.w8_serve_abi_version() == serve.SERVE_ABI_VERSION
    for code in range(16):
        assert serve.status_str(code)


def test_constants_and_struct_layout(tmp_path):
    """Sizes and offsets as a C compiler sees them."""
    src = tmp_path / "s.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "w8_serve.h"\nint main(void) {\n'
                   'printf("%zu %zu %zu ", sizeof(w8_latent_cache), sizeof(w8_latent_paged), sizeof(w8_latent_expanded));\n'
                   'printf("%zu %zu %zu ", offsetof(w8_latent_paged, cache), offsetof(w8_latent_paged, lse), offsetof(w8_latent_paged, scale));\n'
                   'printf("%zu %zu ", offsetof(w8_latent_expanded, cu_q), offsetof(w8_latent_expanded, scale));\n'
                   'printf("%d %d %d %d\\n", W8_MAX_REQUESTS, W8_MAX_LATENT_HEADS, W8_MAX_TOP, W8_LATENT_ROW);\nreturn 0; }\n')
    exe = tmp_path / "s"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got[:3] == [serve._CACHE.size, serve._PAGED.size, serve._EXPANDED.size]
    # a value in each place comes back from there
    raw = serve._PAGED.pack(*range(1, 19), 0, 21, 22, 23, 24, 0.5)
    import struct
    assert struct.unpack_from("@Pqqii", raw, got[3]) == (7, 8, 9, 10, 11)
    assert struct.unpack_from("@f", raw, got[5])[0] == 0.5
    assert struct.unpack_from("@P", raw, got[4])[0] == 0
    raw = serve._EXPANDED.pack(*range(1, 21), 21, 22, 23, 24, 25, 26, 27, 0.25)
    assert struct.unpack_from("@PP", raw, got[6]) == (15, 16)
    assert struct.unpack_from("@f", raw, got[7])[0] == 0.25
    assert got[8:] == [serve.MAX_REQUESTS, serve.MAX_LATENT_HEADS, serve.MAX_TOP, serve.LATENT_ROW]


def status(code):
    return serve.w8.STATUS[code]


TABLES = dict(ctx=P, new=P, n=4, page=16, free=P, n_free=9, head=P, table=P, ld=8, width=8, seq=P, cu=P, slots=P,
              pos=P, toks=5, out=P + 64, status=P)


@pytest.mark.parametrize("kw,want", [
    (dict(n=0), "SHAPE"), (dict(n=16385), "SHAPE"), (dict(n=-1), "SHAPE"), (dict(page=0), "SHAPE"),
    (dict(page=(1 << 20) + 1), "SHAPE"), (dict(n_free=-1), "SHAPE"), (dict(width=0), "SHAPE"),
    (dict(ld=7), "SHAPE"), (dict(toks=-1), "SHAPE"), (dict(toks=(1 << 30) + 1), "SHAPE"),
    (dict(out=P), "SHAPE"), (dict(ctx=None), "NULL"), (dict(new=None), "NULL"), (dict(free=None), "NULL"),
    (dict(head=None), "NULL"), (dict(table=None), "NULL"), (dict(seq=None), "NULL"), (dict(cu=None), "NULL"),
    (dict(slots=None), "NULL"), (dict(pos=None), "NULL"), (dict(out=None), "NULL"), (dict(status=None), "NULL"),
    (dict(slots=P + 4), "ALIGN"), (dict(ctx=P + 2), "ALIGN"), (dict(status=P + 1), "ALIGN")])
def test_block_tables_refusals(kw, want):
    a = {**TABLES, **kw}
    got = serve.lib.w8_block_tables(a["ctx"], a["new"], a["n"], a["page"], a["free"], a["n_free"], a["head"],
                                    a["table"], a["ld"], a["width"], a["seq"], a["cu"], a["slots"], a["pos"],
                                    a["toks"], a["out"], a["status"], None)
    assert status(got) == "W8_ERR_" + want


CACHE = dict(data=P, ld_page=16 * 576, ld_tok=576, pages=4, page=16)
WRITE = dict(lat=P, lld=2624, rope=P, rld=2624, slots=P, n=3)


@pytest.mark.parametrize("kw,cache,want", [
    (dict(n=-1), {}, "SHAPE"), (dict(n=0), {}, "OK"), (dict(n=0, lat=None), {}, "OK"), (dict(lat=None), {}, "NULL"),
    (dict(rope=None), {}, "NULL"), (dict(slots=None), {}, "NULL"), (dict(lld=504), {}, "SHAPE"),
    (dict(rld=56), {}, "SHAPE"), (dict(lld=2620), {}, "ALIGN"), (dict(lat=P + 8), {}, "ALIGN"),
    (dict(rope=P + 2), {}, "ALIGN"), (dict(slots=P + 4), {}, "ALIGN"), ({}, dict(data=None), "NULL"),
    ({}, dict(pages=0), "SHAPE"), ({}, dict(page=0), "SHAPE"), ({}, dict(ld_tok=568), "SHAPE"),
    ({}, dict(ld_page=16 * 576 - 8), "SHAPE"), ({}, dict(ld_tok=580, ld_page=580 * 16), "ALIGN"),
    ({}, dict(data=P + 8), "ALIGN")])
def test_cache_write_refusals(kw, cache, want):
    a, c = {**WRITE, **kw}, {**CACHE, **cache}
    raw = serve._CACHE.pack(c["data"] or 0, c["ld_page"], c["ld_tok"], c["pages"], c["page"])
    got = serve.lib.w8_latent_cache_write(a["lat"], a["lld"], a["rope"], a["rld"], a["slots"], a["n"], raw, None)
    assert status(got) == ("W8_OK" if want == "OK" else "W8_ERR_" + want)


PAGED = dict(q=P, q_t=64 * 512, q_h=512, r=P, r_t=64 * 256, r_h=256, data=P, ld_page=16 * 576, ld_tok=576, pages=4,
             page=16, table=P, ld_table=8, lens=P, cu=P, out=P, o_t=64 * 512, o_h=512, lse=P, width=8, n=4, toks=5,
             heads=64, scale=0.1)


@pytest.mark.parametrize("kw,want", [
    (dict(toks=-1), "SHAPE"), (dict(toks=0), "OK"), (dict(toks=0, q=0, out=0), "OK"), (dict(heads=0), "SHAPE"),
    (dict(heads=257), "SHAPE"), (dict(n=0), "SHAPE"), (dict(n=16385), "SHAPE"), (dict(toks=1 << 25), "SHAPE"),
    (dict(width=0), "SHAPE"), (dict(ld_table=7), "SHAPE"), (dict(scale=0.0), "SCALE"), (dict(scale=-1.0), "SCALE"),
    (dict(scale=float("nan")), "SCALE"), (dict(scale=float("inf")), "SCALE"), (dict(data=0), "NULL"),
    (dict(page=8), "SHAPE"), (dict(page=48, ld_page=48 * 576), "SHAPE"), (dict(page=2048, ld_page=2048 * 576), "SHAPE"),
    (dict(q=0), "NULL"), (dict(r=0), "NULL"), (dict(table=0), "NULL"), (dict(lens=0), "NULL"), (dict(cu=0), "NULL"),
    (dict(out=0), "NULL"), (dict(q_t=504), "SHAPE"), (dict(q_h=504), "SHAPE"), (dict(r_h=60), "SHAPE"),
    (dict(q_h=516), "ALIGN"), (dict(q=P + 8), "ALIGN"), (dict(r=P + 4), "ALIGN"), (dict(r_t=4100), "ALIGN"),
    (dict(o_h=510), "SHAPE"), (dict(o_h=513), "ALIGN"), (dict(out=P + 2), "ALIGN"), (dict(lse=P + 2), "ALIGN"),
    (dict(cu=P + 1), "ALIGN"), (dict(table=P + 2), "ALIGN")])
def test_paged_refusals(kw, want):
    a = {**PAGED, **kw}
    raw = serve._PAGED.pack(a["q"], a["q_t"], a["q_h"], a["r"], a["r_t"], a["r_h"], a["data"], a["ld_page"], a["ld_tok"],
                            a["pages"], a["page"], a["table"], a["ld_table"], a["lens"], a["cu"], a["out"], a["o_t"],
                            a["o_h"], a["lse"], a["width"], a["n"], a["toks"], a["heads"], a["scale"])
    got = serve.lib.w8_latent_attn_paged(raw, P, 1 << 40, None)
    assert status(got) == ("W8_OK" if want == "OK" else "W8_ERR_" + want)


EXPANDED = dict(qn=P, qn_t=64 * 256, qn_h=256, qr=P, qr_t=64 * 256, qr_h=256, kn=P, kn_t=64 * 448, kn_h=448, kr=P,
                kr_t=64, v=P, v_t=64 * 448, v_h=448, cu_q=P, cu_k=P, out=P, o_t=64 * 256, o_h=256, lse=P, n=3, q=7,
                k=9, heads=64, nope=192, dv=256, causal=1, scale=0.1)


@pytest.mark.parametrize("kw,want", [
    (dict(q=0), "OK"), (dict(q=-1), "SHAPE"), (dict(k=-1), "SHAPE"), (dict(n=0), "SHAPE"), (dict(heads=0), "SHAPE"),
    (dict(heads=300), "SHAPE"), (dict(nope=128), "SHAPE"), (dict(dv=128), "SHAPE"), (dict(nope=64, dv=64), "SHAPE"),
    (dict(scale=0.0), "SCALE"), (dict(scale=float("inf")), "SCALE"), (dict(qn=0), "NULL"), (dict(qr=0), "NULL"),
    (dict(kn=0), "NULL"), (dict(kr=0), "NULL"), (dict(v=0), "NULL"), (dict(out=0), "NULL"), (dict(cu_q=0), "NULL"),
    (dict(cu_k=0), "NULL"), (dict(qn_h=184), "SHAPE"), (dict(v_h=248), "SHAPE"), (dict(o_h=248), "SHAPE"),
    (dict(kn_h=452), "ALIGN"), (dict(v=P + 8), "ALIGN"), (dict(out=P + 8), "ALIGN"), (dict(kr_t=68), "ALIGN"),
    (dict(lse=P + 1), "ALIGN"), (dict(cu_q=P + 2), "ALIGN")])
def test_expanded_refusals(kw, want):
    a = {**EXPANDED, **kw}
    raw = serve._EXPANDED.pack(a["qn"], a["qn_t"], a["qn_h"], a["qr"], a["qr_t"], a["qr_h"], a["kn"], a["kn_t"], a["kn_h"],
                               a["kr"], a["kr_t"], a["v"], a["v_t"], a["v_h"], a["cu_q"], a["cu_k"], a["out"], a["o_t"],
                               a["o_h"], a["lse"], a["n"], a["q"], a["k"], a["heads"], a["nope"], a["dv"], a["causal"],
                               a["scale"])
    got = serve.lib.w8_latent_attn_expanded(raw, None)
    assert status(got) == ("W8_OK" if want == "OK" else "W8_ERR_" + want)


LOGPROBS = dict(x=P, dtype=1, ld=1000, rows=4, vocab=1000, tok=P, lp=P, ent=P, top=3, ids=P, tlp=P)


@pytest.mark.parametrize("kw,want", [
    (dict(rows=0), "OK"), (dict(rows=-1), "SHAPE"), (dict(vocab=0), "SHAPE"), (dict(ld=999), "SHAPE"),
    (dict(top=33), "SHAPE"), (dict(top=-1), "SHAPE"), (dict(vocab=2, top=3), "SHAPE"), (dict(dtype=0), "DTYPE"),
    (dict(dtype=3), "DTYPE"), (dict(x=None), "NULL"), (dict(tok=None), "NULL"), (dict(lp=None), "NULL"),
    (dict(ids=None), "NULL"), (dict(tlp=None), "NULL"), (dict(x=P + 1), "ALIGN"), (dict(dtype=2, x=P + 2), "ALIGN"),
    (dict(lp=P + 2), "ALIGN"), (dict(ids=P + 1), "ALIGN")])
def test_logprobs_refusals(kw, want):
    a = {**LOGPROBS, **kw}
    got = serve.lib.w8_token_logprobs(a["x"], a["dtype"], a["ld"], a["rows"], a["vocab"], a["tok"], a["lp"], a["ent"],
                                      a["top"], a["ids"], a["tlp"], P, 1 << 40, None)
    assert status(got) == ("W8_OK" if want == "OK" else "W8_ERR_" + want)


def test_workspace_sizes():
    for sms in (1, 132, 152):
        sizes = [serve.latent_paged_workspace_bytes(t, h, r, sms) for t, h, r in ((0, 1, 1), (1, 64, 1), (512, 128, 256))]
        assert sizes == sorted(sizes)
        assert serve.logprobs_workspace_bytes(0, 154880, 5, sms) == 0
        assert serve.logprobs_workspace_bytes(9000, 154880, 5, sms) == 0  # a CTA a row: nothing to join
    for bad in ((-1, 1, 1, 152), (1, 0, 1, 152), (1, 257, 1, 152), (1, 1, 0, 152), (1, 1, 1, 0), (1 << 25, 64, 1, 152)):
        with pytest.raises(serve.W8Error):
            serve.latent_paged_workspace_bytes(*bad)
    for bad in ((-1, 10, 0, 152), (1, 0, 0, 152), (1, 10, 11, 152), (1, 100, 33, 152), (1, 10, 0, 0)):
        with pytest.raises(serve.W8Error):
            serve.logprobs_workspace_bytes(*bad)
