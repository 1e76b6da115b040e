"""Host-side tests of the serving operators' binding (no GPU): what it hands to
the library, seen by a stand-in for the library that records its arguments."""
from __future__ import annotations

import pytest
import torch

from fp8_weight_only_w8a16_gb300 import serve


class OnGpu(torch.Tensor):
    """A host tensor that the binding takes for one on the GPU."""
    is_cuda = True


def on_gpu(t):
    return t.as_subclass(OnGpu)


def i32(*shape):
    return on_gpu(torch.zeros(*shape, dtype=torch.int32))


def bf16(*shape):
    return on_gpu(torch.zeros(*shape, dtype=torch.bfloat16))


@pytest.fixture
def calls(monkeypatch):
    """Each call's function name and arguments."""
    seen = []

    class Library:
        def __getattr__(self, name):
            def call(*args):
                seen.append((name, args))
                return 0
            return call

    monkeypatch.setattr(serve, "lib", Library())
    monkeypatch.setattr(serve, "_stream", lambda stream: None)
    return seen


def tables(table, n):
    serve.block_tables(i32(n), i32(n), 16, i32(9), i32(1), table, i32(n), i32(n + 1),
                       on_gpu(torch.zeros(5, dtype=torch.int64)), i32(5), i32(1), i32(1))


def paged(table, n):
    serve.latent_attn_paged(bf16(n, 2, 512), bf16(n, 2, 64), bf16(4, 16, 576), table, i32(n), i32(n + 1), 0.1,
                            bf16(n, 2, 512))


def strides(calls, call, table, n):
    """ld_table and max_pages as the library gets them."""
    call(table, n)
    (name, args), = calls
    if name == "w8_block_tables":
        return args[8], args[9]
    fields = serve._PAGED.unpack(args[0])
    return fields[12], fields[19]


@pytest.mark.parametrize("call", [tables, paged])
@pytest.mark.parametrize("table,n,want", [
    (i32(10).expand(8, -1), 8, (0, 10)),  # one row for eight requests: no stride that fits is made up
    (i32(40).as_strided((8, 10), (4, 1)), 8, (4, 10)),
    (i32(8, 10), 8, (10, 10)), (i32(8, 16)[:, :10], 8, (16, 10)), (i32(8, 10), 3, (10, 10)),
    (i32(10).expand(1, -1), 1, (10, 10)), (i32(10).expand(8, -1), 1, (10, 10))])
def test_table_stride_is_the_tensors_own(calls, call, table, n, want):
    """The table's row stride goes to the library as it is (which refuses one below the width), except
    where there is one row."""
    assert strides(calls, call, table, n) == want


# every call with small operands, by name
OPERANDS = {
    "block_tables": lambda: dict(
        ctx_lens=i32(3), new_lens=i32(3), page_size=16, free_pages=i32(9), free_head=i32(1), block_table=i32(3, 4),
        seq_lens=i32(3), cu_new=i32(4), slots=on_gpu(torch.zeros(5, dtype=torch.int64)), positions=i32(5),
        free_head_out=i32(1), status=i32(1)),
    "latent_cache_write": lambda: dict(
        latent=bf16(5, 512), rope=bf16(5, 64), slots=on_gpu(torch.zeros(5, dtype=torch.int64)), cache=bf16(4, 16, 576)),
    "latent_attn_paged": lambda: dict(
        q_lat=bf16(3, 2, 512), q_rope=bf16(3, 2, 64), cache=bf16(4, 16, 576), block_table=i32(3, 4), seq_lens=i32(3),
        cu_q=i32(4), scale=0.1, out=bf16(3, 2, 512), lse=on_gpu(torch.zeros(3, 2)),
        workspace=on_gpu(torch.zeros(256, dtype=torch.uint8))),
    "latent_attn_expanded": lambda: dict(
        q_nope=bf16(3, 2, 128), q_rope=bf16(3, 2, 64), k_nope=bf16(5, 2, 128), k_rope=bf16(5, 64), v=bf16(5, 2, 128),
        cu_q=i32(3), cu_k=i32(3), scale=0.1, causal=True, out=bf16(3, 2, 128), lse=on_gpu(torch.zeros(3, 2))),
    "token_logprobs": lambda: dict(
        logits=bf16(2, 100), tokens=i32(2), logprob=on_gpu(torch.zeros(2)), entropy=on_gpu(torch.zeros(2)), top_ids=i32(2, 3),
        top_logprobs=on_gpu(torch.zeros(2, 3)), workspace=on_gpu(torch.zeros(256, dtype=torch.uint8))),
}
TENSORS = [(f, k) for f, make in OPERANDS.items() for k, v in make().items() if isinstance(v, torch.Tensor)]


@pytest.mark.parametrize("name", OPERANDS)
def test_operands_reach_the_library(calls, name):
    getattr(serve, name)(**OPERANDS[name]())
    assert [c[0] for c in calls] == ["w8_" + name]


@pytest.mark.parametrize("name,operand", TENSORS)
def test_host_tensors_are_refused(calls, name, operand):
    """A tensor on the host is no device pointer: the library is not called."""
    args = OPERANDS[name]()
    args[operand] = args[operand].as_subclass(torch.Tensor)
    with pytest.raises(AssertionError):
        getattr(serve, name)(**args)
    assert not calls


@pytest.mark.parametrize("name,operand", [(f, k) for f, k in TENSORS if k != "logits" and OPERANDS[f]()[k].dtype == torch.bfloat16])
@pytest.mark.parametrize("dtype", [torch.float16, torch.int16, torch.float32])
def test_other_types_than_bf16_are_refused(calls, name, operand, dtype):
    """16 bits of another type would be read as bf16."""
    args = OPERANDS[name]()
    args[operand] = on_gpu(torch.zeros(args[operand].shape, dtype=dtype))
    with pytest.raises(AssertionError):
        getattr(serve, name)(**args)
    assert not calls


def test_logits_of_another_type_are_refused(monkeypatch):
    """The library tells the logits' type by a code; fp16 has none."""
    monkeypatch.setattr(serve, "_stream", lambda stream: None)
    args = OPERANDS["token_logprobs"]()
    args["logits"] = on_gpu(torch.zeros(2, 100, dtype=torch.float16))
    with pytest.raises(serve.W8Error):
        serve.token_logprobs(**args)


@pytest.mark.parametrize("device,want", [
    (0, "cuda:0"), (1, "cuda:1"), (2, "cuda:2"), (None, "cuda:1"), ("cuda:0", "cuda:0"), (torch.device("cuda", 0), "cuda:0")])
def test_workspaces_are_made_for_the_device_that_is_named(monkeypatch, device, want):
    """... and sized for its SMs, device 0 too, with device 1 the current one."""
    made = []
    sms = {0: 10, 1: 152, 2: 80}

    class Properties:
        def __init__(self, device):
            self.multi_processor_count = sms[torch.device(device).index if not isinstance(device, int) else device]

    def make(n, dtype, device):
        made.append((n, str(device)))

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    monkeypatch.setattr(torch.cuda, "get_device_properties", Properties)
    monkeypatch.setattr(torch, "empty", make)
    monkeypatch.setattr(torch, "zeros", make)
    serve.new_latent_paged_workspace(4, 64, 2, device=device)
    serve.new_logprobs_workspace(2, 154880, 5, device=device)
    n = sms[torch.device(want).index]
    assert [d for _, d in made] == [want] * 2
    assert made[0][0] == serve.latent_paged_workspace_bytes(4, 64, 2, n)
    assert made[1][0] >= serve.logprobs_workspace_bytes(2, 154880, 5, n)


def test_the_stride_of_one_entry_says_nothing(calls):
    """One token, one head, one page, a page of one token: a stride that is no multiple of 8, or none at
    all, comes with a slice or an expand of such an axis and refuses nothing."""
    def one(*shape):  # its first axis an odd number of elements apart, and one entry long
        n = 1
        for x in shape[1:]:
            n *= x
        return on_gpu(torch.zeros(2 * n + 13, dtype=torch.bfloat16).as_strided(shape, (n + 13,) + torch.empty(shape).stride()[1:]))

    serve.latent_attn_paged(one(1, 3, 512), one(1, 3, 64), one(1, 16, 576), i32(1, 4), i32(1), i32(2), 0.1, one(1, 3, 512))
    serve.latent_attn_paged(one(1, 3, 512).transpose(0, 1), one(1, 3, 64).transpose(0, 1), one(1, 4, 576).transpose(0, 1),
                            i32(1, 4), i32(1), i32(2), 0.1, one(1, 3, 512).transpose(0, 1))
    serve.latent_attn_expanded(one(1, 3, 128), one(1, 3, 64), one(1, 3, 128), one(1, 64), one(1, 3, 128), i32(2), i32(2),
                               0.1, True, one(1, 3, 128))
    serve.latent_cache_write(one(1, 512), one(1, 64), on_gpu(torch.zeros(1, dtype=torch.int64)), one(1, 16, 576))
    serve.latent_attn_paged(bf16(1, 512).expand(1, 1, 512), bf16(64).expand(1, 1, 64), bf16(16, 576).expand(1, 16, 576),
                            i32(1, 4), i32(1), i32(2), 0.1, bf16(1, 1, 512))
    a, b, c, d, e = (args for _, args in calls)
    pack = serve._PAGED.unpack
    assert pack(a[0])[1:3] == (1536, 512) and pack(a[0])[4:6] == (192, 64) and pack(a[0])[7:9] == (16 * 576, 576)
    assert pack(b[0])[1:3] == (512, 512) and pack(b[0])[4:6] == (64, 64) and pack(b[0])[7:9] == (576, 576)
    fields = serve._EXPANDED.unpack(c[0])
    assert fields[1:3] == (384, 128) and fields[4:6] == (192, 64) and fields[7:9] == (384, 128) and fields[10] == 64
    assert d[1] == 512 and d[3] == 64
    assert pack(e[0])[1:3] == (512, 512) and pack(e[0])[7:9] == (16 * 576, 576)


# ---------------------------------------------------------------------------
# outputs of the bookkeeping that lie on its inputs: refused before any CUDA call
# ---------------------------------------------------------------------------

N, FREE, TOKS, WIDTH, LD = 2000, 700, 3000, 20, 40
BUFFERS = dict(ctx=4 * N, new=4 * N, free=4 * FREE, head=4, table=4 * ((N - 1) * LD + WIDTH), seq=4 * N, cu=4 * (N + 1),
               slots=8 * TOKS, pos=4 * TOKS, out=4, status=4)
PLACES = {name: 0x1000000 * (i + 1) for i, name in enumerate(BUFFERS)}
INPUTS, OUTPUTS = ("ctx", "new", "free", "head"), ("table", "seq", "cu", "slots", "pos", "out", "status")


def on_inputs():
    for i in INPUTS:
        for o in OUTPUTS:
            step = 8 if o == "slots" else 4
            last = BUFFERS[o] - step
            yield i, o, PLACES[i]                                    # the same address
            yield i, o, (PLACES[i] - last) // step * step            # the output's last entry on the input's first
            yield i, o, (PLACES[i] + BUFFERS[i] - 4) // step * step  # its first on the input's last
            if o == "table":  # a row in the middle
                yield i, o, PLACES[i] - 4 * LD * 1000 - 4 * (WIDTH - 1)


@pytest.mark.parametrize("i,o,at", list(on_inputs()))
def test_tables_outputs_on_inputs_are_refused(i, o, at):
    p = {**PLACES, o: at}
    got = serve.lib.w8_block_tables(p["ctx"], p["new"], N, 16, p["free"], FREE, p["head"], p["table"], LD, WIDTH, p["seq"],
                                    p["cu"], p["slots"], p["pos"], TOKS, p["out"], p["status"], None)
    assert serve.w8.STATUS[got] == "W8_ERR_SHAPE"


@pytest.mark.parametrize("sms", [1, 132, 152])
@pytest.mark.parametrize("vocab", [1, 4097, 32003, 154880])
def test_a_workspace_serves_every_smaller_call(sms, vocab):
    """Fewer rows need more bytes than many: a workspace is sized for the worst of them."""
    need = [0] + [serve.logprobs_workspace_bytes(r, vocab, 1, sms) for r in range(1, 1400)]
    worst = 0
    for r in range(1, 1400):
        worst = max(worst, need[r])
        assert serve.logprobs_workspace_bytes_upto(r, vocab, 1, sms) == worst
    for smaller in (1, 100, 4096, 5000, 30000, 100000):
        if smaller < vocab:
            for r in (1, 2, 37, 300, 1399):
                assert serve.logprobs_workspace_bytes(r, smaller, 1, sms) <= serve.logprobs_workspace_bytes_upto(r, vocab, 1, sms)
    with pytest.raises(serve.W8Error):
        serve.logprobs_workspace_bytes_upto(-1, vocab, 0, sms)


def test_new_workspaces_serve_every_smaller_call(monkeypatch):
    class Properties:
        multi_processor_count = 152

    made = []
    monkeypatch.setattr(torch.cuda, "get_device_properties", lambda device: Properties)
    monkeypatch.setattr(torch, "zeros", lambda n, **kw: made.append(n))
    for rows in (1, 304, 305, 9000):
        serve.new_logprobs_workspace(rows, 154880, 5, device=0)
        assert made[-1] >= max(serve.logprobs_workspace_bytes(r, 154880, 5, 152) for r in range(1, rows + 1))
