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
