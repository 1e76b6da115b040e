"""Thin ctypes binding of the serving operators (include/w8_serve.h): argument
marshalling only, like ``w8``.

What a serving step runs between and after the projections: ``block_tables``
(pages, tables and slot map from the requests' lengths), ``latent_cache_write``,
``latent_attn_paged`` (absorbed form over the paged cache),
``latent_attn_expanded`` (expanded form over a prompt) and ``token_logprobs``.
Every call takes its outputs and its workspace from the caller and is
asynchronous on ``stream`` (default: the current stream).  All tensors are on
the GPU.
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import w8
from .w8 import W8Error

LATENT_DIM, LATENT_ROPE, LATENT_ROW = 512, 64, 576
MAX_REQUESTS, MAX_LATENT_HEADS, MAX_TOP = 16384, 256, 32
LOGITS_BF16, LOGITS_F32 = 1, 2
SERVE_ABI_VERSION = 2  # W8_SERVE_ABI_VERSION of include/w8_serve.h

lib = w8.lib

# every symbol include/w8_serve.h declares
EXPORTS = ("w8_serve_abi_version", "w8_serve_status_str", "w8_serve_device_status",
           "w8_block_tables", "w8_latent_cache_write", "w8_latent_attn_paged",
           "w8_latent_paged_workspace_bytes", "w8_latent_attn_expanded", "w8_token_logprobs",
           "w8_logprobs_workspace_bytes", "w8_logprobs_workspace_bytes_upto")

# the structs of w8_serve.h, packed field by field (native sizes and padding)
_CACHE = struct.Struct("@Pqqii")
_PAGED = struct.Struct("@PqqPqqPqqiiPqPPPqqPiiiif0P")
_EXPANDED = struct.Struct("@PqqPqqPqqPqPqqPPPqqPiiiiiiif0P")


def _load():
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
    st = ctypes.c_int
    lib.w8_serve_abi_version.argtypes = []
    lib.w8_serve_abi_version.restype = i32
    lib.w8_serve_status_str.argtypes = [st]
    lib.w8_serve_status_str.restype = ctypes.c_char_p
    lib.w8_serve_device_status.argtypes = [ctypes.POINTER(ctypes.c_int), i32]
    lib.w8_serve_device_status.restype = st
    lib.w8_block_tables.argtypes = [vp, vp, i32, i32, vp, i32, vp, vp, i64, i32, vp, vp, vp, vp, i32,
                                    vp, vp, vp]
    lib.w8_block_tables.restype = st
    lib.w8_latent_cache_write.argtypes = [vp, i64, vp, i64, vp, i32, ctypes.c_char_p, vp]
    lib.w8_latent_cache_write.restype = st
    lib.w8_latent_attn_paged.argtypes = [ctypes.c_char_p, vp, sz, vp]
    lib.w8_latent_attn_paged.restype = st
    lib.w8_latent_paged_workspace_bytes.argtypes = [i32, i32, i32, i32, ctypes.POINTER(sz)]
    lib.w8_latent_paged_workspace_bytes.restype = st
    lib.w8_latent_attn_expanded.argtypes = [ctypes.c_char_p, vp]
    lib.w8_latent_attn_expanded.restype = st
    lib.w8_token_logprobs.argtypes = [vp, i32, i64, i32, i32, vp, vp, vp, i32, vp, vp, vp, sz, vp]
    lib.w8_token_logprobs.restype = st
    lib.w8_logprobs_workspace_bytes.argtypes = [i32, i32, i32, i32, ctypes.POINTER(sz)]
    lib.w8_logprobs_workspace_bytes.restype = st
    lib.w8_logprobs_workspace_bytes_upto.argtypes = [i32, i32, i32, i32, ctypes.POINTER(sz)]
    lib.w8_logprobs_workspace_bytes_upto.restype = st
    if lib.w8_serve_abi_version() != SERVE_ABI_VERSION:
        raise ImportError(f"{w8.LIB_PATH} has serving ABI {lib.w8_serve_abi_version()}, this "
                          f"binding {SERVE_ABI_VERSION}: rebuild it")


_load()


def _check(status: int):
    if status != 0:
        raise W8Error(status, lib.w8_serve_status_str(status).decode())


def status_str(status: int) -> str:
    return lib.w8_serve_status_str(status).decode()


def device_status(reset: bool = False) -> int:
    """The attention kernels' status word on the current device (0: every
    bounded wait ended normally).  Synchronous with all streams."""
    out = ctypes.c_int(0)
    _check(lib.w8_serve_device_status(ctypes.byref(out), 1 if reset else 0))
    return int(out.value)


# the current stream's handle without a Stream object around it (0.3 us
# instead of 3), where torch offers it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> int:
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:
        return _raw_stream(torch.cuda.current_device())
    return torch.cuda.current_stream().cuda_stream


def _ints(t: torch.Tensor, dtype: torch.dtype = torch.int32, n: int | None = None) -> int:
    assert t.is_cuda and t.dtype == dtype and t.is_contiguous() and (n is None or t.numel() >= n)
    return t.data_ptr()


def _rows(t: torch.Tensor, cols: int) -> tuple[int, int]:
    """Pointer and row stride of a 2-D bf16 operand."""
    row, one = t.stride()
    assert t.is_cuda and t.shape[1] == cols and one == 1 and t.dtype == torch.bfloat16
    return t.data_ptr(), row if t.shape[0] > 1 else cols


def _heads(t: torch.Tensor, toks: int, heads: int, cols: int) -> tuple[int, int, int]:
    """Pointer, token stride and head stride of a bf16 operand [toks, heads, cols]."""
    assert t.is_cuda and t.shape == (toks, heads, cols) and t.dtype == torch.bfloat16
    tok, head, one = t.stride()
    assert one == 1
    # the stride of an axis of one entry says nothing: give one that fits
    head = head if heads > 1 else cols
    return t.data_ptr(), tok if toks > 1 else heads * head, head


def _cache_fields(cache: torch.Tensor) -> tuple:
    page, tok, one = cache.stride()
    n, size, cols = cache.shape
    assert cache.is_cuda and cols == LATENT_ROW and one == 1 and cache.dtype == torch.bfloat16
    tok = tok if size > 1 else LATENT_ROW
    return cache.data_ptr(), page if n > 1 else size * tok, tok, n, size


def _table(t: torch.Tensor, n: int) -> tuple[int, int, int]:
    """Pointer, row stride and width of a page table of at least n rows.  The
    stride goes out as it is: rows that share their storage (expand) are the
    library's to refuse."""
    assert t.is_cuda and t.dim() == 2 and t.stride(1) == 1 and t.dtype == torch.int32 and t.shape[0] >= n
    return t.data_ptr(), t.stride(0) if n > 1 else t.shape[1], t.shape[1]


def _workspace(ws: torch.Tensor | None) -> tuple:
    assert ws is None or ws.is_cuda
    return (None, 0) if ws is None else (ws.data_ptr(), ws.numel() * ws.element_size())


def _device(device) -> torch.device:
    """The GPU of a workspace: a device, its name or its number; None: the current one."""
    if device is None:
        device = torch.cuda.current_device()
    return torch.device("cuda", device) if isinstance(device, int) else torch.device(device)


def _sms(device: torch.device) -> int:
    return torch.cuda.get_device_properties(device).multi_processor_count


def block_tables(ctx_lens: torch.Tensor, new_lens: torch.Tensor, page_size: int,
                 free_pages: torch.Tensor, free_head: torch.Tensor, block_table: torch.Tensor,
                 seq_lens: torch.Tensor, cu_new: torch.Tensor, slots: torch.Tensor,
                 positions: torch.Tensor, free_head_out: torch.Tensor, status: torch.Tensor,
                 stream=None) -> None:
    """Take the pages that the appended tokens need from the free list and
    write the tables, lengths, offsets, slots and positions of the step (one
    kernel launch).  ``status`` is 0 when everything fitted.  No output shares
    memory with an input: ``seq_lens`` are copied to ``ctx_lens`` afterwards."""
    n, toks = ctx_lens.numel(), slots.numel()
    _check(lib.w8_block_tables(
        _ints(ctx_lens), _ints(new_lens, n=n), n, page_size, _ints(free_pages), free_pages.numel(),
        _ints(free_head, n=1), *_table(block_table, n),
        _ints(seq_lens, n=n), _ints(cu_new, n=n + 1), _ints(slots, torch.int64),
        _ints(positions, n=toks), toks, _ints(free_head_out, n=1), _ints(status, n=1),
        _stream(stream)))


def latent_cache_write(latent: torch.Tensor, rope: torch.Tensor, slots: torch.Tensor,
                       cache: torch.Tensor, stream=None) -> torch.Tensor:
    """cache.view(-1, 576)[slots[t]] = [latent[t] | rope[t]]; slots outside the
    cache are skipped (one kernel launch)."""
    n = slots.numel()
    lp, lld = _rows(latent, LATENT_DIM)
    rp, rld = _rows(rope, LATENT_ROPE)
    assert latent.shape[0] >= n and rope.shape[0] >= n
    _check(lib.w8_latent_cache_write(lp, lld, rp, rld, _ints(slots, torch.int64), n,
                                     _CACHE.pack(*_cache_fields(cache)), _stream(stream)))
    return cache


def latent_paged_workspace_bytes(n_tok: int, n_heads: int, n_req: int, sm_count: int) -> int:
    out = ctypes.c_size_t(0)
    _check(lib.w8_latent_paged_workspace_bytes(n_tok, n_heads, n_req, sm_count, ctypes.byref(out)))
    return int(out.value)


def new_latent_paged_workspace(n_tok: int, n_heads: int, n_req: int, device=None) -> torch.Tensor:
    """A workspace for latent_attn_paged calls of up to these counts."""
    device = _device(device)
    nbytes = latent_paged_workspace_bytes(n_tok, n_heads, n_req, _sms(device))
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


def latent_attn_paged(q_lat: torch.Tensor, q_rope: torch.Tensor, cache: torch.Tensor,
                      block_table: torch.Tensor, seq_lens: torch.Tensor, cu_q: torch.Tensor,
                      scale: float, out: torch.Tensor, lse: torch.Tensor | None = None,
                      workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """out[t, h] = softmax(scale (q_lat . c + q_rope . e)) c over the cached
    tokens that query token t sees; q_lat [T, H, 512], q_rope [T, H, 64], cache
    [pages, page_size, 576], out [T, H, 512] (two kernel launches)."""
    toks, heads = q_lat.shape[0], q_lat.shape[1]
    n = seq_lens.numel()
    table, ld_table, width = _table(block_table, n)
    args = _PAGED.pack(
        *_heads(q_lat, toks, heads, LATENT_DIM), *_heads(q_rope, toks, heads, LATENT_ROPE),
        *_cache_fields(cache), table, ld_table,
        _ints(seq_lens), _ints(cu_q, n=n + 1), *_heads(out, toks, heads, LATENT_DIM),
        _ints(lse, torch.float32, toks * heads) if lse is not None else 0,
        width, n, toks, heads, scale)
    _check(lib.w8_latent_attn_paged(args, *_workspace(workspace), _stream(stream)))
    return out


def latent_attn_expanded(q_nope: torch.Tensor, q_rope: torch.Tensor, k_nope: torch.Tensor,
                         k_rope: torch.Tensor, v: torch.Tensor, cu_q: torch.Tensor,
                         cu_k: torch.Tensor, scale: float, causal: bool, out: torch.Tensor,
                         lse: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """out[i, h] = softmax(scale (q_nope . k_nope + q_rope . k_rope)) v over the
    keys of the query's request (one kernel launch)."""
    toks, heads, d_nope = q_nope.shape
    n_k, d_v, n = k_rope.shape[0], v.shape[2], cu_q.numel() - 1
    args = _EXPANDED.pack(
        *_heads(q_nope, toks, heads, d_nope), *_heads(q_rope, toks, heads, LATENT_ROPE),
        *_heads(k_nope, n_k, heads, d_nope), *_rows(k_rope, LATENT_ROPE), *_heads(v, n_k, heads, d_v),
        _ints(cu_q), _ints(cu_k, n=n + 1), *_heads(out, toks, heads, d_v),
        _ints(lse, torch.float32, toks * heads) if lse is not None else 0,
        n, toks, n_k, heads, d_nope, d_v, 1 if causal else 0, scale)
    _check(lib.w8_latent_attn_expanded(args, _stream(stream)))
    return out


def logprobs_workspace_bytes(n_rows: int, vocab: int, top: int, sm_count: int) -> int:
    out = ctypes.c_size_t(0)
    _check(lib.w8_logprobs_workspace_bytes(n_rows, vocab, top, sm_count, ctypes.byref(out)))
    return int(out.value)


def logprobs_workspace_bytes_upto(n_rows: int, vocab: int, top: int, sm_count: int) -> int:
    out = ctypes.c_size_t(0)
    _check(lib.w8_logprobs_workspace_bytes_upto(n_rows, vocab, top, sm_count, ctypes.byref(out)))
    return int(out.value)


def new_logprobs_workspace(n_rows: int, vocab: int, top: int = 0, device=None) -> torch.Tensor:
    """A zero-filled workspace for token_logprobs calls of up to these counts
    (its counters must start at zero)."""
    device = _device(device)
    nbytes = logprobs_workspace_bytes_upto(n_rows, vocab, top, _sms(device))
    return torch.zeros(max(nbytes, 256), dtype=torch.uint8, device=device)


def token_logprobs(logits: torch.Tensor, tokens: torch.Tensor, logprob: torch.Tensor,
                   entropy: torch.Tensor | None = None, top_ids: torch.Tensor | None = None,
                   top_logprobs: torch.Tensor | None = None,
                   workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The log probability of tokens[i] under logits[i] (bf16 or fp32), the
    row's entropy and its top_ids.shape[1] most likely tokens (one kernel
    launch)."""
    assert logits.is_cuda and logits.dim() == 2 and logits.stride(1) == 1
    rows, vocab = logits.shape
    dtype = {torch.bfloat16: LOGITS_BF16, torch.float32: LOGITS_F32}.get(logits.dtype, 0)
    top = 0 if top_ids is None else top_ids.shape[1]
    assert top_ids is None or (top_ids.shape[0] == rows and top_logprobs.shape == top_ids.shape)
    _check(lib.w8_token_logprobs(
        logits.data_ptr(), dtype, logits.stride(0) if rows > 1 else vocab, rows, vocab,
        _ints(tokens, n=rows), _ints(logprob, torch.float32, rows),
        _ints(entropy, torch.float32, rows) if entropy is not None else None, top,
        _ints(top_ids) if top else None, _ints(top_logprobs, torch.float32) if top else None,
        *_workspace(workspace), _stream(stream)))
    return logprob
