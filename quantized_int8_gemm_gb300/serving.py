"""Python binding of the serving step around the projections: page tables, K/V
rows into a paged cache, attention over it, verification of drafted tokens.

As in mmq.py these functions only check and marshal arguments; the work is in
the library's kernels and nothing here reads device memory back.  Argument
structs are packed with struct (a call of a decode step is a few microseconds
of host time)."""
from __future__ import annotations

import math
import struct
from typing import NamedTuple

import torch

from .mmq import MMQ_DT_BF16, MMQ_DT_F16, MMQ_DT_F32, _check, load

_TYPES = {torch.float16: MMQ_DT_F16, torch.float32: MMQ_DT_F32, torch.bfloat16: MMQ_DT_BF16}
_I32, _I64, _F32 = torch.int32, torch.int64, torch.float32
# mmq_paged_cache, mmq_attention and mmq_verification of mmq.h
_CACHE = struct.Struct("@QQ7q4i").pack
_ATTENTION = struct.Struct("@6Q7q5if").pack
_VERIFICATION = struct.Struct("@8Q9q2i").pack


def _device(t: torch.Tensor, name: str) -> int:
    """Index of t's device, which has to be the current one."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    dev = t.get_device()
    if dev != torch.cuda.current_device():
        raise ValueError(f"{name} is on device {dev}, the current device is {torch.cuda.current_device()}")
    return dev


def _stream_of(stream, dev: int) -> int:
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _empty(shape, dtype, dev: int, stream):
    """A new tensor that belongs to the stream the call runs on."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(_stream_of(stream, dev), device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


def _ptr(t, name: str, dtype, shape, dev: int) -> int:
    """Address of a contiguous tensor of this type and shape."""
    if not isinstance(t, torch.Tensor) or t.get_device() != dev:
        raise TypeError(f"{name} must be a tensor on CUDA device {dev}")
    if t.dtype != dtype or t.shape != shape:
        raise ValueError(f"{name} must be {dtype} of shape {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _rows3(t, name: str, dev: int):
    """(address, stride 0, stride 1) of a 3-D tensor with contiguous rows."""
    if not isinstance(t, torch.Tensor) or t.get_device() != dev:
        raise TypeError(f"{name} must be a tensor on CUDA device {dev}")
    if t.dim() != 3:
        raise ValueError(f"{name} must have 3 dimensions")
    a, b, c = t.stride()
    if c != 1 and t.shape[2] > 1:
        raise ValueError(f"the last dimension of {name} must be contiguous")
    if (a | b) & 7:  # the stride of a dimension of one element says nothing
        a = 0 if t.shape[0] <= 1 else a
        b = 0 if t.shape[1] <= 1 else b
    return t.data_ptr(), a, b


def _table(t, name: str, nreq: int, dev: int):
    """(address, width, row stride) of the page table."""
    if not isinstance(t, torch.Tensor) or t.get_device() != dev:
        raise TypeError(f"{name} must be a tensor on CUDA device {dev}")
    if t.dtype != _I32 or t.dim() != 2 or t.shape[0] != nreq:
        raise ValueError(f"{name} must be int32 of shape ({nreq}, width)")
    width = t.shape[1]
    row, one = t.stride()
    if one != 1 and width > 1:
        raise ValueError(f"the rows of {name} must be contiguous")
    return t.data_ptr(), width, row if nreq > 1 else max(row, width)


def _cache(k, v, dev: int):
    """The packed mmq_paged_cache of K and V (pages, page_size, heads, head_dim), and its K/V heads, width and type."""
    if not isinstance(k, torch.Tensor) or not isinstance(v, torch.Tensor) or k.get_device() != dev or v.get_device() != dev:
        raise TypeError(f"k_cache and v_cache must be tensors on CUDA device {dev}")
    if k.dim() != 4 or k.shape != v.shape:
        raise ValueError("k_cache and v_cache must be (pages, page_size, heads, head_dim), both the same")
    if k.dtype != v.dtype or k.dtype not in (torch.float16, torch.bfloat16):
        raise ValueError("k_cache and v_cache must both be float16 or bfloat16")
    pages, page, heads, d = k.shape
    ks, vs = k.stride(), v.stride()
    if ks[3] != 1 or vs[3] != 1:
        raise ValueError("the last dimension of the cache must be contiguous")
    if (ks[0] | ks[1] | ks[2] | vs[0] | vs[1] | vs[2]) & 7:
        ks = [0 if n == 1 else s for n, s in zip(k.shape, ks)]
        vs = [0 if n == 1 else s for n, s in zip(k.shape, vs)]
    typ = _TYPES[k.dtype]
    return _CACHE(k.data_ptr(), v.data_ptr(), ks[0], ks[1], ks[2], vs[0], vs[1], vs[2], pages, page, heads, d, typ), heads, d, typ


class PageTables(NamedTuple):
    """What mmq_page_tables gives (or is given to fill)."""

    q_start: torch.Tensor    # (nreq + 1,) int32: first row of each request's new tokens, and their total
    seq_lens: torch.Tensor   # (nreq,) int32: cached + new tokens
    n_blocks: torch.Tensor   # (nreq,) int32: pages held now
    slots: torch.Tensor      # (max_tokens,) int64: slot of each new token, -1 behind the last
    positions: torch.Tensor  # (max_tokens,) int32: its place in its request, -1 behind the last
    taken: torch.Tensor      # (2,) int32: pages taken from the free list, pages missing


def mmq_page_tables(cached_lens: torch.Tensor, new_lens: torch.Tensor, n_blocks: torch.Tensor, block_table: torch.Tensor,
                    free_pages: torch.Tensor, page_size: int, max_tokens: int, out: PageTables | None = None,
                    stream=None) -> PageTables:
    """Pages for each request's new tokens from the front of free_pages (entered into block_table in place), and the
    slot map of the step.  Lengths and pages are int32 CUDA tensors; `out`: buffers to fill instead of new ones."""
    dev = _device(cached_lens, "cached_lens")
    if cached_lens.dim() != 1:
        raise ValueError("cached_lens must have 1 dimension")
    shape = cached_lens.shape
    nreq = shape[0]
    if not isinstance(free_pages, torch.Tensor) or free_pages.dim() != 1:
        raise ValueError("free_pages must be a tensor of 1 dimension")
    if out is None:
        out = PageTables(_empty(nreq + 1, _I32, dev, stream), _empty(nreq, _I32, dev, stream), _empty(nreq, _I32, dev, stream),
                         _empty(max_tokens, _I64, dev, stream), _empty(max_tokens, _I32, dev, stream), _empty(2, _I32, dev, stream))
    q_start, seq_lens, held, slots, positions, taken = out
    table, width, row = _table(block_table, "block_table", nreq, dev)
    _check(load().mmq_page_tables(
        _ptr(cached_lens, "cached_lens", _I32, shape, dev), _ptr(new_lens, "new_lens", _I32, shape, dev),
        _ptr(n_blocks, "n_blocks", _I32, shape, dev), nreq, table, width, row,
        _ptr(free_pages, "free_pages", _I32, free_pages.shape, dev), free_pages.shape[0], page_size, max_tokens,
        _ptr(q_start, "q_start", _I32, (nreq + 1,), dev), _ptr(seq_lens, "seq_lens", _I32, shape, dev),
        _ptr(held, "n_blocks (out)", _I32, shape, dev), _ptr(slots, "slots", _I64, (max_tokens,), dev),
        _ptr(positions, "positions", _I32, (max_tokens,), dev), _ptr(taken, "taken", _I32, (2,), dev),
        _stream_of(stream, dev)), "mmq_page_tables")
    return out if type(out) is PageTables else PageTables(*out)


def mmq_kv_write(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, slots: torch.Tensor,
                 stream=None) -> None:
    """K and V rows (tokens, heads, head_dim; fp32, fp16 or bf16, any row strides) into their slots of the cache
    (pages, page_size, heads, head_dim; fp16 or bf16, any strides but the last).  Slot -1: padding."""
    dev = _device(k, "k")
    cache, heads, d, _ = _cache(k_cache, v_cache, dev)
    kp, kt, kh = _rows3(k, "k", dev)
    vp, vt, vh = _rows3(v, "v", dev)
    n = k.shape[0]
    if k.shape != v.shape or k.dtype != v.dtype or k.dtype not in _TYPES or k.shape[1] != heads or k.shape[2] != d:
        raise ValueError(f"k and v must be (tokens, {heads}, {d}) of one floating type, got {tuple(k.shape)} {k.dtype} and "
                         f"{tuple(v.shape)} {v.dtype}")
    _check(load().mmq_kv_write(cache, kp, kt, kh, vp, vt, vh, _TYPES[k.dtype], _ptr(slots, "slots", _I64, (n,), dev), n,
                               _stream_of(stream, dev)), "mmq_kv_write")


def mmq_paged_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
                        seq_lens: torch.Tensor, q_start: torch.Tensor, *, scale: float | None = None, causal: bool = True,
                        window: int = 0, out: torch.Tensor | None = None, lse: torch.Tensor | bool | None = None,
                        out_dtype: torch.dtype | None = None, stream=None):
    """(out, lse) of each request's new tokens q (tokens, q heads, head_dim) over its pages.  `scale`: 1/sqrt(head_dim)
    if not given; `window` > 0: a token sees that many keys, up to itself; `out`: a buffer, else a new tensor of
    out_dtype (q's type or float32); `lse`: a buffer, True for a new one, or None."""
    dev = _device(q, "q")
    cache, heads, d, typ = _cache(k_cache, v_cache, dev)
    qp, qt, qh = _rows3(q, "q", dev)
    n, hq, dq = q.shape
    if _TYPES.get(q.dtype) != typ or dq != d or hq % heads:
        raise ValueError(f"q must be (tokens, a multiple of {heads}, {d}) of the cache's type, got {tuple(q.shape)} {q.dtype}")
    if out is None:
        out = _empty((n, hq, d), out_dtype or q.dtype, dev, stream)
    elif out.shape != q.shape or (out_dtype is not None and out.dtype != out_dtype):
        raise ValueError(f"out must have shape {tuple(q.shape)}")
    op, ot, oh = _rows3(out, "out", dev)
    if lse is True:
        lse = _empty((n, hq), _F32, dev, stream)
    elif lse is False:
        lse = None
    if not isinstance(seq_lens, torch.Tensor) or seq_lens.dim() != 1:
        raise ValueError("seq_lens must be a tensor of 1 dimension")
    nreq = seq_lens.shape[0]
    table, width, row = _table(block_table, "block_table", nreq, dev)
    args = _ATTENTION(qp, op, 0 if lse is None else _ptr(lse, "lse", _F32, (n, hq), dev), table,
                      _ptr(seq_lens, "seq_lens", _I32, seq_lens.shape, dev), _ptr(q_start, "q_start", _I32, (nreq + 1,), dev),
                      qt, qh, ot, oh, row, nreq, n, width, hq, _TYPES.get(out.dtype, 0), causal, window,
                      1.0 / math.sqrt(d) if scale is None else scale)
    _check(load().mmq_paged_attention(cache, args, _stream_of(stream, dev)), "mmq_paged_attention")
    return out, lse


def mmq_verify_draft(target_probs: torch.Tensor, draft_probs: torch.Tensor | None, draft_tokens: torch.Tensor,
                     n_draft: torch.Tensor | None, u: torch.Tensor, noise: torch.Tensor, stream=None):
    """(tokens (nreq, k + 1) int32, accepted (nreq,) int32): the drafted tokens kept against the target's probabilities
    (nreq, k + 1, vocab), one more token drawn behind them, then -1.  draft_probs (nreq, k, vocab), or None for a draft
    without chance; u (nreq, k) uniform in [0, 1); noise (nreq, vocab) exponential."""
    dev = _device(target_probs, "target_probs")
    tp, tr, tw = _rows3(target_probs, "target_probs", dev)
    nreq, k, vocab = target_probs.shape
    k -= 1
    typ = _TYPES.get(target_probs.dtype, 0)
    dp = dr = dw = 0
    if draft_probs is not None:
        dp, dr, dw = _rows3(draft_probs, "draft_probs", dev)
        if draft_probs.shape != (nreq, k, vocab) or draft_probs.dtype != target_probs.dtype:
            raise ValueError(f"draft_probs must be {target_probs.dtype} of shape {(nreq, k, vocab)}")
    out, accepted = _empty((nreq, k + 1), _I32, dev, stream), _empty(nreq, _I32, dev, stream)
    args = _VERIFICATION(tp, dp, _ptr(draft_tokens, "draft_tokens", _I32, (nreq, k), dev),
                         0 if n_draft is None else _ptr(n_draft, "n_draft", _I32, (nreq,), dev),
                         _ptr(u, "u", _F32, (nreq, k), dev), _ptr(noise, "noise", _F32, (nreq, vocab), dev),
                         out.data_ptr(), accepted.data_ptr(), tr, tw, dr, dw, k, k, vocab, nreq, vocab, k, typ)
    _check(load().mmq_verify_draft(args, _stream_of(stream, dev)), "mmq_verify_draft")
    return out, accepted
