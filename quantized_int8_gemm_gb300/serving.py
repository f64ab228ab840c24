"""Python binding of the serving step around the projections: page tables, K/V
rows into a paged cache, attention over it, verification of drafted tokens.

As in mmq.py these functions only check and marshal arguments (csrc/binding.cpp
does, against the C ABI of mmq.h); the work is in the library's kernels and
nothing here reads device memory back."""
from __future__ import annotations

import ctypes
import importlib.util
import os
from typing import NamedTuple

import torch

from .mmq import MMQError, load

_binding = None


def _load():
    """The compiled binding, bound to the loaded library."""
    global _binding
    from .build import binding_path
    lib = load()
    path = binding_path()
    if not os.path.exists(path):
        raise RuntimeError(f"the serving binding is not built for this Python and torch ({path}); run quantized_int8_gemm_gb300.build.build()")
    spec = importlib.util.spec_from_file_location("quantized_int8_gemm_gb300._serving", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    module.bind(*(ctypes.cast(f, ctypes.c_void_p).value for f in (lib.mmq_page_tables, lib.mmq_kv_write, lib.mmq_paged_attention,
                                                                  lib.mmq_verify_draft)))
    _binding = module
    return module


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
    slot map of the step.  Lengths and pages are int32 CUDA tensors; `out`: buffers to fill instead of new ones, which (like
    block_table) may overlap no other tensor of the call: a step's n_blocks is not the next one's out.n_blocks."""
    got = (_binding or _load()).page_tables(cached_lens, new_lens, n_blocks, block_table, free_pages, page_size, max_tokens, out,
                                            stream)
    rc = got if out is not None else got[0]
    if rc:
        raise MMQError(rc, "mmq_page_tables")
    return out if type(out) is PageTables else PageTables(*(out or got[1]))


def mmq_kv_write(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, slots: torch.Tensor,
                 stream=None) -> None:
    """K and V rows (tokens, heads, head_dim; fp32, fp16 or bf16, any row strides) into their slots of the cache
    (pages, page_size, heads, head_dim; fp16 or bf16, any strides but the last).  Slot -1: padding."""
    rc = (_binding or _load()).kv_write(k, v, k_cache, v_cache, slots, stream)
    if rc:
        raise MMQError(rc, "mmq_kv_write")


def mmq_paged_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
                        seq_lens: torch.Tensor, q_start: torch.Tensor, *, scale: float | None = None, causal: bool = True,
                        window: int = 0, out: torch.Tensor | None = None, lse: torch.Tensor | bool | None = None,
                        out_dtype: torch.dtype | None = None, stream=None):
    """(out, lse) of each request's new tokens q (tokens, q heads, head_dim) over its pages.  `scale`: 1/sqrt(head_dim)
    if not given; `window` > 0: a token sees that many keys, up to itself; `out`: a buffer, else a new tensor of
    out_dtype (q's type or float32); `lse`: a buffer, True for a new one, or None."""
    rc, out, lse = (_binding or _load()).paged_attention(q, k_cache, v_cache, block_table, seq_lens, q_start, scale, causal, window,
                                                         out, lse, out_dtype, stream)
    if rc:
        raise MMQError(rc, "mmq_paged_attention")
    return out, lse


def mmq_verify_draft(target_probs: torch.Tensor, draft_probs: torch.Tensor | None, draft_tokens: torch.Tensor,
                     n_draft: torch.Tensor | None, u: torch.Tensor, noise: torch.Tensor, stream=None):
    """(tokens (nreq, k + 1) int32, accepted (nreq,) int32): the drafted tokens kept against the target's probabilities
    (nreq, k + 1, vocab), one more token drawn behind them, then -1.  draft_probs (nreq, k, vocab), or None for a draft
    without chance; u (nreq, k) uniform in [0, 1); noise (nreq, vocab) exponential."""
    rc, tokens, accepted = (_binding or _load()).verify_draft(target_probs, draft_probs, draft_tokens, n_draft, u, noise, stream)
    if rc:
        raise MMQError(rc, "mmq_verify_draft")
    return tokens, accepted
