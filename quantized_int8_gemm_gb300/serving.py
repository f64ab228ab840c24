"""Python binding of the serving step around the projections: page tables, K/V
rows into a paged cache, attention over it, verification of drafted tokens; and
what differs from request to request: pages shared, given back and copied, rules
on the next token, low-rank adapters.

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
    module.bind(*(ctypes.cast(f, ctypes.c_void_p).value for f in (
        lib.mmq_page_tables, lib.mmq_kv_write, lib.mmq_paged_attention, lib.mmq_verify_draft, lib.mmq_page_fork, lib.mmq_page_compact,
        lib.mmq_page_copy, lib.mmq_token_probs, lib.mmq_lora_plan_words, lib.mmq_lora_plan, lib.mmq_lora)))
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


class PageFork(NamedTuple):
    """What mmq_page_fork gives (or is given to fill)."""

    block_table: torch.Tensor  # (new rows, width) int32: the rows' pages, then -1
    n_blocks: torch.Tensor     # (new rows,) int32: pages held
    pairs: torch.Tensor        # (new rows, 2) int32: page to copy and its copy, -1 -1 for a row without one
    tokens: torch.Tensor       # (new rows,) int32: tokens to copy
    free_pages: torch.Tensor   # (n_pages,) int32: pages that no row holds, ascending, then -1
    counts: torch.Tensor       # (2,) int32: entries of free_pages, copies that found no free page


def mmq_page_fork(block_table: torch.Tensor, n_blocks: torch.Tensor, parents: torch.Tensor, lens: torch.Tensor, page_size: int,
                  n_pages: int, out: PageFork | None = None, stream=None) -> PageFork:
    """The page table's rows made anew: row b continues row parents[b] (-1: empty) with its first lens[b] tokens.  Full pages
    may be shared by rows; the page that a row's next token goes into is its own, a copy where another row has it too
    (mmq_page_copy(k_cache, v_cache, f.pairs, f.tokens) makes them).  Pages of no row are free.  `out` may overlap no other
    tensor of the call."""
    got = (_binding or _load()).page_fork(block_table, n_blocks, parents, lens, page_size, n_pages, out, stream)
    rc = got if out is not None else got[0]
    if rc:
        raise MMQError(rc, "mmq_page_fork")
    return out if type(out) is PageFork else PageFork(*(out or got[1]))


class PageMoves(NamedTuple):
    """What mmq_page_compact gives (or is given to fill)."""

    block_table: torch.Tensor  # (requests, width) int32: the table after the moves, -1 behind a row's pages
    pairs: torch.Tensor        # (n_pages // 2, 2) int32: from, to; then -1 -1
    counts: torch.Tensor       # (2,) int32: pages held, moves


def mmq_page_compact(block_table: torch.Tensor, n_blocks: torch.Tensor, n_pages: int, out: PageMoves | None = None,
                     stream=None) -> PageMoves:
    """Moves that bring the held pages to the front of the cache (mmq_page_copy(k_cache, v_cache, m.pairs) makes them); behind
    them pages counts[0] .. n_pages - 1 are free.  `out` may overlap no other tensor of the call."""
    got = (_binding or _load()).page_compact(block_table, n_blocks, n_pages, out, stream)
    rc = got if out is not None else got[0]
    if rc:
        raise MMQError(rc, "mmq_page_compact")
    return out if type(out) is PageMoves else PageMoves(*(out or got[1]))


def mmq_page_copy(k_cache: torch.Tensor, v_cache: torch.Tensor, pairs: torch.Tensor, tokens: torch.Tensor | None = None,
                  stream=None) -> None:
    """Page pairs[i, 0] of K and V to page pairs[i, 1], its first tokens[i] tokens or all of it; a negative id copies nothing."""
    rc = (_binding or _load()).page_copy(k_cache, v_cache, pairs, tokens, stream)
    if rc:
        raise MMQError(rc, "mmq_page_copy")


def mmq_token_probs(logits: torch.Tensor, *, temperature: torch.Tensor | None = None, tokens: torch.Tensor | None = None,
                    token_lens: torch.Tensor | None = None, prompt_lens: torch.Tensor | None = None,
                    draft_tokens: torch.Tensor | None = None, n_draft: torch.Tensor | None = None,
                    repetition: torch.Tensor | None = None, frequency: torch.Tensor | None = None,
                    presence: torch.Tensor | None = None, bias: tuple | None = None, mask: torch.Tensor | None = None,
                    mask_rows: torch.Tensor | None = None, probs: torch.Tensor | bool | None = True,
                    adjusted: torch.Tensor | bool | None = None, stream=None):
    """(probs, adjusted): probabilities, as mmq_verify_draft reads them, and adjusted logits of logits (nreq, k + 1, vocab) under
    each request's rules.  Row i stands behind the request's tokens (nreq, width; the first token_lens, of which prompt_lens are
    the prompt's) and its first i draft_tokens (nreq, k).  repetition, frequency, presence, temperature (0: greedy): float32,
    one a request.  bias: (start (nreq + 1), ids, values): request b's are start[b] .. start[b + 1] - 1.  mask (masks,
    ceil(vocab / 32)) int32, bit v % 32 of word v // 32 allows token v; mask_rows (nreq, k + 1): each row's mask, -1 for none.
    n_draft: rows past it are left as they are.  probs, adjusted: a buffer, True for a new float32 one, or None; adjusted may
    be logits itself."""
    rc, probs, adjusted = (_binding or _load()).token_probs(logits, temperature, tokens, token_lens, prompt_lens, draft_tokens, n_draft,
                                                            repetition, frequency, presence, bias, mask, mask_rows, probs, adjusted,
                                                            stream)
    if rc:
        raise MMQError(rc, "mmq_token_probs")
    return probs, adjusted


class LoraPlan(NamedTuple):
    """The tokens of a step in the order of their adapters (mmq_lora_plan), for all its mmq_lora calls."""

    words: torch.Tensor  # int32
    tokens: int          # rows of x and y
    requests: int
    adapters: int


def mmq_lora_plan(adapters: torch.Tensor, q_start: torch.Tensor, max_tokens: int, n_adapters: int,
                  out: torch.Tensor | None = None, stream=None) -> LoraPlan:
    """adapters (nreq,) int32: each request's adapter, -1 for none; q_start (nreq + 1,) int32: its first token row, as
    mmq_page_tables gives it; max_tokens: rows of x and y.  `out`: the words of an earlier plan of the same sizes, to fill."""
    rc, words = (_binding or _load()).lora_plan(adapters, q_start, max_tokens, n_adapters, out, stream)
    if rc:
        raise MMQError(rc, "mmq_lora_plan")
    return LoraPlan(words, max_tokens, adapters.shape[0], n_adapters)


def mmq_lora(x: torch.Tensor, y: torch.Tensor, a: torch.Tensor, b: torch.Tensor, plan: LoraPlan, *, scales: torch.Tensor | None = None,
             ranks: torch.Tensor | None = None, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y (tokens, od) float32 plus scale * (x a^T) b^T of each token's adapter: x (tokens, id) float32, float16 or bfloat16;
    a (adapters, rank, id), b (adapters, od, rank) float16 or bfloat16; scales, ranks: one an adapter.  `out`: y itself (the
    adapters are added in place), another buffer, or None for a new tensor."""
    words, tokens, requests, adapters = plan
    rc, out = (_binding or _load()).lora(x, y, a, b, words, tokens, requests, adapters, scales, ranks, out, stream)
    if rc:
        raise MMQError(rc, "mmq_lora")
    return out
