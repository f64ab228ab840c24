"""A serving loop of one attention block on quantized weights: prompts in chunks,
then steps that verify drafted tokens, every step through the library's calls.

    python examples/serving_step.py [--steps N] [--requests B]

One step, for any mixture of requests and new tokens:
  mmq_page_tables      pages and slots for the new tokens, from lengths on the GPU
  mmq_gemm_f32         q, k, v of the new tokens (one fused q4_K projection, fp32)
  mmq_kv_write         k, v rows, straight out of the projection's columns, into the paged fp16 cache
  mmq_paged_attention  the new tokens over their requests' pages, fp32 out
  mmq_gemm_f32         output projection (q6_K), then the vocabulary's (q4_K)
  mmq_verify_draft     drafted tokens against the target's probabilities; the accepted counts are the next lengths
Lengths, page tables and accepted counts stay on the GPU; the host reads how many pages a step took (and whether any
were missing), to cut them off its free list, and the tokens to return.  Weights are synthetic, the block has no norm
weights and no rotation: it shows the calls, not a trained model."""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import quantized_int8_gemm_gb300 as mmq  # noqa: E402
from synth import gen  # noqa: E402


class Block:
    """Embedding, attention over a paged cache, output and vocabulary projections."""

    def __init__(self, hidden=512, q_heads=8, kv_heads=2, head_dim=64, vocab=1000, pages=512, page_size=16, seed=0):
        dev = torch.device("cuda")
        self.hq, self.hkv, self.d, self.vocab, self.page = q_heads, kv_heads, head_dim, vocab, page_size

        def weight(qtype, rows, cols, s):
            return mmq.mmq_register_weights(qtype, torch.from_numpy(gen.weights(qtype, rows, cols, s)).to(dev), rows, cols)

        self.qkv = weight("q4_K", (q_heads + 2 * kv_heads) * head_dim, hidden, seed)
        self.out = weight("q6_K", hidden, q_heads * head_dim, seed + 1)
        self.head = weight("q4_K", vocab, hidden, seed + 2)
        g = torch.Generator(device=dev).manual_seed(seed)
        self.embedding = torch.randn((vocab, hidden), generator=g, device=dev)
        self.k, self.v = (torch.zeros((pages, page_size, kv_heads, head_dim), dtype=torch.float16, device=dev) for _ in range(2))

    @staticmethod
    def _unit(x):
        return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)

    def forward(self, tokens: torch.Tensor, tables: mmq.PageTables, block_table: torch.Tensor) -> torch.Tensor:
        """Logits (tokens, vocab) of the step's new tokens, in the order of tables.q_start."""
        n = tokens.numel()
        x = self.embedding[tokens.long()]
        qkv = self._unit(mmq.mmq_gemm_f32(self.qkv, self._unit(x)).view(n, self.hq + 2 * self.hkv, self.d))
        mmq.mmq_kv_write(qkv[:, self.hq:self.hq + self.hkv], qkv[:, self.hq + self.hkv:], self.k, self.v, tables.slots)
        y, _ = mmq.mmq_paged_attention(qkv[:, :self.hq].to(self.k.dtype), self.k, self.v, block_table, tables.seq_lens,
                                       tables.q_start, out_dtype=torch.float32)
        x = self._unit(x) + self._unit(mmq.mmq_gemm_f32(self.out, y.view(n, -1)))
        return 4.0 * self._unit(mmq.mmq_gemm_f32(self.head, self._unit(x)))


    def draft(self, last: torch.Tensor, n: int, generator: torch.Generator):
        """n drafted tokens behind each of `last` and the probabilities they were drawn from: the block without its
        attention, a guess from one token to the next."""
        tokens, probs = [], []
        for _ in range(n):
            x = self._unit(self.embedding[last.long()])
            p = torch.softmax(4.0 * self._unit(mmq.mmq_gemm_f32(self.head, x)), -1)
            last = torch.multinomial(p, 1, generator=generator)[:, 0].int()
            tokens.append(last)
            probs.append(p)
        return torch.stack(tokens, 1), torch.stack(probs, 1)


def pages_of(lens, steps: int, drafted: int = 3, page_size: int = 16) -> int:
    """Pages that serve() needs at the most for prompts of these lengths."""
    return sum(-(-(n + steps * (drafted + 1)) // page_size) for n in lens)


def serve(block: Block, prompts: list[torch.Tensor], steps: int = 4, drafted: int = 3, chunk: int = 64, seed: int = 1):
    """Runs the prompts through the block in chunks, then `steps` steps of `drafted` drafted tokens.  Returns the
    requests' tokens (lists) and the last step's logits of each request's first new token.  RuntimeError if the block's
    cache is too small (pages_of)."""
    dev = torch.device("cuda")
    b = len(prompts)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    g = torch.Generator(device=dev).manual_seed(seed)
    width = -(-(max(len(p) for p in prompts) + (drafted + 1) * (steps + 1)) // block.page) + 1
    table = torch.full((b, width), -1, dtype=torch.int32, device=dev)
    free = torch.arange(block.k.shape[0], dtype=torch.int32, device=dev)
    cached, held = i32([0] * b), i32([0] * b)

    def step(new, tokens):
        nonlocal free, held
        t = mmq.mmq_page_tables(cached, new, held, table, free, block.page, tokens.numel())
        taken, missing = t.taken.tolist()
        if missing:
            raise RuntimeError(f"the cache is short of {missing} pages")
        free, held = free[taken:], t.n_blocks
        return t, block.forward(tokens, t, table)

    done = [0] * b
    while any(done[i] < len(p) for i, p in enumerate(prompts)):  # prompts, a chunk of each at a time
        part = [p[done[i]:done[i] + chunk] for i, p in enumerate(prompts)]
        _, logits = step(i32([len(p) for p in part]), torch.cat(part))
        cached = cached + i32([len(p) for p in part])
        done = [n + len(p) for n, p in zip(done, part)]
    out = [p.tolist() for p in prompts]
    last = torch.tensor([t[-1] for t in out], device=dev, dtype=torch.int32)
    cached = cached - 1  # the prompt's last token is the first step's first: it is written again, in its place
    for _ in range(steps):
        draft, guessed = block.draft(last, drafted, g)
        tokens = torch.cat([last[:, None], draft], 1)
        _, logits = step(i32([drafted + 1] * b), tokens.flatten())
        probs = torch.softmax(logits.view(b, drafted + 1, -1), -1)
        kept, accepted = mmq.mmq_verify_draft(probs, guessed, draft, None, torch.rand((b, drafted), generator=g, device=dev),
                                              torch.empty((b, block.vocab), device=dev).exponential_(generator=g))
        cached = cached + accepted + 1  # what follows the accepted tokens in the cache is overwritten by the next step
        last = kept.gather(1, accepted[:, None].long())[:, 0]
        for i, row in enumerate(kept.tolist()):
            out[i] += [t for t in row if t >= 0]
    return out, logits.view(b, drafted + 1, -1)[:, 0]


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=8)
    ap.add_argument("--requests", type=int, default=5)
    a = ap.parse_args()
    lens = [7 + 53 * i for i in range(a.requests)]
    block = Block(pages=max(1, pages_of(lens, a.steps)))
    g = torch.Generator(device="cuda").manual_seed(0)
    prompts = [torch.randint(0, block.vocab, (n,), generator=g, device="cuda", dtype=torch.int32) for n in lens]
    out, _ = serve(block, prompts, a.steps)
    for p, t in zip(prompts, out):
        print(f"prompt of {len(p)} tokens, then {len(t) - len(p)}: {t[len(p):]}")
    if mmq.mmq_last_device_error():
        raise SystemExit("a device error was recorded")


if __name__ == "__main__":
    main()
