"""A serving loop of one attention block on quantized weights: prompts in chunks,
then steps that verify drafted tokens, every step through the library's calls.

    python examples/serving_step.py [--steps N] [--requests B] [--samples S]

One step, for any mixture of requests and new tokens:
  mmq_page_tables      pages and slots for the new tokens, from lengths on the GPU
  mmq_gemm_f32         q, k, v of the new tokens (one fused q4_K projection, fp32)
  mmq_lora             each request's own adapter added to it, as to the other projections (mmq_lora_plan: once a step)
  mmq_kv_write         k, v rows, straight out of the projection's columns, into the paged fp16 cache
  mmq_paged_attention  the new tokens over their requests' pages, fp32 out
  mmq_gemm_f32         output projection (q6_K), then the vocabulary's (q4_K)
  mmq_token_probs      the target's probabilities, under each request's temperature, penalties, biases and mask
  mmq_verify_draft     drafted tokens against them; the accepted counts are the next lengths
  mmq_page_fork        pages that refused drafted tokens took given back; behind the prompts, samples that share their pages
                       (mmq_page_copy: all but the one that the next token goes into)
Lengths, page tables and accepted counts stay on the GPU; the host reads how many pages a step took (and whether any
were missing) and how many are free behind it, to cut its free list, and the tokens to return.  Weights are synthetic, the block has no norm
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

    def __init__(self, hidden=512, q_heads=8, kv_heads=2, head_dim=64, vocab=1000, pages=512, page_size=16, seed=0, adapters=0, rank=16):
        dev = torch.device("cuda")
        self.hq, self.hkv, self.d, self.vocab, self.page = q_heads, kv_heads, head_dim, vocab, page_size

        def weight(qtype, rows, cols, s):
            return mmq.mmq_register_weights(qtype, torch.from_numpy(gen.weights(qtype, rows, cols, s)).to(dev), rows, cols)

        self.qkv = weight("q4_K", (q_heads + 2 * kv_heads) * head_dim, hidden, seed)
        self.out = weight("q6_K", hidden, q_heads * head_dim, seed + 1)
        self.head = weight("q4_K", vocab, hidden, seed + 2)
        g = torch.Generator(device=dev).manual_seed(seed)
        self.embedding = torch.randn((vocab, hidden), generator=g, device=dev)
        self.adapters = adapters
        self.lora = {w: (torch.randn((adapters, rank, i), generator=g, device=dev).div(i ** 0.5).bfloat16(),
                         torch.randn((adapters, o, rank), generator=g, device=dev).div(4.0 * rank ** 0.5).bfloat16())
                     for w, o, i in ((self.qkv, (q_heads + 2 * kv_heads) * head_dim, hidden), (self.out, hidden, q_heads * head_dim),
                                     (self.head, vocab, hidden))}
        self.k, self.v = (torch.zeros((pages, page_size, kv_heads, head_dim), dtype=torch.float16, device=dev) for _ in range(2))

    @staticmethod
    def _unit(x):
        return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)

    def project(self, weights, x: torch.Tensor, plan: mmq.LoraPlan | None) -> torch.Tensor:
        y = mmq.mmq_gemm_f32(weights, x)
        return mmq.mmq_lora(x, y, *self.lora[weights], plan, out=y) if plan else y

    def forward(self, tokens: torch.Tensor, tables: mmq.PageTables, block_table: torch.Tensor, adapters: torch.Tensor | None = None) -> torch.Tensor:
        """Logits (tokens, vocab) of the step's new tokens, in the order of tables.q_start; adapters (requests,): each
        request's, -1 for none."""
        n = tokens.numel()
        plan = mmq.mmq_lora_plan(adapters, tables.q_start, n, self.adapters) if adapters is not None else None
        x = self.embedding[tokens.long()]
        qkv = self._unit(self.project(self.qkv, self._unit(x), plan).view(n, self.hq + 2 * self.hkv, self.d))
        mmq.mmq_kv_write(qkv[:, self.hq:self.hq + self.hkv], qkv[:, self.hq + self.hkv:], self.k, self.v, tables.slots)
        y, _ = mmq.mmq_paged_attention(qkv[:, :self.hq].to(self.k.dtype), self.k, self.v, block_table, tables.seq_lens,
                                       tables.q_start, out_dtype=torch.float32)
        x = self._unit(x) + self._unit(self.project(self.out, y.view(n, -1), plan))
        return 4.0 * self._unit(self.project(self.head, self._unit(x), plan))

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


def pages_of(lens, steps: int, drafted: int = 3, page_size: int = 16, samples: int = 1) -> int:
    """Pages that serve() needs at the most for prompts of these lengths."""
    return samples * sum(-(-(n + steps * (drafted + 1)) // page_size) for n in lens)


def serve(block: Block, prompts: list[torch.Tensor], steps: int = 4, drafted: int = 3, chunk: int = 64, seed: int = 1, samples: int = 1,
          adapters: list[int] | None = None, rules: dict | None = None):
    """Runs the prompts through the block in chunks, then `steps` steps of `drafted` drafted tokens for `samples` samples of
    each.  Returns the samples' tokens (lists, a prompt's next to each other) and the last step's logits of each one's first
    new token.  adapters: each prompt's, -1 for none; rules: what mmq_token_probs takes of each sample (temperature,
    repetition, frequency, presence, bias).  RuntimeError if the block's cache is too small (pages_of)."""
    dev = torch.device("cuda")
    b = len(prompts)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    g = torch.Generator(device=dev).manual_seed(seed)
    longest, pages = max(len(p) for p in prompts) + (drafted + 1) * (steps + 1), block.k.shape[0]
    table = torch.full((b, -(-longest // block.page) + 1), -1, dtype=torch.int32, device=dev)
    free = torch.arange(pages, dtype=torch.int32, device=dev)
    cached, held = i32([0] * b), i32([0] * b)
    with_adapter = i32(adapters) if adapters else None

    def step(new, tokens):
        nonlocal free, held
        t = mmq.mmq_page_tables(cached, new, held, table, free, block.page, tokens.numel())
        taken, missing = t.taken.tolist()
        if missing:
            raise RuntimeError(f"the cache is short of {missing} pages")
        free, held = free[taken:], t.n_blocks
        return t, block.forward(tokens, t, table, with_adapter)

    def keep(parents, lens):  # row i goes on from row parents[i], with its first lens[i] tokens
        nonlocal table, held, free, cached
        f = mmq.mmq_page_fork(table, held, parents, lens, block.page, pages)
        mmq.mmq_page_copy(block.k, block.v, f.pairs, f.tokens)
        listed, missing = f.counts.tolist()
        if missing:
            raise RuntimeError(f"the cache is short of {missing} pages")
        table, held, free, cached = f.block_table, f.n_blocks, f.free_pages[:listed], lens

    done = [0] * b
    while any(done[i] < len(p) for i, p in enumerate(prompts)):  # prompts, a chunk of each at a time
        part = [p[done[i]:done[i] + chunk] for i, p in enumerate(prompts)]
        _, logits = step(i32([len(p) for p in part]), torch.cat(part))
        cached = cached + i32([len(p) for p in part])
        done = [n + len(p) for n, p in zip(done, part)]
    # the samples; the prompt's last token is the first step's first: it is written again, each sample's in its own page
    rows = torch.arange(b, dtype=torch.int32, device=dev).repeat_interleave(samples)
    keep(rows, (cached - 1)[rows])
    with_adapter = with_adapter[rows] if adapters else None
    out = [p.tolist() for p in prompts for _ in range(samples)]
    b = len(out)
    rows = torch.arange(b, dtype=torch.int32, device=dev)
    prompt_lens = i32([len(t) for t in out])
    seen, history = prompt_lens, torch.full((b, longest), -1, dtype=torch.int32, device=dev)
    for row, t in zip(history, out):
        row[:len(t)] = i32(t)
    last = history.gather(1, seen[:, None].long() - 1)[:, 0]
    for _ in range(steps):
        draft, guessed = block.draft(last, drafted, g)
        tokens = torch.cat([last[:, None], draft], 1)
        _, logits = step(i32([drafted + 1] * b), tokens.flatten())
        probs, _ = mmq.mmq_token_probs(logits.view(b, drafted + 1, -1), tokens=history, token_lens=seen, prompt_lens=prompt_lens,
                                       draft_tokens=draft, **(rules or {}))
        kept, accepted = mmq.mmq_verify_draft(probs, guessed, draft, None, torch.rand((b, drafted), generator=g, device=dev),
                                              torch.empty((b, block.vocab), device=dev).exponential_(generator=g))
        keep(rows, cached + accepted + 1)
        last = kept.gather(1, accepted[:, None].long())[:, 0]
        history.scatter_(1, seen[:, None].long() + torch.arange(drafted + 1, device=dev), kept)
        seen = seen + accepted + 1
        for i, row in enumerate(kept.tolist()):
            out[i] += [t for t in row if t >= 0]
    return out, logits.view(b, drafted + 1, -1)[:, 0]


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=8)
    ap.add_argument("--requests", type=int, default=5)
    ap.add_argument("--samples", type=int, default=1, help="of each prompt; the requests take turns over two adapters and none")
    a = ap.parse_args()
    lens = [7 + 53 * i for i in range(a.requests)]
    block = Block(pages=max(1, pages_of(lens, a.steps, samples=a.samples)), adapters=2)
    g = torch.Generator(device="cuda").manual_seed(0)
    prompts = [torch.randint(0, block.vocab, (n,), generator=g, device="cuda", dtype=torch.int32) for n in lens]
    penalties = {"repetition": torch.full((a.requests * a.samples,), 1.1, device="cuda"),
                 "temperature": torch.full((a.requests * a.samples,), 0.8, device="cuda")}
    out, _ = serve(block, prompts, a.steps, samples=a.samples, adapters=[i % 3 - 1 for i in range(a.requests)], rules=penalties)
    for p, t in zip((p for p in prompts for _ in range(a.samples)), out):
        print(f"prompt of {len(p)} tokens, then {len(t) - len(p)}: {t[len(p):]}")
    if mmq.mmq_last_device_error():
        raise SystemExit("a device error was recorded")


if __name__ == "__main__":
    main()
