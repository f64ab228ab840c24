"""The serving example with samples that share their prompt's pages, an adapter for each request and rules on its tokens,
against the same block computed densely in the same calls' order."""
import pytest
import torch

from tests.test_gpu_serving_example import example  # noqa: F401

pytestmark = pytest.mark.gpu


def _prompts(block, lens, seed=7):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randint(0, block.vocab, (n,), generator=g, device="cuda", dtype=torch.int32) for n in lens]


def _dense_logits(mmq, block, tokens, adapter):
    """Logits of one sequence's tokens: attention and adapters in fp64, without pages and plans."""
    def project(w, x):
        y = mmq.mmq_gemm_f32(w, x)
        if adapter >= 0:
            a, b = (m[adapter].double() for m in block.lora[w])
            y = (y.double() + x.double() @ a.T @ b.T).float()
        return y

    x = block.embedding[tokens.long()]
    n = tokens.numel()
    qkv = block._unit(project(block.qkv, block._unit(x)).view(n, -1, block.d)).to(torch.float16).double()
    q, k, v = qkv.split([block.hq, block.hkv, block.hkv], 1)
    rep = block.hq // block.hkv
    s = torch.einsum("ihd,jhd->hij", q, k.repeat_interleave(rep, 1)) / block.d ** 0.5
    s.masked_fill_(torch.ones((n, n), dtype=torch.bool, device=s.device).triu(1), -torch.inf)
    y = torch.einsum("hij,jhd->ihd", torch.softmax(s, -1), v.repeat_interleave(rep, 1)).reshape(n, -1)
    x = block._unit(x) + block._unit(project(block.out, y.float()))
    return 4.0 * block._unit(project(block.head, block._unit(x)))


@pytest.mark.parametrize("page", [16, 5])
def test_samples_with_adapters_agree_with_dense_passes(example, page):  # noqa: F811
    import quantized_int8_gemm_gb300 as mmq
    mmq.mmq_last_device_error()
    lens, ids, samples, steps = (1, 33, 80, 130), [0, -1, 1, 0], 3, 4
    block = example.Block(page_size=page, pages=example.pages_of(lens, steps, page_size=page, samples=samples), adapters=2)
    prompts = _prompts(block, lens)
    kw = dict(samples=samples, adapters=ids)
    out, logits = example.serve(block, prompts, steps=steps, **kw)
    again, _ = example.serve(block, prompts, steps=steps - 1, **kw)
    assert mmq.mmq_last_device_error() == 0
    for i, t in enumerate(again):
        p = prompts[i // samples]
        assert t[:len(p)] == p.tolist() and out[i][:len(t)] == t  # (the same random numbers: the same tokens)
        want = _dense_logits(mmq, block, torch.tensor(t, device="cuda", dtype=torch.int32), ids[i // samples])[-1]
        # attention in fp16 weights against fp64 moves the projections' 8-bit inputs by a step here and there:
        # 1 / 127 of a block's largest value each, on logits of size 4
        assert (logits[i] - want).abs().max() <= 0.15, (i, (logits[i] - want).abs().max())
        assert (logits[i] - want).square().mean().sqrt() <= 0.03
    assert len({tuple(t) for t in out}) == len(out)  # each sample its own


def test_a_request_without_an_adapter_is_served_as_alone(example):  # noqa: F811
    block = example.Block(pages=300, adapters=2)
    prompts = _prompts(block, (20, 40))
    plain, logits = example.serve(block, prompts)
    got, same = example.serve(block, prompts, adapters=[-1, -1])
    assert got == plain and torch.equal(same, logits)


def test_rules_hold_over_the_steps(example):  # noqa: F811
    block = example.Block(pages=300)
    lens, samples = (9, 50), 2
    b, dev = len(lens) * samples, "cuda"
    allowed = torch.zeros(block.vocab, dtype=torch.bool)
    allowed[torch.arange(5, block.vocab, 7)] = True
    bits = torch.nn.functional.pad(allowed, (0, -block.vocab % 32)).view(-1, 32).long()
    words = (bits << torch.arange(32)).sum(1)
    mask = torch.where(words >= 2 ** 31, words - 2 ** 32, words).int().to(dev)[None]
    rules = {"mask": mask, "mask_rows": torch.zeros((b, 4), dtype=torch.int32, device=dev),
             # a penalty larger than any difference of the logits (4 times a unit vector's values): no token twice
             "presence": torch.full((b,), 1e4, device=dev)}
    prompts = _prompts(block, lens)
    out, _ = example.serve(block, prompts, steps=6, samples=samples, rules=rules)
    for i, t in enumerate(out):
        new = t[lens[i // samples]:]
        assert len(new) >= 6 and all(allowed[x] for x in new) and len(set(new)) == len(new)
    # temperature 0: every sample the same tokens
    rules = {"temperature": torch.zeros(b, device=dev)}
    out, _ = example.serve(block, prompts, steps=3, samples=samples, rules=rules)
    for i in range(0, b, samples):
        n = min(len(out[i]), len(out[i + 1]))
        assert out[i][:n] == out[i + 1][:n]


def test_refused_tokens_pages_are_given_back(example):  # noqa: F811
    """Drafted tokens that are never accepted leave no page behind: the pool holds the prompts, one token a step and one
    step's drafted ones, where every step's would not fit."""
    lens, steps, drafted, page = (30, 47), 12, 8, 4
    block = example.Block(pages=sum(-(-(n + steps + drafted) // page) for n in lens), page_size=page)
    mask = torch.full((1, -(-block.vocab // 32)), 0, dtype=torch.int32, device="cuda")
    mask[0, 0] = 1  # token 0 alone: drafted ones are refused (but for a drafted 0)
    rules = {"mask": mask, "mask_rows": torch.zeros((len(lens), drafted + 1), dtype=torch.int32, device="cuda")}
    out, _ = example.serve(block, _prompts(block, lens), steps=steps, drafted=drafted, rules=rules)
    accepted = [len(t) - n - steps for t, n in zip(out, lens)]
    assert all(set(t[n:]) == {0} for t, n in zip(out, lens)) and max(accepted) <= page, accepted
