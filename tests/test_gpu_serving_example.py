"""The serving example's loop against the same block computed densely: every step's cache, tables and attention have to
give what one causal pass over the whole sequence gives."""
import importlib.util
import os

import pytest
import torch

from tests.conftest import ROOT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    from quantized_int8_gemm_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("serving_step", os.path.join(ROOT, "examples", "serving_step.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def _dense_logits(mmq, block, tokens):
    """Logits of one sequence's tokens, attention in fp64 without pages."""
    x = block.embedding[tokens.long()]
    n = tokens.numel()
    qkv = block._unit(mmq.mmq_gemm_f32(block.qkv, block._unit(x)).view(n, -1, block.d)).to(torch.float16).double()
    q, k, v = qkv.split([block.hq, block.hkv, block.hkv], 1)
    rep = block.hq // block.hkv
    s = torch.einsum("ihd,jhd->hij", q, k.repeat_interleave(rep, 1)) / block.d ** 0.5
    s.masked_fill_(torch.ones((n, n), dtype=torch.bool, device=s.device).triu(1), -torch.inf)
    y = torch.einsum("hij,jhd->ihd", torch.softmax(s, -1), v.repeat_interleave(rep, 1)).reshape(n, -1)
    x = block._unit(x) + block._unit(mmq.mmq_gemm_f32(block.out, y.float()))
    return 4.0 * block._unit(mmq.mmq_gemm_f32(block.head, block._unit(x)))


@pytest.mark.parametrize("page", [16, 5])
def test_steps_agree_with_one_dense_pass(example, page):
    import quantized_int8_gemm_gb300 as mmq
    mmq.mmq_last_device_error()
    block = example.Block(page_size=page, pages=700)
    g = torch.Generator(device="cuda").manual_seed(3)
    prompts = [torch.randint(0, block.vocab, (n,), generator=g, device="cuda", dtype=torch.int32) for n in (1, 40, 64, 130, 333)]
    drafted = 3
    out, logits = example.serve(block, prompts, steps=5, drafted=drafted)
    assert mmq.mmq_last_device_error() == 0
    for i, (p, t) in enumerate(zip(prompts, out)):
        assert t[:len(p)] == p.tolist() and len(p) + 5 <= len(t) <= len(p) + 5 * (drafted + 1)
        assert all(0 <= x < block.vocab for x in t)
    # the last step's first token of request i: everything but what that step itself drew
    again, _ = example.serve(block, prompts, steps=4, drafted=drafted)
    for i, t in enumerate(again):
        assert out[i][:len(t)] == t  # (the same random numbers: the same tokens)
        want = _dense_logits(mmq, block, torch.tensor(t, device="cuda", dtype=torch.int32))[-1]
        # attention in fp16 weights against fp64 moves the projections' 8-bit inputs by a step here and there:
        # 1 / 127 of a block's largest value each, on logits of size 4
        assert (logits[i] - want).abs().max() <= 0.15, (i, (logits[i] - want).abs().max())
        assert (logits[i] - want).square().mean().sqrt() <= 0.03
