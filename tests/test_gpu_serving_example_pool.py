"""The serving example's pool of pages: no page is handed out twice, and a pool that is too small is an error."""
import pytest
import torch

from tests.test_gpu_serving_example import example  # noqa: F401

pytestmark = pytest.mark.gpu


def _prompts(block, lens):
    g = torch.Generator(device="cuda").manual_seed(5)
    return [torch.randint(0, block.vocab, (n,), generator=g, device="cuda", dtype=torch.int32) for n in lens]


def test_a_pool_that_is_used_up_is_an_error(example):  # noqa: F811
    block = example.Block(pages=12)
    with pytest.raises(RuntimeError, match="pages"):
        example.serve(block, _prompts(block, (100, 90, 30)), steps=2)


def test_a_pool_of_just_enough_pages_serves_as_a_large_one(example):  # noqa: F811
    lens, steps, drafted = (1, 40, 64, 130), 4, 3
    enough = sum(-(-(n + steps * (drafted + 1)) // 16) for n in lens)
    large = example.Block(pages=500)
    want, logits = example.serve(large, _prompts(large, lens), steps=steps, drafted=drafted)
    block = example.Block(pages=enough)
    got, same = example.serve(block, _prompts(block, lens), steps=steps, drafted=drafted)
    assert got == want and torch.equal(logits, same)


def test_many_requests(example, monkeypatch, capsys):  # noqa: F811
    monkeypatch.setattr("sys.argv", ["serving_step.py", "--steps", "2", "--requests", "20"])
    example.main()
    lines = capsys.readouterr().out.splitlines()
    assert [int(x.split()[2]) for x in lines] == [7 + 53 * i for i in range(20)]
