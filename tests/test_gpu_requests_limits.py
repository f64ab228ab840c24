"""What differs from request to request in a step, on the GPU, at the limits of its arguments: logits far from 0, calls of
several threads; and all bits of the adapters' inputs.  Tolerances are those of tests/test_gpu_requests.py, derived there, unless a test says others."""
import ctypes
import math
import threading

import pytest
import torch

from tests.test_gpu_requests import BF16, F16, F32, _check_rules, _f32, _i32, _no_device_error, _rules_problem, mmq  # noqa: F401
from tests.test_requests_host import Fork, Lora, Rules, i64, vp

pytestmark = pytest.mark.gpu

# ---------------------------------------------------------------- logits far below 0
# (b, k, v): rows enough for slices of more than 4096 tokens, which a thread goes over in several parts, the last of them too
# short for most threads: 160 rows of 50257 go by slices of 12576 in fp32 and in 16 bits.
SEVERAL_PARTS = [(40, 3, 50257), (160, 0, 100277)]


def _far(p, shift, temperature=None):
    p["logits"] = (p["logits"].float() + shift).to(p["logits"].dtype)
    if temperature:
        p["temperature"] = _f32([temperature] * p["logits"].shape[0])
    return p


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("b,k,v", SEVERAL_PARTS)
@pytest.mark.parametrize("shift,temperature", [(-100.0, 1.0), (-1000.0, 1.0), (-20.0, 0.05), (1000.0, 1.0)])
def test_probs_of_logits_far_from_zero(mmq, b, k, v, dtype, shift, temperature):  # noqa: F811
    """The parts of a row that a thread has nothing of add nothing, whatever the largest logit is."""
    p = _rules_problem(b, k, v, dtype, seed=v, masks=0, bias=0, hist=0)
    _check_rules(mmq, _far({"logits": p["logits"]}, shift, temperature))


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("b,k,v", [(3, 2, 1000), (2, 1, 10007), *SEVERAL_PARTS[:1]])
@pytest.mark.parametrize("shift", [-100.0, -1000.0])
def test_probs_of_masked_logits_far_below_zero(mmq, b, k, v, dtype, shift):  # noqa: F811
    """Tokens that a mask hides, that have a place of their own outside the stream or that are -inf themselves stand in whole
    fours: their probabilities are 0 and their own, not NaN."""
    p = _far(_rules_problem(b, k, v, dtype, seed=v), shift)
    p["logits"][..., 128:512] = -math.inf
    ids, values = list(range(600, 640)) * b, [0.25 * (i % 7) for i in range(40 * b)]
    p["bias"] = (_i32([40 * i for i in range(b + 1)]), _i32(ids), _f32(values))
    for temperature in (None, 0.05):
        _check_rules(mmq, _far(p, 0.0, temperature))


# ---------------------------------------------------------------- terms of the adapters' operands
def _terms(x, n):  # the sum of n bf16 terms, each what rounding to nearest leaves of those before
    left, got = x.clone(), torch.zeros_like(x, dtype=torch.float64)
    for _ in range(n):
        term = left.to(BF16).float()
        got, left = got + term.double(), left - term
    return got


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("rank", [8, 32, 72])
@pytest.mark.parametrize("tokens", [5, 700, 3000])  # (the kernels of few tokens, of tiles of 16 and of 64)
def test_lora_holds_all_bits_of_x(mmq, tokens, rank, dtype):  # noqa: F811
    """Weights of one 1 a row: out is x's columns, through both products.  Three terms hold an fp32 number's 24 bits, so each
    product's sum is the number itself, cut off at most at the last bit of its first term, 2^-23 of up to twice the number
    (2^-22), twice: 2^-21.  Two terms would leave up to 2^-18."""
    g = torch.Generator(device="cuda").manual_seed(rank)
    x = torch.randn((tokens, 520), generator=g, device="cuda")
    a, b = torch.zeros((1, rank, 520), dtype=dtype, device="cuda"), torch.eye(rank, device="cuda").to(dtype)[None].contiguous()
    columns = torch.arange(rank, device="cuda") * 7
    a[0, torch.arange(rank, device="cuda"), columns] = 1
    want = x[:, columns].double()
    assert torch.equal(_terms(x[:, columns], 3), want)
    assert ((_terms(x[:, columns], 2) - want).abs() > 2.0 ** -20 * want.abs()).any()
    got = mmq.mmq_lora(x, torch.zeros((tokens, rank), device="cuda"), a, b, mmq.mmq_lora_plan(_i32([0]), _i32([0, tokens]), tokens, 1))
    assert ((got.double() - want).abs() <= 2.0 ** -21 * want.abs()).all()


# ---------------------------------------------------------------- threads
def _call(lib, name, *args):
    f = getattr(lib, name)
    return lambda stream: f(*args, stream)


def _rules_call(lib, b, v, tokens):
    logits, probs = torch.zeros((b, v), device="cuda"), torch.empty((b, v), device="cuda")
    said, rho = torch.zeros((b, 4), dtype=torch.int32, device="cuda"), torch.ones(b, device="cuda")
    t = Rules(logits=logits.data_ptr(), probs=probs.data_ptr(), logits_req=v, logits_row=v, probs_req=v, probs_row=v, nreq=b, vocab=v, rows=1,
              type=2, probs_type=2)
    if tokens:
        t.tokens, t.tokens_stride, t.tokens_width, t.repetition = said.data_ptr(), 4, 4, rho.data_ptr()
    return _call(lib, "mmq_token_probs", ctypes.byref(t)), (logits, probs, said, rho)


def _fork_call(lib, pages):
    table, one, zero = _i32([[0]]), _i32([1]), _i32([0])
    out = [torch.empty(n, dtype=torch.int32, device="cuda") for n in (1, 1, 2, 1, pages, 2)]
    f = Fork(**dict(zip(("new_table", "held_out", "pairs", "tokens", "free_pages", "counts"), (x.data_ptr() for x in out))), table=table.data_ptr(),
             held=one.data_ptr(), parents=zero.data_ptr(), lens=one.data_ptr(), nold=1, nnew=1, table_width=1, table_stride=1, new_stride=1,
             npages=pages, page_size=16)
    return _call(lib, "mmq_page_fork", ctypes.byref(f)), (table, one, zero, *out)


def _compact_call(lib, pages):
    table, held = _i32([[0]]), _i32([1])
    out = [torch.empty(n, dtype=torch.int32, device="cuda") for n in (1, pages, 2)]
    p = [vp(x.data_ptr()) for x in (table, held, *out)]
    return _call(lib, "mmq_page_compact", p[0], p[1], i64(1), i64(1), i64(1), i64(pages), p[2], i64(1), p[3], p[4]), (table, held, *out)


def _plan_call(lib, mmq, nreq):  # noqa: F811
    adapters, start = torch.zeros(nreq, dtype=torch.int32, device="cuda"), torch.arange(nreq + 1, dtype=torch.int32, device="cuda")
    words = mmq.mmq_lora_plan(adapters, start, nreq, 1).words
    return _call(lib, "mmq_lora_plan", vp(adapters.data_ptr()), vp(start.data_ptr()), i64(nreq), i64(nreq), i64(1), vp(words.data_ptr())), (
        adapters, start, words)


def _lora_call(lib, mmq, tokens, rank):  # noqa: F811
    x, y = torch.zeros((tokens, 64), device="cuda"), torch.zeros((tokens, 64), device="cuda")
    a, b = (torch.zeros(4096 * 8, dtype=BF16, device="cuda") for _ in range(2))
    words = mmq.mmq_lora_plan(_i32([0]), _i32([0, tokens]), tokens, 1).words
    t = Lora(x=x.data_ptr(), y=y.data_ptr(), out=y.data_ptr(), a=a.data_ptr(), b=b.data_ptr(), plan=words.data_ptr(), x_row=64, y_row=64, out_row=64,
             ntok=tokens, nreq=1, nadapters=1, id=64, od=64, rank=rank, type=3, x_type=2)
    return _call(lib, "mmq_lora", ctypes.byref(t)), (x, y, a, b, words)


@pytest.mark.parametrize("what", ["lists", "probs", "fork", "compact", "plan", "lora16", "lora64"])
def test_calls_of_two_sizes_at_the_same_time(mmq, what):  # noqa: F811
    """How much shared memory a kernel may have is a setting of the kernel, not of a call: a thread that makes small calls
    does not take from one that makes large ones.  (Calls of the C ABI by ctypes, which runs them in parallel.)"""
    lib = mmq.load()
    make = {"lists": lambda n: _rules_call(lib, 1, (32000, 2 ** 18)[n], True), "probs": lambda n: _rules_call(lib, 80, (90000, 100277)[n], False),
            "fork": lambda n: _fork_call(lib, (2 ** 18, 2 ** 20)[n]), "compact": lambda n: _compact_call(lib, (2 ** 18, 2 ** 20)[n]),
            "plan": lambda n: _plan_call(lib, mmq, (3000, 8192)[n]), "lora16": lambda n: _lora_call(lib, mmq, 700, (72, 128)[n]),
            "lora64": lambda n: _lora_call(lib, mmq, 3000, (72, 128)[n])}[what]
    jobs = [make(n) for n in range(2)]
    torch.cuda.synchronize()
    codes, streams = [[], []], [torch.cuda.Stream() for _ in range(2)]

    def run(n):
        for k in range(3000):
            codes[n].append(jobs[n][0](vp(streams[n].cuda_stream)))
            if k % 100 == 99:
                streams[n].synchronize()

    threads = [threading.Thread(target=run, args=(n,)) for n in range(2)]
    for x in threads:
        x.start()
    for x in threads:
        x.join()
    torch.cuda.synchronize()
    assert all(len(c) == 3000 for c in codes) and {x for c in codes for x in c} == {0}


# ---------------------------------------------------------------- rows between rows
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_probs_and_adjusted_in_halves_of_one_array(mmq, dtype):  # noqa: F811
    """Outputs side by side in one array, or beside the logits: the same bits as in arrays of their own with rows that begin
    alike in 16 bytes of memory."""
    v = 1504  # (whole pieces of 16 bytes)
    p = _rules_problem(4, 2, v, dtype, seed=11)
    want = mmq.mmq_token_probs(**p, probs=torch.empty_like(p["logits"]), adjusted=torch.empty_like(p["logits"]))
    both = torch.empty((4, 3, 2 * v), dtype=dtype, device="cuda")
    got = mmq.mmq_token_probs(**p, probs=both[..., v:], adjusted=both[..., :v])
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    both[..., :v] = p["logits"]
    got = mmq.mmq_token_probs(**{**p, "logits": both[..., :v]}, probs=both[..., v:], adjusted=both[..., :v])
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    with pytest.raises(mmq.MMQError):
        mmq.mmq_token_probs(**p, probs=both[..., v - 1:-1], adjusted=both[..., :v])
