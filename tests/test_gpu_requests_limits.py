"""What differs from request to request in a step, on the GPU, at the limits of its arguments: logits far from 0.
Tolerances are those of tests/test_gpu_requests.py, derived there, unless a test says others."""
import math

import pytest

from tests.test_gpu_requests import BF16, F16, F32, _check_rules, _f32, _i32, _no_device_error, _rules_problem, mmq  # noqa: F401

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
