"""What differs from request to request in a step, the host side at the limits of its arguments, without a GPU: what the C ABI
refuses before any device call.  Addresses are made up, so calls that it should take are made only where there is no device
to take them."""
import random

import pytest

from tests.test_requests_host import ARG, BASE, NO_DEVICE, RULES, UNSUPPORTED, _compact, _fork, _probs, lib, no_gpu  # noqa: F401

# One row of one token a request, in one place for all to be read.
MANY = dict(RULES, rows=1, vocab=1, logits_req=0, logits_row=1, probs=1 << 40, probs_req=1, probs_row=1)
LISTS = dict(tokens=4096, tokens_stride=0, tokens_width=1, repetition=1 << 41)
MOST_LISTED = (2 ** 31 - 1) // 18  # eighteen numbers of each request's list, counted in 32 bits


def test_more_requests_with_lists_than_their_places_count(lib):  # noqa: F811
    for lists in (LISTS, dict(bias_start=1 << 41, bias_ids=4096, bias_values=8192, nbias=1),
                  dict(tokens=4096, tokens_width=1, presence=1 << 41), dict(tokens=4096, tokens_width=1, frequency=1 << 41)):
        for n in (MOST_LISTED + 1, 2 ** 27 - 1):
            assert _probs(lib, MANY, nreq=n, **lists) == UNSUPPORTED, (n, lists)


@no_gpu
def test_the_most_requests(lib):  # noqa: F811
    assert _probs(lib, MANY, nreq=MOST_LISTED, **LISTS) == NO_DEVICE
    assert _probs(lib, MANY, nreq=2 ** 27 - 1) == NO_DEVICE  # no lists
    assert _probs(lib, MANY, nreq=2 ** 27 - 1, tokens=4096, tokens_width=1) == NO_DEVICE  # no penalties, so that no tokens are counted
    assert _probs(lib, MANY, nreq=1, **{**LISTS, "tokens_width": 2 ** 29 - 1}) == NO_DEVICE
    assert _probs(lib, MANY, nreq=1, bias_start=4096, bias_ids=1 << 41, bias_values=1 << 42, nbias=2 ** 31 - 2048) == NO_DEVICE


def test_tokens_that_a_count_has_no_bits_for(lib):  # noqa: F811
    """A listed token's count lies in the 29 bits below its flags: said 2^29 times it would be a hidden one."""
    for width in (2 ** 29, 2 ** 31 - 1):
        assert _probs(lib, MANY, nreq=1, **{**LISTS, "tokens_width": width}) == UNSUPPORTED


def test_biases_whose_numbers_would_wrap(lib):  # noqa: F811
    """A CTA's threads go over the biases 1024 at a time, in 32 bits."""
    for n in (2 ** 31 - 2047, 2 ** 31 - 1):
        assert _probs(lib, MANY, nreq=1, bias_start=4096, bias_ids=1 << 41, bias_values=1 << 42, nbias=n) == UNSUPPORTED


WIDEST = 2 ** 31 - 1024


def test_tables_whose_columns_would_wrap(lib):  # noqa: F811
    """A CTA's warps go over a row's entries 256 at a time, in 32 bits."""
    for width in (WIDEST + 1, 2 ** 31 - 256, 2 ** 31 - 1):
        assert _fork(lib, nold=1, nnew=1, table=1 << 40, new_table=1 << 41, table_width=width, table_stride=width, new_stride=width) == UNSUPPORTED
        assert _compact(lib, nreq=1, table=1 << 40, new=1 << 41, width=width, stride=width, new_stride=width) == UNSUPPORTED


@no_gpu
def test_the_widest_tables(lib):  # noqa: F811
    assert _fork(lib, nold=1, nnew=1, table=1 << 40, new_table=1 << 41, table_width=WIDEST, table_stride=WIDEST, new_stride=WIDEST) == NO_DEVICE
    assert _compact(lib, nreq=1, table=1 << 40, new=1 << 41, width=WIDEST, stride=WIDEST, new_stride=WIDEST) == NO_DEVICE


def _elements(at, size, n, req, nreq, row=0, rows=1):
    return {at + size * (b * req + i * row + v) + byte for b in range(nreq) for i in range(rows) for v in range(n) for byte in range(size)}


def _strides(r, n, nreq, rows):  # rows that do not lie on one another, by requests or by rows
    if r.random() < 0.5:
        row = n + r.randint(0, 9)
        return (rows - 1) * row + n + r.randint(0, 9), row
    req = n + r.randint(0, 9)
    return req, (nreq - 1) * req + n + r.randint(0, 9)


@no_gpu
@pytest.mark.parametrize("seed", range(400))
def test_token_probs_written_beside_what_is_read(lib, seed):  # noqa: F811
    """Refused where an element is written that is read, or another output's, and nowhere else: rows lie between rows."""
    r = random.Random(seed)
    nreq, rows, v = r.randint(1, 4), r.randint(1, 3), r.randint(1, 9)
    probs_req, probs_row = _strides(r, v, nreq, rows)
    written = _elements(BASE, 4, v, probs_req, nreq, probs_row, rows)
    at = BASE + 4 * r.randint(-40, max(written) // 4 - BASE // 4 + 8)
    call = dict(nreq=nreq, rows=rows, vocab=v, type=2, probs=BASE, probs_type=2, probs_req=probs_req, probs_row=probs_row, logits=1 << 20,
                logits_req=rows * v, logits_row=v)
    what = r.choice(["logits", "logits", "half", "adjusted", "adjusted", "tokens", "draft", "mask", "temperature"])
    if what == "logits":
        strides = r.choice([(probs_req, probs_row), _strides(r, v, nreq, rows), (0, v), (v, 0), (0, 0), (r.randint(0, 20), r.randint(0, 20))])
        call.update(logits=at, logits_req=strides[0], logits_row=strides[1])
        other = _elements(at, 4, v, strides[0], nreq, strides[1], rows)
    elif what == "half":
        strides = r.choice([(2 * probs_req, 2 * probs_row), _strides(r, v, nreq, rows)])
        call.update(logits=at + 2, type=3, logits_req=strides[0], logits_row=strides[1])
        other = _elements(at + 2, 2, v, strides[0], nreq, strides[1], rows)
    elif what == "adjusted":
        strides = r.choice([(probs_req, probs_row), _strides(r, v, nreq, rows)])
        call.update(adjusted=at, adjusted_type=2, adjusted_req=strides[0], adjusted_row=strides[1])
        other = _elements(at, 4, v, strides[0], nreq, strides[1], rows)
    elif what == "temperature":
        call.update(temperature=at)
        other = _elements(at, 4, nreq, 0, 1)
    else:
        n, many = {"tokens": (5, nreq), "draft": (rows - 1, nreq), "mask": (1, 3)}[what]
        stride = n + r.choice([0, 0, probs_req])
        call.update({"tokens": dict(tokens=at, tokens_width=n, tokens_stride=stride), "draft": dict(draft=at, draft_stride=stride),
                     "mask": dict(mask=at, mask_stride=stride, nmasks=many)}[what])
        other = _elements(at, 4, n, stride, many)
    assert _probs(lib, call) == (ARG if other & written else NO_DEVICE), (what, call)


@no_gpu
def test_halves_of_wider_rows(lib):  # noqa: F811
    half = dict(RULES, logits_req=600, logits_row=200, probs_req=600, probs_row=200)
    assert _probs(lib, half, probs=(1 << 20) + 400) == NO_DEVICE and _probs(lib, half, probs=(1 << 20) + 396) == ARG
    both = dict(half, adjusted=(1 << 21) + 400, adjusted_type=2, adjusted_req=600, adjusted_row=200)
    assert _probs(lib, both) == NO_DEVICE and _probs(lib, both, probs=(1 << 20) + 400, adjusted=1 << 20) == NO_DEVICE
    assert _probs(lib, both, adjusted=(1 << 21) + 404) == ARG
