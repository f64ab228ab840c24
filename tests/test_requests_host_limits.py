"""What differs from request to request in a step, the host side at the limits of its arguments, without a GPU: what the C ABI
refuses before any device call.  Addresses are made up, so calls that it should take are made only where there is no device
to take them."""
from tests.test_requests_host import NO_DEVICE, RULES, UNSUPPORTED, _compact, _fork, _probs, lib, no_gpu  # noqa: F401

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
