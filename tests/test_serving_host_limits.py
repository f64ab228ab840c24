"""The serving step's host side at the limits of its arguments, without a GPU: what the C ABI refuses before any device
call.  Addresses are made up, so calls that it should take are made only where there is no device to take them."""
import ctypes

import pytest
import torch

from tests.test_serving_host import ALIGN, ARG, UNSUPPORTED, i32, i64, lib, vp  # noqa: F401

NO_DEVICE = -8
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are made up")

# nine requests, 40 table columns, 100 free pages, 70 token rows; 4096 bytes for each buffer, 64 for each row of the table
BUFFERS = {"cached": 36, "fresh": 36, "held": 36, "free": 400, "q_start": 40, "seq_lens": 36, "held_out": 36, "slots": 560, "positions": 280,
           "taken": 8}
READ = ["cached", "fresh", "held", "free"]


def _tables(lib, table=1 << 20, width=8, stride=16, **moved):  # noqa: F811
    at = {name: 4096 * (i + 1) for i, name in enumerate(BUFFERS)}
    at.update(moved)
    return lib.mmq_page_tables(vp(at["cached"]), vp(at["fresh"]), vp(at["held"]), i64(9), vp(table), i64(width), i64(stride), vp(at["free"]),
                               i64(100), i32(16), i64(70), vp(at["q_start"]), vp(at["seq_lens"]), vp(at["held_out"]), vp(at["slots"]),
                               vp(at["positions"]), vp(at["taken"]), None)


@pytest.mark.parametrize("other", BUFFERS)
@pytest.mark.parametrize("out", [b for b in BUFFERS if b not in READ])
def test_page_tables_written_over_something_else(lib, out, other):  # noqa: F811
    if out == other:
        return
    base = 1 << 24
    for at in (base, base + BUFFERS[other] - 8, base - BUFFERS[out] + 8):  # all of it, its end, its begin
        assert _tables(lib, **{other: base, out: at}) == ARG, at - base


@pytest.mark.parametrize("name", BUFFERS)
def test_page_tables_written_over_the_table(lib, name):  # noqa: F811
    table, row, pitch = 1 << 24, 32, 64
    for at in (table, table - BUFFERS[name] + 8, table + 3 * pitch + row - 8, table + 8 * pitch + row - 8):
        assert _tables(lib, table, **{name: at}) == ARG, at - table


@no_gpu
def test_page_tables_beside_one_another(lib):  # noqa: F811
    assert _tables(lib) == NO_DEVICE
    base = 1 << 24
    for out in BUFFERS:
        for other in BUFFERS:
            if out != other:
                assert _tables(lib, **{other: base, out: base + (BUFFERS[other] + 7) // 8 * 8}) == NO_DEVICE
        # behind the table's last row; in the gap between two of them, where it is short enough
        assert _tables(lib, base, **{out: base + 8 * 64 + 32}) == NO_DEVICE
        if BUFFERS[out] <= 32:
            assert _tables(lib, base, **{out: base + 4 * 64 + 32}) == NO_DEVICE
    for a, b in (("cached", "fresh"), ("held", "cached"), ("free", "held")):  # what is only read may be one buffer
        assert _tables(lib, **{a: base, b: base}) == NO_DEVICE


def test_attention_rows_whose_numbers_would_wrap(lib):  # noqa: F811
    """A row tile's rows are numbered past the last one: 2^31 less a unit's rows is the most."""
    import tests.test_serving_host as host
    cache = host._cache(heads=1, head_dim=8)
    for heads in (1, 8, 160):
        most = (2 ** 31 - 1 - 512) // heads
        for ntok in (most + 1, (2 ** 31 - 1) // heads):
            a = host.Attention(q=4096, out=4096, table=4096, seq_lens=4096, q_start=4096, q_token=8 * heads, q_head=8, out_token=8 * heads, out_head=8,
                               table_stride=8, nreq=1, ntok=ntok, table_width=8, q_heads=heads, out_type=1, causal=1, scale=0.1)
            assert lib.mmq_paged_attention(ctypes.byref(cache), ctypes.byref(a), None) == ARG


def test_kv_rows_whose_items_would_wrap(lib):  # noqa: F811
    import tests.test_serving_host as host
    for heads, d in ((2 ** 27, 64), (2 ** 26 + 1, 64), (2 ** 31 - 1, 8), (2 ** 25 + 1, 128)):
        cache = host._cache(heads=heads, head_dim=d)
        assert lib.mmq_kv_write(ctypes.byref(cache), vp(4096), i64(128), i64(64), vp(4096), i64(128), i64(64), 2, vp(4096), i64(1), None) == UNSUPPORTED


def test_pointers_off_their_elements_alignment(lib):  # noqa: F811
    """Such an access would fault on the device."""
    import tests.test_serving_host as host
    for name in BUFFERS:
        for off in (1, 2) + ((4,) if name == "slots" else ()):
            assert _tables(lib, **{name: 4096 * 50 + off}) == ALIGN, (name, off)
    assert _tables(lib, (1 << 20) + 2) == ALIGN
    base = dict(q=4096, out=4096, lse=4096, table=4096, seq_lens=4096, q_start=4096, q_token=512, q_head=64, out_token=512, out_head=64, table_stride=8,
                nreq=1, ntok=1, table_width=8, q_heads=8, out_type=1, causal=1, window=0, scale=0.1)
    cache = host._cache()
    for name in ("lse", "table", "seq_lens", "q_start"):
        assert lib.mmq_paged_attention(ctypes.byref(cache), ctypes.byref(host.Attention(**{**base, name: 4098})), None) == ALIGN, name
    base = dict(target=4096, draft=4096, tokens=4096, n_draft=4096, u=4096, noise=4096, out=4096, accepted=4096, target_req=64, target_row=32,
                draft_req=32, draft_row=32, tokens_stride=1, u_stride=1, noise_stride=32, nreq=1, vocab=32, k=1, type=1)
    for name in ("tokens", "n_draft", "u", "noise", "out", "accepted"):
        assert lib.mmq_verify_draft(ctypes.byref(host.Verification(**{**base, name: 4098})), None) == ALIGN, name
