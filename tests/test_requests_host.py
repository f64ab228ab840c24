"""The host side of what differs from request to request in a step, without a GPU: what the C ABI refuses before any device
call, and what the Python binding does.  Addresses are made up, so calls that would be taken are made only where there is
no device to take them."""
import ctypes

import pytest
import torch

from tests.test_serving_host import ALIGN, ARG, CACHE_FAULTS, TYPE, UNSUPPORTED, _cache, i32, i64, lib, vp  # noqa: F401

NO_DEVICE = -8
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are made up")


class Fork(ctypes.Structure):
    _fields_ = [(n, vp) for n in ("table", "held", "parents", "lens", "new_table", "held_out", "pairs", "tokens", "free_pages", "counts")] + [
        (n, i64) for n in ("nold", "nnew", "table_width", "table_stride", "new_stride", "npages")] + [("page_size", i32)]


RULE_POINTERS = ("logits", "probs", "adjusted", "temperature", "tokens", "token_lens", "prompt_lens", "draft", "n_draft", "repetition",
                 "frequency", "presence", "bias_start", "bias_ids", "bias_values", "mask", "mask_rows")


class Rules(ctypes.Structure):
    _fields_ = [(n, vp) for n in RULE_POINTERS] + [
        (n, i64) for n in ("logits_req", "logits_row", "probs_req", "probs_row", "adjusted_req", "adjusted_row", "tokens_stride", "tokens_width",
                           "draft_stride", "nbias", "mask_stride", "nmasks", "nreq", "vocab")] + [
        (n, i32) for n in ("rows", "type", "probs_type", "adjusted_type")]


class Lora(ctypes.Structure):
    _fields_ = [(n, vp) for n in ("x", "y", "out", "a", "b", "scales", "ranks", "plan")] + [
        (n, i64) for n in ("x_row", "y_row", "out_row", "ntok", "nreq", "nadapters", "id", "od")] + [(n, i32) for n in ("rank", "type", "x_type")]


def test_struct_sizes_are_the_headers():
    """The structs above lie as in mmq.h on a 64-bit machine: pointers and int64 of 8 bytes, then int32, filled up to 8."""
    assert [ctypes.sizeof(s) for s in (Fork, Rules, Lora)] == [16 * 8 + 8, 31 * 8 + 16, 16 * 8 + 16]


# Nine old rows, eleven new ones, eight columns in rows of 16, 40 pages: the bytes of each buffer.
FORK = {"held": 36, "parents": 44, "lens": 44, "held_out": 44, "pairs": 88, "tokens": 44, "free_pages": 160, "counts": 8}
FORK_READ = ("held", "parents", "lens")
BASE = 1 << 24


def _fork(lib, **kw):  # noqa: F811
    f = {name: 4096 * (i + 1) for i, name in enumerate(FORK)}
    f.update(table=1 << 20, new_table=1 << 21, nold=9, nnew=11, table_width=8, table_stride=16, new_stride=16, npages=40, page_size=16)
    f.update(kw)
    return lib.mmq_page_fork(ctypes.byref(Fork(**f)), None)


def test_page_fork_checks(lib):  # noqa: F811
    for bad in (dict(nold=-1), dict(nnew=-1), dict(table_width=-1), dict(table_stride=7), dict(new_stride=7), dict(npages=-1), dict(page_size=0),
                dict(page_size=-5), dict(table_width=2 ** 31, table_stride=2 ** 31, new_stride=2 ** 31), dict(table_stride=2 ** 41)):
        assert _fork(lib, **bad) == ARG, bad
    for name in (*FORK, "table", "new_table"):
        assert _fork(lib, **{name: None}) == ARG, name
        assert _fork(lib, **{name: BASE + 2}) == ALIGN, name
    for many in (dict(nold=8193), dict(nnew=8193), dict(npages=2 ** 20 + 1)):
        assert _fork(lib, **many) == UNSUPPORTED, many
    assert lib.mmq_page_fork(None, None) == ARG


@pytest.mark.parametrize("other", FORK)
@pytest.mark.parametrize("out", [n for n in FORK if n not in FORK_READ])
def test_page_fork_written_over_something_else(lib, out, other):  # noqa: F811
    if out == other:
        return
    for at in (BASE, BASE + FORK[other] - 4, BASE - FORK[out] + 4):  # its begin, its end, the end of what is written
        assert _fork(lib, **{other: BASE, out: at}) == ARG, at - BASE


@pytest.mark.parametrize("name", FORK)
@pytest.mark.parametrize("table", ["table", "new_table"])
def test_page_fork_vectors_and_tables(lib, table, name):  # noqa: F811
    if table == "table" and name in FORK_READ:
        return  # (all read)
    rows = 9 if table == "table" else 11
    for at in (BASE, BASE + 64 * (rows - 1) + 28, BASE - FORK[name] + 4):  # rows of 32 bytes, 64 apart
        assert _fork(lib, **{table: BASE, name: at}) == ARG, at - BASE


def test_page_fork_into_its_own_table(lib):  # noqa: F811
    for at in (BASE, BASE + 4, BASE - 28, BASE + 64 * 8 + 28, BASE - 64 * 10 - 28):
        assert _fork(lib, table=BASE, new_table=at) == ARG, at - BASE


@no_gpu
def test_page_fork_that_there_is_no_device_for(lib):  # noqa: F811
    assert _fork(lib) == NO_DEVICE
    assert _fork(lib, table=BASE, new_table=BASE + 32) == NO_DEVICE  # the halves of wider rows
    assert _fork(lib, table=BASE, counts=BASE + 32) == NO_DEVICE     # between rows
    assert _fork(lib, nold=0, table=None, held=None) == NO_DEVICE
    assert _fork(lib, nnew=0, parents=None, lens=None, new_table=None, held_out=None, pairs=None, tokens=None) == NO_DEVICE
    assert _fork(lib, npages=0, free_pages=None) == NO_DEVICE
    assert _fork(lib, table_width=0, table=None, new_table=None) == NO_DEVICE
    assert _fork(lib, nold=8192, nnew=8192, npages=2 ** 20, **{n: 2 ** 28 + 2 ** 23 * i for i, n in enumerate(FORK)}) == NO_DEVICE


def _compact(lib, table=1 << 20, held=4096, nreq=9, width=8, stride=16, pages=40, new=1 << 21, new_stride=16, pairs=8192, counts=12288):  # noqa: F811
    return lib.mmq_page_compact(vp(table), vp(held), i64(nreq), i64(width), i64(stride), i64(pages), vp(new), i64(new_stride), vp(pairs),
                                vp(counts), None)


def test_page_compact_checks(lib):  # noqa: F811
    for bad in (dict(nreq=-1), dict(width=-1), dict(stride=7), dict(new_stride=7), dict(pages=-1), dict(table=None), dict(held=None),
                dict(new=None), dict(pairs=None), dict(counts=None)):
        assert _compact(lib, **bad) == ARG, bad
    for bad in (dict(table=BASE + 2), dict(held=BASE + 1), dict(new=BASE + 2), dict(pairs=BASE + 4), dict(counts=BASE + 2)):
        assert _compact(lib, **bad) == ALIGN, bad
    assert _compact(lib, nreq=8193) == UNSUPPORTED and _compact(lib, pages=2 ** 20 + 1) == UNSUPPORTED
    for bad in (dict(table=BASE, new=BASE), dict(table=BASE, new=BASE + 64 + 28), dict(held=BASE, counts=BASE + 32), dict(held=BASE, pairs=BASE),
                dict(pairs=BASE, counts=BASE + 152), dict(new=BASE, counts=BASE + 8 * 64), dict(new=BASE, pairs=BASE - 152),
                dict(new=BASE, held=BASE), dict(table=BASE, pairs=BASE + 64), dict(table=BASE, counts=BASE + 8 * 64 + 24)):
        assert _compact(lib, **bad) == ARG, bad


@no_gpu
def test_page_compact_that_there_is_no_device_for(lib):  # noqa: F811
    assert _compact(lib) == NO_DEVICE
    assert _compact(lib, nreq=0, table=None, held=None, new=None) == NO_DEVICE
    assert _compact(lib, pages=1, pairs=None) == NO_DEVICE and _compact(lib, pages=0, pairs=None) == NO_DEVICE


@pytest.mark.parametrize("change,code", CACHE_FAULTS, ids=str)
def test_page_copy_checks_the_cache(lib, change, code):  # noqa: F811
    assert lib.mmq_page_copy(ctypes.byref(_cache(**change)), vp(4096), vp(4096), i64(1), None) == code


def test_page_copy_checks(lib):  # noqa: F811
    def call(n, pairs=4096, tokens=None, **kw):
        return lib.mmq_page_copy(ctypes.byref(_cache(**kw)), vp(pairs), vp(tokens), i64(n), None)

    assert lib.mmq_page_copy(None, vp(4096), None, i64(1), None) == ARG
    assert call(-1) == ARG and call(2 ** 31) == ARG and call(1, pairs=None) == ARG
    assert call(1, pairs=4098) == ALIGN and call(1, tokens=4097) == ALIGN
    assert call(1, page_size=2 ** 26, heads=2) == UNSUPPORTED  # 2^27 * 64 elements
    assert call(0) == 0 and call(0, pairs=None) == 0


# Five requests of three rows, 100 tokens: rows end to end.
RULES = dict(logits=1 << 20, probs=1 << 21, adjusted=None, logits_req=300, logits_row=100, probs_req=300, probs_row=100, nreq=5, vocab=100, rows=3,
             type=2, probs_type=2)
EXTRA = {"temperature": 20, "token_lens": 20, "prompt_lens": 20, "n_draft": 20, "repetition": 20, "frequency": 20, "presence": 20,
         "bias_start": 24, "bias_ids": 28, "bias_values": 28, "mask_rows": 60, "tokens": 160, "draft": 40, "mask": 32}
FULL = dict(RULES, tokens_stride=8, tokens_width=8, draft_stride=2, nbias=7, mask_stride=4, nmasks=2,
            **{n: 4096 * (i + 1) for i, n in enumerate(EXTRA)})


def _probs(lib, base=RULES, **kw):  # noqa: F811
    return lib.mmq_token_probs(ctypes.byref(Rules(**{**base, **kw})), None)


def test_token_probs_checks(lib):  # noqa: F811
    assert lib.mmq_token_probs(None, None) == ARG
    for bad in (dict(type=0), dict(type=4), dict(type=9), dict(probs_type=0), dict(adjusted=1 << 22, adjusted_type=0)):
        assert _probs(lib, **bad) == TYPE, bad
    for bad in (dict(nreq=-1), dict(rows=0), dict(vocab=0), dict(tokens_width=-1), dict(nbias=-1), dict(nmasks=-1), dict(logits=None),
                dict(probs=None), dict(tokens_width=1), dict(nbias=1), dict(nbias=1, bias_ids=4096), dict(logits_req=-1), dict(logits_row=-1),
                dict(probs_req=-1), dict(adjusted_row=-1), dict(tokens_stride=-1), dict(draft_stride=-1), dict(mask_stride=-1),
                dict(logits_req=2 ** 62), dict(probs_row=2 ** 62), dict(mask_stride=2 ** 62, nmasks=4), dict(tokens_width=2 ** 31),
                dict(mask=4096, nmasks=2, mask_stride=3)):
        assert _probs(lib, **bad) == ARG, bad
    assert _probs(lib, vocab=2 ** 18 + 1) == UNSUPPORTED and _probs(lib, nreq=2 ** 26, rows=2, logits_req=0, probs_req=0) == UNSUPPORTED
    assert _probs(lib, logits=(1 << 20) + 2) == ALIGN and _probs(lib, probs=(1 << 21) + 2) == ALIGN
    assert _probs(lib, logits=(1 << 20) + 1, type=1) == ALIGN
    for name in EXTRA:
        assert _probs(lib, FULL, **{name: BASE + 2}) == ALIGN, name
    assert _probs(lib, nreq=0) == 0 and _probs(lib, nreq=0, logits=None, probs=None) == 0


def test_token_probs_written_over_something_else(lib):  # noqa: F811
    size = 4 * 1500
    for bad in (dict(probs=1 << 20), dict(probs=(1 << 20) + size - 4), dict(probs=(1 << 20) - size + 4),            # on the logits
                dict(probs_row=99), dict(probs_req=299), dict(probs_req=0), dict(probs_row=0),                       # rows on one another
                dict(adjusted=1 << 21, adjusted_type=2, adjusted_req=300, adjusted_row=100),                         # on the probabilities
                dict(adjusted=1 << 20, adjusted_type=1, adjusted_req=300, adjusted_row=100),                         # the logits' place, another type
                dict(adjusted=1 << 20, adjusted_type=2, adjusted_req=301, adjusted_row=100),                         # other strides
                dict(adjusted=(1 << 20) + 4, adjusted_type=2, adjusted_req=300, adjusted_row=100),                   # one further
                dict(adjusted=1 << 20, adjusted_type=2, adjusted_req=300, adjusted_row=50, logits_row=50),           # in place, rows on one another
                dict(adjusted=1 << 22, adjusted_type=2, adjusted_req=0, adjusted_row=100)):
        assert _probs(lib, **bad) == ARG, bad
    for name, n in EXTRA.items():
        for at in ((1 << 21), (1 << 21) + size - 4, (1 << 21) - n + 4):
            assert _probs(lib, FULL, **{name: at}) == ARG, (name, at - (1 << 21))
        assert _probs(lib, FULL, adjusted=BASE, adjusted_type=2, adjusted_req=300, adjusted_row=100, **{name: BASE + size - 4}) == ARG, name


@no_gpu
def test_token_probs_that_there_is_no_device_for(lib):  # noqa: F811
    assert _probs(lib) == NO_DEVICE and _probs(lib, FULL) == NO_DEVICE
    assert _probs(lib, adjusted=1 << 20, adjusted_type=2, adjusted_req=300, adjusted_row=100) == NO_DEVICE  # in place
    assert _probs(lib, logits_req=0, logits_row=0) == NO_DEVICE  # one row of logits for all
    assert _probs(lib, logits_req=100, logits_row=500, probs_req=100, probs_row=500) == NO_DEVICE  # (row, request) in memory
    assert _probs(lib, type=3, logits=(1 << 20) + 2) == NO_DEVICE and _probs(lib, vocab=2 ** 18, nreq=1, rows=1) == NO_DEVICE


def test_lora_plan_checks(lib):  # noqa: F811
    lib.mmq_lora_plan_words.restype = i64

    def words(ntok=100, nreq=5, many=7):
        return lib.mmq_lora_plan_words(i64(ntok), i64(nreq), i64(many))

    assert 100 < words() < 2000 and words(0, 0, 0) > 0
    top = 2 ** 31 // 64 - 1
    assert words(ntok=top) > top and words(nreq=8192) > 0 and words(many=2 ** 18) > 0
    for bad in (dict(ntok=-1), dict(nreq=-1), dict(many=-1), dict(ntok=top + 1), dict(nreq=8193), dict(many=2 ** 18 + 1)):
        assert words(**bad) == -1, bad

    def call(adapters=4096, start=8192, nreq=5, ntok=100, many=7, plan=BASE):
        return lib.mmq_lora_plan(vp(adapters), vp(start), i64(nreq), i64(ntok), i64(many), vp(plan), None)

    for bad in (dict(nreq=-1), dict(ntok=-1), dict(many=-1), dict(adapters=None), dict(start=None), dict(plan=None), dict(plan=4096),
                dict(plan=8192 + 20), dict(adapters=BASE + 4 * words() - 4), dict(start=BASE - 20)):
        assert call(**bad) == ARG, bad
    for bad in (dict(adapters=4098), dict(start=8193), dict(plan=BASE + 2)):
        assert call(**bad) == ALIGN, bad
    for bad in (dict(nreq=8193), dict(ntok=top + 1), dict(many=2 ** 18 + 1)):
        assert call(**bad) == UNSUPPORTED, bad
    if not torch.cuda.is_available():
        assert call() == NO_DEVICE and call(nreq=0, adapters=None) == NO_DEVICE and call(adapters=BASE + 4 * words()) == NO_DEVICE


# 100 tokens of 64 values to 40, seven adapters of rank 16.
LORA = dict(x=1 << 20, y=1 << 21, out=1 << 21, a=1 << 22, b=1 << 23, scales=None, ranks=None, plan=BASE, x_row=64, y_row=40, out_row=40, ntok=100,
            nreq=5, nadapters=7, id=64, od=40, rank=16, type=1, x_type=2)


def _lora(lib, **kw):  # noqa: F811
    return lib.mmq_lora(ctypes.byref(Lora(**{**LORA, **kw})), None)


def test_lora_checks(lib):  # noqa: F811
    assert lib.mmq_lora(None, None) == ARG
    for bad in (dict(type=2), dict(type=0), dict(x_type=0), dict(x_type=4)):
        assert _lora(lib, **bad) == TYPE, bad
    for bad in (dict(ntok=-1), dict(nreq=-1), dict(nadapters=-1), dict(id=0), dict(id=60), dict(od=0), dict(rank=0), dict(rank=12), dict(rank=136),
                dict(rank=-8), dict(x_row=-64), dict(y_row=-1), dict(out_row=-1), dict(x=None), dict(y=None), dict(out=None), dict(a=None),
                dict(b=None), dict(plan=None), dict(y_row=39, out_row=39), dict(out=1 << 25, out_row=39), dict(y_row=41), dict(x_row=2 ** 62)):
        assert _lora(lib, **bad) == ARG, bad
    for bad in (dict(x=(1 << 20) + 8), dict(a=(1 << 22) + 8), dict(b=(1 << 23) + 2), dict(x_row=66), dict(y=(1 << 21) + 2, out=(1 << 21) + 2),
                dict(scales=4098), dict(ranks=4097), dict(plan=BASE + 1), dict(x_row=68, x_type=1)):
        assert _lora(lib, **bad) == ALIGN, bad
    for bad in (dict(ntok=2 ** 31 // 64, x_row=0), dict(nreq=8193), dict(nadapters=2 ** 18 + 1), dict(id=2 ** 28 + 8), dict(od=2 ** 28 + 1)):
        assert _lora(lib, **bad) == UNSUPPORTED, bad
    assert _lora(lib, ntok=0) == 0 and _lora(lib, nreq=0) == 0


def test_lora_written_over_something_else(lib):  # noqa: F811
    out, size = 1 << 26, 4 * 40 * 100
    for name, n in dict(x=4 * 64 * 100, y=size, a=2 * 7 * 16 * 64, b=2 * 7 * 16 * 40, scales=28, ranks=28, plan=400).items():
        for at in (out + 16 * (name == "y"), out + size - 16, out - n // 16 * 16 + 16):
            assert _lora(lib, **{"out": out, name: at}) == ARG, (name, at - out)
    # within rows: columns of one array apart and not
    assert _lora(lib, x=out + 16, x_row=128, out=out, y=out, out_row=128, y_row=128) == ARG
    assert _lora(lib, y=out + 4 * 39, y_row=128, out=out, out_row=128) == ARG


@no_gpu
def test_lora_that_there_is_no_device_for(lib):  # noqa: F811
    out = 1 << 26
    assert _lora(lib) == NO_DEVICE and _lora(lib, out=out) == NO_DEVICE
    assert _lora(lib, nadapters=0, a=None, b=None) == NO_DEVICE
    assert _lora(lib, x=out + 160, x_row=128, out=out, y=out, out_row=128, y_row=128) == NO_DEVICE  # columns of one array
    assert _lora(lib, y=out + 160, y_row=128, out=out, out_row=128) == NO_DEVICE
    assert _lora(lib, ntok=1, y_row=0, out_row=40) == NO_DEVICE
    assert _lora(lib, x_row=0) == NO_DEVICE  # one x for all tokens


def test_binding_refuses_tensors_that_are_not_on_the_gpu():
    import quantized_int8_gemm_gb300 as mmq
    x = torch.zeros((2, 16, 2, 64), dtype=torch.float16)
    y = torch.zeros((2, 64))
    i = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: mmq.mmq_page_fork(i[:, None], i, i, i, 16, 4),
                 lambda: mmq.mmq_page_compact(i[:, None], i, 4),
                 lambda: mmq.mmq_page_copy(x, x, i[:, None]),
                 lambda: mmq.mmq_token_probs(y[None]),
                 lambda: mmq.mmq_lora_plan(i, i, 4, 2),
                 lambda: mmq.mmq_lora(y, y, x[0, :, :1], x[0, :, :1], mmq.LoraPlan(i, 2, 1, 1)),
                 lambda: mmq.mmq_page_fork(None, i, i, i, 16, 4),
                 lambda: mmq.mmq_token_probs(None)):
        with pytest.raises(TypeError, match="must be a CUDA tensor"):
            call()
