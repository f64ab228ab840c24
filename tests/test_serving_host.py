"""The serving step's host side without a GPU: argument checks of the C ABI, which come before any device call, and of
the Python binding."""
import ctypes

import pytest
import torch

vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32

ARG, ALIGN, TYPE, UNSUPPORTED = -1, -2, -3, -7


class Cache(ctypes.Structure):
    _fields_ = [("k", vp), ("v", vp)] + [(n, i64) for n in ("k_page", "k_token", "k_head", "v_page", "v_token", "v_head", "pages")] + [
        (n, i32) for n in ("page_size", "heads", "head_dim", "type")]


class Attention(ctypes.Structure):
    _fields_ = [(n, vp) for n in ("q", "out", "lse", "table", "seq_lens", "q_start")] + [
        (n, i64) for n in ("q_token", "q_head", "out_token", "out_head", "table_stride", "nreq", "ntok")] + [
        (n, i32) for n in ("table_width", "q_heads", "out_type", "causal", "window")] + [("scale", ctypes.c_float)]


class Verification(ctypes.Structure):
    _fields_ = [(n, vp) for n in ("target", "draft", "tokens", "n_draft", "u", "noise", "out", "accepted")] + [
        (n, i64) for n in ("target_req", "target_row", "draft_req", "draft_row", "tokens_stride", "u_stride", "noise_stride", "nreq", "vocab")] + [
        (n, i32) for n in ("k", "type")]


@pytest.fixture(scope="module")
def lib():
    from quantized_int8_gemm_gb300 import build
    return ctypes.CDLL(build.build())


def _cache(**kw):
    c = dict(k=4096, v=8192, k_page=2048, k_token=128, k_head=64, v_page=2048, v_token=128, v_head=64, pages=4, page_size=16, heads=2,
             head_dim=64, type=1)
    c.update(kw)
    return Cache(**c)


CACHE_FAULTS = [(dict(k=None), ARG), (dict(v=None), ARG), (dict(pages=0), ARG), (dict(page_size=0), ARG), (dict(heads=0), ARG),
                (dict(head_dim=0), ARG), (dict(head_dim=20), ARG), (dict(head_dim=264), ARG), (dict(k_token=-8), ARG), (dict(type=2), TYPE),
                (dict(type=9), TYPE), (dict(k=4104), ALIGN), (dict(v_head=4), ALIGN)]


@pytest.mark.parametrize("change,code", CACHE_FAULTS, ids=str)
def test_cache_checks(lib, change, code):
    c = _cache(**change)
    assert lib.mmq_kv_write(ctypes.byref(c), vp(4096), i64(128), i64(64), vp(4096), i64(128), i64(64), 2, vp(4096), i64(1), None) == code
    assert lib.mmq_paged_attention(ctypes.byref(c), ctypes.byref(Attention(out_type=1)), None) == code
    assert lib.mmq_paged_attention(None, None, None) == ARG


def test_kv_write_checks(lib):
    c = _cache()

    def call(k=4096, kt=128, src=2, slots=4096, n=1):
        return lib.mmq_kv_write(ctypes.byref(c), vp(k), i64(kt), i64(64), vp(4096), i64(128), i64(64), src, vp(slots), i64(n), None)

    assert call(n=-1) == ARG and call(src=7) == TYPE and call(k=None) == ARG and call(slots=None) == ARG
    assert call(k=4100) == ALIGN and call(kt=129) == ALIGN and call(kt=-8) == ARG
    assert call(n=0) == 0  # nothing to do


def test_attention_checks(lib):
    c = _cache()

    def call(**kw):
        a = dict(q=4096, out=4096, lse=None, table=4096, seq_lens=4096, q_start=4096, q_token=512, q_head=64, out_token=512, out_head=64,
                 table_stride=8, nreq=1, ntok=1, table_width=8, q_heads=8, out_type=1, causal=1, window=0, scale=0.1)
        a.update(kw)
        return lib.mmq_paged_attention(ctypes.byref(c), ctypes.byref(Attention(**a)), None)

    assert call(out_type=3) == TYPE and call(out_type=0) == TYPE
    for bad in (dict(nreq=-1), dict(ntok=-1), dict(q_heads=0), dict(q_heads=7), dict(window=-1), dict(scale=0.0), dict(scale=float("nan")),
                dict(scale=float("inf")), dict(q=None), dict(out=None), dict(table=None), dict(seq_lens=None), dict(q_start=None),
                dict(table_stride=7), dict(table_width=-1), dict(q_token=-8), dict(ntok=2 ** 31)):
        assert call(**bad) == ARG, bad
    assert call(q=4104) == ALIGN and call(out_head=4) == ALIGN
    assert call(nreq=0) == 0 and call(ntok=0) == 0


def test_page_tables_checks(lib):
    def call(nreq=1, width=4, stride=4, nfree=2, page=16, room=4, cached=4096, table=4096, free=4096, slots=4096, q_start=4096):
        return lib.mmq_page_tables(vp(cached), vp(4096), vp(4096), i64(nreq), vp(table), i64(width), i64(stride), vp(free), i64(nfree),
                                   i32(page), i64(room), vp(q_start), vp(4096), vp(4096), vp(slots), vp(4096), vp(4096), None)

    for bad in (dict(nreq=-1), dict(width=-1), dict(stride=3), dict(nfree=-1), dict(page=0), dict(room=-1), dict(cached=None),
                dict(table=None), dict(free=None), dict(slots=None), dict(q_start=None), dict(room=2 ** 31)):
        assert call(**bad) == ARG, bad
    assert call(nreq=8193) == UNSUPPORTED


def test_verify_checks(lib):
    def call(**kw):
        a = dict(target=4096, draft=4096, tokens=4096, n_draft=None, u=4096, noise=4096, out=4096, accepted=4096, target_req=64, target_row=32,
                 draft_req=32, draft_row=32, tokens_stride=1, u_stride=1, noise_stride=32, nreq=1, vocab=32, k=1, type=2)
        a.update(kw)
        return lib.mmq_verify_draft(ctypes.byref(Verification(**a)), None)

    assert call(type=0) == TYPE
    for bad in (dict(nreq=-1), dict(nreq=65536), dict(vocab=0), dict(vocab=2 ** 31), dict(k=-1), dict(target=None), dict(noise=None),
                dict(out=None), dict(accepted=None), dict(tokens=None), dict(u=None), dict(target_row=-1)):
        assert call(**bad) == ARG, bad
    assert call(target=4098) == ALIGN and call(noise=4098) == ALIGN
    assert call(nreq=0) == 0
    assert lib.mmq_verify_draft(None, None) == ARG


def test_binding_refuses_tensors_that_are_not_on_the_gpu():
    import quantized_int8_gemm_gb300 as mmq
    x = torch.zeros((2, 2, 64), dtype=torch.float16)
    i = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: mmq.mmq_kv_write(x, x, x[None], x[None], i.long()),
                 lambda: mmq.mmq_paged_attention(x, x[None], x[None], i[None], i, i),
                 lambda: mmq.mmq_page_tables(i, i, i, i[:, None], i, 16, 4),
                 lambda: mmq.mmq_verify_draft(x.float(), None, i[:, None], i, x[0, :, :1].float(), x[0].float()),
                 lambda: mmq.mmq_kv_write(None, x, x, x, i)):
        with pytest.raises(TypeError, match="must be a CUDA tensor"):
            call()


def test_struct_sizes_are_the_headers():
    """The structs above lie as in mmq.h: 88, 128 and 144 bytes on a 64-bit machine."""
    assert [ctypes.sizeof(s) for s in (Cache, Attention, Verification)] == [88, 128, 144]
