"""The serving step's operators on the GPU against plain implementations in 64 bits.

Tolerances, derived before any run.  Attention in a type of unit roundoff u (half an ulp of 1: fp16 2^-11, bf16 2^-8): the output is
rounded once (u |out|), every softmax weight once (u sum p|v|); fp16 weights below 2^-14 of the row's largest lose up to
2^-25 each; fp32 sums and exp2 add a few 1e-6 of sum p|v| and of the exponents, covered by 1e-4 sum p|v|.  lse carries the
fp32 sum of head_dim products, 2^-20 of sum |q k| scale at the most.  Everything else is exact.
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
UNIT = {F16: 2.0 ** -11, BF16: 2.0 ** -8}


@pytest.fixture(scope="module")
def mmq():
    from quantized_int8_gemm_gb300 import build
    build.build()
    import quantized_int8_gemm_gb300 as m
    m.load()
    assert torch.cuda.is_available()
    return m


@pytest.fixture(autouse=True)
def _no_device_error(mmq):
    mmq.mmq_last_device_error()
    yield
    assert mmq.mmq_last_device_error() == 0


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------- attention
def _problem(dtype, q_lens, kv_lens, hq, hkv, d, page, layout="nhd", seed=0, poison=math.nan, gain=1.5):
    """kv_lens: keys of each request, the new tokens among them.  Everything no request holds is `poison`."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    blocks = [-(-n // page) for n in kv_lens]
    pages = sum(blocks) + 2
    shape = (pages, page, hkv, d) if layout == "nhd" else (pages, hkv, page, d)
    kc, vc = (torch.full(shape, poison, dtype=dtype, device="cuda") for _ in range(2))
    if layout == "hnd":
        kc, vc = kc.permute(0, 2, 1, 3), vc.permute(0, 2, 1, 3)
    order = torch.randperm(pages, generator=g, device="cuda").tolist()
    table = torch.full((len(kv_lens), max(blocks + [1]) + 1), -1, dtype=torch.int32)
    keys, values, at = [], [], 0
    for b, n in enumerate(kv_lens):
        k, v = (torch.randn((n, hkv, d), generator=g, device="cuda").to(dtype) for _ in range(2))
        keys.append(k)
        values.append(v)
        for j in range(blocks[b]):
            p = order[at]
            at += 1
            table[b, j] = p
            m = min(page, n - j * page)
            kc[p, :m] = k[j * page:j * page + m]
            vc[p, :m] = v[j * page:j * page + m]
    q = (torch.randn((sum(q_lens), hq, d), generator=g, device="cuda") * gain).to(dtype)
    starts = np.concatenate([[0], np.cumsum(q_lens)]).tolist()
    return {"q": q, "kc": kc, "vc": vc, "table": table.cuda(), "seq_lens": _i32(kv_lens), "q_start": _i32(starts),
            "keys": keys, "values": values, "q_lens": q_lens, "kv_lens": kv_lens}


def _reference(p, scale, causal, window):
    """out, lse, and the tolerances of both, in fp64."""
    q = p["q"].double()
    t, hq, d = q.shape
    dev = q.device
    out = torch.zeros((t, hq, d), dtype=torch.float64, device=dev)
    lse = torch.full((t, hq), -math.inf, dtype=torch.float64, device=dev)
    tol, lse_tol = torch.zeros_like(out), torch.zeros_like(lse)
    u = UNIT[p["q"].dtype]
    at = 0
    for n, length, k, v in zip(p["q_lens"], p["kv_lens"], p["keys"], p["values"]):
        if n and length:
            hkv = k.shape[1]
            kk, vv = (x.double().repeat_interleave(hq // hkv, 1).permute(1, 0, 2) for x in (k, v))
            x = q[at:at + n].permute(1, 0, 2)
            s = x @ kk.transpose(1, 2) * scale
            size = (x.abs() @ kk.abs().transpose(1, 2) * scale).amax(-1)
            pos = torch.arange(length - n, length, device=dev)[:, None]
            j = torch.arange(length, device=dev)
            seen = torch.ones((n, length), dtype=torch.bool, device=dev)
            if causal:
                seen &= j <= pos
            if window:
                seen &= j > pos - window
            s.masked_fill_(~seen, -math.inf)
            some = seen.any(-1)
            top = torch.where(some, s.amax(-1), 0.0)
            w = torch.exp(s - top[..., None])
            total = w.sum(-1)
            z = torch.where(some, top + torch.log(total), -math.inf)
            div = torch.where(total > 0, total, 1.0)[..., None]
            o, mass = w @ vv / div, w @ vv.abs() / div
            tiny = 2.0 ** -25 * (seen.double() @ vv.abs()) / div if p["q"].dtype == F16 else 0.0
            out[at:at + n] = o.permute(1, 0, 2)
            lse[at:at + n] = z.T
            tol[at:at + n] = (u * (mass + o.abs()) * 1.0625 + 1e-4 * mass + tiny).permute(1, 0, 2)
            lse_tol[at:at + n] = (2.0 ** -20 * size + 1e-5).T
        at += n
    return out, lse, tol, lse_tol


def _check(p, out, lse, scale, causal=True, window=0):
    ref, z, tol, z_tol = _reference(p, scale, causal, window)
    assert torch.isfinite(out).all()
    worst = ((out.double() - ref).abs() - tol).max().item() if out.numel() else 0
    assert worst <= 0, worst
    if lse is not None:
        none = torch.isinf(z)
        assert torch.equal(torch.isinf(lse) & (lse < 0), none)
        off = torch.where(none, 0.0, (lse.double() - torch.where(none, 0.0, z)).abs() - z_tol)
        assert off.max().item() <= 0, off.max().item()


def _attend(mmq, p, **kw):
    return mmq.mmq_paged_attention(p["q"], p["kc"], p["vc"], p["table"], p["seq_lens"], p["q_start"], lse=True, **kw)


SHAPES = [
    # q lens, key lens, q heads, K/V heads, head width, page
    ([1], [1], 1, 1, 64, 16),
    ([1], [257], 8, 8, 128, 16),
    ([1, 1, 1], [700, 1, 129], 28, 4, 128, 16),
    ([1] * 40, [5 + 61 * i for i in range(40)], 8, 2, 64, 64),
    ([1] * 300, [1 + (37 * i) % 290 for i in range(300)], 8, 1, 128, 16),
    ([0, 1, 2] * 400, [(53 * i) % 200 for i in range(1200)], 2, 2, 64, 8),
    ([1, 3] * 70, [(29 * i) % 150 for i in range(140)], 2, 1, 256, 16),
    ([5, 1, 3], [133, 640, 3], 28, 4, 128, 8),
    ([130], [130], 7, 1, 128, 32),
    ([300, 1, 77], [1000, 2049, 77], 12, 4, 64, 128),
    ([40, 0, 9], [44, 0, 700], 4, 2, 128, 256),
    ([33], [97], 6, 2, 80, 16),
    ([2, 100], [300, 180], 8, 4, 96, 24),
    ([70, 4], [90, 515], 3, 3, 8, 16),
    ([61], [200], 4, 1, 256, 16),
    ([1, 9], [2000, 130], 8, 1, 192, 1),
    ([45, 1], [300, 333], 6, 3, 128, 5),
    ([3], [400], 160, 1, 64, 16),       # more query heads to a K/V head than rows of a tile
    ([1], [9000], 4, 1, 128, 64),       # one row, split over the keys
    ([1], [6000], 4, 1, 256, 16),
    ([1, 2], [20000, 3000], 4, 2, 96, 16),
    ([20], [30000], 1, 1, 64, 256),
    ([513], [4097], 4, 1, 64, 64),
]


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"q{s[0][0]}x{len(s[0])}_kv{max(s[1])}_h{s[2]}-{s[3]}_d{s[4]}_p{s[5]}")
def test_attention_against_64_bits(mmq, shape, dtype):
    q_lens, kv_lens, hq, hkv, d, page = shape
    for layout, causal, window in (("nhd", True, 0), ("hnd", True, 50), ("nhd", False, 0)):
        p = _problem(dtype, q_lens, kv_lens, hq, hkv, d, page, layout, seed=page + d)
        out, lse = _attend(mmq, p, causal=causal, window=window)
        _check(p, out, lse, 1 / math.sqrt(d), causal, window)


@pytest.mark.parametrize("d,page", [(128, 16), (64, 64), (96, 3), (256, 16)])
def test_rows_that_see_nothing(mmq, d, page):
    """A request without keys, and a chunk longer than its keys (its first rows have none)."""
    p = _problem(BF16, [3, 20, 1], [0, 12, 30], 4, 2, d, page)
    out, lse = _attend(mmq, p)
    _check(p, out, lse, 1 / math.sqrt(d))
    assert not out[:3].any() and not out[3:11].any() and torch.isinf(lse[:11]).all()


@pytest.mark.parametrize("poison", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("d,page", [(128, 16), (128, 7)])
def test_what_lies_past_the_last_key_is_not_used(mmq, d, page, poison):
    p = _problem(F16, [1, 150, 5], [100, 150, 513], 8, 2, d, page, poison=poison)
    out, lse = _attend(mmq, p)
    _check(p, out, lse, 1 / math.sqrt(d))


@pytest.mark.parametrize("d,page", [(64, 8), (128, 5)])
def test_very_many_requests(mmq, d, page):
    """More groups of 32 requests than a CTA keeps sums of: few requests have tokens, the last one among them."""
    n = 40000
    some = {0: (1, 40), 7: (3, 130), 16351: (1, 9), 16352: (2, 300), 20011: (1, 1), n - 1: (4, 600)}
    p = _problem(F16, [x for x, _ in some.values()], [x for _, x in some.values()], 4, 2, d, page)
    q_lens, kv_lens = torch.zeros(n, dtype=torch.int32), torch.zeros(n, dtype=torch.int32)
    table = torch.full((n, p["table"].shape[1]), -1, dtype=torch.int32, device="cuda")
    for row, (at, (x, y)) in enumerate(some.items()):
        q_lens[at], kv_lens[at] = x, y
        table[at] = p["table"][row]
    starts = torch.cat([torch.zeros(1, dtype=torch.int32), q_lens.cumsum(0).int()]).cuda()
    out, lse = mmq.mmq_paged_attention(p["q"], p["kc"], p["vc"], table, kv_lens.cuda(), starts, lse=True)
    _check(p, out, lse, 1 / math.sqrt(d))


@pytest.mark.parametrize("d,page,hq,hkv", [(64, 16, 8, 2), (128, 8, 28, 4), (128, 64, 4, 4), (128, 256, 4, 1), (256, 16, 4, 2), (64, 5, 4, 1)])
@pytest.mark.parametrize("window", [1, 13, 100, 300])
def test_what_lies_behind_the_window_is_not_used(mmq, d, page, hq, hkv, window):
    """Pages and keys that no new token's window reaches may be gone: ids out of the cache, NaN in their memory."""
    q_lens, kv_lens = [1, 1, 5, 300, 2, 1], [4097, 640, 517, 1333, 90, 7000]
    p = _problem(F16, q_lens, kv_lens, hq, hkv, d, page, seed=window)
    for b, (n, length) in enumerate(zip(q_lens, kv_lens)):
        first = max(0, length - n - window + 1)
        for j in range(first // page):
            for x in (p["kc"], p["vc"]):
                x[p["table"][b, j]] = math.nan
            if (b + j) % 2:
                p["table"][b, j] = -1 if j % 4 else 2 ** 30
        if first % page:
            for x in (p["kc"], p["vc"]):
                x[p["table"][b, first // page], :first % page] = math.nan
    out, lse = _attend(mmq, p, window=window)
    _check(p, out, lse, 1 / math.sqrt(d), window=window)


@pytest.mark.parametrize("d,page,q_lens", [(128, 16, [1, 1]), (128, 16, [200, 1]), (64, 5, [3, 90])])
def test_strides_scale_and_fp32_output(mmq, d, page, q_lens):
    """q as columns of a wider tensor, an output with its own strides, fp32 output, another scale."""
    p = _problem(BF16, q_lens, [400, 300], 8, 2, d, page)
    t = sum(q_lens)
    wide = torch.full((t, 12, d), math.nan, dtype=BF16, device="cuda")
    wide[:, 2:10] = p["q"]
    p["q"] = wide[:, 2:10]
    buf = torch.zeros((8, t, d + 8), dtype=F32, device="cuda")
    out = buf[:, :, :d].permute(1, 0, 2)
    got, lse = mmq.mmq_paged_attention(p["q"], p["kc"], p["vc"], p["table"], p["seq_lens"], p["q_start"], scale=0.11, out=out,
                                       lse=True)
    assert got is out and not buf[:, :, d:].any()
    _check(p, out, lse, 0.11)
    rounded, none = mmq.mmq_paged_attention(p["q"], p["kc"], p["vc"], p["table"], p["seq_lens"], p["q_start"], scale=0.11)
    assert none is None and torch.equal(rounded, out.to(BF16))


def test_scores_of_any_size(mmq):
    """Scores far from zero on either side, rising along the keys, so that the running maximum moves in every tile."""
    for sign in (1.0, -1.0):
        p = _problem(BF16, [140, 1], [900, 700], 4, 2, 128, 16)
        for b in range(2):
            n = p["kv_lens"][b]
            ramp = torch.linspace(0.1, 3.0, n, device="cuda")[:, None, None] * sign
            p["keys"][b] = (torch.ones_like(p["keys"][b]).float() * ramp).to(BF16)
            for j in range(-(-n // 16)):
                m = min(16, n - j * 16)
                p["kc"][p["table"][b, j].item(), :m] = p["keys"][b][j * 16:j * 16 + m]
        p["q"] = torch.full_like(p["q"], 2.0)
        out, lse = _attend(mmq, p)
        _check(p, out, lse, 1 / math.sqrt(128))


def test_rows_behind_the_last_request_are_left_alone(mmq):
    p = _problem(F16, [2, 3], [600, 40], 4, 2, 64, 16)
    pad = torch.randn((4, 4, 64), device="cuda").to(F16)
    out = torch.full((9, 4, 64), 7.0, dtype=F16, device="cuda")
    lse = torch.full((9, 4), 7.0, device="cuda")
    mmq.mmq_paged_attention(torch.cat([p["q"], pad]), p["kc"], p["vc"], p["table"], p["seq_lens"], p["q_start"], out=out, lse=lse)
    _check(p, out[:5], lse[:5], 1 / 8)
    assert (out[5:] == 7).all() and (lse[5:] == 7).all()


def test_repeated_calls_give_the_same_bits(mmq):
    for q_lens, kv_lens in (([1] * 6, [3000, 17, 900, 4000, 1, 250]), ([700], [4000])):
        p = _problem(BF16, q_lens, kv_lens, 28, 4, 128, 16)
        first = _attend(mmq, p)
        for _ in range(3):
            again = _attend(mmq, p)
            assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_another_stream_and_graph_replay_on_other_lengths(mmq):
    """A captured call reads the lengths and pages that lie there when it is replayed."""
    a = _problem(F16, [1] * 5, [3000, 2, 1111, 64, 4000], 8, 2, 128, 16, seed=1)
    b = _problem(F16, [1] * 5, [5, 4000, 900, 3500, 33], 8, 2, 128, 16, seed=2)
    width = max(a["table"].shape[1], b["table"].shape[1])
    pages = max(a["kc"].shape[0], b["kc"].shape[0])
    q, lens, start = a["q"].clone(), a["seq_lens"].clone(), a["q_start"].clone()
    kc, vc = (torch.zeros((pages, 16, 2, 128), dtype=F16, device="cuda") for _ in range(2))
    table = torch.full((5, width), -1, dtype=torch.int32, device="cuda")
    out, lse = torch.empty_like(q), torch.empty((5, 8), device="cuda")

    def fill(p):
        q.copy_(p["q"])
        lens.copy_(p["seq_lens"])
        start.copy_(p["q_start"])
        kc[:p["kc"].shape[0]] = p["kc"]
        vc[:p["vc"].shape[0]] = p["vc"]
        table[:, :p["table"].shape[1]] = p["table"]

    fill(a)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    mmq.mmq_paged_attention(q, kc, vc, table, lens, start, out=out, lse=lse, stream=s)
    new, new_lse = mmq.mmq_paged_attention(q, kc, vc, table, lens, start, lse=True, stream=s.cuda_stream)
    s.synchronize()
    _check(a, out, lse, 1 / math.sqrt(128))
    assert torch.equal(new, out) and torch.equal(new_lse, lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mmq.mmq_paged_attention(q, kc, vc, table, lens, start, out=out, lse=lse)
    for p in (b, a, b):
        fill(p)
        out.fill_(math.nan)
        graph.replay()
        torch.cuda.synchronize()
        _check(p, out, lse, 1 / math.sqrt(128))


@pytest.mark.parametrize("d,page", [(128, 16), (128, 6)])
def test_cache_past_32_bits_of_elements(mmq, d, page):
    """Pages whose first element lies past 2^31 (and past 2^32 bytes)."""
    p = _problem(BF16, [1, 40], [300, 500], 2, 2, d, page)
    small = p["kc"].shape[0]
    pages = 2 ** 31 // (page * 2 * d) + small + 5
    kc, vc = (torch.empty((pages, page, 2, d), dtype=BF16, device="cuda") for _ in range(2))
    kc[pages - small:], vc[pages - small:] = p["kc"], p["vc"]
    p["kc"], p["vc"] = kc, vc
    p["table"] = torch.where(p["table"] >= 0, p["table"] + (pages - small), -1)
    out, lse = _attend(mmq, p)
    _check(p, out, lse, 1 / math.sqrt(d))
    k = torch.randn((3, 2, d), device="cuda")
    slots = torch.tensor([pages * page - 1, -1, (pages - small) * page], device="cuda")
    mmq.mmq_kv_write(k, -k, kc, vc, slots)
    assert torch.equal(kc[-1, -1], k[0].to(BF16)) and torch.equal(vc[pages - small, 0], -k[2].to(BF16))


@pytest.mark.parametrize("page", [16, 5])
def test_page_ids_out_of_the_cache_are_reported(mmq, page):
    p = _problem(F16, [1, 1], [100, 100], 4, 2, 64, page)
    for bad in (-1, p["kc"].shape[0], 2 ** 31 - 1, -(2 ** 31)):
        table = p["table"].clone()
        table[1, 1] = bad
        out, lse = mmq.mmq_paged_attention(p["q"], p["kc"], p["vc"], table, p["seq_lens"], p["q_start"], lse=True)
        assert mmq.mmq_last_device_error() == mmq.MMQ_ERR_DEVICE_INDEX
        assert mmq.mmq_last_device_error() == 0
        ref, _, tol, _ = _reference(p, 1 / 8, True, 0)
        assert ((out.double() - ref).abs() <= tol)[0].all()  # the other request is as it was
    mmq.mmq_paged_attention(p["q"], p["kc"], p["vc"], p["table"], _i32([100, 10 ** 6]), p["q_start"])
    assert mmq.mmq_last_device_error() == mmq.MMQ_ERR_DEVICE_INDEX


def test_attention_refusals(mmq):
    p = _problem(F16, [2], [40], 4, 2, 64, 16)
    args = [p["q"], p["kc"], p["vc"], p["table"], p["seq_lens"], p["q_start"]]

    def refused(error, *swap, **kw):
        a = list(args)
        for i, x in zip(swap[::2], swap[1::2]):
            a[i] = x
        with pytest.raises(error) as e:
            mmq.mmq_paged_attention(*a, **kw)
        return e.value

    refused(TypeError, 0, p["q"].cpu())
    refused(ValueError, 0, p["q"].to(BF16))
    refused(ValueError, 0, p["q"][:, :3])
    refused(ValueError, 0, p["q"].transpose(1, 2))
    refused(ValueError, 2, p["vc"].float())
    refused(ValueError, 3, p["table"].long())
    refused(ValueError, 4, p["seq_lens"].long())
    refused(ValueError, 5, p["q_start"][:1])
    refused(ValueError, out=p["q"][:1])
    refused(ValueError, lse=torch.empty(3, device="cuda"))
    assert refused(mmq.MMQError, out=torch.empty((2, 4, 64), dtype=BF16, device="cuda")).code == -3
    assert refused(mmq.MMQError, scale=0.0).code == -1
    assert refused(mmq.MMQError, scale=-1.0).code == -1
    assert refused(mmq.MMQError, window=-1).code == -1
    odd = torch.empty((2, 4, 65), dtype=F16, device="cuda")[:, :, 1:]
    assert refused(mmq.MMQError, 0, odd).code == -2
    kc = torch.zeros((2, 16, 2, 20), dtype=F16, device="cuda")
    assert refused(mmq.MMQError, 0, p["q"][:, :, :20], 1, kc, 2, kc).code == -1  # head width 20
    for empty in (mmq.mmq_paged_attention(p["q"][:0], *args[1:])[0],
                  mmq.mmq_paged_attention(p["q"][:0], p["kc"], p["vc"], p["table"][:0], p["seq_lens"][:0], p["q_start"][:1])[0]):
        assert empty.shape == (0, 4, 64)


# ---------------------------------------------------------------- K and V rows
@pytest.mark.parametrize("src", [F32, F16, BF16], ids=["f32", "f16", "bf16"])
@pytest.mark.parametrize("dst", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("t,heads,d,page", [(1, 1, 8, 1), (3, 2, 64, 16), (1000, 4, 128, 16), (77, 3, 96, 7), (130, 8, 256, 64)])
def test_kv_write(mmq, src, dst, t, heads, d, page):
    g = torch.Generator(device="cuda").manual_seed(t + d)
    qkv = torch.randn((t, 3 * heads, d), generator=g, device="cuda").to(src)
    pages = t // page + 5
    for layout in ("nhd", "hnd"):
        shape = (pages, page, heads, d) if layout == "nhd" else (pages, heads, page, d)
        kc, vc = (torch.randn(shape, generator=g, device="cuda").to(dst) for _ in range(2))
        if layout == "hnd":
            kc, vc = kc.permute(0, 2, 1, 3), vc.permute(0, 2, 1, 3)
        want_k, want_v = kc.clone(), vc.clone()
        slots = torch.randperm(pages * page, generator=g, device="cuda")[:t]
        slots[2::5] = -1
        for i, s in enumerate(slots.tolist()):
            if s >= 0:
                want_k[s // page, s % page] = qkv[i, heads:2 * heads].to(dst)
                want_v[s // page, s % page] = qkv[i, 2 * heads:].to(dst)
        mmq.mmq_kv_write(qkv[:, heads:2 * heads], qkv[:, 2 * heads:], kc, vc, slots.contiguous())
        assert torch.equal(kc, want_k) and torch.equal(vc, want_v)


def test_kv_write_reports_slots_past_the_cache(mmq):
    kc, vc = (torch.zeros((4, 8, 2, 16), dtype=F16, device="cuda") for _ in range(2))
    k = torch.ones((3, 2, 16), device="cuda")
    mmq.mmq_kv_write(k, k, kc, vc, torch.tensor([31, 32, -5], device="cuda"))
    assert mmq.mmq_last_device_error() == mmq.MMQ_ERR_DEVICE_INDEX
    assert kc.sum() == 32 and (kc[3, 7] == 1).all()
    mmq.mmq_kv_write(k[:0], k[:0], kc, vc, torch.empty(0, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        mmq.mmq_kv_write(k, k[:2], kc, vc, torch.zeros(3, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        mmq.mmq_kv_write(k, k, kc, vc, torch.zeros(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(mmq.MMQError):
        mmq.mmq_kv_write(torch.ones((3, 2, 17), device="cuda")[:, :, 1:], k, kc, vc, torch.zeros(3, dtype=torch.int64, device="cuda"))


# ---------------------------------------------------------------- page tables
def _tables_reference(cached, new, held, table, free, page, room):
    table = table.copy()
    n = len(cached)
    width = table.shape[1]
    q_start, seq, now, missing, at, want = [0], [], [], 0, 0, 0
    slots, positions = np.full(room, -1, np.int64), np.full(room, -1, np.int32)
    for b in range(n):
        total = cached[b] + new[b]
        need = -(-total // page)
        got = held[b]
        for j in range(held[b], need):
            if j >= width:
                missing += 1
                continue
            if want < len(free):
                table[b, j] = free[want]
                at += 1
                got += 1
            else:
                table[b, j] = -1
                missing += 1
            want += 1
        for i in range(new[b]):
            t = q_start[-1] + i
            if t < room:
                pos = cached[b] + i
                positions[t] = pos
                j = pos // page
                if j < min(max(need, held[b]), width) and table[b, j] >= 0:
                    slots[t] = int(table[b, j]) * page + pos % page
        q_start.append(q_start[-1] + new[b])
        seq.append(total)
        now.append(got)
    return q_start, seq, now, slots, positions, [at, missing], table


@pytest.mark.parametrize("n,old,fresh,page,spare,short,room_off", [
    (1, 0, 1, 16, 0, 0, 0), (1, 40, 5, 1, 0, 0, 7), (8, 300, 1, 16, 1, 0, 0), (33, 50, 20, 8, 2, 0, 100), (700, 400, 90, 64, 1, 0, 3),
    (600, 10, 3, 4, 1, 0, -50), (40, 100, 30, 16, 1, 25, 0), (5000, 20, 2, 16, 1, 0, 0), (0, 1, 1, 16, 0, 0, 5)])
def test_page_tables(mmq, n, old, fresh, page, spare, short, room_off):
    """short: that many pages fewer than needed; room_off: token rows beyond (or short of) the new tokens."""
    rng = np.random.default_rng(n + page)
    cached = rng.integers(0, old + 1, n)
    new = rng.integers(0, fresh + 1, n) if n > 1 else np.array([fresh] * n)
    held = -(-cached // page) + rng.integers(0, spare + 1, n)
    need = int(np.maximum(-(-(cached + new) // page) - held, 0).sum())
    width = int(max((-(-(cached + new) // page)).max(initial=0), held.max(initial=0))) + 1
    ids = rng.permutation(int(held.sum() + need) + 10)
    table = np.full((n, width), -1, np.int32)
    at = 0
    for b in range(n):
        table[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
    free = ids[at:at + need + 10 - (short + 10 if short else 0)].astype(np.int32)
    room = int(new.sum()) + room_off
    want = _tables_reference(cached.tolist(), new.tolist(), held.tolist(), table, free, page, room)
    tab = torch.from_numpy(table).cuda()
    for _ in range(2):  # the second call finds what the first wrote
        t = mmq.mmq_page_tables(_i32(cached.tolist()), _i32(new.tolist()), _i32(held.tolist()), tab, _i32(free.tolist()), page, room)
        for got, ref in zip((*t, tab), want):
            assert np.array_equal(got.cpu().numpy().ravel(), np.asarray(ref).ravel())


def test_page_tables_with_a_narrow_table(mmq):
    """Needs beyond the table's row are missing pages, not writes past it; the row pitch is the caller's."""
    wide = torch.full((3, 8), 77, dtype=torch.int32, device="cuda")
    wide[0, 0] = 5
    t = mmq.mmq_page_tables(_i32([4, 0, 0]), _i32([9, 40, 0]), _i32([1, 0, 0]), wide[:, :3], _i32(list(range(20, 40))), 4, 60)
    want = _tables_reference([4, 0, 0], [9, 40, 0], [1, 0, 0], wide[:, :3].cpu().numpy() * 0 + np.array([[5, 77, 77], [77] * 3, [77] * 3]),
                             list(range(20, 40)), 4, 60)
    for got, ref in zip((*t, wide[:, :3]), want):
        assert np.array_equal(got.cpu().numpy().ravel(), np.asarray(ref).ravel())
    assert (wide[:, 3:] == 77).all()
    assert t.taken.tolist() == [5, 8]


def test_page_tables_refusals(mmq):
    one = _i32([1])
    with pytest.raises(TypeError):
        mmq.mmq_page_tables(one.cpu(), one, one, one[None], one, 16, 4)
    with pytest.raises(ValueError):
        mmq.mmq_page_tables(one, _i32([1, 2]), one, one[None], one, 16, 4)
    with pytest.raises(ValueError):
        mmq.mmq_page_tables(one, one, one, one, one, 16, 4)
    with pytest.raises(mmq.MMQError):
        mmq.mmq_page_tables(one, one, one, one[None], one, 0, 4)
    many = torch.zeros(8193, dtype=torch.int32, device="cuda")
    with pytest.raises(mmq.MMQError) as e:
        mmq.mmq_page_tables(many, many, many, many[:, None], one, 16, 4)
    assert e.value.code == -7


# ---------------------------------------------------------------- verification
def _verify_reference(target, draft, tokens, n_draft, u, noise):
    """(tokens, accepted) by the definition, fp32 operation by operation, and each request's weights."""
    nreq, k1, vocab = target.shape
    out, accepted, weights = np.full((nreq, k1), -1, np.int32), np.zeros(nreq, np.int32), []
    for b in range(nreq):
        a = 0
        while a < n_draft[b]:
            x = tokens[b, a]
            q = draft[b, a, x] if draft is not None else np.float32(1)
            if not (np.float32(u[b, a] * q) < target[b, a, x]):
                break
            out[b, a] = x
            a += 1
        w = target[b, a].copy()
        if a < n_draft[b]:
            left = w.copy()
            if draft is not None:
                left = w - draft[b, a]
            else:
                left[tokens[b, a]] = 0
            left = np.where(left > 0, left, np.float32(0))
            if (left > 0).any():
                w = left
        key = np.where(w > 0, w / noise[b], np.float32(0))
        out[b, a] = int(np.argmax(key)) if (key > 0).any() else -1
        accepted[b] = a
        weights.append(w)
    return out, accepted, weights


def _drafts(nreq, k, vocab, seed, dtype=F32, sharp=3.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    z = torch.randn((nreq, k + 1, vocab), generator=g, device="cuda") * sharp
    target = torch.softmax(z, -1).to(dtype)
    q = torch.softmax(z[:, :k] + 0.5 * torch.randn((nreq, k, vocab), generator=g, device="cuda"), -1)
    tokens = torch.multinomial(q.reshape(-1, vocab), 1, generator=g).view(nreq, k).int() if k else torch.zeros((nreq, 0), dtype=torch.int32, device="cuda")
    n_draft = torch.randint(0, k + 1, (nreq,), generator=g, device="cuda", dtype=torch.int32)
    u = torch.rand((nreq, k), generator=g, device="cuda")
    noise = torch.empty((nreq, vocab), device="cuda").exponential_(generator=g)
    return target, q.to(dtype), tokens, n_draft, u, noise


@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=["f32", "f16", "bf16"])
@pytest.mark.parametrize("nreq,k,vocab", [(1, 0, 1), (3, 1, 5), (17, 4, 1000), (40, 7, 4097), (2, 40, 333), (5, 3, 32000), (32, 2, 40000), (33, 2, 20000)])
def test_verify_against_the_definition(mmq, dtype, nreq, k, vocab):
    target, draft, tokens, n_draft, u, noise = _drafts(nreq, k, vocab, seed=vocab, dtype=dtype)
    for q, n in ((draft, n_draft), (None, n_draft), (draft, None)):
        got, accepted = mmq.mmq_verify_draft(target, q, tokens, n, u, noise)
        f = lambda x: None if x is None else x.float().cpu().numpy()  # noqa: E731
        count = np.full(nreq, k) if n is None else n.cpu().numpy()
        want, kept, weights = _verify_reference(f(target), f(q), tokens.cpu().numpy(), count, f(u), f(noise))
        assert np.array_equal(accepted.cpu().numpy(), kept)
        assert np.array_equal(got.cpu().numpy(), want)
        # in 64 bits no other token's key is larger by more than the two fp32 roundings
        e = f(noise).astype(np.float64)
        for b in range(nreq):
            drawn = got[b, kept[b]].item()
            key = weights[b].astype(np.float64) / e[b]
            assert drawn >= 0 and key[drawn] * (1 + 2.0 ** -22) >= key.max()


def test_verify_edges(mmq):
    """Refusal at certainty, ties, rows without weight, NaN, p equal to q, strided probabilities."""
    v = 37
    noise = torch.ones((6, v), device="cuda")
    target = torch.zeros((6, 3, v), device="cuda")
    draft = torch.zeros((6, 2, v), device="cuda")
    tokens = torch.zeros((6, 2), dtype=torch.int32, device="cuda")
    n = _i32([2, 2, 1, 2, 0, 2])
    u = torch.zeros((6, 2), device="cuda")
    target[0, 0, [9, 20]] = 0.5     # token 0 has no weight: refused at u = 0; two equal weights behind it
    draft[0, 0, 0] = 1
    target[1, :2, 0] = 1            # both kept, then nothing to draw from
    draft[1, :, 0] = 1
    target[2, 0] = math.nan         # NaN is never kept and never drawn
    target[2, 0, 11] = 0.25
    draft[2, 0, 0] = 1
    target[3, 0, 0] = 0.5           # p = q everywhere, refused by chance: drawn from p
    draft[3, 0, 0] = 0.5
    u[3, 0] = 1.0
    target[4, 0, 36] = 1            # nothing drafted
    target[5, 0, 0] = 1             # kept, then refused: p - q on the rest
    target[5, 1, 4] = 0.3
    target[5, 1, 5] = 0.7
    draft[5, 0, 0] = 1
    draft[5, 1, 5] = 0.65
    draft[5, 1, 4] = 0.1
    tokens[5, 1] = 4
    u[5, 1] = 0.999999
    target[5, 1, 4], draft[5, 1, 4] = 0.1, 0.35
    got, accepted = mmq.mmq_verify_draft(target, draft, tokens, n, u, noise)
    assert got.tolist() == [[9, -1, -1], [0, 0, -1], [11, -1, -1], [0, -1, -1], [36, -1, -1], [0, 5, -1]]
    assert accepted.tolist() == [0, 2, 0, 0, 0, 1]
    wide = torch.zeros((6, 4, v + 3), device="cuda")
    wide[:, :3, 1:v + 1] = target
    again, _ = mmq.mmq_verify_draft(wide[:, :3, 1:v + 1], draft, tokens, n, u, noise)
    assert torch.equal(again, got)


def test_verify_reports_tokens_outside_the_vocabulary(mmq):
    for vocab, draft_given in ((50, True), (50, False), (48, False)):
        target, draft, tokens, _, u, noise = _drafts(3, 2, vocab, seed=3)
        tokens[1, 0] = vocab
        tokens[2, 0] = -1
        got, accepted = mmq.mmq_verify_draft(target, draft if draft_given else None, tokens, None, u, noise)
        assert mmq.mmq_last_device_error() == mmq.MMQ_ERR_DEVICE_INDEX
        assert accepted[1:].tolist() == [0, 0]
        assert ((got[1:, 0] >= 0) & (got[1:, 0] < vocab)).all()


def test_verify_draws_from_the_target(mmq):
    """Kept and drawn tokens together follow p whatever the draft was: 40000 requests, each count within 5 deviations."""
    n, v = 40000, 6
    g = torch.Generator(device="cuda").manual_seed(5)
    p = torch.tensor([0.4, 0.05, 0.25, 0.0, 0.2, 0.1], device="cuda")
    q = torch.tensor([0.1, 0.3, 0.2, 0.1, 0.2, 0.1], device="cuda")
    tokens = torch.multinomial(q, n, replacement=True, generator=g).int()[:, None]
    got, _ = mmq.mmq_verify_draft(p.expand(n, 2, v).contiguous(), q.expand(n, 1, v).contiguous(), tokens, None,
                                  torch.rand((n, 1), generator=g, device="cuda"),
                                  torch.empty((n, v), device="cuda").exponential_(generator=g))
    count = torch.bincount(got[:, 0].long(), minlength=v).double()
    sd = (n * p * (1 - p)).sqrt().clamp(min=1e-9)
    assert ((count - n * p).abs() <= 5 * sd).all()


def test_verify_refusals(mmq):
    target, draft, tokens, n, u, noise = _drafts(2, 3, 64, seed=1)
    with pytest.raises(TypeError):
        mmq.mmq_verify_draft(target.cpu(), draft, tokens, n, u, noise)
    with pytest.raises(ValueError):
        mmq.mmq_verify_draft(target, draft[:, :2], tokens, n, u, noise)
    with pytest.raises(ValueError):
        mmq.mmq_verify_draft(target, draft, tokens.long(), n, u, noise)
    with pytest.raises(ValueError):
        mmq.mmq_verify_draft(target, draft, tokens, n, u, noise[:, :63])
    with pytest.raises(ValueError):
        mmq.mmq_verify_draft(target.transpose(1, 2), None, tokens, n, u, noise)
    with pytest.raises(mmq.MMQError) as e:
        mmq.mmq_verify_draft(target.double(), None, tokens, n, u, noise)
    assert e.value.code == -3
