"""What differs from request to request in a step, on the GPU against plain implementations: pages in Python integers, token
probabilities and adapters in 64 bits.

Tolerances, derived before any run.  Adjusted logits: four fp32 operations and one for each bias, each half a step
(2^-24) of what has been added up to there.  Probabilities: those errors over the temperature, twice (the largest logit has
them too); the exponent's argument carries 2^-23 of itself; exp2, the sum, the division and the joins stay within 2^-20.
Adapters: x and the inner sums as three bf16 terms, 2^-27 each, fp16 weights as two terms of which the products of the
smallest ones are left out, 2^-26; fp32 sums in chains of at most 128 steps of 2^-23: 2^-15 of the sum of magnitudes in all;
the last addition rounds to fp32."""
import math
import random

import pytest
import torch

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
ARG, ALIGN, UNSUPPORTED = -1, -2, -7
HALF_STEP = {F32: 2.0 ** -24, F16: 2.0 ** -11, BF16: 2.0 ** -8}


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


def _f32(x):
    return torch.tensor(x, dtype=torch.float32, device="cuda")


def _recorded(mmq):
    return mmq.mmq_last_device_error() == mmq.MMQ_ERR_DEVICE_INDEX


# ---------------------------------------------------------------- forks
def _fork_reference(rows, parents, lens, page, pages, width):
    """rows: each old row's pages.  Returns what mmq_page_fork gives, as lists."""
    fresh, writable = [], []
    for p, n in zip(parents, lens):
        had = rows[p] if p >= 0 else []
        need = min(-(-max(n, 0) // page), len(had), width)
        fresh.append(had[:need])
        full = max(n, 0) // page
        writable.append(had[full] if full < need and n % page else None)
    full_pages = {x for got, w, n in zip(fresh, writable, lens) for x in got[: max(n, 0) // page]}
    first = {}
    for b, w in enumerate(writable):
        if w is not None:
            first.setdefault(w, b)
    keeps = [w is not None and w not in full_pages and first[w] == b for b, w in enumerate(writable)]
    held = full_pages | {w for w, k in zip(writable, keeps) if k}
    free = [x for x in range(pages) if x not in held]
    pairs, tokens, missing = [], [], 0
    for b, (w, k) in enumerate(zip(writable, keeps)):
        pairs.append([-1, -1])
        tokens.append(0)
        if w is None or k:
            continue
        if free:
            to = free.pop(0)
            pairs[b], tokens[b] = [w, to], lens[b] % page
        else:
            to, missing = -1, missing + 1
        fresh[b] = fresh[b][:-1] + [to]
    return {"table": [x + [-1] * (width - len(x)) for x in fresh], "n_blocks": [len(x) for x in fresh], "pairs": pairs, "tokens": tokens,
            "free": free + [-1] * (pages - len(free)), "counts": [len(free), missing]}


def _rows(r, count, page, most, pages, shared=0.5, spare=True):
    """Rows of random pages, some of them sharing the front of the row before; their lengths."""
    ids = r.sample(range(pages), pages)
    rows, lens = [], []
    for b in range(count):
        n = r.randint(0, most)
        need = -(-n // page) + (spare and r.random() < 0.2)
        front = []
        if rows and r.random() < shared:
            same = min(need, lens[-1] // page, n // page)
            front = rows[-1][: r.randint(0, same)]
        own = need - len(front)
        if own > len(ids):
            n, own, need = 0, 0, 0
            front = []
        rows.append(front + [ids.pop() for _ in range(own)])
        lens.append(min(n, len(rows[-1]) * page))
    return rows, lens


def _table(rows, width, stride=None):
    t = torch.full((len(rows), stride or width), -7, dtype=torch.int32)[:, :width]
    for b, x in enumerate(rows):
        t[b, : len(x)] = torch.tensor(x, dtype=torch.int32)
    if not stride:
        return t.contiguous().cuda()
    whole = torch.full((len(rows), stride), -7, dtype=torch.int32, device="cuda")
    whole[:, :width] = t.cuda()
    return whole[:, :width]


def _same_fork(f, want):
    assert f.block_table.tolist() == want["table"]
    assert f.n_blocks.tolist() == want["n_blocks"] and f.pairs.tolist() == want["pairs"] and f.tokens.tolist() == want["tokens"]
    assert f.counts.tolist() == want["counts"] and f.free_pages.tolist() == want["free"]


FORKS = [
    # old rows, new rows, page, longest, pages of the cache
    (1, 1, 16, 1, 1), (1, 3, 16, 40, 9), (4, 4, 1, 30, 200), (8, 8, 16, 500, 700), (5, 40, 4, 60, 100), (40, 3, 8, 100, 600),
    (33, 300, 16, 900, 1500), (300, 300, 16, 700, 9000), (1100, 1300, 8, 90, 8000), (9, 9, 256, 5000, 70), (60, 60, 16, 2000, 40000),
    (3, 2000, 32, 3000, 5000), (700, 8192, 2, 11, 6000),
]


@pytest.mark.parametrize("old,new,page,most,pages", FORKS)
@pytest.mark.parametrize("seed", [0, 1])
def test_fork(mmq, old, new, page, most, pages, seed):
    r = random.Random(seed)
    rows, lens = _rows(r, old, page, most, pages)
    width = max(len(x) for x in rows) + r.randint(0, 2) or 1
    parents = [-1 if r.random() < 0.1 else r.randrange(old) for _ in range(new)]
    keep = [r.choice([0, 5]) if p < 0 else max(0, lens[p] - r.choice([0, 0, 0, 1, 3, lens[p] // 2, lens[p]])) for p in parents]
    table, held = _table(rows, width, width + 3 if seed else None), _i32([len(x) for x in rows])
    f = mmq.mmq_page_fork(table, held, _i32(parents), _i32(keep), page, pages)
    want = _fork_reference(rows, parents, [0 if p < 0 else n for p, n in zip(parents, keep)], page, pages, width)
    _same_fork(f, want)
    # the same bits into the caller's buffers, the rows of a wider table among them
    into = mmq.PageFork(torch.full((new, width + 5), 9, dtype=torch.int32, device="cuda")[:, :width], *(torch.empty_like(x) for x in f[1:]))
    got = mmq.mmq_page_fork(table, held, _i32(parents), _i32(keep), page, pages, out=into)
    assert got is into
    _same_fork(got, want)
    if new > 1:
        assert (into.block_table.as_strided((new, 5), (width + 5, 1), into.block_table.storage_offset() + width) == 9).all()


def test_fork_edges(mmq):
    # one parent, three children in the middle of a page: the lowest keeps it
    f = mmq.mmq_page_fork(_table([[3, 5, 1]], 4), _i32([3]), _i32([0, 0, 0]), _i32([9, 9, 9]), 4, 8)
    assert f.block_table.tolist() == [[3, 5, 1, -1], [3, 5, 0, -1], [3, 5, 2, -1]]
    assert f.pairs.tolist() == [[-1, -1], [1, 0], [1, 2]] and f.tokens.tolist() == [0, 1, 1]
    assert f.free_pages.tolist() == [4, 6, 7, -1, -1, -1, -1, -1] and f.counts.tolist() == [3, 0]
    # a child whose writable page is full in its sibling gets a copy, though it is the lowest
    f = mmq.mmq_page_fork(_table([[3, 5, 1]], 3), _i32([3]), _i32([0, 0]), _i32([6, 12]), 4, 8)
    assert f.block_table.tolist() == [[3, 0, -1], [3, 5, 1]] and f.pairs.tolist() == [[5, 0], [-1, -1]] and f.tokens.tolist() == [2, 0]
    # no page left
    f = mmq.mmq_page_fork(_table([[0, 1]], 2), _i32([2]), _i32([0, 0, 0]), _i32([5, 6, 7]), 4, 3)
    assert f.block_table.tolist() == [[0, 1], [0, 2], [0, -1]] and f.counts.tolist() == [0, 1]
    assert f.pairs.tolist() == [[-1, -1], [1, 2], [-1, -1]] and f.tokens.tolist() == [0, 2, 0]
    # nothing there, nothing wanted
    f = mmq.mmq_page_fork(_table([], 0).view(0, 3), _i32([]), _i32([-1, -1]), _i32([4, 0]), 4, 40)
    assert f.block_table.tolist() == [[-1] * 3] * 2 and f.free_pages.tolist() == list(range(40)) and f.counts.tolist() == [40, 0]
    f = mmq.mmq_page_fork(_table([[1]], 1), _i32([1]), _i32([]), _i32([]), 4, 3)
    assert f.free_pages.tolist() == [0, 1, 2] and f.n_blocks.numel() == 0
    f = mmq.mmq_page_fork(_table([[]], 1), _i32([0]), _i32([0]), _i32([0]), 4, 0)
    assert f.counts.tolist() == [0, 0] and f.n_blocks.tolist() == [0]


@pytest.mark.parametrize("many", [False, True])
def test_fork_faults(mmq, many):
    """Bad parents, lengths beyond the pages held and page ids out of the cache are left out and reported."""
    n = 2000 if many else 3
    table = _table([[0, 1]] * n, 6)
    assert not _recorded(mmq)
    f = mmq.mmq_page_fork(table, _i32([2] * n), _i32([n] + [0] * (n - 1)), _i32([8] * n), 4, 9)
    assert _recorded(mmq)
    assert f.n_blocks.tolist() == [0] + [2] * (n - 1) and f.free_pages.tolist() == [2, 3, 4, 5, 6, 7, 8, -1, -1]
    f = mmq.mmq_page_fork(table, _i32([2] * n), _i32([0] * n), _i32([9] + [8] * (n - 1)), 4, 9)
    assert _recorded(mmq)
    assert f.n_blocks.tolist() == [2] * n
    table[0, 1] = 9
    f = mmq.mmq_page_fork(table, _i32([2] * n), _i32([0] * n), _i32([8] * n), 4, 9)
    assert _recorded(mmq) and f.block_table[:, :2].tolist() == [[0, -1]] * n
    f = mmq.mmq_page_fork(table, _i32([2] * n), _i32([0] * n), _i32([7] * n), 4, 9)
    assert _recorded(mmq) and f.block_table[:, :2].tolist() == [[0, -1]] * n and f.counts.tolist() == [8, 0]
    # -1 is no page either
    table[0, 1] = -1
    mmq.mmq_page_fork(table, _i32([2] * n), _i32([0] * n), _i32([8] * n), 4, 9)
    assert _recorded(mmq)


# ---------------------------------------------------------------- compaction
@pytest.mark.parametrize("count,page,most,pages", [(1, 16, 1, 1), (1, 16, 90, 8), (8, 16, 500, 700), (3, 4, 70, 200), (300, 16, 700, 9000),
                                                   (1100, 8, 90, 40001), (9, 1, 3000, 70000), (2, 16, 40, 1 << 20), (40, 8, 60, 301)])
def test_compact(mmq, count, page, most, pages):
    r = random.Random(count)
    rows, _ = _rows(r, count, page, most, pages)
    width = max(len(x) for x in rows) + 1
    held = sorted({x for row in rows for x in row})
    h = len(held)
    moved, holes = [x for x in held if x >= h], [x for x in range(h) if x not in set(held)]
    to = dict(zip(moved, holes))
    table, n = _table(rows, width, width + 2), _i32([len(x) for x in rows])
    m = mmq.mmq_page_compact(table, n, pages)
    assert m.counts.tolist() == [h, len(moved)]
    assert m.block_table.tolist() == [[to.get(x, x) for x in row] + [-1] * (width - len(row)) for row in rows]
    pairs = [[a, b] for a, b in zip(moved, holes)]
    assert m.pairs[: len(pairs)].tolist() == pairs and (m.pairs[len(pairs):] == -1).all() and m.pairs.shape == (pages // 2, 2)
    into = mmq.PageMoves(*(torch.full_like(x, 5) for x in m))
    assert mmq.mmq_page_compact(table, n, pages, out=into) is into
    assert all(torch.equal(a, b) for a, b in zip(m, into))


def test_compact_faults(mmq):
    for n in (2, 3000):
        m = mmq.mmq_page_compact(_table([[4, 9]] * n, 3), _i32([2] * n), 5)
        assert _recorded(mmq)
        assert m.block_table.tolist() == [[0, -1, -1]] * n and m.counts.tolist() == [1, 1] and m.pairs.tolist() == [[4, 0], [-1, -1]]


# ---------------------------------------------------------------- copies
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("layout", ["nhd", "hnd", "columns"])
@pytest.mark.parametrize("n,page,heads,d", [(1, 1, 1, 8), (5, 16, 4, 128), (9, 5, 3, 72), (300, 16, 2, 64), (3, 256, 8, 256), (40, 64, 1, 96)])
@pytest.mark.parametrize("partial", [False, True])
def test_copy(mmq, dtype, layout, n, page, heads, d, partial):
    g = torch.Generator(device="cuda").manual_seed(n)
    pages = 2 * n + 3
    shape = (pages, heads, page, d) if layout == "hnd" else (pages, page, heads, d)
    kc, vc = (torch.randn(shape, generator=g, device="cuda").to(dtype) for _ in range(2))
    if layout == "columns":  # K and V side by side, NaN behind them
        both = torch.full((pages, page, 3 * heads, d), math.nan, dtype=dtype, device="cuda")
        both[:, :, :heads], both[:, :, heads:2 * heads] = kc, vc
        kc, vc = both[:, :, :heads], both[:, :, heads:2 * heads]
    elif layout == "hnd":
        kc, vc = kc.permute(0, 2, 1, 3), vc.permute(0, 2, 1, 3)
    pairs = torch.randperm(pages, generator=g, device="cuda")[: 2 * n].to(torch.int32).view(n, 2).contiguous()
    pairs[3::5, 0], pairs[4::5, 1] = -1, -1
    tokens = _i32([(3 * i) % (page + 3) - 1 for i in range(n)]) if partial else None
    want = [c.clone() for c in (kc, vc)]
    for c in want:
        for i, (a, b) in enumerate(pairs.tolist()):
            if a >= 0 and b >= 0:
                m = min(max((3 * i) % (page + 3) - 1, 0), page) if partial else page
                c[b, :m] = c[a, :m]
    mmq.mmq_page_copy(kc, vc, pairs, tokens)
    assert torch.equal(kc, want[0]) and torch.equal(vc, want[1])
    if layout == "columns":
        assert both[:, :, 2 * heads:].isnan().all()


def test_copy_edges(mmq):
    kc, vc = torch.randn((2, 4, 3, 2, 8), device="cuda").half()
    k0, v0 = kc.clone(), vc.clone()
    mmq.mmq_page_copy(kc, vc, _i32([]).view(0, 2))
    mmq.mmq_page_copy(kc, vc, _i32([[4, 1], [0, 2], [1, 2 ** 31 - 1]]))
    assert _recorded(mmq)
    k0[2], v0[2] = k0[0], v0[0]
    assert torch.equal(kc, k0) and torch.equal(vc, v0)


def test_copy_past_32_bits(mmq):
    """Pages beyond 2^31 elements of a cache."""
    pages = 2 ** 31 // (16 * 8 * 128) + 40
    kc = torch.empty((pages, 16, 8, 128), dtype=F16, device="cuda")
    vc = torch.empty_like(kc)
    kc[-1], vc[-1] = 1.5, 2.5
    kc[3], vc[3] = -3.0, -4.0
    mmq.mmq_page_copy(kc, vc, _i32([[pages - 1, 2], [3, pages - 2]]))
    assert (kc[2] == 1.5).all() and (vc[2] == 2.5).all() and (kc[-2] == -3).all() and (vc[-2] == -4).all()


# ---------------------------------------------------------------- token probabilities
def _rules_problem(b, k, v, dtype, seed=0, hist=50, bias=5, masks=3, pad=0):
    r = random.Random(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    logits = (torch.randn((b, k + 1, v + pad), generator=g, device="cuda") * 3).to(dtype)[..., :v]
    words = lambda n: [min(v - 1, int(v * r.random() ** 3)) for _ in range(n)]  # noqa: E731
    lens = [r.choice([0, 1, hist, r.randint(0, hist)]) for _ in range(b)]
    tokens = torch.full((b, hist + 2), -5, dtype=torch.int32)
    for i, n in enumerate(lens):
        tokens[i, :n] = torch.tensor(words(n), dtype=torch.int32)
    lists = [[(w, r.uniform(-4, 4)) for w in words(r.choice([0, bias, 2 * bias]))] for _ in range(b)]
    start = [0]
    for x in lists:
        start.append(start[-1] + len(x))
    flat = [x for y in lists for x in y]
    p = {"logits": logits, "tokens": tokens.cuda(), "token_lens": _i32(lens), "prompt_lens": _i32([r.randint(0, n) for n in lens]),
         "draft_tokens": _i32([words(k) for _ in range(b)]).view(b, k), "temperature": _f32([r.choice([0.3, 1.0, 1.7, 0.0]) for _ in range(b)]),
         "repetition": _f32([r.choice([1.0, 1.3, 0.8]) for _ in range(b)]), "frequency": _f32([r.uniform(-0.2, 0.5) for _ in range(b)]),
         "presence": _f32([r.uniform(-0.3, 0.5) for _ in range(b)])}
    if bias:
        p["bias"] = (_i32(start), _i32([x for x, _ in flat]), _f32([x for _, x in flat]))
    if masks:
        bits = torch.rand((masks, -(-v // 32) * 32), generator=g, device="cuda") < 0.4
        bits[0] = False
        if masks > 1:
            bits[1] = False
            bits[1, v - 1] = True
        p["mask"] = (bits.view(masks, -1, 32).long() << torch.arange(32, device="cuda")).sum(-1).to(torch.int32)
        p["mask_rows"] = _i32([[r.randint(-1, masks - 1) for _ in range(k + 1)] for _ in range(b)])
    return p


def _rules_reference(p):
    """probs, adjusted and their tolerances in fp64."""
    b, rows, v = p["logits"].shape
    x = p["logits"].double().clone()
    size = x.abs()
    one = lambda n, z: p[n].tolist() if p.get(n) is not None else [z] * b  # noqa: E731
    rho, alpha, beta, temperature = one("repetition", 1.0), one("frequency", 0.0), one("presence", 0.0), one("temperature", 1.0)
    for i in range(b):
        width = p["tokens"].shape[1] if p.get("tokens") is not None else 0
        n = int(p["token_lens"][i]) if p.get("token_lens") is not None else width
        m = int(p["prompt_lens"][i]) if p.get("prompt_lens") is not None else 0
        said = p["tokens"][i, :n].tolist() if width else []
        for j in range(rows):
            drafted = p["draft_tokens"][i, :j].tolist() if p.get("draft_tokens") is not None else []
            times = {}
            for t in said[m:] + drafted:
                times[t] = times.get(t, 0) + 1
            ids = torch.tensor(sorted(set(said + drafted)), dtype=torch.long, device="cuda")
            if ids.numel():
                c = torch.tensor([times.get(t, 0) for t in ids.tolist()], dtype=torch.float64, device="cuda")
                y = x[i, j, ids]
                y = torch.where(y > 0, y / rho[i], y * rho[i])
                size[i, j, ids] = y.abs() + c * abs(alpha[i]) + abs(beta[i])
                x[i, j, ids] = y - c * alpha[i] - (c > 0) * beta[i]
            if p.get("bias") is not None:
                start, at, value = (z.tolist() for z in p["bias"])
                for e in range(start[i], start[i + 1]):
                    x[i, j, at[e]] += value[e]
                    size[i, j, at[e]] += 2 * abs(value[e])
            if p.get("mask") is not None:
                which = int(p["mask_rows"][i, j]) if p.get("mask_rows") is not None else i * rows + j
                if which >= 0:
                    bits = (p["mask"][which][:, None] >> torch.arange(32, device="cuda", dtype=torch.int32) & 1).flatten()[:v].bool()
                    x[i, j] = torch.where(bits, x[i, j], -math.inf)
    off = size * 6 * 2.0 ** -24
    heat = torch.tensor(temperature, dtype=torch.float64, device="cuda")[:, None, None]
    z = x / torch.where(heat > 0, heat, 1.0)
    top = z.amax(-1, keepdim=True)
    z = z - torch.where(top > -math.inf, top, 0.0)
    e = torch.exp(z)
    total = e.sum(-1, keepdim=True)
    probs = torch.where(total > 0, e / total, 0.0)
    worst = torch.where(x > -math.inf, off, 0.0).amax(-1, keepdim=True) / torch.where(heat > 0, heat, 1.0)
    tol = probs * (2.0 ** -20 + 2 * worst + 2.0 ** -23 * torch.where(z > -math.inf, z.abs(), 0.0)) + 2.0 ** -126
    first = (x == x.amax(-1, keepdim=True)) & (x > -math.inf)
    first &= torch.cumsum(first, -1) == 1
    probs, tol = torch.where(heat > 0, probs, first.double()), torch.where(heat > 0, tol, 0.0)
    return probs, x, tol, off


def _check_rules(mmq, p, probs=True, adjusted=True, ref=None):
    logits = p["logits"]
    got, x = mmq.mmq_token_probs(**p, probs=probs, adjusted=adjusted)
    want, wx, tol, off = ref or _rules_reference(p)
    if got is not None:
        more = HALF_STEP[got.dtype] * want if got.dtype != F32 else 0.0
        small = 2.0 ** -25 if got.dtype == F16 else 2.0 ** -134 if got.dtype == BF16 else 0.0  # half the smallest step
        assert got.shape == logits.shape and torch.isfinite(got).all()
        worst = ((got.double() - want).abs() - tol * 1.01 - more - small).max().item()
        assert worst <= 0, worst
    if x is not None:
        assert torch.equal(torch.isinf(x), torch.isinf(wx))
        fine = ~torch.isinf(wx)
        assert ((x.double() - wx).abs()[fine] - (off + HALF_STEP[x.dtype] * wx.abs() * 1.01 + (2.0 ** -25 if x.dtype == F16 else 0))[fine]).max().item() <= 0 if fine.any() else True
    return got, x


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("b,k,v", [(1, 0, 1), (2, 1, 7), (1, 0, 33), (3, 2, 255), (2, 0, 1000), (5, 3, 1003), (2, 4, 4096), (3, 1, 10007), (2, 2, 32000), (1, 1, 100277)])
def test_probs(mmq, b, k, v, dtype):
    _check_rules(mmq, _rules_problem(b, k, v, dtype, seed=v))


@pytest.mark.parametrize("left", ["tokens", "draft_tokens", "temperature", "repetition", "frequency", "presence", "bias", "mask", "prompt_lens", "token_lens", "all"])
def test_probs_without(mmq, left):
    p = _rules_problem(4, 2, 1203, F32, seed=5)
    if left == "token_lens":
        p["tokens"].clamp_(min=0)
    gone = {"tokens": ["tokens", "token_lens", "prompt_lens"], "mask": ["mask", "mask_rows"], "all": [n for n in p if n != "logits"]}.get(left, [left])
    _check_rules(mmq, {n: x for n, x in p.items() if n not in gone})


@pytest.mark.parametrize("out", [F32, F16, BF16])
@pytest.mark.parametrize("pad", [0, 1, 4, 5])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_probs_strides_and_types(mmq, out, pad, dtype):
    p = _rules_problem(3, 2, 2049, dtype, seed=pad, pad=pad)
    whole = [torch.full((3, 3, 2049 + 2 * pad), 7.0, dtype=out, device="cuda") for _ in range(2)]
    a, x = (w[..., pad:pad + 2049] for w in whole)
    _check_rules(mmq, p, probs=a, adjusted=x)
    for w in whole:
        assert (w[..., :pad] == 7).all() and (w[..., pad + 2049:] == 7).all()


def test_probs_in_place_and_alone(mmq):
    for dtype in (F32, F16):
        p = _rules_problem(5, 3, 5003, dtype, seed=1)
        ref = _rules_reference(p)
        a, none = _check_rules(mmq, p, adjusted=None, ref=ref)
        assert none is None
        none, x = _check_rules(mmq, p, probs=None, ref=ref)
        assert none is None
        b, x = _check_rules(mmq, p, adjusted=p["logits"], ref=ref)
        assert x is p["logits"] and torch.equal(a, b)


def test_probs_of_a_request_without_all_rows(mmq):
    p = _rules_problem(4, 3, 777, F32, seed=2)
    a, _ = mmq.mmq_token_probs(**p)
    n = [0, 3, 1, 2]
    into = torch.full_like(a, -2.0)
    adjusted = torch.full_like(a, -3.0)
    mmq.mmq_token_probs(**p, n_draft=_i32(n), probs=into, adjusted=adjusted)
    for i, m in enumerate(n):
        assert torch.equal(into[i, : m + 1], a[i, : m + 1]) and (into[i, m + 1:] == -2).all() and (adjusted[i, m + 1:] == -3).all()


def test_probs_edges(mmq):
    inf, nan = math.inf, math.nan
    v = 300
    x = torch.randn((8, 1, v), device="cuda")
    x[1, 0] = -inf                      # no token at all
    x[2, 0, 7], x[2, 0, 200] = inf, nan  # hidden by the mask
    x[3, 0, 100] = nan
    x[4, 0, 100] = inf
    x[5, 0] = 2.5                       # ties
    x[6, 0] = torch.finfo(F32).min      # the type's lowest value, and one token above
    x[6, 0, 150] = -1.0
    x[7, 0, 9] = nan
    mask = torch.full((1, 10), -1, dtype=torch.int32, device="cuda")
    mask[0, 0] = ~(1 << 7)
    mask[0, 200 // 32] = ~(1 << 200 % 32)
    rows = _i32([[-1], [-1], [0], [-1], [-1], [-1], [-1], [-1]])
    p, adjusted = mmq.mmq_token_probs(x, mask=mask, mask_rows=rows, adjusted=True)
    p = p[:, 0]
    assert abs(p[0].sum().item() - 1) < 1e-5 and (p[1] == 0).all()
    assert p[2, 7] == 0 and p[2, 200] == 0 and abs(p[2].double().sum().item() - 1) < 1e-5 and adjusted[2, 0, 200] == -inf
    assert p[3].isnan().all() and p[4].isnan().all() and p[7].isnan().all()
    assert (p[5] - 1 / v).abs().max() < 1e-8
    assert p[6, 150] == 1 and p[6].sum() == 1
    q = mmq.mmq_token_probs(x, mask=mask, mask_rows=rows, temperature=_f32([0.0, 0, 0, 0, 0, 0, -1, nan]))[0][:, 0]
    assert q[0, x[0, 0].argmax()] == 1 and q[0].sum() == 1 and (q[1] == 0).all() and q[2].sum() == 1 and q[3].isnan().all()
    assert q[4, 100] == 1 and q[4].sum() == 1 and q[5, 0] == 1 and q[5].sum() == 1 and q[6, 150] == 1 and q[6].sum() == 1
    assert q[7].isnan().all()
    # temperatures at the ends of their range; 0 and -0 are a tie
    x = torch.randn((3, 1, 1000), device="cuda")
    x[2] = -1.0
    x[2, 0, 900], x[2, 0, 500] = 0.0, -0.0
    q = mmq.mmq_token_probs(x, temperature=_f32([1e-44, 3e38, 0.0]))[0][:, 0]
    assert q[0, x[0, 0].argmax()] == 1 and q[0].sum() == 1 and (q[1] - 1e-3).abs().max() < 1e-8 and q[2, 500] == 1 and q[2, 900] == 0


def test_probs_biases_of_one_token_add_up_in_order(mmq):
    x = torch.zeros((1, 1, 500), device="cuda")
    ids, values = [400] * 70 + [3, 400, 3], [1.0, 1e8, -1e8, 0.5] * 17 + [0.25, 2.0] + [7.0, 3.0, 1e-3]
    want = {3: torch.zeros((), dtype=F32), 400: torch.zeros((), dtype=F32)}
    for i, value in zip(ids, values):
        want[i] = want[i] + torch.tensor(value, dtype=F32)
    _, y = mmq.mmq_token_probs(x, bias=(_i32([0, 73]), _i32(ids), _f32(values)), probs=None, adjusted=True)
    assert y[0, 0, 400].item() == want[400].item() and y[0, 0, 3].item() == want[3].item() and (y != 0).sum() == 2


@pytest.mark.parametrize("width", [32000, 40000])
def test_probs_of_long_rows_of_tokens(mmq, width):
    v = 3001
    tokens = torch.full((2, width), 17, dtype=torch.int32, device="cuda")
    tokens[1, : width // 2] = 18
    x = torch.zeros((2, 1, v), device="cuda")
    _, y = mmq.mmq_token_probs(x, tokens=tokens, frequency=_f32([1.0, 1.0]), prompt_lens=_i32([0, 100]), probs=None, adjusted=True)
    assert y[0, 0, 17] == -width and y[1, 0, 17] == -width // 2 and y[1, 0, 18] == -(width // 2 - 100)
    assert (y[0, 0, 16], y[0, 0, 18]) == (0, 0)


def test_probs_largest_vocabulary(mmq):
    v = 2 ** 18
    for dtype in (F32, BF16):
        _check_rules(mmq, _rules_problem(1, 1, v, dtype, seed=3, hist=300, bias=50, masks=2))
    with pytest.raises(mmq.MMQError) as e:
        mmq.mmq_token_probs(torch.empty((1, 1, v + 1), device="cuda"))
    assert e.value.code == -7


def test_probs_faults(mmq):
    """What is out of range is left out and reported; the rest stays as it is."""
    p = _rules_problem(2, 2, 400, F32, seed=9)
    p["token_lens"], p["prompt_lens"] = _i32([6, 6]), _i32([2, 2])
    p["tokens"][:, :6] = _i32([[1, 2, 3, 3, 4, 5], [7, 7, 8, 8, 9, 9]])
    want = mmq.mmq_token_probs(**p, adjusted=True)
    assert not _recorded(mmq)

    def same(**kw):
        got = mmq.mmq_token_probs(**{**p, **kw}, adjusted=True)
        assert _recorded(mmq), kw.keys()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), kw.keys()

    tokens = torch.cat([p["tokens"][:, :6], _i32([[400, -1], [2 ** 31 - 1, -2 ** 31]])], 1)
    same(tokens=tokens, token_lens=_i32([8, 8]))
    same(tokens=p["tokens"][:, :6].contiguous(), token_lens=_i32([7, 6]))
    start, ids, values = p["bias"]
    same(bias=(start, torch.cat([ids]), values), mask_rows=torch.where(p["mask_rows"] < 0, 3, p["mask_rows"]))
    same(mask_rows=torch.where(p["mask_rows"] < 0, -2, p["mask_rows"]))
    n = start[1].item()
    more = (_i32([0, n + 2, start[2].item() + 2]), torch.cat([ids[:n], _i32([400, -1]), ids[n:]]), torch.cat([values[:n], _f32([1, 1]), values[n:]]))
    same(bias=more)
    far = start.clone()
    far[2] += 1
    same(bias=(far, ids, values))
    same(n_draft=_i32([3, 2]))


# ---------------------------------------------------------------- adapters
def _lora_problem(lens, adapters, n, into, out, rank, dtype, x_dtype=F32, seed=0, tail=0, ranks=None, x_pad=0, y_pad=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = sum(lens) + tail
    start = [0]
    for m in lens:
        start.append(start[-1] + m)
    p = {"x": torch.randn((t, into + x_pad), generator=g, device="cuda").to(x_dtype)[:, :into],
         "y": torch.randn((t, out + y_pad), generator=g, device="cuda")[:, :out],
         "a": (torch.randn((n, rank, into), generator=g, device="cuda") / math.sqrt(into)).to(dtype),
         "b": torch.randn((n, out, rank), generator=g, device="cuda").to(dtype),
         "scales": _f32([0.5 + 0.25 * i for i in range(n)]), "ranks": _i32(ranks) if ranks else None}
    return p, _i32(adapters), _i32(start), t


def _lora_reference(p, lens, adapters):
    out, tol = p["y"].double().clone(), p["y"].abs().double() * 2.0 ** -24
    at = 0
    for m, a in zip(lens, adapters):
        if a >= 0 and m:
            r = min(max(int(p["ranks"][a]), 0), p["a"].shape[1]) if p.get("ranks") is not None else p["a"].shape[1]
            scale = p["scales"][a].double() if p.get("scales") is not None else 1.0
            x, down, up = p["x"][at:at + m].double(), p["a"][a, :r].double(), p["b"][a, :, :r].double()
            out[at:at + m] += scale * (x @ down.T @ up.T)
            tol[at:at + m] += 2.0 ** -15 * abs(scale) * (x.abs() @ down.abs().T @ up.abs().T)
        at += m
    return out, tol + out.abs() * 2.0 ** -23


def _check_lora(mmq, p, start, adapters, lens, ids, n, t, **kw):
    plan = mmq.mmq_lora_plan(adapters, start, t, n)
    got = mmq.mmq_lora(**p, plan=plan, **kw)
    want, tol = _lora_reference({**p, "y": kw["was"] if "was" in kw else p["y"]}, lens, ids)
    rows = sum(lens)
    worst = ((got[:rows].double() - want[:rows]).abs() - tol[:rows]).max().item() if rows else 0
    assert worst <= 0, worst
    return got


LORAS = [
    # tokens of each request, adapters, how many there are, id, od, rank
    ([1], [0], 1, 8, 1, 8), ([1], [2], 3, 3584, 4608, 16), ([1, 1, 1, 1], [1, -1, 0, 1], 2, 512, 768, 64),
    ([1] * 40, [(7 * i) % 11 - 1 for i in range(40)], 10, 1024, 1000, 32), ([3, 0, 5, 1, 9], [0, 1, 1, 2, 0], 3, 520, 333, 24),
    ([17, 64, 65, 1], [3, 2, 3, -1], 4, 264, 1026, 128), ([200, 130], [1, 1], 2, 1024, 512, 40), ([700, 1, 500], [0, 1, 2], 3, 512, 2080, 72),
    ([2100], [0], 1, 256, 260, 8), ([1, 2] * 300, [i % 50 - 1 for i in range(600)], 49, 128, 96, 16), ([0, 0], [0, 1], 2, 64, 64, 8),
    ([5] * 90, [i % 3 for i in range(90)], 3, 3584, 512, 56),
]


@pytest.mark.parametrize("case", LORAS, ids=lambda c: f"{len(c[0])}x{c[0][0]}-{c[3]}-{c[4]}-r{c[5]}")
@pytest.mark.parametrize("dtype,x_dtype", [(BF16, F32), (F16, F32), (F16, F16), (BF16, F16), (F16, BF16)])
def test_lora(mmq, case, dtype, x_dtype):
    lens, ids, n, into, out, rank = case
    ranks = [(5 * i + rank) % (rank + 2) for i in range(n)] if n > 1 else None
    p, adapters, start, t = _lora_problem(lens, ids, n, into, out, rank, dtype, x_dtype, tail=2, ranks=ranks)
    for a, r in enumerate(ranks or []):  # nothing past a rank is used
        p["a"][a, min(r, rank):] = math.nan
        p["b"][a, :, min(r, rank):] = math.inf
    y = p["y"].clone()
    buffer = torch.full_like(y, 5.0)
    got = _check_lora(mmq, p, start, adapters, lens, ids, n, t, out=buffer)
    assert got is buffer and (got[sum(lens):] == 5).all() and torch.equal(p["y"], y)
    none = torch.tensor([a < 0 for m, a in zip(lens, ids) for _ in range(m)] + [False] * 2, device="cuda")
    assert torch.equal(got[none], y[none])
    # in place, the same bits; rows of no request are left as they are
    plan = mmq.mmq_lora_plan(adapters, start, t, n)
    assert mmq.mmq_lora(**p, plan=plan, out=p["y"]) is p["y"]
    assert torch.equal(p["y"][: sum(lens)], got[: sum(lens)]) and torch.equal(p["y"][sum(lens):], y[sum(lens):])


@pytest.mark.parametrize("x_pad,y_pad,out", [(8, 4, 512), (24, 3, 512), (0, 1, 511), (8, 0, 510)])
def test_lora_strides(mmq, x_pad, y_pad, out):
    lens, ids = [3, 40, 1], [1, 0, -1]
    p, adapters, start, t = _lora_problem(lens, ids, 2, 320, out, 16, BF16, x_pad=x_pad, y_pad=y_pad)
    _check_lora(mmq, p, start, adapters, lens, ids, 2, t)
    # columns of one array: the middle of a fused projection's output, in place
    whole = torch.randn((t, 3 * out), device="cuda")
    was = whole.clone()
    want, tol = _lora_reference({**p, "y": whole[:, out:2 * out]}, lens, ids)
    got = mmq.mmq_lora(p["x"], whole[:, out:2 * out], p["a"], p["b"], mmq.mmq_lora_plan(adapters, start, t, 2), scales=p["scales"], out=whole[:, out:2 * out])
    assert ((got.double() - want).abs() <= tol).all()
    assert torch.equal(whole[:, :out], was[:, :out]) and torch.equal(whole[:, 2 * out:], was[:, 2 * out:])
    # x beside y in one array
    both = torch.randn((t, 320 + out + 8 - out % 8), device="cuda")
    got = mmq.mmq_lora(both[:, :320], both[:, 320:320 + out], p["a"], p["b"], mmq.mmq_lora_plan(adapters, start, t, 2), out=None)
    want, tol = _lora_reference({**p, "x": both[:, :320], "y": both[:, 320:320 + out], "scales": None}, lens, ids)
    assert ((got.double() - want).abs() <= tol).all()


def test_lora_without_adapters(mmq):
    p, _, start, t = _lora_problem([3, 4], [-1, -1], 0, 64, 96, 8, BF16)
    plan = mmq.mmq_lora_plan(_i32([-1, -1]), start, t, 0)
    p["scales"] = None
    assert torch.equal(mmq.mmq_lora(**p, plan=plan), p["y"])
    got = mmq.mmq_lora(p["x"][:0], p["y"][:0], p["a"], p["b"], mmq.mmq_lora_plan(_i32([]), _i32([0]), 0, 0))
    assert got.shape == (0, 96)


def test_lora_large_values(mmq):
    """Numbers beyond fp16's range, and far below its smallest."""
    for gain in (1e6, 1e-12):
        p, adapters, start, t = _lora_problem([30], [0], 1, 512, 256, 16, F16)
        p["x"] *= gain
        p["y"] *= gain
        _check_lora(mmq, p, start, adapters, [30], [0], 1, t)


@pytest.mark.parametrize("lens", [[1], [30, 25], [700, 600]], ids=str)
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_lora_long_sums_of_one_sign(mmq, lens, dtype):
    """Numbers of one sign, so that every rounding counts in full and a sum cut off always errs to one side: at most 37 sums
    of 32 columns a warp (18944 / 8 CTAs / 2 warps / 32), each of 6 steps of the tensor cores (8 more products with fp16
    weights) of 2^-23, added up with 2^-24 each, then 2 warps and 8 CTAs; the second product's 6 steps (10); the splits 2^-26."""
    p, _, start, t = _lora_problem(lens, [0] * len(lens), 1, 18944, 256, 32, dtype)
    p = {**p, "x": p["x"].abs() + 1, "a": p["a"].abs() + 2.0 ** -6, "b": p["b"].abs() + 1, "y": torch.zeros_like(p["y"])}
    got = mmq.mmq_lora(**p, plan=mmq.mmq_lora_plan(_i32([0] * len(lens)), start, t, 1))
    want, _ = _lora_reference(p, lens, [0] * len(lens))
    steps = (6 + 6 if dtype == BF16 else 10 + 10)
    assert ((got.double() - want).abs() / want).max() <= (2 * steps + 37 + 10 + 2) * 2.0 ** -24


@pytest.mark.parametrize("nreq", [1, 2, 31, 300, 1025, 8192])
def test_lora_plan(mmq, nreq):
    """Every token of a request once, tiles of one adapter, adapters ascending and none last."""
    r = random.Random(nreq)
    n = r.choice([1, 5, 700])
    lens = [r.choice([0, 1, 1, r.randint(0, 9)]) for _ in range(nreq)]
    ids = [r.randint(-1, n - 1) for _ in range(nreq)]
    start = [0]
    for m in lens:
        start.append(start[-1] + m)
    t = start[-1] + 5
    words = mmq.mmq_lora_plan(_i32(ids), _i32(start), t, n).words.tolist()
    tiles, with_adapter = words[:2]
    order, entries = words[4:4 + t], words[4 + t:]
    want = sorted((a if a >= 0 else n, b) for b, a in enumerate(ids))
    tokens = [start[b] + i for _, b in want for i in range(lens[b])]
    assert order[: len(tokens)] == tokens
    of = [(-1 if a == n else a) for a, b in want for _ in range(lens[b])]
    at = 0
    for k in range(tiles):
        a, first, count = entries[3 * k: 3 * k + 3]
        assert first == at and count >= 1 and set(of[at: at + count]) == {a} and (a >= 0) == (k < with_adapter)
        at += count
    assert at == len(tokens)


def test_lora_faults(mmq):
    p, _, start, t = _lora_problem([2, 3], [0, 1], 2, 64, 96, 8, BF16)
    plan = mmq.mmq_lora_plan(_i32([2, 1]), start, t, 2)
    assert _recorded(mmq)
    got = mmq.mmq_lora(**p, plan=plan)
    assert torch.equal(got[:2], p["y"][:2])
    want, tol = _lora_reference(p, [2, 3], [-1, 1])
    assert ((got.double() - want).abs() <= tol).all()
    mmq.mmq_lora_plan(_i32([-2, 1]), start, t, 2)
    assert _recorded(mmq)
    plan = mmq.mmq_lora_plan(_i32([0, 1]), _i32([0, 3, 2]), t, 2)
    assert _recorded(mmq)
    buffer = torch.full_like(p["y"], 3.0)
    assert (mmq.mmq_lora(**p, plan=plan, out=buffer) == 3).all()
    # row starts past the token rows: the rows that are there
    plan = mmq.mmq_lora_plan(_i32([0, 1]), _i32([0, 2, 9]), t, 2)
    got = mmq.mmq_lora(**p, plan=plan)
    want, tol = _lora_reference(p, [2, 3], [0, 1])
    assert ((got.double() - want).abs() <= tol).all()


# ---------------------------------------------------------------- refusals
def test_refused_pages(mmq):
    table, held, parents, lens = _table([[1, 2], [3]], 4), _i32([2, 1]), _i32([0, 1]), _i32([20, 3])
    kc, vc = (torch.zeros((8, 16, 2, 64), dtype=F16, device="cuda") for _ in range(2))
    f, m = mmq.mmq_page_fork(table, held, parents, lens, 16, 8), mmq.mmq_page_compact(table, held, 8)
    fork = lambda **kw: mmq.mmq_page_fork(**{**dict(block_table=table, n_blocks=held, parents=parents, lens=lens, page_size=16, n_pages=8), **kw})  # noqa: E731
    compact = lambda **kw: mmq.mmq_page_compact(**{**dict(block_table=table, n_blocks=held, n_pages=8), **kw})  # noqa: E731
    copy = lambda **kw: mmq.mmq_page_copy(**{**dict(k_cache=kc, v_cache=vc, pairs=f.pairs, tokens=f.tokens), **kw})  # noqa: E731
    for call, bad in [(fork, dict(block_table=table.long())), (fork, dict(block_table=table[0])), (fork, dict(block_table=table.t())),
                      (fork, dict(n_blocks=held[:1])), (fork, dict(n_blocks=held.float())), (fork, dict(parents=parents[:1])),
                      (fork, dict(lens=lens.long())), (fork, dict(lens=lens[:, None])), (fork, dict(n_pages=-1)), (fork, dict(n_pages=2 ** 31)),
                      (fork, dict(out=f._replace(counts=f.counts[:1]))), (fork, dict(out=f._replace(block_table=f.block_table[:, :3]))),
                      (fork, dict(out=f._replace(free_pages=f.free_pages[:7]))), (fork, dict(out=f._replace(pairs=f.pairs.float()))),
                      (compact, dict(block_table=table[:1])), (compact, dict(n_pages=-1)), (compact, dict(out=m._replace(pairs=m.pairs[:2]))),
                      (copy, dict(pairs=f.pairs.long())), (copy, dict(pairs=f.tokens)), (copy, dict(tokens=f.tokens[:1])),
                      (copy, dict(v_cache=vc[:4])), (copy, dict(v_cache=vc.bfloat16())), (copy, dict(k_cache=kc.float(), v_cache=vc.float()))]:
        with pytest.raises(ValueError):
            call(**bad)
    for call, bad in [(fork, dict(parents=parents.cpu())), (fork, dict(out=(f.pairs,))), (fork, dict(lens=None)), (compact, dict(out=m.counts)),
                      (copy, dict(pairs=None)), (copy, dict(tokens=[1, 2]))]:
        with pytest.raises(TypeError):
            call(**bad)
    for call, bad, code in [(fork, dict(page_size=0), ARG), (fork, dict(out=f._replace(block_table=table)), ARG),
                            (fork, dict(out=f._replace(n_blocks=held)), ARG), (fork, dict(n_pages=2 ** 20 + 1), UNSUPPORTED),
                            (compact, dict(out=m._replace(block_table=table)), ARG)]:
        with pytest.raises(mmq.MMQError) as e:
            call(**bad)
        assert e.value.code == code, bad.keys()
    _same_fork(f, _fork_reference([[1, 2], [3]], [0, 1], [20, 3], 16, 8, 4))


def test_refused_rules(mmq):
    p = _rules_problem(2, 1, 320, F32, seed=1)
    one, ids = torch.ones(2, device="cuda"), _i32([0, 1])
    for bad in (dict(logits=p["logits"].double()), dict(logits=p["logits"][0]), dict(logits=p["logits"].transpose(1, 2)), dict(temperature=one[:1]),
                dict(temperature=one.half()), dict(tokens=p["tokens"][:1]), dict(tokens=p["tokens"].long()), dict(tokens=None), dict(token_lens=ids[:1]),
                dict(prompt_lens=one), dict(draft_tokens=p["draft_tokens"][:, :0]), dict(n_draft=one), dict(repetition=one[:1]), dict(frequency=ids),
                dict(presence=one[:1]), dict(bias=(ids, *p["bias"][1:])), dict(bias=(p["bias"][0], p["bias"][1], p["bias"][2][:-1])),
                dict(mask=p["mask"][:, :-1]), dict(mask=p["mask"].long()), dict(mask=None), dict(mask_rows=ids), dict(probs=None), dict(probs=False),
                dict(probs=p["logits"][:, :1].clone()), dict(probs=p["logits"].double()), dict(adjusted=p["logits"][..., :-1])):
        with pytest.raises(ValueError):
            mmq.mmq_token_probs(**{**p, **bad})
    for bad in (dict(temperature=one.cpu()), dict(bias=p["bias"][0]), dict(bias=p["bias"][:2]), dict(tokens=[1]), dict(probs=3)):
        with pytest.raises(TypeError):
            mmq.mmq_token_probs(**{**p, **bad})
    for bad in (dict(probs=p["logits"]), dict(adjusted=torch.empty(320, device="cuda").expand(2, 2, 320))):
        with pytest.raises(mmq.MMQError) as e:
            mmq.mmq_token_probs(**{**p, **bad})
        assert e.value.code == ARG


def test_refused_adapters(mmq):
    p, adapters, start, t = _lora_problem([2, 3], [0, 1], 2, 64, 96, 8, BF16)
    plan = mmq.mmq_lora_plan(adapters, start, t, 2)
    for bad in ((adapters[:1], start, t, 2), (adapters.long(), start, t, 2), (adapters, start[:2], t, 2), (adapters, start.float(), t, 2),
                (adapters, start, t, 2, plan.words[:-1])):
        with pytest.raises(ValueError):
            mmq.mmq_lora_plan(*bad)
    for bad, code in (((adapters, start, -1, 2), ARG), ((adapters, start, t, -1), ARG),
                      ((adapters, start, 2 ** 30, 2), UNSUPPORTED), ((adapters, start, t, 2 ** 19), UNSUPPORTED)):
        with pytest.raises(mmq.MMQError) as e:
            mmq.mmq_lora_plan(*bad)
        assert e.value.code == code, bad
    lora = lambda **kw: mmq.mmq_lora(**{**p, "plan": plan, **kw})  # noqa: E731
    for bad in (dict(x=p["x"][:-1]), dict(x=p["x"].double()), dict(x=p["x"].t()), dict(y=p["y"].half()), dict(y=p["y"][:, :-1]), dict(a=p["a"].half()),
                dict(a=p["a"].float(), b=p["b"].float()), dict(a=p["a"][:1]), dict(b=p["b"][:, :, :4]), dict(b=p["b"].transpose(1, 2)),
                dict(scales=p["scales"].half()), dict(ranks=_i32([1])), dict(out=p["y"][:-1]), dict(out=p["y"].half()),
                dict(plan=plan._replace(words=plan.words[:-1])), dict(plan=plan._replace(tokens=4)), dict(plan=plan._replace(requests=1)),
                dict(plan=plan._replace(adapters=1))):
        with pytest.raises(ValueError):
            lora(**bad)
    wide, flat = torch.zeros((t, 70), device="cuda"), torch.zeros(t * 96 + 4, device="cuda")
    for bad, code in ((dict(x=wide[:, 1:65]), ALIGN), (dict(x=wide[:, :64]), ALIGN),
                      (dict(a=p["a"][:, :4].contiguous(), b=p["b"][..., :4].contiguous()), ARG),
                      (dict(out=p["y"].new_empty(96).expand(t, 96)), ARG),
                      (dict(y=flat[4:].view(t, 96), out=flat[:-4].view(t, 96)), ARG)):  # four further on in one buffer
        with pytest.raises(mmq.MMQError) as e:
            lora(**bad)
        assert e.value.code == code, bad.keys()
    with pytest.raises(TypeError):
        lora(x=p["x"].cpu())


# ---------------------------------------------------------------- together, streams, graphs
def test_repeated_bits(mmq):
    p = _rules_problem(6, 3, 20011, F32, seed=4, hist=3000, bias=30)
    q, adapters, start, t = _lora_problem([40, 1, 90], [0, 1, 0], 2, 1024, 768, 32, BF16)
    first = None
    for _ in range(20):
        got = [*mmq.mmq_token_probs(**p, adjusted=True), mmq.mmq_lora(**q, plan=mmq.mmq_lora_plan(adapters, start, t, 2))]
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(got, first))


def test_other_stream_and_current_device(mmq):
    s = torch.cuda.Stream()
    p = _rules_problem(2, 1, 5000, F32, seed=8)
    want = mmq.mmq_token_probs(**p)[0]
    torch.cuda.synchronize()
    got = mmq.mmq_token_probs(**p, stream=s)[0]
    s.synchronize()
    assert torch.equal(got, want)
    with torch.cuda.stream(s):
        got = mmq.mmq_token_probs(**p)[0]
    s.synchronize()
    assert torch.equal(got, want)


def test_two_threads_on_two_streams(mmq):
    """Calls with scratch at the same time: each its own."""
    import threading
    jobs = []
    for seed in range(2):
        probs = _rules_problem(5, 3, 30011, (F32, BF16)[seed], seed=seed, hist=900, bias=20)
        lora, adapters, start, t = _lora_problem([200, 3, 90 + seed], [0, 1, 0], 2, 768, 1024, (32, 64)[seed], BF16, seed=seed)
        plan = mmq.mmq_lora_plan(adapters, start, t, 2)
        jobs.append((probs, lora, plan, [*mmq.mmq_token_probs(**probs, adjusted=True), mmq.mmq_lora(**lora, plan=plan)]))
    torch.cuda.synchronize()
    wrong = []

    def run(probs, lora, plan, want):
        s = torch.cuda.Stream()
        for _ in range(40):
            with torch.cuda.stream(s):
                got = [*mmq.mmq_token_probs(**probs, adjusted=True), mmq.mmq_lora(**lora, plan=plan)]
            s.synchronize()
            wrong.extend(k for k, (a, b) in enumerate(zip(got, want)) if not torch.equal(a, b))

    threads = [threading.Thread(target=run, args=job) for job in jobs]
    for x in threads:
        x.start()
    for x in threads:
        x.join()
    assert not wrong


def test_a_row_for_all(mmq):
    """Inputs that are one row seen many times (stride 0): logits, tokens, x and y."""
    v, b = 3001, 4
    g = torch.Generator(device="cuda").manual_seed(2)
    logits = torch.randn((1, 1, v), generator=g, device="cuda")
    tokens = torch.randint(0, v, (1, 50), generator=g, device="cuda", dtype=torch.int32)
    rho = _f32([1.3] * b)
    got, adjusted = mmq.mmq_token_probs(logits.expand(b, 1, v), tokens=tokens.expand(b, 50), repetition=rho, adjusted=True)
    want = mmq.mmq_token_probs(logits.repeat(b, 1, 1), tokens=tokens.repeat(b, 1), repetition=rho, adjusted=True)
    # 3001 elements: the repeated rows begin anywhere in 16 bytes of memory, so that their sums go by other groups and their
    # exponentials against other maxima; each is within 2^-20 and 2^-23 of an exponent below 16: 2 (1 + 2) 2^-20 in all
    assert ((got - want[0]).abs() <= 6 * 2.0 ** -20 * want[0]).all() and torch.equal(adjusted, want[1])
    for n in (5, 300):
        p, adapters, start, t = _lora_problem([n - 1, 1], [0, 1], 2, 256, 512, 16, BF16)
        plan = mmq.mmq_lora_plan(adapters, start, t, 2)
        x, y = p["x"][:1], p["y"][:1]
        got = mmq.mmq_lora(**{**p, "x": x.expand(t, 256), "y": y.expand(t, 512)}, plan=plan)
        assert torch.equal(got, mmq.mmq_lora(**{**p, "x": x.repeat(t, 1), "y": y.repeat(t, 1)}, plan=plan))


@pytest.mark.parametrize("old,new,width,pages", [(3, 5, 40, 2 ** 20), (8192, 8192, 3, 30000), (40, 70, 300, 2 ** 20)])
def test_fork_and_compact_at_the_limits(mmq, old, new, width, pages):
    """The largest caches and the most rows: what is held, what is free and what moves, by sets."""
    r, page = random.Random(old), 16
    g = torch.Generator(device="cuda").manual_seed(old)
    table = torch.randperm(pages, generator=g, device="cuda")[: old * width].view(old, width).int()
    n = [r.randint(0, width * page) for _ in range(old)]
    held = [-(-x // page) for x in n]
    parents = [r.randrange(old) for _ in range(new)]
    lens = [max(0, n[p] - r.choice([0, 0, 1, 40])) for p in parents]
    rows = [row[:h] for row, h in zip(table.tolist(), held)]
    f = mmq.mmq_page_fork(table, _i32(held), _i32(parents), _i32(lens), page, pages)
    _same_fork(f, _fork_reference(rows, parents, lens, page, pages, width))
    m = mmq.mmq_page_compact(f.block_table, f.n_blocks, pages)
    used = sorted({x for row, k in zip(f.block_table.tolist(), f.n_blocks.tolist()) for x in row[:k]})
    h = len(used)
    moved = [x for x in used if x >= h]
    to = sorted(set(range(h)) - set(used))
    assert m.counts.tolist() == [h, len(moved)] and m.pairs[: len(moved)].tolist() == [list(x) for x in zip(moved, to)]
    assert (m.pairs[len(moved):] == -1).all()
    place = dict(zip(moved, to))
    want = [[place.get(x, x) for x in row[:k]] + [-1] * (width - k) for row, k in zip(f.block_table.tolist(), f.n_blocks.tolist())]
    assert m.block_table.tolist() == want


def test_graphs_on_other_inputs(mmq):
    """Two captured graphs, replayed in turn on other tables, lengths, tokens and adapters."""
    page, pages, width = 8, 300, 30
    r = random.Random(0)
    probs = _rules_problem(3, 2, 3001, F32, seed=1)
    lora, adapters, start, t = _lora_problem([3, 9, 2], [0, 1, -1], 2, 256, 512, 16, F16)
    table, held, parents, lens = _table([[0] * width] * 6, width), _i32([0] * 6), _i32([0] * 6), _i32([0] * 6)

    def step():
        f = mmq.mmq_page_fork(table, held, parents, lens, page, pages)
        m = mmq.mmq_page_compact(f.block_table, f.n_blocks, pages)
        return f, m, mmq.mmq_token_probs(**probs)[0], mmq.mmq_lora(**lora, plan=mmq.mmq_lora_plan(adapters, start, t, 2))

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = step()
        graphs.append((g, got))
    for seed in range(6):
        rows, n = _rows(random.Random(seed), 6, page, 150, pages)
        table.copy_(_table(rows, width))
        held.copy_(_i32([len(x) for x in rows]))
        p = [r.randrange(6) for _ in range(6)]
        parents.copy_(_i32(p))
        lens.copy_(_i32([n[x] for x in p]))
        fresh = _rules_problem(3, 2, 3001, F32, seed=seed)
        for name, x in fresh.items():
            if name != "bias":
                probs[name].copy_(x)
        cut = r.randint(0, 12)
        start.copy_(_i32([0, cut, cut + 1, 14]))
        adapters.copy_(_i32([r.randint(-1, 1) for _ in range(3)]))
        lora["x"].normal_()
        g, (f, m, q, y) = graphs[seed % 2]
        g.replay()
        want = step()
        for a, b in zip([*f, *m, q, y], [*want[0], *want[1], *want[2:]]):
            assert torch.equal(a, b)
        _same_fork(f, _fork_reference(rows, p, [n[x] for x in p], page, pages, width))


def test_beams_over_a_paged_cache(mmq):
    """Page tables, K/V rows, forks, copies, compactions and attention together: every row's attention is that over its own
    tokens, held beside in a list, whatever pages they went through."""
    page, pages, heads, d, width = 4, 120, 2, 64, 12
    r = random.Random(3)
    g = torch.Generator(device="cuda").manual_seed(3)
    kc, vc = (torch.full((pages, page, heads, d), math.nan, dtype=F16, device="cuda") for _ in range(2))
    b = 5
    table = torch.full((b, width), -1, dtype=torch.int32, device="cuda")
    held, cached, free = _i32([0] * b), [0] * b, torch.arange(pages, dtype=torch.int32, device="cuda")
    kept = [(torch.empty((0, heads, d), device="cuda", dtype=F16),) * 2 for _ in range(b)]
    for step in range(14):
        new = [r.choice([0, 1, 1, 3]) for _ in range(b)]
        n = sum(new)
        t = mmq.mmq_page_tables(_i32(cached), _i32(new), held, table, free, page, n)
        taken, missing = t.taken.tolist()
        assert not missing
        free, held = free[taken:], t.n_blocks
        k, v, q = (torch.randn((n, heads, d), generator=g, device="cuda").half() for _ in range(3))
        mmq.mmq_kv_write(k, v, kc, vc, t.slots)
        y, _ = mmq.mmq_paged_attention(q, kc, vc, table, t.seq_lens, t.q_start, out_dtype=F32)
        at = 0
        for i, m in enumerate(new):
            keys, values = (torch.cat([old, x[at:at + m]]) for old, x in zip(kept[i], (k, v)))
            kept[i] = keys, values
            cached[i] += m
            for j in range(m):
                seen = cached[i] - m + j + 1
                s = torch.einsum("hd,jhd->hj", q[at + j].double(), keys[:seen].double()) / d ** 0.5
                want = torch.einsum("hj,jhd->hd", torch.softmax(s, -1), values[:seen].double())
                assert (y[at + j].double() - want).abs().max() < 4e-3  # fp16 weights: 2^-11 of values below 4
            at += m
        parents = [r.choice([i, i, r.randrange(b)]) for i in range(b)]
        if step % 5 == 4:
            parents[r.randrange(b)] = -1
        lens = [0 if p < 0 else max(0, cached[p] - r.choice([0, 0, 1, 2])) for p in parents]
        f = mmq.mmq_page_fork(table, held, _i32(parents), _i32(lens), page, pages)
        mmq.mmq_page_copy(kc, vc, f.pairs, f.tokens)
        table, held, cached = f.block_table, f.n_blocks, lens
        kept = [tuple(x[:n] for x in kept[p]) if p >= 0 else tuple(x[:0] for x in kept[0]) for p, n in zip(parents, lens)]
        listed, missing = f.counts.tolist()
        assert not missing
        free = f.free_pages[:listed]
        used = {x for row, n in zip(table.tolist(), held.tolist()) for x in row[:n]}
        assert len(used) + listed == pages
        for i in free.tolist():  # what is free holds nothing
            kc[i], vc[i] = math.nan, math.nan
        if step % 4 == 3:
            m = mmq.mmq_page_compact(table, held, pages)
            mmq.mmq_page_copy(kc, vc, m.pairs)
            table, first = m.block_table, m.counts.tolist()[0]
            assert first == len(used)
            kc[first:], vc[first:] = math.nan, math.nan
            free = torch.arange(first, pages, dtype=torch.int32, device="cuda")
