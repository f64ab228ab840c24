"""The operators of a serving step next to the projections, as cases to measure: page tables and slot maps from
request lengths, K and V written into the paged cache, attention of a chunk of new tokens over that cache, and
the verification of drafted tokens.

`run` computes each one in elementary torch operations in 32 bits (`own` false) or by the library's entry points
(`own` true).  Lengths follow from a case alone (`spread`), values from the seed."""
import itertools
import math
import random

import torch

own = False

_DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def listed():
    """28 query heads of 128 are the 3584 rows of the repository's q-proj; 512 and 2630 are its token counts."""
    return [
        # one user, one token: the call's latency
        _attention("decode_b1_ctx900", "bf16", 1, 1, 1, 900, 900, 28, 4, 128, 16, "nhd"),
        # a decode batch of requests of very different ages
        _attention("decode_b64_ragged", "f16", 64, 1, 1, 97, 12001, 28, 4, 128, 64, "hnd"),
        # a decode batch that also carries a few drafted tokens for each request, to be verified
        _attention("draft_b24_q5", "bf16", 24, 5, 5, 700, 5000, 28, 4, 128, 16, "nhd"),
        # one prompt's chunk of the ordinary size on what came before it
        _attention("chunk512_ctx8k", "bf16", 1, 512, 512, 8000, 8000, 28, 4, 128, 16, "nhd"),
        # whole prompts, heads of 64, a sliding window, odd lengths
        _attention("prompts_d64_window", "f16", 5, 301, 2630, 0, 0, 24, 8, 64, 32, "hnd", window=1000),
        # the largest: a long chunk of a long document
        _attention("chunk4096_ctx28k", "bf16", 1, 4096, 4096, 28001, 28001, 28, 4, 128, 64, "nhd"),
        # a decode batch's new K and V, out of the fused projection's fp32 rows
        _write("write_64", 64, 28, 4, 128, 16, 600, "f32", "f16"),
        # the rows of several prompts' chunks, padded as a captured step pads them
        _write("write_16k", 16384, 28, 4, 128, 64, 1200, "f32", "bf16"),
        # tables of a small decode batch
        _tables("tables_b8", 8, 1, 1, 60, 3000, 16, 16),
        # tables of a large batch that mixes decodes and chunks
        _tables("tables_b700", 700, 1, 500, 0, 9000, 16, 65536),
        # four drafted tokens of a few requests
        _verify("verify_b6_k4", 6, 4, 32000, "f32"),
        # a full batch, a vocabulary with an odd size
        _verify("verify_b160_k5", 160, 5, 100277, "f32"),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["attention"] * 5 + ["write", "tables", "verify"])
    if op == "attention":
        hkv = rng.choice([1, 2, 4, 8])
        hq = hkv * rng.choice([1, 2, 3, 4, 7, 8])
        d = rng.choice([64, 96, 128, 128])
        q = log(1, 4096) if rng.random() < 0.6 else rng.choice([1, 1, 5])
        kv = log(1, 30000)
        room = 1.5e9 / (hq * (q + kv))  # keeps the plain form's scores within the largest case's
        b = max(1, min(log(1, 96), int(room / q), int(2e6 / (hkv * (q + kv))) or 1))
        kv = min(kv, max(1, int(3.6e9 / (b * hq * q)) - q)) if q > 1 else kv
        kv = max(kv, 1)
        return _attention(None, rng.choice(["bf16", "f16"]), b, rng.choice([1, q]), q, rng.choice([1, kv]), kv, hq, hkv, d,
                          rng.choice([8, 16, 32, 64, 128, 256]), rng.choice(["nhd", "hnd"]),
                          window=rng.choice([0, 0, 0, log(100, 4000)]))
    if op == "write":
        page = rng.choice([8, 16, 32, 64])
        t = log(1, 16384)
        hkv = rng.choice([1, 2, 4, 8])
        return _write(None, t, hkv * rng.choice([1, 4, 7]), hkv, rng.choice([64, 96, 128]), page, t // page + log(50, 1000),
                      rng.choice(["f32", "f16", "bf16"]), rng.choice(["f16", "bf16"]))
    if op == "tables":
        b = log(1, 1000)
        hi = max(1, min(log(1, 1000), 65536 // b))
        return _tables(None, b, rng.choice([0, 1]), hi, rng.choice([0, 50]), log(50, 12000), rng.choice([1, 8, 16, 64]), b * hi)
    v = log(1000, 131072)
    return _verify(None, log(1, 160), rng.randint(1, 8), v, rng.choice(["f32", "f32", "bf16"]))


def _named(name, case):
    return case if name is None else {"name": name, **case}


def _attention(name, dtype, b, q_lo, q_hi, kv_lo, kv_hi, hq, hkv, d, page, layout, window=0):
    return _named(name, {"op": "attention", "dtype": dtype, "b": b, "q_lo": q_lo, "q_hi": q_hi, "kv_lo": kv_lo, "kv_hi": kv_hi,
                         "hq": hq, "hkv": hkv, "d": d, "page": page, "layout": layout, "window": window})


def _write(name, tokens, hq, hkv, d, page, pages, src, dtype):
    return _named(name, {"op": "write", "tokens": tokens, "hq": hq, "hkv": hkv, "d": d, "page": page, "pages": pages, "src": src, "dtype": dtype})


def _tables(name, b, new_lo, new_hi, old_lo, old_hi, page, room):
    return _named(name, {"op": "tables", "b": b, "new_lo": new_lo, "new_hi": new_hi, "old_lo": old_lo, "old_hi": old_hi, "page": page, "room": room})


def _verify(name, b, k, v, dtype):
    return _named(name, {"op": "verify", "b": b, "k": k, "v": v, "dtype": dtype})


def spread(lo, hi, n, salt=0):
    """n lengths from lo to hi, even in their logarithm, in a fixed mixed order."""
    if n == 1:
        return [hi]
    got = [int(round((lo + 1) * ((hi + 1) / (lo + 1)) ** (i / (n - 1)))) - 1 for i in range(n)]
    random.Random(1000 * n + salt).shuffle(got)
    return got


def _lens(case):
    return spread(case["q_lo"], case["q_hi"], case["b"], 1), spread(case["kv_lo"], case["kv_hi"], case["b"], 2)


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return {"attention": _prepare_attention, "write": _prepare_write, "tables": _prepare_tables,
            "verify": _prepare_verify}[case["op"]](case, g, seed) | {"op": case["op"]}


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _randn(g, shape, dtype, scale=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype).mul_(scale)


def _cumulated(x):
    return [0, *itertools.accumulate(x)]


def _prepare_attention(case, g, seed):
    """Pages lie in a random order in the cache; what no request holds (other pages, the ends of last pages) is NaN, as
    memory that nothing was written to may be.  The scores' deviation is 1.5, so that a few keys carry most of a row."""
    dt, page, hkv, d, b = _DT[case["dtype"]], case["page"], case["hkv"], case["d"], case["b"]
    q_lens, old = _lens(case)
    lens = [o + q for o, q in zip(old, q_lens)]
    blocks = [-(-n // page) for n in lens]
    pages = sum(blocks) + 3
    shape = (pages, page, hkv, d) if case["layout"] == "nhd" else (pages, hkv, page, d)
    kc, vc = _randn(g, shape, dt), _randn(g, shape, dt)
    if case["layout"] == "hnd":
        kc, vc = kc.permute(0, 2, 1, 3), vc.permute(0, 2, 1, 3)
    width = max(blocks) + 2
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    n_blocks, seq_lens = _i32(blocks), _i32(lens)
    j = torch.arange(width, device="cuda", dtype=torch.int32)
    first = torch.cumsum(n_blocks, 0, dtype=torch.int32) - n_blocks
    table = torch.where(j < n_blocks[:, None], order[(first[:, None] + j).clamp(max=pages - 1).long()], -1)
    held = torch.zeros((pages, page), dtype=torch.bool, device="cuda")
    filled = j[:, None] * page + torch.arange(page, device="cuda") < seq_lens[:, None, None]
    rows = table >= 0
    held[table[rows].long()] = filled[rows]
    for c in (kc, vc):
        c[~held] = math.nan
    tokens = sum(q_lens)
    return {"q": _randn(g, (tokens, case["hq"], d), dt, 1.5), "kc": kc, "vc": vc, "table": table.contiguous(), "seq_lens": seq_lens,
            "q_start": _i32(_cumulated(q_lens)), "max_q": max(q_lens), "max_kv": max(lens), "window": case["window"],
            "out": torch.empty((tokens, case["hq"], d), dtype=dt, device="cuda"),
            "lse": torch.empty((tokens, case["hq"]), dtype=torch.float32, device="cuda")}


def _prepare_write(case, g, seed):
    """K and V are columns of the fused projection's output; one token in nine is padding (slot -1)."""
    hq, hkv, d, t = case["hq"], case["hkv"], case["d"], case["tokens"]
    qkv = _randn(g, (t, hq + 2 * hkv, d), _DT[case["src"]])
    shape = (case["pages"], case["page"], hkv, d)
    slots = torch.randperm(case["pages"] * case["page"], generator=g, device="cuda")[:t].contiguous()
    slots[4::9] = -1
    return {"k": qkv[:, hq:hq + hkv], "v": qkv[:, hq + hkv:], "slots": slots,
            "kc": _randn(g, shape, _DT[case["dtype"]]), "vc": _randn(g, shape, _DT[case["dtype"]])}


def _tables_lens(case):
    return spread(case["new_lo"], case["new_hi"], case["b"], 3), spread(case["old_lo"], case["old_hi"], case["b"], 4)


def _prepare_tables(case, g, seed):
    """Every fifth request still holds a page more than its tokens need, left by drafted tokens that were refused."""
    new, old = _tables_lens(case)
    page, b = case["page"], case["b"]
    held = [-(-o // page) + (i % 5 == 3) for i, o in enumerate(old)]
    width = max(max(-(-(o + n) // page), h) for o, n, h in zip(old, new, held)) + 1
    need = sum(max(0, -(-(o + n) // page) - h) for o, n, h in zip(old, new, held))
    order = torch.randperm(sum(held) + need + 64, generator=g, device="cuda").to(torch.int32)
    n_blocks = _i32(held)
    first = torch.cumsum(n_blocks, 0, dtype=torch.int32) - n_blocks
    j = torch.arange(width, device="cuda", dtype=torch.int32)
    table = torch.where(j < n_blocks[:, None], order[(first[:, None] + j).clamp(max=order.numel() - 1).long()], -1)
    empty = lambda n, dt=torch.int32: torch.empty(n, dtype=dt, device="cuda")  # noqa: E731
    return {"cached": _i32(old), "new": _i32(new), "n_blocks": n_blocks, "table": table.contiguous(), "free": order[sum(held):].contiguous(),
            "page": page, "room": case["room"],
            "out": (empty(b + 1), empty(b), empty(b), empty(case["room"], torch.int64), empty(case["room"]), empty(2))}


def _prepare_verify(case, g, seed):
    """The draft's distribution is the target's, a little off; requests bring 0 to k drafted tokens; the last one brings tokens
    that the target gives nothing."""
    b, k, v, dt = case["b"], case["k"], case["v"], _DT[case["dtype"]]
    target = torch.empty((b, k + 1, v), dtype=dt, device="cuda")
    draft = torch.empty((b, k, v), dtype=dt, device="cuda")
    tokens = torch.empty((b, k), dtype=torch.int32, device="cuda")
    for i in range(k + 1):
        z = _randn(g, (b, v), torch.float32, 3.0)
        target[:, i] = torch.softmax(z, -1).to(dt)
        if i < k:
            q = torch.softmax(z + _randn(g, (b, v), torch.float32, 0.7), -1)
            draft[:, i] = q.to(dt)
            tokens[:, i] = torch.multinomial(q, 1, generator=g)[:, 0].to(torch.int32)
    n = torch.arange(b, device="cuda", dtype=torch.int32) % (k + 1)
    n_draft = torch.where(torch.arange(b, device="cuda") % 2 == 0, torch.full_like(n, k), n).contiguous()
    target[b - 1, 0, tokens[b - 1, 0].long()] = 0
    noise = torch.empty((b, v), dtype=torch.float32, device="cuda").exponential_(generator=g)
    return {"target": target, "draft": draft, "tokens": tokens, "n_draft": n_draft,
            "u": torch.rand((b, k), generator=g, device="cuda"), "noise": noise}


# ---------------------------------------------------------------- one pass
def run(s):
    if own:
        return _own(s)
    return {"attention": _plain_attention, "write": _plain_write, "tables": _plain_tables, "verify": _plain_verify}[s["op"]](s)


def _own(s):
    import quantized_int8_gemm_gb300 as mmq
    if s["op"] == "attention":
        out, lse = mmq.mmq_paged_attention(s["q"], s["kc"], s["vc"], s["table"], s["seq_lens"], s["q_start"],
                                           window=s["window"], out=s["out"], lse=s["lse"])
        return {"out": out, "lse": lse}
    if s["op"] == "write":
        mmq.mmq_kv_write(s["k"], s["v"], s["kc"], s["vc"], s["slots"])
        return {"k_cache": s["kc"], "v_cache": s["vc"]}
    if s["op"] == "tables":
        t = mmq.mmq_page_tables(s["cached"], s["new"], s["n_blocks"], s["table"], s["free"], s["page"], s["room"], out=s["out"])
        return {"q_start": t.q_start, "seq_lens": t.seq_lens, "n_blocks": t.n_blocks, "slots": t.slots, "positions": t.positions,
                "taken": t.taken, "table": s["table"]}
    tokens, accepted = mmq.mmq_verify_draft(s["target"], s["draft"], s["tokens"], s["n_draft"], s["u"], s["noise"])
    return {"tokens": tokens, "accepted": accepted}


def _plain_attention(s):
    q, kc, vc, seq_lens, q_start = s["q"], s["kc"], s["vc"], s["seq_lens"], s["q_start"]
    (tokens, hq, d), page, hkv, b = q.shape, kc.shape[1], kc.shape[2], seq_lens.numel()
    dev, rep, scale = q.device, hq // hkv, 1.0 / math.sqrt(d)
    pages = s["table"][:, :-(-s["max_kv"] // page)].clamp(min=0).long()
    length = pages.shape[1] * page
    at = torch.arange(length, device=dev)
    held = (at < seq_lens[:, None])[:, :, None, None]
    k = torch.where(held, kc[pages].reshape(b, length, hkv, d).float(), 0.0).permute(0, 2, 3, 1)
    v = torch.where(held, vc[pages].reshape(b, length, hkv, d).float(), 0.0).permute(0, 2, 1, 3)
    # the ragged chunks, padded to the longest
    i = torch.arange(s["max_q"], device=dev)
    row = (q_start[:-1, None] + i).clamp(max=tokens - 1).long()
    qp = q[row].float().view(b, s["max_q"], hkv, rep, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, rep * s["max_q"], d)
    score = torch.matmul(qp, k).mul_(scale).view(b, hkv, rep, s["max_q"], length)
    q_pos = (seq_lens - (q_start[1:] - q_start[:-1]))[:, None] + i
    seen = (at <= q_pos[:, :, None]) & (at < seq_lens[:, None, None])
    if s["window"]:
        seen &= at > q_pos[:, :, None] - s["window"]
    score.masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score.sub_(torch.where(top == -math.inf, 0.0, top)))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(b, hkv, rep * s["max_q"], length), v).view(b, hkv, rep, s["max_q"], d)
    o = torch.where(total > 0, o / total, 0.0)
    lse = (top + torch.log(total))[..., 0]
    # back to the ragged rows
    t = torch.arange(tokens, device=dev)
    of = torch.searchsorted(q_start[1:].contiguous(), t.int(), right=True)
    nth = t - q_start.long()[of]
    return {"out": o[of, :, :, nth].reshape(tokens, hq, d).to(q.dtype), "lse": lse[of, :, :, nth].reshape(tokens, hq)}


def _plain_write(s):
    hkv, d = s["k"].shape[1:]
    kept = s["slots"] >= 0
    at = s["slots"][kept]
    s["kc"].view(-1, hkv, d)[at] = s["k"][kept].float().to(s["kc"].dtype)
    s["vc"].view(-1, hkv, d)[at] = s["v"][kept].float().to(s["vc"].dtype)
    return {"k_cache": s["kc"], "v_cache": s["vc"]}


def _plain_tables(s):
    cached, new, held, table, free, page, room = s["cached"], s["new"], s["n_blocks"], s["table"], s["free"], s["page"], s["room"]
    seq_lens = cached + new
    q_start = torch.cat([torch.zeros_like(new[:1]), torch.cumsum(new, 0, dtype=torch.int32)])
    n_blocks = torch.maximum(held, (seq_lens + page - 1) // page)
    more = n_blocks - held
    first = torch.cumsum(more, 0, dtype=torch.int32) - more
    j = torch.arange(table.shape[1], device=table.device, dtype=torch.int32)
    nth = first[:, None] + j - held[:, None]
    fresh = (j >= held[:, None]) & (j < n_blocks[:, None])
    table = torch.where(fresh, free[nth.clamp(0, free.numel() - 1).long()], table)
    t = torch.arange(room, device=table.device, dtype=torch.int32)
    of = torch.searchsorted(q_start[1:].contiguous(), t, right=True).clamp(max=new.numel() - 1)
    real = t < q_start[-1]
    position = torch.where(real, cached[of] + t - q_start[of], -1)
    inside = position.clamp(min=0)
    slots = torch.where(real, table[of, (inside // page).long()].long() * page + inside % page, -1)
    taken = torch.stack([more.sum(), torch.zeros_like(more[0])]).to(torch.int32)
    return {"q_start": q_start, "seq_lens": seq_lens, "n_blocks": n_blocks, "slots": slots, "positions": position, "taken": taken,
            "table": table}


def _plain_verify(s):
    target, draft, tokens, n_draft, u = s["target"], s["draft"], s["tokens"].long(), s["n_draft"], s["u"]
    b, k, v = draft.shape
    dev = target.device
    p = target[:, :k].gather(2, tokens[:, :, None])[:, :, 0].float()
    q = draft.gather(2, tokens[:, :, None])[:, :, 0].float()
    i = torch.arange(k, device=dev)
    passed = (u * q < p) & (i < n_draft[:, None])
    accepted = torch.cumprod(passed.int(), 1).sum(1).int()
    rows = torch.arange(b, device=dev)
    p = target[rows, accepted.long()].float()
    q = draft[rows, accepted.clamp(max=k - 1).long()].float()
    left = torch.where((accepted < n_draft)[:, None], (p - q).clamp(min=0), p)
    left = torch.where(left.amax(1, keepdim=True) > 0, left, p)
    key = left / s["noise"]
    best = key.amax(1, keepdim=True)
    ids = torch.arange(v, device=dev)
    drawn = torch.where(best[:, 0] > 0, torch.where(key == best, ids, v).amin(1), -1)
    at = torch.arange(k + 1, device=dev)
    kept = torch.cat([tokens, tokens[:, :1]], 1)
    out = torch.where(at < accepted[:, None], kept, torch.where(at == accepted[:, None], drawn[:, None], -1))
    return {"tokens": out.int(), "accepted": accepted}


# ---------------------------------------------------------------- what a pass cannot do without
def _size(name):
    return 4 if name == "f32" else 2


def work(case):
    if case["op"] == "attention":
        q_lens, old = _lens(case)
        seen = read = 0
        for n, o in zip(q_lens, old):
            w = case["window"] or n + o
            if n:
                # token i sees min(o + i + 1, w) keys
                short = max(0, min(n, w - o))
                seen += short * o + short * (short + 1) // 2 + (n - short) * w
                read += min(n + o, n - 1 + w)
        e = _size(case["dtype"])
        tokens = sum(q_lens)
        return {"bytes": 2 * read * case["hkv"] * case["d"] * e + tokens * case["hq"] * (2 * case["d"] * e + 4),
                "flops": 4 * seen * case["hq"] * case["d"]}
    if case["op"] == "write":
        kept = case["tokens"] - len(range(4, case["tokens"], 9))
        return {"bytes": 2 * kept * case["hkv"] * case["d"] * (_size(case["src"]) + _size(case["dtype"])) + 8 * case["tokens"],
                "flops": 0}
    if case["op"] == "tables":
        new, old = _tables_lens(case)
        page = case["page"]
        need = sum(max(0, -(-(o + n) // page) - (-(-o // page) + (i % 5 == 3))) for i, (o, n) in enumerate(zip(old, new)))
        return {"bytes": 6 * 4 * case["b"] + 8 * need + 12 * case["room"], "flops": 0}
    # one row each of the target's, the draft's and the noise
    return {"bytes": case["b"] * case["v"] * (2 * _size(case["dtype"]) + 4) + case["b"] * case["k"] * 24, "flops": 3 * case["b"] * case["v"]}


# ---------------------------------------------------------------- in 64 bits
def exact(case, seed):
    if case["op"] == "attention":
        return _exact_attention(case, prepare(case, seed))
    if case["op"] == "write":
        s = prepare(case, seed)
        got = {}
        for name, x, cache in (("k_cache", s["k"], s["kc"]), ("v_cache", s["v"], s["vc"])):
            flat = cache.double().reshape(-1, *x.shape[1:])
            kept = torch.nonzero(s["slots"] >= 0)[:, 0]
            flat.index_copy_(0, s["slots"].index_select(0, kept), x.double().index_select(0, kept))
            got[name] = flat.reshape(cache.shape)
        return got
    return None


def _exact_attention(case, s):
    """Request by request and a few rows at a time, over the keys that the rows see and no others."""
    q, kc, vc = s["q"], s["kc"], s["vc"]
    rep, d = case["hq"] // case["hkv"], case["d"]
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=q.device)
    q_lens, old = _lens(case)
    begin = 0
    for r, (n, o) in enumerate(zip(q_lens, old)):
        used = s["table"][r][: -(-(n + o) // case["page"])].long()
        k = kc.index_select(0, used).flatten(0, 1)[: n + o].double().transpose(0, 1)
        v = vc.index_select(0, used).flatten(0, 1)[: n + o].double().transpose(0, 1)
        for i in range(0, n, 256):
            c = min(256, n - i)
            lo = max(0, o + i + 1 - case["window"]) if case["window"] else 0
            hi = o + i + c
            mine = q[begin + i: begin + i + c].double().view(c, case["hkv"], rep, d).permute(1, 2, 0, 3)
            w = torch.einsum("hrid,hjd->hrij", mine, k[:, lo:hi]) / math.sqrt(d)
            j = torch.arange(lo, hi, device=q.device)
            pos = torch.arange(o + i, o + i + c, device=q.device)[:, None]
            hidden = j > pos
            if case["window"]:
                hidden |= j <= pos - case["window"]
            w.masked_fill_(hidden, -math.inf)
            z = torch.logsumexp(w, -1)
            o64 = torch.einsum("hrij,hjd->ihrd", torch.exp(w - z[..., None]), v[:, lo:hi])
            out[begin + i: begin + i + c] = o64.reshape(c, -1, d)
            lse[begin + i: begin + i + c] = z.permute(2, 0, 1).reshape(c, -1)
        begin += n
    return {"out": out, "lse": lse}
