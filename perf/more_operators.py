"""The parts of a batched serving step that differ from request to request, as cases to measure: the pages that requests
share, give back or get copies of; the rules that each request puts on its next token; the low-rank adapter that each
request brings beside the shared projections.

`run` computes each one in elementary torch operations in 32 bits (`own` false) or by the library's entry points
(`own` true).  Lengths follow from a case alone (`spread`), everything else from the seed."""
import math
import random

import torch

own = False

_DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def listed():
    """3584, 4608 (28 + 2 * 4 heads of 128) and 18944 are the rows of the repository's projections; 512 and 2630 its token counts."""
    return [
        # four users with two samples each; one sample ends, another is continued twice
        _fork("fork_b8", 8, 8, 2, 60, 3000, 16),
        # a full batch of beams: every step some are dropped and others continued several times
        _fork("fork_b700", 700, 700, 4, 30, 9000, 16),
        # a small cache put in order
        _compact("compact_b8", 8, 60, 3000, 16, 700),
        # a large cache in small pages after a day of requests, half of it held
        _compact("compact_b500", 500, 30, 12000, 16, 131072),
        # the last pages of a few forked requests
        _copy("copy_8", 8, 16, 4, 128, "nhd", "f16", 900, partial=True),
        # the moves of a compaction
        _copy("copy_2k", 2048, 64, 4, 128, "hnd", "bf16", 6000, partial=False),
        # one user's next token: temperature and penalties
        _probs("probs_b1", 1, 0, 32000, "f32", 700, 700, bias=0, masks=0),
        # a batch with drafted tokens, biases and grammars, 16-bit logits, adjusted logits wanted too
        _probs("probs_b24_k4", 24, 4, 128256, "bf16", 50, 6000, bias=40, masks=5, adjusted=True),
        # a full batch to be verified, a vocabulary with an odd size
        _probs("probs_b160_k5", 160, 5, 100277, "f32", 20, 4000, bias=300, masks=8),
        # one user's token through the attention's projections
        _lora("lora_b1", 1, 1, 1, 3584, 4608, 3584, 16, 4, "f16"),
        # a decode batch, nearly as many adapters as requests
        _lora("lora_b96", 96, 1, 1, 3584, 4608, 3584, 64, 64, "bf16"),
        # prompts of several requests through the feed-forward block's up and down projections
        _lora("lora_prompts_ffn", 9, 100, 1000, 3584, 18944, 3584, 32, 6, "bf16"),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["fork", "compact", "copy", "probs", "probs", "probs", "lora", "lora", "lora"])
    if op == "fork":
        return _fork(None, log(1, 700), log(1, 700), rng.randint(1, 5), rng.choice([0, 30]), log(50, 9000), rng.choice([8, 16, 32, 64]))
    if op == "compact":
        return _compact(None, log(1, 500), rng.choice([0, 30]), log(50, 9000), rng.choice([16, 32, 64]), log(1000, 131072))
    if op == "copy":
        page = rng.choice([8, 16, 32, 64, 128])
        n = log(1, 2048 * 64 // page)
        return _copy(None, n, page, rng.choice([1, 2, 4, 8][: 4 if n * page < 60000 else 3]), rng.choice([64, 96, 128]),
                     rng.choice(["nhd", "hnd"]), rng.choice(["f16", "bf16"]), 2 * n + log(2, 1000), partial=rng.random() < 0.5)
    if op == "probs":
        v = log(1000, 152064)
        k = rng.randint(0, 6)
        b = log(1, max(1, min(256, int(9e7 / ((k + 1) * v)))))
        return _probs(None, b, k, v, rng.choice(["f32", "f32", "f16", "bf16"]), rng.choice([0, 30]), log(50, 8000), bias=rng.choice([0, log(1, 500)]),
                      masks=rng.choice([0, rng.randint(1, 8)]), adjusted=rng.random() < 0.3)
    hidden = rng.choice([512, 1024, 2048, 3584])
    wide = rng.choice([hidden, 4608, 18944, 1000])
    b = log(1, 128)
    hi = log(1, max(1, min(2000, 3000 // b)))
    return _lora(None, b, rng.choice([1, hi]), hi, hidden, wide, hidden, rng.choice([8, 16, 24, 32, 64, 128]), log(1, 64), rng.choice(["f16", "bf16"]))


def _named(name, case):
    return case if name is None else {"name": name, **case}


def _fork(name, old, new, beams, kv_lo, kv_hi, page):
    return _named(name, {"op": "fork", "old": old, "new": new, "beams": beams, "kv_lo": kv_lo, "kv_hi": kv_hi, "page": page})


def _compact(name, b, kv_lo, kv_hi, page, pages):
    return _named(name, {"op": "compact", "b": b, "kv_lo": kv_lo, "kv_hi": kv_hi, "page": page, "pages": pages})


def _copy(name, n, page, hkv, d, layout, dtype, pages, partial):
    return _named(name, {"op": "copy", "n": n, "page": page, "hkv": hkv, "d": d, "layout": layout, "dtype": dtype, "pages": pages, "partial": partial})


def _probs(name, b, k, v, dtype, hist_lo, hist_hi, bias, masks, adjusted=False):
    return _named(name, {"op": "probs", "b": b, "k": k, "v": v, "dtype": dtype, "hist_lo": hist_lo, "hist_hi": hist_hi, "bias": bias,
                         "masks": masks, "adjusted": adjusted})


def _lora(name, b, q_lo, q_hi, into, wide, out, rank, adapters, dtype):
    """Two projections of one step: (tokens, into) -> wide, and (tokens, wide or into) -> out."""
    return _named(name, {"op": "lora", "b": b, "q_lo": q_lo, "q_hi": q_hi, "into": into, "wide": wide, "out": out, "rank": rank,
                         "adapters": adapters, "dtype": dtype})


def spread(lo, hi, n, salt=0):
    """n lengths from lo to hi, even in their logarithm, in a fixed mixed order."""
    if n == 1:
        return [hi]
    got = [int(round((lo + 1) * ((hi + 1) / (lo + 1)) ** (i / (n - 1)))) - 1 for i in range(n)]
    random.Random(1000 * n + salt).shuffle(got)
    return got


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return {"fork": _prepare_fork, "compact": _prepare_compact, "copy": _prepare_copy, "probs": _prepare_probs,
            "lora": _prepare_lora}[case["op"]](case, g, seed) | {"op": case["op"]}


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _f32(x):
    return torch.tensor(x, dtype=torch.float32, device="cuda")


def _randn(g, shape, dtype, scale=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype).mul_(scale)


def _old_rows(case):
    """Lengths of the rows that there are: the samples of one request are of one age, a few tokens apart."""
    groups = spread(case["kv_lo"], case["kv_hi"], -(-case["old"] // case["beams"]), 1)
    return [max(0, groups[i // case["beams"]] - i % case["beams"]) for i in range(case["old"])]


def _shared(case, lens):
    """Pages that a row has in common with the first row of its request: about two thirds of them."""
    return [0 if i % case["beams"] == 0 else min(lens[i], lens[i - i % case["beams"]]) * 2 // 3 // case["page"] for i in range(len(lens))]


def _new_rows(case, seed):
    """The old row that each new one continues (-1: none, one in 16) and the tokens that it keeps: all, or a few less."""
    r = random.Random(seed)
    old = _old_rows(case)
    parents = [-1 if r.random() < 1 / 16 else min(i, case["old"] - 1) if r.random() < 0.6 else r.randrange(case["old"]) for i in range(case["new"])]
    return parents, [0 if p < 0 else max(0, old[p] - r.choice([0, 0, 0, 1, 2, 5])) for p in parents]


def _held_of(case, lens):
    """Every fifth row still holds a page more than its tokens need."""
    return [-(-n // case["page"]) + (i % 5 == 3) for i, n in enumerate(lens)]


def _prepare_fork(case, g, seed):
    lens = _old_rows(case)
    shared, held = _shared(case, lens), _held_of(case, lens)
    pages = sum(held) + case["new"] + 5
    width = max(held) + 2
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    n_blocks = _i32(held)
    first = torch.cumsum(n_blocks, 0, dtype=torch.int32) - n_blocks
    leader = first[torch.arange(len(lens), device="cuda") // case["beams"] * case["beams"]]
    j = torch.arange(width, device="cuda", dtype=torch.int32)
    at = torch.where(j < _i32(shared)[:, None], leader[:, None] + j, first[:, None] + j)
    table = torch.where(j < n_blocks[:, None], order[at.clamp(max=pages - 1).long()], -1)
    parents, keep = _new_rows(case, seed)
    return {"table": table.contiguous(), "n_blocks": n_blocks, "parents": _i32(parents), "lens": _i32(keep), "page": case["page"], "pages": pages}


def _compact_lens(case):
    """Lengths, cut so that at least a third of the cache is free."""
    lens = spread(case["kv_lo"], case["kv_hi"], case["b"], 2)
    room = case["pages"] * 2 // 3
    got = []
    for n in lens:
        n = min(n, room * case["page"])
        got.append(n)
        room -= -(-n // case["page"])
    return got


def _prepare_compact(case, g, seed):
    held = [-(-n // case["page"]) for n in _compact_lens(case)]
    width = max(held) + 2
    order = torch.randperm(case["pages"], generator=g, device="cuda").to(torch.int32)
    n_blocks = _i32(held)
    first = torch.cumsum(n_blocks, 0, dtype=torch.int32) - n_blocks
    j = torch.arange(width, device="cuda", dtype=torch.int32)
    table = torch.where(j < n_blocks[:, None], order[(first[:, None] + j).clamp(max=case["pages"] - 1).long()], -1)
    return {"table": table.contiguous(), "n_blocks": n_blocks, "pages": case["pages"]}


def _copy_tokens(case):
    return [1 + (7 * i) % case["page"] if case["partial"] else case["page"] for i in range(case["n"])]


def _prepare_copy(case, g, seed):
    """One pair in nine is padding (-1, -1), as of a row that needed no copy."""
    n, page, hkv, d = case["n"], case["page"], case["hkv"], case["d"]
    shape = (case["pages"], page, hkv, d) if case["layout"] == "nhd" else (case["pages"], hkv, page, d)
    kc, vc = _randn(g, shape, _DT[case["dtype"]]), _randn(g, shape, _DT[case["dtype"]])
    if case["layout"] == "hnd":
        kc, vc = kc.permute(0, 2, 1, 3), vc.permute(0, 2, 1, 3)
    order = torch.randperm(case["pages"], generator=g, device="cuda")[: 2 * n].to(torch.int32)
    pairs = order.view(n, 2).clone()
    pairs[4::9] = -1
    return {"kc": kc, "vc": vc, "pairs": pairs, "tokens": _i32(_copy_tokens(case)) if case["partial"] else None}


def _hist_lens(case):
    return spread(case["hist_lo"], case["hist_hi"], case["b"], 5)


def _bias_lens(case):
    """Two requests in three bring biases."""
    return [0 if i % 3 == 1 else min(case["bias"], case["v"]) for i in range(case["b"])]


def _prepare_probs(case, g, seed):
    """Tokens of a request repeat as words do (the cube of a uniform number); a mask allows one token in four or a few tokens;
    one request in eight is greedy."""
    b, k, v, dt = case["b"], case["k"], case["v"], _DT[case["dtype"]]
    lens = _hist_lens(case)
    width = max(max(lens), 1) + 3

    def words(shape):
        return (torch.rand(shape, generator=g, device="cuda").pow_(3) * v).long().clamp_(max=v - 1).to(torch.int32)

    def uniform(lo, hi):
        return torch.rand(b, generator=g, device="cuda") * (hi - lo) + lo

    tokens = words((b, width))
    token_lens = _i32(lens)
    tokens[torch.arange(width, device="cuda") >= token_lens[:, None]] = -1  # nothing was written there
    temperature = uniform(0.4, 1.3)
    temperature[5::8] = 0.0
    s = {"logits": _randn(g, (b, k + 1, v), dt, 3.0), "tokens": tokens, "token_lens": token_lens, "prompt_lens": _i32([n // 2 for n in lens]),
         "draft": words((b, k)) if k else None, "temperature": temperature, "repetition": uniform(1.0, 1.5),
         "frequency": uniform(0.0, 0.4), "presence": uniform(-0.2, 0.6), "bias": None, "mask": None, "mask_rows": None,
         "adjusted": torch.empty((b, k + 1, v), dtype=torch.float32, device="cuda") if case["adjusted"] else None,
         "probs": torch.empty((b, k + 1, v), dtype=torch.float32, device="cuda")}
    if case["bias"]:
        n = _bias_lens(case)
        start = [0]
        for m in n:
            start.append(start[-1] + m)
        step = max(1, v // max(1, case["bias"]))  # distinct tokens: one of each stretch of the vocabulary
        at = torch.arange(start[-1], device="cuda") % min(case["bias"], v)
        ids = at * step + torch.randint(0, step, (start[-1],), generator=g, device="cuda")
        s["bias"] = (_i32(start), ids.to(torch.int32), _randn(g, (start[-1],), torch.float32, 2.0))
    if case["masks"]:
        m, words_of = case["masks"], -(-v // 32)
        bits = [torch.randint(-2 ** 31, 2 ** 31, (m, words_of), generator=g, device="cuda") for _ in range(2)]
        mask = bits[0] & bits[1]
        few = torch.rand((m, words_of), generator=g, device="cuda") < 40 / words_of
        few[:, 3] = True
        mask = torch.where((torch.arange(m, device="cuda") % 2 == 1)[:, None], torch.where(few, bits[0] | 1, 0), mask)
        s["mask"] = mask.to(torch.int32)
        rows = torch.randint(0, m, (b, k + 1), generator=g, device="cuda", dtype=torch.int32)
        rows[torch.arange(b, device="cuda") % 2 == 1] = -1
        s["mask_rows"] = rows
    return s


def _q_lens(case):
    return spread(case["q_lo"], case["q_hi"], case["b"], 6)


def _down(case):
    """Rows that the second projection reads: a feed-forward block's are the first's columns."""
    return case["wide"] if case["wide"] == 18944 else case["into"]


def _adapter_of(case, seed):
    """One request in seven brings no adapter."""
    r = random.Random(seed)
    return [-1 if i % 7 == 6 else r.randrange(case["adapters"]) for i in range(case["b"])]


def _ranks(case):
    """Every third adapter is of half the rank."""
    return [case["rank"] // 2 if i % 3 == 2 else case["rank"] for i in range(case["adapters"])]


def _prepare_lora(case, g, seed):
    dt, r, n = _DT[case["dtype"]], case["rank"], case["adapters"]
    lens = _q_lens(case)
    t = sum(lens)
    start = [0]
    for m in lens:
        start.append(start[-1] + m)
    s = {"adapters": _i32(_adapter_of(case, seed)), "q_start": _i32(start), "tokens": t, "n": n, "ranks": _i32(_ranks(case)),
         "scales": _f32([2.0 if i % 2 else 0.5 for i in range(n)]), "sides": []}
    for into, out in ((case["into"], case["wide"]), (_down(case), case["out"])):
        s["sides"].append({"x": _randn(g, (t, into), torch.float32), "y": _randn(g, (t, out), torch.float32),
                           "a": _randn(g, (n, r, into), dt, 1 / math.sqrt(into)), "b": _randn(g, (n, out, r), dt, 0.3 / math.sqrt(r)),
                           "out": torch.empty((t, out), dtype=torch.float32, device="cuda")})
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    if own:
        return _own(s)
    return {"fork": _plain_fork, "compact": _plain_compact, "copy": _plain_copy, "probs": _plain_probs, "lora": _plain_lora}[s["op"]](s)


def _own(s):
    import quantized_int8_gemm_gb300 as mmq
    if s["op"] == "fork":
        f = mmq.mmq_page_fork(s["table"], s["n_blocks"], s["parents"], s["lens"], s["page"], s["pages"])
        return {"table": f.block_table, "n_blocks": f.n_blocks, "pairs": f.pairs, "tokens": f.tokens, "free_pages": f.free_pages, "counts": f.counts}
    if s["op"] == "compact":
        c = mmq.mmq_page_compact(s["table"], s["n_blocks"], s["pages"])
        return {"table": c.block_table, "pairs": c.pairs, "counts": c.counts}
    if s["op"] == "copy":
        mmq.mmq_page_copy(s["kc"], s["vc"], s["pairs"], s["tokens"])
        return {"k_cache": s["kc"], "v_cache": s["vc"]}
    if s["op"] == "probs":
        probs, adjusted = mmq.mmq_token_probs(
            s["logits"], temperature=s["temperature"], tokens=s["tokens"], token_lens=s["token_lens"], prompt_lens=s["prompt_lens"],
            draft_tokens=s["draft"], repetition=s["repetition"], frequency=s["frequency"], presence=s["presence"], bias=s["bias"],
            mask=s["mask"], mask_rows=s["mask_rows"], probs=s["probs"], adjusted=s["adjusted"])
        return {"probs": probs, "adjusted": adjusted}
    plan = mmq.mmq_lora_plan(s["adapters"], s["q_start"], s["tokens"], s["n"])
    return [mmq.mmq_lora(p["x"], p["y"], p["a"], p["b"], plan, scales=s["scales"], ranks=s["ranks"], out=p["out"]) for p in s["sides"]]


def _plain_fork(s):
    table, held, parents, page, pages = s["table"], s["n_blocks"], s["parents"], s["page"], s["pages"]
    width, new, dev = table.shape[1], parents.numel(), table.device
    p = parents.clamp(min=0).long()
    length = torch.where(parents >= 0, s["lens"], 0)
    need = torch.minimum((length + page - 1) // page, held[p]).clamp(max=width)
    j = torch.arange(width, device=dev, dtype=torch.int32)
    rows = torch.where(j < need[:, None], table[p], -1)
    b = torch.arange(new, device=dev)
    last = (length // page).clamp(max=width - 1).long()
    part = (length % page > 0) & (length // page < need)
    w = torch.where(part, rows[b, last], pages).long()  # (pages: an entry for those that have none)
    full = j < torch.minimum(length // page, need)[:, None]
    is_full = torch.zeros(pages + 1, dtype=torch.bool, device=dev)
    is_full[torch.where(full, rows, pages).long()] = True
    keeper = torch.full((pages + 1,), new, device=dev).scatter_reduce(0, w, b, "amin")
    keeps = part & ~is_full[w] & (keeper[w] == b)
    copied = part & ~keeps
    is_held = is_full.clone()
    is_held[torch.where(keeps, w, pages)] = True
    free = ~is_held[:pages]
    nth = torch.cumsum(free, 0) - 1
    ids = torch.arange(pages, device=dev)
    n_free, n_copied = free.sum(), copied.sum()
    listed_free = torch.full((pages + 1,), -1, device=dev).scatter(0, torch.where(free, nth, pages), torch.where(free, ids, -1))
    which = torch.cumsum(copied, 0) - 1
    target = torch.where(copied & (which < n_free), listed_free[which.clamp(0, pages)], -1)
    rows[b, last] = torch.where(copied, target, rows[b, last].long()).int()
    found = copied & (target >= 0)
    pairs = torch.where(found[:, None], torch.stack([w, target], 1), -1)
    left = ids + n_copied
    free_pages = torch.where(left < n_free, listed_free[left.clamp(max=pages)], -1)
    counts = torch.stack([(n_free - n_copied).clamp(min=0), (n_copied - n_free).clamp(min=0)])
    return {"table": rows, "n_blocks": need.int(), "pairs": pairs.int(), "tokens": torch.where(found, length % page, 0).int(),
            "free_pages": free_pages.int(), "counts": counts.int()}


def _plain_compact(s):
    table, pages, dev = s["table"], s["pages"], s["table"].device
    j = torch.arange(table.shape[1], device=dev, dtype=torch.int32)
    valid = j < s["n_blocks"][:, None]
    held = torch.zeros(pages + 1, dtype=torch.bool, device=dev)
    held[torch.where(valid, table, pages).long()] = True
    held = held[:pages]
    n = held.sum()
    ids = torch.arange(pages, device=dev)
    moved, hole = held & (ids >= n), ~held & (ids < n)
    room = pages // 2
    nth_moved, nth_hole = torch.cumsum(moved, 0) - 1, torch.cumsum(hole, 0) - 1
    none = torch.full((room + 1,), -1, device=dev)
    src = none.scatter(0, torch.where(moved, nth_moved, room), torch.where(moved, ids, -1))
    dst = none.scatter(0, torch.where(hole, nth_hole, room), torch.where(hole, ids, -1))
    to = torch.where(moved, dst[nth_moved.clamp(0, room)], ids)
    return {"table": torch.where(valid, to[table.clamp(min=0).long()], -1).int(), "pairs": torch.stack([src[:room], dst[:room]], 1).int(),
            "counts": torch.stack([n, moved.sum()]).int()}


def _plain_copy(s):
    kept = s["pairs"][:, 0] >= 0
    src, dst = s["pairs"][kept].long().unbind(1)
    for c in (s["kc"], s["vc"]):
        new = c[src]
        if s["tokens"] is not None:
            i = torch.arange(c.shape[1], device=c.device)
            new = torch.where((i < s["tokens"][kept][:, None])[:, :, None, None], new, c[dst])
        c[dst] = new
    return {"k_cache": s["kc"], "v_cache": s["vc"]}


def _plain_probs(s):
    logits, tokens, dev = s["logits"], s["tokens"], s["logits"].device
    b, rows, v = logits.shape
    width = tokens.shape[1]
    i = torch.arange(width, device=dev)
    there = i < s["token_lens"][:, None]
    answered = there & (i >= s["prompt_lens"][:, None])
    at = torch.where(there, tokens, v).long()
    counts = torch.zeros((b, v + 1), device=dev).scatter_add_(1, at, answered.float())[:, None]
    seen = torch.zeros((b, v + 1), device=dev).scatter_add_(1, at, there.float())[:, None]
    if s["draft"] is not None:
        # row i has the drafted tokens before it
        before = (torch.arange(rows - 1, device=dev) < torch.arange(rows, device=dev)[:, None]).float().expand(b, -1, -1)
        more = torch.zeros((b, rows, v + 1), device=dev).scatter_add_(2, s["draft"].long()[:, None].expand(-1, rows, -1), before)
        counts, seen = counts + more, seen + more
    counts, seen = counts[..., :v], seen[..., :v]
    x = logits.float()
    rho = s["repetition"][:, None, None]
    x = torch.where(seen > 0, torch.where(x > 0, x / rho, x * rho), x)
    x = x - s["frequency"][:, None, None] * counts
    x = x - torch.where(counts > 0, s["presence"][:, None, None], 0.0)
    if s["bias"] is not None:
        start, ids, values = s["bias"]
        of = torch.searchsorted(start[1:].contiguous(), torch.arange(ids.numel(), device=dev, dtype=torch.int32), right=True)
        x = x + torch.zeros((b, v), device=dev).index_put_((of, ids.long()), values)[:, None]
    if s["mask"] is not None:
        t = torch.arange(v, device=dev)
        bits = (s["mask"][:, t // 32] >> (t % 32).int() & 1).bool()
        which = s["mask_rows"]
        x = torch.where((which < 0)[..., None] | bits[which.clamp(min=0).long()], x, -math.inf)
    temperature = s["temperature"][:, None, None]
    top = x.amax(-1, keepdim=True)
    some = top > -math.inf
    e = torch.exp((x - torch.where(some, top, 0.0)) / torch.where(temperature > 0, temperature, 1.0))
    total = e.sum(-1, keepdim=True)
    p = torch.where(some, e / total, 0.0)
    ids = torch.arange(v, device=dev)
    first = torch.where(x == top, ids, v).amin(-1, keepdim=True)
    p = torch.where(temperature > 0, p, ((ids == first) & some).float())
    return {"probs": p, "adjusted": x if s["adjusted"] is not None else None}


def _plain_lora(s):
    """The products with every adapter at once, of which a token keeps its own adapter's columns."""
    t, n = s["tokens"], s["n"]
    dev = s["q_start"].device
    of = torch.searchsorted(s["q_start"][1:].contiguous(), torch.arange(t, device=dev, dtype=torch.int32), right=True)
    mine = s["adapters"][of]
    got = []
    for p in s["sides"]:
        r = p["a"].shape[1]
        h = torch.matmul(p["x"], p["a"].float().view(n * r, -1).t()).view(t, n, r)
        kept = (torch.arange(n, device=dev) == mine[:, None])[:, :, None] & (torch.arange(r, device=dev) < s["ranks"][:, None])
        h = torch.where(kept, h * s["scales"][:, None], 0.0)
        got.append(p["y"] + torch.matmul(h.view(t, n * r), p["b"].float().permute(0, 2, 1).reshape(n * r, -1)))
    return got


# ---------------------------------------------------------------- what a pass cannot do without
def _size(name):
    return 4 if name == "f32" else 2


def work(case):
    op = case["op"]
    if op == "fork":
        old = _old_rows(case)
        held = _held_of(case, old)
        width, pages = max(held) + 2, sum(held) + case["new"] + 5
        # the parents' entries; the new rows and the free list
        return {"bytes": 4 * (sum(old) // case["page"] * case["new"] // case["old"] + width * case["new"] + pages + 6 * case["new"]), "flops": 0}
    if op == "compact":
        held = [-(-n // case["page"]) for n in _compact_lens(case)]
        return {"bytes": 4 * (sum(held) + (max(held) + 2) * case["b"] + 2 * (case["pages"] // 2) + case["b"]), "flops": 0}
    if op == "copy":
        kept = sum(t for i, t in enumerate(_copy_tokens(case)) if i % 9 != 4)
        return {"bytes": 2 * 2 * kept * case["hkv"] * case["d"] * 2 + 8 * case["n"], "flops": 0}
    if op == "probs":
        b, rows, v = case["b"], case["k"] + 1, case["v"]
        masked = (b + 1) // 2 * rows if case["masks"] else 0
        return {"bytes": b * rows * v * (_size(case["dtype"]) + 4 + 4 * case["adjusted"]) + min(masked, case["masks"]) * v // 8 +
                4 * sum(_hist_lens(case)) + 8 * sum(_bias_lens(case)) + 4 * b * (8 + 2 * rows), "flops": 6 * b * rows * v}
    t = sum(_q_lens(case))
    used = min(case["adapters"], case["b"])
    ranks = sum(sorted(_ranks(case))[:used])
    into, out = case["into"] + _down(case), case["wide"] + case["out"]
    return {"bytes": 4 * t * (into + 2 * out) + 2 * ranks * (into + out) + 8 * t, "flops": 2 * t * case["rank"] * (into + out)}


# ---------------------------------------------------------------- in 64 bits
def exact(case, seed):
    if case["op"] == "copy":
        return _exact_copy(case, prepare(case, seed))
    if case["op"] == "probs":
        return _exact_probs(case, prepare(case, seed))
    if case["op"] == "lora":
        return _exact_lora(case, seed, prepare(case, seed))
    return None


def _exact_copy(case, s):
    got = {}
    for name, cache in (("k_cache", s["kc"]), ("v_cache", s["vc"])):
        page = case["page"]
        flat = cache.double().reshape(case["pages"] * page, -1)
        src, dst = [], []
        for (a, z), n in zip(s["pairs"].tolist(), _copy_tokens(case)):
            if a >= 0:
                src += range(a * page, a * page + n)
                dst += range(z * page, z * page + n)
        src, dst = torch.tensor(src, device="cuda"), torch.tensor(dst, device="cuda")
        got[name] = flat.index_copy(0, dst, flat.index_select(0, src)).reshape(cache.shape)
    return got


def _exact_probs(case, s):
    """Row by row, over counts that are taken from the tokens as they stand."""
    b, k, v = case["b"], case["k"], case["v"]
    probs = torch.zeros((b, k + 1, v), dtype=torch.float64, device="cuda")
    adjusted = torch.zeros((b, k + 1, v), dtype=torch.float64, device="cuda") if case["adjusted"] else None
    rule = {n: s[n].double().tolist() for n in ("temperature", "repetition", "frequency", "presence")}
    bias_at = s["bias"][0].tolist() if s["bias"] is not None else None
    rows = s["mask_rows"].tolist() if s["mask"] is not None else None
    open_bits = None
    if rows is not None:
        open_bits = torch.stack([s["mask"] >> i & 1 for i in range(32)], -1).flatten(1)[:, :v].bool()
    for i, n in enumerate(_hist_lens(case)):
        for j in range(k + 1):
            drafted = s["draft"][i, :j] if k else s["tokens"][i, :0]
            said = torch.cat([s["tokens"][i, n // 2: n], drafted]).long()
            known = torch.cat([s["tokens"][i, : n // 2].long(), said])
            times = torch.bincount(said, minlength=v).double()
            x = s["logits"][i, j].double()
            met = torch.bincount(known, minlength=v) > 0
            x = torch.where(met, torch.where(x < 0, x * rule["repetition"][i], x / rule["repetition"][i]), x)
            x = x - rule["frequency"][i] * times - rule["presence"][i] * (times > 0)
            if bias_at is not None:
                lo, hi = bias_at[i], bias_at[i + 1]
                x = x.index_add(0, s["bias"][1][lo:hi].long(), s["bias"][2][lo:hi].double())
            if rows is not None and rows[i][j] >= 0:
                x = x.masked_fill(~open_bits[rows[i][j]], -math.inf)
            if adjusted is not None:
                adjusted[i, j] = x
            if rule["temperature"][i] > 0:
                z = x / rule["temperature"][i]
                probs[i, j] = torch.exp(z - torch.logsumexp(z, 0))
            else:
                probs[i, j, torch.argmax(x)] = 1.0
    return {"probs": probs, "adjusted": adjusted}


def _exact_lora(case, seed, s):
    """Request by request, a few hundred tokens at a time."""
    got = []
    for p in s["sides"]:
        out = p["y"].double()
        begin = 0
        for n, a in zip(_q_lens(case), _adapter_of(case, seed)):
            if a >= 0:
                r = _ranks(case)[a]
                down, up = p["a"][a, :r].double(), p["b"][a, :, :r].double()
                scale = 2.0 if a % 2 else 0.5
                for i in range(begin, begin + n, 512):
                    x = p["x"][i: min(i + 512, begin + n)].double()
                    out[i: i + x.shape[0]] += torch.einsum("tr,or->to", torch.einsum("ti,ri->tr", x, down), up) * scale
            begin += n
        got.append(out)
    return got
