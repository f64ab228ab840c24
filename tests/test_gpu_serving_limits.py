"""The serving step's operators at the limits of their arguments: rows that a step has no room for, extreme windows, waits
that run out, buffers given by the caller.  Problems, references and tolerances are those of test_gpu_serving.py."""
import math
import threading

import pytest
import torch

from tests.test_gpu_serving import BF16, F16, UNIT, _i32, _no_device_error, _problem, _reference, mmq  # noqa: F401

pytestmark = pytest.mark.gpu


def _check_rows(p, out, lse, scale, causal, window):
    """The rows that were given, against the whole problem's."""
    n = out.shape[0]
    ref, z, tol, z_tol = (x[:n] for x in _reference(p, scale, causal, window))
    assert torch.isfinite(out).all()
    assert ((out.double() - ref).abs() <= tol).all()
    none = torch.isinf(z)
    assert torch.equal(torch.isinf(lse) & (lse < 0), none)
    assert (torch.where(none, 0.0, (lse.double() - torch.where(none, 0.0, z)).abs()) <= z_tol).all()


@pytest.mark.parametrize("d,page", [(64, 16), (128, 64), (128, 5), (256, 16)])
@pytest.mark.parametrize("room", [1, 3, 150, 203])
def test_attention_of_a_step_with_more_tokens_than_rows(mmq, d, page, room):  # noqa: F811
    """q_start counts tokens that q has no row for (the tables' new tokens past max_tokens): the rows that are there keep
    their places, and the keys of the others, which nothing wrote, are not seen by them."""
    q_lens, kv_lens = [3, 200, 1, 40], [700, 1500, 33, 40]
    for causal, window in ((True, 0), (True, 70), (False, 0)):
        p = _problem(F16, q_lens, kv_lens, 8, 2, d, page, seed=room)
        if causal:
            at = 0
            for b, (n, length) in enumerate(zip(q_lens, kv_lens)):
                for i in range(max(0, min(n, room - at)), n):
                    key = length - n + i
                    for x in (p["kc"], p["vc"]):
                        x[p["table"][b, key // page], key % page] = math.nan
                at += n
        guard = 5
        out = torch.full((room + guard, 8, d), 7.0, dtype=F16, device="cuda")
        lse = torch.full((room + guard, 8), 7.0, device="cuda")
        mmq.mmq_paged_attention(p["q"][:room], p["kc"], p["vc"], p["table"], p["seq_lens"], p["q_start"], causal=causal, window=window,
                                out=out[:room], lse=lse[:room])
        _check_rows(p, out[:room], lse[:room], 1 / math.sqrt(d), causal, window)
        assert (out[room:] == 7).all() and (lse[room:] == 7).all()


@pytest.mark.parametrize("d,page", [(64, 16), (128, 16), (96, 3), (256, 16)])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 5, 2 ** 30])
@pytest.mark.parametrize("causal", [True, False])
def test_the_widest_windows(mmq, d, page, window, causal):  # noqa: F811
    """Windows near the largest number, in a chunk longer than its keys (places below zero)."""
    p = _problem(BF16, [3, 20, 300], [5, 12, 40], 4, 2, d, page)
    out, lse = mmq.mmq_paged_attention(p["q"], p["kc"], p["vc"], p["table"], p["seq_lens"], p["q_start"], causal=causal, window=window, lse=True)
    _check_rows(p, out, lse, 1 / math.sqrt(d), causal, window)


# ---------------------------------------------------------------- infinities and NaN that rows do see
def _put(p, which, b, key, at, value):
    page = p["kc"].shape[1]
    (p["keys"] if which == "kc" else p["values"])[b][key, :, at] = value
    p[which][p["table"][b, key // page], key % page, :, at] = value


def _reference_without(p, gone, scale):
    """As _reference (causal), with the key gone[b] of request b left out of its rows' sums."""
    q = p["q"].double()
    out, tol = torch.zeros_like(q), torch.zeros_like(q)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    lse_tol = torch.zeros_like(lse)
    u = UNIT[p["q"].dtype]
    at = 0
    for n, length, k, v, key in zip(p["q_lens"], p["kv_lens"], p["keys"], p["values"], gone):
        rep = q.shape[1] // k.shape[1]
        keep = [j for j in range(length) if j != key]
        kk, vv = (x[keep].double().repeat_interleave(rep, 1).permute(1, 0, 2) for x in (k, v))
        x = q[at:at + n].permute(1, 0, 2)
        s = x @ kk.transpose(1, 2) * scale
        size = (x.abs() @ kk.abs().transpose(1, 2) * scale).amax(-1)
        hidden = torch.tensor(keep, device="cuda") > torch.arange(length - n, length, device="cuda")[:, None]
        w = torch.softmax(s.masked_fill(hidden, -math.inf), -1)
        o, mass = w @ vv, w @ vv.abs()
        out[at:at + n] = o.permute(1, 0, 2)
        tol[at:at + n] = (u * (mass + o.abs()) * 1.0625 + 1e-4 * mass).permute(1, 0, 2)
        lse[at:at + n] = torch.logsumexp(s.masked_fill(hidden, -math.inf), -1).T
        lse_tol[at:at + n] = (2.0 ** -20 * size + 1e-5).T
        at += n
    return out, lse, tol, lse_tol


NOT_FINITE = [(64, 16, [150, 1], [900, 700]), (128, 16, [150, 1], [900, 700]), (128, 5, [70, 1], [300, 700]), (256, 16, [40, 1], [130, 700]),
              (128, 64, [1, 2], [9000, 20000]), (64, 16, [1, 2], [9000, 20000]), (128, 3, [1, 2], [9000, 20000])]


@pytest.mark.parametrize("d,page,q_lens,kv_lens", NOT_FINITE)
@pytest.mark.parametrize("back", [0, 30, 600])
@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_a_key_that_is_not_finite(mmq, d, page, q_lens, kv_lens, back, value):  # noqa: F811
    """One element of one key of each request, `back` places before the last.  Rows whose score of it is NaN or +inf are NaN;
    rows whose score is -inf give it no weight; rows that do not see it are as they were.  (bf16: no smallest weight to add
    to the tolerance.)"""
    p = _problem(BF16, q_lens, kv_lens, 8, 2, d, page, seed=back)
    p["q"][:, :, 1][p["q"][:, :, 1] == 0] = 1
    gone = [max(0, length - 1 - back) for length in kv_lens]
    for b, key in enumerate(gone):
        _put(p, "kc", b, key, 1, value)
    out, lse = mmq.mmq_paged_attention(p["q"], p["kc"], p["vc"], p["table"], p["seq_lens"], p["q_start"], lse=True)
    seen = torch.cat([torch.arange(length - n, length) >= key for n, length, key in zip(q_lens, kv_lens, gone)]).cuda()[:, None]
    spoilt = seen & (p["q"][:, :, 1] > 0) if value == math.inf else seen.expand(lse.shape)
    assert torch.isnan(out[spoilt]).all() and torch.isnan(lse[spoilt]).all()
    ref, z, tol, z_tol = _reference_without(p, gone, 1 / math.sqrt(d))
    assert ((out.double() - ref).abs() <= tol)[~spoilt].all()
    assert ((lse.double() - z).abs() <= z_tol)[~spoilt].all()


@pytest.mark.parametrize("d,page,q_lens,kv_lens", NOT_FINITE)
@pytest.mark.parametrize("back", [0, 30, 600])
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
def test_a_value_that_is_not_finite(mmq, d, page, q_lens, kv_lens, back, value):  # noqa: F811
    """One element of one V row of each request: that column of the rows that see it is not finite (a row of the same chunk
    that does not see it may be either), the other columns and every lse are as they were."""
    p = _problem(BF16, q_lens, kv_lens, 8, 2, d, page, seed=back)
    ref, z, tol, z_tol = _reference(p, 1 / math.sqrt(d), True, 0)
    for b, length in enumerate(kv_lens):
        _put(p, "vc", b, max(0, length - 1 - back), 1, value)
    out, lse = mmq.mmq_paged_attention(p["q"], p["kc"], p["vc"], p["table"], p["seq_lens"], p["q_start"], lse=True)
    seen = torch.cat([torch.arange(length - n, length) >= max(0, length - 1 - back) for n, length in zip(q_lens, kv_lens)]).cuda()
    assert not torch.isfinite(out[seen][:, :, 1]).any()
    others = [i for i in range(d) if i != 1]
    assert ((out.double() - ref).abs() <= tol)[:, :, others].all()
    assert ((lse.double() - z).abs() <= z_tol).all()


def test_calls_of_two_threads_on_two_streams(mmq):  # noqa: F811
    """Each call has scratch of its own: the bits are those of calls one after another."""
    problems = [_problem(BF16, [300, 1, 5], [4000, 900, 3000], 28, 4, 128, 16, seed=1), _problem(F16, [1] * 6, [3000, 17, 900, 4000, 1, 250], 8, 2, 64, 16, seed=2)]

    def call(p, stream=None):
        return mmq.mmq_paged_attention(p["q"], p["kc"], p["vc"], p["table"], p["seq_lens"], p["q_start"], lse=True, stream=stream)

    want = [call(p) for p in problems]
    torch.cuda.synchronize()
    got, streams = [[], []], [torch.cuda.Stream(), torch.cuda.Stream()]
    threads = [threading.Thread(target=lambda i=i: got[i].extend(call(problems[i], streams[i]) for _ in range(50))) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert len(g) == 50 and all(torch.equal(x, y) for pair in g for x, y in zip(pair, w))


# ---------------------------------------------------------------- waits that run out
@pytest.fixture
def short_waits(mmq):  # noqa: F811
    """Waits give up as soon as they look at the clock (after 256 polls, about a millisecond)."""
    mmq.mmq_set_wait_timeout_ns(1)
    yield
    mmq.mmq_set_wait_timeout_ns(2 * 10 ** 9)


def _late_problem(n, kv_len, d):
    """Requests of which only the last ten have tokens (the first stretches of the plan's line, then, are theirs): adding up
    the rooms of the others takes a CTA several milliseconds."""
    p = _problem(F16, [1] * 10, [kv_len] * 10, 4, 2, d, 16)
    lens, starts = torch.zeros(n, dtype=torch.int32, device="cuda"), torch.zeros(n + 1, dtype=torch.int32, device="cuda")
    table = torch.full((n, p["table"].shape[1]), -1, dtype=torch.int32, device="cuda")
    lens[-10:], table[-10:] = kv_len, p["table"]
    starts[-10:] = torch.arange(1, 11, dtype=torch.int32)
    return p, (p["kc"], p["vc"], table, lens, starts)


def _run_out(mmq, p, args, d):  # noqa: F811
    """A call whose waits run out, between guard rows; then the same one with time."""
    out, lse = torch.full((30, 4, d), 7.0, dtype=F16, device="cuda"), torch.full((30, 4), 7.0, device="cuda")
    mmq.mmq_paged_attention(p["q"], *args, out=out[10:20], lse=lse[10:20])
    assert mmq.mmq_last_device_error() == mmq.mmq.MMQ_ERR_DEVICE_TIMEOUT
    for guard in (out[:10], out[20:], lse[:10], lse[20:]):
        assert (guard == 7).all()
    assert mmq.mmq_last_device_error() == 0
    mmq.mmq_set_wait_timeout_ns(2 * 10 ** 9)
    mmq.mmq_paged_attention(p["q"], *args, out=out[10:20], lse=lse[10:20])
    _check_rows(p, out[10:20], lse[10:20], 1 / math.sqrt(d), True, 0)


@pytest.mark.parametrize("d", [64, 128])
def test_waits_that_run_out_without_pieces(mmq, short_waits, d):  # noqa: F811
    """A table too narrow for units to be cut: no partial results and no join, only the kernel's own way out."""
    p, args = _late_problem(3 * 10 ** 6, 250, d)
    assert args[2].shape[1] * 16 > 256
    _run_out(mmq, p, (args[0], args[1], args[2][:, :16], *args[3:]), d)


@pytest.mark.parametrize("d", [64, 128])
def test_waits_that_run_out_with_pieces(mmq, short_waits, d):  # noqa: F811
    """Long keys, so that units are cut and a second kernel joins them: it may use nothing that no CTA wrote, whatever the
    scratch holds from a larger call before."""
    big = _problem(F16, [300, 200], [4000, 3000], 28, 4, d, 16)
    for _ in range(2):
        mmq.mmq_set_wait_timeout_ns(2 * 10 ** 9)
        mmq.mmq_paged_attention(big["q"], big["kc"], big["vc"], big["table"], big["seq_lens"], big["q_start"])
        mmq.mmq_set_wait_timeout_ns(1)
        p, args = _late_problem(3 * 10 ** 6, 3000, d)
        _run_out(mmq, p, args, d)


@pytest.mark.parametrize("d", [64, 128])
def test_every_replay_of_a_captured_call_tells_of_its_waits(mmq, short_waits, d):  # noqa: F811
    """A captured call that gave up once is not taken for one that has given up when it is replayed."""
    p, args = _late_problem(3 * 10 ** 6, 3000, d)
    out = torch.full((10, 4, d), 7.0, dtype=F16, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mmq.mmq_paged_attention(p["q"], *args, out=out)
    for _ in range(3):
        graph.replay()
        assert mmq.mmq_last_device_error() == mmq.mmq.MMQ_ERR_DEVICE_TIMEOUT
        assert mmq.mmq_last_device_error() == 0


# ---------------------------------------------------------------- page tables
def _tables_problem(n, seed=0):
    g = torch.Generator().manual_seed(seed)
    cached = torch.randint(0, 400, (n,), generator=g)
    new = torch.randint(0, 9, (n,), generator=g)
    held = (cached + 15) // 16
    width = int(((cached + new + 15) // 16).max()) + 1
    need = int(((cached + new + 15) // 16 - held).sum())
    order = torch.randperm(int(held.sum()) + need + 5, generator=g).int()
    table = torch.full((n, width), -1, dtype=torch.int32)
    at = 0
    for b in range(n):
        table[b, :held[b]] = order[at:at + held[b]]
        at += int(held[b])
    return [x.int().cuda() for x in (cached, new, held, table, order[at:])], int(new.sum()) + 3


@pytest.mark.parametrize("n", [1, 7, 900])
def test_page_tables_into_buffers(mmq, n):  # noqa: F811
    (cached, new, held, table, free), room = _tables_problem(n)
    other = table.clone()
    want = mmq.mmq_page_tables(cached, new, held, table, free, 16, room)
    buffers = [torch.full_like(x, 77) for x in want]
    for out in (tuple(buffers), mmq.PageTables(*buffers)):
        got = mmq.mmq_page_tables(cached, new, held, other, free, 16, room, out=out)
        assert all(x is y for x, y in zip(got, buffers))
        assert all(torch.equal(x, y) for x, y in zip(got, want)) and torch.equal(other, table)
    # buffers of other shapes or types, and buffers that are the call's inputs or one another's
    for i, x in enumerate(buffers):
        for bad in (x[:-1], x.float()):
            with pytest.raises(ValueError):
                mmq.mmq_page_tables(cached, new, held, other, free, 16, room, out=tuple(buffers[:i] + [bad] + buffers[i + 1:]))
    q_start, lens, blocks, slots, positions, taken = buffers
    for out in ((q_start, lens, held, slots, positions, taken), (q_start, cached, blocks, slots, positions, taken),
                (q_start, new, blocks, slots, positions, taken), (q_start, lens, lens, slots, positions, taken),
                (q_start, lens, q_start[1:], slots, positions, taken)):
        before = [x.clone() for x in (cached, new, held, other)]
        with pytest.raises(mmq.MMQError) as e:
            mmq.mmq_page_tables(cached, new, held, other, free, 16, room, out=out)
        assert e.value.code == -1
        assert all(torch.equal(x, y) for x, y in zip(before, (cached, new, held, other)))


def test_steps_that_hand_their_buffers_on(mmq):  # noqa: F811
    """A captured step with two sets of buffers that take turns, on lengths that stay on the device."""
    (cached, new, held, table, free), room = _tables_problem(40, seed=4)
    table = torch.cat([table, torch.full_like(table, -1)], 1)
    again, lens, blocks = table.clone(), cached.clone(), held.clone()
    sets = [tuple(torch.empty_like(x) for x in mmq.mmq_page_tables(cached, new, held, table.clone(), free, 16, room)) for _ in range(2)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mmq.mmq_page_tables(cached, new, held, table, free, 16, room, out=sets[0])
        mmq.mmq_page_tables(sets[0][1], new, sets[0][2], table, free, 16, room, out=sets[1])
    graph.replay()
    for got in sets:
        want = mmq.mmq_page_tables(lens, new, blocks, again, free, 16, room)
        assert all(torch.equal(x, y) for x, y in zip(got, want))
        lens, blocks = want.seq_lens, want.n_blocks
    assert torch.equal(table, again)


def test_page_tables_of_the_most_token_rows(mmq):  # noqa: F811
    """2^31 - 1 rows: the CTAs' threads together are 2^31."""
    room = 2 ** 31 - 1
    table = torch.full((3, 9), 77, dtype=torch.int32, device="cuda")
    table[:, 0] = _i32([5, 6, 7])
    free = _i32(list(range(20, 40)))
    t = mmq.mmq_page_tables(_i32([4, 0, 9]), _i32([9, 40, 0]), _i32([1, 1, 1]), table, free, 16, room)
    assert t.q_start.tolist() == [0, 9, 49, 49] and t.taken.tolist() == [2, 0] and t.n_blocks.tolist() == [1, 3, 1]
    assert table.tolist() == [[5] + [77] * 8, [6, 20, 21] + [77] * 6, [7] + [77] * 8]
    want = [5 * 16 + 4 + i for i in range(9)] + [(6, 20, 21)[i // 16] * 16 + i % 16 for i in range(40)]
    assert t.slots[:49].tolist() == want and t.positions[:49].tolist() == list(range(4, 13)) + list(range(40))
    for x in (t.slots, t.positions):
        for part in x[49:].split(2 ** 28):
            assert int(part.max()) == -1 and int(part.min()) == -1


# ---------------------------------------------------------------- the binding
def test_a_cache_without_heads_is_refused(mmq):  # noqa: F811
    p = _problem(F16, [2], [40], 4, 2, 64, 16)
    none = p["kc"][:, :, :0]
    with pytest.raises(mmq.MMQError) as e:
        mmq.mmq_paged_attention(p["q"], none, none, p["table"], p["seq_lens"], p["q_start"])
    assert e.value.code == -1
    with pytest.raises(mmq.MMQError) as e:
        mmq.mmq_kv_write(p["q"][:, :0], p["q"][:, :0], none, none, torch.zeros(2, dtype=torch.int64, device="cuda"))
    assert e.value.code == -1


def test_an_argument_without_a_truth_value_is_an_error(mmq):  # noqa: F811
    p = _problem(F16, [2], [40], 4, 2, 64, 16)
    out = torch.full_like(p["q"], 7.0)
    with pytest.raises(RuntimeError, match="ambiguous"):
        mmq.mmq_paged_attention(p["q"], p["kc"], p["vc"], p["table"], p["seq_lens"], p["q_start"], causal=torch.ones(2), out=out)
    assert (out == 7).all()


@pytest.mark.parametrize("d,page", [(64, 16), (128, 16), (128, 5)])
def test_row_starts_that_descend_are_reported(mmq, d, page):  # noqa: F811
    """Rows of two requests: what comes out for them is not said, but it is reported, and the rows of others stay."""
    p = _problem(F16, [4, 3, 2], [40, 30, 300], 4, 2, d, page)
    guard = torch.full((12, 4, d), 7.0, dtype=F16, device="cuda")
    for starts in ([0, 4, 2, 9], [0, 4, -3, 7], [0, 9, 4, 7], [2 ** 31 - 1, 0, 2, 9]):
        mmq.mmq_paged_attention(p["q"], p["kc"], p["vc"], p["table"], p["seq_lens"], _i32(starts), out=guard[:9])
        assert mmq.mmq_last_device_error() == mmq.MMQ_ERR_DEVICE_INDEX
        assert (guard[9:] == 7).all()
    mmq.mmq_paged_attention(p["q"], p["kc"], p["vc"], p["table"], p["seq_lens"], p["q_start"], out=guard[:9])
    assert mmq.mmq_last_device_error() == 0
