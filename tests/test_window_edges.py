"""Windowed attention and the 4-bit cache where calls and kernels meet: repeated launches, rows that
are not finite, streams, workspaces, limits.  Helpers and tolerances are those of test_window.py."""
import contextlib
import math

import pytest
import torch

from adaptive_top_sparse_b200 import twl
from test_window import ALL, D, PAGE, _attend, _check, _deal, _rand, _rows, _seen, _unquantise


@pytest.mark.gpu
@pytest.mark.parametrize("hq,hkv", [(8, 8), (8, 1)])
@pytest.mark.parametrize("sinks,window", [(0, ALL), (4, 130)])
def test_chunks_repeat_bit_for_bit(hq, hkv, sinks, window):
    """Units of one and two query tiles and of one to many key tiles, several to a run and some cut
    by runs: every launch gives the same bits, and what the definition gives."""
    from adaptive_top_sparse_b200.layer import DecodeLayer
    lens = [40, 128, 129, 700, 5000] + [90 + 37 * i for i in range(40)]
    qn = [40, 1, 129, 300, 260] + [1 + (53 * i) % (90 + 37 * i) for i in range(40)]
    table, n, pages = _deal(lens, 4)
    k, v = _rand(1, pages, hkv, PAGE, D), _rand(2, pages, hkv, PAGE, D)
    start = torch.tensor([0] + qn).cumsum(0).int()
    q = _rand(3, int(start[-1]), hq, D, scale=4.0)
    layer = DecodeLayer(k, v, table, n, hq, hkv)
    first = layer.window_prefill(q, start.cuda(), sinks, window)
    for _ in range(10):
        again = layer.window_prefill(q, start.cuda(), sinks, window)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    for b, m in enumerate(lens):
        rows = slice(int(start[b]), int(start[b + 1]))
        t = torch.arange(m - qn[b], m, device="cuda")
        want, wlse, big = _attend(q[rows].double(), _rows(k, table, b, m).double(),
                                  _rows(v, table, b, m).double(), _seen(t, m, sinks, window))
        _check(first[0][rows], first[1][rows], want, wlse, 6.0, big, True)
    assert layer.status() == (0, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("bad", ["nan", "inf", "-inf"])
@pytest.mark.parametrize("where", [160, 300, 520])    # a tile all see, one at the edge, the last one
@pytest.mark.parametrize("qn", [150, 5])              # two query tiles, one
@pytest.mark.parametrize("copies", [1, 50])           # units cut by runs, and whole ones
def test_a_score_that_is_not_finite_counts_at_every_key(bad, where, qn, copies):
    """A K row with a NaN, or with an infinity that makes a score of +inf, at eight keys in a row: no
    query that sees it gets a finite o or lse, the others are exact.  A score of -inf has weight 0."""
    from adaptive_top_sparse_b200.layer import DecodeLayer
    n, hq, hkv, sinks, window = 600, 4, 2, 0, 300
    table, lens, pages = _deal([n], 5)
    k, v = _rand(1, pages, hkv, PAGE, D), _rand(2, pages, hkv, PAGE, D)
    q = _rand(3, qn, hq, D)
    q[..., 3] = -1.0 if bad == "-inf" else 1.0
    start = torch.arange(copies + 1, dtype=torch.int32, device="cuda") * qn
    t = torch.arange(n - qn, n, device="cuda")
    seen = _seen(t, n, sinks, window)
    group = torch.arange(hq, device="cuda") < hq // hkv
    for key in range(where, where + 8):
        kk = k.clone()
        kk[table[0, key // PAGE], 0, key % PAGE, 3] = math.nan if bad == "nan" else math.inf
        # sequences that share all their pages
        layer = DecodeLayer(kk, v, table.repeat(copies, 1), lens.repeat(copies), hq, hkv)
        os, lses = layer.window_prefill(q.repeat(copies, 1, 1), start, sinks, window)
        one, lse1 = layer.window_decode(q[-1:].repeat(copies, 1, 1), sinks, window)
        # what rows see without the planted one, and heads of the other kv-head with it
        keep = seen.clone()
        keep[:, key] = False
        rows = _rows(k, table, 0, n).double(), _rows(v, table, 0, n).double()
        without = _attend(q.double(), *rows, keep)
        whole = _attend(q.double(), *rows, seen)
        hit = seen[:, key, None] & group
        want = torch.where(hit[..., None], without[0], whole[0])
        wlse = torch.where(hit, without[1], whole[1])
        for c in range(copies):
            o, lse = os[c * qn:(c + 1) * qn], lses[c * qn:(c + 1) * qn]
            if bad != "-inf":
                assert not o[hit].isfinite().any() and not lse[hit].isfinite().any()
                assert not one[c][hit[-1]].isfinite().any()
                assert not lse1[c][hit[-1]].isfinite().any()
            near = torch.zeros_like(hit) if bad == "-inf" else hit
            _check(o[~near], lse[~near], want[~near], wlse[~near], 6.0, whole[2], True)
            _check(one[c][~near[-1]], lse1[c][~near[-1]], want[-1][~near[-1]], wlse[-1][~near[-1]],
                   6.0, whole[2], False)
        assert layer.status() == (0, 0)


# ------------------------------------------------------------------ streams
class _FakeStream:
    def __init__(self, device=None):
        self.device, self.waits = device, 0

    def synchronize(self):
        self.waits += 1


@pytest.mark.parametrize("capturing", [False, True])
def test_a_workspace_is_zero_when_it_is_handed_out(monkeypatch, capturing):
    """Without a GPU: alloc_workspace waits for its zeros, except within a capture."""
    class Zeros:
        is_cuda, device = True, "a device"
    stream, order = _FakeStream("a device"), []
    monkeypatch.setattr(torch, "zeros", lambda *a, **k: order.append(stream.waits) or Zeros())
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device: stream)
    ws = twl.alloc_workspace(twl.TWL_OP_PAGES, "cuda", batch=1, max_pages=1, rows=1)
    assert isinstance(ws, Zeros) and order == [0]
    assert stream.waits == (0 if capturing else 1)


@contextlib.contextmanager
def _busy():
    """The current stream has about 0.2 s of work queued while the body runs."""
    torch.cuda.synchronize()
    torch.cuda._sleep(400_000_000)
    yield
    torch.cuda.synchronize()


@pytest.mark.gpu
def test_a_manager_made_on_a_busy_stream_serves_another():
    """A manager, its layer and a 4-bit layer are made while the current stream is busy; their first
    calls, on another stream, give what calls in order give."""
    from adaptive_top_sparse_b200.layer import DecodeLayer, Int4Layer
    side, got = torch.cuda.Stream(), []
    for busy in (False, True):
        table, n, pages = _deal([300, 45, 2000], 3, extra_pages=2, spare=8)
        k, v = _rand(1, pages, 2, PAGE, D), _rand(2, pages, 2, PAGE, D)
        kn, q = _rand(3, 3, 2, D), _rand(4, 3, 8, D)
        codes = (torch.arange(2 * pages * 2 * PAGE * 64, device="cuda") % 251).to(torch.uint8)
        codes = codes.view(2, pages, 2, PAGE, 64)
        sz = _rand(5, 2, pages, 2, PAGE, 2).abs()
        parent = torch.tensor([0, 0, 2], dtype=torch.int32, device="cuda")
        with _busy() if busy else contextlib.nullcontext():
            stream = side if busy else None
            four = Int4Layer(codes[0], sz[0], codes[1], sz[1], table.clone(), n.clone(), 8, 2)
            four.pages().remap(parent, parent, stream=stream)
            four.decode(q, kn, kn, 4, 100, stream=stream)
            side.synchronize()
            out = [x.clone() for x in (four.page_table, four.seq_lens, four.k, four.o, four.lse)]
        got.append(out)
    assert all(torch.equal(x, y) for x, y in zip(*got))


def test_chunks_make_their_outputs_and_workspace_on_the_launch_stream(monkeypatch):
    """Without a GPU, on meta tensors: what window_prefill allocates is allocated with the launch's
    stream current, and its first call is refused when that stream is being captured."""
    from adaptive_top_sparse_b200.layer import DecodeLayer
    now, seen = ["current"], []

    @contextlib.contextmanager
    def stream_context(stream):
        now.append(stream)
        try:
            yield
        finally:
            now.pop()
    empty, empty_like = torch.empty, torch.empty_like
    monkeypatch.setattr(torch.cuda, "stream", stream_context)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: now[-1])
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: now[-1] == "captured")
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: seen.append(("record", s)))
    monkeypatch.setattr(torch, "empty", lambda *a, **k: seen.append(("o", now[-1])) or empty(*a, **k))
    monkeypatch.setattr(torch, "empty_like",
                        lambda *a, **k: seen.append(("o", now[-1])) or empty_like(*a, **k))
    monkeypatch.setattr(twl, "alloc_workspace", lambda *a, **k: seen.append(("ws", now[-1])) or "ws")
    monkeypatch.setattr(twl, "twl_window_prefill",
                        lambda *a: seen.append(("launch", a[-1], a[-2], now[-1])))
    q = empty((5, 8, 128), dtype=torch.float16, device="meta")
    start = empty((4,), dtype=torch.int32, device="meta")
    out = (empty_like(q), empty((5, 8), dtype=torch.float32, device="meta"))
    layer = DecodeLayer.__new__(DecodeLayer)
    layer.k, layer.kv = empty((4, 2, 16, 128), dtype=torch.float16, device="meta"), None
    layer.batch, layer.num_q_heads, layer.num_kv_heads, layer.ws_prefill = 3, 8, 2, None
    with pytest.raises(RuntimeError):
        layer.window_prefill(q, start, out=out, stream="captured")
    assert seen == [] and layer.ws_prefill is None
    layer.window_prefill(q, start, stream="side")
    assert sorted(seen[:2]) == [("o", "side")] * 2 and ("ws", "side") in seen
    assert seen.count(("record", "current")) == 2
    assert seen[-1] == ("launch", "side", "ws", "current")
    seen.clear()
    layer.window_prefill(q, start, out=out, stream="captured")
    assert seen == [("launch", "captured", "ws", "current")]
    seen.clear()
    layer.window_prefill(q, start)
    assert seen == [("o", "current")] * 2 + [("launch", None, "ws", "current")]


@pytest.mark.gpu
@pytest.mark.parametrize("raw", [False, True])        # the stream, or its handle
def test_first_chunks_on_another_stream_than_the_busy_one(raw):
    from adaptive_top_sparse_b200.layer import DecodeLayer
    lens, qn = [3000, 700, 40], [900, 300, 40]
    table, n, pages = _deal(lens, 3)
    k, v = _rand(1, pages, 2, PAGE, D), _rand(2, pages, 2, PAGE, D)
    start = torch.tensor([0] + qn).cumsum(0).int().cuda()
    q = _rand(3, sum(qn), 8, D)
    want = [x.clone() for x in DecodeLayer(k, v, table, n, 8, 2).window_prefill(q, start, 4, 500)]
    side = torch.cuda.Stream()
    layer = DecodeLayer(k, v, table, n, 8, 2)
    with _busy():
        got = layer.window_prefill(q, start, 4, 500, stream=side.cuda_stream if raw else side)
        side.synchronize()
        with torch.cuda.stream(side):
            assert all(torch.equal(x, y) for x, y in zip(want, got))
    assert all(torch.equal(x, y) for x, y in zip(want, got))
    assert layer.status() == (0, 0)


def test_a_4_bit_cache_is_filled_and_quantised_on_one_stream(monkeypatch):
    """Without a GPU, on meta tensors: from_fp16 fills its codes with the stream current that the
    quantiser runs on."""
    from adaptive_top_sparse_b200.layer import Int4Layer
    now, seen = ["current"], []

    @contextlib.contextmanager
    def stream_context(stream):
        now.append(stream)
        try:
            yield
        finally:
            now.pop()
    zeros = torch.zeros
    monkeypatch.setattr(torch.cuda, "stream", stream_context)
    monkeypatch.setattr(torch, "zeros", lambda *a, **k: seen.append(now[-1]) or zeros(*a, **k))
    monkeypatch.setattr(twl, "alloc_workspace", lambda *a, **k: seen.append(now[-1]))
    monkeypatch.setattr(twl, "twl_quantize_k", lambda *a: seen.append(a[-1]))
    k = torch.empty((4, 2, 16, 128), dtype=torch.float16, device="meta")
    table = torch.empty((3, 5), dtype=torch.int32, device="meta")
    Int4Layer.from_fp16(k, k, table, table[:, 0].clone(), 8, 2, stream="side")
    assert len(seen) == 9 and set(seen) == {"side"}      # K and V; o, lse and the workspace


@pytest.mark.gpu
def test_a_4_bit_cache_made_on_another_stream_than_the_busy_one():
    from adaptive_top_sparse_b200.layer import Int4Layer
    table, n, pages = _deal([3000, 700, 40], 3)
    k, v, q = _rand(1, pages, 2, PAGE, D), _rand(2, pages, 2, PAGE, D), _rand(3, 3, 8, D)
    ref = Int4Layer.from_fp16(k, v, table, n, 8, 2)
    want = [x.clone() for x in (*ref.decode(q), ref.k, ref.k_sz, ref.v, ref.v_sz)]
    side = torch.cuda.Stream()
    with _busy():
        four = Int4Layer.from_fp16(k, v, table, n, 8, 2, stream=side)
        o, lse = four.decode(q, stream=side)
        side.synchronize()
        with torch.cuda.stream(side):
            got = [x.clone() for x in (o, lse, four.k, four.k_sz, four.v, four.v_sz)]
    assert all(torch.equal(x, y) for x, y in zip(want, got))
    assert all(torch.equal(x, y) for x, y in
               zip(want, (four.o, four.lse, four.k, four.k_sz, four.v, four.v_sz)))


def test_status_reads_behind_the_stream_it_is_given(monkeypatch):
    from adaptive_top_sparse_b200.layer import DecodeLayer, Int4Layer, PageManager
    seen = []
    monkeypatch.setattr(twl, "twl_device_status",
                        lambda ws, clear, stream: seen.append((ws, clear, stream)) or (0, 0))
    for cls, spaces in ((DecodeLayer, ("ws", "ws_window", "ws_prefill")), (Int4Layer, ("ws",)),
                        (PageManager, ("ws",))):
        one = cls.__new__(cls)
        one.device = torch.device("meta")
        for name in spaces:
            setattr(one, name, name)
        assert one.status(True, stream="side") == (0, 0)
        assert one.status() == (0, 0)
        assert seen == [(x, c, s) for c, s in ((True, "side"), (False, None)) for x in spaces]
        seen.clear()


@pytest.mark.gpu
def test_status_of_calls_on_a_busy_stream():
    """A bad page met behind 0.2 s of other work on a side stream shows in the status read there."""
    from adaptive_top_sparse_b200.layer import DecodeLayer, Int4Layer, PageManager
    table, n, pages = _deal([300, 45], 3)
    k, v, q = _rand(1, pages, 2, PAGE, D), _rand(2, pages, 2, PAGE, D), _rand(3, 2, 8, D)
    four = Int4Layer.from_fp16(k, v, table, n, 8, 2)
    layer, manager = DecodeLayer(k, v, table.clone(), n, 8, 2), PageManager([k, v], table, n)
    bad = torch.tensor([0, 2], dtype=torch.int32, device="cuda")
    table[0, 3], layer.page_table[0, 3] = pages, -1
    side = torch.cuda.Stream()
    for what, call in ((layer, lambda: layer.window_decode(q, stream=side)),
                       (four, lambda: four.decode(q, stream=side)),
                       (manager, lambda: manager.remap(bad, stream=side))):
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(400_000_000)
        call()
        assert what.status(clear=True, stream=side) == (twl.TWL_ERR_BAD_INDEX, twl.TWL_FLAG_BAD_INDEX)
        assert what.status(stream=side) == (0, 0)


# ------------------------------------------------------------------ workspaces
@pytest.mark.gpu
def test_one_workspace_serves_attention_of_every_shape():
    """One token, chunks and a 4-bit cache, groups of 8, 1 and 4 heads and batches of 1 to 40 in turn
    through one workspace give the bits that each gives in its own."""
    from adaptive_top_sparse_b200.layer import DecodeLayer, Int4Layer
    calls = []
    for i, (hq, hkv, lens, qn) in enumerate([
            (16, 2, [5000], [60]), (4, 4, [3000, 900], [500, 10]),
            (8, 2, [100 + 90 * i for i in range(40)], [1 + 3 * i for i in range(40)]),
            (8, 1, [9000, 17], [300, 17]), (1, 1, [20000], [1])]):
        table, n, pages = _deal(lens, i)
        k, v = _rand(1, pages, hkv, PAGE, D), _rand(2, pages, hkv, PAGE, D)
        layer, four = DecodeLayer(k, v, table, n, hq, hkv), Int4Layer.from_fp16(k, v, table, n, hq, hkv)
        q, qp = _rand(3, len(lens), hq, D), _rand(4, sum(qn), hq, D)
        start = torch.tensor([0] + qn).cumsum(0).int().cuda()
        for call in (lambda l=layer, q=q: l.window_decode(q, 4, 10000),
                     lambda l=layer, q=qp, s=start: l.window_prefill(q, s, 4, 3000),
                     lambda l=four, q=q: l.decode(q)):
            calls.append((call, [x.clone() for x in call()], layer, four))
    shared = twl.alloc_workspace(twl.TWL_OP_WINDOW_PREFILL, "cuda", batch=1, num_q_heads=1,
                                 num_kv_heads=1)
    for _, _, layer, four in calls:
        layer.ws_window = layer.ws_prefill = four.ws = shared
    for order in (calls, calls[::-1], calls):
        for call, want, layer, four in order:
            for x in (layer.o, layer.lse, four.o, four.lse):
                x.fill_(math.nan)
            assert all(torch.equal(x, y) for x, y in zip(call(), want))
    assert twl.twl_device_status(shared) == (0, 0)


@pytest.mark.gpu
def test_one_workspace_serves_pools_and_tables_of_every_size():
    """Page steps and compactions of small and large pools and tables in turn through one workspace
    give what each gives in its own."""
    from adaptive_top_sparse_b200.layer import PageManager
    sides = []
    for lens, spare in (([40, 17], 6), ([4000, 30000], 60000), ([300] * 50, 900), ([5], 30)):
        for shared in (False, True):
            table, n, pages = _deal(lens, 7, extra_pages=2, spare=spare)
            pool = torch.arange(pages * 4, dtype=torch.int32, device="cuda").view(pages, 4)
            sides.append((shared, PageManager([pool], table, n),
                          torch.arange(len(lens), dtype=torch.int32, device="cuda") // 2))
    ws = max((m.ws for _, m, _ in sides), key=lambda t: t.nbytes)
    ws = torch.zeros_like(ws)
    for shared, m, _ in sides:
        if shared:
            m.ws = ws
    for step in range(4):
        for part in (False, True):
            for shared, m, parent in sides[::-1] if step % 2 else sides:
                if shared == part:
                    m.remap(parent, parent, 4, 2000)
                    m.compact()
        for (_, a, _), (_, b, _) in zip(sides[::2], sides[1::2]):
            assert torch.equal(a.page_table, b.page_table) and torch.equal(a.pools[0], b.pools[0])
            assert torch.equal(a.seq_lens, b.seq_lens) and int(a.num_used) == int(b.num_used)
            assert a.status() == (0, 0) and b.status() == (0, 0)


def test_workspaces_keep_their_zeroed_words_in_one_place():
    """The words that a launch leaves zero for the next lie before everything whose size depends on
    the call's: 4096 arrival counters, and a bit for each of 2^23 pages."""
    wb = twl.twl_workspace_bytes
    for op in (twl.TWL_OP_WINDOW_DECODE, twl.TWL_OP_INT4_DECODE, twl.TWL_OP_WINDOW_PREFILL):
        assert wb(op, 1, 1, 1) == wb(op, 64, 8, 8) >= 256 + 4 * 4097
    assert wb(twl.TWL_OP_PAGES, 1, 0, 0, 1, 0, 1) >= 256 + (1 << 23) // 8
    assert wb(twl.TWL_OP_PAGES, 4, 0, 0, 64, 0, 16) == wb(twl.TWL_OP_PAGES, 4, 0, 0, 64, 0, 1 << 23)


# ------------------------------------------------------------------ waits that give up
@pytest.mark.gpu
@pytest.mark.parametrize("hq,hkv,lens,qn", [(8, 1, [9000], [2000]), (4, 4, [20000, 300], [5, 300]),
                                            (8, 8, [400] * 30, [150] * 30)])
def test_a_chunk_launch_that_gives_up_leaves_a_valid_workspace(hq, hkv, lens, qn):
    """Through the test hook every second CTA of a chunk launch waits for what never happens: the
    launch returns with the timeout flag, and the next ones, of the same chunks and of others, are
    exact, bit for bit those of a layer that never gave up."""
    from adaptive_top_sparse_b200.layer import DecodeLayer
    table, n, pages = _deal(lens, 3)
    k, v = _rand(1, pages, hkv, PAGE, D), _rand(2, pages, hkv, PAGE, D)
    start = torch.tensor([0] + qn).cumsum(0).int().cuda()
    q = _rand(3, sum(qn), hq, D)
    ref = DecodeLayer(k, v, table, n, hq, hkv)
    want = [[x.clone() for x in ref.window_prefill(q, start, 4, w)] for w in (ALL, 700)]
    layer = DecodeLayer(k, v, table, n, hq, hkv)
    out = tuple(torch.empty_like(x) for x in want[0])
    layer.window_prefill(q, start, 4, ALL, out)
    for _ in range(2):
        try:
            twl.twl_test_set_waits(32, True)
            layer.window_prefill(q, start, 4, ALL, out)
            torch.cuda.synchronize()
        finally:
            twl.twl_test_set_waits(0, False)
        assert layer.status(clear=True) == (twl.TWL_ERR_TIMEOUT, twl.TWL_FLAG_TIMEOUT)
        for i in (0, 1, 0):
            for x in out:
                x.fill_(math.nan)
            layer.window_prefill(q, start, 4, (ALL, 700)[i], out)
            assert all(torch.equal(x, y) for x, y in zip(want[i], out))
        assert layer.status() == (0, 0)


@pytest.mark.gpu
def test_a_page_call_that_gives_up_changes_nothing_and_leaves_a_valid_workspace():
    """Through the test hook every CTA of a page call waits for one more than there are: the call
    returns with the timeout flag, nothing has changed, and the next calls are exact."""
    from adaptive_top_sparse_b200.layer import PageManager
    sides = []
    for _ in range(2):
        table, n, pages = _deal([40, 17, 300], 4, extra_pages=2, spare=20)
        pool = torch.arange(pages * 4, dtype=torch.int32, device="cuda").view(pages, 4)
        sides.append((PageManager([pool], table, n), (table, n, pool)))
    (m, mine), (ref, theirs) = sides
    parent = torch.tensor([0, 0, 2], dtype=torch.int32, device="cuda")
    for call, ref_call in ((lambda: m.remap(parent, parent), lambda: ref.remap(parent, parent)),
                           (m.compact, ref.compact)):
        before = [x.clone() for x in mine]
        try:
            twl.twl_test_set_waits(64, True)
            call()
            torch.cuda.synchronize()
        finally:
            twl.twl_test_set_waits(0, False)
        assert m.status(clear=True) == (twl.TWL_ERR_TIMEOUT, twl.TWL_FLAG_TIMEOUT)
        assert all(torch.equal(x, y) for x, y in zip(before, mine))
        call()
        ref_call()
        assert m.status() == (0, 0)
        assert all(torch.equal(x, y) for x, y in zip(mine, theirs))
    assert int(m.num_used) == int(ref.num_used) > 0


# ------------------------------------------------------------------ host threads
@pytest.mark.gpu
@pytest.mark.parametrize("call", ["decode", "int4", "remap", "compact"])
def test_host_threads_with_calls_of_different_sizes(call):
    """Two host threads, each with its own tensors, workspace and stream, one with the smallest
    shapes and one with large ones: every call launches, and they give what they give alone."""
    import threading
    from adaptive_top_sparse_b200.layer import DecodeLayer, Int4Layer, PageManager
    lib, jobs = twl._lib, []
    for batch in (1, 4000):
        table, n, pages = _deal([20] * batch, 3, extra_pages=1, spare=40000 if batch > 1 else 3)
        stream, same = torch.cuda.Stream(), torch.arange(batch, dtype=torch.int32, device="cuda")
        if call in ("decode", "int4"):
            k, v, q = _rand(1, pages, 1, PAGE, D), _rand(2, pages, 1, PAGE, D), _rand(3, batch, 1, D)
            layer = DecodeLayer(k, v, table, n, 1, 1) if call == "decode" else \
                Int4Layer.from_fp16(k, v, table, n, 1, 1)
            ws = layer.ws_window if call == "decode" else layer.ws
            kv, rest = layer.kv.c(), (0, ALL, 0.1, layer.o.data_ptr(), layer.lse.data_ptr(),
                                      ws.data_ptr(), ws.nbytes, stream.cuda_stream)
            fn, args = (lib.twl_window_decode, (q.data_ptr(), 1, kv)) if call == "decode" else \
                (lib.twl_int4_decode, (q.data_ptr(), 1, kv, None, None, 0))
            keep, result = (layer, k, v, q), (layer.o, layer.lse)
        else:
            manager = PageManager([torch.zeros((pages, 4), dtype=torch.int32, device="cuda")],
                                  table, n)
            out = torch.empty_like(table)
            pools, ws = twl._pools(manager.pools), manager.ws
            rest = (ws.data_ptr(), ws.nbytes, stream.cuda_stream)
            fn, args = (lib.twl_remap_pages, (pools, 1, table.data_ptr(), n.data_ptr(), batch,
                                              table.shape[1], pages, same.data_ptr(), None, 0, ALL)) \
                if call == "remap" else \
                (lib.twl_compact_pages, (pools, 1, table.data_ptr(), out.data_ptr(), batch,
                                         table.shape[1], pages, manager.num_used.data_ptr()))
            keep, result = (manager, out, pools), (table, n) if call == "remap" else (out,)
        assert fn(*args, *rest) == 0
        torch.cuda.synchronize()
        jobs.append((fn, args + rest, stream, keep, result, [x.clone() for x in result]))
    failed = []

    def loop(fn, args, stream):
        for i in range(4000):
            if fn(*args) != 0:
                failed.append(i)
            if i % 100 == 99:
                stream.synchronize()
    threads = [threading.Thread(target=loop, args=job[:3]) for job in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert failed == []
    for job in jobs:
        assert all(torch.equal(x, y) for x, y in zip(job[4], job[5]))


# ------------------------------------------------------------------ pools
def test_a_manager_refuses_pools_when_it_is_made():
    from adaptive_top_sparse_b200.layer import PageManager
    e = lambda *s, dt=torch.float16: torch.empty(s, dtype=dt, device="meta")
    table, lens = e(3, 5, dt=torch.int32), e(3, dt=torch.int32)
    for pool in (e(4, 3), e(4), e(4, 0), e(0, 8), e(4, 2, 17, dt=torch.uint8)):
        with pytest.raises(ValueError):
            PageManager([e(pool.shape[0], 8), pool], table, lens)
    m = PageManager.__new__(PageManager)
    m.device, m.num_phys_pages, m.pools = table.device, 4, []
    for pool in (None, e(5, 8), e(4, 3), e(4, 8, 2).transpose(1, 2), torch.zeros(4, 8)):
        with pytest.raises(ValueError):
            m.add(pool)
    assert m.pools == []


@pytest.mark.gpu
def test_a_manager_of_as_many_pools_as_layers_have():
    """300 pools step and compact as one pool whose page holds all of theirs does; a step that
    cannot be carried out changes none of them."""
    from adaptive_top_sparse_b200.layer import PageManager
    count, lens = 300, [40, 17, 0, 300]
    table, n, pages = _deal(lens, 4, extra_pages=2, spare=20)
    whole = torch.arange(pages * count * 4, dtype=torch.int32, device="cuda").view(pages, count, 4)
    pools = [whole[:, i].contiguous() for i in range(count)]
    one = PageManager([whole], table.clone(), n.clone())
    many = PageManager(pools, table, n)

    def same():
        return torch.equal(one.page_table, many.page_table) and torch.equal(one.seq_lens, many.seq_lens) \
            and torch.equal(whole, torch.stack(pools, 1)) and one.status() == many.status()
    side = torch.cuda.Stream()
    for parent, stream in (([0, 0, 0, 3], None), ([1, 1, 3, 0], side), ([0, 1, 2, -1], None)):
        reserve = torch.tensor([1, 16, 5, 40], dtype=torch.int32, device="cuda")
        parent = torch.tensor(parent, dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        for m in (one, many):
            m.remap(parent, reserve, 4, 1000, stream=stream)
        torch.cuda.synchronize()
        assert same() and one.status() == (0, 0)
    out = [torch.empty_like(table) for _ in range(2)]
    for m, x in ((one, out[0]), (many, out[1])):
        assert int(m.compact(x)) > 0
        m.page_table.copy_(x)
    assert same() and int(one.num_used) == int(many.num_used)
    many.page_table[0, 0] = one.page_table[0, 0] = 0 if int(table[0, 0]) else 1
    for m in (one, many):
        m.compact()
    assert same() and one.status() == (0, 0)
    before = whole.clone(), table.clone(), n.clone()
    reserve.fill_(PAGE * (pages + 1))
    for m in (one, many):
        m.remap(parent, reserve)
    assert many.status() == one.status() != (0, 0)
    assert same() and all(torch.equal(x, y) for x, y in zip(before, (whole, table, n)))


@pytest.mark.gpu
@pytest.mark.parametrize("manager_first", [False, True])
def test_centroids_follow_their_pages(manager_first):
    """After forks, frees and a compaction the two-level path reads what centroids built anew hold,
    whether its buffers were made before the manager or behind it."""
    from adaptive_top_sparse_b200.layer import DecodeLayer
    table, n, pages = _deal([300, 45, 70, 160], 3, extra_pages=2, spare=30)
    k, v = _rand(1, pages, 2, PAGE, D), _rand(2, pages, 2, PAGE, D)
    layer, q = DecodeLayer(k, v, table, n, 8, 2), _rand(3, 4, 8, D)
    if manager_first:
        layer.pages()
    dp = layer.double_p()
    layer.build_aux()
    dp.build_centroids()
    used = lambda: layer.page_table[layer.page_table >= 0].unique().long()
    for parent in ([0, 0, 2, 0], [1, 1, -1, 3]):
        layer.pages().remap(torch.tensor(parent, dtype=torch.int32, device="cuda"))
        layer.pages().compact()
        n.copy_(torch.where(n == 0, 1, n))             # the freed slot: one token, on no page
        o, lse = (x.clone() for x in dp.decode(q))
        kept = dp.centroids[used()].clone()
        dp.build_centroids()
        assert torch.equal(kept, dp.centroids[used()])
        o2, lse2 = dp.decode(q)
        live = [b for b, p in enumerate(parent) if p >= 0]
        assert torch.equal(o[live], o2[live]) and torch.equal(lse[live], lse2[live])
    assert layer.pages().status() == (0, 0)


# ------------------------------------------------------------------ limits
@pytest.mark.gpu
@pytest.mark.parametrize("size", [2.0 ** e for e in range(0, 16, 3)] + [30000.0, 60000.0])
def test_scores_up_to_the_largest_of_fp16_rows(size):
    """Rows of one repeated value, so that scores are +-128 size x: 2^4 up to 2^36 in log2 units, and
    next to one another at every distance.  One token, fp16 and in 4 bits (which hold such rows
    exactly), and chunks, units of one and two query tiles.

    Tolerances: scores are exact sums (128 equal products), their scaling rounds once (2^-24 of the
    score, on both sides of a difference), so a weight that is not 0 or 1 is off by at most
    2^-22 |score| in log2 units; such weights only count where scores lie within 40 of one another."""
    from adaptive_top_sparse_b200.layer import DecodeLayer, Int4Layer
    n, hq, hkv = 900, 4, 2
    table, lens, pages = _deal([n], 5)
    g = torch.Generator().manual_seed(int(size))
    steps = torch.randint(-8, 9, (pages, hkv, PAGE, 1), generator=g)
    k = (size * (1 + steps / 1024) * torch.sign(steps + 0.5)).expand(-1, -1, -1, D)
    k = k.contiguous().half().cuda()
    v = _rand(2, pages, hkv, PAGE, D)
    for qn in (300, 3):
        sign = torch.where(torch.arange(qn * hq) % 3 == 0, -1.0, 1.0).view(qn, hq, 1)
        q = (sign * size).expand(-1, -1, D).contiguous().half().cuda()
        start = torch.tensor([0, qn], dtype=torch.int32, device="cuda")
        layer = DecodeLayer(k, v, table, lens, hq, hkv)
        o, lse = layer.window_prefill(q, start, 0, 700)
        one, lse1 = layer.window_decode(q[-1:].contiguous(), 0, 700)
        t = torch.arange(n - qn, n, device="cuda")
        want, wlse, big = _attend(q.double(), _rows(k, table, 0, n).double(),
                                  _rows(v, table, 0, n).double(), _seen(t, n, 0, 700))
        # an error of e in the exponents moves o by at most e max|v| (weights sum to 1)
        off = min(2.0, 2.0 ** -22 * big * 1.5) if 128 * size * size / 1024 * 0.08 < 40 else 0.0
        assert (o.double() - want).abs().max().item() <= (3 * 2.0 ** -11 + off) * 6.0
        assert (one.double() - want[-1:]).abs().max().item() <= (2.0 ** -17 + off) * 6.0
        assert (lse.double() - wlse).abs().max().item() <= 2.0 ** -18 * (1 + big)
        assert (lse1.double() - wlse[-1:]).abs().max().item() <= 2.0 ** -18 * (1 + big)
        four = Int4Layer.from_fp16(k, v, table, lens, hq, hkv)
        one, lse1 = four.decode(q[-1:].contiguous(), window=700)
        vv = _unquantise(_rows(four.v, table, 0, n), _rows(four.v_sz, table, 0, n))
        want, wlse, big = _attend(q[-1:].double(), _rows(k, table, 0, n).double(), vv,
                                  _seen(t[-1:], n, 0, 700))
        assert (one.double() - want).abs().max().item() <= (2.0 ** -17 + off) * 6.0
        assert (lse1.double() - wlse).abs().max().item() <= 2.0 ** -18 * (1 + big)

@pytest.mark.parametrize("scale", [2.0 ** 48 * (1 + 2.0 ** -20), 1e30, 3e38, -1.0, 0.0])
def test_scales_out_of_range_are_refused(scale):
    """Above 2^48 a score of fp16 or 4-bit rows could pass the kernels' lowest maximum (-1e30):
    |q.k| < 2^43 for rows of up to 16 x 65504, so scores in log2 units stay below 2^92."""
    from test_window import _decode, _decode4, _prefill
    for call in (_decode, _prefill, _decode4):
        assert call(scale=scale) == twl.TWL_ERR_INVALID_ARG


@pytest.mark.gpu
def test_the_largest_scale():
    """Scores of up to 2^48 |q.k|: one key wins, whatever the sign of its score."""
    from adaptive_top_sparse_b200.layer import DecodeLayer, Int4Layer
    table, n, pages = _deal([1, 300], 3)
    k, v, q = _rand(1, pages, 2, PAGE, D), _rand(2, pages, 2, PAGE, D), _rand(3, 2, 8, D)
    first = k[table[0, 0], :, 0].float()                       # the only key of sequence 0
    q[0] = (-q[0].float() * (q[0].float().view(2, 4, D) @ first[..., None]).sign().view(8, 1)).half()
    scale, start = 2.0 ** 48, torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    layer, four = DecodeLayer(k, v, table, n, 8, 2), Int4Layer.from_fp16(k, v, table, n, 8, 2)
    half, lse = torch.empty_like(q), torch.empty((2, 8), device="cuda")
    layer.window_prefill(q, start, out=(half, lse))
    twl.twl_window_decode(q, 8, layer.kv, 0, ALL, scale, layer.o, layer.lse, layer.ws_window)
    twl.twl_int4_decode(q, 8, four.kv, None, None, False, 0, ALL, scale, four.o, four.lse, four.ws)
    twl.twl_window_prefill(q, start, 2, 8, layer.kv, 0, ALL, scale, half, lse, layer.ws_prefill)
    for b, m in enumerate((1, 300)):
        fp16 = [_rows(x, table, b, m).double() for x in (k, v)]
        int4 = [_unquantise(_rows(c, table, b, m), _rows(z, table, b, m))
                for c, z in ((four.k, four.k_sz), (four.v, four.v_sz))]
        for o, l, (kk, vv), u in ((layer.o, layer.lse, fp16, 2.0 ** -17), (half, lse, fp16, 3 * 2.0 ** -11),
                                  (four.o, four.lse, int4, 2.0 ** -17)):
            s = torch.einsum("hd,thd->ht", q[b].double(), kk.repeat_interleave(4, 1)) * scale
            assert (l[b].double() - s.amax(1)).abs().max() <= 2.0 ** -18 * s.abs().max()
            best = vv.repeat_interleave(4, 1)[s.argmax(1), torch.arange(8, device="cuda")]
            assert (o[b].double() - best).abs().max().item() <= u * 6.0
            assert b == 1 or bool((s < 0).all())
