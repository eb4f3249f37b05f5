"""The page-table step and the compaction against a restatement in plain Python, and the windowed
calls, the 4-bit cache and the page calls used together as a decoding loop uses them."""
import math
import random

import pytest
import torch

from adaptive_top_sparse_b200 import twl

pytestmark = pytest.mark.gpu

PAGE, ALL = 16, 2 ** 31 - 1


def remap_plain(table, lens, parent, reserve, sinks, window, pages):
    """(new table, new lengths, [(from, to)] copies) or None when it cannot be carried out."""
    batch, width = len(table), len(table[0])
    keeper = {}
    for b, p in enumerate(parent):
        if p >= 0:
            keeper[p] = p if parent[p] == p else min(keeper.get(p, b), b)
    new, n_new, wants, copies = [], [], [], []
    for b, p in enumerate(parent):
        n = lens[p] if p >= 0 else 0
        need = -(-(n + reserve[b]) // PAGE)
        if need > width:
            return None
        row = [-1] * width
        for j in range(need):
            full = PAGE * (j + 1) <= n
            if full:                     # seen by the query at n: a sink, or in its window
                if any(t < sinks or t > n - window for t in range(PAGE * j, PAGE * j + PAGE)):
                    row[j] = table[p][j]
                continue
            held = PAGE * j < n
            if held and keeper[p] != b:
                if table[p][j] >= 0:
                    copies.append((table[p][j], b, j))
            elif held or p == b:
                row[j] = table[p][j]
            if row[j] < 0:
                row[j] = -1
                wants.append((b, j))
        new.append(row)
        n_new.append(n)
    taken = {x for row in new for x in row if x >= 0}
    free = [x for x in range(pages) if x not in taken]
    if len(free) < len(wants):
        return None
    for (b, j), x in zip(wants, free):
        new[b][j] = x
    return new, n_new, [(f, new[b][j]) for f, b, j in copies]


def make(seed, batch, longest, pages, pools=((4, PAGE, 8), (3, 16)), extra=4):
    """Random sequences over a pool; pools: (shape behind the page axis) of int32 tensors."""
    r = random.Random(seed)
    lens = [r.choice([0, 1, 15, 16, 17, r.randint(1, max(1, longest))]) for _ in range(batch)]
    need = [-(-n // PAGE) for n in lens]
    assert sum(need) <= pages
    ids = list(range(pages))
    r.shuffle(ids)
    width = max(need) + extra
    table = []
    for m in need:
        spare = r.randint(0, 1) if len(ids) > sum(need) + batch else 0
        table.append([ids.pop() for _ in range(m + spare)] + [-1] * (width - m - spare))
    g = torch.Generator(device="cuda").manual_seed(seed)
    made = [torch.randint(-2 ** 31, 2 ** 31 - 1, (pages, *s), generator=g, device="cuda").int()
            for s in pools]
    return (torch.tensor(table, dtype=torch.int32, device="cuda"),
            torch.tensor(lens, dtype=torch.int32, device="cuda"), made)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("batch,longest,pages", [(1, 40, 8), (2, 100, 40), (9, 700, 900),
                                                 (70, 90, 600), (700, 300, 20000), (3, 30000, 6000)])
@pytest.mark.parametrize("sinks,window", [(0, ALL), (4, 32), (17, 1), (0, 16), (64, 100)])
def test_remap(batch, longest, pages, sinks, window):
    from adaptive_top_sparse_b200.layer import PageManager
    table, lens, pools = make(batch + window % 31, batch, longest, pages)
    m = PageManager(pools, table, lens)
    r = random.Random(batch)
    for step in range(3):
        parent = [r.choice([b, b, r.randrange(batch), -1]) for b in range(batch)]
        reserve = [r.choice([0, 1, 16, 40]) for _ in range(batch)]
        reserve = reserve if step else None
        want = remap_plain(table.tolist(), lens.tolist(), parent, reserve or [0] * batch, sinks,
                           window, pages)
        before = [t.clone() for t in (table, lens, *pools)]
        m.remap(i32(parent), i32(reserve) if reserve else None, sinks, window)
        if want is None:
            assert m.status(clear=True)[0] in (twl.TWL_ERR_NO_PAGES, twl.TWL_ERR_BAD_INDEX)
            assert all(torch.equal(x, y) for x, y in zip(before, (table, lens, *pools)))
            continue
        assert m.status() == (twl.TWL_OK, 0)
        assert table.tolist() == want[0] and lens.tolist() == want[1]
        for old, pool in zip(before[2:], pools):
            for src, dst in want[2]:
                old[dst] = old[src]
            assert torch.equal(pool, old)


def test_remap_all_fork_one_and_pool_sizes():
    """Every slot becomes a fork of one (its own slot among them, or freed), with pools whose page
    is 16 bytes, a piece and a bit, and many pools at once."""
    from adaptive_top_sparse_b200.layer import PageManager
    for own in (True, False):
        pools = [(4,), (1024,), (1028,), (2051, 4)] + [(8,)] * 100
        table, lens, pools = make(5, 6, 0, 60, pools)
        lens.copy_(i32([37, 20, 0, 5, 16, 1]))
        table.fill_(-1)
        table[0, :3], table[1, :2], table[3, 0] = i32([9, 3, 50]), i32([0, 1]), 2
        m = PageManager(pools, table, lens)
        parent = [0 if own else -1] + [0] * 5
        want = remap_plain(table.tolist(), lens.tolist(), parent, [0] * 6, 0, ALL, 60)
        before = [p.clone() for p in pools]
        m.remap(i32(parent))
        assert table.tolist() == want[0] and lens.tolist() == want[1]
        assert len(want[2]) == (5 if own else 4)
        for old, pool in zip(before, pools):
            for src, dst in want[2]:
                old[dst] = old[src]
            assert torch.equal(pool, old)


def test_remap_changes_nothing_when_it_cannot_be_carried_out():
    from adaptive_top_sparse_b200.layer import PageManager
    table, lens, pools = make(7, 4, 0, 12, extra=2)
    lens.copy_(i32([20, 33, 16, 0]))
    table.fill_(-1)
    table[0, :2], table[1, :3], table[2, 0] = i32([1, 2]), i32([3, 4, 5]), 6
    table = torch.nn.functional.pad(table, (0, 2), value=-1).contiguous()
    m = PageManager(pools, table, lens)
    same = [0, 1, 2, 3]
    bad = [([0, 1, 2, 4], [0] * 4, twl.TWL_ERR_BAD_INDEX),        # a parent outside the batch
           ([0, 1, 2, -2], [0] * 4, twl.TWL_ERR_BAD_INDEX),
           (same, [0, 0, -1, 0], twl.TWL_ERR_BAD_INDEX),          # a negative reserve
           (same, [0, 0, 0, PAGE * table.shape[1] + 1], twl.TWL_ERR_BAD_INDEX),
           (same, [2 ** 31 - 1] * 4, twl.TWL_ERR_BAD_INDEX),
           ([1, 1, 1, 1], [0, 0, 0, 0], twl.TWL_OK),
           ]
    for parent, reserve, status in bad:
        before = [t.clone() for t in (table, lens, *pools)]
        m.remap(i32(parent), i32(reserve))
        assert m.status(clear=True)[0] == status
        if status != twl.TWL_OK:
            assert all(torch.equal(x, y) for x, y in zip(before, (table, lens, *pools)))
    # 12 pages: four slots of 33 tokens hold 2 shared and 4 partial ones, 6 are free
    before = [t.clone() for t in (table, lens, *pools)]
    m.remap(i32(same), i32([15, 31, 31, 15]))                     # 0 + 1 + 1 + 0 more pages
    assert m.status(clear=True)[0] == twl.TWL_OK
    before = [t.clone() for t in (table, lens, *pools)]
    m.remap(i32([-1, -1, 2, 2]), i32([0, 0, 31, 16 * 7 + 1]))     # more than are free
    status = m.status(clear=True)[0]
    assert status in (twl.TWL_ERR_NO_PAGES, twl.TWL_ERR_BAD_INDEX)
    assert all(torch.equal(x, y) for x, y in zip(before, (table, lens, *pools)))
    table[1, 0] = 12                                              # an entry outside the pool
    before = [t.clone() for t in (table, lens, *pools)]
    m.remap(i32(same))
    assert m.status(clear=True)[0] == twl.TWL_ERR_BAD_INDEX
    used = m.compact(torch.empty_like(table))
    assert m.status(clear=True)[0] == twl.TWL_ERR_BAD_INDEX
    assert all(torch.equal(x, y) for x, y in zip(before, (table, lens, *pools)))
    m.remap(i32([0, -1, 2, 3]))                                   # freed: no longer held
    assert m.status(clear=True)[0] == twl.TWL_OK
    lens[0] = -1
    m.remap(i32(same))
    assert m.status(clear=True)[0] == twl.TWL_ERR_BAD_INDEX
    assert used.device.type == "cuda"


def test_remap_too_few_pages():
    from adaptive_top_sparse_b200.layer import PageManager
    table, lens, pools = make(8, 2, 0, 4, extra=6)
    lens.copy_(i32([17, 0]))
    table.fill_(-1)
    table[0, :2] = i32([3, 1])
    m = PageManager(pools, table, lens)
    before = [t.clone() for t in (table, lens, *pools)]
    m.remap(i32([0, 0]), i32([32, 0]))            # wants 2 + 1 pages of 2
    assert m.status(clear=True) == (twl.TWL_ERR_NO_PAGES, twl.TWL_FLAG_NO_PAGES)
    assert all(torch.equal(x, y) for x, y in zip(before, (table, lens, *pools)))
    m.remap(i32([0, 0]), i32([31, 0]))            # 1 + 1: the last free ones
    assert m.status() == (twl.TWL_OK, 0)
    assert sorted(x for x in table.flatten().tolist() if x >= 0) == [0, 1, 2, 3, 3]


@pytest.mark.parametrize("pages,used", [(1, 1), (5, 0), (40, 17), (256, 256), (257, 100),
                                        (9000, 4000), (9000, 8990), (70000, 300)])
@pytest.mark.parametrize("in_place", [False, True])
def test_compact(pages, used, in_place):
    from adaptive_top_sparse_b200.layer import PageManager
    r = random.Random(pages + used)
    ids = r.sample(range(pages), used)
    width = -(-max(used, 1) // 3) + 2
    flat = ids + [r.choice([-1, -7] + ids[:5]) for _ in range(3 * width - used)]
    table = i32(flat).view(3, width).contiguous()
    g = torch.Generator(device="cuda").manual_seed(1)
    pools = [torch.randint(0, 2 ** 31 - 1, (pages, n), generator=g, device="cuda").int()
             for n in (12, 1500)]
    before = [p.clone() for p in pools]
    m = PageManager(pools, table, torch.zeros(3, dtype=torch.int32, device="cuda"))
    ref = table.clone()
    out = None if in_place else torch.full_like(table, 99)
    count = m.compact(out)
    assert m.status() == (twl.TWL_OK, 0)
    out = table if in_place else out
    assert int(count) == used
    inside = {x for x in ids if x < used}
    to = dict(zip(sorted(x for x in ids if x >= used),
                  [x for x in range(used) if x not in inside]))
    assert out.flatten().tolist() == [to.get(x, x) for x in ref.flatten().tolist()]
    src = torch.arange(pages, device="cuda")
    if to:
        src[torch.tensor(list(to.values()), device="cuda")] = torch.tensor(list(to), device="cuda")
    for old, pool in zip(before, pools):
        assert torch.equal(pool, old[src])


def test_a_decoding_loop_of_beams():
    """Prompts prefilled in two chunks, then beams that fork, append, attend and drop pages, with
    the cache in fp16 and in 4 bits; every step's outputs against contiguous per-beam copies."""
    from test_window import D, _attend, _check, _rand, _seen, _unquantise
    from adaptive_top_sparse_b200.layer import DecodeLayer, Int4Layer
    batch, hq, hkv, sinks, window, pages = 4, 8, 2, 4, 48, 64
    prompt = [70, 33]
    table = torch.full((batch, 12), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
    k, v = _rand(1, pages, hkv, PAGE, D), _rand(2, pages, hkv, PAGE, D)
    layer = DecodeLayer(k, v, table, lens, hq, hkv)
    manager = layer.pages()
    r = random.Random(3)
    # pages for the prompts: empty slots that go on with a reserve
    manager.remap(i32([0, 1, 2, 3]), i32(prompt + [0, 0]), sinks, window)
    lens[:2] = i32(prompt)
    rows = [[(k[table[b, j // PAGE], :, j % PAGE].clone(), v[table[b, j // PAGE], :, j % PAGE].clone())
             for j in range(n)] for b, n in enumerate(prompt)] + [[], []]
    for cut in (40, 10):                          # the last 40 tokens, then the last 10, of both
        cut = [min(cut, n) for n in prompt]
        start = i32([0, cut[0], sum(cut), sum(cut), sum(cut)])
        q = _rand(4 + cut[0], sum(cut), hq, D)
        o, lse = layer.window_prefill(q, start, sinks, window)
        for b in range(2):
            part = slice(int(start[b]), int(start[b + 1]))
            t = torch.arange(prompt[b] - cut[b], prompt[b], device="cuda")
            kk, vv = (torch.stack(x).double() for x in zip(*rows[b]))
            want = _attend(q[part].double(), kk, vv, _seen(t, prompt[b], sinks, window))
            _check(o[part], lse[part], want[0], want[1], 6.0, want[2], True)
    layer.build_aux()
    layer.status(clear=True)                      # it flags the two slots that are still empty
    four = Int4Layer.from_fp16(k, v, table.clone(), lens.clone(), hq, hkv)
    codes = None
    for step in range(24):
        parent = [0, 1, 0, 1] if step == 0 else [r.choice([b, b, r.randrange(batch)]) for b in range(batch)]
        manager.remap(i32(parent), i32([1] * batch), sinks, window)
        four.pages().remap(i32(parent), i32([1] * batch), sinks, window)
        assert torch.equal(table, four.page_table) and torch.equal(lens, four.seq_lens)
        rows = [list(rows[p]) for p in parent]
        kn, vn = _rand(100 + step, batch, hkv, D), _rand(200 + step, batch, hkv, D)
        q = _rand(300 + step, batch, hq, D)
        layer.append(kn, vn)
        o, lse = layer.window_decode(q, sinks, window)
        o4, lse4 = four.decode(q, kn, vn, sinks, window)
        assert torch.equal(lens, four.seq_lens)
        for b in range(batch):
            rows[b].append((kn[b], vn[b]))
            m = len(rows[b])
            assert int(lens[b]) == m
            kk, vv = (torch.stack(x).double() for x in zip(*rows[b]))
            seen = _seen(torch.tensor([m - 1], device="cuda"), m, sinks, window)
            want = _attend(q[b:b + 1].double(), kk, vv, seen)
            _check(o[b:b + 1], lse[b:b + 1], want[0], want[1], 6.0, want[2], False)
            qk, qv = (_quantised(x) for x in (kk, vv))
            want = _attend(q[b:b + 1].double(), qk, qv, seen)
            _check(o4[b:b + 1], lse4[b:b + 1], want[0], want[1], 6.0, want[2], False)
        if step == 12:                            # move everything to the front on the way
            count = int(manager.compact())
            assert int(table.max()) < count
            four.pages().compact()
    assert layer.status() == (twl.TWL_OK, 0) and manager.status() == (twl.TWL_OK, 0)
    assert four.status() == (twl.TWL_OK, 0) and four.pages().status() == (twl.TWL_OK, 0)
    # pages behind the window were dropped on the way: a beam holds its window, sinks and tail
    held = [int((table[b] >= 0).sum()) for b in range(batch)]
    assert max(held) <= window // PAGE + 3 and codes is None


def _quantised(x):
    """The rows that the 4-bit scheme stores for x [T][Hkv][128] (64 bits in and out)."""
    f = x.float()
    lo, hi = f.amin(-1, keepdim=True), f.amax(-1, keepdim=True)
    s = ((hi - lo) / 15.0).half().float()
    n = torch.where(s == 0, torch.zeros_like(f), torch.round((f - lo) / s).clamp(0, 15))
    return n.double() * s.double() + lo.double()


def test_captured_steps_share_a_workspace_and_replay():
    """A page step, an append and attention captured twice (two graphs over one layer) and replayed
    in turn give what eager calls give, also on another stream than the tensors were made on."""
    from test_window import D, _rand
    from adaptive_top_sparse_b200.layer import DecodeLayer, Int4Layer
    results = []
    for mode in ("eager", "graph"):
        table = torch.full((2, 12), -1, dtype=torch.int32, device="cuda")
        lens = torch.zeros(2, dtype=torch.int32, device="cuda")
        k, v = _rand(1, 40, 2, PAGE, D), _rand(2, 40, 2, PAGE, D)
        layer = DecodeLayer(k, v, table, lens, 8, 2)
        four = Int4Layer.from_fp16(k, v, table, lens, 8, 2)
        manager = layer.pages()
        manager.remap(i32([0, 1]), i32([50, 20]))
        lens.copy_(i32([50, 20]))
        parents = [i32([0, 1]), i32([1, 1])]
        one, start = i32([1, 1]), i32([0, 3, 7])
        q, qp = _rand(3, 2, 8, D), _rand(4, 7, 8, D)
        kn, vn = _rand(5, 2, 2, D), _rand(6, 2, 2, D)
        out = layer.window_prefill(qp, start)

        def step(parent):
            manager.remap(parent, one, 4, 30)
            layer.append(kn, vn)
            layer.window_decode(q, 4, 30)
            layer.window_prefill(qp, start, 4, 20, out)
            four.decode(q, sinks=4, window=30)

        got = []
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            if mode == "graph":
                graphs = []
                for parent in parents:
                    g = torch.cuda.CUDAGraph()
                    with torch.cuda.graph(g, stream=stream):
                        step(parent)
                    graphs.append(g)
            for i in (0, 0, 1, 0, 1):
                graphs[i].replay() if mode == "graph" else step(parents[i])
                got += [x.clone() for x in (layer.o, layer.lse, *out, four.o, four.lse, table, lens)]
        torch.cuda.synchronize()
        assert layer.status() == (twl.TWL_OK, 0) and manager.status() == (twl.TWL_OK, 0)
        results.append(got)
    assert all(torch.equal(x, y) for x, y in zip(*results))
    assert not any(x.isnan().any() for x in results[0] if x.is_floating_point())


def test_bad_pages_and_lengths_are_skipped():
    """A bad page hides its tokens, a bad length its sequence; the others stay exact."""
    from test_window import D, _attend, _check, _rand, _rows, _seen, _unquantise
    from adaptive_top_sparse_b200.layer import DecodeLayer, Int4Layer
    lens, hq, hkv = [100, 60, 70, 33], 8, 2
    table = torch.arange(32, dtype=torch.int32, device="cuda").view(4, 8).contiguous()
    n = i32(lens)
    k, v = _rand(1, 32, hkv, PAGE, D), _rand(2, 32, hkv, PAGE, D)
    four = Int4Layer.from_fp16(k, v, table.clone(), n.clone(), hq, hkv)
    layer = DecodeLayer(k, v, table, n, hq, hkv)
    for x, y in ((table, n), (four.page_table, four.seq_lens)):
        x[0, 2], x[0, 4] = 32, -1                  # outside the pool, unmapped
        y[1], y[2] = PAGE * 8 + 1, -3              # too long, negative
    q = _rand(3, 4, hq, D)
    start = i32([0, 1, 3, 3, 7])
    qp = _rand(4, 7, hq, D)
    for got, cache in ((layer.window_decode(q), None), (four.decode(q), four),
                       (layer.window_prefill(qp, start), "chunk")):
        o, lse = got
        for b in (0, 3):
            kk, vv = _rows(k, table.clamp(max=31), b, lens[b]), _rows(v, table.clamp(max=31), b, lens[b])
            if isinstance(cache, Int4Layer):
                kk, vv = (_quantised(x.double()) for x in (kk, vv))
            rows = slice(int(start[b]), int(start[b + 1])) if cache == "chunk" else slice(b, b + 1)
            count = rows.stop - rows.start
            t = torch.arange(lens[b] - count, lens[b], device="cuda")
            seen = _seen(t, lens[b], 0, ALL)
            if b == 0:
                seen[:, 32:48] = False
                seen[:, 64:80] = False
            want = _attend((qp if cache == "chunk" else q)[rows].double(), kk.double(), vv.double(), seen)
            _check(o[rows], lse[rows], want[0], want[1], 6.0, want[2], cache == "chunk")
        if cache != "chunk":
            assert bool((o[1:3] == 0).all()) and bool((lse[1:3] == -math.inf).all())
    assert layer.status(clear=True) == (twl.TWL_ERR_BAD_INDEX, twl.TWL_FLAG_BAD_INDEX)
    assert four.status(clear=True) == (twl.TWL_ERR_BAD_INDEX, twl.TWL_FLAG_BAD_INDEX)
    # a token whose page is not mapped: left alone and flagged; an empty slot: no flag
    four.seq_lens.copy_(i32([128, 20, 0, 5]))
    four.page_table[1, 1], four.page_table[2, 0] = -1, -1
    kn = _rand(5, 4, hkv, D)
    before = four.k.clone()
    o, lse = four.decode(q, kn, kn)
    assert four.seq_lens.tolist() == [128, 20, 0, 6]
    assert bool((o[:3] == 0).all()) and bool((lse[:3] == -math.inf).all())
    changed = (four.k != before).flatten(1).any(1).nonzero().flatten().tolist()
    assert changed == [24]
    assert four.status()[0] == twl.TWL_ERR_BAD_INDEX
