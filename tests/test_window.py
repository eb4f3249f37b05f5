"""Attention under a sliding window with sinks (one token, prompt chunks), a cache held in 4 bits,
and the page-table step and compaction, each against its definition in 64 bits.

Tolerances, from the number formats (u16 = 2^-11 and u32 = 2^-24 are half-step roundings):
  o of one token   fp32; the weights enter as two fp16 parts (2^-22 each at most) and sums of up to
                   64 K terms lose well under 2^-18 relative to sum p|v| / sum p, so
                   |o - o64| <= 2^-17 max|v|
  o of a chunk     fp16; weights rounded to fp16 (2 u16: weight and its tail) and the result (u16):
                   |o - o64| <= 3 u16 max|v|
  lse              fp32 of a score of up to a few hundred: |lse - lse64| <= 2^-18 (1 + max|score|)
Page numbers, lengths and copied rows are equal.
"""
import ctypes as C
import math

import numpy as np
import pytest
import torch

from adaptive_top_sparse_b200 import twl

D, PAGE = 128, 16
ALL = 2 ** 31 - 1
A = 1 << 20                        # a fake aligned address: those calls fail before any launch
SCALE = 1.0 / math.sqrt(D)


# ------------------------------------------------------------------ refusals (no GPU needed)
def _kv(**over):
    d = dict(k=A, v=A, page_table=A, seq_lens=A, batch=2, num_kv_heads=8, head_dim=128,
             page_size=16, max_pages=64, num_phys_pages=128)
    d.update(over)
    return twl._PagedKV(*d.values())


def _kv4(**over):
    d = dict(k=A, k_scale_zero=A, v=A, v_scale_zero=A, page_table=A, seq_lens=A, batch=2,
             num_kv_heads=8, head_dim=128, page_size=16, max_pages=64, num_phys_pages=128)
    d.update(over)
    return twl._Int4KV(*d.values())


BAD_WINDOW = [(dict(sinks=-1), -1), (dict(window=0), -1), (dict(window=-3), -1),
              (dict(scale=0.0), -1), (dict(scale=float("inf")), -1),
              (dict(scale=float("nan")), -1), (dict(q=0), -1), (dict(q=A + 8), -1),
              (dict(o=0), -1), (dict(o=A + 4), -1), (dict(lse=0), -1), (dict(hq=24), -2),
              (dict(hq=12), -1), (dict(hq=128), -2), (dict(ws=0), -5), (dict(ws=A + 16), -5),
              (dict(ws_bytes=300), -5)]
BAD_CACHE = [(dict(k=0), -1), (dict(v=0), -1), (dict(v=A + 8), -1), (dict(page_table=0), -1),
             (dict(seq_lens=A + 1), -1), (dict(batch=0), -1), (dict(batch=513), -2),
             (dict(head_dim=64), -2), (dict(page_size=32), -2), (dict(max_pages=32769), -2),
             (dict(num_phys_pages=0), -1), (dict(num_phys_pages=1 << 26), -2)]


def _decode(kv=None, q=A, hq=32, sinks=4, window=100, scale=SCALE, o=A, lse=A, ws=A,
            ws_bytes=1 << 40):
    return twl._lib.twl_window_decode(q, hq, C.byref(kv or _kv()), sinks, window, scale, o, lse,
                                      ws, ws_bytes, None)


def _prefill(kv=None, q=A, start=A, total=16, hq=32, sinks=4, window=100, scale=SCALE, o=A, lse=A,
             ws=A, ws_bytes=1 << 40):
    return twl._lib.twl_window_prefill(q, start, total, hq, C.byref(kv or _kv()), sinks, window,
                                       scale, o, lse, ws, ws_bytes, None)


def _decode4(kv=None, q=A, hq=32, k_new=A, v_new=A, advance=1, sinks=4, window=100, scale=SCALE,
             o=A, lse=A, ws=A, ws_bytes=1 << 40):
    return twl._lib.twl_int4_decode(q, hq, C.byref(kv or _kv4()), k_new, v_new, advance, sinks,
                                    window, scale, o, lse, ws, ws_bytes, None)


@pytest.mark.parametrize("call", [_decode, _prefill, _decode4])
@pytest.mark.parametrize("kw,code", BAD_WINDOW)
def test_attention_refuses_bad_arguments(call, kw, code):
    if call is _prefill and "ws_bytes" in kw:
        kw = dict(ws_bytes=128)
    assert call(**kw) == code


@pytest.mark.parametrize("kw,code", BAD_CACHE)
def test_attention_refuses_bad_caches(kw, code):
    assert _decode(kv=_kv(**kw)) == code
    assert _prefill(kv=_kv(**kw)) == code
    assert _decode4(kv=_kv4(**kw)) == code


def test_prefill_and_int4_refuse_their_own():
    assert _prefill(start=0) == -1
    assert _prefill(start=A + 2) == -1
    assert _prefill(total=-1) == -1
    assert _prefill(total=0, q=0, o=0, lse=0) == 0           # nothing to do, nothing launched
    assert _decode4(k_new=None) == -1                        # one without the other
    assert _decode4(v_new=None) == -1
    assert _decode4(k_new=None, v_new=None, advance=1) == -1
    assert _decode4(k_new=A + 8) == -1
    assert _decode4(kv=_kv4(k_scale_zero=0)) == -1
    assert _decode4(kv=_kv4(v_scale_zero=A + 8)) == -1
    assert twl._lib.twl_int4_decode(A, 32, None, A, A, 1, 0, 1, SCALE, A, A, A, 1 << 40, None) == -1


def _pools(n=2, data=A, nbytes=4096):
    return (twl._PagePool * max(n, 1))(*[(data, nbytes)] * n)


def _remap(pools=None, n=2, table=A, lens=A, batch=4, max_pages=64, phys=256, parent=A, reserve=A,
           sinks=0, window=ALL, ws=A, ws_bytes=1 << 40):
    return twl._lib.twl_remap_pages(pools if pools is not None else _pools(), n, table, lens,
                                    batch, max_pages, phys, parent, reserve, sinks, window, ws,
                                    ws_bytes, None)


def _compact(pools=None, n=2, table=A, out=A, batch=4, max_pages=64, phys=256, used=A, ws=A,
             ws_bytes=1 << 40):
    return twl._lib.twl_compact_pages(pools if pools is not None else _pools(), n, table, out,
                                      batch, max_pages, phys, used, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(n=0), -1), (dict(n=129), -1), (dict(table=0), -1), (dict(table=A + 2), -1),
    (dict(batch=0), -1), (dict(batch=4097), -2), (dict(max_pages=0), -1),
    (dict(max_pages=32769), -2), (dict(phys=0), -1), (dict(phys=(1 << 23) + 1), -2),
    (dict(pools=_pools(data=0)), -1), (dict(pools=_pools(data=A + 8)), -1),
    (dict(pools=_pools(nbytes=24)), -1), (dict(pools=_pools(nbytes=0)), -1),
    (dict(ws=0), -5), (dict(ws=A + 8), -5), (dict(ws_bytes=256), -5)])
def test_page_calls_refuse_bad_arguments(kw, code):
    assert _remap(**kw) == code
    assert _compact(**kw) == code


def test_page_calls_refuse_their_own():
    assert _remap(lens=0) == -1
    assert _remap(parent=0) == -1
    assert _remap(reserve=A + 2) == -1
    assert _remap(sinks=-1) == -1
    assert _remap(window=0) == -1
    assert _compact(out=0) == -1
    assert _compact(used=0) == -1
    assert _compact(used=A + 1) == -1
    assert twl._lib.twl_remap_pages(None, 1, A, A, 4, 64, 256, A, A, 0, 1, A, 1 << 40, None) == -1


def test_workspaces_and_status_of_the_new_calls():
    wb = twl.twl_workspace_bytes
    for op in (twl.TWL_OP_WINDOW_DECODE, twl.TWL_OP_INT4_DECODE, twl.TWL_OP_WINDOW_PREFILL):
        assert wb(op, 2, 32, 8) >= 256 and wb(op, 2, 32, 8) % 256 == 0
        assert wb(op, 2, 32, 0) == 0 and wb(op, 2, 4, 8) == 0
    assert wb(twl.TWL_OP_PAGES, 4, 0, 0, 64, 0, 4096) >= 256 + 4 * 64 * 4 + 4096 // 8
    assert wb(twl.TWL_OP_PAGES, 4, 0, 0, 64, 0, -1) == 0
    assert twl.twl_status_string(twl.TWL_ERR_NO_PAGES) != "unknown status"


def test_wrappers_refuse_bad_tensors():
    from adaptive_top_sparse_b200.layer import DecodeLayer, Int4Layer, PageManager
    f16, i32, u8 = torch.float16, torch.int32, torch.uint8
    e = lambda *s, dt=f16: torch.empty(s, dtype=dt, device="meta")
    layer = DecodeLayer.__new__(DecodeLayer)
    layer.k, layer.batch, layer.num_q_heads, layer.num_kv_heads = e(4, 2, 16, 128), 3, 8, 2
    start = e(4, dt=i32)
    for q, s in ((e(5, 8, 64), start), (e(5, 4, 128), start), (e(5, 8, 128, dt=torch.float32), start),
                 (e(5, 128, 8).transpose(1, 2), start), (torch.zeros(5, 8, 128, dtype=f16), start),
                 (e(8, 128), start), (e(5, 8, 128), e(3, dt=i32)),
                 (e(5, 8, 128), e(4, dt=torch.int64))):
        with pytest.raises(ValueError):
            layer.window_prefill(q, s)
    with pytest.raises(ValueError):
        layer.window_prefill(e(5, 8, 128), start, out=(e(4, 8, 128), e(5, 8, dt=torch.float32)))
    with pytest.raises(ValueError):
        layer.window_decode(e(3, 8, 64))
    good = [e(4, 2, 16, 64, dt=u8), e(4, 2, 16, 2), e(4, 2, 16, 64, dt=u8), e(4, 2, 16, 2),
            e(3, 5, dt=i32), e(3, dt=i32)]
    for i, bad in ((0, e(4, 2, 16, 64)), (1, e(4, 2, 16)), (2, e(4, 1, 16, 64, dt=u8)),
                   (3, e(5, 2, 16, 2)), (4, e(3, 5, dt=torch.int64)), (5, e(4, dt=i32)),
                   (0, e(4, 2, 64, dt=u8)), (4, e(15, dt=i32)), (4, torch.zeros(3, 5, dtype=i32))):
        with pytest.raises(ValueError):
            Int4Layer(*[bad if j == i else t for j, t in enumerate(good)], 8, 2)
    with pytest.raises(ValueError):
        Int4Layer.from_fp16(e(4, 2, 16, 64), e(4, 2, 16, 64), good[4], good[5], 8, 2)
    for pools in ([], [e(4, 8), e(5, 8)], [e(4, 8), torch.zeros(4, 8)], [e(4, 8, 2).transpose(1, 2)]):
        with pytest.raises(ValueError):
            PageManager(pools, good[4], good[5])
    four = Int4Layer.__new__(Int4Layer)
    four.device, four.batch, four.num_q_heads, four.num_kv_heads = torch.device("meta"), 3, 8, 2
    with pytest.raises(ValueError):
        four.decode(e(3, 8, 128), e(3, 2, 128))
    with pytest.raises(ValueError):
        four.decode(e(3, 8, 128), e(3, 2, 128), e(3, 8, 128))


# ------------------------------------------------------------------ the definition, in 64 bits
def _seen(t, n, sinks, window):
    j = torch.arange(n, device=t.device)
    return (j <= t[:, None]) & ((j < sinks) | (j > t[:, None] - window))


def _attend(q, k, v, seen):
    """q [R][Hq][128], k and v [T][Hkv][128] (64 bits), seen [R][T] -> o, lse, and max|score|."""
    group = q.shape[1] // k.shape[1]
    k, v = k.repeat_interleave(group, 1), v.repeat_interleave(group, 1)
    any_seen = seen.any(0)
    k, v = k[any_seen], v[any_seen]                # rows nobody sees may hold anything
    s = torch.einsum("rhd,thd->rht", q, k) * SCALE
    s = s.masked_fill(~seen[:, None, any_seen], -math.inf)
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - torch.where(lse.isinf(), torch.zeros_like(lse), lse)[..., None])
    big = s[s.isfinite()].abs().max().item() if s.isfinite().any() else 0.0
    return torch.einsum("rht,thd->rhd", p, v), lse, big


def _deal(lens, seed, extra_pages=1, spare=3, device="cuda"):
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // PAGE) + extra_pages for n in lens]
    total = sum(need) + spare
    perm = torch.randperm(total, generator=g).to(torch.int32)
    table = torch.full((len(lens), max(need) + 1), -1, dtype=torch.int32)
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = perm[at:at + m]
        at += m
    return table.to(device), torch.tensor(lens, dtype=torch.int32, device=device), total


def _rand(seed, *shape, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).half()


def _rows(pool, table, b, n):
    j = torch.arange(n, device=pool.device)
    return pool[table[b].long()[j // PAGE].clamp(min=0), :, j % PAGE]


def _unquantise(codes, sz):
    n = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).double()
    return n * sz[..., :1].double() + sz[..., 1:].double()


def _check(o, lse, want_o, want_lse, vmax, big, half):
    tol = 3 * 2.0 ** -11 * vmax if half else 2.0 ** -17 * vmax
    assert o.shape == want_o.shape and not o.isnan().any()
    assert (o.double() - want_o).abs().max().item() <= tol + 1e-30
    none = want_lse.isinf()
    assert torch.equal(lse.isinf(), none) and bool((lse[none] < 0).all())
    if (~none).any():
        far = (lse.double() - want_lse)[~none].abs().max().item()
        assert far <= 2.0 ** -18 * (1 + big)


WINDOWS = [(0, ALL), (4, 20), (0, 1), (17, 33), (64, 100), (1, 16), (ALL, 5), (3, 5000)]


@pytest.mark.gpu
@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 2), (8, 2), (16, 2), (32, 8)])
@pytest.mark.parametrize("sinks,window", WINDOWS)
def test_window_decode(hq, hkv, sinks, window):
    from adaptive_top_sparse_b200.layer import DecodeLayer
    lens = [1, 15, 16, 17, 130, 1000, 0, 2047]
    table, n, pages = _deal(lens, hq + window % 97)
    k, v = _rand(1, pages, hkv, PAGE, D), _rand(2, pages, hkv, PAGE, D)
    q = _rand(3, len(lens), hq, D, scale=2.0)
    for b, m in enumerate(lens):        # stale rows behind a sequence and rows outside its window
        first = min(sinks, m)
        for j in list(range(m, table.shape[1] * PAGE)) + list(range(first, max(first, m - window))):
            if table[b, j // PAGE] >= 0:
                k[table[b, j // PAGE], :, j % PAGE] = math.nan
                v[table[b, j // PAGE], :, j % PAGE] = math.inf
    layer = DecodeLayer(k, v, table, n, hq, hkv)
    for _ in range(2):                  # the second call finds the workspace as the first left it
        layer.o.fill_(math.nan)
        o, lse = layer.window_decode(q, sinks, window)
        for b, m in enumerate(lens):
            t = torch.tensor([m - 1], device="cuda")
            want, wlse, big = _attend(q[b:b + 1].double(), _rows(k, table, b, m).double(),
                                      _rows(v, table, b, m).double(), _seen(t, m, sinks, window))
            _check(o[b:b + 1], lse[b:b + 1], want, wlse, 6.0, big, False)
    assert layer.status() == (twl.TWL_OK, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 2), (8, 2), (16, 2), (32, 8)])
@pytest.mark.parametrize("sinks,window", WINDOWS)
def test_window_prefill(hq, hkv, sinks, window):
    from adaptive_top_sparse_b200.layer import DecodeLayer
    lens, qn = [1, 33, 64, 700, 0, 300, 257, 40], [1, 33, 5, 300, 0, 1, 257, 0]
    table, n, pages = _deal(lens, hq + window % 89)
    k, v = _rand(1, pages, hkv, PAGE, D), _rand(2, pages, hkv, PAGE, D)
    first_row = 3                       # rows before, and 5 behind, belong to no chunk
    start = torch.tensor([first_row + sum(qn[:i]) for i in range(len(qn) + 1)], dtype=torch.int32)
    total = int(start[-1]) + 5
    q = _rand(3, total, hq, D, scale=2.0)
    q[:first_row] = math.nan
    for b, m in enumerate(lens):        # stale rows behind a sequence, and rows no query sees
        first, t0 = min(sinks, m), m - qn[b]
        for j in list(range(m, table.shape[1] * PAGE)) + \
                list(range(first, max(first, t0 - window + 1))):
            if table[b, j // PAGE] >= 0:
                k[table[b, j // PAGE], :, j % PAGE] = math.nan
                v[table[b, j // PAGE], :, j % PAGE] = math.inf
    layer = DecodeLayer(k, v, table, n, hq, hkv)
    for _ in range(2):
        out = (torch.full((total, hq, D), 7.0, dtype=torch.float16, device="cuda"),
               torch.full((total, hq), 7.0, device="cuda"))
        o, lse = layer.window_prefill(q, start.cuda(), sinks, window, out)
        for x in out:
            assert bool((x[:first_row] == 7).all()) and bool((x[int(start[-1]):] == 7).all())
        for b, m in enumerate(lens):
            rows = slice(int(start[b]), int(start[b + 1]))
            if qn[b] == 0:
                continue
            t = torch.arange(m - qn[b], m, device="cuda")
            want, wlse, big = _attend(q[rows].double(), _rows(k, table, b, m).double(),
                                      _rows(v, table, b, m).double(), _seen(t, m, sinks, window))
            _check(o[rows], lse[rows], want, wlse, 6.0, big, True)
    assert layer.status() == (twl.TWL_OK, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 2), (8, 2), (16, 2), (32, 8)])
@pytest.mark.parametrize("sinks,window", WINDOWS)
@pytest.mark.parametrize("vscale", [1.0, 1e-3, 300.0])
def test_int4_decode(hq, hkv, sinks, window, vscale):
    from adaptive_top_sparse_b200.layer import Int4Layer
    lens = [1, 15, 16, 17, 130, 1000, 0, 2047]
    table, n, pages = _deal(lens, hq + window % 83)
    k, v = _rand(1, pages, hkv, PAGE, D), _rand(2, pages, hkv, PAGE, D, scale=vscale)
    v[::3, :, 5] = 0.25 * vscale        # constant rows: scale 0
    layer = Int4Layer.from_fp16(k, v, table, n, hq, hkv)
    layer.k_sz[table[7, -2].long()] = math.nan           # a mapped page behind a sequence
    q = _rand(3, len(lens), hq, D, scale=2.0)
    for step in range(3):
        kn, vn = _rand(10 + step, 8, hkv, D), _rand(20 + step, 8, hkv, D, scale=vscale)
        o, lse = layer.decode(q, kn, vn, sinks, window)
        ends = [m + step + 1 for m in lens]
        assert n.tolist() == ends
        for b, m in enumerate(ends):
            kk = _unquantise(_rows(layer.k, table, b, m), _rows(layer.k_sz, table, b, m))
            vv = _unquantise(_rows(layer.v, table, b, m), _rows(layer.v_sz, table, b, m))
            for new, row in ((kn, kk[-1]), (vn, vv[-1])):      # at most half a code away
                lo, hi = new[b].double().aminmax(dim=-1)
                # half a code, plus the scale's own rounding over 15 codes
                near = (hi - lo) / 30 * (1 + 2.0 ** -5)
                assert bool(((new[b].double() - row).abs().amax(-1) <= near).all())
            t = torch.tensor([m - 1], device="cuda")
            want, wlse, big = _attend(q[b:b + 1].double(), kk, vv, _seen(t, m, sinks, window))
            _check(o[b:b + 1], lse[b:b + 1], want, wlse, 6.0 * vscale, big, False)
    # without a new token: the same answers from the last cached one, and nothing moves
    again, lse2 = (x.clone() for x in (o, lse))
    before = [x.clone() for x in (layer.k, layer.v, n)]
    o, lse = layer.decode(q, sinks=sinks, window=window)
    assert torch.equal(o, again) and torch.equal(lse, lse2)
    assert all(torch.equal(x, y) for x, y in zip(before, (layer.k, layer.v, n)))
    assert layer.status() == (twl.TWL_OK, 0)


# ------------------------------------------------------------------ where such kernels go wrong
@pytest.mark.gpu
@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 2), (16, 2)])
@pytest.mark.parametrize("sinks,window", [(0, ALL), (4, 60), (150, 40)])
def test_rows_that_are_not_finite_reach_only_their_queries(hq, hkv, sinks, window):
    from adaptive_top_sparse_b200.layer import DecodeLayer
    n, qn = 420, 333
    table, lens, pages = _deal([n], 5)
    k, v = _rand(1, pages, hkv, PAGE, D), _rand(2, pages, hkv, PAGE, D)
    q = _rand(3, qn, hq, D)
    kk, vv = _rows(k, table, 0, n).double(), _rows(v, table, 0, n).double()   # before the planting
    spoilt_v = {100: (7, math.nan), 300: (100, math.inf), 333: (64, -math.inf)}
    for key, (col, value) in spoilt_v.items():
        v[table[0, key // PAGE], 0, key % PAGE, col] = value
    bad_k = 380
    k[table[0, bad_k // PAGE], 0, bad_k % PAGE, 3] = math.nan
    layer = DecodeLayer(k, v, table, lens, hq, hkv)
    start = torch.tensor([0, qn], dtype=torch.int32, device="cuda")
    o, lse = layer.window_prefill(q, start, sinks, window)
    t = torch.arange(n - qn, n, device="cuda")
    seen = _seen(t, n, sinks, window)
    want, wlse, big = _attend(q.double(), kk, vv, seen)
    group = hq // hkv
    spoilt = torch.zeros_like(o, dtype=torch.bool)
    for key, (col, _) in spoilt_v.items():
        spoilt[seen[:, key], :group, col] = True
    spoilt[seen[:, bad_k], :group] = True
    assert torch.equal(~o.isfinite(), spoilt)
    far = (o.double() - want).abs()[~spoilt].max().item()
    assert far <= 3 * 2.0 ** -11 * 6.0
    fine = ~seen[:, bad_k, None] | (torch.arange(hq, device="cuda") >= group)
    assert (lse.double() - wlse)[fine].abs().max().item() <= 2.0 ** -18 * (1 + big)
    assert not lse[~fine].isfinite().any()
    # one token: the same for its heads
    o, lse = layer.window_decode(q[-1:], sinks, window)
    spoilt = spoilt[-1]
    assert torch.equal(~o[0].isfinite(), spoilt)
    assert (o[0].double() - want[-1]).abs()[~spoilt].numel() == 0 or \
        (o[0].double() - want[-1]).abs()[~spoilt].max().item() <= 2.0 ** -17 * 6.0


@pytest.mark.gpu
@pytest.mark.parametrize("batch,hq,hkv", [(4096, 1, 1), (500, 16, 8), (161, 4, 2), (160, 8, 1)])
def test_many_sequences(batch, hq, hkv):
    """Batches up to the largest, ragged, some empty: one token, chunks of 0-40, a 4-bit cache."""
    from adaptive_top_sparse_b200.layer import DecodeLayer, Int4Layer
    g = torch.Generator().manual_seed(batch)
    lens = torch.randint(0, 70, (batch,), generator=g).tolist()
    lens[7], lens[8] = 900, 0
    table, n, pages = _deal(lens, 3, extra_pages=1, spare=0)
    k, v = _rand(1, pages, hkv, PAGE, D), _rand(2, pages, hkv, PAGE, D)
    qn = [min(m, int(x)) for m, x in zip(lens, torch.randint(0, 41, (batch,), generator=g))]
    start = torch.tensor([0] + qn).cumsum(0).int()
    q, qp = _rand(3, batch, hq, D), _rand(4, int(start[-1]), hq, D)
    sinks, window = 3, 48
    layer = DecodeLayer(k, v, table, n, hq, hkv)
    o, lse = layer.window_decode(q, sinks, window)
    op, lsep = layer.window_prefill(qp, start.cuda(), sinks, window)
    four = Int4Layer.from_fp16(k, v, table, n.clone(), hq, hkv)
    kn, vn = _rand(5, batch, hkv, D), _rand(6, batch, hkv, D)
    o4, lse4 = four.decode(q, kn, vn, sinks, window)
    assert four.seq_lens.tolist() == [m + 1 for m in lens]
    assert layer.status() == (twl.TWL_OK, 0) and four.status() == (twl.TWL_OK, 0)
    assert bool((o[8] == 0).all()) and bool((lse[8] == -math.inf).all())
    for b in [0, 1, 7, 8, 9, batch // 2, batch - 1] + list(range(100, batch, batch // 12)):
        m = lens[b]
        t = torch.tensor([m - 1], device="cuda")
        kk, vv = _rows(k, table, b, m).double(), _rows(v, table, b, m).double()
        if m:
            want = _attend(q[b:b + 1].double(), kk, vv, _seen(t, m, sinks, window))
            _check(o[b:b + 1], lse[b:b + 1], want[0], want[1], 6.0, want[2], False)
        rows = slice(int(start[b]), int(start[b + 1]))
        if qn[b]:
            t = torch.arange(m - qn[b], m, device="cuda")
            want = _attend(qp[rows].double(), kk, vv, _seen(t, m, sinks, window))
            _check(op[rows], lsep[rows], want[0], want[1], 6.0, want[2], True)
        m += 1
        t = torch.tensor([m - 1], device="cuda")
        kk = _unquantise(_rows(four.k, table, b, m), _rows(four.k_sz, table, b, m))
        vv = _unquantise(_rows(four.v, table, b, m), _rows(four.v_sz, table, b, m))
        want = _attend(q[b:b + 1].double(), kk, vv, _seen(t, m, sinks, window))
        _check(o4[b:b + 1], lse4[b:b + 1], want[0], want[1], 6.0, want[2], False)


@pytest.mark.gpu
@pytest.mark.parametrize("hq,hkv,lens,qn,sinks,window", [
    (8, 1, [9000], [4000], 0, ALL),              # one long chunk, keys of many runs
    (4, 4, [33000, 5], [7, 5], 4, 32000),        # a few queries far behind: every unit is cut
    (2, 1, [2500, 2500, 0], [2500, 1, 0], 130, 700),
    (16, 2, [5000] * 9, [1] * 9, 64, 4096)])
def test_long_chunks(hq, hkv, lens, qn, sinks, window):
    from adaptive_top_sparse_b200.layer import DecodeLayer
    table, n, pages = _deal(lens, 11)
    k, v = _rand(1, pages, hkv, PAGE, D), _rand(2, pages, hkv, PAGE, D)
    start = torch.tensor([0] + qn).cumsum(0).int()
    q = _rand(3, int(start[-1]), hq, D, scale=2.0)
    layer = DecodeLayer(k, v, table, n, hq, hkv)
    for _ in range(2):
        o, lse = layer.window_prefill(q, start.cuda(), sinks, window)
        for b, m in enumerate(lens):
            kk, vv = _rows(k, table, b, m).double(), _rows(v, table, b, m).double()
            for r in range(0, qn[b], 500):       # the definition in 64 bits, 500 rows at a time
                rows = slice(int(start[b]) + r, min(int(start[b]) + r + 500, int(start[b + 1])))
                t = torch.arange(m - qn[b] + r, m - qn[b] + r + rows.stop - rows.start, device="cuda")
                want, wlse, big = _attend(q[rows].double(), kk, vv, _seen(t, m, sinks, window))
                _check(o[rows], lse[rows], want, wlse, 6.0, big, True)
    assert layer.status() == (twl.TWL_OK, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("hq,hkv", [(4, 4), (8, 1)])
def test_long_contexts(hq, hkv):
    """One token behind the longest context a table may hold, fp16 and in 4 bits."""
    from adaptive_top_sparse_b200.layer import DecodeLayer, Int4Layer
    lens = [PAGE * 32768 - 1, 39999]
    table, n, pages = _deal(lens, 2, extra_pages=0, spare=0)
    table = torch.nn.functional.pad(table, (0, 32768 - table.shape[1]), value=-1)[:, :32768].contiguous()
    k, v = _rand(1, pages, hkv, PAGE, D), _rand(2, pages, hkv, PAGE, D)
    q = _rand(3, 2, hq, D, scale=2.0)
    layer = DecodeLayer(k, v, table, n, hq, hkv)
    four = Int4Layer.from_fp16(k, v, table, n.clone(), hq, hkv)
    kn, vn = _rand(4, 2, hkv, D), _rand(5, 2, hkv, D)
    for sinks, window in ((0, ALL), (5, 300000)):
        four.seq_lens.copy_(n)
        o, lse = (x.clone() for x in layer.window_decode(q, sinks, window))
        o4, lse4 = four.decode(q, kn, vn, sinks, window)
        for b, m in enumerate(lens):
            t = torch.tensor([m - 1], device="cuda")
            want = _attend(q[b:b + 1].double(), _rows(k, table, b, m).double(),
                           _rows(v, table, b, m).double(), _seen(t, m, sinks, window))
            _check(o[b:b + 1], lse[b:b + 1], want[0], want[1], 6.0, want[2], False)
            m, t = m + 1, t + 1
            kk = _unquantise(_rows(four.k, table, b, m), _rows(four.k_sz, table, b, m))
            vv = _unquantise(_rows(four.v, table, b, m), _rows(four.v_sz, table, b, m))
            want = _attend(q[b:b + 1].double(), kk, vv, _seen(t, m, sinks, window))
            _check(o4[b:b + 1], lse4[b:b + 1], want[0], want[1], 6.0, want[2], False)
    o4, _ = four.decode(q, kn, vn)               # the first sequence is full now: left alone
    assert four.seq_lens.tolist() == [PAGE * 32768, 40000]
    assert bool((o4[0] == 0).all()) and four.status()[0] == twl.TWL_ERR_BAD_INDEX


@pytest.mark.gpu
def test_two_streams_at_once():
    """Two layers on two streams, all calls in flight together, give what they give alone."""
    from adaptive_top_sparse_b200.layer import DecodeLayer, Int4Layer
    sides = []
    for s in range(2):
        lens = [300 + 700 * s, 2000, 17]
        table, n, pages = _deal(lens, s, extra_pages=2, spare=8)
        k, v = _rand(10 + s, pages, 2, PAGE, D), _rand(20 + s, pages, 2, PAGE, D)
        layer = DecodeLayer(k, v, table, n, 8, 2)
        four = Int4Layer.from_fp16(k, v, table, n, 8, 2)
        start = torch.tensor([0, 200, 500, 517], dtype=torch.int32, device="cuda")
        q, qp = _rand(30 + s, 3, 8, D), _rand(40 + s, 517, 8, D)
        parent = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
        out = layer.window_prefill(qp, start)
        manager = layer.pages()
        sides.append((layer, four, manager, q, qp, start, parent, out, torch.cuda.Stream()))

    def calls(layer, four, manager, q, qp, start, parent, out, stream):
        manager.remap(parent, None, 4, 100000, stream=stream)
        layer.window_decode(q, 4, 500, stream=stream)
        four.decode(q, sinks=4, window=500, stream=stream)
        layer.window_prefill(qp, start, 4, 300, out, stream=stream)

    def results(layer, four, manager, q, qp, start, parent, out, stream):
        return [x.clone() for x in (layer.o, layer.lse, four.o, four.lse, *out, layer.page_table)]

    alone = []
    for side in sides:
        calls(*side)
        torch.cuda.synchronize()
        alone.append(results(*side))
    for _ in range(20):
        for side in sides:
            calls(*side)
    torch.cuda.synchronize()
    for side, want in zip(sides, alone):
        assert all(torch.equal(x, y) for x, y in zip(results(*side), want))
        assert side[0].status() == (twl.TWL_OK, 0) and side[2].status() == (twl.TWL_OK, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("four_bit", [False, True])
def test_pools_beyond_32_bit_offsets(four_bit):
    """Pools of more than 2^32 bytes whose used pages lie at the far end: attention there, then a
    compaction that moves them to the front, then the same attention bit for bit."""
    from adaptive_top_sparse_b200.layer import DecodeLayer, Int4Layer, PageManager
    hq, hkv, lens = 16, 8, [700, 33]
    pages = 530000 if four_bit else 140000
    need = [-(-(m + 2) // PAGE) for m in lens]
    table = torch.full((2, max(need)), -1, dtype=torch.int32, device="cuda")
    far = pages - 1 - 7 * torch.arange(sum(need), dtype=torch.int32, device="cuda")
    table[0, :need[0]], table[1, :need[1]] = far[:need[0]], far[need[0]:]
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    q = _rand(1, 2, hq, D)
    if four_bit:
        k, v = (torch.zeros((pages, hkv, PAGE, 64), dtype=torch.uint8, device="cuda") for _ in "kv")
        ks, vs = (torch.zeros((pages, hkv, PAGE, 2), dtype=torch.float16, device="cuda") for _ in "kv")
        for i, (c, sz) in enumerate(((k, ks), (v, vs))):
            g = torch.Generator(device="cuda").manual_seed(i)
            c[far.long()] = torch.randint(0, 256, (len(far), hkv, PAGE, 64), generator=g,
                                          device="cuda").to(torch.uint8)
            sz[far.long()] = _rand(5 + i, len(far), hkv, PAGE, 2, scale=0.3).abs()
        layer = Int4Layer(k, ks, v, vs, table, n, hq, hkv)
        kn, vn = _rand(2, 2, hkv, D), _rand(3, 2, hkv, D)
        o, lse = (x.clone() for x in layer.decode(q, kn, vn))
        for b in range(2):
            m = lens[b] + 1
            kk = _unquantise(_rows(k, table, b, m), _rows(ks, table, b, m))
            vv = _unquantise(_rows(v, table, b, m), _rows(vs, table, b, m))
            want = _attend(q[b:b + 1].double(), kk, vv,
                           torch.ones((1, m), dtype=torch.bool, device="cuda"))
            _check(o[b:b + 1], lse[b:b + 1], want[0], want[1], vv.abs().max().item(), want[2], False)
        again = lambda: layer.decode(q)
    else:
        k, v = (torch.empty((pages, hkv, PAGE, D), dtype=torch.float16, device="cuda") for _ in "kv")
        for i, x in enumerate((k, v)):
            x[far.long()] = _rand(7 + i, len(far), hkv, PAGE, D)
        layer = DecodeLayer.__new__(DecodeLayer)        # without the derived K data: two pools only
        layer.k, layer.v, layer.num_q_heads, layer.num_kv_heads, layer.batch = k, v, hq, hkv, 2
        layer.kv = twl.PagedKV(k, v, table, n, hkv, pages)
        layer.o = torch.zeros((2, hq, D), device="cuda")
        layer.lse = torch.zeros((2, hq), device="cuda")
        layer.ws_window = twl.alloc_workspace(twl.TWL_OP_WINDOW_DECODE, "cuda", batch=2,
                                              num_q_heads=hq, num_kv_heads=hkv)
        layer.ws_prefill = None
        start = torch.tensor([0, 300, 310], dtype=torch.int32, device="cuda")
        qp = _rand(4, 310, hq, D)
        o, lse = (x.clone() for x in layer.window_decode(q))
        op, lsep = layer.window_prefill(qp, start)
        for b in range(2):
            m = lens[b]
            kk, vv = _rows(k, table, b, m).double(), _rows(v, table, b, m).double()
            t = torch.tensor([m - 1], device="cuda")
            want = _attend(q[b:b + 1].double(), kk, vv, _seen(t, m, 0, ALL))
            _check(o[b:b + 1], lse[b:b + 1], want[0], want[1], 6.0, want[2], False)
            rows = slice(int(start[b]), int(start[b + 1]))
            t = torch.arange(m - (rows.stop - rows.start), m, device="cuda")
            want = _attend(qp[rows].double(), kk, vv, _seen(t, m, 0, ALL))
            _check(op[rows], lsep[rows], want[0], want[1], 6.0, want[2], True)
        again = lambda: layer.window_decode(q)
    pools = [layer.k, layer.k_sz, layer.v, layer.v_sz] if four_bit else [k, v]
    manager = PageManager(pools, table, n)
    parent = torch.tensor([0, 0], dtype=torch.int32, device="cuda")      # a fork of a far page
    manager.remap(parent)
    assert int(manager.compact()) == need[0] + (1 if int(n[0]) % PAGE else 0) and \
        manager.status() == (twl.TWL_OK, 0)
    o2, lse2 = again()
    # the fork's second slot attends with its own query; the first is unchanged
    assert torch.equal(o2[0], o[0]) and torch.equal(lse2[0], lse[0])


@pytest.mark.gpu
def test_empty_and_allocating_calls():
    from adaptive_top_sparse_b200.layer import DecodeLayer
    table, n, pages = _deal([20, 5], 1)
    k, v = _rand(1, pages, 2, PAGE, D), _rand(2, pages, 2, PAGE, D)
    layer = DecodeLayer(k, v, table, n, 4, 2)
    start = torch.zeros(3, dtype=torch.int32, device="cuda")
    o, lse = layer.window_prefill(_rand(3, 0, 4, D), start)        # no rows at all
    assert o.shape == (0, 4, D) and lse.shape == (0, 4)
    q = _rand(4, 6, 4, D)
    o, lse = layer.window_prefill(q, start)                        # rows, but every chunk empty
    start = torch.tensor([2, 4, 5], dtype=torch.int32, device="cuda")
    o, lse = layer.window_prefill(q, start)
    same = layer.window_prefill(q, start, out=(torch.empty_like(o), torch.empty_like(lse)))
    assert torch.equal(o[2:5], same[0][2:5]) and torch.equal(lse[2:5], same[1][2:5])
    for bad in ([0, 7, 7], [3, 2, 6], [-1, 2, 3], [0, 0, 6]):      # outside q, backwards, too long
        layer.window_prefill(q, torch.tensor(bad, dtype=torch.int32, device="cuda"))
        assert layer.status(clear=True) == (twl.TWL_ERR_BAD_INDEX, twl.TWL_FLAG_BAD_INDEX)
    assert layer.status() == (twl.TWL_OK, 0)
