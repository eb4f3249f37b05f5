"""Windowed attention and the 4-bit cache where calls and kernels meet: repeated launches, rows that
are not finite, streams, workspaces, limits.  Helpers and tolerances are those of test_window.py."""
import math

import pytest
import torch

from test_window import ALL, D, PAGE, _attend, _check, _deal, _rand, _rows, _seen


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
