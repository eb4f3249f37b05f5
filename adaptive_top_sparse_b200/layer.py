"""Device-side state of one decode-attention layer and the calls a user makes on it.

``DecodeLayer`` is a layer with an fp16 cache, ``Int4Layer`` one whose cache is held in 4 bits, and
``PageManager`` forks, frees, grows and compacts the pages either of them (or many) uses.

``DecodeLayer`` owns device tensors (PyTorch is only the allocator here): the paged fp16 K/V, the
page table, the derived INT4 K and page bounds, a workspace, and the outputs.  Every computation
is a call into libtwl.so.
"""
from __future__ import annotations

import contextlib
import math

import torch

from . import twl


def budget_bound(max_pages: int, budget_pages: int, budget_div: int) -> int:
    """Largest page budget any sequence can get (the sel_pages row stride)."""
    if budget_pages > 0:
        return min(budget_pages, max_pages)
    return -(-max_pages // budget_div)


def expect_tensor(name: str, t, shape, dtype, device) -> None:
    """Raises unless `t` is a contiguous tensor of `shape` and `dtype` on `device`.  The library
    takes raw pointers: it cannot tell a host buffer, a tensor on another GPU or a mis-shaped one
    from a good one, and a kernel would read or write the wrong memory."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if t.device != device:
        raise ValueError(f"{name}: tensor on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if t.shape != shape and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: tensor is not contiguous")


ALL_TOKENS = 2 ** 31 - 1        # a window of every token


def on_device(device, call, *args):
    """call(*args) with `device` current: a stream of None is then that device's current stream,
    and the launch goes there whatever device the caller has current."""
    if device.index is None or device.index == torch.cuda.current_device():
        return call(*args)
    with torch.cuda.device(device):
        return call(*args)


def launch_stream(device, stream):
    """A context in which `stream` (a torch stream or a raw handle) is the current one: what is
    allocated and filled there is ordered before a launch on it.  None is the current stream."""
    if stream is None:
        return contextlib.nullcontext()
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=device) if stream else \
            torch.cuda.default_stream(device)
    return torch.cuda.stream(stream)


class DecodeLayer:
    """One layer's paged KV cache on a GPU and its decode step.

    k, v: fp16 [num_phys_pages][num_kv_heads][16][128]; page_table: int32 [B][max_pages] (logical
    page -> physical page, -1 unmapped); seq_lens: int32 [B].  Arrays on the host are copied to
    `device`.  budget_pages > 0 fixes the pages each head selects, else ceil(P_b / budget_div).
    Every call on a layer uses the layer's one workspace: issue them in order on one stream (the
    current stream when `stream` is None)."""

    def __init__(self, k, v, page_table, seq_lens, num_q_heads: int, num_kv_heads: int,
                 budget_pages: int = 0, budget_div: int = 4, device="cuda"):
        dev = torch.device(device)
        t = lambda x, dt: torch.as_tensor(x).to(device=dev, dtype=dt).contiguous()
        self.k = t(k, torch.float16)
        self.v = t(v, torch.float16)
        self.page_table = t(page_table, torch.int32)
        self.seq_lens = t(seq_lens, torch.int32)
        self.num_q_heads = num_q_heads
        self.num_kv_heads = num_kv_heads
        self.budget_pages = budget_pages
        self.budget_div = budget_div
        self.device = dev
        p_phys = self.k.shape[0]
        self.kv = twl.PagedKV(self.k, self.v, self.page_table, self.seq_lens, num_kv_heads,
                              p_phys)
        self.batch = self.kv.batch
        self.max_pages = self.kv.max_pages
        self.max_budget = budget_bound(self.max_pages, budget_pages, budget_div)
        self.aux = twl.KAux(
            torch.zeros((p_phys, num_kv_heads, 16, 64), dtype=torch.uint8, device=dev),
            torch.zeros((p_phys, num_kv_heads, 16, 2), dtype=torch.float16, device=dev),
            torch.zeros((p_phys, num_kv_heads, 2, 128), dtype=torch.float16, device=dev))
        self.ws = twl.alloc_workspace(twl.TWL_OP_DECODE_STEP, dev, batch=self.batch,
                                      num_q_heads=num_q_heads, num_kv_heads=num_kv_heads,
                                      max_pages=self.max_pages, max_budget=self.max_budget)
        self.o = torch.zeros((self.batch, num_q_heads, 128), dtype=torch.float32, device=dev)
        self.lse = torch.zeros((self.batch, num_q_heads), dtype=torch.float32, device=dev)
        self.ws_window = twl.alloc_workspace(twl.TWL_OP_WINDOW_DECODE, dev, batch=self.batch,
                                             num_q_heads=num_q_heads, num_kv_heads=num_kv_heads)
        # made by the first window_prefill (not during a capture), or set to another layer's: layers
        # of one shape whose calls run in order on one stream can share it
        self.ws_prefill = None
        self._pages = None
        self._centroids = None

    @classmethod
    def from_workload(cls, wl, device="cuda"):
        return cls(wl.k, wl.v, wl.page_table, wl.seq_lens, wl.num_q_heads, wl.num_kv_heads,
                   wl.budget_pages, wl.budget_div, device)

    # ------------------------------------------------------------------ cache maintenance
    def build_aux(self, stream=None) -> None:
        """INT4 K and page bounds for every referenced page."""
        twl.twl_quantize_k(self.kv, self.aux.k_int4, self.aux.k_scale_zero, self.ws, stream)
        twl.twl_page_bounds(self.kv, self.aux.bounds, self.ws, stream)

    def append(self, k_new, v_new, stream=None) -> None:
        """Append one token per sequence at position seq_lens[b] (K, V, INT4 K and page bounds
        in one launch) and advance seq_lens.  The page for the position must be mapped."""
        for name, t in (("k_new", k_new), ("v_new", v_new)):
            expect_tensor(name, t, (self.batch, self.num_kv_heads, 128), torch.float16,
                          self.k.device)
        twl.twl_append_token(self.kv, self.aux, k_new, v_new, True, self.ws, stream)

    # ------------------------------------------------------------------ stats buffers
    def alloc_stats(self) -> dict:
        b, hq, hkv, mb = self.batch, self.num_q_heads, self.num_kv_heads, self.max_budget
        dev, i32, f32 = self.device, torch.int32, torch.float32
        cs, us = 16 * mb, 16 * self.max_pages
        return dict(
            sel_pages=torch.full((b, hq, mb), -1, dtype=i32, device=dev),
            sel_count=torch.zeros((b, hq), dtype=i32, device=dev),
            weights=torch.zeros((b, hq, cs), dtype=f32, device=dev),
            cand_tok=torch.full((b, hq, cs), -1, dtype=i32, device=dev),
            cand_count=torch.zeros((b, hq), dtype=i32, device=dev),
            threshold=torch.zeros((b, hq), dtype=f32, device=dev),
            kept_count=torch.zeros((b, hq), dtype=i32, device=dev),
            union_tok=torch.full((b, hkv, us), -1, dtype=i32, device=dev),
            union_count=torch.zeros((b, hkv), dtype=i32, device=dev))

    # ------------------------------------------------------------------ the decode step
    def decode(self, q, p: float = 0.85, eps: float = 1e-6, stats: dict | None = None,
               stream=None):
        """One select -> estimate -> prune -> union -> attend step for query q [B][Hq][128] fp16
        (device tensor), one launch of the library's persistent step kernel.  Returns the
        layer's (o, lse) device tensors (o and lse are attributes a caller may point at slices
        of its own buffers)."""
        self.expect_query(q)
        st = twl.make_stats(**stats) if stats is not None else None
        twl.twl_decode_step(q, self.num_q_heads, self.kv, self.aux, self.budget_pages,
                            self.budget_div, self.max_budget, p, eps, self.o, self.lse, st,
                            self.ws, stream)
        return self.o, self.lse

    # ------------------------------------------------------------------ windowed attention
    def window_decode(self, q, sinks: int = 0, window: int = ALL_TOKENS, stream=None):
        """The last token of every sequence (already appended) attends to the first `sinks` tokens
        and the last `window` ones: q [B][Hq][128] fp16 -> the layer's (o, lse)."""
        self.expect_query(q)
        on_device(self.k.device, twl.twl_window_decode, q, self.num_q_heads, self.kv, sinks,
                  window, SM_SCALE, self.o, self.lse, self.ws_window, stream)
        return self.o, self.lse

    def window_prefill(self, q, q_start, sinks: int = 0, window: int = ALL_TOKENS, out=None,
                       stream=None):
        """Chunks of many tokens: rows q_start[b] .. q_start[b + 1] - 1 of q [T][Hq][128] fp16 are
        the last tokens of sequence b (already in its cache) and attend causally under the window.
        Returns (o fp16 [T][Hq][128], lse fp32 [T][Hq]), new tensors (made on the launch's stream)
        or the pair `out`; rows outside every chunk are not written."""
        dev = self.k.device
        if not isinstance(q, torch.Tensor) or q.dim() != 3:
            raise ValueError("q: expected a tensor [T][Hq][128]")
        expect_tensor("q", q, (q.shape[0], self.num_q_heads, 128), torch.float16, dev)
        expect_tensor("q_start", q_start, (self.batch + 1,), torch.int32, dev)
        if out is None and stream is None:
            out = (torch.empty_like(q), torch.empty(q.shape[:2], dtype=torch.float32, device=dev))
        elif out is None:
            with launch_stream(dev, stream):
                out = (torch.empty_like(q),
                       torch.empty(q.shape[:2], dtype=torch.float32, device=dev))
                capturing = torch.cuda.is_current_stream_capturing()
            if not capturing:
                for t in out:                  # the caller reads them on the current stream
                    t.record_stream(torch.cuda.current_stream(dev))
        o, lse = out
        expect_tensor("o", o, q.shape, torch.float16, dev)
        expect_tensor("lse", lse, q.shape[:2], torch.float32, dev)
        if self.ws_prefill is None:
            with launch_stream(dev, stream):
                if torch.cuda.is_current_stream_capturing():
                    raise RuntimeError("window_prefill: the layer's first call makes its "
                                       "workspace, so it cannot be captured")
                self.ws_prefill = twl.alloc_workspace(
                    twl.TWL_OP_WINDOW_PREFILL, dev, batch=self.batch,
                    num_q_heads=self.num_q_heads, num_kv_heads=self.num_kv_heads)
        on_device(dev, twl.twl_window_prefill, q, q_start, q.shape[0], self.num_q_heads, self.kv,
                  sinks, window, SM_SCALE, o, lse, self.ws_prefill, stream)
        return o, lse

    # ------------------------------------------------------------------ pages
    def pages(self) -> "PageManager":
        """The page manager of this layer's cache and its derived K data, the centroids of the
        two-level path among it once they exist (built on first use)."""
        if self._pages is None:
            more = [] if self._centroids is None else [self._centroids]
            self._pages = PageManager([self.k, self.v, self.aux.k_int4, self.aux.k_scale_zero,
                                       self.aux.bounds, *more], self.page_table, self.seq_lens)
        return self._pages

    def expect_query(self, q) -> None:
        """q must be fp16 [B][Hq][128], contiguous, on the layer's GPU."""
        expect_tensor("q", q, (self.batch, self.num_q_heads, 128), torch.float16, self.k.device)

    # ------------------------------------------------------------------ other paths
    def staged(self) -> "Staged":
        """The same step as five separate library calls (see Staged)."""
        return Staged(self)

    def centroids(self):
        """fp16 [num_phys_pages][num_kv_heads][128], made on first use: page centroids, filled by
        DoubleP.build_centroids.  They move and fork with their pages."""
        if self._centroids is None:
            self._centroids = torch.zeros((self.k.shape[0], self.num_kv_heads, 128),
                                          dtype=torch.float16, device=self.device)
            if self._pages is not None:
                self._pages.add(self._centroids)
        return self._centroids

    def double_p(self) -> "DoubleP":
        """The two-level top-p path on this layer's cache (built on first use)."""
        if getattr(self, "_double_p", None) is None:
            self._double_p = DoubleP(self)
        return self._double_p

    def status(self, clear: bool = False, stream=None):
        """(status, flags) of the layer's device flags, over all of its workspaces, behind the
        calls issued on `stream`, which it waits for."""
        got = [on_device(self.device, twl.twl_device_status, ws, clear, stream)
               for ws in (self.ws, self.ws_window, self.ws_prefill) if ws is not None]
        return next((st for st, _ in got if st != twl.TWL_OK), twl.TWL_OK), \
            got[0][1] | got[1][1] | (got[2][1] if len(got) > 2 else 0)


SM_SCALE = 1.0 / math.sqrt(128.0)


class Int4Layer:
    """One layer whose paged cache is held in 4 bits, and attention over it.

    k, v: uint8 codes [num_phys_pages][num_kv_heads][16][64]; k_sz, v_sz: fp16 scale and zero of
    every row [..][16][2]; page_table, seq_lens as DecodeLayer.  All are device tensors that the
    layer uses in place.  Issue the calls on a layer in order on one stream: they share its
    workspace."""

    def __init__(self, k, k_sz, v, v_sz, page_table, seq_lens, num_q_heads: int,
                 num_kv_heads: int):
        if not isinstance(k, torch.Tensor) or k.dim() != 4:
            raise ValueError("k: expected a tensor [P][Hkv][16][64]")
        dev, p_phys = k.device, k.shape[0]
        for name, t in (("k", k), ("v", v)):
            expect_tensor(name, t, (p_phys, num_kv_heads, 16, 64), torch.uint8, dev)
        for name, t in (("k_sz", k_sz), ("v_sz", v_sz)):
            expect_tensor(name, t, (p_phys, num_kv_heads, 16, 2), torch.float16, dev)
        expect_table(page_table, seq_lens, dev)
        self.k, self.k_sz, self.v, self.v_sz = k, k_sz, v, v_sz
        self.page_table, self.seq_lens = page_table, seq_lens
        self.num_q_heads, self.num_kv_heads = num_q_heads, num_kv_heads
        self.device = dev
        self.kv = twl.Int4KV(k, k_sz, v, v_sz, page_table, seq_lens, num_kv_heads, p_phys)
        self.batch = self.kv.batch
        self.o = torch.zeros((self.batch, num_q_heads, 128), dtype=torch.float32, device=dev)
        self.lse = torch.zeros((self.batch, num_q_heads), dtype=torch.float32, device=dev)
        # behind the other buffers: they too are filled once it is there
        self.ws = twl.alloc_workspace(twl.TWL_OP_INT4_DECODE, dev, batch=self.batch,
                                      num_q_heads=num_q_heads, num_kv_heads=num_kv_heads)
        self._pages = None

    @classmethod
    def from_fp16(cls, k, v, page_table, seq_lens, num_q_heads: int, num_kv_heads: int,
                  stream=None):
        """The layer of an fp16 cache (device tensors, layout of DecodeLayer): quantises K and V
        of every page the sequences use, on `stream`, where the layer's buffers are made too."""
        if not isinstance(k, torch.Tensor) or k.dim() != 4:
            raise ValueError("k: expected a tensor [P][Hkv][16][128]")
        dev, p_phys = k.device, k.shape[0]
        for name, t in (("k", k), ("v", v)):
            expect_tensor(name, t, (p_phys, num_kv_heads, 16, 128), torch.float16, dev)
        expect_table(page_table, seq_lens, dev)
        with launch_stream(dev, stream):      # the zeros before the rows, on one stream
            made = []
            for x in (k, v):
                codes = torch.zeros((p_phys, num_kv_heads, 16, 64), dtype=torch.uint8, device=dev)
                sz = torch.zeros((p_phys, num_kv_heads, 16, 2), dtype=torch.float16, device=dev)
                on_device(dev, twl.twl_quantize_k, twl.PagedKV(x, x, page_table, seq_lens,
                                                               num_kv_heads, p_phys),
                          codes, sz, None, stream)
                made += [codes, sz]
            return cls(*made, page_table, seq_lens, num_q_heads, num_kv_heads)

    def decode(self, q, k_new=None, v_new=None, sinks: int = 0, window: int = ALL_TOKENS,
               advance: bool = True, stream=None):
        """Appends the token (k_new, v_new) [B][Hkv][128] fp16 of every sequence in 4 bits (its
        page must be mapped) and attends from it, in one launch: q [B][Hq][128] fp16 -> the
        layer's (o, lse).  With advance, seq_lens moves on.  Without k_new and v_new the last
        cached token attends and nothing is written."""
        dev = self.device
        expect_tensor("q", q, (self.batch, self.num_q_heads, 128), torch.float16, dev)
        if (k_new is None) != (v_new is None):
            raise ValueError("k_new and v_new go together")
        if k_new is not None:
            for name, t in (("k_new", k_new), ("v_new", v_new)):
                expect_tensor(name, t, (self.batch, self.num_kv_heads, 128), torch.float16, dev)
        on_device(dev, twl.twl_int4_decode, q, self.num_q_heads, self.kv, k_new, v_new,
                  advance and k_new is not None, sinks, window, SM_SCALE, self.o, self.lse,
                  self.ws, stream)
        return self.o, self.lse

    def pages(self) -> "PageManager":
        """The page manager of this layer's cache (built on first use)."""
        if self._pages is None:
            self._pages = PageManager([self.k, self.k_sz, self.v, self.v_sz], self.page_table,
                                      self.seq_lens)
        return self._pages

    def status(self, clear: bool = False, stream=None):
        """(status, flags) of the device flags, behind the calls issued on `stream`, which it
        waits for."""
        return on_device(self.device, twl.twl_device_status, self.ws, clear, stream)


def expect_table(page_table, seq_lens, device) -> None:
    """page_table int32 [B][max_pages] and seq_lens int32 [B], contiguous, on `device`."""
    if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2:
        raise ValueError("page_table: expected a tensor [B][max_pages]")
    expect_tensor("page_table", page_table, page_table.shape, torch.int32, device)
    expect_tensor("seq_lens", seq_lens, page_table.shape[:1], torch.int32, device)


class PageManager:
    """The pages of one page table and of every pool (tensor [num_phys_pages][...]) it indexes:
    the K and V of one layer, or of all layers that share the table.  Uses the tensors in place.
    A pool's page is a multiple of 16 bytes, 16-byte aligned; any number of pools will do.
    A page is in use when the table names it; nothing else is kept.  Issue the calls in order on
    one stream, the one that the attention calls on the same cache use."""

    def __init__(self, pools, page_table, seq_lens):
        pools = list(pools)
        if not pools or not all(isinstance(t, torch.Tensor) and t.dim() >= 1 for t in pools):
            raise ValueError("pools: expected tensors [num_phys_pages][...]")
        dev, p_phys = pools[0].device, pools[0].shape[0]
        self.device, self.num_phys_pages = dev, p_phys
        for t in pools:
            self._expect_pool(t)
        expect_table(page_table, seq_lens, dev)
        self.pools, self.page_table, self.seq_lens = pools, page_table, seq_lens
        self.batch, self.max_pages = page_table.shape
        self.num_used = torch.zeros((), dtype=torch.int32, device=dev)
        # table and lengths that the calls for pools behind the first TWL_MAX_POOLS work on
        self._copies = None
        self._make_copies()
        self.ws = twl.alloc_workspace(twl.TWL_OP_PAGES, dev, batch=self.batch,
                                      max_pages=self.max_pages, rows=p_phys)

    def _expect_pool(self, t) -> None:
        p_phys = self.num_phys_pages
        expect_tensor("pool", t, (p_phys, *t.shape[1:]), t.dtype, self.device)
        if t.nbytes == 0 or t.nbytes // p_phys % 16 or (not t.is_meta and t.data_ptr() % 16):
            raise ValueError("pool: expected pages of a multiple of 16 bytes, 16-byte aligned, "
                             f"got {t.nbytes} bytes in {p_phys} pages")

    def _make_copies(self) -> None:
        if len(self.pools) > twl.TWL_MAX_POOLS and self._copies is None:
            self._copies = torch.empty_like(self.page_table), torch.empty_like(self.seq_lens)

    def add(self, pool) -> None:
        """One more pool [num_phys_pages][...] that the table indexes, from the next call on (a
        captured call keeps the pools it was captured with)."""
        if not isinstance(pool, torch.Tensor) or pool.dim() < 1:
            raise ValueError("pool: expected a tensor [num_phys_pages][...]")
        self._expect_pool(pool)
        self.pools.append(pool)
        self._make_copies()

    def remap(self, parent, reserve=None, sinks: int = 0, window: int = ALL_TOKENS,
              stream=None) -> None:
        """One page-table step: slot b goes on as parent[b]'s sequence (itself, a fork of another
        slot, or -1: freed) with pages for reserve[b] more tokens; pages that no later query sees
        under (sinks, window) are dropped.  parent, reserve: int32 [B] device tensors.  A step
        that cannot be carried out changes nothing and shows in status()."""
        expect_tensor("parent", parent, (self.batch,), torch.int32, self.device)
        if reserve is not None:
            expect_tensor("reserve", reserve, (self.batch,), torch.int32, self.device)
        args = self.num_phys_pages, parent, reserve, sinks, window, self.ws, stream
        # a call's outcome follows from table, lengths and arguments alone: it is the same for all
        for pools in self._further():
            with launch_stream(self.device, stream):
                for copy, of in zip(self._copies, (self.page_table, self.seq_lens)):
                    copy.copy_(of)
            on_device(self.device, twl.twl_remap_pages, pools, *self._copies, *args)
        on_device(self.device, twl.twl_remap_pages, self._first(), self.page_table, self.seq_lens,
                  *args)

    def compact(self, table_out=None, stream=None):
        """Moves the used pages to the front of the pools.  The table with the new numbers goes to
        table_out, or replaces the page table.  Returns the manager's device scalar with the
        number of used pages."""
        if table_out is None:
            table_out = self.page_table
        expect_tensor("table_out", table_out, self.page_table.shape, torch.int32, self.device)
        args = self.num_phys_pages, self.num_used, self.ws, stream
        for pools in self._further():
            on_device(self.device, twl.twl_compact_pages, pools, self.page_table,
                      self._copies[0], *args)
        on_device(self.device, twl.twl_compact_pages, self._first(), self.page_table, table_out,
                  *args)
        return self.num_used

    def _first(self):
        """The pools that one call takes ..."""
        return self.pools if self._copies is None else self.pools[:twl.TWL_MAX_POOLS]

    def _further(self):
        """... and those behind them, in lists that a call takes."""
        if self._copies is None:
            return ()
        n = twl.TWL_MAX_POOLS
        return [self.pools[i:i + n] for i in range(n, len(self.pools), n)]

    def status(self, clear: bool = False, stream=None):
        """(status, flags) of the device flags, behind the calls issued on `stream`, which it
        waits for."""
        return on_device(self.device, twl.twl_device_status, self.ws, clear, stream)


class DoubleP:
    """The two-level top-p step: top-p over page clusters scored by size-weighted centroids
    (twl_select_clusters_top_p), then the token-level path on the kept pages: INT4 estimate,
    top-p prune, group union, sparse attention.  Five library calls; this class only owns the
    buffers between them."""

    def __init__(self, layer: DecodeLayer):
        self.layer = layer
        L, dev = layer, layer.device
        b, hq, hkv, mp = L.batch, L.num_q_heads, L.num_kv_heads, L.max_pages
        i32, f32 = torch.int32, torch.float32
        self.centroids = L.centroids()
        self.sel = torch.full((b, hq, mp), -1, dtype=i32, device=dev)
        self.sel_count = torch.zeros((b, hq), dtype=i32, device=dev)
        self.cluster_w = torch.zeros((b, hq, mp), dtype=f32, device=dev)
        cs = 16 * mp
        self.weights = torch.zeros((b, hq, cs), dtype=f32, device=dev)
        self.cand_tok = torch.full((b, hq, cs), -1, dtype=i32, device=dev)
        self.cand_count = torch.zeros((b, hq), dtype=i32, device=dev)
        self.m = torch.zeros(b * hq, dtype=f32, device=dev)
        self.kept_count = torch.zeros(b * hq, dtype=i32, device=dev)
        self.kept_idx = torch.zeros((b * hq, cs), dtype=i32, device=dev)
        self.union_tok = torch.full((b, hkv, cs), -1, dtype=i32, device=dev)
        self.union_count = torch.zeros((b, hkv), dtype=i32, device=dev)
        dims = dict(batch=b, num_q_heads=hq, num_kv_heads=hkv, max_pages=mp, max_budget=mp)
        self.ws_sel = twl.alloc_workspace(twl.TWL_OP_SELECT_CLUSTERS, dev, **dims)
        self.ws_est = twl.alloc_workspace(twl.TWL_OP_ESTIMATE, dev, **dims)
        self.ws_att = twl.alloc_workspace(twl.TWL_OP_SPARSE_DECODE, dev, batch=b, num_q_heads=hq,
                                          num_kv_heads=hkv, row_stride=cs)
        self.ws_cache = twl.alloc_workspace(twl.TWL_OP_CACHE, dev)

    def build_centroids(self, stream=None) -> None:
        twl.twl_page_centroids(self.layer.kv, self.centroids, self.ws_cache, stream)

    def decode(self, q, p_cluster: float = 0.95, p: float = 0.85, eps: float = 1e-6,
               stream=None):
        L = self.layer
        L.expect_query(q)
        hq, mp = L.num_q_heads, L.max_pages
        cs = 16 * mp
        twl.twl_select_clusters_top_p(q, hq, L.kv, self.centroids, p_cluster, eps, self.sel,
                                      self.sel_count, self.cluster_w, self.ws_sel, stream)
        twl.twl_estimate(q, hq, L.kv, L.aux.k_int4, L.aux.k_scale_zero, self.sel,
                         self.sel_count, mp, self.weights, self.cand_tok, self.cand_count,
                         self.ws_est, stream)
        rows = L.batch * hq
        twl.twl_prune_top_p(self.weights.view(rows, cs), self.cand_count.view(rows), rows, cs,
                            p, eps, self.m, self.kept_count, self.kept_idx, None, stream)
        twl.twl_group_union(hq, L.kv, self.cand_tok, self.kept_idx, self.kept_count, cs,
                            self.union_tok, self.union_count, None, stream)
        twl.twl_sparse_decode(q, hq, L.kv, self.union_tok, self.union_count, cs, SM_SCALE, L.o,
                              L.lse, self.ws_att, stream)
        return L.o, L.lse


class Staged:
    """The decode step as its five staged library calls (twl_select_pages, twl_estimate,
    twl_prune_top_p, twl_group_union, twl_sparse_decode) instead of the one fused launch: the
    comparison the flattened per-stage work lists give.  Only owns the buffers between calls."""

    def __init__(self, layer: DecodeLayer):
        self.layer = layer
        L, dev = layer, layer.device
        b, hq, hkv, mb = L.batch, L.num_q_heads, L.num_kv_heads, L.max_budget
        i32, f32 = torch.int32, torch.float32
        cs = 16 * mb
        self.sel = torch.full((b, hq, mb), -1, dtype=i32, device=dev)
        self.sel_count = torch.zeros((b, hq), dtype=i32, device=dev)
        self.weights = torch.zeros((b, hq, cs), dtype=f32, device=dev)
        self.cand_tok = torch.full((b, hq, cs), -1, dtype=i32, device=dev)
        self.cand_count = torch.zeros((b, hq), dtype=i32, device=dev)
        self.m = torch.zeros(b * hq, dtype=f32, device=dev)
        self.kept_count = torch.zeros(b * hq, dtype=i32, device=dev)
        self.kept_idx = torch.zeros((b * hq, cs), dtype=i32, device=dev)
        us = 16 * L.max_pages  # union rows: up to every token of the sequence
        self.union_tok = torch.full((b, hkv, us), -1, dtype=i32, device=dev)
        self.union_count = torch.zeros((b, hkv), dtype=i32, device=dev)
        dims = dict(batch=b, num_q_heads=hq, num_kv_heads=hkv, max_pages=L.max_pages,
                    max_budget=mb)
        self.ws_sel = twl.alloc_workspace(twl.TWL_OP_SELECT, dev, **dims)
        self.ws_est = twl.alloc_workspace(twl.TWL_OP_ESTIMATE, dev, **dims)
        self.ws_att = twl.alloc_workspace(twl.TWL_OP_SPARSE_DECODE, dev, batch=b, num_q_heads=hq,
                                          num_kv_heads=hkv, row_stride=us)

    def decode(self, q, p: float = 0.85, eps: float = 1e-6, stream=None):
        L = self.layer
        L.expect_query(q)
        hq, mb = L.num_q_heads, L.max_budget
        cs = 16 * mb
        twl.twl_select_pages(q, hq, L.kv, L.aux.bounds, L.budget_pages, L.budget_div, mb,
                             self.sel, self.sel_count, None, self.ws_sel, stream)
        twl.twl_estimate(q, hq, L.kv, L.aux.k_int4, L.aux.k_scale_zero, self.sel,
                         self.sel_count, mb, self.weights, self.cand_tok, self.cand_count,
                         self.ws_est, stream)
        rows = L.batch * hq
        twl.twl_prune_top_p(self.weights.view(rows, cs), self.cand_count.view(rows), rows, cs,
                            p, eps, self.m, self.kept_count, self.kept_idx, None, stream)
        twl.twl_group_union(hq, L.kv, self.cand_tok, self.kept_idx, self.kept_count, cs,
                            self.union_tok, self.union_count, None, stream)
        twl.twl_sparse_decode(q, hq, L.kv, self.union_tok, self.union_count, 16 * L.max_pages,
                              SM_SCALE, L.o, L.lse, self.ws_att, stream)
        return L.o, L.lse
