"""The cache operators and how they are measured: attention of one token or of prompt chunks over a
sliding window with sink tokens, attention over a cache held in 4 bits, and the page-table step and
compaction that manage the cache's pages.

``run`` computes an operator in its plain form (elementary torch operations in 32 bits), or, with
``own`` set, through the library.  ``exact`` computes it from its definition in 64 bits.
Shapes: head_dim 128, 16-token pages, fp16 K and V [P][Hkv][16][128] (or 4-bit codes with an fp16
scale and zero per row), page table int32 [B][max_pages], lengths int32 [B].
"""
import math
import random

import torch

own = False

D, PAGE = 128, 16
ALL = 2 ** 31 - 1               # a window of every token
SCALE = 1.0 / math.sqrt(D)
DEV = "cuda"


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one token of one sequence at 32K context, a streaming window: latency
        dict(name="window_decode_1x32k", op="window_decode", batch=1, hq=32, hkv=8, min_len=32768,
             max_len=32768, sinks=4, window=1024),
        # a serving batch with ragged lengths, every token visible: bandwidth
        dict(name="window_decode_16_ragged", op="window_decode", batch=16, hq=32, hkv=8,
             min_len=8192, max_len=32768, sinks=0, window=ALL),
        # verification of a few drafted tokens per sequence behind long contexts
        dict(name="prefill_verify", op="window_prefill", batch=8, hq=32, hkv=8, min_q=1, max_q=8,
             min_len=2000, max_len=8192, sinks=4, window=4096),
        # one long prompt, a window with sinks
        dict(name="prefill_8k_window", op="window_prefill", batch=1, hq=32, hkv=8, min_q=8192,
             max_q=8192, min_len=8192, max_len=8192, sinks=4, window=2048),
        # ragged prompt chunks of several sequences over what they have cached, causal
        dict(name="prefill_4_chunks", op="window_prefill", batch=4, hq=32, hkv=8, min_q=1500,
             max_q=2048, min_len=2048, max_len=8192, sinks=0, window=ALL),
        # one token over a 4-bit cache, batch 1: latency and split
        dict(name="int4_decode_1x32k", op="int4_decode", batch=1, hq=32, hkv=8, min_len=32768,
             max_len=32768, sinks=0, window=ALL),
        # a serving batch over a 4-bit cache: bandwidth
        dict(name="int4_decode_64x8k", op="int4_decode", batch=64, hq=32, hkv=8, min_len=8192,
             max_len=8192, sinks=0, window=ALL),
        # groups of 8 heads, ragged lengths, a window with sinks
        dict(name="int4_decode_window", op="int4_decode", batch=16, hq=64, hkv=8, min_len=5000,
             max_len=32768, sinks=4, window=4000),
        # beams of short sequences change their parents and get a page for the next token
        dict(name="remap_beams", op="remap_pages", batch=8, hkv=8, min_len=200, max_len=1000,
             forks=5, frees=0, reserve=1, sinks=0, window=ALL, spare=64),
        # a serving batch forks, frees and grows, and drops what fell out of its window
        dict(name="remap_serving", op="remap_pages", batch=256, hkv=8, min_len=100, max_len=4000,
             forks=100, frees=20, reserve=16, sinks=4, window=2000, spare=4096),
        # a small pool, three quarters free
        dict(name="compact_512", op="compact_pages", batch=8, hkv=8, pages=512, used=128),
        # a large pool, half of it free: bandwidth
        dict(name="compact_32k", op="compact_pages", batch=64, hkv=8, pages=32768, used=16384),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["window_decode", "window_prefill", "int4_decode", "remap_pages",
                     "compact_pages"])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 4, 8])
    sinks = rng.choice([0, 1, 4, 17, 64])
    window = rng.choice([ALL, _log(rng, 1, 8192), _log(rng, 64, 4096)])
    if op in ("window_decode", "int4_decode"):
        batch = _log(rng, 1, 64)
        # tokens x kv-heads of the batch at most those of the largest case of this operator
        most = min(131072, (2560000 if op == "window_decode" else 4000000) // (batch * hkv))
        hi = _log(rng, 17, max(18, most))
        return dict(op=op, batch=batch, hq=hq, hkv=hkv, min_len=_log(rng, 1, hi), max_len=hi,
                    sinks=sinks, window=window)
    if op == "window_prefill":
        batch = _log(rng, 1, 16)
        max_q = _log(rng, 1, 8192)
        hi = _log(rng, max_q, max(max_q, 16384))
        while batch * max_q * hi * hq > 1 << 30:       # score elements of the padded batch
            if batch > 1:
                batch = max(1, batch // 2)
            elif hq > hkv:
                hq //= 2
            elif hkv > 1:
                hkv //= 2
                hq //= 2
            else:
                max_q, hi = max(1, max_q // 2), max(1, hi // 2)
        return dict(op=op, batch=batch, hq=hq, hkv=hkv, min_q=_log(rng, 1, max_q), max_q=max_q,
                    min_len=max_q, max_len=hi, sinks=sinks, window=window)
    if op == "remap_pages":
        batch = _log(rng, 2, 256)
        hi = _log(rng, 20, min(16000, 1000000 // batch))
        forks = rng.randint(0, batch - 1)
        return dict(op=op, batch=batch, hkv=hkv, min_len=_log(rng, 1, hi), max_len=hi, forks=forks,
                    frees=rng.randint(0, batch - 1 - forks), reserve=rng.choice([1, 5, 16, 100]),
                    sinks=sinks, window=window, spare=batch * 9)
    pages = _log(rng, 40, 32768)
    return dict(op=op, batch=_log(rng, 1, 64), hkv=hkv, pages=pages,
                used=max(1, int(pages * rng.uniform(0.1, 0.95))))


# ------------------------------------------------------------------ inputs
def _lens(case):
    """(cached lengths, chunk lengths) of the sequences: spread over the case's ranges, the first
    ones the longest.  They belong to the case and not to the seed, so that outputs of two seeds
    have one shape."""
    r = random.Random("%d %d %d" % (case["batch"], case["min_len"], case["max_len"]))
    lens = [r.randint(case["min_len"], case["max_len"]) for _ in range(case["batch"])]
    lens[0] = case["max_len"]
    if case["op"] != "window_prefill":
        return lens, None
    qn = [r.randint(case["min_q"], case["max_q"]) for _ in lens]
    qn[0] = case["max_q"]
    return [max(n, m) for n, m in zip(lens, qn)], qn


def _tables(g, lens, extra_pages, spare):
    """Every sequence's pages, dealt from one random permutation of the pool; -1 where unmapped."""
    need = [-(-n // PAGE) for n in lens]
    max_pages = max(need) + extra_pages
    total = sum(need) + spare
    perm = torch.randperm(total, generator=g).to(torch.int32)
    table = torch.full((len(lens), max_pages), -1, dtype=torch.int32)
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = perm[at:at + m]
        at += m
    return table, total


def _normal(seed, *shape):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float16)


def _queries(g, seed, rows, hq):
    """Queries of heads between focused and diffuse: N(0, I) over a logit temperature that is
    log-uniform in [0.25, 8]."""
    tau = torch.exp(torch.rand(hq, generator=g) * math.log(32.0) + math.log(0.25)).to(DEV)
    return (_normal(seed, rows, hq, D).float() / tau[None, :, None]).half()


def _quantise(x):
    """Packed 4-bit codes [..., 64] and (scale, zero) fp16 [..., 2] of fp16 rows [..., 128]."""
    f = x.float()
    lo, hi = f.amin(-1, keepdim=True), f.amax(-1, keepdim=True)
    s = ((hi - lo) / 15.0).half()
    code = torch.round((f - lo) / s.float()).clamp(0, 15)
    code = torch.where(s == 0, torch.zeros_like(code), code).to(torch.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), torch.cat([s, lo.half()], -1)


def _quantised_pool(seed, pages, hkv):
    codes, szs, step = [], [], 4096
    for at in range(0, pages, step):
        c, s = _quantise(_normal(seed + 7919 * at, min(step, pages - at), hkv, PAGE, D))
        codes.append(c)
        szs.append(s)
    return torch.cat(codes), torch.cat(szs)


def prepare(case, seed):
    g = torch.Generator().manual_seed(seed)
    st = dict(case)
    op, hkv, batch = case["op"], case["hkv"], case["batch"]
    if op in ("window_decode", "int4_decode"):
        lens, _ = _lens(case)
        append = op == "int4_decode"          # the new token goes behind the cached ones
        table, pages = _tables(g, [n + 1 for n in lens] if append else lens, 0, 0)
        st.update(table=table.to(DEV), lens=torch.tensor(lens, dtype=torch.int32, device=DEV),
                  q=_queries(g, seed + 1, batch, case["hq"]))
        if append:
            st["kc"], st["ks"] = _quantised_pool(seed + 2, pages, hkv)
            st["vc"], st["vs"] = _quantised_pool(seed + 3, pages, hkv)
            st["k_new"] = _normal(seed + 4, batch, hkv, D)
            st["v_new"] = _normal(seed + 5, batch, hkv, D)
        else:
            st["k"] = _normal(seed + 2, pages, hkv, PAGE, D)
            st["v"] = _normal(seed + 3, pages, hkv, PAGE, D)
        if own:
            from adaptive_top_sparse_b200 import layer
            if append:
                st["layer"] = layer.Int4Layer(st["kc"], st["ks"], st["vc"], st["vs"], st["table"],
                                              st["lens"], case["hq"], hkv)
            else:
                st["layer"] = layer.DecodeLayer(st["k"], st["v"], st["table"], st["lens"],
                                                case["hq"], hkv)
    elif op == "window_prefill":
        lens, qn = _lens(case)
        table, pages = _tables(g, lens, 0, 0)
        start = torch.tensor([0] + qn).cumsum(0).to(torch.int32)
        total = int(start[-1])
        st.update(table=table.to(DEV), lens=torch.tensor(lens, dtype=torch.int32, device=DEV),
                  q=_queries(g, seed + 1, total, case["hq"]), start=start.to(DEV),
                  k=_normal(seed + 2, pages, hkv, PAGE, D),
                  v=_normal(seed + 3, pages, hkv, PAGE, D),
                  longest_q=max(qn), longest=max(lens))
        if own:
            from adaptive_top_sparse_b200 import layer
            st["layer"] = layer.DecodeLayer(st["k"], st["v"], st["table"], st["lens"],
                                            case["hq"], hkv)
    elif op == "remap_pages":
        lens, _ = _lens(case)
        reserve = torch.randint(0, case["reserve"] + 1, (batch,), generator=g)
        extra = -(-case["reserve"] // PAGE) + 1
        # room for the partial pages of the forks and for every slot's reserved tokens
        spare = case["spare"] + batch * (extra + 1)
        table, pages = _tables(g, lens, extra, spare)
        slots = torch.randperm(batch, generator=g).tolist()
        nf, nd = case["forks"], case["frees"]
        kept = slots[nf + nd:]
        parent = torch.arange(batch)
        for b in slots[:nf]:
            parent[b] = kept[int(torch.randint(0, len(kept), (1,), generator=g))]
        for b in slots[nf:nf + nd]:
            parent[b] = -1
        reserve[slots[nf:nf + nd]] = 0
        st.update(table=table.to(DEV), lens=torch.tensor(lens, dtype=torch.int32, device=DEV),
                  parent=parent.to(torch.int32).to(DEV), extra=reserve.to(torch.int32).to(DEV),
                  k=_normal(seed + 2, pages, hkv, PAGE, D),
                  v=_normal(seed + 3, pages, hkv, PAGE, D))
        if own:
            from adaptive_top_sparse_b200 import layer
            st["pages"] = layer.PageManager([st["k"], st["v"]], st["table"], st["lens"])
    else:
        # the used pages lie anywhere in the pool; some are shared by two sequences
        pages, used = case["pages"], case["used"]
        ids = torch.randperm(pages, generator=g)[:used].to(torch.int32)
        per = -(-used // batch)
        table = torch.full((batch, per + 8), -1, dtype=torch.int32)
        for b in range(batch):
            mine = ids[b * per:(b + 1) * per]
            table[b, :len(mine)] = mine
            table[b, len(mine):len(mine) + min(8, used)] = ids[:8]
        st.update(table=table.to(DEV), table_out=torch.empty_like(table, device=DEV),
                  lens=torch.full((batch,), 16 * (per + 8), dtype=torch.int32, device=DEV),
                  k=_normal(seed + 2, pages, hkv, PAGE, D),
                  v=_normal(seed + 3, pages, hkv, PAGE, D))
        if own:
            from adaptive_top_sparse_b200 import layer
            st["pages"] = layer.PageManager([st["k"], st["v"]], st["table"], st["lens"])
    return st


# ------------------------------------------------------------------ one pass
def run(st):
    op = st["op"]
    if own:
        if op == "window_decode":
            return list(st["layer"].window_decode(st["q"], st["sinks"], st["window"]))
        if op == "window_prefill":
            return list(st["layer"].window_prefill(st["q"], st["start"], st["sinks"],
                                                   st["window"]))
        if op == "int4_decode":
            o, lse = st["layer"].decode(st["q"], st["k_new"], st["v_new"], st["sinks"],
                                        st["window"], advance=False)
            return [o, lse, st["ks"], st["vs"]]
        if op == "remap_pages":
            st["pages"].remap(st["parent"], st["extra"], st["sinks"], st["window"])
            return [st["table"], st["lens"], st["k"], st["v"]]
        used = st["pages"].compact(st["table_out"])
        return [st["table_out"], used, st["k"], st["v"]]
    if op == "window_decode":
        return _plain_decode(st, st["lens"].long(), _rows_fp16)
    if op == "window_prefill":
        return _plain_prefill(st)
    if op == "int4_decode":
        _plain_append(st)
        return _plain_decode(st, st["lens"].long() + 1, _rows_int4) + [st["ks"], st["vs"]]
    if op == "remap_pages":
        return _plain_remap(st)
    return _plain_compact(st)


def _rows_fp16(st, page, row):
    """K and V rows [B][T][Hkv][128] in 32 bits at physical pages and rows [B][T]."""
    return st["k"][page, :, row].float(), st["v"][page, :, row].float()


def _rows_int4(st, page, row):
    def rows(codes, sz):
        c = codes[page, :, row]
        s = sz[page, :, row].float()
        n = torch.stack([c & 15, c >> 4], -1).flatten(-2).float()
        return n * s[..., :1] + s[..., 1:]
    return rows(st["kc"], st["ks"]), rows(st["vc"], st["vs"])


def _plain_append(st):
    n = st["lens"].long()
    page = st["table"].gather(1, (n // PAGE)[:, None])[:, 0].long()
    for x, codes, sz in ((st["k_new"], st["kc"], st["ks"]), (st["v_new"], st["vc"], st["vs"])):
        c, s = _quantise(x)
        codes[page, :, n % PAGE] = c
        sz[page, :, n % PAGE] = s


def _plain_decode(st, n, rows):
    """The token at position n - 1 of each sequence attends to the sinks and its window."""
    batch, hq, hkv = st["batch"], st["hq"], st["hkv"]
    longest = st["max_len"] + (1 if rows is _rows_int4 else 0)
    tail = min(st["window"], longest)
    first = torch.clamp(n - tail, min=0)                     # the window's first position
    ns = min(st["sinks"], longest)
    sink = torch.arange(ns, device=DEV)[None, :].expand(batch, ns)
    win = first[:, None] + torch.arange(tail, device=DEV)[None, :]
    pos = torch.cat([sink, win], 1)
    seen = torch.cat([sink < torch.minimum(first, n)[:, None], win < n[:, None]], 1)
    pos = torch.where(seen, pos, torch.zeros_like(pos))
    page = torch.clamp(st["table"].gather(1, pos // PAGE).long(), min=0)
    k, v = rows(st, page, pos % PAGE)
    q = st["q"].float().view(batch, hkv, hq // hkv, D)
    s = torch.matmul(q, k.permute(0, 2, 3, 1)) * SCALE        # [B][Hkv][G][T]
    s = s.masked_fill(~seen[:, None, None, :], float("-inf"))
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - m)
    z = p.sum(-1, keepdim=True)
    o = torch.matmul(p / z, v.permute(0, 2, 1, 3))
    return [o.reshape(batch, hq, D), (m + torch.log(z)).reshape(batch, hq)]


def _plain_prefill(st):
    """The last q_len tokens of each sequence attend causally to the sinks and their windows."""
    batch, hq, hkv = st["batch"], st["hq"], st["hkv"]
    n, start = st["lens"].long(), st["start"].long()
    qn = start[1:] - start[:-1]
    lq, lk = st["longest_q"], st["longest"]
    i = torch.arange(lq, device=DEV)[None, :]
    valid = i < qn[:, None]
    row = torch.where(valid, start[:-1, None] + i, torch.zeros_like(i))
    q = st["q"][row].float().view(batch, lq, hkv, hq // hkv, D).permute(0, 2, 3, 1, 4)
    j = torch.arange(lk, device=DEV)
    page = torch.clamp(st["table"].gather(1, (j // PAGE)[None, :].expand(batch, lk)).long(), min=0)
    k, v = _rows_fp16(st, page, (j % PAGE)[None, :].expand(batch, lk))
    t = (n - qn)[:, None] + i                                 # positions of the query rows
    seen = (j <= t[..., None]) & ((j < st["sinks"]) | (j > t[..., None] - st["window"]))
    s = torch.matmul(q, k.permute(0, 2, 3, 1)[:, :, None]) * SCALE
    s.masked_fill_(~seen[:, None, None], float("-inf"))
    m = s.amax(-1, keepdim=True)
    p = s.sub_(m).exp_()
    z = p.sum(-1, keepdim=True)
    o = torch.matmul(p.div_(z), v.permute(0, 2, 1, 3)[:, :, None])
    o = o.permute(0, 3, 1, 2, 4).reshape(batch, lq, hq, D)
    lse = (m + torch.log(z))[..., 0].permute(0, 3, 1, 2).reshape(batch, lq, hq)
    return [o[valid].half(), lse[valid]]


def _plain_remap(st):
    table, lens = st["table"].long(), st["lens"].long()
    parent = st["parent"].long()
    batch, max_pages = table.shape
    b, j = torch.arange(batch, device=DEV), torch.arange(max_pages, device=DEV)[None, :]
    src = parent.clamp(min=0)
    n = torch.where(parent >= 0, lens[src], torch.zeros_like(lens))[:, None]
    rows = table[src]
    need = (n + st["extra"].long()[:, None] + PAGE - 1) // PAGE
    partial = (j == n // PAGE) & (n % PAGE != 0)
    out = (PAGE * j >= st["sinks"]) & (PAGE * j + PAGE - 1 <= n - st["window"]) & ~partial
    hold = (parent >= 0)[:, None] & (j < (n + PAGE - 1) // PAGE) & ~out
    # the partial page stays with the parent's own slot, else with its lowest fork
    key = torch.where(parent == b, torch.full_like(b, -1), b)
    first = torch.full((batch,), batch, device=DEV).scatter_reduce(0, src, torch.where(
        parent >= 0, key, torch.full_like(key, batch)), "amin")
    copy = hold & partial & (first[src] != key)[:, None] & (rows >= 0)
    mine = (parent == b)[:, None] & (j >= (n + PAGE - 1) // PAGE) & (j < need)
    new = torch.where((hold & ~copy) | mine, rows, torch.full_like(rows, -1))
    want = copy | ((j >= n // PAGE) & (j < need) & (new < 0))
    used = torch.zeros(st["k"].shape[0], dtype=torch.bool, device=DEV)
    used[new[new >= 0]] = True
    free = torch.nonzero(~used)[:, 0]
    at = torch.nonzero(want)
    new[at[:, 0], at[:, 1]] = free[:at.shape[0]]
    for pool in (st["k"], st["v"]):
        pool[new[copy]] = pool[rows[copy]]
    st["table"].copy_(new)
    st["lens"].copy_(n[:, 0])
    return [st["table"], st["lens"], st["k"], st["v"]]


def _plain_compact(st):
    table, pages = st["table"].long(), st["k"].shape[0]
    used = torch.zeros(pages, dtype=torch.bool, device=DEV)
    used[table[table >= 0]] = True
    count = used.sum()
    ids = torch.arange(pages, device=DEV)
    movers = torch.nonzero(used & (ids >= count))[:, 0]
    holes = torch.nonzero(~used & (ids < count))[:, 0]
    ids[movers] = holes
    for pool in (st["k"], st["v"]):
        pool[holes] = pool[movers]
    st["table_out"].copy_(torch.where(table >= 0, ids[table.clamp(min=0)], table))
    return [st["table_out"], count.to(torch.int32), st["k"], st["v"]]


# ------------------------------------------------------------------ what a pass cannot do without
def _keys(n, qn, case):
    """Visible (query, key) pairs of a chunk of qn queries that ends at length n, and the keys
    that any of them sees."""
    limit = case["sinks"] + case["window"]
    whole = min(max(limit - (n - qn), 0), qn)       # rows that see every earlier key
    first = n - qn
    pairs = whole * first + whole * (whole + 1) // 2 + (qn - whole) * limit
    return pairs, min(n, qn - 1 + limit)


def work(case):
    op, batch, hkv = case["op"], case["batch"], case["hkv"]
    if op in ("window_decode", "int4_decode"):
        new = 1 if op == "int4_decode" else 0
        seen = sum(min(n + new, case["sinks"] + case["window"]) for n in _lens(case)[0])
        token = 2 * (2 * D if op == "window_decode" else D // 2 + 4)    # K and V of one kv-head
        out = batch * case["hq"] * (D * 6 + 4) + new * batch * hkv * (4 * D + 136)
        return {"bytes": hkv * seen * token + seen / PAGE * 4 + out,
                "flops": 4.0 * D * case["hq"] * seen}
    if op == "window_prefill":
        lens, qn = _lens(case)
        both = [_keys(n, m, case) for n, m in zip(lens, qn)]
        return {"bytes": sum(qn) * case["hq"] * (4 * D + 4) + sum(x[1] for x in both) * hkv * 4 * D,
                "flops": 4.0 * D * case["hq"] * sum(x[0] for x in both)}
    page = 2 * hkv * PAGE * D * 2                               # K and V of one page
    if op == "remap_pages":
        copies = case["forks"] * 15 / 16
        entries = sum(-(-n // PAGE) for n in _lens(case)[0])
        return {"bytes": copies * 2 * page + 8 * entries + 20 * batch, "flops": 0}
    moved = case["used"] * (case["pages"] - case["used"]) / case["pages"]
    return {"bytes": moved * 2 * page + 8 * (case["used"] + 16 * batch), "flops": 0}


# ------------------------------------------------------------------ the definition, in 64 bits
def _sequence(st, b, count):
    """K and V [count][Hkv][128] of sequence b, in 64 bits."""
    j = torch.arange(count, device=DEV)
    page, row = st["table"][b].long()[j // PAGE].clamp(min=0), j % PAGE
    if "kc" not in st:
        return st["k"][page, :, row].double(), st["v"][page, :, row].double()
    both = []
    for codes, sz in ((st["kc"], st["ks"]), (st["vc"], st["vs"])):
        c, s = codes[page, :, row], sz[page, :, row].double()
        x = torch.empty(*c.shape[:-1], D, dtype=torch.float64, device=DEV)
        x[..., 0::2], x[..., 1::2] = (c % 16).double(), (c // 16).double()
        both.append(s[..., 0:1] * x + s[..., 1:2])
    return both


def _attend(q, k, v, seen):
    """softmax(q k^T / sqrt(128)) v over the seen keys; q [R][Hq][128], seen [R][T]."""
    group = q.shape[1] // k.shape[1]
    o = torch.zeros_like(q)
    lse = torch.zeros(q.shape[:2], dtype=torch.float64, device=DEV)
    for h in range(q.shape[1]):
        s = (q[:, h] @ k[:, h // group].T) / math.sqrt(128.0)
        s[~seen] = -math.inf
        lse[:, h] = torch.logsumexp(s, 1)
        o[:, h] = torch.exp(s - lse[:, h, None]) @ v[:, h // group]
    return o, lse


def exact(case, seed):
    st = prepare(case, seed)
    op, batch = case["op"], case["batch"]
    lens = st["lens"].tolist()
    if op in ("window_decode", "int4_decode"):
        if op == "int4_decode":
            for x, codes, sz in ((st["k_new"], st["kc"], st["ks"]), (st["v_new"], st["vc"], st["vs"])):
                f = x.double()
                lo = f.min(-1).values
                s = ((f.max(-1).values - lo).float() / 15).half()
                # a code is defined with its quotient in 32 bits, halves to even
                code = torch.round((f - lo[..., None]).float() / s.float()[..., None])
                code = code.clamp(0, 15).to(torch.uint8)
                for b in range(batch):
                    page, row = int(st["table"][b, lens[b] // PAGE]), lens[b] % PAGE
                    codes[page, :, row] = code[b, :, 0::2] + 16 * code[b, :, 1::2]
                    sz[page, :, row, 0], sz[page, :, row, 1] = s[b], lo[b].half()
            lens = [n + 1 for n in lens]
        os, ls = [], []
        for b, n in enumerate(lens):
            k, v = _sequence(st, b, n)
            j = torch.arange(n, device=DEV)
            seen = (j < case["sinks"]) | (j > n - 1 - case["window"])
            o, lse = _attend(st["q"][b:b + 1].double(), k, v, seen[None])
            os.append(o)
            ls.append(lse)
        got = [torch.cat(os), torch.cat(ls)]
        return got + [st["ks"].double(), st["vs"].double()] if op == "int4_decode" else got
    if op == "window_prefill":
        start = st["start"].tolist()
        os, ls = [], []
        for b, n in enumerate(lens):
            q = st["q"][start[b]:start[b + 1]].double()
            k, v = _sequence(st, b, n)
            t = torch.arange(n - len(q), n, device=DEV)[:, None]
            j = torch.arange(n, device=DEV)[None, :]
            o, lse = _attend(q, k, v, (j <= t) & ((j < case["sinks"]) | (j > t - case["window"])))
            os.append(o)
            ls.append(lse)
        return [torch.cat(os), torch.cat(ls)]
    table = st["table"].tolist()
    if op == "remap_pages":
        parent, extra = st["parent"].tolist(), st["extra"].tolist()
        width, sinks, window = len(table[0]), case["sinks"], case["window"]
        new, wants, moves, held = [], [], [], {}
        for b in range(batch):
            p = parent[b]
            n = lens[p] if p >= 0 else 0
            row = [-1] * width
            whole = n // PAGE
            for j in range(whole):
                if any(x < sinks or x > n - window for x in (PAGE * j, PAGE * j + PAGE - 1)):
                    row[j] = table[p][j]
            if n % PAGE and table[p][whole] >= 0:
                keeper = p if parent[p] == p else parent.index(p)
                if keeper == b:
                    row[whole] = table[p][whole]
                else:
                    wants.append((b, whole))
                    moves.append((b, whole, table[p][whole]))
            need = -(-(n + extra[b]) // PAGE)
            for j in range(whole, need):
                if p == b and j >= -(-n // PAGE):
                    row[j] = table[b][j]
                if row[j] < 0 and (b, j) not in wants[-1:]:
                    wants.append((b, j))
            new.append(row)
            held[b] = n
        taken = {x for row in new for x in row if x >= 0}
        free = (x for x in range(st["k"].shape[0]) if x not in taken)
        for b, j in wants:
            new[b][j] = next(free)
        for b, j, p in moves:
            for pool in (st["k"], st["v"]):
                pool[new[b][j]] = pool[p]
        return [torch.tensor(new, dtype=torch.int32), torch.tensor([held[b] for b in range(batch)],
                                                                   dtype=torch.int32),
                st["k"], st["v"]]
    taken = sorted({x for row in table for x in row if x >= 0})
    count = len(taken)
    inside = {x for x in taken if x < count}
    holes = [x for x in range(count) if x not in inside]
    to = dict(zip([x for x in taken if x >= count], holes))
    for pool in (st["k"], st["v"]):
        for x, y in to.items():
            pool[y] = pool[x]
    return [torch.tensor([[to.get(x, x) for x in row] for row in table], dtype=torch.int32),
            torch.tensor(count, dtype=torch.int32), st["k"], st["v"]]
