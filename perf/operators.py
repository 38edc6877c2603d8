"""The page operators of the FP4 cache and the attention over a shared prefix: cases, inputs, plain forms and calls.

Pages: sequences of a paged cache share pages. refs[p] counts the sequences that hold physical page p (0: free).
  copy     page src[i] -> page dst[i] (FP4 codes, E4M3 scales, indexer keys); -1 is an empty slot
  fork     child[i] becomes a copy of the first min(length[i], seq_len[parent[i]]) entries of parent[i]: whole pages are
           shared, a partial last page is copied to the lowest free page
  resize   seq[i] gets new_len[i] entries: pages behind it are released, missing pages are taken (lowest first), and a
           partial last page that others hold too is replaced by a copy of its own
  compact  the live pages behind the first n_live pages move into the free ones among those, both in ascending order
Attention: sequences are listed in groups; a group's first prefix_len entries are read through the pages of its first
member, later entries through each sequence's own pages, and a window of E4M3 rows is attended as well:
  o = sum_j softmax_j(scale * <q, v_j>) v_j over the entries below the query's limit and its window rows.
"""
import math

import torch

own = False

D = 512
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def listed():
    return [
        # one prompt sampled four times, first tokens: the smallest decode call, latency counts
        dict(name="attn_small", op="attn", groups="4", prefix="1000", h=16, qps=1, ps=64, tail=40, window=128, limits=False),
        # three prompts of uneven length with uneven batches, two draft tokens a sequence, each with its own limit
        dict(name="attn_groups", op="attn", groups="3,10,7", prefix="5011,257,20480", h=64, qps=2, ps=128, tail=300, window=256,
             limits=True),
        # a serving batch of 64 sequences behind one system prompt, 64-entry pages
        dict(name="attn_batch", op="attn", groups="64", prefix="32768", h=32, qps=1, ps=64, tail=600, window=512, limits=False),
        # eight questions on one very long document
        dict(name="attn_long", op="attn", groups="8", prefix="200001", h=64, qps=1, ps=64, tail=100, window=512, limits=False),
        # a few pages swapped in for a scheduler; a large block of a cache duplicated
        dict(name="copy_few", op="copy", pages=64, n=8, ps=64, di=64, empty=0),
        dict(name="copy_many", op="copy", pages=12000, n=5001, ps=64, di=128, empty=300),
        # four samples of one short prompt; 63 samples of a 256K-entry prompt
        dict(name="fork_few", op="fork", batch=8, pages=256, max_pages=64, ps=64, di=64, n=4, parents=1, length=1999),
        dict(name="fork_many", op="fork", batch=128, pages=12000, max_pages=4096, ps=64, di=64, n=96, parents=2, length=250021),
        # one decode step of a batch (some sequences cross into a new page); a batch of finished and rolled back sequences
        dict(name="resize_step", op="resize", batch=64, pages=8192, max_pages=512, ps=64, di=64, n=64, length=5000, to="step"),
        dict(name="resize_free", op="resize", batch=128, pages=12000, max_pages=2048, ps=64, di=128, n=100, length=100000, to="free"),
        # a small pool, and a large one of which six in ten pages are live
        dict(name="compact_few", op="compact", batch=8, pages=200, max_pages=40, ps=64, di=64, length=700, live=0.5),
        dict(name="compact_many", op="compact", batch=64, pages=16000, max_pages=4096, ps=64, di=64, length=30000, live=0.6),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "copy", "fork", "resize", "compact"])
    ps = rng.choice([32, 64, 128, 256])
    di = rng.choice([64, 128])
    if op == "attn":
        n = rng.randint(1, 3)
        h = rng.choice([16, 32, 64])
        qps = rng.choice([1, 1, 2, 4])
        sizes = [max(1, _log(rng, 1, 96) // (n * qps)) for _ in range(n)]
        prefix = [_log(rng, 1, 30000) for _ in range(n)]
        return dict(op="attn", groups=",".join(map(str, sizes)), prefix=",".join(map(str, prefix)), h=h, qps=qps, ps=ps,
                    tail=_log(rng, 1, 900), window=rng.choice([0, 1, 100, 128, 333, 512]), limits=rng.random() < 0.5)
    if op == "copy":
        n = _log(rng, 1, 1500)
        return dict(op="copy", pages=2 * n + rng.randint(1, 50), n=n, ps=ps, di=di, empty=rng.randint(0, n // 2))
    if op == "fork":
        n = _log(rng, 1, 60)
        length = _log(rng, 1, 60000)
        return dict(op="fork", batch=n + 4, pages=2 * (length // ps + 1) + n + 5, max_pages=length // ps + 3, ps=ps, di=di, n=n,
                    parents=rng.randint(1, 2), length=length)
    if op == "resize":
        batch = _log(rng, 2, 64)
        length = _log(rng, 10, 20000)
        room = max(2, int((length // ps + 3) * rng.uniform(0.1, 1.2)))
        return dict(op="resize", batch=batch, pages=batch * (room + 2) + 10 + length // ps, max_pages=2 * (length // ps + 2), ps=ps, di=di,
                    n=rng.randint(1, batch), length=length, to=rng.choice(["step", "free"]))
    batch = _log(rng, 1, 64)
    length = _log(rng, 10, 10000)
    live = rng.uniform(0.2, 0.95)
    return dict(op="compact", batch=batch, pages=int(batch * (length // ps + 1) / live) + 2, max_pages=length // ps + 2, ps=ps, di=di,
                length=length, live=round(live, 3))


# ---- inputs ---------------------------------------------------------------------------------------


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _quantised(rows, g):
    """N(0, 1) rows as FP4 codes (two a byte, element 2i in the low half) and one E4M3 scale per 16 values."""
    codes = torch.empty((rows, D // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((rows, D // 16), dtype=torch.uint8, device="cuda")
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    for a in range(0, rows, 65536):
        b = min(rows, a + 65536)
        x = torch.randn((b - a, D // 16, 16), generator=g, device="cuda")
        s = (x.abs().amax(-1) / 6).to(torch.float8_e4m3fn)
        y = x / s.float().clamp_min(2.0**-9)[..., None]
        c = torch.bucketize(y.abs(), edges).to(torch.uint8) | ((y < 0).to(torch.uint8) << 3)
        c = c.view(b - a, D // 2, 2)
        codes[a:b] = c[..., 0] | (c[..., 1] << 4)
        scales[a:b] = s.view(torch.uint8)
    return codes, scales


def _pool(pages, ps, di, g):
    """A cache of `pages` pages filled with plausible bytes (page operators move bytes, whatever they stand for)."""
    rows = pages * ps
    return dict(codes=torch.randint(0, 256, (rows, D // 2), dtype=torch.uint8, device="cuda", generator=g),
                scales=torch.randint(40, 70, (rows, D // 16), dtype=torch.uint8, device="cuda", generator=g),
                kidx=torch.randint(0, 120, (rows, di), dtype=torch.uint8, device="cuda", generator=g))


def _room(case):
    """Pages of its own for each sequence of a resize case, with some left to take."""
    return max(1, (case["pages"] - 2 * case["batch"] - 8 - -(-case["length"] // case["ps"])) // case["batch"])


def _tables(start, page_table, refs, seq_len):
    """The tables, the counts and the lengths in one buffer, so that one copy puts them back before each pass."""
    flat = torch.cat([t.reshape(-1).to(torch.int32) for t in (page_table, refs, seq_len)])
    work = flat.clone()
    a, b = page_table.numel(), page_table.numel() + refs.numel()
    start.update(saved=flat, work=work, page_table=work[:a].view(page_table.shape), refs=work[a:b], seq_len=work[b:])


def prepare(case, seed):
    g = _gen(seed)
    op, ps = case["op"], case["ps"]
    i32 = dict(dtype=torch.int32, device="cuda")
    if op == "attn":
        sizes = [int(x) for x in case["groups"].split(",")]
        prefix = [int(x) for x in case["prefix"].split(",")]
        h, qps, w = case["h"], case["qps"], case["window"]
        batch = sum(sizes)
        tails = torch.randint(0, case["tail"] + 1, (batch,), generator=g, device="cuda").tolist()
        order = torch.randperm(batch, generator=g, device="cuda").tolist()
        lens = [0] * batch
        begin = [0]
        for n in sizes:
            begin.append(begin[-1] + n)
        for k, p in enumerate(prefix):
            for j in range(begin[k], begin[k + 1]):
                lens[order[j]] = p + tails[j]
        shared = [p // ps for p in prefix]
        ends = [(n + ps - 1) // ps for n in lens]
        need = sum(shared) + sum(ends[order[j]] - shared[k] for k in range(len(prefix)) for j in range(begin[k], begin[k + 1]))
        # a partial last page of the prefix is a sequence's own copy, with the same entries: made equal below
        phys = torch.randperm(need + 2, generator=g, device="cuda").tolist()
        table = torch.full((batch, max(max(ends), 1)), -1, dtype=torch.int32)
        codes, scales = _quantised((need + 2) * ps, g)
        at = 0
        for k, p in enumerate(prefix):
            common = phys[at:at + shared[k]]
            at += shared[k]
            first = None
            for j in range(begin[k], begin[k + 1]):
                s = order[j]
                mine = phys[at:at + ends[s] - shared[k]]
                at += len(mine)
                table[s, :ends[s]] = torch.tensor(common + mine, dtype=torch.int32)
                if p % ps and mine:
                    if first is None:
                        first = mine[0]
                    else:
                        n = p % ps
                        codes[mine[0] * ps:mine[0] * ps + n] = codes[first * ps:first * ps + n]
                        scales[mine[0] * ps:mine[0] * ps + n] = scales[first * ps:first * ps + n]
        nq = batch * qps
        seq_len = torch.tensor(lens, **i32)
        limit = None
        if case["limits"]:  # the tokens of one step see one entry more each, the last of them all
            back = torch.arange(qps - 1, -1, -1, **i32)
            limit = (seq_len[:, None] - back[None, :]).clamp_min(0).reshape(-1).contiguous()
        ring = max(w, 1) + 37
        swa = torch.randn((batch, ring, D), generator=g, device="cuda").to(torch.float8_e4m3fn).view(torch.uint8)
        wb = torch.randint(0, ring, (nq,), generator=g, **i32)
        return dict(op=op, ps=ps, lut=torch.tensor(E2M1, device="cuda"), codes=codes, scales=scales, page_table=table.cuda(), seq_len=seq_len,
                    q=torch.randn((nq, h, D), generator=g, device="cuda").to(torch.bfloat16), qps=qps,
                    members=torch.tensor(order, **i32), group_begin=torch.tensor(begin, **i32),
                    prefix_len=torch.tensor(prefix, **i32), spans=tuple(zip(begin, begin[1:], prefix)), q_limit=limit,
                    swa=swa if w else None, swa_begin=wb if w else None, swa_end=wb + w if w else None, w=w,
                    most=max(lens) if lens else 0, tail=max(1, max(tails)), scale=1 / math.sqrt(D))
    di = case["di"]
    pages = case["pages"]
    s = dict(op=op, ps=ps, **_pool(pages, ps, di, g))
    if op == "copy":
        n = case["n"]
        perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        src, dst = perm[:n].clone(), perm[n:2 * n].clone()
        gone = torch.randperm(n, generator=g, device="cuda")[:case["empty"]]
        src[gone] = -1
        s.update(src=src, dst=dst, empty=case["empty"] > 0)
        return s
    batch, width, length = case["batch"], case["max_pages"], case["length"]
    table = torch.full((batch, width), -1, **i32)
    seq_len = torch.zeros(batch, **i32)
    refs = torch.zeros(pages, **i32)
    perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    if op == "fork":
        n, np_ = case["n"], case["parents"]
        per = (length + ps - 1) // ps
        slots = torch.randperm(batch, generator=g, device="cuda").to(torch.int32)
        parents, child = slots[:np_], slots[np_:np_ + n].clone()
        table[parents.long(), :per] = perm[:np_ * per].view(np_, per)
        refs[perm[:np_ * per].long()] = 1
        seq_len[parents.long()] = length
        parent = parents[torch.randint(0, np_, (n,), generator=g, device="cuda")].contiguous()
        cut = torch.randint(0, max(1, min(3 * ps, length // 4 + 1)), (n,), generator=g, **i32)
        s.update(parent=parent, child=child, length=(length - cut).contiguous())
    else:
        if op == "resize":  # where the pool is too small for pages of their own, all sequences share their first ones
            room = _room(case)
            common = max(0, -(-length // ps) - room)
            lens = torch.randint(max(length // 2, common * ps + 1), length + 1, (batch,), generator=g, **i32)
            per = lens // ps + (lens % ps > 0)
        else:
            lens = torch.randint(length // 2, length + 1, (batch,), generator=g, **i32)
            room = int(pages * case["live"]) // batch
            per = torch.minimum(lens // ps + (lens % ps > 0), torch.tensor(min(room, width), **i32))
            lens = torch.minimum(lens, per * ps)
            common = 0
        col = torch.arange(width, **i32)[None, :]
        mine = (col >= common) & (col < per[:, None])
        rank = mine.reshape(-1).cumsum(0).view(mine.shape) - 1 + common
        assert int(rank[-1, -1]) < pages, "a pool too small for its sequences"
        table = torch.where(col < common, perm[col.clamp_max(max(common - 1, 0)).long()],
                            torch.where(mine, perm[rank.clamp_min(0)], table))
        refs.index_add_(0, table[table >= 0].long(), torch.ones_like(table[table >= 0]))
        seq_len = lens.clone()
        if op == "resize":
            n = case["n"]
            seq = torch.randperm(batch, generator=g, device="cuda")[:n]
            if case["to"] == "step":
                new = lens[seq] + 1
            else:  # half of them end, the others are rolled back
                keep = torch.rand((n,), generator=g, device="cuda") * (torch.rand((n,), generator=g, device="cuda") < 0.5)
                new = (lens[seq] * keep).to(torch.int32)
            s.update(seq=seq.to(torch.int32).contiguous(), new_len=new.to(torch.int32).contiguous())
    _tables(s, table, refs, seq_len)
    return s


# ---- plain forms ----------------------------------------------------------------------------------


def _values(lut, codes, scales):
    """The rows that FP4 codes and their scales stand for, in 32 bits."""
    v = torch.stack((lut[(codes & 15).int()], lut[(codes >> 4).int()]), -1).view(*codes.shape[:-1], D // 16, 16)
    return (v * scales.view(torch.float8_e4m3fn).float()[..., None]).view(*codes.shape[:-1], D)


def _plain_attn(s):
    ps, qps, w = s["ps"], s["qps"], s["w"]
    nq, h = s["q"].shape[:2]
    q = s["q"].float()
    batch = nq // qps
    seq = torch.arange(nq, device="cuda") // qps
    limit = s["q_limit"] if s["q_limit"] is not None else s["seq_len"][seq]
    o = torch.empty((nq, h, D), device="cuda")
    lse = torch.empty((nq, h), device="cuda")
    for a, b, prefix in s["spans"]:
        who = s["members"][a:b].long()
        mine = (who[:, None] * qps + torch.arange(qps, device="cuda")).reshape(-1)  # the group's queries
        qg = q[mine]
        lim = limit[mine][:, None]
        t = torch.arange(prefix, device="cuda")
        page = s["page_table"][who[0]].long()[t // ps]
        rows = page * ps + t % ps
        v = _values(s["lut"], s["codes"][rows], s["scales"][rows])
        x = (qg.reshape(-1, D) @ v.T).view(-1, h, prefix) * s["scale"]
        x = x.masked_fill((t[None, :] >= lim)[:, None, :], -math.inf)
        t = prefix + torch.arange(s["tail"], device="cuda")
        page = s["page_table"][who].long()[:, (t // ps).clamp_max(s["page_table"].shape[1] - 1)]
        rows = (page * ps + t % ps).clamp_min(0)
        vt = _values(s["lut"], s["codes"][rows], s["scales"][rows])  # [members, tail, D]
        xt = (qg.view(len(who), qps * h, D) @ vt.transpose(1, 2)).view(-1, h, len(t)) * s["scale"]
        xt = xt.masked_fill((t[None, :] >= lim)[:, None, :], -math.inf)
        m = torch.maximum(x.amax(-1), xt.amax(-1))
        if w:
            slot = (s["swa_begin"][mine].long()[:, None] + torch.arange(w, device="cuda")) % s["swa"].shape[1]
            vw = s["swa"].view(torch.float8_e4m3fn)[seq[mine][:, None], slot].float()  # [queries, w, D]
            xw = (qg @ vw.transpose(1, 2)) * s["scale"]
            m = torch.maximum(m, xw.amax(-1))
        at = m.masked_fill(m == -math.inf, 0)[..., None]
        p, pt = torch.exp(x - at), torch.exp(xt - at)
        total = p.sum(-1) + pt.sum(-1)
        acc = (p.view(-1, prefix) @ v).view(-1, h, D) + (pt.view(len(who), qps * h, -1) @ vt).view(-1, h, D)
        if w:
            pw = torch.exp(xw - at)
            total = total + pw.sum(-1)
            acc = acc + pw @ vw
        o[mine] = torch.where(total[..., None] > 0, acc / total[..., None], 0.0)
        lse[mine] = at[..., 0] + torch.log(total)
    return o.to(torch.bfloat16), lse


def _paged(s):
    return [s[k].view(-1, s["ps"], s[k].shape[1]) for k in ("codes", "scales", "kidx")]


def _plain_copy(s):
    src, dst = s["src"].long(), s["dst"].long()
    if s["empty"]:
        some = (src >= 0) & (dst >= 0)
        src, dst = src[some], dst[some]
    for t in _paged(s):
        t[dst] = t[src]
    return s["codes"], s["scales"], s["kidx"]


def _free_page(refs, rank):
    """The page that is free and has `rank` free pages below it."""
    return torch.searchsorted((refs == 0).cumsum(0), rank + 1)


def _copy_part(s, some, src, dst, rows):
    """The first rows[i] rows of page src[i] into page dst[i], where some[i]."""
    src, dst, rows = src[some], dst[some], rows[some]
    r = torch.arange(s["ps"], device="cuda")
    for t in _paged(s):
        t[dst] = torch.where((r[None, :] < rows[:, None])[..., None], t[src], t[dst])


def _plain_fork(s):
    s["work"].copy_(s["saved"])
    table, refs, seq_len, ps = s["page_table"], s["refs"], s["seq_len"], s["ps"]
    parent, child = s["parent"].long(), s["child"].long()
    n = torch.minimum(s["length"], seq_len[parent])
    whole, rest = n // ps, n % ps
    part = rest > 0
    new = _free_page(refs, part.cumsum(0) - 1).to(torch.int32)
    col = torch.arange(table.shape[1], device="cuda")[None, :]
    rows = table[parent]
    old = rows.gather(1, whole.clamp_max(table.shape[1] - 1)[:, None].long())[:, 0]
    shared = col < whole[:, None]
    refs.index_add_(0, torch.where(shared, rows, 0).reshape(-1), shared.reshape(-1).int())
    rows = torch.where(shared, rows, -1)
    table[child] = torch.where((col == whole[:, None]) & part[:, None], new[:, None], rows)
    refs[new[part].long()] = 1
    seq_len[child] = n
    src, dst = torch.where(part, old, -1), torch.where(part, new, -1)
    _copy_part(s, part, src.long(), dst.long(), rest)
    return table, refs, seq_len, src, dst, s["codes"], s["scales"], s["kidx"]


def _plain_resize(s):
    s["work"].copy_(s["saved"])
    table, refs, seq_len, ps = s["page_table"], s["refs"], s["seq_len"], s["ps"]
    seq, new = s["seq"].long(), s["new_len"]
    before = refs.clone()
    had, has = (seq_len[seq] + ps - 1) // ps, (new + ps - 1) // ps
    kept = torch.minimum(seq_len[seq], new)
    last = ((kept - 1) // ps).clamp_min(0)
    rows = table[seq]
    old = rows.gather(1, last[:, None].long())[:, 0]
    apart = (kept % ps > 0) & (before[old.clamp_min(0).long()] > 1)  # a partial last page that others hold too
    grown = (has - had).clamp_min(0)
    first = (apart + grown).cumsum(0) - (apart + grown)
    page = _free_page(before, first).to(torch.int32)
    col = torch.arange(table.shape[1], device="cuda")[None, :]
    out = (col >= has[:, None]) & (col < had[:, None])
    refs.index_add_(0, torch.where(out, rows, 0).reshape(-1), -out.reshape(-1).int())
    rows = torch.where(out, -1, rows)
    added = (col >= had[:, None]) & (col < has[:, None])
    fresh = _free_page(before, torch.where(added, (first + apart)[:, None] + col - had[:, None], 0)).to(torch.int32)
    refs.index_add_(0, torch.where(added, fresh, 0).reshape(-1), added.reshape(-1).int())
    rows = torch.where(added, fresh, rows)
    refs.index_add_(0, old.clamp_min(0), -apart.int())
    refs.index_add_(0, torch.where(apart, page, 0), apart.int())
    rows = torch.where((col == last[:, None]) & apart[:, None], page[:, None], rows)
    table[seq] = rows
    seq_len[seq] = new
    src, dst = torch.where(apart, old, -1), torch.where(apart, page, -1)
    _copy_part(s, apart, src.long(), dst.long(), kept % ps)
    return table, refs, seq_len, src, dst, s["codes"], s["scales"], s["kidx"]


def _plain_compact(s):
    s["work"].copy_(s["saved"])
    table, refs = s["page_table"], s["refs"]
    live = refs > 0
    n = live.sum()
    page = torch.arange(len(refs), device="cuda", dtype=torch.int32)
    src, dst = page[live & (page >= n)], page[~live & (page < n)]
    to = page.clone()
    to[src.long()] = dst
    table.copy_(torch.where(table >= 0, to[table.clamp_min(0).long()], table))
    refs[dst.long()] = refs[src.long()]
    refs[src.long()] = 0
    for t in _paged(s):
        t[dst.long()] = t[src.long()]
    pad = torch.full((2, len(refs) // 2), -1, dtype=torch.int32, device="cuda")
    pad[0, :len(src)], pad[1, :len(dst)] = src, dst
    return table, refs, s["seq_len"], pad[0], pad[1], n.to(torch.int32).view(1), s["codes"], s["scales"], s["kidx"]


# ---- the framework's calls ------------------------------------------------------------------------


def _kept(s):
    """What a program keeps beside its tensors: the cache's descriptor, the workspace and the output buffers."""
    from sparse_fp4_kv_b200 import binding as B
    if "kept" in s:
        return B, s["kept"]
    i32 = dict(dtype=torch.int32, device="cuda")
    k = {}
    if s["op"] == "attn":
        nq, h = s["q"].shape[:2]
        k["kv"] = B.KvCache(s["codes"], s["scales"], None, s["page_table"], s["seq_len"], s["ps"])
        k["o"] = torch.empty((nq, h, D), dtype=torch.bfloat16, device="cuda")
        k["lse"] = torch.empty((nq, h), dtype=torch.float32, device="cuda")
        k["ws"] = B.workspace(B.csa2_prefix_attn_workspace_size(len(s["members"]), len(s["prefix_len"]), s["qps"], h), "cuda")
    else:
        pages = s["codes"].shape[0] // s["ps"]
        table = s["page_table"] if "page_table" in s else torch.zeros((1, 1), **i32)
        k["kv"] = B.KvCache(s["codes"], s["scales"], s["kidx"], table, s["seq_len"] if "seq_len" in s else torch.zeros(1, **i32), s["ps"])
        n = {"fork": "parent", "resize": "seq"}.get(s["op"])
        n = len(s[n]) if n else 0
        k["ws"] = B.workspace(B.csa2_pages_workspace_size(n, table.shape[0], pages), "cuda")
        k["src"], k["dst"] = (torch.empty(n or pages // 2, **i32) for _ in range(2))
        k["live"] = torch.empty(1, **i32)
    s["kept"] = k
    return B, k


def _own_run(s):
    B, k = _kept(s)
    op, kv, ws = s["op"], k["kv"], k["ws"]
    if op == "attn":
        B.csa2_prefix_attn_decode(s["q"], s["qps"], kv, s["members"], s["group_begin"], s["prefix_len"], s["q_limit"], s["swa"],
                                  s["swa"].shape[1] if s["w"] else 0, s["swa_begin"], s["swa_end"], s["w"], s["scale"], k["o"],
                                  k["lse"], ws)
        return k["o"], k["lse"]
    if op == "copy":
        B.csa2_pages_copy(kv, s["src"], s["dst"])
        return s["codes"], s["scales"], s["kidx"]
    s["work"].copy_(s["saved"])
    data = s["codes"], s["scales"], s["kidx"]
    if op == "fork":
        B.csa2_pages_fork(kv, s["refs"], s["parent"], s["child"], s["length"], k["src"], k["dst"], ws)
        return s["page_table"], s["refs"], s["seq_len"], k["src"], k["dst"], *data
    if op == "resize":
        B.csa2_pages_resize(kv, s["refs"], s["seq"], s["new_len"], k["src"], k["dst"], ws)
        return s["page_table"], s["refs"], s["seq_len"], k["src"], k["dst"], *data
    B.csa2_pages_compact(kv, s["refs"], k["src"], k["dst"], k["live"], ws)
    return s["page_table"], s["refs"], s["seq_len"], k["src"], k["dst"], k["live"], *data


def run(state):
    """One pass. Page operators first put the tables back, so that each pass does the same work."""
    if own:
        return _own_run(state)
    return dict(attn=_plain_attn, copy=_plain_copy, fork=_plain_fork, resize=_plain_resize, compact=_plain_compact)[state["op"]](state)


def work(case):
    op, ps = case["op"], case["ps"]
    if op == "attn":
        sizes = [int(x) for x in case["groups"].split(",")]
        prefix = [int(x) for x in case["prefix"].split(",")]
        h, qps, w = case["h"], case["qps"], case["window"]
        nq = sum(sizes) * qps
        tail = case["tail"] / 2
        entries = sum(prefix) + sum(sizes) * tail
        pairs = qps * sum(n * (p + tail + w) for n, p in zip(sizes, prefix))
        ring = min(w + 37, qps * w) if w else 0
        return dict(bytes=entries * 288 + entries / ps * 4 + sum(sizes) * ring * D + nq * h * (2 * D * 2 + 4), flops=pairs * h * D * 4)
    row = D // 2 + D // 16 + case["di"]
    if op == "copy":
        return dict(bytes=2 * (case["n"] - case["empty"]) * ps * row + 8 * case["n"], flops=0)
    if op == "fork":
        n, per = case["n"], case["length"] // ps
        return dict(bytes=n * ps * row + 4 * case["pages"] + 4 * per * (n + 2 * case["parents"]), flops=0)
    if op == "resize":
        n, per = case["n"], 0.75 * case["length"] / ps
        parts = n / 2 if case["to"] == "free" and -(-case["length"] // ps) > _room(case) else 0
        cells = 0.75 * n * per if case["to"] == "free" else n / ps
        return dict(bytes=parts * ps * row + 4 * case["pages"] + 4 * 3 * cells, flops=0)
    pages, live = case["pages"], case["live"]
    table = case["batch"] * case["max_pages"]
    held = min(live * pages, 0.75 * case["batch"] * case["length"] / ps)
    moved = held * (1 - held / pages)
    return dict(bytes=2 * moved * ps * row + 8 * pages + 4 * table, flops=0)


# ---- the attention's definition in 64 bits --------------------------------------------------------


def exact(case, seed):
    if case["op"] != "attn":
        return None  # whole numbers and moved bytes: nothing is computed
    s = prepare(case, seed)
    nq, h, _ = s["q"].shape
    o = torch.zeros((nq, h, D), dtype=torch.float64, device="cuda")
    lse = torch.full((nq, h), -math.inf, dtype=torch.float64, device="cuda")
    members = s["members"].tolist()
    level = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")

    def number(code):
        return level[(code & 7).long()] * (1 - 2 * (code >> 3).double())

    for a, b, prefix in s["spans"]:
        for j in range(a, b):
            for i in range(members[j] * s["qps"], (members[j] + 1) * s["qps"]):
                n = int(s["q_limit"][i] if s["q_limit"] is not None else s["seq_len"][members[j]])
                t = torch.arange(n, device="cuda")
                holder = torch.where(t < prefix, members[a], members[j])
                at = s["page_table"][holder, t // s["ps"]].long() * s["ps"] + t % s["ps"]
                byte = s["codes"][at]
                v = torch.empty((n, D), dtype=torch.float64, device="cuda")
                v[:, 0::2], v[:, 1::2] = number(byte & 15), number(byte >> 4)
                v *= s["scales"][at].view(torch.float8_e4m3fn).double().repeat_interleave(16, dim=1)
                if s["w"]:
                    r = torch.arange(int(s["swa_begin"][i]), int(s["swa_end"][i]), device="cuda") % s["swa"].shape[1]
                    v = torch.cat([v, s["swa"][members[j], r].view(torch.float8_e4m3fn).double()])
                if len(v):
                    x = s["q"][i].double() @ v.T * s["scale"]
                    lse[i] = torch.logsumexp(x, -1)
                    o[i] = torch.softmax(x, -1) @ v
    return o, lse
