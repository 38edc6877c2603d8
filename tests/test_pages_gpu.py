"""The page operators against a sequential model: tables, counts, lengths,
copy lists and every byte of the pool equal."""
import numpy as np
import pytest
import torch

from pages_model import Pool

pytestmark = pytest.mark.gpu
PAGES = 16  # the error word's bit of a refused entry
BAD_ROW = 1


@pytest.fixture(scope="module")
def B():
    from sparse_fp4_kv_b200 import build
    build.build()
    from sparse_fp4_kv_b200 import binding
    return binding


class Gpu:
    """The model's pool on the device."""

    def __init__(self, B, pool, dev, n=64, shift=0):
        t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)
        self.B, self.dev = B, dev
        self.data = [t(d.reshape(-1, d.shape[-1])) for d in pool.data]
        self.table, self.seq_len, self.refs = t(pool.table), t(pool.seq_len), t(pool.refs)
        if shift:  # counts that start inside a larger buffer
            self.refs = torch.cat([self.refs.new_full((shift,), 9), self.refs])[shift:]
        self.kv = B.KvCache(self.data[0], self.data[1], self.data[2] if len(self.data) > 2 else None, self.table, self.seq_len, pool.ps)
        self.ws = B.workspace(B.csa2_pages_workspace_size(n, len(pool.seq_len), pool.pages), dev)

    def i32(self, a):
        return None if a is None else torch.tensor(np.asarray(a, np.int32), device=self.dev)

    def lists(self, n):
        return [torch.full((max(n, 1),), -7, dtype=torch.int32, device=self.dev) for _ in range(2)]

    def fork(self, parent, child, length=None, lists=True):
        c = self.lists(len(parent)) if lists else (None, None)
        self.B.csa2_pages_fork(self.kv, self.refs, self.i32(parent), self.i32(child), self.i32(length), *c, self.ws)
        return c

    def resize(self, seq, new_len, lists=True):
        c = self.lists(len(seq)) if lists else (None, None)
        self.B.csa2_pages_resize(self.kv, self.refs, self.i32(seq), self.i32(new_len), *c, self.ws)
        return c

    def compact(self, pages):
        c, live = self.lists(pages // 2), self.i32([-1])
        self.B.csa2_pages_compact(self.kv, self.refs, *c, live, self.ws)
        return c, live

    def copy(self, src, dst):
        self.B.csa2_pages_copy(self.kv, self.i32(src), self.i32(dst))

    def same(self, pool, status=0):
        assert self.B.csa2_device_status() == status
        for got, want in ((self.refs, pool.refs), (self.seq_len, pool.seq_len), (self.table, pool.table)):
            np.testing.assert_array_equal(got.cpu().numpy(), want)
        for got, want in zip(self.data, pool.data):
            np.testing.assert_array_equal(got.cpu().numpy().reshape(want.shape), want)


def _pair(got, want):
    for g, w in zip(got, want):
        np.testing.assert_array_equal(g.cpu().numpy()[:len(w)], w)


@pytest.mark.parametrize("ps,di,n", [(32, 64, 1), (64, 128, 7), (128, 0, 33), (256, 64, 5), (64, 64, 300)])
def test_copy(B, cuda_device, ps, di, n):
    rng = np.random.default_rng(ps + n)
    pool = Pool(rng, 2 * n + 3, ps, di, 1, 1)
    g = Gpu(B, pool, cuda_device)
    perm = rng.permutation(pool.pages)
    src, dst = perm[:n].copy(), perm[n:2 * n].copy()
    if n > 4:
        src[1], dst[3], src[4] = -1, -1, dst[4]  # empty slots; a page onto itself
    pool.copy(src, dst)
    g.copy(src, dst)
    g.same(pool)


def test_copy_outside_the_cache_is_reported_and_skipped(B, cuda_device):
    rng = np.random.default_rng(1)
    pool = Pool(rng, 6, 32, 64, 1, 1)
    g = Gpu(B, pool, cuda_device)
    g.copy([0, 6, -2, 2], [3, 4, 5, 1 << 30])
    pool.copy([0], [3])
    g.same(pool, BAD_ROW)


@pytest.mark.parametrize("ps,di", [(32, 64), (64, 128), (256, 0)])
@pytest.mark.parametrize("length", [0, 1, 31, 32, 255, 256, 257, 1000])
def test_fork(B, cuda_device, ps, di, length):
    rng = np.random.default_rng(ps * 1000 + length)
    pool = Pool(rng, 3 * (1000 // ps + 2) + 20, ps, di, 12, 1000 // ps + 2)
    pool.fill(rng, [length, 700])
    g = Gpu(B, pool, cuda_device)
    parent, child = [0, 1, 0, 0, 1], [5, 2, 11, 3, 7]
    lens = [length, 700, max(0, length - 1), length // 2, 10 ** 6]
    want = pool.fork(parent, child, lens)
    _pair(g.fork(parent, child, lens), want)
    g.same(pool)
    # the rest of the batch: no lengths, a child as parent, no lists
    pool.fork([5, 2], [4, 6])
    g.fork([5, 2], [4, 6], lists=False)
    g.same(pool)


def test_fork_refusals(B, cuda_device):
    rng = np.random.default_rng(3)
    pool = Pool(rng, 14, 32, 64, 8, 4)
    pool.fill(rng, [100, 33])  # 4 + 2 pages, 8 free
    g = Gpu(B, pool, cuda_device)
    # out of the batch, itself, not empty, twice, a negative length, then fine ones
    parent, child = [0, 9, 0, 0, 0, 1, 0, 0], [8, 2, 0, 1, 3, 3, 4, 5]
    lens = [5, 5, 5, 5, 100, 33, -1, 40]
    want = pool.fork(parent, child, lens)
    assert pool.refused
    _pair(g.fork(parent, child, lens), want)
    g.same(pool, PAGES)
    # a child of this call is an empty parent
    pool.fork([0, 7], [7, 6])
    g.fork([0, 7], [7, 6])
    g.same(pool)


def test_no_pages_left_in_the_order_of_the_entries(B, cuda_device):
    rng = np.random.default_rng(4)
    pool = Pool(rng, 12, 32, 64, 10, 12)
    pool.fill(rng, [5 * 32 + 1, 3 * 32])  # 9 of 12 pages
    g = Gpu(B, pool, cuda_device)
    parent, child, lens = [0, 0, 1, 0, 0, 1], [2, 3, 4, 5, 6, 7], [40, 64, 90, 161, 3, 96]
    want = pool.fork(parent, child, lens)  # three pages for four partial ones
    assert pool.refused
    _pair(g.fork(parent, child, lens), want)
    g.same(pool, PAGES)
    # growth: two freed, then one entry too large and whatever comes later
    for seq, new in (([2, 3], [0, 0]), ([4, 0, 1, 6], [90 + 32, 12 * 32, 97, 0])):
        pool.refused = False
        want = pool.resize(seq, new)
        _pair(g.resize(seq, new), want)
        g.same(pool, PAGES if pool.refused else 0)


@pytest.mark.parametrize("ps,di,seed", [(32, 64, 0), (64, 128, 1), (128, 0, 2), (64, 64, 3), (4096, 64, 4)])
def test_random_turns(B, cuda_device, ps, di, seed):
    """Forks, growth, rollbacks into shared pages, frees and compactions in turn."""
    rng = np.random.default_rng(seed)
    batch, width = 24, 9  # refs at every alignment
    pool = Pool(rng, 90, ps, di, batch, width)
    pool.fill(rng, [ps * 4 + 5, ps * 3, 1])
    g = Gpu(B, pool, cuda_device, shift=seed)
    for turn in range(12):
        pool.refused = False
        n = int(rng.integers(1, 9))
        some = rng.permutation(batch)[:n]
        kind = turn % 4
        if kind == 0:
            empty = [s for s in range(batch) if pool.seq_len[s] == 0][:n]
            full = [s for s in range(batch) if pool.seq_len[s] > 0]
            parent = [int(rng.choice(full)) for _ in empty]
            lens = [int(rng.integers(0, pool.seq_len[a] + 1)) for a in parent]
            if empty:
                _pair(g.fork(parent, empty, lens), pool.fork(parent, empty, lens))
        elif kind in (1, 2):
            new = [min(width * ps, int(pool.seq_len[s] + rng.integers(0, 2 * ps))) if kind == 1
                   else int(rng.integers(0, pool.seq_len[s] + 1)) for s in some]
            _pair(g.resize(some, new), pool.resize(some, new))
        else:
            moves, live = pool.compact()
            got, n_live = g.compact(pool.pages)
            _pair(got, moves)
            assert int(n_live) == live
        g.same(pool, PAGES if pool.refused else 0)
    # the counts are those of the tables
    held = np.bincount(pool.table[pool.table >= 0], minlength=pool.pages)
    np.testing.assert_array_equal(held, pool.refs)


def test_resize_refusals(B, cuda_device):
    rng = np.random.default_rng(5)
    pool = Pool(rng, 20, 64, 64, 4, 3)
    pool.fill(rng, [100, 192])
    g = Gpu(B, pool, cuda_device)
    seq, new = [-1, 4, 0, 0, 1, 2], [1, 1, 120, 10, 193, -5]
    want = pool.resize(seq, new)
    _pair(g.resize(seq, new), want)
    g.same(pool, PAGES)


@pytest.mark.parametrize("pages", [1, 2, 3, 33, 5000, 70001])
def test_compact_sizes(B, cuda_device, pages):
    """Pool sizes around the runs of the plan's CTAs; no, one and many moves."""
    rng = np.random.default_rng(pages)
    pool = Pool(rng, pages, 32, 0, 3, pages)
    used = int(pages * 0.6)
    pool.fill(rng, [32 * (used // 2), 32 * (used - used // 2) - (1 if used > 1 else 0)])
    g = Gpu(B, pool, cuda_device)
    for _ in range(2):  # the second finds nothing to move
        moves, live = pool.compact()
        got, n_live = g.compact(pages)
        _pair(got, moves)
        assert int(n_live) == live
        g.same(pool)


@pytest.mark.parametrize("n", [1, 31, 1025, 2500])
def test_many_entries(B, cuda_device, n):
    """More entries than the plan's block has threads."""
    rng = np.random.default_rng(n)
    pool = Pool(rng, n + 40, 32, 0, n + 1, 4)
    pool.fill(rng, [97])
    g = Gpu(B, pool, cuda_device, n=n)
    child = rng.permutation(n) + 1
    lens = rng.integers(0, 98, n)
    _pair(g.fork([0] * n, child, lens), pool.fork([0] * n, child, lens))
    g.same(pool)
    new = np.where(rng.random(n) < 0.5, 0, rng.integers(0, 129, n))
    pool.refused = False
    _pair(g.resize(child, new), pool.resize(child, new))
    g.same(pool, PAGES if pool.refused else 0)


def test_no_entries_do_nothing(B, cuda_device):
    rng = np.random.default_rng(6)
    pool = Pool(rng, 8, 32, 64, 2, 4)
    pool.fill(rng, [40])
    g = Gpu(B, pool, cuda_device)
    none = torch.empty(0, dtype=torch.int32, device=cuda_device)
    B.csa2_pages_copy(g.kv, none, none)
    B.csa2_pages_fork(g.kv, g.refs, none, none, None, None, None, g.ws)
    B.csa2_pages_resize(g.kv, g.refs, none, none, None, None, g.ws)
    g.same(pool)


def test_captured_and_replayed(B, cuda_device):
    """A fork and its release in one graph, on a stream of its own, replayed twice."""
    rng = np.random.default_rng(7)
    pool = Pool(rng, 40, 32, 64, 6, 8)
    pool.fill(rng, [170, 64])
    g = Gpu(B, pool, cuda_device)
    parent, child, zero = g.i32([0, 1, 0]), g.i32([3, 4, 5]), g.i32([0, 0, 0])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):  # attributes are set outside the capture
        B.csa2_pages_fork(g.kv, g.refs, parent, child, None, None, None, g.ws)
        B.csa2_pages_resize(g.kv, g.refs, child, zero, None, None, g.ws)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        B.csa2_pages_fork(g.kv, g.refs, parent, child, None, None, None, g.ws)
        B.csa2_pages_resize(g.kv, g.refs, child, zero, None, None, g.ws)
    for _ in range(2):
        graph.replay()
        pool.fork([0, 1, 0], [3, 4, 5])
        pool.resize([3, 4, 5], [0, 0, 0])
    torch.cuda.synchronize()
    g.same(pool)


def test_needs_that_pass_32_bits_are_refused(B, cuda_device):
    """Rows of 2^26 pages: what the entries ask for together passes 2^31 pages, and every entry behind the first large
    one that needs pages is refused."""
    ps, width, batch, pages = 32, 1 << 26, 40, 12
    i32 = dict(dtype=torch.int32, device=cuda_device)
    table = torch.full((batch, width), -1, **i32)
    seq_len, refs = torch.zeros(batch, **i32), torch.zeros(pages, **i32)
    table[39, :2], seq_len[39], refs[3], refs[5] = torch.tensor([3, 5], **i32), 64, 1, 1
    z = lambda w: torch.zeros((pages * ps, w), dtype=torch.uint8, device=cuda_device)
    kv = B.KvCache(z(256), z(32), None, table, seq_len, ps)
    ws = B.workspace(B.csa2_pages_workspace_size(batch, batch, pages), cuda_device)
    most = 2 ** 31 - 1
    seq = torch.tensor([1, *range(2, 37), 37, 39, 38], **i32)
    new = torch.tensor([70, *[most] * 35, 1, 20, 64], **i32)
    src, dst = (torch.full((len(seq),), -7, **i32) for _ in range(2))
    B.csa2_pages_resize(kv, refs, seq, new, src, dst, ws)
    assert B.csa2_device_status() == PAGES
    assert table[1, :4].tolist() == [0, 1, 2, -1] and table[39, :3].tolist() == [3, -1, -1]
    assert refs.tolist() == [1, 1, 1, 1] + [0] * 8
    want = torch.zeros(batch, **i32)
    want[1], want[39] = 70, 20
    assert torch.equal(seq_len, want) and (src == -1).all() and (dst == -1).all()
    assert int((table >= 0).sum()) == 4


def test_rows_as_wide_as_32_bits(B, cuda_device):
    """A fork and its release in rows of 2^31 - 1 columns."""
    ps, width, pages = 64, 2 ** 31 - 1, 9
    i32 = dict(dtype=torch.int32, device=cuda_device)
    table = torch.full((2, width), -1, **i32)
    table[0, :3] = torch.tensor([7, 2, 4], **i32)
    seq_len, refs = torch.tensor([150, 0], **i32), torch.zeros(pages, **i32)
    refs[[7, 2, 4]] = 1
    z = lambda w: torch.zeros((pages * ps, w), dtype=torch.uint8, device=cuda_device)
    kv = B.KvCache(z(256), z(32), None, table, seq_len, ps)
    ws = B.workspace(B.csa2_pages_workspace_size(1, 2, pages), cuda_device)
    one = lambda x: torch.tensor([x], **i32)
    B.csa2_pages_fork(kv, refs, one(0), one(1), None, None, None, ws)
    assert B.csa2_device_status() == 0
    assert table[1, :4].tolist() == [7, 2, 0, -1] and seq_len.tolist() == [150, 150]
    assert refs.tolist() == [1, 0, 2, 0, 1, 0, 0, 2, 0]
    assert int(table[1].max()) == 7 and int((table[1, 3:] != -1).sum()) == 0 and int((table[0, 3:] != -1).sum()) == 0
    B.csa2_pages_resize(kv, refs, one(1), one(0), None, None, ws)
    assert B.csa2_device_status() == 0
    assert refs.tolist() == [0, 0, 1, 0, 1, 0, 0, 1, 0] and int((table[1] != -1).sum()) == 0
    live, (src, dst) = one(-1), (torch.full((pages // 2,), -7, **i32) for _ in range(2))
    B.csa2_pages_compact(kv, refs, src, dst, live, ws)
    # live are 2, 4 and 7: 4 moves to 0 and 7 to 1
    assert B.csa2_device_status() == 0 and int(live) == 3 and table[0, :4].tolist() == [1, 2, 0, -1]


@pytest.mark.parametrize("n,ps,width", [(1, 32, 8000), (1, 32, 70000), (1, 16384, 4), (1, 65536, 4), (2, 64, 20000), (5, 32, 6000), (3, 4096, 5)])
def test_wide_rows_and_large_pages(B, cuda_device, n, ps, width):
    """Few entries with long rows of the table or large partial pages: forked, grown, rolled back and freed."""
    rng = np.random.default_rng(n * ps + width)
    long = (width - 1) * ps - 5 if ps * width < 400_000 else min(width - 3, 900) * ps - 5
    pages = -(-long // ps) + (3 * n + 4 if ps > 1000 else 300)
    pool = Pool(rng, pages, ps, 64 if ps > 1000 else 0, n + 2, width)
    pool.fill(rng, [long])
    g = Gpu(B, pool, cuda_device)
    child = [1 + i for i in range(n)]
    lens = [long - i * (ps // 2 + 1) for i in range(n)]
    _pair(g.fork([0] * n, child, lens), pool.fork([0] * n, child, lens))
    g.same(pool)
    room = width * ps
    for new in ([min(room, int(x) + ps) for x in pool.seq_len[child]], [int(x) // 2 + 1 for x in lens], [min(room, 200 * ps // n)] * n, [0] * n):
        pool.refused = False
        _pair(g.resize(child, new), pool.resize(child, new))
        g.same(pool, PAGES if pool.refused else 0)


def test_compaction_reports_entries_outside_the_cache(B, cuda_device):
    """Within a sequence's length a page that is none is reported and left as it is, with or without moves; what lies
    behind the length is not looked at."""
    rng = np.random.default_rng(8)
    for holes in (True, False):
        for bad in (-1, -7, 24, 2 ** 31 - 1, None):
            pool = Pool(rng, 24, 32, 64, 4, 6)
            pool.fill(rng, [130, 64, 96], shuffle=holes)
            pool.table[1, 4] = 99  # behind its two pages
            if bad is not None:
                pool.table[2, 1], keep = bad, pool.table[2, 1]
            g = Gpu(B, pool, cuda_device)
            if bad is not None:
                pool.table[2, 1] = keep
            moves, live = pool.compact()
            if bad is not None:
                pool.table[2, 1] = bad
            got, n_live = g.compact(pool.pages)
            _pair(got, moves)
            assert int(n_live) == live
            g.same(pool, BAD_ROW if bad is not None else 0)
