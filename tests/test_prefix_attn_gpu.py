"""Attention over shared prefixes against dense attention in 64 bits."""
import math

import numpy as np
import pytest
import torch

import prefix_oracle as ref
from sparse_fp4_kv_b200 import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from sparse_fp4_kv_b200 import build
    build.build()
    from sparse_fp4_kv_b200 import binding
    return binding


class Case:
    """Sequences of `groups` (sizes) behind prefixes, each with a tail, on shuffled pages; inputs and the oracle."""

    def __init__(self, dev, groups, prefix, tails, h, ps, w=0, qps=1, seed=0, spare=1, ring=None, limits=None, qscale=1.0,
                 scale=1 / math.sqrt(512)):
        rng = np.random.default_rng(seed)
        n = sum(groups)
        self.batch = batch = n + spare
        slots = rng.permutation(batch)
        self.members = slots[:n].astype(np.int32)
        self.begin = np.concatenate([[0], np.cumsum(groups)]).astype(np.int32)
        self.prefix = np.array(prefix, np.int32)
        tails = np.resize(np.array(tails), n)
        self.seq_len = np.zeros(batch, np.int32)
        self.group = np.repeat(np.arange(len(groups)), groups)
        for j in range(n):
            self.seq_len[self.members[j]] = prefix[self.group[j]] + tails[j]
        width = max(1, -(-int(self.seq_len.max()) // ps)) + 1
        self.table = np.full((batch, width), -1, np.int32)
        need = sum(-(-int(x) // ps) for x in self.seq_len) + 2
        phys = rng.permutation(need)
        at = 0
        rows = need * ps
        self.codes = rng.integers(0, 256, (rows, 256)).astype(np.uint8)
        self.scales = rng.integers(40, 60, (rows, 32)).astype(np.uint8)  # 0.25 ... 1.75
        for g, size in enumerate(groups):
            shared = prefix[g] // ps
            common = phys[at:at + shared]
            at += shared
            for j in range(self.begin[g], self.begin[g + 1]):
                s = self.members[j]
                c = -(-int(self.seq_len[s]) // ps) - shared
                self.table[s, :shared + c] = np.concatenate([common, phys[at:at + c]])
                at += c
        self.ps, self.h, self.qps, self.w, self.scale = ps, h, qps, w, scale
        self.nq = batch * qps
        self.q = (synth.normal_bf16(seed + 1, 3, 0, self.nq * h * 512).view(self.nq, h, 512).float() * qscale).to(torch.bfloat16)
        self.limit = None
        if limits is not None:
            self.limit = np.array([limits(rng, int(self.seq_len[u // qps])) for u in range(self.nq)], np.int32)
        self.swa = self.wb = self.we = None
        if w:
            ring = ring or w + 11
            self.swa = synth.normal_e4m3(seed + 2, 4, 0, batch * ring * 512).view(batch, ring, 512)
            self.wb = rng.integers(0, ring, self.nq).astype(np.int32)
            self.we = (self.wb + rng.integers(0, w + 1, self.nq)).astype(np.int32)
            self.we[0] = self.wb[0] + w
        self.dev = dev

    def run(self, B, lse=True, ws=None, stream=None):
        t = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(self.dev)
        self.kv = B.KvCache(t(self.codes), t(self.scales), None, t(self.table), t(self.seq_len), self.ps)
        o = torch.full((self.nq, self.h, 512), 77.0, dtype=torch.bfloat16, device=self.dev)
        l = torch.full((self.nq, self.h), 77.0, device=self.dev) if lse else None
        if ws is None:
            ws = B.workspace(B.csa2_prefix_attn_workspace_size(len(self.members), len(self.prefix), self.qps, self.h), self.dev)
            ws.fill_(0xFF)  # what an earlier use left there must not matter
        swa = self.swa.to(self.dev) if self.w else None
        self.args = (self.q.to(self.dev), self.qps, self.kv, t(self.members), t(self.begin), t(self.prefix), t(self.limit), swa,
                     swa.shape[1] if self.w else 0, t(self.wb), t(self.we), self.w, self.scale, o, l, ws)
        B.csa2_prefix_attn_decode(*self.args, stream=stream)
        return o, l

    def rows(self, j, u):
        """The rows that query u of member j attends, in 64 bits."""
        s = int(self.members[j])
        first = int(self.members[self.begin[self.group[j]]])
        n = int(self.limit[u]) if self.limit is not None else int(self.seq_len[s])
        t = np.arange(max(n, 0))
        at = self.table[np.where(t < self.prefix[self.group[j]], first, s), t // self.ps].astype(np.int64) * self.ps + t % self.ps
        at = at[(at >= 0) & (at < len(self.codes))]
        v = ref.fp4_rows(self.codes[at], self.scales[at])
        if self.w:
            slot = np.arange(self.wb[u], self.we[u]) % self.swa.shape[1]
            v = np.concatenate([v, ref.e4m3_rows(self.swa[s].numpy()[slot])])
        return v

    def check(self, o, lse):
        o = o.double().cpu().numpy()
        lse = lse.double().cpu().numpy() if lse is not None else None
        listed = np.zeros(self.nq, bool)
        for j in range(len(self.members)):
            for u in range(self.members[j] * self.qps, (self.members[j] + 1) * self.qps):
                listed[u] = True
                want, wl, tol, tl = ref.attend(self.q[u].double().numpy(), self.rows(j, u), self.scale)
                off = np.abs(o[u] - want)
                assert (off <= tol).all(), f"query {u}: {off.max()} where {tol[np.unravel_index(off.argmax(), off.shape)]} may be"
                if lse is not None:
                    if np.isinf(wl).any():
                        assert (lse[u] == wl).all()
                    else:
                        assert (np.abs(lse[u] - wl) <= tl).all(), f"query {u}: lse"
        assert (o[~listed] == 77.0).all()  # sequences in no group stay as they were
        if lse is not None:
            assert (lse[~listed] == 77.0).all()


def _run(B, case, status=0, **kw):
    o, lse = case.run(B, **kw)
    assert B.csa2_device_status() == status
    case.check(o, lse)
    return o, lse


@pytest.mark.parametrize("h", [1, 3, 16, 32, 48, 64, 100, 128])
def test_head_counts(B, cuda_device, h):
    _run(B, Case(cuda_device, [3, 2], [300, 70], [0, 5, 40, 129], h, 64, w=20, seed=h))


@pytest.mark.parametrize("prefix", [0, 1, 31, 32, 63, 64, 65, 127, 128, 129, 255, 256, 257, 500])
def test_prefix_lengths(B, cuda_device, prefix):
    _run(B, Case(cuda_device, [4], [prefix], [0, 1, 64, 130], 16, 32, seed=prefix))


@pytest.mark.parametrize("ps", [32, 64, 128, 256, 1024])
@pytest.mark.parametrize("w", [0, 1, 130])
def test_pages_and_windows(B, cuda_device, ps, w):
    _run(B, Case(cuda_device, [2, 1, 3], [257, 0, 700], [3, 90, 0, 33], 32, ps, w=w, seed=ps + w))


@pytest.mark.parametrize("sizes", [[1], [1, 1, 1], [9], [5, 1, 17]])
@pytest.mark.parametrize("qps", [1, 3])
def test_groups_and_queries(B, cuda_device, sizes, qps):
    _run(B, Case(cuda_device, sizes, [200, 33, 400][:len(sizes)], [7, 0, 70], 16, 64, w=9, qps=qps, seed=len(sizes) * 10 + qps))


@pytest.mark.parametrize("sizes,prefix,h", [([13], [5000], 32), ([3, 20], [3001, 999], 64), ([2], [20011], 128), ([40], [1500], 16)])
def test_long_prefixes(B, cuda_device, sizes, prefix, h):
    _run(B, Case(cuda_device, sizes, prefix, [60, 1, 200], h, 64, w=33, seed=prefix[0]))


def test_limits_inside_the_prefix_and_empty_queries(B, cuda_device):
    """Limits of every kind: none visible, inside the prefix, at its end, inside the tail, all."""
    pick = lambda rng, n: int(rng.choice([0, -3, 1, 130, 256, 257, n // 2, n]).clip(max=n))
    _run(B, Case(cuda_device, [6, 3], [257, 300], [0, 40, 150], 16, 64, qps=4, seed=5, limits=pick))
    _run(B, Case(cuda_device, [6, 3], [257, 300], [0, 40, 150], 16, 64, qps=4, w=10, seed=6, limits=lambda rng, n: 0))


def test_rows_that_nobody_sees_may_hold_anything(B, cuda_device):
    """Entries behind every limit and spare pages hold NaN scales."""
    c = Case(cuda_device, [3], [200], [10, 20, 0], 16, 64, seed=8, limits=lambda rng, n: min(n, 205))
    used = np.zeros(len(c.codes), bool)
    for j in range(3):
        s, first = c.members[j], c.members[0]
        t = np.arange(min(205, c.seq_len[s]))
        used[c.table[np.where(t < 200, first, s), t // 64] * 64 + t % 64] = True
    c.scales[~used] = 0x7F
    _run(B, c)


@pytest.mark.parametrize("qscale,scale", [(1.0, 1.0), (30.0, 1 / math.sqrt(512)), (1.0, -0.3), (1.0, 0.0)])
def test_peaked_and_flat_scores(B, cuda_device, qscale, scale):
    """Scores far apart (the running maximum moves often), turned round, and all equal."""
    _run(B, Case(cuda_device, [5], [1200], [50, 3], 32, 64, w=17, seed=9, qscale=qscale, scale=scale))


def test_rising_scores(B, cuda_device):
    """Each tile raises the maximum: rows grow along the sequence."""
    c = Case(cuda_device, [3], [1000], [30], 16, 64, seed=10)
    first = c.members[0]
    for j in range(3):
        for t in range(int(c.seq_len[c.members[j]])):
            c.scales[c.table[first if t < 1000 else c.members[j], t // 64] * 64 + t % 64] = 16 + t // 18
    _run(B, c)


def test_bad_pages_are_left_out_and_reported(B, cuda_device):
    c = Case(cuda_device, [2], [256], [100, 70], 16, 64, seed=11)
    c.table[c.members[0], 1] = -1
    c.table[c.members[1], 4] = 10 ** 6
    _run(B, c, status=1)


def test_bad_windows_are_dropped_and_reported(B, cuda_device):
    c = Case(cuda_device, [4], [100], [5], 16, 64, w=8, seed=12)
    for j, (b, e) in enumerate([(-1, 4), (19, 20), (0, 9), (3, 3)]):
        c.wb[c.members[j]], c.we[c.members[j]] = b, e
    o, lse = c.run(B)
    assert B.csa2_device_status() == 1
    for j in range(4):
        c.wb[c.members[j]] = c.we[c.members[j]] = 0
    c.check(o, lse)


def test_bad_members_and_groups_are_skipped_and_reported(B, cuda_device):
    c = Case(cuda_device, [2, 2], [100, 64], [5, 80], 16, 64, seed=13, spare=2)
    o, lse = c.run(B)
    B.csa2_device_status()
    bad = list(c.args)
    for members, begin in ((c.members.copy(), [0, 2, 5]), (c.members.copy(), [-1, 2, 4]), (np.where(np.arange(4) == 1, 99, c.members), [0, 2, 4])):
        o2 = torch.full_like(o, 77.0)
        bad[3], bad[4] = (torch.tensor(np.asarray(x, np.int32), device=cuda_device) for x in (members, begin))
        bad[13] = o2
        B.csa2_prefix_attn_decode(*bad)
        assert B.csa2_device_status() == 1
        fine = [c.members[j] for j in range(4) if (begin[c.group[j]] >= 0 and begin[c.group[j] + 1] <= 4) and 0 <= members[j] < c.batch]
        for s in range(c.batch):
            if s in fine:
                assert torch.equal(o2[s], o[s])
            else:
                assert (o2[s] == 77.0).all()


def test_no_lse_and_repeatable(B, cuda_device):
    c = Case(cuda_device, [7], [2000], [300, 2], 32, 64, w=50, seed=14)
    o, lse = _run(B, c)
    o2, _ = c.run(B, lse=False)
    assert torch.equal(o, o2)


def test_two_streams_and_a_graph(B, cuda_device):
    """Two calls at once with workspaces of their own; a captured call replayed on new inputs."""
    a, b = (Case(cuda_device, [6], [3000], [40], 32, 64, w=16, seed=s) for s in (15, 16))
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    ra, rb = a.run(B), b.run(B)
    torch.cuda.synchronize()
    keep = [x.clone() for x in (*ra, *rb)]
    for x in (*ra, *rb):
        x.fill_(77.0)
    torch.cuda.synchronize()
    for _ in range(3):
        B.csa2_prefix_attn_decode(*a.args, stream=s1)
        B.csa2_prefix_attn_decode(*b.args, stream=s2)
    torch.cuda.synchronize()
    for x, y in zip((*ra, *rb), keep):
        assert torch.equal(x, y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.csa2_prefix_attn_decode(*a.args)
    a.args[0].copy_(b.args[0])
    a.q = b.q
    graph.replay()
    torch.cuda.synchronize()
    a.check(*ra)


def test_out_of_range_q_leaves_other_queries_alone(B, cuda_device):
    c = Case(cuda_device, [5], [700], [20], 16, 64, seed=17)
    o, lse = c.run(B)
    keep = o.clone()
    s = int(c.members[2])
    c.args[0][s, 3, 100] = 1e6
    B.csa2_prefix_attn_decode(*c.args)
    B.csa2_device_status()
    for j in (0, 1, 3, 4):
        assert torch.equal(o[int(c.members[j])], keep[int(c.members[j])])


def test_a_descending_group_list_computes_nothing(B, cuda_device):
    c = Case(cuda_device, [2, 2], [100, 64], [5, 80], 16, 64, seed=18)
    o, _ = c.run(B)
    B.csa2_device_status()
    args = list(c.args)
    for begin in ([0, 4, 2], [2, 0, 4]):
        args[4] = torch.tensor(begin, dtype=torch.int32, device=cuda_device)
        o.fill_(77.0)
        B.csa2_prefix_attn_decode(*args)
        assert B.csa2_device_status() == 1
        assert (o == 77.0).all()


def test_limits_beyond_the_table_are_cut_and_reported(B, cuda_device):
    """Two queries ask for more entries than a row of the table holds; the last pages of the rows are not there either."""
    c = Case(cuda_device, [3], [130], [10, 62, 0], 16, 64, seed=19)
    c.limit = c.seq_len.copy()
    c.limit[c.members[0]] = 2 ** 31 - 1
    c.limit[c.members[2]] = 10 ** 6
    o, lse = c.run(B)
    assert B.csa2_device_status() == 1
    c.limit = np.minimum(c.limit, c.table.shape[1] * c.ps)
    full = (c.table >= 0).sum(1) * c.ps  # rows of the pages that are there
    c.limit = np.minimum(c.limit, full).astype(np.int32)
    c.check(o, lse)


def test_empty_groups_and_an_unlisted_batch(B, cuda_device):
    """Groups without members between others, and a call without groups."""
    c = Case(cuda_device, [2, 0, 3, 0], [70, 5, 300, 9], [5, 80], 16, 64, seed=20, spare=4)
    _run(B, c)
    o = torch.full_like(c.args[13], 77.0)
    none = torch.empty(0, dtype=torch.int32, device=cuda_device)
    B.csa2_prefix_attn_decode(*c.args[:3], none, torch.zeros(1, dtype=torch.int32, device=cuda_device), none, *c.args[6:13], o, *c.args[14:])
    assert (o == 77.0).all() and B.csa2_device_status() == 0


def test_two_graphs_share_a_workspace(B, cuda_device):
    """Captured calls of different shapes over one workspace, replayed in turn on one stream."""
    a = Case(cuda_device, [6], [3000], [40], 32, 64, w=16, seed=21)
    b = Case(cuda_device, [1, 4], [90, 700], [5, 300], 64, 64, seed=22)
    size = max(B.csa2_prefix_attn_workspace_size(6, 1, 1, 32), B.csa2_prefix_attn_workspace_size(5, 2, 1, 64))
    ws = B.workspace(size, cuda_device)
    outs = [c.run(B, ws=ws) for c in (a, b)]
    torch.cuda.synchronize()
    graphs = []
    for c in (a, b):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            B.csa2_prefix_attn_decode(*c.args)
    for x in (*outs[0], *outs[1]):
        x.fill_(77.0)
    for i in (0, 1, 1, 0, 0, 1):
        graphs[i].replay()
    torch.cuda.synchronize()
    assert B.csa2_device_status() == 0
    a.check(*outs[0])
    b.check(*outs[1])


@pytest.mark.parametrize("n,split", [(200, 200), (256, 256), (5000, 5000), (5000, 0), (5000, 137)])
@pytest.mark.parametrize("gap", [17.0, 20.0, 23.0, 24.5, 25.5, 27.0])
def test_weak_weights_count_beside_a_strong_one(B, cuda_device, n, split, gap):
    """One entry 2^gap times as heavy as each of the others, which alone fill the latent values that it leaves zero.
    Their weights count in o as they do in lse: rounded to f16 they are off by at most 2^-11, or by 2^-32 of the
    heaviest one (half a step of f16's least numbers, the probabilities being at least 2^7 at the maximum)."""
    c = Case(cuda_device, [2], [split], [n - split], 16, 64, seed=int(gap), spare=0, scale=math.log(2))
    rng = np.random.default_rng(n + int(gap))
    c.codes &= 0x77  # no signs: nothing cancels
    c.codes[:, :8] = 0
    c.scales[:] = 0x38  # 1
    for s, first in ((int(c.members[0]), int(c.members[0])), (int(c.members[1]), int(c.members[0]))):
        t = int(rng.integers(0, n)) if split == 0 else 7  # in the prefix it is the first member's
        at = c.table[first if t < split else s, t // 64] * 64 + t % 64
        c.codes[at] = 0
        c.codes[at, :8] = 0x22  # sixteen values of 1
    c.q[:] = 0
    c.q[:, :, :16] = gap / 16  # a multiple of 1/32 below 2: exact
    o, lse = c.run(B)
    assert B.csa2_device_status() == 0
    for j in range(2):
        u = int(c.members[j])
        q, v = c.q[u].double().numpy(), c.rows(j, u)
        want, wl, _, tl = ref.attend(q, v, c.scale)
        s = q @ v.T * c.scale
        p = np.exp(s - s.max(1, keepdims=True))
        l = p.sum(1, keepdims=True)
        es = 512 * 2.0 ** -23 * (np.abs(q) @ np.abs(v).T).max(1) * c.scale + 2.0 ** -21 * (np.abs(s).max(1) + 1)
        tol = 2.0 ** -8 * np.abs(want) + ((2.0 ** -11 + 2 * es[:, None]) * p @ np.abs(v) + 2.0 ** -32 * np.abs(v).sum(0)) / l * 1.01
        off = np.abs(o[u].double().cpu().numpy() - want)
        assert (off <= tol).all(), f"member {j}: {(off / tol).max():.3g} times what it may be"
        assert (np.abs(lse[u].double().cpu().numpy() - wl) <= tl).all()


def test_more_than_65535_queries(B, cuda_device):
    """Two sequences with 35,001 queries each, each with a limit of its own."""
    c = Case(cuda_device, [2], [70], [30, 5], 2, 32, qps=35001, seed=23, spare=0, limits=lambda rng, n: int(rng.integers(0, n + 1)))
    o, lse = c.run(B)
    assert B.csa2_device_status() == 0
    for j in range(2):
        for u in range(int(c.members[j]) * c.qps, (int(c.members[j]) + 1) * c.qps, 1009):
            want, wl, tol, tl = ref.attend(c.q[u].double().numpy(), c.rows(j, u), c.scale)
            assert (np.abs(o[u].double().cpu().numpy() - want) <= tol).all()
            got = lse[u].double().cpu().numpy()
            assert (got == wl).all() if np.isinf(wl).any() else (np.abs(got - wl) <= tl).all()
    assert not (o == 77.0).all(-1).any()


@pytest.mark.parametrize("members,qps", [(1024, 1), (1025, 1), (512, 2), (205, 5), (1250, 2)])
def test_queries_around_the_plans_block(B, cuda_device, members, qps):
    """More queries than the plan's block has threads; many of them have no rows of their own."""
    third = members // 3
    _run(B, Case(cuda_device, [third, members - third], [65, 40], [0, 0, 3, 0, 40, 0, 0], 2, 32, qps=qps, seed=members + qps))


@pytest.mark.parametrize("groups", [1023, 1024, 1025, 1500])
def test_groups_around_the_plans_block(B, cuda_device, groups):
    """As many groups as the plan keeps in shared memory, and more: most of one member, some empty, runs of them
    without a prefix, and sequences without entries."""
    sizes = [0 if g % 7 == 3 else 3 if g % 11 == 5 else 1 for g in range(groups)]
    prefix = [0 if g % 5 == 0 or 300 <= g < 420 or g > groups - 9 else 1 + g % (90 if sizes[g] else 30)
              for g in range(groups)]
    _run(B, Case(cuda_device, sizes, prefix, [0, 2, 0, 0, 35], 2, 32, seed=groups))


@pytest.mark.parametrize("value", [65536.0, -65536.0, 3e38, -3e38, math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("at", [0, 511, 100, 101])
def test_out_of_range_q_is_reported(B, cuda_device, value, at):
    """Either half of a packed pair; the largest value in range is not reported, nor are queries that no group lists."""
    c = Case(cuda_device, [3], [90], [20], 16, 64, seed=24)
    c.run(B)
    assert B.csa2_device_status() == 0
    q = c.args[0]
    q[int(c.members[1]), 5, at] = 65280.0  # the bf16 value below 65536
    B.csa2_prefix_attn_decode(*c.args)
    assert B.csa2_device_status() == 0
    spare = (set(range(c.batch)) - set(c.members.tolist())).pop()
    q[spare, 5, at] = value
    B.csa2_prefix_attn_decode(*c.args)
    assert B.csa2_device_status() == 0
    q[int(c.members[1]), 5, at] = value
    B.csa2_prefix_attn_decode(*c.args)
    assert B.csa2_device_status() == 8


@pytest.mark.parametrize("qps,cut", [(2, 1), (4, 3), (7, 2)])
def test_fewer_queries_of_the_last_sequence(B, cuda_device, qps, cut):
    """nq that q_per_seq does not divide: what lies behind the last query is neither read nor written."""
    c = Case(cuda_device, [2, 3], [70, 300], [3, 90, 0], 16, 64, qps=qps, w=20, seed=25, spare=0, limits=lambda rng, n: int(rng.integers(1, n + 1)))
    full = c.nq
    c.nq -= cut
    for name in ("q", "limit", "wb", "we"):
        setattr(c, name, getattr(c, name)[:c.nq])
    o, lse = c.run(B)
    assert B.csa2_device_status() == 0
    seen = 0
    for j in range(len(c.members)):
        for u in range(c.members[j] * qps, min(c.nq, (c.members[j] + 1) * qps)):
            want, wl, tol, tl = ref.attend(c.q[u].double().numpy(), c.rows(j, u), c.scale)
            assert (np.abs(o[u].double().cpu().numpy() - want) <= tol).all()
            assert (np.abs(lse[u].double().cpu().numpy() - wl) <= tl).all()
            seen += 1
    assert seen == full - cut
