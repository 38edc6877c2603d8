"""The page operators and the attention over shared prefixes together, as a
serving loop uses them, next to the appends and the sparse attention; and rows
whose offsets pass 32 bits."""
import math

import numpy as np
import pytest
import torch

import prefix_oracle as ref
from helpers import normal_bf16_rows
from sparse_fp4_kv_b200 import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from sparse_fp4_kv_b200 import build
    build.build()
    from sparse_fp4_kv_b200 import binding
    return binding


def _i32(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


class Server:
    """A pool, its tables and the calls a scheduler makes of them."""

    def __init__(self, B, dev, batch, pages, ps, width, caches=1):
        self.B, self.dev, self.ps, self.pages = B, dev, ps, pages
        self.table = torch.full((batch, width), -1, dtype=torch.int32, device=dev)
        self.seq_len = torch.zeros(batch, dtype=torch.int32, device=dev)
        self.refs = torch.zeros(pages, dtype=torch.int32, device=dev)
        z = lambda w: torch.zeros((pages * ps, w), dtype=torch.uint8, device=dev)
        self.kvs = [B.KvCache(z(256), z(32), z(64), self.table, self.seq_len, ps) for _ in range(caches)]
        self.ws = B.workspace(B.csa2_pages_workspace_size(batch, batch, pages), dev)

    def lists(self, n):
        return torch.empty(n, dtype=torch.int32, device=self.dev), torch.empty(n, dtype=torch.int32, device=self.dev)

    def resize(self, seq, new_len):
        src, dst = self.lists(len(seq))
        self.B.csa2_pages_resize(self.kvs[0], self.refs, _i32(seq, self.dev), _i32(new_len, self.dev), src, dst, self.ws)
        for kv in self.kvs[1:]:
            self.B.csa2_pages_copy(kv, src, dst)

    def fork(self, parent, child):
        src, dst = self.lists(len(parent))
        self.B.csa2_pages_fork(self.kvs[0], self.refs, _i32(parent, self.dev), _i32(child, self.dev), None, src, dst, self.ws)
        for kv in self.kvs[1:]:
            self.B.csa2_pages_copy(kv, src, dst)

    def compact(self):
        src, dst = self.lists(self.pages // 2)
        live = _i32([0], self.dev)
        self.B.csa2_pages_compact(self.kvs[0], self.refs, src, dst, live, self.ws)
        for kv in self.kvs[1:]:
            self.B.csa2_pages_copy(kv, src, dst)
        return int(live)

    def append(self, seq, pos, rows):
        for c, kv in enumerate(self.kvs):
            x = (rows.float() * (1 + c)).to(torch.bfloat16)
            self.B.csa2_append_fp4(x.to(self.dev), _i32(seq, self.dev), torch.tensor(pos, device=self.dev), kv)

    def rows(self, c, b):
        n = int(self.seq_len[b])
        t = torch.arange(n, device=self.dev)
        at = self.table[b].long()[t // self.ps] * self.ps + t % self.ps
        return ref.fp4_rows(self.kvs[c].codes[at].cpu().numpy(), self.kvs[c].scales[at].cpu().numpy())


def test_a_serving_loop(B, cuda_device):
    """A prompt, four samples of it over a few steps, a compaction between two steps, and everything freed. Two
    caches behind one table. After each step the prefix attention is compared with dense attention over each
    sequence's rows, and with the sparse attention given all ids."""
    dev, ps, h, prompt = cuda_device, 32, 16, 300
    s = Server(B, dev, 6, 80, ps, 16, caches=2)
    s.resize([5, 0], [90, prompt])
    s.append([5] * 90, list(range(90)), normal_bf16_rows(1, 1, 90))
    s.append([0] * prompt, list(range(prompt)), normal_bf16_rows(2, 1, prompt))
    s.resize([5], [0])  # another request ended: its pages are holes now
    s.fork([0, 0, 0], [2, 1, 4])
    members = [0, 2, 1, 4]
    contents = None
    for step in range(4):
        lens = [int(s.seq_len[b]) for b in members]
        s.resize(members, [n + 1 for n in lens])
        s.append(members, lens, normal_bf16_rows(10 + step, 1, 4))
        if step == 2:
            before = [s.rows(c, b) for c in range(2) for b in members]
            live = s.compact()
            assert live == int((s.refs > 0).sum()) and (s.refs[live:] == 0).all()
            for x, y in zip(before, [s.rows(c, b) for c in range(2) for b in members]):
                np.testing.assert_array_equal(x, y)
        q = synth.normal_bf16(step, 3, 0, 6 * h * 512).view(6, h, 512).to(dev)
        for c, kv in enumerate(s.kvs):
            o, lse = torch.zeros_like(q), torch.zeros((6, h), device=dev)
            ws = B.workspace(B.csa2_prefix_attn_workspace_size(4, 1, 1, h), dev)
            B.csa2_prefix_attn_decode(q, 1, kv, _i32(members, dev), _i32([0, 4], dev), _i32([prompt], dev), None, None, 0, None, None, 0,
                                      1 / math.sqrt(512), o, lse, ws)
            k = prompt + 8
            topk = torch.arange(k, dtype=torch.int32, device=dev)[None].expand(6, k)
            topk = torch.where(topk < s.seq_len[:, None], topk, -1).contiguous()
            o2, lse2 = torch.zeros_like(q), torch.zeros((6, h), device=dev)
            ws2 = B.workspace(B.csa2_sparse_attn_workspace_size(6, h, k, 0), dev)
            B.csa2_sparse_attn_decode(q, 1, kv, topk, None, 0, None, None, 0, 1 / math.sqrt(512), o2, lse2, ws2)
            for b in members:
                want, wl, tol, tl = ref.attend(q[b].double().cpu().numpy(), s.rows(c, b), 1 / math.sqrt(512))
                for got, gl in ((o, lse), (o2, lse2)):
                    assert (np.abs(got[b].double().cpu().numpy() - want) <= tol).all()
                    assert (np.abs(gl[b].double().cpu().numpy() - wl) <= tl).all()
    assert B.csa2_device_status() == 0
    # samples differ from each other behind the prompt and share its whole pages
    a, b = s.rows(0, 0), s.rows(0, 2)
    np.testing.assert_array_equal(a[:prompt], b[:prompt])
    assert not np.array_equal(a[prompt:], b[prompt:])
    assert int((s.refs > 1).sum()) == prompt // ps
    s.resize(members, [0] * 4)
    assert int(s.refs.abs().sum()) == 0 and (s.table == -1).all() and (s.seq_len == 0).all()
    assert B.csa2_device_status() == 0


def test_offsets_past_32_bits(B, cuda_device):
    """A cache of 18 million rows (4.6 GB of codes): pages at its end are copied, forked, compacted and attended."""
    dev, ps, rows = cuda_device, 64, 18_000_000 // 64 * 64
    pages = rows // ps
    codes = torch.empty((rows, 256), dtype=torch.uint8, device=dev)
    scales = torch.empty((rows, 32), dtype=torch.uint8, device=dev)
    table = torch.full((3, 8), -1, dtype=torch.int32, device=dev)
    seq_len = _i32([200, 0, 70], dev)
    refs = torch.zeros(pages, dtype=torch.int32, device=dev)
    kv = B.KvCache(codes, scales, None, table, seq_len, ps)
    rng = np.random.default_rng(0)
    hc = rng.integers(0, 256, (300, 256)).astype(np.uint8)
    hs = rng.integers(40, 60, (300, 32)).astype(np.uint8)
    top = pages - 4
    codes[top * ps:] = torch.from_numpy(hc[:256]).to(dev)
    scales[top * ps:] = torch.from_numpy(hs[:256]).to(dev)
    table[0, :4] = _i32([top, top + 1, top + 2, top + 3], dev)
    refs[top:] = 1
    # page 3 of the sequence copied to a page at 4.4 GB
    mid = 17_200_000 // ps
    B.csa2_pages_copy(kv, _i32([top + 3, top + 1], dev), _i32([mid, mid + 1], dev))
    assert torch.equal(codes[mid * ps:mid * ps + ps], codes[(top + 3) * ps:])
    table[2, :2] = _i32([mid, mid + 1], dev)
    refs[mid:mid + 2] = 1
    ws = B.workspace(B.csa2_pages_workspace_size(1, 3, pages), dev)
    B.csa2_pages_fork(kv, refs, _i32([0], dev), _i32([1], dev), None, None, None, ws)

    def attend():
        q = synth.normal_bf16(5, 3, 0, 3 * 16 * 512).view(3, 16, 512).to(dev)
        o, lse = torch.zeros_like(q), torch.zeros((3, 16), device=dev)
        wa = B.workspace(B.csa2_prefix_attn_workspace_size(3, 2, 1, 16), dev)
        B.csa2_prefix_attn_decode(q, 1, kv, _i32([0, 1, 2], dev), _i32([0, 2, 3], dev), _i32([192, 0], dev), None, None, 0, None, None,
                                  0, 1 / math.sqrt(512), o, lse, wa)
        whole = ref.fp4_rows(hc, hs)
        for b, v in ((0, whole[:200]), (1, whole[:200]), (2, np.concatenate([whole[192:256], whole[64:70]]))):
            want, wl, tol, _ = ref.attend(q[b].double().cpu().numpy(), v, 1 / math.sqrt(512))
            assert (np.abs(o[b].double().cpu().numpy() - want) <= tol).all()

    attend()
    src, dst = (torch.empty(pages // 2, dtype=torch.int32, device=dev) for _ in range(2))
    live = _i32([0], dev)
    B.csa2_pages_compact(kv, refs, src, dst, live, ws)
    assert int(live) == 7 and int(table.max()) == 6
    attend()
    assert B.csa2_device_status() == 0
