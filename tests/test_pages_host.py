"""Host-side checks of the page operators and of the attention over shared
prefixes (no GPU needed), and the page model's own invariants."""
import ctypes

import numpy as np
import pytest

from pages_model import Pool


@pytest.fixture(scope="module")
def binding():
    from sparse_fp4_kv_b200 import build
    build.build()
    from sparse_fp4_kv_b200 import binding as b
    return b


def _desc(binding, **kw):
    d = binding.csa2_kv_desc()
    base = dict(codes=0x10000, scales=0x20000, kidx=0x30000, page_table=0x40000, seq_len=0x50000, rows_cap=4096, d=512, di=64,
                page_size=64, max_pages=8, batch=4)
    for k, v in {**base, **kw}.items():
        setattr(d, k, v)
    return ctypes.pointer(d)


def test_page_operators_refuse_on_the_host(binding):
    L = binding._lib
    kv = _desc(binding)
    ws = binding.csa2_pages_workspace_size(3, 4, 64)
    # copy: descriptor, unsupported layout, keys of an unsupported width, lists
    assert L.csa2_pages_copy(None, 0x1000, 0x2000, 3, None) == 1
    assert L.csa2_pages_copy(_desc(binding, page_size=48), 0x1000, 0x2000, 3, None) == 2
    assert L.csa2_pages_copy(_desc(binding, di=32), 0x1000, 0x2000, 3, None) == 2
    assert L.csa2_pages_copy(_desc(binding, rows_cap=63), 0x1000, 0x2000, 3, None) in (1, 2)
    assert L.csa2_pages_copy(kv, 0x1000, None, 3, None) == 1
    assert L.csa2_pages_copy(kv, 0x1002, 0x2000, 3, None) == 1
    assert L.csa2_pages_copy(kv, 0x1000, 0x2000, -1, None) == 1
    assert L.csa2_pages_copy(kv, None, None, 0, None) == 0
    # fork and resize: arrays, one list without the other, the workspace
    assert L.csa2_pages_fork(kv, None, 0x1000, 0x2000, None, 3, None, None, 0x100, ws, None) == 1
    assert L.csa2_pages_fork(kv, 0x3000, 0x1000, None, None, 3, None, None, 0x100, ws, None) == 1
    assert L.csa2_pages_fork(kv, 0x3000, 0x1000, 0x2000, None, 3, 0x4000, None, 0x100, ws, None) == 1
    assert L.csa2_pages_fork(kv, 0x3000, 0x1000, 0x2000, None, 3, None, None, 0x100, ws - 1, None) == 3
    assert L.csa2_pages_fork(kv, 0x3000, 0x1000, 0x2000, None, 3, None, None, 0x110, ws, None) == 3
    assert L.csa2_pages_fork(kv, 0x3000, 0x1000, 0x2000, None, 0, None, None, None, 0, None) == 0
    assert L.csa2_pages_resize(kv, 0x3000, 0x1000, None, 3, None, None, 0x100, ws, None) == 1
    assert L.csa2_pages_resize(kv, 0x3000, 0x1000, 0x2000, -3, None, None, 0x100, ws, None) == 1
    assert L.csa2_pages_resize(kv, 0x3000, 0x1000, 0x2000, 3, None, None, None, 0, None) == 3
    # compact: lists and the workspace
    assert L.csa2_pages_compact(kv, 0x3000, None, 0x2000, None, 0x100, ws, None) == 1
    assert L.csa2_pages_compact(kv, 0x3000, 0x1000, 0x2000, None, None, 0, None) == 3
    assert binding.csa2_pages_workspace_size(-1, 4, 64) == 0
    assert binding.csa2_pages_workspace_size(0, 0, 64) == 0
    assert 0 < binding.csa2_pages_workspace_size(0, 4, 64) <= ws


def test_prefix_attention_refuses_on_the_host(binding):
    L = binding._lib
    f = L.csa2_prefix_attn_decode

    def call(nq=4, qps=1, h=16, kv=None, members=0x1000, n_members=3, begin=0x2000, prefix=0x3000, n_groups=2, limit=None, swa=None,
             stride=0, wb=None, we=None, w=0, scale=0.1, o=0x4000, lse=None, ws=0x10000, wsb=None, q=0x5000):
        if wsb is None:
            wsb = binding.csa2_prefix_attn_workspace_size(n_members, n_groups, qps, h)
        return f(q, nq, qps, h, kv or _desc(binding), members, n_members, begin, prefix, n_groups, limit, swa, stride, wb, we, w, scale,
                 o, lse, ws, wsb, None)

    assert call(h=0) == 2 and call(h=129) == 2
    assert call(nq=5) == 1 and call(nq=0) == 1 and call(qps=0, wsb=1 << 20) == 1
    assert call(n_members=5) == 1 and call(n_groups=4) == 1 and call(n_members=-1, n_groups=-1) == 1
    assert call(qps=2**31 - 1, n_members=1, n_groups=1, wsb=1 << 30) == 1  # more queries than a call takes
    assert call(members=None) == 1 and call(begin=None) == 1 and call(prefix=0x3001) == 1
    assert call(q=0x5008) == 1 and call(o=None) == 1 and call(lse=0x4002) == 1
    assert call(scale=float("nan")) == 1 and call(scale=float("inf")) == 1
    assert call(w=8) == 1 and call(wb=0x6000, w=8) == 1 and call(wb=0x6000, we=0x6100, swa=0x7000, stride=0, w=8) == 1
    assert call(kv=_desc(binding, d=256)) == 2
    swa = dict(wb=0x6000, we=0x6100, swa=0x7000)
    assert call(w=1 << 30, stride=8, **swa) == 2 and call(w=8, stride=1 << 30, **swa) == 2
    assert call(wsb=16) == 3 and call(ws=None) == 3 and call(ws=0x10010) == 3
    assert call(n_groups=0, wsb=0) == 0  # nothing to do
    assert binding.csa2_prefix_attn_workspace_size(3, 2, 1, 129) == 0
    assert binding.csa2_prefix_attn_workspace_size(0, 0, 1, 16) == 0


def test_page_model_keeps_counts(binding):
    rng = np.random.default_rng(0)
    pool = Pool(rng, 60, 32, 0, 10, 6)
    pool.fill(rng, [100, 64])
    pool.fork([0, 1, 0], [4, 5, 6], [100, 64, 40])
    pool.resize([0, 6, 4], [70, 0, 150])
    pool.compact()
    held = np.bincount(pool.table[pool.table >= 0], minlength=60)
    np.testing.assert_array_equal(held, pool.refs)
    assert not pool.refused and (pool.refs[int((pool.refs > 0).sum()):] == 0).all()


def test_prefix_attention_takes_up_to_2_17_listed_queries(binding):
    """The limit is on the listed queries; the check of the workspace comes behind it (nothing is launched)."""
    f = binding._lib.csa2_prefix_attn_decode

    def call(nq, qps, n_members):
        return f(0x5000, nq, qps, 2, _desc(binding, batch=1 << 20), 0x1000, n_members, 0x2000, 0x3000, 1, None, None, 0, None, None, 0, 0.1,
                 0x4000, None, 0x10000, 16, None)

    assert call(65535, 1, 65535) == 3 and call(65536, 1, 65536) == 3 and call(1 << 17, 1, 1 << 17) == 3
    assert call(70002, 35001, 2) == 3 and call(1 << 20, 1, 7) == 3
    assert call((1 << 17) + 1, 1, (1 << 17) + 1) == 1 and call(1 << 20, 1 << 16, 3) == 1
    assert binding.csa2_prefix_attn_workspace_size(1 << 17, 1, 1, 2) > 0
    assert binding.csa2_prefix_attn_workspace_size((1 << 17) + 1, 1, 1, 2) == 0


class _Tensor:
    """What the binding asks of a device tensor, without a device."""
    is_cuda = True

    def __init__(self, *shape, dtype=None):
        import torch
        self.shape, self.dtype = shape, dtype or torch.int32

    def numel(self):
        return int(np.prod(self.shape))

    def element_size(self):
        return self.dtype.itemsize

    @property
    def nbytes(self):
        return self.numel() * self.element_size()

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0x10000


@pytest.fixture
def calls(binding, monkeypatch):
    """The names of the library's calls that the binding makes; none of them runs."""
    made = []

    class Lib:
        def __getattr__(self, name):
            return lambda *args: made.append(name) or 0

    monkeypatch.setattr(binding, "_lib", Lib())
    monkeypatch.setattr(binding, "_stream", lambda stream: None)
    return made


def test_the_binding_checks_lists_and_tables(binding, calls):
    import torch
    u8, i64 = torch.uint8, torch.int64
    T = _Tensor

    def cache(rows=4 * 64, scales=None, keys=None, table=None, lens=None):
        return binding.KvCache(T(rows, 256, dtype=u8), scales or T(rows, 32, dtype=u8), keys or T(rows, 64, dtype=u8), table or T(3, 8),
                               lens or T(3), 64)

    kv, ws = cache(), T(4096, dtype=u8)
    # of each call: fine arguments (n = 5, 4 pages) and which of them have a least length of their own
    copy, fork, resize, compact = (getattr(binding, "csa2_pages_" + x) for x in ("copy", "fork", "resize", "compact"))
    table = [(copy, [kv, T(5), T(5)], [2]), (fork, [kv, T(4), T(5), T(5), T(5), T(5), T(5), ws], [1, 3, 4, 5, 6]),
             (resize, [kv, T(4), T(5), T(5), T(5), T(5), ws], [1, 3, 4, 5]), (compact, [kv, T(4), T(2), T(2), T(1), ws], [1, 2, 3, 4])]
    for f, args, _ in table:
        f(*args)
    fork(*table[1][1][:4], None, None, None, ws)
    resize(kv, T(9), T(5), T(6), None, None, ws)
    compact(kv, T(4), T(7), T(2), None, ws)
    assert len(calls) == 7
    unfit = [cache(scales=T(255, 32, dtype=u8)), cache(keys=T(255, 64, dtype=u8)), cache(table=T(3, 8, dtype=i64)),
             cache(lens=T(3, dtype=i64)), cache(lens=T(2))]
    for f, args, least in table:
        for i in range(1, len(args) - (f is not copy)):
            for bad in [T(*args[i].shape, dtype=i64)] + ([T(args[i].shape[0] - 1)] if i in least else []):
                with pytest.raises(ValueError):
                    f(*args[:i], bad, *args[i + 1:])
        for bad in unfit:
            with pytest.raises(ValueError):
                f(bad, *args[1:])
    assert len(calls) == 7


def test_the_binding_checks_the_prefix_attention(binding, calls):
    import torch
    T = _Tensor
    bf16, f32, u8 = torch.bfloat16, torch.float32, torch.uint8
    kv = binding.KvCache(T(256, 256, dtype=u8), T(256, 32, dtype=u8), None, T(3, 8), T(3), 64)
    fine = dict(q_bf16=T(6, 4, 512, dtype=bf16), q_per_seq=2, kv=kv, members=T(3), group_begin=T(3), prefix_len=T(2), q_limit=T(6),
                swa=T(3, 9, 512, dtype=u8), swa_seq_stride=9, swa_begin=T(6), swa_end=T(6), w_max=8, softmax_scale=0.1,
                o_bf16=T(6, 4, 512, dtype=bf16), lse=T(6, 4, dtype=f32), ws=T(1 << 20, dtype=u8))
    f = binding.csa2_prefix_attn_decode
    f(**fine)
    f(**{**fine, "q_limit": None, "lse": None})
    f(**{**fine, "swa": None, "swa_seq_stride": 0, "swa_begin": None, "swa_end": None, "w_max": 0})
    assert len(calls) == 3
    i64 = torch.int64
    for name, bad in [("q_bf16", T(6, 4, 512, dtype=f32)), ("q_bf16", T(6, 4, 256, dtype=bf16)), ("members", T(3, dtype=i64)),
                      ("group_begin", T(2)), ("group_begin", T(3, dtype=i64)), ("prefix_len", T(2, dtype=i64)), ("q_limit", T(5)),
                      ("q_limit", T(6, dtype=i64)), ("swa", T(3, 8, 512, dtype=u8)), ("swa_begin", T(5)), ("swa_end", T(6, dtype=f32)),
                      ("o_bf16", T(6, 4, 512, dtype=f32)), ("o_bf16", T(5, 4, 512, dtype=bf16)), ("lse", T(6, 4, dtype=bf16)),
                      ("lse", T(6, 3, dtype=f32))]:
        with pytest.raises(ValueError):
            f(**{**fine, name: bad})
    assert len(calls) == 3
