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
