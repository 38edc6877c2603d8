"""Python binding of libcsa2.so: the C-ABI calls under the same names.

Argument marshalling only: torch tensors are turned into device pointers and
sizes, the caller's current CUDA stream is passed along, and a non-OK status
raises. The page operators and the attention over shared prefixes refuse lists,
tables and outputs of another type or too short, which the C ABI cannot see.
Every step of the computation runs in the library's kernels; there is
no fallback of any kind. If the library is missing the import fails.
"""
import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libcsa2.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is not built; run `python -m sparse_fp4_kv_b200.build` (nvcc, sm_100a)")

_lib = ctypes.CDLL(LIB_PATH)

_INT32 = torch.int32
_raw_stream, _current_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice

CSA2_D = 512
CSA2_ATTN_STATIC_SCRATCH_BYTES = 16 << 20
STATUS = {0: "ok", 1: "invalid argument", 2: "unsupported configuration",
          3: "workspace missing or too small", 4: "CUDA error", 5: "device-side error recorded"}


class Csa2Error(RuntimeError):
    def __init__(self, call, status):
        super().__init__(f"{call}: {STATUS.get(status, status)} (status {status})")
        self.status = status


class csa2_kv_desc(ctypes.Structure):
    _fields_ = [
        ("codes", ctypes.c_void_p),
        ("scales", ctypes.c_void_p),
        ("kidx", ctypes.c_void_p),
        ("page_table", ctypes.c_void_p),
        ("seq_len", ctypes.c_void_p),
        ("rows_cap", ctypes.c_int64),
        ("d", ctypes.c_int32),
        ("di", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("max_pages", ctypes.c_int32),
        ("batch", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
    ]


_vp, _i32, _i64, _sz, _f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
_kvp = ctypes.POINTER(csa2_kv_desc)
_SIGS = {
    "csa2_append_fp4": (_i32, [_vp, _i32, _vp, _vp, _kvp, _vp]),
    "csa2_index_full": (_i32, [_vp, _vp, _i32, _i32, _i32, _vp, _i64, _kvp, _i32, _i32, _vp, _vp, _vp, _sz,
                               _vp]),
    "csa2_append_swa_e4m3": (_i32, [_vp, _i32, _vp, _vp, _vp, _i32, _i64, _vp]),
    "csa2_append_kidx_e4m3": (_i32, [_vp, _i32, _vp, _vp, _kvp, _vp]),
    "csa2_index_full_workspace_size": (_sz, [_i32, _i64]),
    "csa2_index_reindex": (_i32, [_vp, _vp, _i32, _i32, _i32, _vp, _i32, _kvp, _i32, _vp, _vp, _sz, _vp]),
    "csa2_index_reindex_workspace_size": (_sz, [_i32, _i32]),
    "csa2_sparse_attn_decode": (_i32, [_vp, _i32, _i32, _i32, _kvp, _vp, _i32, _vp, _i64, _vp, _vp, _i32,
                                       _f32, _vp, _vp, _vp, _sz, _vp]),
    "csa2_sparse_attn_workspace_size": (_sz, [_i32, _i32, _i32, _i32]),
    "csa2_sparse_attn_decode_nvfp4": (_i32, [_vp, _i32, _i32, _i32, _kvp, _vp, _i32, _vp, _i64, _vp, _vp, _i32,
                                             _f32, _vp, _vp, _vp, _sz, _vp]),
    "csa2_sparse_attn_nvfp4_workspace_size": (_sz, [_i32, _i32, _i32, _i32]),
    "csa2_sparse_attn_decode_static": (_i32, [_vp, _i32, _i32, _i32, _kvp, _vp, _i32, _vp, _i64, _vp, _vp, _i32,
                                              _f32, _vp, _vp, _vp]),
    "csa2_pages_copy": (_i32, [_kvp, _vp, _vp, _i32, _vp]),
    "csa2_pages_fork": (_i32, [_kvp, _vp, _vp, _vp, _vp, _i32, _vp, _vp, _vp, _sz, _vp]),
    "csa2_pages_resize": (_i32, [_kvp, _vp, _vp, _vp, _i32, _vp, _vp, _vp, _sz, _vp]),
    "csa2_pages_compact": (_i32, [_kvp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "csa2_pages_workspace_size": (_sz, [_i32, _i32, _i64]),
    "csa2_prefix_attn_decode": (_i32, [_vp, _i32, _i32, _i32, _kvp, _vp, _i32, _vp, _vp, _i32, _vp, _vp, _i64, _vp,
                                       _vp, _i32, _f32, _vp, _vp, _vp, _sz, _vp]),
    "csa2_prefix_attn_workspace_size": (_sz, [_i32, _i32, _i32, _i32]),
    "csa2_score_ids": (_i32, [_vp, _vp, _i32, _i32, _i32, _vp, _i32, _kvp, _i32, _vp, _vp]),
    "csa2_select_keys": (_i32, [_vp, _i32, _i32, _i32, _vp, _vp]),
    "csa2_sparse_attn_partial": (_i32, [_vp, _i32, _i32, _i32, _kvp, _vp, _i32, _vp, _i64, _vp, _vp, _i32,
                                        _f32, _vp, _vp, _vp, _sz, _vp]),
    "csa2_attn_merge": (_i32, [_vp, _vp, _i32, _i32, _i32, _vp, _vp, _vp]),
    "csa2_device_status": (_i32, [_vp, ctypes.POINTER(ctypes.c_uint32)]),
    "csa2_check_wait_timeout": (_i32, [ctypes.c_uint32, _vp]),
    "csa2_status_string": (ctypes.c_char_p, [_i32]),
    "csa2_version": (_i32, []),
}
for _name, (_res, _args) in _SIGS.items():
    _fn = getattr(_lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args

EXPORTED = tuple(_SIGS)


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("device tensor expected")
    if not t.is_contiguous():
        raise ValueError("contiguous tensor expected")
    return t.data_ptr()


def _ints(t, n, what):
    """The address of a list of at least n int32 values (None: null)."""
    if t is None:
        return None
    if t.dtype is _INT32 and t.numel() >= n and t.is_cuda and t.is_contiguous():
        return t.data_ptr()
    return _refused(t, _INT32, n, what)


def _refused(t, dtype, n, what):
    """Raises what is wrong with a tensor that should hold n values of dtype on the device."""
    if t.dtype is not dtype or t.numel() < n:
        raise ValueError(f"{what}: at least {n} values of {dtype} expected, got {t.numel()} of {t.dtype}")
    return _ptr(t)


def _stream(stream):
    if stream is not None:
        return stream.cuda_stream
    # the current stream's handle without building a Stream object (4.6 us a call, as long as a small kernel); a
    # tensor on the device has initialised CUDA
    return _raw_stream(_current_device())


def _check(call, st):
    if st != 0:
        raise Csa2Error(call, st)


class KvCache:
    """The shared global KV cache: torch tensors plus the C descriptor.

    codes [rows_cap, 256] u8, scales [rows_cap, 32] u8, kidx [rows_cap, di] u8,
    page_table [batch, max_pages] i32, seq_len [batch] i32 (all on the device).
    """

    def __init__(self, codes, scales, kidx, page_table, seq_len, page_size):
        self.codes, self.scales, self.kidx = codes, scales, kidx
        self.page_table, self.seq_len = page_table, seq_len
        self.page_size = int(page_size)
        d = ctypes.pointer(csa2_kv_desc())
        d.contents.codes = _ptr(codes)
        d.contents.scales = _ptr(scales)
        d.contents.kidx = _ptr(kidx) if kidx is not None else None
        d.contents.page_table = _ptr(page_table)
        d.contents.seq_len = _ptr(seq_len)
        d.contents.rows_cap = codes.shape[0]
        d.contents.d = CSA2_D
        d.contents.di = kidx.shape[1] if kidx is not None else 0
        d.contents.page_size = self.page_size
        d.contents.max_pages = page_table.shape[1]
        d.contents.batch = page_table.shape[0]
        self.desc = d
        rows, batch = codes.shape[0], page_table.shape[0]
        self.num_pages = rows // self.page_size if self.page_size > 0 else 0
        # what keeps the page operators from writing this cache (None: nothing)
        self.unwritable = None
        for name, t, n in (("codes", codes, rows * CSA2_D // 2), ("scales", scales, rows * CSA2_D // 16),
                           ("kidx", kidx, rows * self.di)):
            if t is not None and t.numel() * t.element_size() < n:
                self.unwritable = f"{name}: {n} bytes expected for {rows} rows, got {t.numel() * t.element_size()}"
        for name, t, n in (("page_table", page_table, page_table.numel()), ("seq_len", seq_len, batch)):
            if t.dtype is not torch.int32 or t.numel() < n:
                self.unwritable = f"{name}: at least {n} int32 values expected, got {t.numel()} of {t.dtype}"

    def written(self):
        """The descriptor, for a call that writes tables, lengths and rows."""
        if self.unwritable is not None:
            raise ValueError(self.unwritable)
        return self.desc

    @property
    def di(self):
        return self.desc.contents.di


def csa2_append_fp4(x_bf16, seq, pos, kv: KvCache, stream=None):
    n = x_bf16.shape[0] if x_bf16.dim() == 2 else 0
    _check("csa2_append_fp4", _lib.csa2_append_fp4(_ptr(x_bf16), n, _ptr(seq), _ptr(pos), kv.desc,
                                                   _stream(stream)))


def csa2_index_full_workspace_size(nq, n_max):
    return _lib.csa2_index_full_workspace_size(nq, n_max)


def csa2_index_full(qidx, w, q_per_seq, q_limit, n_max, kv: KvCache, k, p, topk, pool, ws, stream=None):
    nq, hi = qidx.shape[0], qidx.shape[1]
    _check("csa2_index_full", _lib.csa2_index_full(
        _ptr(qidx), _ptr(w), nq, q_per_seq, hi, _ptr(q_limit), int(n_max), kv.desc, k, p, _ptr(topk),
        _ptr(pool), _ptr(ws), ws.numel() * ws.element_size() if ws is not None else 0, _stream(stream)))


def csa2_index_reindex_workspace_size(nq, p):
    return _lib.csa2_index_reindex_workspace_size(nq, p)


def csa2_index_reindex(qidx, w, q_per_seq, pool, kv: KvCache, k, topk, ws, stream=None):
    nq, hi = qidx.shape[0], qidx.shape[1]
    p = pool.shape[1]
    _check("csa2_index_reindex", _lib.csa2_index_reindex(
        _ptr(qidx), _ptr(w), nq, q_per_seq, hi, _ptr(pool), p, kv.desc, k, _ptr(topk), _ptr(ws),
        ws.numel() * ws.element_size() if ws is not None else 0, _stream(stream)))


def csa2_sparse_attn_workspace_size(nq, h, k, w_max):
    return _lib.csa2_sparse_attn_workspace_size(nq, h, k, w_max)


def csa2_sparse_attn_decode(q_bf16, q_per_seq, kv: KvCache, topk, swa, swa_seq_stride, swa_begin, swa_end,
                            w_max, softmax_scale, o_bf16, lse, ws, stream=None):
    nq, h = q_bf16.shape[0], q_bf16.shape[1]
    k = topk.shape[1] if topk is not None else 0
    _check("csa2_sparse_attn_decode", _lib.csa2_sparse_attn_decode(
        _ptr(q_bf16), nq, q_per_seq, h, kv.desc, _ptr(topk), k, _ptr(swa), int(swa_seq_stride),
        _ptr(swa_begin), _ptr(swa_end), int(w_max), float(softmax_scale), _ptr(o_bf16), _ptr(lse),
        _ptr(ws), ws.numel() * ws.element_size() if ws is not None else 0, _stream(stream)))


def csa2_sparse_attn_decode_static(q_bf16, q_per_seq, kv: KvCache, topk, swa, swa_seq_stride, swa_begin, swa_end,
                                   w_max, softmax_scale, o_bf16, lse, stream=None):
    """csa2_sparse_attn_decode with the library's fixed device scratch
    (CSA2_ATTN_STATIC_SCRATCH_BYTES) in place of a caller workspace, for
    callers that cannot allocate device memory. Calls whose kernels can
    overlap on one device share that scratch and race."""
    nq, h = q_bf16.shape[0], q_bf16.shape[1]
    k = topk.shape[1] if topk is not None else 0
    _check("csa2_sparse_attn_decode_static", _lib.csa2_sparse_attn_decode_static(
        _ptr(q_bf16), nq, q_per_seq, h, kv.desc, _ptr(topk), k, _ptr(swa), int(swa_seq_stride),
        _ptr(swa_begin), _ptr(swa_end), int(w_max), float(softmax_scale), _ptr(o_bf16), _ptr(lse),
        _stream(stream)))


def csa2_sparse_attn_nvfp4_workspace_size(nq, h, k, w_max):
    return _lib.csa2_sparse_attn_nvfp4_workspace_size(nq, h, k, w_max)


def csa2_sparse_attn_decode_nvfp4(q_bf16, q_per_seq, kv: KvCache, topk, swa, swa_seq_stride, swa_begin, swa_end,
                                  w_max, softmax_scale, o_bf16, lse, ws, stream=None):
    """csa2_sparse_attn_decode with q quantised to NVFP4 for the scores (FP4
    block-scaled products on the selected entries); h = 64."""
    nq, h = q_bf16.shape[0], q_bf16.shape[1]
    k = topk.shape[1] if topk is not None else 0
    _check("csa2_sparse_attn_decode_nvfp4", _lib.csa2_sparse_attn_decode_nvfp4(
        _ptr(q_bf16), nq, q_per_seq, h, kv.desc, _ptr(topk), k, _ptr(swa), int(swa_seq_stride),
        _ptr(swa_begin), _ptr(swa_end), int(w_max), float(softmax_scale), _ptr(o_bf16), _ptr(lse),
        _ptr(ws), ws.numel() * ws.element_size() if ws is not None else 0, _stream(stream)))


def csa2_append_swa_e4m3(x_bf16, seq, pos, swa, stream=None):
    """Window rows x [n][512] into ring slots pos % ring_rows of swa [batch][ring_rows][512]."""
    _check("csa2_append_swa_e4m3", _lib.csa2_append_swa_e4m3(
        _ptr(x_bf16), x_bf16.shape[0], _ptr(seq), _ptr(pos), _ptr(swa), swa.shape[0], swa.shape[1],
        _stream(stream)))


def csa2_append_kidx_e4m3(x_bf16, seq, pos, kv: KvCache, stream=None):
    """Indexer keys x [n][di] into the physical rows of (seq, pos) of the key array."""
    _check("csa2_append_kidx_e4m3", _lib.csa2_append_kidx_e4m3(
        _ptr(x_bf16), x_bf16.shape[0], _ptr(seq), _ptr(pos), kv.desc, _stream(stream)))


def _bytes(ws):
    return ws.nbytes if ws is not None else 0


def csa2_pages_workspace_size(n, batch, num_pages):
    return _lib.csa2_pages_workspace_size(n, batch, num_pages)


def csa2_pages_copy(kv: KvCache, src, dst, stream=None):
    """Pages src[i] -> dst[i] (codes, scales, keys); -1 is an empty slot."""
    n = src.numel()
    _check("csa2_pages_copy", _lib.csa2_pages_copy(kv.written(), _ints(src, n, "src"), _ints(dst, n, "dst"), n, _stream(stream)))


def csa2_pages_fork(kv: KvCache, refs, parent, child, length, copy_src, copy_dst, ws, stream=None):
    """Empty sequences child[i] become the first length[i] entries (None: all) of parent[i], sharing whole pages."""
    n = parent.numel()
    _check("csa2_pages_fork", _lib.csa2_pages_fork(
        kv.written(), _ints(refs, kv.num_pages, "refs"), _ints(parent, n, "parent"), _ints(child, n, "child"),
        _ints(length, n, "length"), n, _ints(copy_src, n, "copy_src"), _ints(copy_dst, n, "copy_dst"), _ptr(ws), _bytes(ws),
        _stream(stream)))


def csa2_pages_resize(kv: KvCache, refs, seq, new_len, copy_src, copy_dst, ws, stream=None):
    """seq[i] gets new_len[i] entries: pages are released or taken, 0 frees the sequence."""
    n = seq.numel()
    _check("csa2_pages_resize", _lib.csa2_pages_resize(
        kv.written(), _ints(refs, kv.num_pages, "refs"), _ints(seq, n, "seq"), _ints(new_len, n, "new_len"), n,
        _ints(copy_src, n, "copy_src"), _ints(copy_dst, n, "copy_dst"), _ptr(ws), _bytes(ws), _stream(stream)))


def csa2_pages_compact(kv: KvCache, refs, move_src, move_dst, n_live, ws, stream=None):
    """Live pages move into the lowest page numbers; the moves go to move_src / move_dst (then -1)."""
    moves = kv.num_pages // 2
    _check("csa2_pages_compact", _lib.csa2_pages_compact(
        kv.written(), _ints(refs, kv.num_pages, "refs"), _ints(move_src, moves, "move_src"), _ints(move_dst, moves, "move_dst"),
        _ints(n_live, 1, "n_live"), _ptr(ws), _bytes(ws), _stream(stream)))


def csa2_prefix_attn_workspace_size(n_members, n_groups, q_per_seq, h):
    return _lib.csa2_prefix_attn_workspace_size(n_members, n_groups, q_per_seq, h)


def csa2_prefix_attn_decode(q_bf16, q_per_seq, kv: KvCache, members, group_begin, prefix_len, q_limit, swa, swa_seq_stride,
                            swa_begin, swa_end, w_max, softmax_scale, o_bf16, lse, ws, stream=None):
    """Attention over whole sequences and their windows, each group's first prefix_len entries read once for all of it."""
    nq, h = q_bf16.shape[0], q_bf16.shape[1]
    n_groups, n = prefix_len.shape[0], nq * h * CSA2_D
    for t, name in ((q_bf16, "q_bf16"), (o_bf16, "o_bf16")):
        if t.dtype is not torch.bfloat16 or t.numel() < n:
            _refused(t, torch.bfloat16, n, name)
    if lse is not None and (lse.dtype is not torch.float32 or lse.numel() < nq * h):
        _refused(lse, torch.float32, nq * h, "lse")
    if swa is not None and q_per_seq > 0 and _bytes(swa) < -(-nq // q_per_seq) * int(swa_seq_stride) * CSA2_D:
        raise ValueError(f"swa: {_bytes(swa)} bytes are not {int(swa_seq_stride)} rows for each sequence")
    _check("csa2_prefix_attn_decode", _lib.csa2_prefix_attn_decode(
        _ptr(q_bf16), nq, q_per_seq, h, kv.desc, _ints(members, 0, "members"), members.shape[0],
        _ints(group_begin, n_groups + 1, "group_begin"), _ints(prefix_len, n_groups, "prefix_len"), n_groups,
        _ints(q_limit, nq, "q_limit"), _ptr(swa), int(swa_seq_stride), _ints(swa_begin, nq, "swa_begin"),
        _ints(swa_end, nq, "swa_end"), int(w_max), float(softmax_scale), _ptr(o_bf16), _ptr(lse), _ptr(ws), _bytes(ws),
        _stream(stream)))


def csa2_score_ids(qidx, w, q_per_seq, ids, kv: KvCache, id_offset, keys, stream=None):
    """Unique 64-bit keys (score key << 32 | ~(id + id_offset)) of ids [nq][m] (local to kv)."""
    nq, hi = qidx.shape[0], qidx.shape[1]
    _check("csa2_score_ids", _lib.csa2_score_ids(_ptr(qidx), _ptr(w), nq, q_per_seq, hi, _ptr(ids), ids.shape[1],
                                                 kv.desc, int(id_offset), _ptr(keys), _stream(stream)))


def csa2_select_keys(keys, k, ids, stream=None):
    """The ids carried by the k largest of each query's keys [nq][m] (padded with -1)."""
    _check("csa2_select_keys", _lib.csa2_select_keys(_ptr(keys), keys.shape[0], keys.shape[1], int(k), _ptr(ids),
                                                     _stream(stream)))


def csa2_sparse_attn_partial(q_bf16, q_per_seq, kv: KvCache, topk, swa, swa_seq_stride, swa_begin, swa_end,
                             w_max, softmax_scale, o_f32, lse, ws, stream=None):
    nq, h = q_bf16.shape[0], q_bf16.shape[1]
    k = topk.shape[1] if topk is not None else 0
    _check("csa2_sparse_attn_partial", _lib.csa2_sparse_attn_partial(
        _ptr(q_bf16), nq, q_per_seq, h, kv.desc, _ptr(topk), k, _ptr(swa), int(swa_seq_stride),
        _ptr(swa_begin), _ptr(swa_end), int(w_max), float(softmax_scale), _ptr(o_f32), _ptr(lse),
        _ptr(ws), ws.numel() * ws.element_size() if ws is not None else 0, _stream(stream)))


def csa2_attn_merge(o_parts, lse_parts, o_bf16, lse, stream=None):
    """Merge g partials o_parts [g][nq][h][512] f32, lse_parts [g][nq][h] into bf16 o and lse."""
    g, nq, h = o_parts.shape[0], o_parts.shape[1], o_parts.shape[2]
    _check("csa2_attn_merge", _lib.csa2_attn_merge(_ptr(o_parts), _ptr(lse_parts), g, nq, h, _ptr(o_bf16), _ptr(lse),
                                                   _stream(stream)))


def csa2_device_status(stream=None):
    code = ctypes.c_uint32(0)
    st = _lib.csa2_device_status(_stream(stream), ctypes.byref(code))
    if st not in (0, 5):
        raise Csa2Error("csa2_device_status", st)
    return code.value


def csa2_check_wait_timeout(limit_us, stream=None):
    """Launch the bounded-wait self-check (a wait that runs out after limit_us)."""
    _check("csa2_check_wait_timeout", _lib.csa2_check_wait_timeout(int(limit_us), _stream(stream)))


def csa2_status_string(status):
    return _lib.csa2_status_string(status).decode()


def csa2_version():
    return _lib.csa2_version()


def workspace(nbytes, device):
    """A device byte buffer (256-byte aligned by the caching allocator)."""
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)
