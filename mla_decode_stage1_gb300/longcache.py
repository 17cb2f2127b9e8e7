"""Binding of the operators that read less of a long cache: decode attention for
groups of requests that share a prefix, and the selection of pages by a score.

Marshalling only, like the package's other calls.  Shapes, dtypes and devices
(the current one) are checked here (ValueError); everything else is checked by the library
(MlaError).  Nothing synchronises but ``mla_shared_check``.
"""
from __future__ import annotations

import ctypes

import torch

from . import DTYPES, HEADS, QK_DIM, V_DIM, _check, _i32_array, _lib, _ptr
from .layer import (_dense, _need, _on_current_device, _pool, _POOLS, _several_devices, _stream, _vec,
                    _word)


class SharedInfo(ctypes.Structure):
    _fields_ = [("batch_size", ctypes.c_int32), ("num_groups", ctypes.c_int32),
                ("q_len", ctypes.c_int32), ("num_clusters", ctypes.c_int32),
                ("block_rows", ctypes.c_int32), ("num_items", ctypes.c_int32),
                ("prefix_tokens", ctypes.c_int64),
                ("own_tokens", ctypes.c_int64), ("workspace_bytes", ctypes.c_size_t)]


def _declare(lib):
    P, i32, i64, sz, e = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t,
                          ctypes.c_int)
    args = {
        "mla_shared_plan": [P, P, i32, P, P, i32, i32, e, e, i32, e, ctypes.POINTER(P)],
        "mla_shared_get_info": [P, ctypes.POINTER(SharedInfo)],
        "mla_shared_destroy": [P],
        "mla_shared_run": [P, P, P, P, P, P, i64, i64, P, P, P, sz, P, P, P],
        "mla_shared_check": [P, P, P],
        "mla_page_bounds": [P, e, P, i64, i64, i32, P, P, i32, P, i64, i32, P, i64, P, P],
        "mla_page_scores": [P, e, P, P, P, i64, P, i32, i32, i32, P, i64, i32, P, i64, P, P],
        "mla_page_select": [P, i64, P, i32, i32, i32, P, i64, i32, i32, i32, i32, P, P, P, i64, P, P,
                            P],
    }
    for name, a in args.items():
        fn = getattr(lib, name)
        fn.argtypes = a
        fn.restype = None if name == "mla_shared_destroy" else ctypes.c_int


_declare(_lib)
_shared_run, _page_bounds, _page_scores, _page_select = (
    _lib.mla_shared_run, _lib.mla_page_bounds, _lib.mla_page_scores, _lib.mla_page_select)

# (a look-up in torch costs 50 ns, a call makes up to ten)
_I32, _F32, _BF16, _U8 = torch.int32, torch.float32, torch.bfloat16, torch.uint8

FORMS = {"auto": 0, "once": 1, "each": 2}


class SharedPlan:
    """Owns an mla_shared* (host object)."""

    def __init__(self, handle, q_dtype, kv_dtype, prefix_entries, page_entries):
        self._h = handle
        self.q_dtype, self.kv_dtype = q_dtype, kv_dtype
        self.prefix_entries, self.page_entries = prefix_entries, page_entries
        info = self.info()
        self.query_tokens = info.batch_size * info.q_len
        self.workspace_bytes = info.workspace_bytes

    @property
    def handle(self):
        return self._h

    def info(self) -> SharedInfo:
        info = SharedInfo()
        _check("mla_shared_get_info", _lib.mla_shared_get_info(self._h, ctypes.byref(info)))
        return info

    def __del__(self):
        if getattr(self, "_h", None):
            _lib.mla_shared_destroy(self._h)
            self._h = None


def mla_shared_plan(group_indptr, prefix_indptr, kv_indptr, kv_last_page_len=None, *, page_size: int,
                    q_dtype: str, kv_dtype: str, q_len: int = 1, num_sms: int = 0,
                    form: str = "auto") -> SharedPlan:
    """Plan a decode call from HOST offsets: group_indptr (requests of each
    group), prefix_indptr (pages of each group's shared prefix, all full) and
    kv_indptr (pages of each request's own) with optional last-page lengths.
    form: "once" (a prefix is read once for up to 16 query tokens), "each" (for
    every request), or "auto" (what is expected to be faster)."""
    _need(form in FORMS, f"form must be one of {tuple(FORMS)}")
    grp, grp_p = _i32_array(group_indptr)
    pre, pre_p = _i32_array(prefix_indptr)
    kvp, kvp_p = _i32_array(kv_indptr)
    last, last_p = _i32_array(kv_last_page_len)
    groups = len(grp) - 1
    _need(groups >= 1, "group_indptr must have at least two entries")
    _need(len(pre) == groups + 1, f"prefix_indptr must have {groups + 1} entries")
    bs = int(grp[-1])
    _need(len(kvp) == bs + 1, f"kv_indptr must have {bs + 1} entries")
    _need(last is None or len(last) == bs, f"kv_last_page_len must have {bs} entries")
    h = ctypes.c_void_p()
    _check("mla_shared_plan", _lib.mla_shared_plan(
        grp_p, pre_p, groups, kvp_p, last_p, int(q_len), int(page_size), DTYPES[q_dtype],
        DTYPES[kv_dtype], int(num_sms), FORMS[form], ctypes.byref(h)))
    return SharedPlan(h, q_dtype, kv_dtype, int(pre[-1]), int(kvp[-1]))


_Q_DTYPES = {"bf16": _BF16, "fp8": _U8}


def _table(name, t, entries):
    """Pointer of a page table with room for the plan's entries, or None."""
    if t is None:
        return None
    if not (t.is_cuda and t.dtype is _I32 and t.dim() == 1 and t.is_contiguous()
            and t.shape[0] >= entries):
        _vec(name, t, _I32)
        raise ValueError(f"{name} must hold the plan's {entries} pages")
    return t.data_ptr()


def _query_ok(q, dtype, tokens):
    """Whether q is [tokens, 16, 576] (or [requests, q_len, 16, 576]), dense."""
    size = q.shape
    return (q.is_cuda and q.dtype is dtype and q.is_contiguous() and len(size) >= 3
            and size[-1] == QK_DIM and size[-2] == HEADS and q.numel() == tokens * (HEADS * QK_DIM))


def mla_shared_run(plan: SharedPlan, q, kv, out, *, workspace, prefix_indices=None, kv_indices=None,
                   q_scale=None, kv_scale=None, kv_e8m0=None, lse=None, stream=None) -> None:
    """Enqueue one decode call of the plan: q [tokens, 16, 576] bf16 or uint8
    (e4m3 bytes), kv the pool as mla_decode_run takes it, out bf16 [tokens, 16,
    512], lse fp32 [tokens, 16] or None (tokens: requests x q_len), workspace a
    uint8 CUDA tensor of at least plan.workspace_bytes."""
    if _several_devices:
        _on_current_device(stream, q, kv, out, workspace, prefix_indices, kv_indices, q_scale, kv_scale,
                           kv_e8m0, lse)
    T = plan.query_tokens
    if not _query_ok(q, _Q_DTYPES[plan.q_dtype], T):
        raise ValueError(f"q must be a contiguous CUDA tensor [{T}, {HEADS}, {QK_DIM}] of "
                         f"{_Q_DTYPES[plan.q_dtype]}")
    if not (out.is_cuda and out.dtype is _BF16 and out.is_contiguous()
            and out.numel() == T * (HEADS * V_DIM)):
        _dense("out", out, _BF16, (T, HEADS, V_DIM))
    if lse is not None and not (lse.is_cuda and lse.dtype is _F32 and lse.is_contiguous()
                                and lse.numel() == T * HEADS):
        _dense("lse", lse, _F32, (T, HEADS))
    qs = None
    if plan.q_dtype == "fp8":
        _need(q_scale is not None, "fp8 q needs q_scale")
        _word("q_scale", q_scale, _F32)
        qs = q_scale.data_ptr()
    if not (workspace.is_cuda and workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous CUDA tensor")
    scale, e8, e8_stride = _pool(kv, plan.kv_dtype, kv_scale, kv_e8m0)
    status = _shared_run(
        plan.handle, q.data_ptr(), qs, kv.data_ptr(), scale, e8, e8_stride, kv.shape[0],
        _table("prefix_indices", prefix_indices, plan.prefix_entries),
        _table("kv_indices", kv_indices, plan.page_entries), workspace.data_ptr(), workspace.nbytes,
        out.data_ptr(), None if lse is None else lse.data_ptr(), _stream(stream, q))
    if status:
        _check("mla_shared_run", status)


def mla_shared_check(plan: SharedPlan, workspace, stream=None) -> None:
    """mla_decode_check for a shared plan's workspace."""
    if _several_devices:
        _on_current_device(stream, workspace)
    _check("mla_shared_check", _lib.mla_shared_check(plan.handle, workspace.data_ptr(),
                                                     _stream(stream, workspace)))


class MlaShared:
    """Convenience owner of a shared plan and its workspace."""

    def __init__(self, group_indptr, prefix_indptr, kv_indptr, kv_last_page_len=None, *, page_size,
                 q_dtype, kv_dtype, q_len=1, form="auto", device="cuda"):
        self.plan = mla_shared_plan(group_indptr, prefix_indptr, kv_indptr, kv_last_page_len,
                                    page_size=page_size, q_dtype=q_dtype, kv_dtype=kv_dtype,
                                    q_len=q_len, form=form)
        self.workspace = torch.empty(self.plan.workspace_bytes, dtype=_U8, device=device)

    def __call__(self, q, kv, out, **kw):
        mla_shared_run(self.plan, q, kv, out, workspace=self.workspace, **kw)
        return out


def _blocks(block_table, bs):
    """(pointer, row stride, columns) of a block table with dense rows."""
    size, strides = block_table.shape, block_table.stride()
    if not (block_table.is_cuda and block_table.dtype is _I32 and len(size) == 2
            and size[0] == bs and (strides[1] == 1 or size[1] <= 1)):
        raise ValueError(f"block_table must be a CUDA tensor [{bs}, columns] of torch.int32 with "
                         "dense rows")
    return block_table.data_ptr(), strides[0] if bs > 1 else size[1], size[1]


def _bounds(bounds):
    size = bounds.shape
    if not (bounds.is_cuda and bounds.dtype is _BF16 and len(size) == 3 and size[1] == 2
            and size[2] == QK_DIM and bounds.is_contiguous()):
        raise ValueError(f"bounds must be a contiguous CUDA tensor [pages, 2, {QK_DIM}] of bfloat16")
    return size[0]


def _lengths(name, t):
    if not (t.is_cuda and t.dtype is _I32 and t.dim() == 1 and t.is_contiguous()):
        _vec(name, t, _I32)
    return t.shape[0]


def mla_page_bounds(kv, bounds, block_table, old_lens, new_lens=None, *, page_size: int,
                    kv_dtype: str, kv_e8m0=None, err=None, stream=None) -> None:
    """Bring the bounds of the pages that got rows up to date: bounds bf16
    [pages, 2, 576], the smallest and the largest stored value of every dim over
    a page's rows.  kv the pool as mla_decode_run takes it, block_table int32
    [requests, columns], old_lens / new_lens int32 [requests] (new_lens None: one
    new token each) as for mla_cache_step.  With old_lens 0 everything is done
    anew."""
    if _several_devices:
        _on_current_device(stream, kv, bounds, block_table, old_lens, new_lens, kv_e8m0, err)
    bs = _lengths("old_lens", old_lens)
    if new_lens is not None and _lengths("new_lens", new_lens) != bs:
        raise ValueError(f"new_lens must have {bs} elements")
    table, stride, columns = _blocks(block_table, bs)
    pages = _bounds(bounds)
    _word("err", err, _I32)
    width, dtype = _POOLS[kv_dtype]
    size = kv.shape
    if not (kv.is_cuda and kv.dtype is dtype and len(size) == 2 and size[1] == width
            and kv.is_contiguous()):
        raise ValueError(f"kv must be a contiguous CUDA tensor [rows, {width}] of {dtype}")
    e8, e8_stride = None, 0
    if kv_dtype == "mxfp4":
        _, e8, e8_stride = _pool(kv, kv_dtype, None, kv_e8m0)
    status = _page_bounds(kv.data_ptr(), DTYPES[kv_dtype], e8, e8_stride, size[0], page_size,
                          old_lens.data_ptr(), _ptr(new_lens), bs, table, stride, columns,
                          bounds.data_ptr(), pages, _ptr(err), _stream(stream, kv))
    if status:
        _check("mla_page_bounds", status)


def _scores(scores, rows, columns):
    """Row stride of scores [rows, at least columns] with dense rows."""
    size, strides = scores.shape, scores.stride()
    if not (scores.is_cuda and scores.dtype is _F32 and len(size) == 2 and size[0] == rows
            and size[1] >= columns and (strides[1] == 1 or size[1] <= 1)):
        raise ValueError(f"scores must be a CUDA tensor [{rows}, >= {columns}] of float32 with dense "
                         "rows")
    return strides[0] if rows > 1 else size[1]


def mla_page_scores(q, bounds, block_table, lens, scores, *, page_size: int, q_len: int = 1,
                    q_scale=None, kv_scale=None, err=None, stream=None) -> None:
    """Upper bounds of the decode call's scores, page by page: scores fp32
    [requests * q_len, columns], -inf where a query token sees no token of a
    page.  q as mla_decode_run takes it (uint8: e4m3 bytes, with q_scale, which a
    bf16 q ignores), lens int32 [requests] with the new tokens."""
    if _several_devices:
        _on_current_device(stream, q, bounds, block_table, lens, scores, q_scale, kv_scale, err)
    bs = _lengths("lens", lens)
    table, stride, columns = _blocks(block_table, bs)
    pages = _bounds(bounds)
    fp8 = q.dtype is _U8
    if not _query_ok(q, _U8 if fp8 else _BF16, bs * q_len):
        raise ValueError(f"q must be a contiguous CUDA tensor [{bs * q_len}, {HEADS}, {QK_DIM}] of "
                         "bfloat16 or uint8")
    _need(q_scale is not None or not fp8, "fp8 q needs q_scale")
    _word("q_scale", q_scale, _F32)
    _word("kv_scale", kv_scale, _F32)
    _word("err", err, _I32)
    status = _page_scores(q.data_ptr(), 1 if fp8 else 0, _ptr(q_scale), _ptr(kv_scale),
                          bounds.data_ptr(), pages, lens.data_ptr(), bs, q_len, page_size, table,
                          stride, columns, scores.data_ptr(), _scores(scores, bs * q_len, columns),
                          _ptr(err), _stream(stream, q))
    if status:
        _check("mla_page_scores", status)


def mla_page_select(scores, block_table, lens, *, page_size: int, top_pages: int,
                    first_pages: int = 1, last_pages: int = 1, q_len: int = 1, kv_indptr,
                    kv_last_page_len, kv_indices, columns=None, err=None, stream=None) -> None:
    """The page table of the best pages of every row (requests * q_len): all of
    a row with at most top_pages, else the first, the last, and of those between
    the ones with the largest scores.  Outputs: kv_indptr int32 [rows+1],
    kv_last_page_len int32 [rows], kv_indices int32 [capacity], columns int32
    [rows, top_pages] (-1 past the kept ones)."""
    if _several_devices:
        _on_current_device(stream, scores, block_table, lens, kv_indptr, kv_last_page_len, kv_indices,
                           columns, err)
    bs = _lengths("lens", lens)
    rows = bs * q_len
    table, stride, cols = _blocks(block_table, bs)
    if not (kv_indptr.is_cuda and kv_indptr.dtype is _I32 and kv_indptr.is_contiguous()
            and kv_indptr.shape == (rows + 1,) and kv_last_page_len.is_cuda
            and kv_last_page_len.dtype is _I32 and kv_last_page_len.is_contiguous()
            and kv_last_page_len.shape == (rows,) and kv_indices.is_cuda and kv_indices.dtype is _I32
            and kv_indices.is_contiguous() and kv_indices.dim() == 1):
        _vec("kv_indptr", kv_indptr, _I32, rows + 1)
        _vec("kv_last_page_len", kv_last_page_len, _I32, rows)
        _vec("kv_indices", kv_indices, _I32)
    if columns is not None:
        _dense("columns", columns, _I32, (rows, top_pages))
    _word("err", err, _I32)
    status = _page_select(scores.data_ptr(), _scores(scores, rows, cols), lens.data_ptr(), bs, q_len,
                          page_size, table, stride, cols, top_pages, first_pages, last_pages,
                          kv_indptr.data_ptr(), kv_last_page_len.data_ptr(), kv_indices.data_ptr(),
                          kv_indices.shape[0], _ptr(columns), _ptr(err), _stream(stream, scores))
    if status:
        _check("mla_page_select", status)
