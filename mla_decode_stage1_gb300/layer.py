"""Binding of the operators around the decode call: the cache step, the cache
write, the absorbed form's two products and the expanded form.

Marshalling only, like the package's other calls.  Shapes, dtypes and devices
(the current one) are checked here (ValueError); everything else is checked by the library
(MlaError).  Nothing synchronises but the ``_check`` calls.
"""
from __future__ import annotations

import ctypes

import torch

from . import DTYPES, _check, _i32_array, _lib, _ptr

LATENT, ROPE, NOPE, V_HEAD = 512, 64, 128, 128
ROW = LATENT + ROPE
ROPES = {"interleaved": 0, "half": 1}


class PrefillInfo(ctypes.Structure):
    _fields_ = [("batch_size", ctypes.c_int32), ("heads", ctypes.c_int32),
                ("num_ctas", ctypes.c_int32), ("num_items", ctypes.c_int32),
                ("num_partials", ctypes.c_int32), ("query_tokens", ctypes.c_int64),
                ("key_tokens", ctypes.c_int64), ("workspace_bytes", ctypes.c_size_t)]


def _declare(lib):
    P, i32, i64, sz, f32 = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t,
                            ctypes.c_float)
    e = ctypes.c_int
    args = {
        "mla_cache_step": [P, P, i32, i32, P, i64, i32, P, i32, P, P, P, i64, P, P, P, i64, P, P, P],
        "mla_cache_write": [P, i64, P, i64, P, f32, P, i64, P, e, P, i64, e, P, P, P, i64, i64, P,
                            P, P],
        "mla_absorb_q": [P, i64, i64, P, i64, i32, f32, P, i64, P, e, e, P, P, P, P],
        "mla_absorb_out": [P, P, i64, i32, P, P],
        "mla_absorb_out_ex": [P, P, i64, i32, P, P, P],
        "mla_selftest_absorb_wait": [P, P, i64, i32, P, P, i32, ctypes.c_uint32, P, P],
        "mla_prefill_plan": [P, P, P, i32, i32, i32, e, i32, ctypes.POINTER(P)],
        "mla_prefill_get_info": [P, ctypes.POINTER(PrefillInfo)],
        "mla_prefill_destroy": [P],
        "mla_prefill_run": [P, P, i64, i64, P, P, P, i64, i64, P, P, f32, P, i64, P, e, P, sz, P, P,
                            P],
        "mla_prefill_check": [P, P, P],
        "mla_error_check": [P, P],
    }
    for name, a in args.items():
        fn = getattr(lib, name)
        fn.argtypes = a
        fn.restype = None if name == "mla_prefill_destroy" else ctypes.c_int


_declare(_lib)
_cache_step, _cache_write, _absorb_q, _absorb_out, _prefill_run = (
    _lib.mla_cache_step, _lib.mla_cache_write, _lib.mla_absorb_q, _lib.mla_absorb_out_ex,
    _lib.mla_prefill_run)

# The handle of a device's current stream.  torch.cuda.current_stream builds a
# Stream object first, 2.8 us a call on the Grace host against 0.1 us.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)


def _stream(stream, t):
    """The stream to enqueue on: the caller's, or the current one of t's device."""
    return _raw_stream(t.get_device()) if stream is None else stream.cuda_stream


# The library launches on the current device.  Only with several devices can a
# tensor be on another one; asking each costs 0.5 us a call.
_several_devices = torch.cuda.device_count() > 1
_current_device = torch.cuda.current_device


def _on_current_device(stream, *tensors):
    dev = _current_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"every tensor must be on the current CUDA device, {dev}")
    if stream is not None and stream.device.index != dev:
        raise ValueError(f"stream must be one of the current CUDA device, {dev}")


def _need(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


def _vec(name, t, dtype, n=None):
    """A contiguous one-dimensional CUDA tensor of this type (and length)."""
    if not (t.is_cuda and t.dtype is dtype and t.dim() == 1 and t.is_contiguous()
            and (n is None or t.shape[0] == n)):
        raise ValueError(f"{name} must be a contiguous CUDA tensor of {dtype}"
                         + ("" if n is None else f" with {n} elements"))


def _word(name, t, dtype):
    """A CUDA scalar (one element) of this type, or None."""
    if t is not None and not (t.is_cuda and t.dtype is dtype and t.numel() == 1):
        raise ValueError(f"{name} must be a CUDA tensor of one {dtype}")


def _rotation(cos_sin, positions, tokens):
    """(cos_sin pointer, its rows, positions pointer), checked."""
    if cos_sin is None and positions is None:
        return None, 0, None
    _need(cos_sin is not None and positions is not None,
          "cos_sin and positions go together (both or neither)")
    size = cos_sin.shape
    if not (cos_sin.is_cuda and cos_sin.dtype is torch.float32 and len(size) == 2
            and size[1] == ROPE and cos_sin.is_contiguous()):
        raise ValueError(f"cos_sin must be a contiguous CUDA tensor [positions, {ROPE}] of float32")
    if not (positions.is_cuda and positions.dtype is torch.int32 and positions.is_contiguous()
            and positions.numel() == tokens):
        _vec("positions", positions, torch.int32, tokens)
    return cos_sin.data_ptr(), size[0], positions.data_ptr()


_POOLS = {"bf16": (ROW, torch.bfloat16), "fp8": (ROW, torch.uint8),
          "mxfp4": (ROW // 2, torch.uint8)}


def _pool(kv, kv_dtype, kv_scale, kv_e8m0):
    """(scale pointer, e8m0 pointer, e8m0 row stride) of a checked pool."""
    width, dtype = _POOLS[kv_dtype]
    size = kv.shape
    if not (kv.is_cuda and kv.dtype is dtype and len(size) == 2 and size[1] == width
            and kv.is_contiguous()):
        raise ValueError(f"kv must be a contiguous CUDA tensor [rows, {width}] of {dtype}")
    if kv_dtype == "fp8":
        _need(kv_scale is not None, "fp8 KV needs kv_scale")
        _word("kv_scale", kv_scale, torch.float32)
        return kv_scale.data_ptr(), None, 0
    if kv_dtype == "mxfp4":
        if kv_e8m0 is None or not (kv_e8m0.is_cuda and kv_e8m0.dtype is torch.uint8
                                   and kv_e8m0.dim() == 2 and kv_e8m0.shape[0] >= kv.shape[0]
                                   and kv_e8m0.shape[1] >= ROW // 32 and kv_e8m0.stride(1) == 1):
            raise ValueError(f"MXFP4 KV needs kv_e8m0, a CUDA tensor [rows, >= {ROW // 32}] of uint8")
        return None, kv_e8m0.data_ptr(), kv_e8m0.stride(0)
    return None, None, 0


def _weights(w):
    size = w.shape
    if not (w.is_cuda and w.dtype is torch.bfloat16 and len(size) == 3
            and size[1] == NOPE + V_HEAD and size[2] == LATENT and w.is_contiguous()):
        raise ValueError(f"w must be a contiguous CUDA tensor [heads, {NOPE + V_HEAD}, {LATENT}] "
                         "of bfloat16")
    return size[0]


def _query(q, heads):
    """(tokens, token stride, head stride) of q [tokens, heads, 192]; the
    stride of a dimension of size 1 is never used and takes its dense value."""
    size, strides = q.shape, q.stride()
    if not (q.is_cuda and q.dtype is torch.bfloat16 and len(size) == 3 and size[1] == heads
            and size[2] == NOPE + ROPE and strides[2] == 1):
        raise ValueError(f"q must be a CUDA tensor [tokens, {heads}, {NOPE + ROPE}] of bfloat16 "
                         "with a dense last dimension")
    return (size[0], strides[0] if size[0] > 1 else heads * (NOPE + ROPE),
            strides[1] if heads > 1 else NOPE + ROPE)


def _dense(name, t, dtype, shape):
    if not (t.is_cuda and t.dtype is dtype and t.shape == shape and t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous CUDA tensor {list(shape)} of {dtype}")


def mla_cache_step(old_lens, new_lens, block_table, free_pages, *, page_size: int, kv_indptr,
                   kv_last_page_len, kv_indices, qo_indptr, slots, positions, pages_used=None,
                   err=None, stream=None) -> None:
    """Hand out pages for a step and build its page table, slots and positions
    from request lengths on the device (one launch, nothing read on the host).

    old_lens / new_lens int32 [bs] (new_lens None: one token each); block_table
    int32 [bs, columns] with dense rows, updated in place; free_pages int32.
    Outputs: kv_indptr, qo_indptr int32 [bs+1], kv_last_page_len int32 [bs],
    kv_indices int32 [capacity], slots int64 [capacity] (-1 past the last
    token), positions int32 [capacity], pages_used int32 [1].  What went wrong
    on the device (pages ran out, ...) is in err, read by mla_error_check.
    """
    if _several_devices:
        _on_current_device(stream, old_lens, new_lens, block_table, free_pages, kv_indptr,
                           kv_last_page_len, kv_indices, qo_indptr, slots, positions, pages_used,
                           err)
    i32 = torch.int32
    bs = old_lens.shape[0]
    # one pass over the common case; what is wrong is worked out only if it fails
    # (arrays of a given length may have any shape, the others are lists)
    if not (old_lens.dtype is i32 and old_lens.is_cuda and old_lens.is_contiguous()
            and old_lens.dim() == 1
            and (new_lens is None or (new_lens.dtype is i32 and new_lens.is_cuda
                                      and new_lens.is_contiguous() and new_lens.numel() == bs))
            and block_table.dtype is i32 and block_table.is_cuda and block_table.dim() == 2
            and free_pages.dtype is i32 and free_pages.is_cuda and free_pages.is_contiguous()
            and free_pages.dim() == 1
            and kv_indptr.dtype is i32 and kv_indptr.is_cuda and kv_indptr.is_contiguous()
            and kv_indptr.numel() == bs + 1
            and kv_last_page_len.dtype is i32 and kv_last_page_len.is_cuda
            and kv_last_page_len.is_contiguous() and kv_last_page_len.numel() == bs
            and kv_indices.dtype is i32 and kv_indices.is_cuda and kv_indices.is_contiguous()
            and kv_indices.dim() == 1
            and qo_indptr.dtype is i32 and qo_indptr.is_cuda and qo_indptr.is_contiguous()
            and qo_indptr.numel() == bs + 1
            and slots.dtype is torch.int64 and slots.is_cuda and slots.is_contiguous()
            and slots.dim() == 1
            and positions.dtype is i32 and positions.is_cuda and positions.is_contiguous()
            and positions.numel() == slots.numel()
            and (pages_used is None or (pages_used.dtype is i32 and pages_used.is_cuda
                                        and pages_used.numel() == 1))
            and (err is None or (err.dtype is i32 and err.is_cuda and err.numel() == 1))):
        _vec("old_lens", old_lens, i32)
        if new_lens is not None:
            _vec("new_lens", new_lens, i32, bs)
        for name, x, n in (("free_pages", free_pages, None), ("kv_indptr", kv_indptr, bs + 1),
                           ("kv_last_page_len", kv_last_page_len, bs),
                           ("kv_indices", kv_indices, None), ("qo_indptr", qo_indptr, bs + 1)):
            _vec(name, x, i32, n)
        _vec("slots", slots, torch.int64)
        _vec("positions", positions, i32, slots.numel())
        _word("pages_used", pages_used, i32)
        _word("err", err, i32)
        raise ValueError("block_table must be a CUDA tensor [requests, columns] of torch.int32")
    rows, columns = block_table.shape
    stride, dense = block_table.stride()
    if rows != bs or (columns > 1 and dense != 1):
        raise ValueError(f"block_table must be [{bs}, columns] with dense rows")
    status = _cache_step(
        old_lens.data_ptr(), None if new_lens is None else new_lens.data_ptr(), bs, page_size,
        block_table.data_ptr(), stride if bs > 1 else columns, columns, free_pages.data_ptr(),
        free_pages.numel(), kv_indptr.data_ptr(), kv_last_page_len.data_ptr(),
        kv_indices.data_ptr(), kv_indices.numel(), qo_indptr.data_ptr(), slots.data_ptr(),
        positions.data_ptr(), slots.numel(), None if pages_used is None else pages_used.data_ptr(),
        None if err is None else err.data_ptr(), _stream(stream, old_lens))
    if status:
        _check("mla_cache_step", status)


def mla_cache_write(latent, k_rope, kv, slots, *, kv_dtype: str, norm_weight=None,
                    eps: float = 1e-6, positions=None, cos_sin=None, rope: str = "interleaved",
                    kv_scale=None, kv_e8m0=None, rows=None, err=None, stream=None) -> None:
    """Write the rows of new tokens into the cache: norm of the latent
    (norm_weight None: none), rotation of the position dims, the pool's encoding.

    latent bf16 [T,512] and k_rope bf16 [T,64] (dense last dimension; the row
    stride of latent a multiple of 8 elements), slots int64 [T] (-1: not
    stored), kv the pool as mla_decode_run takes it, rows (optional) bf16
    [T,576]: the values that the stored encoding stands for.
    """
    if _several_devices:
        _on_current_device(stream, latent, k_rope, kv, slots, norm_weight, positions, cos_sin,
                           kv_scale, kv_e8m0, rows, err)
    T = slots.numel()
    bf16 = torch.bfloat16
    ls, rs = latent.stride(), k_rope.stride()
    if not (slots.dtype is torch.int64 and slots.is_cuda and slots.is_contiguous()
            and latent.dtype is bf16 and latent.is_cuda and latent.shape == (T, LATENT)
            and ls[1] == 1 and k_rope.dtype is bf16 and k_rope.is_cuda
            and k_rope.shape == (T, ROPE) and rs[1] == 1
            and (norm_weight is None
                 or (norm_weight.dtype is bf16 and norm_weight.is_cuda
                     and norm_weight.is_contiguous() and norm_weight.numel() == LATENT))
            and (err is None or (err.dtype is torch.int32 and err.is_cuda and err.numel() == 1))):
        _vec("slots", slots, torch.int64)
        for name, x, n in (("latent", latent, LATENT), ("k_rope", k_rope, ROPE)):
            _need(x.is_cuda and x.dtype is bf16 and tuple(x.shape) == (T, n) and x.stride(1) == 1,
                  f"{name} must be a CUDA tensor [{T}, {n}] of bfloat16 with a dense last dimension")
        if norm_weight is not None:
            _vec("norm_weight", norm_weight, bf16, LATENT)
        _word("err", err, torch.int32)
    if rows is not None:
        _dense("rows", rows, bf16, (T, ROW))
    scale, e8, e8_stride = _pool(kv, kv_dtype, kv_scale, kv_e8m0)
    cs, npos, pos = _rotation(cos_sin, positions, T)
    status = _cache_write(
        latent.data_ptr(), ls[0] if T > 1 else LATENT, k_rope.data_ptr(),
        rs[0] if T > 1 else ROPE, _ptr(norm_weight), eps, cs, npos, pos, ROPES[rope],
        slots.data_ptr(), T, DTYPES[kv_dtype], kv.data_ptr(), scale, e8, e8_stride, kv.shape[0],
        _ptr(rows), _ptr(err), _stream(stream, slots))
    if status:
        _check("mla_cache_write", status)


def mla_absorb_q(q, w, q_out, *, sm_scale: float, positions=None, cos_sin=None,
                 rope: str = "interleaved", q_scale=None, err=None, stream=None) -> None:
    """The decode call's query from a layer's query q bf16 [T, heads, 192]:
    q_out [T, heads, 576], bf16, or uint8 (e4m3 bytes of the value divided by
    q_scale).  The decode call's scores then carry sm_scale."""
    if _several_devices:
        _on_current_device(stream, q, w, q_out, positions, cos_sin, q_scale, err)
    heads = _weights(w)
    T, st, sh = _query(q, heads)
    fp8 = q_scale is not None
    _word("q_scale", q_scale, torch.float32)
    _dense("q_out", q_out, torch.uint8 if fp8 else torch.bfloat16, (T, heads, ROW))
    _word("err", err, torch.int32)
    cs, npos, pos = _rotation(cos_sin, positions, T)
    status = _absorb_q(q.data_ptr(), st, sh, w.data_ptr(), T, heads, sm_scale, cs, npos, pos,
                               ROPES[rope], 1 if fp8 else 0, _ptr(q_scale), q_out.data_ptr(),
                               _ptr(err), _stream(stream, q))
    if status:
        _check("mla_absorb_q", status)


def mla_absorb_out(o, w, out, *, err=None, stream=None) -> None:
    """The layer's attention output bf16 [T, heads, 128] from the decode
    output o bf16 [T, heads, 512]."""
    if _several_devices:
        _on_current_device(stream, o, w, out, err)
    heads = _weights(w)
    T = o.shape[0]
    _dense("o", o, torch.bfloat16, (T, heads, LATENT))
    _dense("out", out, torch.bfloat16, (T, heads, V_HEAD))
    _word("err", err, torch.int32)
    status = _absorb_out(o.data_ptr(), w.data_ptr(), T, heads, out.data_ptr(), _ptr(err),
                         _stream(stream, o))
    if status:
        _check("mla_absorb_out", status)


def mla_selftest_absorb_wait(x, w, y, *, q_scale=None, limit_us: int = 2000, err=None,
                             stream=None) -> None:
    """mla_absorb_out (y [T, heads, 128]) or mla_absorb_q (y [T, heads, 576]) in
    which the waits for operands run out after limit_us: y's products become
    NaN, and mla_error_check of err raises MlaError with status 5."""
    if _several_devices:
        _on_current_device(stream, x, w, y, q_scale, err)
    heads = _weights(w)
    T, to_out = x.shape[0], y.shape[-1] == V_HEAD
    _word("q_scale", q_scale, torch.float32)
    _word("err", err, torch.int32)
    _dense("x", x, torch.bfloat16, (T, heads, LATENT if to_out else NOPE + ROPE))
    _dense("y", y, torch.bfloat16 if q_scale is None else torch.uint8,
           (T, heads, V_HEAD if to_out else ROW))
    _check("mla_selftest_absorb_wait", _lib.mla_selftest_absorb_wait(
        x.data_ptr(), w.data_ptr(), T, heads, _ptr(q_scale), y.data_ptr(), int(to_out),
        int(limit_us), _ptr(err), _stream(stream, x)))


class PrefillPlan:
    """Owns an mla_prefill* (host object)."""

    def __init__(self, handle, heads, kv_dtype, page_entries):
        self._h = handle
        self.heads, self.kv_dtype, self.page_entries = heads, kv_dtype, page_entries
        info = self.info()
        self.query_tokens, self.workspace_bytes = info.query_tokens, info.workspace_bytes

    @property
    def handle(self):
        return self._h

    def info(self) -> PrefillInfo:
        info = PrefillInfo()
        _check("mla_prefill_get_info", _lib.mla_prefill_get_info(self._h, ctypes.byref(info)))
        return info

    def __del__(self):
        if getattr(self, "_h", None):
            _lib.mla_prefill_destroy(self._h)
            self._h = None


def mla_prefill_plan(qo_indptr, kv_indptr, kv_last_page_len=None, *, page_size: int,
                     kv_dtype: str, heads: int = 16, num_sms: int = 0) -> PrefillPlan:
    """Plan an expanded-form call from HOST offsets: qo_indptr (query tokens)
    and kv_indptr (pages) with optional last-page lengths.  A request's query
    tokens are the last positions of its cached sequence."""
    qo, qo_p = _i32_array(qo_indptr)
    kvp, kvp_p = _i32_array(kv_indptr)
    last, last_p = _i32_array(kv_last_page_len)
    bs = len(qo) - 1
    _need(len(kvp) == bs + 1, f"kv_indptr must have {bs + 1} entries")
    _need(last is None or len(last) == bs, f"kv_last_page_len must have {bs} entries")
    h = ctypes.c_void_p()
    _check("mla_prefill_plan", _lib.mla_prefill_plan(qo_p, kvp_p, last_p, bs, int(page_size),
                                                     int(heads), DTYPES[kv_dtype], int(num_sms),
                                                     ctypes.byref(h)))
    return PrefillPlan(h, int(heads), kv_dtype, int(kvp[-1]))


def mla_prefill_run(plan: PrefillPlan, q, kv, w, out, *, workspace, sm_scale: float,
                    positions=None, cos_sin=None, rope: str = "interleaved", kv_scale=None,
                    kv_e8m0=None, kv_indices=None, lse=None, stream=None) -> None:
    """Enqueue one expanded-form attention call: q bf16 [T, heads, 192], kv the
    pool as mla_decode_run takes it, w bf16 [heads, 256, 512], out bf16
    [T, heads, 128], lse fp32 [T, heads] or None, workspace a uint8 CUDA tensor
    of at least plan.workspace_bytes."""
    if _several_devices:
        _on_current_device(stream, q, kv, w, out, workspace, positions, cos_sin, kv_scale, kv_e8m0,
                           kv_indices, lse)
    heads = _weights(w)
    _need(heads == plan.heads, f"w must have the plan's {plan.heads} heads")
    T, st, sh = _query(q, heads)
    _need(T == plan.query_tokens, f"q must have the plan's {plan.query_tokens} tokens")
    _dense("out", out, torch.bfloat16, (T, heads, V_HEAD))
    if lse is not None:
        _dense("lse", lse, torch.float32, (T, heads))
    if kv_indices is not None:
        _vec("kv_indices", kv_indices, torch.int32)
        _need(kv_indices.shape[0] >= plan.page_entries,
              f"kv_indices must hold the plan's {plan.page_entries} pages")
    _need(workspace.is_cuda and workspace.is_contiguous(), "workspace must be a contiguous CUDA tensor")
    scale, e8, e8_stride = _pool(kv, plan.kv_dtype, kv_scale, kv_e8m0)
    cs, npos, pos = _rotation(cos_sin, positions, T)
    status = _prefill_run(plan.handle, q.data_ptr(), st, sh, kv.data_ptr(), scale, e8,
                                  e8_stride, kv.shape[0], _ptr(kv_indices), w.data_ptr(), sm_scale,
                                  cs, npos, pos, ROPES[rope], workspace.data_ptr(),
                                  workspace.nbytes, out.data_ptr(), _ptr(lse), _stream(stream, q))
    if status:
        _check("mla_prefill_run", status)


def mla_prefill_check(plan: PrefillPlan, workspace, stream=None) -> None:
    """mla_decode_check for a prefill plan's workspace."""
    if _several_devices:
        _on_current_device(stream, workspace)
    _check("mla_prefill_check", _lib.mla_prefill_check(plan.handle, workspace.data_ptr(),
                                                       _stream(stream, workspace)))


class MlaPrefill:
    """Convenience owner of a prefill plan and its workspace."""

    def __init__(self, qo_indptr, kv_indptr, kv_last_page_len=None, *, page_size, kv_dtype,
                 heads=16, device="cuda"):
        self.plan = mla_prefill_plan(qo_indptr, kv_indptr, kv_last_page_len, page_size=page_size,
                                     kv_dtype=kv_dtype, heads=heads)
        self.workspace = torch.empty(max(self.plan.workspace_bytes, 256), dtype=torch.uint8,
                                     device=device)

    def __call__(self, q, kv, w, out, **kw):
        mla_prefill_run(self.plan, q, kv, w, out, workspace=self.workspace, **kw)
        return out


def mla_error_check(err, stream=None) -> None:
    """Synchronise, read and clear a device error word; raise MlaError if it
    was set: status 6 (pages or entries ran out), 1 (a length, page, slot or
    position out of range)."""
    if _several_devices:
        _on_current_device(stream, err)
    _word("err", err, torch.int32)
    _check("mla_error_check", _lib.mla_error_check(err.data_ptr(), _stream(stream, err)))
