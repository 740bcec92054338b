"""Kernels on sequences of different lengths, on torch tensors.

Packed causal attention (forward and backward), the paged key/value cache and
the attention of single tokens over it: the calls of include/llm_kernels.h
with their arguments taken from tensors.  Every call checks its tensors
(device, type, shape), allocates what it returns and its workspace, and
enqueues on the current stream of the tensors' device; nothing synchronises.
Inputs must be ready on that stream, as for any torch operation.

Nothing is recorded for autograd: outputs carry no gradient whatever the inputs
require (attention_packed and attention_paged warn where an input asks for one);
the gradient of attention_packed is attention_packed_backward's.

`flag`, where a call takes it, is an int32 tensor of one element on the same
device: error bits (LLM_PACKED_BAD_CU, LLM_KV_BAD_PAGE, LLM_PACKED_TIMEOUT)
are OR-ed into it on the device and never cleared.
"""
import ctypes as C
import functools
import struct
import warnings

import torch

from . import _lib as L

_DTYPES = {torch.float32: L.LLM_FP32, torch.bfloat16: L.LLM_BF16}
_FORMATS = {torch.float32: L.LLM_KV_F32, torch.bfloat16: L.LLM_KV_BF16,
            torch.float8_e4m3fn: L.LLM_KV_E4M3, torch.int8: L.LLM_KV_INT8}
_NAMES = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn,
          "int8": torch.int8}
_i32, _f32 = torch.int32, torch.float32
# llm_kv as the C compiler lays it out; a call takes the packed bytes
_KV = struct.Struct("@PPPqqiiiiiP")
assert _KV.size == C.sizeof(L.llm_kv)
# The current stream's handle as an integer: torch.cuda.current_stream() builds
# a Stream object for it (2 us of a call whose kernel takes 5).  A torch built
# without CUDA has none, and no tensors that a call gets as far as this with.
_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current = torch.cuda.current_device
_empty = torch.empty
_packed_fwd = L.lib.llm_kernel_attention_packed_fwd
_packed_bwd = L.lib.llm_kernel_attention_packed_bwd
_write, _read = L.lib.llm_kernel_kv_write, L.lib.llm_kernel_kv_read
_paged = L.lib.llm_kernel_attention_paged


def _bad(what):
    raise ValueError(what)


def _unrecorded(name, t, what):
    if t.requires_grad and torch.is_grad_enabled():
        warnings.warn(f"{name} records nothing for autograd: its outputs carry no gradient of "
                      f"{what}; pass {what}.detach(), or call it under torch.no_grad()", stacklevel=3)


def _on(i, fn, *args):
    """fn(*args, stream) with the tensors' device (index i) current."""
    if i == _current():
        rc = fn(*args, _stream(i))
    else:
        with torch.cuda.device(i):
            rc = fn(*args, _stream(i))
    if rc:
        L.check(rc, fn.__name__)


def _rows(name, t):
    """dtype code, device index and row stride of a 2-D float32/bfloat16 tensor
    of rows, which may be spaced (stride(1) == 1)."""
    dt = _DTYPES.get(t.dtype) if isinstance(t, torch.Tensor) and t.dim() == 2 else None
    i = t.get_device() if dt is not None else -1
    if i < 0:
        _bad(f"{name} must be a 2-D float32 or bfloat16 tensor on a CUDA device")
    ld, step = t.stride()
    w = t.shape[1]
    if step != 1 and w != 1:
        _bad(f"{name}: the elements of a row must be adjacent")
    if ld < w:
        if t.shape[0] > 1:
            _bad(f"{name}: its rows overlap")
        ld = w
    return dt, i, ld


def _at(name, t, i, shape, dtype):
    """Address of a contiguous tensor of this device, shape and type."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.get_device() != i or \
            t.shape != shape or not t.is_contiguous():
        _bad(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on cuda:{i}")
    return t.data_ptr()


def _flag(t, i):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.get_device() != i or t.dtype is not _i32 or \
            t.numel() != 1:
        _bad(f"flag must be one int32 element on cuda:{i}")
    return t.data_ptr()


def _offsets(t, i):
    """Address of cu_seqlens and the number of sequences."""
    if not isinstance(t, torch.Tensor) or t.dtype is not _i32 or t.get_device() != i or \
            t.dim() != 1 or not t.is_contiguous() or t.shape[0] < 1:
        _bad(f"cu_seqlens must be a contiguous 1-D int32 tensor on cuda:{i}, one offset more than "
             "there are sequences")
    return t.data_ptr(), t.shape[0] - 1


def _head_dim(width, n_head, n_kv_head):
    if n_head < 1 or n_kv_head < 1 or n_head % n_kv_head:
        _bad("n_kv_head must divide n_head")
    hd, rest = divmod(width, n_head + 2 * n_kv_head)
    if rest:
        _bad("qkv must have (n_head + 2 n_kv_head) * head_dim columns")
    return hd


@functools.lru_cache(maxsize=256)
def _packed_bytes(n_rows, n_seq, n_head, backward):
    b = C.c_int64(0)
    L.check(L.lib.llm_kernel_attention_packed_workspace(n_rows, n_seq, n_head, backward,
                                                        C.byref(b)),
            "llm_kernel_attention_packed_workspace")
    return b.value


def attention_packed(qkv, cu_seqlens, n_head, n_kv_head, out=None, lse=None, flag=None):
    """Causal attention of packed sequences (llm_kernel_attention_packed_fwd).

    qkv: [rows, (n_head + 2 n_kv_head) * head_dim] float32 or bfloat16, q heads,
    then k heads, then v heads of each row, RoPE applied; its rows may be spaced.
    cu_seqlens: int32 [n_seq + 1]; sequence s is rows cu_seqlens[s] to
    cu_seqlens[s + 1] - 1.  Returns (out [rows, n_head * head_dim] in qkv's
    type, lse float32 [n_head, rows]); rows of no sequence keep what out and
    lse held (nothing useful unless they are given)."""
    dt, i, ld = _rows("qkv", qkv)
    _unrecorded("attention_packed", qkv, "qkv")
    n_rows, width = qkv.shape
    hd, dev = _head_dim(width, n_head, n_kv_head), qkv.device
    cu, n_seq = _offsets(cu_seqlens, i)
    nb = _packed_bytes(n_rows, n_seq, n_head, 0)
    if out is None:
        out = _empty((n_rows, n_head * hd), dtype=qkv.dtype, device=dev)
        o = out.data_ptr()
    else:
        o = _at("out", out, i, (n_rows, n_head * hd), qkv.dtype)
    if lse is None:
        lse = _empty((n_head, n_rows), dtype=_f32, device=dev)
        ls = lse.data_ptr()
    else:
        ls = _at("lse", lse, i, (n_head, n_rows), _f32)
    ws = _empty(nb, dtype=torch.uint8, device=dev)
    _on(i, _packed_fwd, qkv.data_ptr(), ld, dt, cu, n_seq, n_rows, n_head, n_kv_head, hd, o, ls,
        ws.data_ptr(), nb, _flag(flag, i))
    return out, lse


def attention_packed_backward(qkv, cu_seqlens, n_head, n_kv_head, out, lse, dout, dqkv=None,
                              flag=None):
    """Gradient of attention_packed (llm_kernel_attention_packed_bwd): from its
    inputs, its out and lse, and the gradient dout of out, the gradient of qkv
    (rows of no sequence keep what dqkv held: nothing useful unless it is
    given; its rows may be spaced)."""
    dt, i, ld = _rows("qkv", qkv)
    n_rows, width = qkv.shape
    hd, dev = _head_dim(width, n_head, n_kv_head), qkv.device
    cu, n_seq = _offsets(cu_seqlens, i)
    nb = _packed_bytes(n_rows, n_seq, n_head, 1)
    o = _at("out", out, i, (n_rows, n_head * hd), qkv.dtype)
    ls = _at("lse", lse, i, (n_head, n_rows), _f32)
    do = _at("dout", dout, i, (n_rows, n_head * hd), qkv.dtype)
    if dqkv is None:
        dqkv = _empty((n_rows, width), dtype=qkv.dtype, device=dev)
        dld = width
    else:
        ddt, di, dld = _rows("dqkv", dqkv)
        if ddt != dt or di != i or dqkv.shape != qkv.shape:
            _bad(f"dqkv must be of qkv's type and shape, on cuda:{i}")
    ws = _empty(nb, dtype=torch.uint8, device=dev)
    _on(i, _packed_bwd, qkv.data_ptr(), ld, dt, cu, n_seq, n_rows, n_head, n_kv_head, hd, o, ls,
        do, dqkv.data_ptr(), dld, ws.data_ptr(), nb, _flag(flag, i))
    return dqkv


def kv_pages(n_pages, page_size, n_kv_head, head_dim, format="bf16", device="cuda"):
    """An empty paged cache: (pages [n_pages, 2, n_kv_head, page_size, head_dim],
    scales [n_pages, 2, n_kv_head, page_size] or None); format "f32", "bf16",
    "e4m3" or "int8"."""
    if format not in _NAMES:
        _bad(f"format must be one of {sorted(_NAMES)}")
    shape = (n_pages, 2, n_kv_head, page_size, head_dim)
    if format in ("e4m3", "int8"):
        pages = torch.zeros(shape, dtype=torch.int8, device=device).view(_NAMES[format])
        return pages, torch.zeros(shape[:4], device=device)
    return torch.zeros(shape, dtype=_NAMES[format], device=device), None


def _kv(pages, scales, table, flag):
    """The cache's packed llm_kv, its device index and shape."""
    fmt = _FORMATS.get(pages.dtype) if isinstance(pages, torch.Tensor) and pages.dim() == 5 else None
    i = pages.get_device() if fmt is not None else -1
    shape = pages.shape if i >= 0 else (0, 0)
    if shape[1] != 2 or not pages.is_contiguous():
        _bad("pages must be a contiguous [n_pages, 2, n_kv_head, page_size, head_dim] tensor on a "
             "CUDA device, of float32, bfloat16, float8_e4m3fn or int8")
    n, _, g, ps, hd = shape
    sc = 0
    if fmt >= L.LLM_KV_E4M3:
        if scales is None:
            _bad("an 8-bit cache needs its scales")
        sc = _at("scales", scales, i, (n, 2, g, ps), _f32)
    if not isinstance(table, torch.Tensor) or table.dtype is not _i32 or \
            table.get_device() != i or table.dim() != 2:
        _bad(f"table must be a 2-D int32 tensor on cuda:{i}")
    ld, step = table.stride()
    cols = table.shape[1]
    if step != 1 and cols > 1:
        _bad("table: the entries of a row must be adjacent")
    if ld < cols:
        if table.shape[0] > 1:
            _bad("table: its rows overlap")
        ld = cols
    return _KV.pack(pages.data_ptr(), sc, table.data_ptr(), ld, n, cols, fmt, g, hd, ps,
                    0 if flag is None else _flag(flag, i)), i, g, hd, ps, cols


def kv_write(qkv, cu_seqlens, n_head, pages, table, scales=None, starts=None, flag=None):
    """The k and v of packed rows into the cache (llm_kernel_kv_write): row i of
    sequence s becomes position starts[s] + i - cu_seqlens[s].

    qkv, cu_seqlens: as in attention_packed; pages, scales: of kv_pages; table:
    int32 [n_seq, pages a sequence]; starts: int32 [n_seq] (None: all 0)."""
    dt, qi, ld = _rows("qkv", qkv)
    kv, i, g, hd, _, _ = _kv(pages, scales, table, flag)
    n_rows, width = qkv.shape
    if qi != i or width != (n_head + 2 * g) * hd:
        _bad(f"qkv must have (n_head + 2 n_kv_head) * head_dim columns, on cuda:{i}")
    cu, n_seq = _offsets(cu_seqlens, i)
    if table.shape[0] < n_seq:
        _bad("table must have a row for every sequence")
    st = None if starts is None else _at("starts", starts, i, (n_seq,), _i32)
    _on(i, _write, kv, qkv.data_ptr(), ld, dt, cu, st, n_seq, n_rows, n_head)


def kv_read(pages, table, cu_seqlens, n_rows, dtype, scales=None, starts=None, k=None, v=None,
            flag=None):
    """The inverse of kv_write (llm_kernel_kv_read): (k, v), each [n_rows,
    n_kv_head, head_dim] of dtype (float32 or bfloat16); rows of no sequence
    keep what k and v held (nothing useful unless they are given)."""
    dt = _DTYPES.get(dtype)
    if dt is None:
        _bad("dtype must be torch.float32 or torch.bfloat16")
    kv, i, g, hd, _, _ = _kv(pages, scales, table, flag)
    cu, n_seq = _offsets(cu_seqlens, i)
    if table.shape[0] < n_seq:
        _bad("table must have a row for every sequence")
    shape, dev = (n_rows, g, hd), pages.device
    st = None if starts is None else _at("starts", starts, i, (n_seq,), _i32)
    if k is None:
        k = _empty(shape, dtype=dtype, device=dev)
        kp = k.data_ptr()
    else:
        kp = _at("k", k, i, shape, dtype)
    if v is None:
        v = _empty(shape, dtype=dtype, device=dev)
        vp = v.data_ptr()
    else:
        vp = _at("v", v, i, shape, dtype)
    _on(i, _read, kv, cu, st, n_seq, n_rows, kp, vp, dt)
    return k, v


@functools.lru_cache(maxsize=256)
def _paged_bytes(n_kv_head, head_dim, page_size, table_pages, n_seq, n_head):
    # what the size depends on; the addresses only have to be plausible
    kv = L.llm_kv(16, 16, 16, table_pages, 1, table_pages, L.LLM_KV_F32, n_kv_head, head_dim,
                  page_size, None)
    b = C.c_int64(0)
    L.check(L.lib.llm_kernel_attention_paged_workspace(C.byref(kv), n_seq, n_head, C.byref(b)),
            "llm_kernel_attention_paged_workspace")
    return b.value


def attention_paged(q, pages, table, lens, scales=None, out=None, lse=None, flag=None):
    """Attention of one new token per sequence over its first lens[s] cached
    positions (llm_kernel_attention_paged).

    q: [n_seq, n_head * head_dim] float32 or bfloat16 (its rows may be spaced:
    the q columns of a q|k|v tensor will do); pages, scales, table: as in
    kv_write; lens: int32 [n_seq].  Returns (out [n_seq, n_head * head_dim] in
    q's type, lse float32 [n_seq, n_head]); a sequence of length 0 gets out 0
    and lse -inf."""
    kv, i, g, hd, ps, cols = _kv(pages, scales, table, flag)
    dt, qi, ld = _rows("q", q)
    _unrecorded("attention_paged", q, "q")
    n_seq, width = q.shape
    n_head = width // hd if hd else 0
    if qi != i or not hd or width % hd or not g or n_head % g:
        _bad(f"q must have n_head * head_dim columns, n_head a multiple of n_kv_head, on cuda:{i}")
    if table.shape[0] < n_seq:
        _bad("table must have a row for every sequence")
    ln = _at("lens", lens, i, (n_seq,), _i32)
    nb = _paged_bytes(g, hd, ps, cols, n_seq, n_head)
    dev = q.device
    if out is None:
        out = _empty((n_seq, width), dtype=q.dtype, device=dev)
        o = out.data_ptr()
    else:
        o = _at("out", out, i, (n_seq, width), q.dtype)
    if lse is None:
        lse = _empty((n_seq, n_head), dtype=_f32, device=dev)
        ls = lse.data_ptr()
    else:
        ls = _at("lse", lse, i, (n_seq, n_head), _f32)
    # a call that splits nothing needs no workspace
    ws = _empty(nb, dtype=torch.uint8, device=dev) if nb else None
    _on(i, _paged, kv, q.data_ptr(), ld, dt, ln, n_seq, n_head, o, ls,
        ws.data_ptr() if nb else None, nb)
    return out, lse
