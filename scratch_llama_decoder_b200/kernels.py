"""Kernels on sequences of different lengths, on torch tensors.

Packed causal attention (forward and backward), the paged key/value cache and
the attention of single tokens over it: the calls of include/llm_kernels.h
with their arguments taken from tensors.  Every call checks its tensors
(device, type, shape), allocates what it returns and its workspace, and
enqueues on the current stream of the tensors' device; nothing synchronises.
Inputs must be ready on that stream, as for any torch operation.

`flag`, where a call takes it, is an int32 tensor of one element on the same
device: error bits (LLM_PACKED_BAD_CU, LLM_KV_BAD_PAGE, LLM_PACKED_TIMEOUT)
are OR-ed into it on the device and never cleared.
"""
import ctypes as C
import functools
import struct

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
# a Stream object for it (2 us of a call whose kernel takes 5).
_stream = torch._C._cuda_getCurrentRawStream
_packed_fwd = L.lib.llm_kernel_attention_packed_fwd
_packed_bwd = L.lib.llm_kernel_attention_packed_bwd
_write, _read = L.lib.llm_kernel_kv_write, L.lib.llm_kernel_kv_read
_paged = L.lib.llm_kernel_attention_paged


def _bad(what):
    raise ValueError(what)


def _on(dev, fn, *args):
    """fn(*args, stream) with the tensors' device current."""
    i = dev.index
    if i == torch.cuda.current_device():
        rc = fn(*args, _stream(i))
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, _stream(i))
    if rc:
        L.check(rc, fn.__name__)


def _rows(name, t):
    """dtype code and row stride of a 2-D float32/bfloat16 tensor of rows, which
    may be spaced (stride(1) == 1)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dim() != 2 or t.dtype not in _DTYPES:
        _bad(f"{name} must be a 2-D float32 or bfloat16 tensor on a CUDA device")
    n, w = t.shape
    ld, step = t.stride()
    if step != 1 and w != 1:
        _bad(f"{name}: the elements of a row must be adjacent")
    if ld < w:
        if n > 1:
            _bad(f"{name}: its rows overlap")
        ld = w
    return _DTYPES[t.dtype], ld


def _at(name, t, dev, shape, dtype):
    """Address of a contiguous tensor of this device, shape and type."""
    if not isinstance(t, torch.Tensor) or t.device != dev or t.dtype != dtype or \
            t.shape != shape or not t.is_contiguous():
        _bad(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {dev}")
    return t.data_ptr()


def _flag(t, dev):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.device != dev or t.dtype != _i32 or t.numel() != 1:
        _bad(f"flag must be one int32 element on {dev}")
    return t.data_ptr()


def _offsets(t, dev):
    """Address of cu_seqlens and the number of sequences."""
    if not isinstance(t, torch.Tensor) or t.device != dev or t.dtype != _i32 or t.dim() != 1 or \
            t.shape[0] < 1 or not t.is_contiguous():
        _bad(f"cu_seqlens must be a contiguous 1-D int32 tensor on {dev}, one offset more than "
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
    dt, ld = _rows("qkv", qkv)
    n_rows, width = qkv.shape
    hd, dev = _head_dim(width, n_head, n_kv_head), qkv.device
    cu, n_seq = _offsets(cu_seqlens, dev)
    nb = _packed_bytes(n_rows, n_seq, n_head, 0)
    if out is None:
        out = torch.empty((n_rows, n_head * hd), dtype=qkv.dtype, device=dev)
        o = out.data_ptr()
    else:
        o = _at("out", out, dev, (n_rows, n_head * hd), qkv.dtype)
    if lse is None:
        lse = torch.empty((n_head, n_rows), dtype=_f32, device=dev)
        ls = lse.data_ptr()
    else:
        ls = _at("lse", lse, dev, (n_head, n_rows), _f32)
    ws = torch.empty(nb, dtype=torch.uint8, device=dev)
    _on(dev, _packed_fwd, qkv.data_ptr(), ld, dt, cu, n_seq, n_rows, n_head, n_kv_head, hd, o, ls,
        ws.data_ptr(), nb, _flag(flag, dev))
    return out, lse


def attention_packed_backward(qkv, cu_seqlens, n_head, n_kv_head, out, lse, dout, dqkv=None,
                              flag=None):
    """Gradient of attention_packed (llm_kernel_attention_packed_bwd): from its
    inputs, its out and lse, and the gradient dout of out, the gradient of qkv
    (rows of no sequence keep what dqkv held: nothing useful unless it is
    given; its rows may be spaced)."""
    dt, ld = _rows("qkv", qkv)
    n_rows, width = qkv.shape
    hd, dev = _head_dim(width, n_head, n_kv_head), qkv.device
    cu, n_seq = _offsets(cu_seqlens, dev)
    nb = _packed_bytes(n_rows, n_seq, n_head, 1)
    o = _at("out", out, dev, (n_rows, n_head * hd), qkv.dtype)
    ls = _at("lse", lse, dev, (n_head, n_rows), _f32)
    do = _at("dout", dout, dev, (n_rows, n_head * hd), qkv.dtype)
    if dqkv is None:
        dqkv = torch.empty((n_rows, width), dtype=qkv.dtype, device=dev)
        dld = width
    else:
        ddt, dld = _rows("dqkv", dqkv)
        if ddt != dt or dqkv.device != dev or dqkv.shape != qkv.shape:
            _bad(f"dqkv must be of qkv's type and shape, on {dev}")
    ws = torch.empty(nb, dtype=torch.uint8, device=dev)
    _on(dev, _packed_bwd, qkv.data_ptr(), ld, dt, cu, n_seq, n_rows, n_head, n_kv_head, hd, o, ls,
        do, dqkv.data_ptr(), dld, ws.data_ptr(), nb, _flag(flag, dev))
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
    """The cache's packed llm_kv, its device, kv heads and head size."""
    if not isinstance(pages, torch.Tensor) or not pages.is_cuda or pages.dim() != 5 or \
            pages.shape[1] != 2 or pages.dtype not in _FORMATS or not pages.is_contiguous():
        _bad("pages must be a contiguous [n_pages, 2, n_kv_head, page_size, head_dim] tensor on a "
             "CUDA device, of float32, bfloat16, float8_e4m3fn or int8")
    fmt, dev, shape = _FORMATS[pages.dtype], pages.device, pages.shape
    sc = 0
    if fmt >= L.LLM_KV_E4M3:
        if scales is None:
            _bad("an 8-bit cache needs its scales")
        sc = _at("scales", scales, dev, shape[:4], _f32)
    if not isinstance(table, torch.Tensor) or table.device != dev or table.dtype != _i32 or \
            table.dim() != 2:
        _bad(f"table must be a 2-D int32 tensor on {dev}")
    cols = table.shape[1]
    ld, step = table.stride()
    if step != 1 and cols > 1:
        _bad("table: the entries of a row must be adjacent")
    if ld < cols:
        if table.shape[0] > 1:
            _bad("table: its rows overlap")
        ld = cols
    n, _, g, ps, hd = shape
    return _KV.pack(pages.data_ptr(), sc, table.data_ptr(), ld, n, cols, fmt, g, hd, ps,
                    _flag(flag, dev) or 0), dev, g, hd


def kv_write(qkv, cu_seqlens, n_head, pages, table, scales=None, starts=None, flag=None):
    """The k and v of packed rows into the cache (llm_kernel_kv_write): row i of
    sequence s becomes position starts[s] + i - cu_seqlens[s].

    qkv, cu_seqlens: as in attention_packed; pages, scales: of kv_pages; table:
    int32 [n_seq, pages a sequence]; starts: int32 [n_seq] (None: all 0)."""
    dt, ld = _rows("qkv", qkv)
    kv, dev, g, hd = _kv(pages, scales, table, flag)
    n_rows, width = qkv.shape
    if qkv.device != dev or width != (n_head + 2 * g) * hd:
        _bad(f"qkv must have (n_head + 2 n_kv_head) * head_dim columns, on {dev}")
    cu, n_seq = _offsets(cu_seqlens, dev)
    if table.shape[0] < n_seq:
        _bad("table must have a row for every sequence")
    st = None if starts is None else _at("starts", starts, dev, (n_seq,), _i32)
    _on(dev, _write, kv, qkv.data_ptr(), ld, dt, cu, st, n_seq, n_rows, n_head)


def kv_read(pages, table, cu_seqlens, n_rows, dtype, scales=None, starts=None, k=None, v=None,
            flag=None):
    """The inverse of kv_write (llm_kernel_kv_read): (k, v), each [n_rows,
    n_kv_head, head_dim] of dtype (float32 or bfloat16); rows of no sequence
    keep what k and v held (nothing useful unless they are given)."""
    if dtype not in _DTYPES:
        _bad("dtype must be torch.float32 or torch.bfloat16")
    kv, dev, g, hd = _kv(pages, scales, table, flag)
    cu, n_seq = _offsets(cu_seqlens, dev)
    if table.shape[0] < n_seq:
        _bad("table must have a row for every sequence")
    shape = (n_rows, g, hd)
    st = None if starts is None else _at("starts", starts, dev, (n_seq,), _i32)
    if k is None:
        k = torch.empty(shape, dtype=dtype, device=dev)
    if v is None:
        v = torch.empty(shape, dtype=dtype, device=dev)
    _on(dev, _read, kv, cu, st, n_seq, n_rows, _at("k", k, dev, shape, dtype),
        _at("v", v, dev, shape, dtype), _DTYPES[dtype])
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
    kv, dev, g, hd = _kv(pages, scales, table, flag)
    dt, ld = _rows("q", q)
    n_seq, width = q.shape
    n_head = width // hd if hd else 0
    if q.device != dev or not hd or width % hd or not g or n_head % g:
        _bad(f"q must have n_head * head_dim columns, n_head a multiple of n_kv_head, on {dev}")
    if table.shape[0] < n_seq:
        _bad("table must have a row for every sequence")
    ln = _at("lens", lens, dev, (n_seq,), _i32)
    nb = _paged_bytes(g, hd, pages.shape[3], table.shape[1], n_seq, n_head)
    if out is None:
        out = torch.empty((n_seq, width), dtype=q.dtype, device=dev)
        o = out.data_ptr()
    else:
        o = _at("out", out, dev, (n_seq, width), q.dtype)
    if lse is None:
        lse = torch.empty((n_seq, n_head), dtype=_f32, device=dev)
        ls = lse.data_ptr()
    else:
        ls = _at("lse", lse, dev, (n_seq, n_head), _f32)
    # a call that splits nothing needs no workspace
    ws = torch.empty(nb, dtype=torch.uint8, device=dev) if nb else None
    _on(dev, _paged, kv, q.data_ptr(), ld, dt, ln, n_seq, n_head, o, ls,
        ws.data_ptr() if nb else None, nb)
    return out, lse
