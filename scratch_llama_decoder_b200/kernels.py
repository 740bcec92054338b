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

import torch

from . import _lib as L

_DTYPES = {torch.float32: L.LLM_FP32, torch.bfloat16: L.LLM_BF16}
_FORMATS = {torch.float32: L.LLM_KV_F32, torch.bfloat16: L.LLM_KV_BF16,
            torch.float8_e4m3fn: L.LLM_KV_E4M3, torch.int8: L.LLM_KV_INT8}
_NAMES = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn,
          "int8": torch.int8}


def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _same(dev, **tensors):
    for name, t in tensors.items():
        if t is not None:
            _need(isinstance(t, torch.Tensor) and t.device == dev,
                  f"{name} must be a tensor on {dev}")


def _rows(name, t, width=None):
    """A 2-D float32/bfloat16 tensor whose rows may be spaced (stride(1) == 1)."""
    _need(isinstance(t, torch.Tensor) and t.is_cuda and t.dim() == 2 and t.dtype in _DTYPES,
          f"{name} must be a 2-D float32 or bfloat16 tensor on a CUDA device")
    _need(t.stride(1) == 1 or t.shape[1] == 1, f"{name}: the elements of a row must be adjacent")
    _need(width is None or t.shape[1] == width, f"{name} must have {width} columns")
    ld = t.stride(0) if t.shape[0] > 1 else max(t.stride(0), t.shape[1])
    _need(ld >= t.shape[1], f"{name}: its rows overlap")
    return ld


def _full(name, t, shape, dtype):
    _need(tuple(t.shape) == tuple(shape) and t.dtype == dtype and t.is_contiguous(),
          f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)}")


def _ints(name, t, n):
    _need(t.dtype == torch.int32 and t.dim() == 1 and t.shape[0] == n and t.is_contiguous(),
          f"{name} must be a contiguous int32 tensor of {n} elements")


def _flag(t):
    if t is not None:
        _need(t.dtype == torch.int32 and t.numel() == 1, "flag must be one int32 element")
        return t.data_ptr()
    return None


def _offsets(t):
    _need(isinstance(t, torch.Tensor) and t.dim() == 1 and t.shape[0] >= 1,
          "cu_seqlens must be a 1-D tensor of one offset more than sequences")
    _ints("cu_seqlens", t, t.shape[0])
    return t.shape[0] - 1


class _On:
    """The tensors' device made current for a call; its current stream."""

    def __init__(self, dev):
        self.dev = dev
        self.guard = None
        if dev.index != torch.cuda.current_device():
            self.guard = torch.cuda.device(dev)

    def __enter__(self):
        if self.guard:
            self.guard.__enter__()
        return torch.cuda.current_stream(self.dev).cuda_stream

    def __exit__(self, *exc):
        if self.guard:
            self.guard.__exit__(*exc)


def _head_dim(width, n_head, n_kv_head):
    _need(n_head >= 1 and n_kv_head >= 1 and n_head % n_kv_head == 0,
          "n_kv_head must divide n_head")
    hd, rest = divmod(width, n_head + 2 * n_kv_head)
    _need(rest == 0, "qkv must have (n_head + 2 n_kv_head) * head_dim columns")
    return hd


def _workspace(n_rows, n_seq, n_head, backward, dev):
    b = C.c_int64(0)
    L.check(L.lib.llm_kernel_attention_packed_workspace(n_rows, n_seq, n_head, backward,
                                                        C.byref(b)),
            "llm_kernel_attention_packed_workspace")
    return torch.empty(b.value, dtype=torch.uint8, device=dev)


def attention_packed(qkv, cu_seqlens, n_head, n_kv_head, out=None, lse=None, flag=None):
    """Causal attention of packed sequences (llm_kernel_attention_packed_fwd).

    qkv: [rows, (n_head + 2 n_kv_head) * head_dim] float32 or bfloat16, q heads,
    then k heads, then v heads of each row, RoPE applied; its rows may be spaced.
    cu_seqlens: int32 [n_seq + 1]; sequence s is rows cu_seqlens[s] to
    cu_seqlens[s + 1] - 1.  Returns (out [rows, n_head * head_dim] in qkv's
    type, lse float32 [n_head, rows]); rows of no sequence keep what out and
    lse held (nothing useful unless they are given)."""
    ld = _rows("qkv", qkv)
    hd = _head_dim(qkv.shape[1], n_head, n_kv_head)
    n_rows, dev = qkv.shape[0], qkv.device
    n_seq = _offsets(cu_seqlens)
    _same(dev, cu_seqlens=cu_seqlens, out=out, lse=lse, flag=flag)
    if out is None:
        out = torch.empty(n_rows, n_head * hd, dtype=qkv.dtype, device=dev)
    else:
        _full("out", out, (n_rows, n_head * hd), qkv.dtype)
    if lse is None:
        lse = torch.empty(n_head, n_rows, dtype=torch.float32, device=dev)
    else:
        _full("lse", lse, (n_head, n_rows), torch.float32)
    with _On(dev) as stream:
        ws = _workspace(n_rows, n_seq, n_head, 0, dev)
        L.check(L.lib.llm_kernel_attention_packed_fwd(
            qkv.data_ptr(), ld, _DTYPES[qkv.dtype], cu_seqlens.data_ptr(), n_seq, n_rows, n_head,
            n_kv_head, hd, out.data_ptr(), lse.data_ptr(), ws.data_ptr(), ws.numel(),
            _flag(flag), stream), "llm_kernel_attention_packed_fwd")
    return out, lse


def attention_packed_backward(qkv, cu_seqlens, n_head, n_kv_head, out, lse, dout, dqkv=None,
                              flag=None):
    """Gradient of attention_packed (llm_kernel_attention_packed_bwd): from its
    inputs, its out and lse, and the gradient dout of out, the gradient of qkv
    (rows of no sequence keep what dqkv held: nothing useful unless it is given)."""
    ld = _rows("qkv", qkv)
    hd = _head_dim(qkv.shape[1], n_head, n_kv_head)
    n_rows, dev = qkv.shape[0], qkv.device
    n_seq = _offsets(cu_seqlens)
    _same(dev, cu_seqlens=cu_seqlens, out=out, lse=lse, dout=dout, dqkv=dqkv, flag=flag)
    _full("out", out, (n_rows, n_head * hd), qkv.dtype)
    _full("dout", dout, (n_rows, n_head * hd), qkv.dtype)
    _full("lse", lse, (n_head, n_rows), torch.float32)
    if dqkv is None:
        dqkv = torch.empty(n_rows, qkv.shape[1], dtype=qkv.dtype, device=dev)
    _need(dqkv.dtype == qkv.dtype and dqkv.shape[0] == n_rows, "dqkv must be like qkv")
    dld = _rows("dqkv", dqkv, qkv.shape[1])
    with _On(dev) as stream:
        ws = _workspace(n_rows, n_seq, n_head, 1, dev)
        L.check(L.lib.llm_kernel_attention_packed_bwd(
            qkv.data_ptr(), ld, _DTYPES[qkv.dtype], cu_seqlens.data_ptr(), n_seq, n_rows, n_head,
            n_kv_head, hd, out.data_ptr(), lse.data_ptr(), dout.data_ptr(), dqkv.data_ptr(), dld,
            ws.data_ptr(), ws.numel(), _flag(flag), stream), "llm_kernel_attention_packed_bwd")
    return dqkv


def kv_pages(n_pages, page_size, n_kv_head, head_dim, format="bf16", device="cuda"):
    """An empty paged cache: (pages [n_pages, 2, n_kv_head, page_size, head_dim],
    scales [n_pages, 2, n_kv_head, page_size] or None); format "f32", "bf16",
    "e4m3" or "int8"."""
    _need(format in _NAMES, f"format must be one of {sorted(_NAMES)}")
    shape = (n_pages, 2, n_kv_head, page_size, head_dim)
    pages = torch.zeros(shape, dtype=torch.uint8, device=device) if format in ("e4m3", "int8") \
        else torch.zeros(shape, dtype=_NAMES[format], device=device)
    if format in ("e4m3", "int8"):
        return pages.view(_NAMES[format]), torch.zeros(shape[:4], device=device)
    return pages, None


def _kv(pages, scales, table, flag):
    _need(isinstance(pages, torch.Tensor) and pages.is_cuda and pages.dim() == 5 and
          pages.shape[1] == 2 and pages.dtype in _FORMATS and pages.is_contiguous(),
          "pages must be a contiguous [n_pages, 2, n_kv_head, page_size, head_dim] tensor on a "
          "CUDA device, of float32, bfloat16, float8_e4m3fn or int8")
    fmt = _FORMATS[pages.dtype]
    _same(pages.device, table=table, scales=scales, flag=flag)
    if fmt >= L.LLM_KV_E4M3:
        _need(scales is not None, "an 8-bit cache needs its scales")
        _full("scales", scales, pages.shape[:4], torch.float32)
    _need(isinstance(table, torch.Tensor) and table.dim() == 2 and table.dtype == torch.int32 and
          (table.stride(1) == 1 or table.shape[1] <= 1), "table must be a 2-D int32 tensor of rows")
    n, _, g, ps, hd = pages.shape
    return L.llm_kv(pages.data_ptr(), scales.data_ptr() if fmt >= L.LLM_KV_E4M3 else None,
                    table.data_ptr(), max(table.stride(0), table.shape[1]), n, table.shape[1],
                    fmt, g, hd, ps, _flag(flag))


def kv_write(qkv, cu_seqlens, n_head, pages, table, scales=None, starts=None, flag=None):
    """The k and v of packed rows into the cache (llm_kernel_kv_write): row i of
    sequence s becomes position starts[s] + i - cu_seqlens[s].

    qkv, cu_seqlens: as in attention_packed; pages, scales: of kv_pages; table:
    int32 [n_seq, pages a sequence]; starts: int32 [n_seq] (None: all 0)."""
    ld = _rows("qkv", qkv)
    kv = _kv(pages, scales, table, flag)
    _need(qkv.shape[1] == (n_head + 2 * kv.n_kv_head) * kv.head_dim,
          "qkv must have (n_head + 2 n_kv_head) * head_dim columns")
    n_seq = _offsets(cu_seqlens)
    _need(table.shape[0] >= n_seq, "table must have a row for every sequence")
    _same(pages.device, qkv=qkv, cu_seqlens=cu_seqlens, starts=starts)
    if starts is not None:
        _ints("starts", starts, n_seq)
    with _On(pages.device) as stream:
        L.check(L.lib.llm_kernel_kv_write(
            C.byref(kv), qkv.data_ptr(), ld, _DTYPES[qkv.dtype], cu_seqlens.data_ptr(),
            starts.data_ptr() if starts is not None else None, n_seq, qkv.shape[0], n_head,
            stream), "llm_kernel_kv_write")


def kv_read(pages, table, cu_seqlens, n_rows, dtype, scales=None, starts=None, k=None, v=None,
            flag=None):
    """The inverse of kv_write (llm_kernel_kv_read): (k, v), each [n_rows,
    n_kv_head, head_dim] of dtype (float32 or bfloat16); rows of no sequence
    keep what k and v held (nothing useful unless they are given)."""
    _need(dtype in _DTYPES, "dtype must be torch.float32 or torch.bfloat16")
    kv = _kv(pages, scales, table, flag)
    n_seq = _offsets(cu_seqlens)
    _need(table.shape[0] >= n_seq, "table must have a row for every sequence")
    dev, shape = pages.device, (n_rows, kv.n_kv_head, kv.head_dim)
    _same(dev, cu_seqlens=cu_seqlens, starts=starts, k=k, v=v)
    if starts is not None:
        _ints("starts", starts, n_seq)
    if k is None:
        k = torch.empty(shape, dtype=dtype, device=dev)
    else:
        _full("k", k, shape, dtype)
    if v is None:
        v = torch.empty(shape, dtype=dtype, device=dev)
    else:
        _full("v", v, shape, dtype)
    with _On(dev) as stream:
        L.check(L.lib.llm_kernel_kv_read(
            C.byref(kv), cu_seqlens.data_ptr(),
            starts.data_ptr() if starts is not None else None, n_seq, n_rows, k.data_ptr(),
            v.data_ptr(), _DTYPES[dtype], stream), "llm_kernel_kv_read")
    return k, v


def attention_paged(q, pages, table, lens, scales=None, out=None, lse=None, flag=None):
    """Attention of one new token per sequence over its first lens[s] cached
    positions (llm_kernel_attention_paged).

    q: [n_seq, n_head * head_dim] float32 or bfloat16 (its rows may be spaced:
    the q columns of a q|k|v tensor will do); pages, scales, table: as in
    kv_write; lens: int32 [n_seq].  Returns (out [n_seq, n_head * head_dim] in
    q's type, lse float32 [n_seq, n_head]); a sequence of length 0 gets out 0
    and lse -inf."""
    kv = _kv(pages, scales, table, flag)
    ld = _rows("q", q)
    n_seq, dev = q.shape[0], pages.device
    n_head, rest = divmod(q.shape[1], kv.head_dim) if kv.head_dim else (0, 1)
    _need(rest == 0 and n_head % max(kv.n_kv_head, 1) == 0,
          "q must have n_head * head_dim columns, n_head a multiple of n_kv_head")
    _need(table.shape[0] >= n_seq, "table must have a row for every sequence")
    _same(dev, q=q, lens=lens, out=out, lse=lse)
    _ints("lens", lens, n_seq)
    if out is None:
        out = torch.empty(n_seq, q.shape[1], dtype=q.dtype, device=dev)
    else:
        _full("out", out, q.shape, q.dtype)
    if lse is None:
        lse = torch.empty(n_seq, n_head, dtype=torch.float32, device=dev)
    else:
        _full("lse", lse, (n_seq, n_head), torch.float32)
    with _On(dev) as stream:
        b = C.c_int64(0)
        L.check(L.lib.llm_kernel_attention_paged_workspace(C.byref(kv), n_seq, n_head,
                                                           C.byref(b)),
                "llm_kernel_attention_paged_workspace")
        ws = torch.empty(b.value, dtype=torch.uint8, device=dev)
        L.check(L.lib.llm_kernel_attention_paged(
            C.byref(kv), q.data_ptr(), ld, _DTYPES[q.dtype], lens.data_ptr(), n_seq, n_head,
            out.data_ptr(), lse.data_ptr(), ws.data_ptr(), b.value, stream),
            "llm_kernel_attention_paged")
    return out, lse
