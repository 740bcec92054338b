"""Host-side refusals of the packed attention and paged cache entries, and
their 64-bit reference forms (no GPU)."""
import ctypes as C
import math

import torch

from tests import packed_ref as ref

X = 1 << 20  # a non-null, aligned stand-in: never dereferenced on the host


def _fwd(P, **kw):
    a = dict(qkv=X, ld=768, dtype=1, cu=X, n_seq=2, n_rows=100, h=8, g=2, hd=64, o=X, lse=X, ws=X,
             wsb=1 << 30, flag=None)
    a.update(kw)
    return P.lib.llm_kernel_attention_packed_fwd(
        a["qkv"], a["ld"], a["dtype"], a["cu"], a["n_seq"], a["n_rows"], a["h"], a["g"], a["hd"],
        a["o"], a["lse"], a["ws"], a["wsb"], a["flag"], None)


def _bwd(P, **kw):
    a = dict(qkv=X, ld=768, dtype=1, cu=X, n_seq=2, n_rows=100, h=8, g=2, hd=64, o=X, lse=X,
             dout=X, dx=2 * X, dld=768, ws=X, wsb=1 << 30, flag=None)
    a.update(kw)
    return P.lib.llm_kernel_attention_packed_bwd(
        a["qkv"], a["ld"], a["dtype"], a["cu"], a["n_seq"], a["n_rows"], a["h"], a["g"], a["hd"],
        a["o"], a["lse"], a["dout"], a["dx"], a["dld"], a["ws"], a["wsb"], a["flag"], None)


def test_packed_refusals():
    import scratch_llama_decoder_b200 as P
    bad = [dict(qkv=None), dict(qkv=X + 1), dict(cu=None), dict(cu=X + 2), dict(o=None),
           dict(lse=None), dict(lse=X + 2), dict(ws=None), dict(ws=X + 8), dict(wsb=16),
           dict(ld=767), dict(dtype=2), dict(n_seq=-1), dict(n_seq=65537), dict(n_rows=-1),
           dict(n_rows=(1 << 20) + 1), dict(g=3), dict(g=0), dict(h=0), dict(hd=63), dict(hd=0),
           dict(hd=130, ld=4096), dict(flag=X + 1), dict(h=1025, g=1, ld=1 << 20)]
    for kw in bad:
        assert _fwd(P, **kw) == P.LLM_ERR_ARG, kw
        assert _bwd(P, **kw) == P.LLM_ERR_ARG, kw
    for kw in [dict(dout=None), dict(dout=X + 1), dict(dx=None), dict(dx=X), dict(dld=700)]:
        assert _bwd(P, **kw) == P.LLM_ERR_ARG, kw
    # nothing to do: no pointer is looked at
    assert _fwd(P, n_rows=0, qkv=None, o=None) == P.LLM_OK
    assert _bwd(P, n_seq=0, qkv=None, dx=None) == P.LLM_OK
    b = C.c_int64(0)
    ws = P.lib.llm_kernel_attention_packed_workspace
    assert ws(100, 2, 8, 0, None) == P.LLM_ERR_ARG
    assert ws(-1, 2, 8, 0, C.byref(b)) == P.LLM_ERR_ARG
    assert ws((1 << 20) + 1, 2, 8, 0, C.byref(b)) == P.LLM_ERR_ARG
    assert ws(100, 2, 0, 0, C.byref(b)) == P.LLM_ERR_ARG
    assert ws(1 << 20, 65536, 16, 1, C.byref(b)) == P.LLM_OK and b.value > 4 * 16 << 20
    assert ws(0, 0, 1, 1, C.byref(b)) == P.LLM_OK


def _kv(P, **kw):
    a = dict(d_pages=X, d_scales=X, d_table=X, table_ld=400, n_pages=10, table_pages=400, format=3,
             n_kv_head=2, head_dim=64, page_size=16, d_flag=None)
    a.update(kw)
    return P._lib.llm_kv(**a)


BAD_KV = [dict(d_pages=None), dict(d_scales=None), dict(d_scales=X + 2), dict(d_table=None),
          dict(d_table=X + 2), dict(table_ld=3), dict(n_pages=0), dict(table_pages=-1),
          dict(format=4), dict(format=-1), dict(n_kv_head=0), dict(n_kv_head=1025),
          dict(head_dim=0), dict(head_dim=3), dict(head_dim=130), dict(page_size=0),
          dict(page_size=65537), dict(d_flag=X + 1), dict(n_pages=1 << 60),
          dict(format=0, d_pages=X + 2), dict(format=1, d_pages=X + 1),
          dict(table_pages=1 << 20, table_ld=1 << 20, page_size=65536)]


def test_cache_refusals():
    import scratch_llama_decoder_b200 as P
    b = C.c_int64(0)

    def write(kv, qkv=X, ld=768, dtype=1, cu=X, st=None, n_seq=2, n_rows=9, h=8):
        return P.lib.llm_kernel_kv_write(C.byref(kv), qkv, ld, dtype, cu, st, n_seq, n_rows, h,
                                         None)

    def read(kv, cu=X, st=None, n_seq=2, n_rows=9, k=X, v=X, dtype=1):
        return P.lib.llm_kernel_kv_read(C.byref(kv), cu, st, n_seq, n_rows, k, v, dtype, None)

    def attend(kv, q=X, ld=512, dtype=1, lens=X, n_seq=2, h=8, o=X, lse=X, ws=X, wsb=1 << 40):
        return P.lib.llm_kernel_attention_paged(C.byref(kv), q, ld, dtype, lens, n_seq, h, o, lse,
                                                ws, wsb, None)

    for kw in BAD_KV:
        kv = _kv(P, **kw)
        assert write(kv) == read(kv) == attend(kv) == P.LLM_ERR_ARG, kw
        assert P.lib.llm_kernel_attention_paged_workspace(C.byref(kv), 2, 8, C.byref(b)) == \
            P.LLM_ERR_ARG, kw
    kv = _kv(P)
    for kw in [dict(qkv=None), dict(qkv=X + 1), dict(ld=767), dict(dtype=-1), dict(cu=None),
               dict(st=X + 2), dict(n_seq=-1), dict(n_rows=-1), dict(h=7), dict(h=0)]:
        assert write(kv, **kw) == P.LLM_ERR_ARG, kw
    for kw in [dict(cu=None), dict(st=X + 1), dict(n_seq=65537), dict(k=None), dict(v=X + 1),
               dict(dtype=9)]:
        assert read(kv, **kw) == P.LLM_ERR_ARG, kw
    for kw in [dict(q=None), dict(ld=511), dict(dtype=5), dict(lens=None), dict(lens=X + 3),
               dict(n_seq=-1), dict(n_seq=8193), dict(h=9), dict(o=None), dict(lse=X + 2),
               dict(ws=None), dict(ws=X + 4)]:
        assert attend(kv, **kw) == P.LLM_ERR_ARG, kw
    assert write(kv, n_rows=0, qkv=None) == read(kv, n_seq=0, k=None) == P.LLM_OK
    assert attend(kv, n_seq=0, q=None) == P.LLM_OK
    assert P.lib.llm_kernel_attention_paged_workspace(C.byref(kv), 2, 8, None) == P.LLM_ERR_ARG
    assert P.lib.llm_kernel_kv_write(None, X, 768, 1, X, None, 1, 1, 8, None) == P.LLM_ERR_ARG


def test_python_calls_refuse_cpu_tensors():
    import pytest

    import scratch_llama_decoder_b200 as P
    cu = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError):
        P.attention_packed(torch.zeros(4, 512), cu, 4, 2)
    pages, scales = P.kv_pages(2, 16, 2, 64, "e4m3", device="cpu")
    assert pages.dtype == torch.float8_e4m3fn and scales.shape == (2, 2, 2, 16)
    with pytest.raises(ValueError):
        P.kv_write(torch.zeros(4, 512), cu, 4, pages, torch.zeros(1, 1, dtype=torch.int32),
                   scales=scales)
    with pytest.raises(ValueError):
        P.attention_paged(torch.zeros(1, 512), pages, torch.zeros(1, 1, dtype=torch.int32),
                          cu[1:], scales=scales)


# ------------------------------------------------------- the reference forms
def test_reference_gradient_against_differences():
    gen = torch.Generator().manual_seed(0)
    h, g, hd, cu = 4, 2, 6, [0, 5, 5, 12, 13]
    x = torch.randn(13, (h + 2 * g) * hd, generator=gen, dtype=torch.float64)
    do = torch.randn(13, h * hd, generator=gen, dtype=torch.float64)
    out, lse, _, _ = ref.attention(x, cu, h, g)
    dx, _ = ref.backward(x, cu, h, g, out, lse, do, torch.float32)
    for _ in range(5):
        d = torch.randn(x.shape, generator=gen, dtype=torch.float64)
        t = 1e-5
        f = [float((ref.attention(x + s * t * d, cu, h, g)[0] * do).sum()) for s in (1, -1)]
        num, got = (f[0] - f[1]) / (2 * t), float((dx * d).sum())
        assert abs(num - got) <= 1e-7 * (1 + abs(num))


def test_reference_attention_is_causal_and_apart():
    gen = torch.Generator().manual_seed(1)
    h, g, hd, cu = 2, 1, 4, [0, 3, 7]
    x = torch.randn(7, (h + 2 * g) * hd, generator=gen, dtype=torch.float64)
    out, lse, _, _ = ref.attention(x, cu, h, g)
    y = x.clone()
    y[5] += 1.0
    o2, l2, _, _ = ref.attention(y, cu, h, g)
    assert torch.equal(out[:5], o2[:5]) and torch.equal(lse[:, :5], l2[:, :5])
    assert not torch.equal(out[5], o2[5])
    # the first row of a sequence is its own value
    v = x.view(7, 4, hd)[:, 3]
    assert torch.allclose(out.view(7, h, hd)[3, 0], v[3])
    assert math.isclose(float(lse[0, 0]), float((x.view(7, 4, hd)[0, 0] * x.view(7, 4, hd)[0, 2])
                                                .sum()) / 2, rel_tol=1e-12)


def test_reference_e4m3_matches_torch():
    """Every finite code is itself, and points between codes round as torch's
    conversion does."""
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn)
    val = codes.float()
    val = val[torch.isfinite(val)].unique()
    assert torch.equal(ref.e4m3(val.double()), val.double())
    mid = (val[1:] + val[:-1]) / 2
    x = torch.cat([mid, torch.nextafter(mid, val[1:]), torch.nextafter(mid, val[:-1]),
                   torch.linspace(-448, 448, 10001)])
    assert torch.equal(ref.e4m3(x.double()).float(), x.to(torch.float8_e4m3fn).float())


def test_reference_scales():
    x = torch.tensor([[448.0], [448.0 * (1 + 2 ** -23)], [447.0], [224.0], [225.0], [0.0],
                      [1e-45], [3e38]])
    _, unit = ref.stored(x, "e4m3")
    assert unit.tolist() == [1.0, 2.0, 1.0, 0.5, 1.0, 2.0 ** -126, 2.0 ** -126,
                             2.0 ** math.ceil(math.log2(float(x[7]) / 448))]
