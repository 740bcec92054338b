"""Packed attention and the paged cache on the GPU at what their calls allow
beside ordinary inputs: non-finite keys before the queries, bad offsets,
gradients that nothing records."""
import itertools
import math

import pytest
import torch

from tests import packed_ref as ref

pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.bfloat16]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("hd", [32, 64, 128])
@pytest.mark.parametrize("rows", [200, 400])
@pytest.mark.parametrize("what", ["nan", "inf", "-inf"])
def test_one_key_that_is_not_finite(what, rows, hd, dtype):
    """One element of one key, at every offset of 32 keys, in the first or a
    later block of 128: a NaN or an infinite score reaches every later row of
    the heads that read the key, whichever way its exponential is taken; a
    score of -inf is a weight of 0, and earlier rows and other heads keep
    their values."""
    import scratch_llama_decoder_b200 as P
    h, g, n = 4, 2, 32
    gen = torch.Generator(device="cuda").manual_seed(31)
    x = torch.randn(n, rows, h + 2 * g, hd, generator=gen, device="cuda").to(dtype)
    x[:, :, :h, 0] = -1.0 if what == "-inf" else 1.0
    at = [32 * (s % 4) + s for s in range(n)]
    for s, p in enumerate(at):
        x[s, p, h + 1, 0] = math.nan if what == "nan" else math.inf
    qkv = x.reshape(n * rows, -1)
    cu = torch.arange(0, n * rows + 1, rows, dtype=torch.int32, device="cuda")
    out, lse = P.attention_packed(qkv, cu, h, g)
    out = out.view(n, rows, h, hd)
    lse = lse.view(h, n, rows)
    r, ex, u, c = ref.R[dtype], ref.EXP[dtype], ref.U, 1 / math.sqrt(hd)
    for s, p in enumerate(at):
        for i in range(h):
            q, k, v = (x[s, :, j].double() for j in (i, h + i // 2, h + g + i // 2))
            k = k.nan_to_num(nan=0.0, posinf=0.0)
            hit = i // 2 == 1
            if hit and what != "-inf":
                assert not bool(torch.isfinite(out[s, p:, i]).any()), (s, i)
                assert not bool(torch.isfinite(lse[i, s, p:]).any()), (s, i)
            sc = q @ k.t() * c
            z = sc.masked_fill(torch.ones_like(sc).triu(1) > 0, -math.inf)
            if hit:
                z[:, p] = -math.inf  # the row p of "-inf" has its other keys
            live = torch.isfinite(z).any(1)
            if hit and what != "-inf":
                live[p:] = False
            z, sc, q, o, l = (t[live] for t in (z, sc, q, out[s, :, i], lse[i, s]))
            L = torch.logsumexp(z, 1)
            w = torch.exp(z - L[:, None])
            # as packed_ref.attention
            es = ((hd + 3) * u * (q.abs() @ k.abs().t()) * c + 2 * u * sc.abs()).tril().amax(1)
            rel = 2 * (es + ex) + (2 * rows + 16) * u + r
            O = w @ v
            ref.check(o, O, rel[:, None] * (w @ v.abs()) + r * O.abs() + 1e-30, (s, i, "out"))
            ref.check(l, L, es + ex + (rows + 8) * u + 4 * u * L.abs() + 1e-30, (s, i, "lse"))


def _bad_offsets(n, n_seq, seed):
    """Offsets that decrease or leave [0, n] in several places, and the same
    clamped and raised to the largest before them."""
    gen = torch.Generator().manual_seed(seed)
    bad = torch.sort(torch.randint(0, n + 1, (n_seq + 1,), generator=gen))[0].tolist()
    bad[0], bad[n_seq // 2], bad[n_seq // 2 - 1] = -3, -(1 << 31), n // 2 + 1
    if n_seq > 6:
        bad[5], bad[-1] = 1, (1 << 31) - 1
    good, top = [], 0
    for c in bad:
        top = max(top, min(max(c, 0), n))
        good.append(top)
    return bad, good


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("hd,g", [(64, 2), (128, 5), (6, 1)])
@pytest.mark.parametrize("n,n_seq", [(100, 3), (33, 40), (5000, 300), (20000, 5000), (300, 65536),
                                     (700, 1025)])
@pytest.mark.parametrize("fmt", ["f32", "bf16", "e4m3", "int8"])
def test_cache_offsets_count_as_mended(fmt, n, n_seq, hd, g, dtype):
    """kv_write and kv_read take bad offsets as attention_packed does, and say
    so in the flag."""
    import scratch_llama_decoder_b200 as P
    h, ps = g, 8
    gen = torch.Generator(device="cuda").manual_seed(32)
    qkv = torch.randn(n, (h + 2 * g) * hd, generator=gen, device="cuda").to(dtype)
    for bad, good in (_bad_offsets(n, n_seq, 33), ([0, 60, 20, 100], [0, 60, 60, 100])):
        if good[-1] > n:
            continue
        lens = [b - a for a, b in zip(good[:-1], good[1:])]
        starts = [i % 11 for i in range(len(lens))]
        need = [-(-(a + x) // ps) if x else 0 for a, x in zip(starts, lens)]
        cols = max(need)
        table = torch.full((len(lens), cols), -1, dtype=torch.int32)
        at = 0
        for s, x in enumerate(need):
            table[s, :x] = torch.arange(at, at + x)
            at += x
        table = table.cuda()
        st = torch.tensor(starts, dtype=torch.int32, device="cuda")
        got = []
        for cu in (bad, good):
            pages, scales = P.kv_pages(at, ps, g, hd, fmt)
            flag = torch.zeros(3, dtype=torch.int32, device="cuda")
            cut = torch.tensor(cu, dtype=torch.int32, device="cuda")
            k, v = (torch.full((n, g, hd), 9.0, device="cuda").to(dtype) for _ in range(2))
            P.kv_write(qkv, cut, h, pages, table, scales=scales, starts=st, flag=flag[:1])
            P.kv_read(pages, table, cut, n, dtype, scales=scales, starts=st, k=k, v=v,
                      flag=flag[1:2])
            P.kv_write(qkv, cut, h, pages, table, scales=scales, starts=st, flag=flag[2:])
            assert flag.tolist() == [int(cu is bad)] * 3
            got.append((pages, scales, k, v))
        for a, b in zip(*got):
            assert a is None or torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        # in a sequence: the stored values, rounded to dtype; elsewhere as it was
        k, lo, hi = got[1][2], good[0], good[-1]
        want, _ = ref.stored(qkv.view(n, h + 2 * g, hd)[:, h:h + g], fmt)
        tol = max(ref.R[dtype], ref.U) * want.abs()
        assert bool(((k.double() - want).abs() <= tol)[lo:hi].all())
        assert bool((k[:lo] == 9).all() and (k[hi:] == 9).all())


@pytest.mark.parametrize("fmt", ["bf16", "int8"])
def test_cache_of_the_most_sequences(fmt):
    """65536 sequences of 16 rows each: written and read whole."""
    import scratch_llama_decoder_b200 as P
    n, n_seq, g, hd, ps = 1 << 20, 65536, 1, 32, 16
    gen = torch.Generator(device="cuda").manual_seed(34)
    qkv = torch.randn(n, 3 * hd, generator=gen, device="cuda").bfloat16()
    cut = torch.arange(0, n + 1, 16, dtype=torch.int32, device="cuda")
    pages, scales = P.kv_pages(n_seq, ps, g, hd, fmt)
    table = torch.randperm(n_seq, generator=gen, device="cuda").to(torch.int32)[:, None]
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    P.kv_write(qkv, cut, 1, pages, table, scales=scales, flag=flag)
    k, v = P.kv_read(pages, table, cut, n, torch.bfloat16, scales=scales, flag=flag)
    assert int(flag) == 0
    for got, x in ((k, qkv[:, hd:2 * hd]), (v, qkv[:, 2 * hd:])):
        if fmt == "bf16":
            assert torch.equal(got[:, 0], x)
        else:
            want, _ = ref.stored(x, fmt)
            # the code's value, rounded to bfloat16
            assert bool(((got[:, 0].double() - want).abs() <= 2.0 ** -8 * want.abs()).all())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("hd", [32, 64, 128, 20])
@pytest.mark.parametrize("n,n_seq,cu,bad", [
    (1, 40, [0] + [1] * 40, {36: -9}),
    (20, 40, list(range(21)) + [20] * 20, {35: 3}),
    (20, 200, list(range(21)) + [20] * 180, {199: 21}),
    (20, 40, list(range(21)) + [20] * 20, {40: 7}),
    (6000, 40, list(range(0, 6001, 600)) + [6000] * 30, {35: 5999}),
])
def test_bad_offsets_behind_the_last_row_are_flagged(n, n_seq, cu, bad, hd, dtype):
    """Offsets that no row needs, past those of every tile: reported, and
    the outputs as without them."""
    import scratch_llama_decoder_b200 as P
    gen = torch.Generator(device="cuda").manual_seed(35)
    qkv = torch.randn(n, 3 * hd, generator=gen, device="cuda").to(dtype)
    dout = torch.randn(n, hd, generator=gen, device="cuda").to(dtype)
    res = []
    for broken in (False, True):
        c = list(cu)
        for i, x in (bad if broken else {}).items():
            c[i] = x
        flags = torch.zeros(2, dtype=torch.int32, device="cuda")
        cut = torch.tensor(c, dtype=torch.int32, device="cuda")
        out, lse = P.attention_packed(qkv, cut, 1, 1, flag=flags[:1])
        dx = P.attention_packed_backward(qkv, cut, 1, 1, out, lse, dout, flag=flags[1:])
        assert flags.tolist() == [int(broken)] * 2
        res.append((out, lse, dx))
    assert all(torch.equal(a, b) for a, b in zip(*res))


def test_gradients_that_nothing_records_are_told():
    """Inputs that require a gradient: a warning, the same outputs, none of
    them with a gradient; no warning where none is asked for."""
    import warnings

    import scratch_llama_decoder_b200 as P
    h, g, hd = 2, 1, 32
    qkv = torch.randn(9, (h + 2 * g) * hd, device="cuda")
    cu = torch.tensor([0, 4, 9], dtype=torch.int32, device="cuda")
    pages, _ = P.kv_pages(2, 8, g, hd, "f32")
    table = torch.tensor([[0], [1]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([4, 5], dtype=torch.int32, device="cuda")
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        want = P.attention_packed(qkv, cu, h, g)
        P.kv_write(qkv, cu, h, pages, table)
        paged = P.attention_paged(qkv[[3, 8], :h * hd], pages, table, lens)
        leaf = qkv.clone().requires_grad_()
        with torch.no_grad():
            P.attention_packed(leaf, cu, h, g)
        P.attention_packed_backward(leaf, cu, h, g, *want, torch.ones_like(want[0]))
    with pytest.warns(UserWarning, match="attention_packed records nothing"):
        got = P.attention_packed(leaf, cu, h, g)
    with pytest.warns(UserWarning, match="attention_paged records nothing"):
        one = P.attention_paged(leaf[[3, 8], :h * hd], pages, table, lens)
    for a, b in zip((*want, *paged), (*got, *one)):
        assert torch.equal(a, b) and not b.requires_grad
