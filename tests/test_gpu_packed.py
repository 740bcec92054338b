"""Packed causal attention on the GPU against 64-bit forms (packed_ref.py has
the error bounds): lengths, heads, types, strides, rows of no sequence, bad
offsets, streams and graphs."""
import itertools
import math

import pytest
import torch

from tests import packed_ref as ref

pytestmark = pytest.mark.gpu

LENS = [[1], [0, 1, 0, 2], [127, 128, 129], [64, 65, 63, 1, 192], [300, 5, 513], [1] * 130,
        [0, 0, 0]]
HEADS = [(4, 4), (8, 2), (3, 1)]
DTYPES = [torch.float32, torch.bfloat16]


def _cu(lens, first=0):
    return [first] + [first + x for x in itertools.accumulate(lens)]


def _data(lens, h, g, hd, dtype, seed=0, first=0, behind=0, big=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    cu = _cu(lens, first)
    n = cu[-1] + behind
    qkv = (torch.randn(n, (h + 2 * g) * hd, generator=gen, device="cuda") * big).to(dtype)
    dout = torch.randn(n, h * hd, generator=gen, device="cuda").to(dtype)
    return qkv, dout, cu, torch.tensor(cu, dtype=torch.int32, device="cuda")


def _check(qkv, dout, cu, cut, h, g, back=True):
    import scratch_llama_decoder_b200 as P
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = P.attention_packed(qkv, cut, h, g, flag=flag)
    a, b = cu[0], cu[-1]
    ro, rl, bo, bl = ref.attention(qkv, cu, h, g, qkv.dtype)
    ref.check(lse[:, a:b], rl[:, a:b], bl[:, a:b], "lse")
    ref.check(out[a:b], ro[a:b], bo[a:b], "out")
    if back:
        dx = P.attention_packed_backward(qkv, cut, h, g, out, lse, dout, flag=flag)
        rx, bx = ref.backward(qkv, cu, h, g, out, lse, dout, qkv.dtype)
        ref.check(dx[a:b], rx[a:b], bx[a:b], "dqkv")
        again = P.attention_packed_backward(qkv, cut, h, g, out, lse, dout)
        assert torch.equal(again[a:b].view(torch.int8), dx[a:b].view(torch.int8))
    again = P.attention_packed(qkv, cut, h, g)
    assert torch.equal(again[0][a:b], out[a:b]) and torch.equal(again[1][:, a:b], lse[:, a:b])
    assert int(flag) == 0
    return out, lse


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("hd", [32, 64, 128])
@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("lens", LENS, ids=lambda x: "-".join(map(str, x[:5])))
def test_forward_and_backward(lens, heads, hd, dtype):
    h, g = heads
    qkv, dout, cu, cut = _data(lens, h, g, hd, dtype)
    _check(qkv, dout, cu, cut, h, g)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("hd", [2, 4, 6, 16, 40, 48, 80, 96, 126])
def test_other_head_sizes(hd, dtype):
    qkv, dout, cu, cut = _data([70, 1, 130], 4, 2, hd, dtype, seed=hd)
    _check(qkv, dout, cu, cut, 4, 2)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("hd", [32, 64, 128])
def test_large_scores(hd, dtype):
    """Scores in the hundreds: the running maximum moves, weights under flow."""
    qkv, dout, cu, cut = _data([200, 333], 4, 2, hd, dtype, seed=3, big=4.0)
    _check(qkv, dout, cu, cut, 4, 2)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("hd", [32, 64, 128])
def test_scores_that_rise_along_the_row(hd, dtype):
    """Each key scores higher than the ones before it by far: the maximum of
    every block replaces the last one's."""
    qkv, dout, cu, cut = _data([600], 2, 1, hd, dtype, seed=4)
    x = qkv.view(600, 4, hd)
    x[:, :2, 0] = 8.0
    x[:, 2, 0] = (torch.arange(600, device="cuda") * 0.25 * math.sqrt(hd) / 8).to(dtype)
    _check(qkv, dout, cu, cut, 2, 1)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("hd", [64, 128, 48])
@pytest.mark.parametrize("pad,off", [(8, 0), (16, 8), (3, 0), (0, 1), (5, 3)])
def test_spaced_and_unaligned_rows(pad, off, hd, dtype):
    import scratch_llama_decoder_b200 as P
    h, g, lens = 4, 2, [130, 1, 67]
    w = (h + 2 * g) * hd
    base = torch.full((198 * (w + pad) + off + 8,), 7.0, device="cuda").to(dtype)
    qkv = base[off:off + 198 * (w + pad)].view(198, w + pad)[:, :w]
    dense, dout, cu, cut = _data(lens, h, g, hd, dtype, seed=5)
    qkv.copy_(dense)
    out, lse = _check(qkv, dout, cu, cut, h, g)
    store = torch.full_like(base, 7.0)
    dst = store[off:off + 198 * (w + pad)].view(198, w + pad)[:, :w]
    P.attention_packed_backward(qkv, cut, h, g, out, lse, dout, dqkv=dst)
    want = P.attention_packed_backward(dense, cut, h, g, out, lse, dout)
    # other strides may take other kernels: equal within both's bounds
    rx, bx = ref.backward(dense, cu, h, g, out, lse, dout, dtype)
    ref.check(dst, rx, bx, "spaced dqkv")
    ref.check(want, rx, bx, "dense dqkv")
    dst.fill_(7.0)
    assert bool((store == 7.0).all())  # nothing outside the rows was written


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("hd", [32, 64, 128, 20])
@pytest.mark.parametrize("poison", [math.nan, math.inf])
def test_rows_of_no_sequence(poison, hd, dtype):
    """Rows before the first and behind the last sequence hold anything and
    their outputs stay; so do the neighbours' non-finite values."""
    import scratch_llama_decoder_b200 as P
    h, g = 4, 2
    for lens in ([1], [100, 37], [127, 0, 130, 5], [256]):
        qkv, dout, cu, cut = _data(lens, h, g, hd, dtype, seed=6, first=9, behind=140)
        a, b = cu[0], cu[-1]
        n = qkv.shape[0]
        dirty, ddirty = qkv.clone(), dout.clone()
        for t in (dirty, ddirty):
            t[:a] = poison
            t[b:] = poison
        out = torch.full((n, h * hd), 3.0, device="cuda").to(dtype)
        lse = torch.full((h, n), 3.0, device="cuda")
        P.attention_packed(dirty, cut, h, g, out=out, lse=lse)
        assert bool((out[:a] == 3).all() and (out[b:] == 3).all())
        assert bool((lse[:, :a] == 3).all() and (lse[:, b:] == 3).all())
        ro, rl, bo, bl = ref.attention(qkv, cu, h, g, dtype)
        ref.check(out[a:b], ro[a:b], bo[a:b], "out")
        ref.check(lse[:, a:b], rl[:, a:b], bl[:, a:b], "lse")
        o2, l2 = out.clone(), lse.clone()
        o2[:a] = poison
        o2[b:] = poison
        l2[:, :a] = poison
        l2[:, b:] = poison
        dx = torch.full_like(qkv, 3.0)
        P.attention_packed_backward(dirty, cut, h, g, o2, l2, ddirty, dqkv=dx)
        assert bool((dx[:a] == 3).all() and (dx[b:] == 3).all())
        rx, bx = ref.backward(qkv, cu, h, g, out, lse, dout, dtype)
        ref.check(dx[a:b], rx[a:b], bx[a:b], "dqkv")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("hd", [32, 64, 128, 20])
def test_a_sequences_nan_stays_in_it(hd, dtype):
    import scratch_llama_decoder_b200 as P
    h, g, lens = 4, 2, [130, 200, 61]
    qkv, dout, cu, cut = _data(lens, h, g, hd, dtype, seed=7)
    ro, rl, bo, bl = ref.attention(qkv, cu, h, g, dtype)
    dirty = qkv.clone()
    dirty[cu[1]:cu[2]] = math.nan
    out, lse = P.attention_packed(dirty, cut, h, g)
    dx = P.attention_packed_backward(dirty, cut, h, g, out, lse, dout)
    assert bool(torch.isnan(out[cu[1]:cu[2]]).all())
    clean = P.attention_packed(qkv, cut, h, g)
    want = P.attention_packed_backward(qkv, cut, h, g, *clean, dout)
    for a, b in ((cu[0], cu[1]), (cu[2], cu[3])):
        ref.check(out[a:b], ro[a:b], bo[a:b], "out")
        ref.check(lse[:, a:b], rl[:, a:b], bl[:, a:b], "lse")
        assert torch.equal(dx[a:b], want[a:b])


@pytest.mark.parametrize("dtype", DTYPES)
def test_many_short_sequences(dtype):
    gen = torch.Generator().manual_seed(8)
    lens = torch.randint(0, 4, (5000,), generator=gen).tolist()
    h, g, hd = 2, 1, 64
    qkv, dout, cu, cut = _data(lens, h, g, hd, dtype, seed=8)
    import scratch_llama_decoder_b200 as P
    out, lse = P.attention_packed(qkv, cut, h, g)
    dx = P.attention_packed_backward(qkv, cut, h, g, out, lse, dout)
    # a reference by neighbours: at most 3 rows a sequence
    n = qkv.shape[0]
    q, k, v = ref.split(qkv, h, g)
    seq = torch.repeat_interleave(torch.arange(5000), torch.tensor(lens)).cuda()
    o = torch.zeros(n, h, hd, dtype=torch.float64, device="cuda")
    z = torch.full((n, h, 3), -math.inf, dtype=torch.float64, device="cuda")
    for back in range(3):
        ok = torch.zeros(n, dtype=torch.bool, device="cuda")
        ok[back:] = seq[back:] == seq[:n - back]
        kk = torch.roll(k, back, 0)
        s = (q * kk).sum(2) / math.sqrt(hd)
        z[:, :, back] = torch.where(ok[:, None], s, z[:, :, back])
    p = torch.softmax(z, 2)
    for back in range(3):
        o += p[:, :, back:back + 1] * torch.roll(v, back, 0)
    tol = 2.0 ** -6 if dtype == torch.bfloat16 else 1e-5  # several roundings of values below 4
    assert float((out.double().view(n, h, hd) - o).abs().max()) <= 4 * tol
    assert bool(torch.isfinite(dx).all())


def test_bad_offsets_are_clamped_and_flagged():
    """Offsets that decrease or leave the rows count as clamped and raised to
    the largest before them: outputs as for the mended offsets, nothing
    outside the rows written."""
    import scratch_llama_decoder_b200 as P
    h, g, hd, n = 4, 2, 64, 300
    for dtype in DTYPES:
        gen = torch.Generator(device="cuda").manual_seed(9)
        qkv = torch.randn(n, (h + 2 * g) * hd, generator=gen, device="cuda").to(dtype)
        dout = torch.randn(n, h * hd, generator=gen, device="cuda").to(dtype)
        for bad, good in (([0, 200, 100, 250], [0, 200, 200, 250]),
                          ([-5, 100, 1 << 30], [0, 100, 300]),
                          ([0, 2147483647, -2147483648, 10], [0, 300, 300, 300])):
            store = torch.full((3 * n, h * hd), 5.0, device="cuda").to(dtype)
            out = store[n:2 * n]
            lse = torch.full((h, n), 5.0, device="cuda")
            flag = torch.zeros(1, dtype=torch.int32, device="cuda")
            cut = torch.tensor(bad, dtype=torch.int32, device="cuda")
            P.attention_packed(qkv, cut, h, g, out=out, lse=lse, flag=flag)
            assert int(flag) == 1
            want = torch.full((n, h * hd), 5.0, device="cuda").to(dtype)
            wl = torch.full((h, n), 5.0, device="cuda")
            gut = torch.tensor(good, dtype=torch.int32, device="cuda")
            P.attention_packed(qkv, gut, h, g, out=want, lse=wl)
            assert torch.equal(out, want) and torch.equal(lse, wl)
            assert bool((store[:n] == 5).all() and (store[2 * n:] == 5).all())
            dx = torch.zeros_like(qkv)
            dw = torch.zeros_like(qkv)
            P.attention_packed_backward(qkv, cut, h, g, out, lse, dout, dqkv=dx)
            P.attention_packed_backward(qkv, gut, h, g, want, wl, dout, dqkv=dw)
            assert torch.equal(dx, dw)


def test_nothing_to_do():
    import scratch_llama_decoder_b200 as P
    z = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = P.attention_packed(torch.zeros(0, 8 * 64, device="cuda"), z, 4, 2)
    assert out.shape == (0, 256) and lse.shape == (4, 0)
    keep = torch.full((5, 256), 2.0, device="cuda")
    P.attention_packed(torch.zeros(5, 512, device="cuda"), z, 4, 2, out=keep)
    assert bool((keep == 2).all())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("hd", [64, 128])
def test_gradient_against_differences(hd, dtype):
    """d/dt sum(dout * out(qkv + t d)) by central differences of the 64-bit
    form, against the kernels' gradient along d."""
    import scratch_llama_decoder_b200 as P
    h, g, lens = 4, 2, [40, 1, 150]
    qkv, dout, cu, cut = _data(lens, h, g, hd, dtype, seed=10)
    out, lse = P.attention_packed(qkv, cut, h, g)
    dx = P.attention_packed_backward(qkv, cut, h, g, out, lse, dout).double()
    gen = torch.Generator(device="cuda").manual_seed(11)
    for part in range(3):  # q, k and v alone
        d = torch.zeros_like(dx).view(-1, h + 2 * g, hd)
        lo, hi = ((0, h), (h, h + g), (h + g, h + 2 * g))[part]
        d[:, lo:hi] = torch.randn(d[:, lo:hi].shape, generator=gen, device="cuda",
                                  dtype=torch.float64)
        d = d.view_as(dx)
        t = 1e-4

        def f(x):
            return float((ref.attention(x, cu, h, g)[0] * dout.double()).sum())

        num = (f(qkv.double() + t * d) - f(qkv.double() - t * d)) / (2 * t)
        got = float((dx * d).sum())
        # each element of dx is off by its bound at most; D comes from the
        # rounded out: r |dout . out| more in every dS
        rx, bx = ref.backward(qkv, cu, h, g, out, lse, dout, dtype)
        tol = float((bx * d.abs()).sum()) * 2 + 1e-5 * abs(num) + 1e-4
        assert abs(num - got) <= tol, (part, num, got, tol)


def test_streams_and_graphs():
    """A captured call serves other offsets and contents; calls on two streams
    at once, each on its own tensors."""
    import scratch_llama_decoder_b200 as P
    h, g, hd = 8, 2, 64
    n = 700
    sets = []
    for seed, lens in ((12, [300, 400]), (13, [1, 0, 698, 1]), (14, [700])):
        qkv, dout, cu, cut = _data(lens, h, g, hd, torch.bfloat16, seed=seed)
        cu4 = torch.full((5,), n, dtype=torch.int32, device="cuda")
        cu4[:len(cu)] = cut
        out, lse = P.attention_packed(qkv, cu4, h, g)
        sets.append((qkv, dout, cu4, out, lse,
                     P.attention_packed_backward(qkv, cu4, h, g, out, lse, dout)))
    x, d, c = (sets[0][i].clone() for i in range(3))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            o, l = P.attention_packed(x, c, h, g)
            dx = P.attention_packed_backward(x, c, h, g, o, l, d)
    torch.cuda.synchronize()
    for s in sets:
        x.copy_(s[0])
        d.copy_(s[1])
        c.copy_(s[2])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, s[3]) and torch.equal(l, s[4]) and torch.equal(dx, s[5])
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for st, s in zip(streams, sets):
            with torch.cuda.stream(st):
                o2, l2 = P.attention_packed(s[0], s[2], h, g)
                got.append((s, o2, l2, P.attention_packed_backward(s[0], s[2], h, g, o2, l2, s[1])))
    torch.cuda.synchronize()
    for s, o2, l2, d2 in got:
        assert torch.equal(o2, s[3]) and torch.equal(l2, s[4]) and torch.equal(d2, s[5])


def test_equal_lengths_agree_with_the_batch_kernels():
    """Sequences of one length: the same attention as the rectangular entry."""
    import ctypes as C

    import scratch_llama_decoder_b200 as P
    h, g, hd, b, t = 8, 2, 64, 3, 256
    qkv, dout, cu, cut = _data([t] * b, h, g, hd, torch.bfloat16, seed=15)
    out, lse = P.attention_packed(qkv, cut, h, g)
    o = torch.empty_like(out)
    l = torch.empty(b, h, t, device="cuda")
    s = C.c_void_p(torch.cuda.current_stream().cuda_stream)
    P.check(P.lib.llm_kernel_attention_fwd_bf16(qkv.data_ptr(), o.data_ptr(), l.data_ptr(), b, t,
                                                h, g, hd, 2, s), "fwd")
    ro, rl, bo, bl = ref.attention(qkv, cu, h, g, torch.bfloat16)
    ref.check(out, ro, bo, "out")
    ref.check(o, ro, bo, "rectangular out")
    ref.check(l.transpose(0, 1).reshape(h, b * t), rl, bl, "rectangular lse")


def test_refused_arguments():
    import scratch_llama_decoder_b200 as P
    qkv = torch.zeros(8, 8 * 64, device="cuda")
    cu = torch.tensor([0, 8], dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        P.attention_packed(qkv.half(), cu, 4, 2)
    with pytest.raises(ValueError):
        P.attention_packed(qkv, cu.long(), 4, 2)
    with pytest.raises(ValueError):
        P.attention_packed(qkv, cu.cpu(), 4, 2)
    with pytest.raises(ValueError):
        P.attention_packed(qkv, cu, 4, 3)
    with pytest.raises(ValueError):
        P.attention_packed(qkv.t(), cu, 4, 2)
    with pytest.raises(ValueError):
        P.attention_packed(qkv, cu, 4, 2, out=torch.zeros(8, 255, device="cuda"))
    with pytest.raises(ValueError):
        P.attention_packed(qkv[:1].expand(8, -1), cu, 4, 2)
    with pytest.raises(P.LLMError):  # head size 129 x 2
        P.attention_packed(torch.zeros(8, 3 * 258, device="cuda"), cu, 1, 1)
    out, lse = P.attention_packed(qkv, cu, 4, 2)
    with pytest.raises(ValueError):
        P.attention_packed_backward(qkv, cu, 4, 2, out, lse[:3], out)
    with pytest.raises(P.LLMError):
        P.attention_packed_backward(qkv, cu, 4, 2, out, lse, out, dqkv=qkv)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("hd", [32, 64, 128])
def test_many_sequences_against_the_formulas(hd, dtype):
    """More sequences than one pass of the plan's search takes, both passes."""
    gen = torch.Generator().manual_seed(16)
    lens = torch.randint(0, 30, (400,), generator=gen).tolist() + [700, 0, 131]
    qkv, dout, cu, cut = _data(lens, 2, 1, hd, dtype, seed=16)
    _check(qkv, dout, cu, cut, 2, 1)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("hd", [64, 128, 20])
@pytest.mark.parametrize("n_seq", [12, 256, 600])
def test_bad_offsets_of_many_rows(n_seq, hd, dtype):
    """Bad offsets where the work is planned ahead (few and many sequences):
    as for the mended offsets, and nothing outside the rows written."""
    import scratch_llama_decoder_b200 as P
    h, g, n = 8, 2, 6000
    gen = torch.Generator().manual_seed(17)
    qkv, dout, _, _ = _data([n], h, g, hd, dtype, seed=17)
    good = torch.sort(torch.randint(0, n + 1, (n_seq + 1,), generator=gen))[0].tolist()
    bad = list(good)
    bad[3], good[3] = -7, good[2]
    good[-2:] = [n, n]
    bad[-2:] = [(1 << 31) - 1, -(1 << 31)]
    at = n_seq // 2
    bad[at] = 0
    good[at] = good[at - 1]
    wide = (h + 2 * g) * hd
    res = []
    for cu in (bad, good):
        store = torch.full((n + 512, wide), 5.0, device="cuda").to(dtype)
        out = torch.full((n + 512, h * hd), 5.0, device="cuda").to(dtype)
        lse = torch.full((h, n), 5.0, device="cuda")
        cut = torch.tensor(cu, dtype=torch.int32, device="cuda")
        flags = torch.zeros(2, dtype=torch.int32, device="cuda")
        P.attention_packed(qkv, cut, h, g, out=out[256:-256], lse=lse, flag=flags[:1])
        P.attention_packed_backward(qkv, cut, h, g, out[256:-256], lse, dout,
                                    dqkv=store[256:-256], flag=flags[1:])
        assert flags.tolist() == [int(cu is bad)] * 2
        for x in (out, store):
            assert bool((x[:256] == 5).all() and (x[-256:] == 5).all())
        res.append((out, lse, store))
    assert all(torch.equal(a, b) for a, b in zip(*res))


@pytest.mark.parametrize("dtype", DTYPES)
def test_most_rows_and_sequences(dtype):
    """The limits, in rows so far apart that offsets pass 2^31 elements: the
    same bits as in calls of 1024 sequences each on rows next to another."""
    import scratch_llama_decoder_b200 as P
    h, g, hd, n, part = 1, 1, 32, 1 << 20, 1 << 14
    gen = torch.Generator(device="cuda").manual_seed(18)
    wide = torch.empty(n, 2112, dtype=dtype, device="cuda")
    qkv, dqkv = wide[:, 1000:1096], wide[:, 1200:1296]
    qkv.copy_(torch.randn(n, 96, generator=gen, device="cuda"))
    dout = torch.randn(n, hd, generator=gen, device="cuda").to(dtype)
    cut = torch.arange(0, n + 1, 16, dtype=torch.int32, device="cuda")
    out, lse = P.attention_packed(qkv, cut, h, g)
    P.attention_packed_backward(qkv, cut, h, g, out, lse, dout, dqkv=dqkv)
    for a in range(0, n, part):
        x = qkv[a:a + part].contiguous()
        o, l = P.attention_packed(x, cut[:part // 16 + 1], h, g)
        assert torch.equal(o, out[a:a + part]) and torch.equal(l, lse[:, a:a + part])
        d = P.attention_packed_backward(x, cut[:part // 16 + 1], h, g, o, l, dout[a:a + part])
        assert torch.equal(d, dqkv[a:a + part])


def test_longest_sequence():
    """One sequence of 2^20 rows: rows of the output and of dq, and the last
    keys' gradients, against the formulas."""
    import scratch_llama_decoder_b200 as P
    hd, n = 32, 1 << 20
    qkv, dout, cu, cut = _data([n], 1, 1, hd, torch.bfloat16, seed=19)
    out, lse = P.attention_packed(qkv, cut, 1, 1)
    dx = P.attention_packed_backward(qkv, cut, 1, 1, out, lse, dout)
    q, k, v = (t[:, 0] for t in ref.split(qkv, 1, 1))
    r, u, c = 2.0 ** -8, ref.U, 1 / math.sqrt(hd)
    for i in (0, 127, 128, 77777, n - 2, n - 1):
        s = k[:i + 1] @ q[i] * c
        L = torch.logsumexp(s, 0)
        p = torch.exp(s - L)
        o, m = p @ v[:i + 1], p @ v[:i + 1].abs()
        # as packed_ref.attention: scores to (hd + 5) u |q||k|, weights 2^-12 and
        # rounded; m terms of a sum to u each
        es = float(((hd + 5) * u * (k[:i + 1].abs() @ q[i].abs()) * c).max()) + 2.0 ** -12
        rel = 2 * es + (2 * i + 18) * u + r
        ref.check(lse[0, i], L, es + (i + 9) * u + 4 * u * L.abs(), "lse")
        ref.check(out[i], o, rel * m + r * o.abs() + 1e-30, "out")
        do = dout[i].double()
        dP = v[:i + 1] @ do
        ds = p * (dP - p @ dP)
        bD = do.abs() @ (rel * m + r * o.abs())
        eds = (p * (bD + 2 * es * (dP - p @ dP).abs() + (hd + 2) * u * (v[:i + 1].abs() @ do.abs()))
               + (r + (i + 9) * u) * ds.abs())
        dq = ds @ k[:i + 1] * c
        ref.check(dx[i, :hd], dq, eds @ k[:i + 1].abs() * c + r * dq.abs() + 1e-30, "dq")
    # the last key meets the last query alone
    p = torch.exp(q[-1] @ k[-1] * c - L)
    dv = p * dout[-1].double()
    ref.check(dx[-1, 2 * hd:], dv, (2 * es + 2 * r + (i + 20) * u) * dv.abs() + 1e-30, "dv")


def test_gradient_at_the_longest_weights_underflow():
    """Scores so far apart that all weights but one underflow: the gradient of
    q and k is zero but for roundings, v's is dout's rows."""
    import scratch_llama_decoder_b200 as P
    for dtype in DTYPES:
        for hd in (32, 64, 128):
            n = 200
            qkv = torch.zeros(n, 3 * hd, dtype=dtype, device="cuda")
            qkv[:, 0] = 64.0
            qkv[:, hd] = torch.arange(n, device="cuda").to(dtype)  # the row's own key wins
            qkv[:, 2 * hd:] = torch.randn(n, hd, device="cuda").to(dtype)
            dout = torch.randn(n, hd, device="cuda").to(dtype)
            cut = torch.tensor([0, n], dtype=torch.int32, device="cuda")
            out, lse = P.attention_packed(qkv, cut, 1, 1)
            dx = P.attention_packed_backward(qkv, cut, 1, 1, out, lse, dout)
            ro, rl, bo, bl = ref.attention(qkv, [0, n], 1, 1, dtype)
            ref.check(out, ro, bo, "out")
            rx, bx = ref.backward(qkv, [0, n], 1, 1, out, lse, dout, dtype)
            ref.check(dx, rx, bx, "dqkv")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("hd", [32, 64, 128])
def test_many_long_sequences(hd, dtype):
    """Hundreds of sequences of several tiles: the same bits as in calls of a
    few sequences each; and shorter ones, against the formulas."""
    import scratch_llama_decoder_b200 as P
    h, g, count = 2, 2, 300
    gen = torch.Generator().manual_seed(20)
    lens = torch.randint(300, 700, (count,), generator=gen).tolist()
    qkv, dout, cu, cut = _data(lens, h, g, hd, dtype, seed=20)
    out, lse = P.attention_packed(qkv, cut, h, g)
    dx = P.attention_packed_backward(qkv, cut, h, g, out, lse, dout)
    for s in (0, 100, 296):
        a, b = cu[s], cu[s + 4]
        part = cut[s:s + 5] - a
        o, l = P.attention_packed(qkv[a:b].contiguous(), part, h, g)
        d = P.attention_packed_backward(qkv[a:b].contiguous(), part, h, g, o, l, dout[a:b])
        assert torch.equal(o, out[a:b]) and torch.equal(l, lse[:, a:b])
        assert torch.equal(d, dx[a:b])
    lens = torch.randint(1, 300, (40,), generator=gen).tolist()
    for h, g in ((8, 8), (4, 2)):
        qkv, dout, cu, cut = _data(lens, h, g, hd, dtype, seed=21)
        _check(qkv, dout, cu, cut, h, g)
