"""The paged key/value cache and the attention over it on the GPU, against
64-bit forms (packed_ref.py)."""
import math

import pytest
import torch

from tests import packed_ref as ref

pytestmark = pytest.mark.gpu

FORMATS = ["f32", "bf16", "e4m3", "int8"]
DTYPES = [torch.float32, torch.bfloat16]


def _tables(need, n_pages, seed, spare=1):
    """Random distinct pages for sequences of need[i] pages; unused entries -1."""
    order = torch.randperm(n_pages, generator=torch.Generator().manual_seed(seed)).tolist()
    t = torch.full((len(need), max(need + [1]) + spare), -1, dtype=torch.int32)
    for i, n in enumerate(need):
        for j in range(n):
            t[i, j] = order.pop()
    return t.cuda()


def _filled(fmt, n_pages, ps, g, hd, seed):
    """A cache whose every row holds random values."""
    import scratch_llama_decoder_b200 as P
    gen = torch.Generator(device="cuda").manual_seed(seed)
    pages, scales = P.kv_pages(n_pages, ps, g, hd, fmt)
    x = torch.randn(pages.shape, generator=gen, device="cuda")
    if fmt == "e4m3":
        pages.copy_((x * 100).clamp(-448, 448).to(pages.dtype))
    elif fmt == "int8":
        pages.copy_((x * 40).round().clamp(-127, 127).to(torch.int8))
    else:
        pages.copy_(x.to(pages.dtype))
    if scales is not None:
        scales.copy_(torch.exp2(torch.randn(scales.shape, generator=gen, device="cuda")) / 60)
        if fmt == "e4m3":
            scales.copy_(torch.exp2(torch.round(torch.log2(scales))))
    return pages, scales


def _values(pages, scales):
    return pages.double() if scales is None else pages.double() * scales.double()[..., None]


# ------------------------------------------------------------ write and read
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("ps,g,hd", [(16, 2, 64), (64, 16, 64), (7, 1, 32), (1, 3, 128), (5, 2, 2),
                                     (16, 1, 40), (8, 3, 6), (32, 2, 126), (300, 5, 16)])
def test_write_and_read(ps, g, hd, dtype, fmt):
    import scratch_llama_decoder_b200 as P
    h, lens, starts = 2 * g, [0, 1, 37, 5, 64], [4, 0, 11, 63, 1]
    gen = torch.Generator(device="cuda").manual_seed(hd + ps)
    cu = torch.tensor([2, 2, 3, 40, 45, 109], dtype=torch.int32, device="cuda")
    n = 113  # 2 rows before, 4 behind
    qkv = torch.randn(n, h + 2 * g, hd, generator=gen, device="cuda")
    qkv = (qkv * torch.exp(3 * torch.randn(n, h + 2 * g, 1, generator=gen, device="cuda")))
    qkv[5, h] = 0.0
    qkv = qkv.to(dtype).reshape(n, -1)
    need = [-(-(a + b) // ps) for a, b in zip(starts, lens)]
    n_pages = sum(need) + 2
    table = _tables(need, n_pages, 1)
    pages, scales = _filled(fmt, n_pages, ps, g, hd, 2)
    before, sbefore = pages.clone(), None if scales is None else scales.clone()
    st = torch.tensor(starts, dtype=torch.int32, device="cuda")
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    P.kv_write(qkv, cu, h, pages, table, scales=scales, starts=st, flag=flag)
    assert int(flag) == 0
    kv = qkv.view(n, h + 2 * g, hd)[:, h:].reshape(n, 2, g, hd)
    val, unit = ref.stored(kv, fmt)
    if fmt == "e4m3":
        assert bool((kv.double().abs() <= 448 * unit[..., None]).all())
    want, swant = _values(before, sbefore), sbefore
    if scales is not None:
        swant = sbefore.double()
    for s in range(len(lens)):
        for t in range(lens[s]):
            p = starts[s] + t
            page, row, i = int(table[s, p // ps]), p % ps, int(cu[s]) + t
            want[page, :, :, row] = val[i]
            if swant is not None:
                swant[page, :, :, row] = unit[i]
    got = _values(pages, scales)
    assert torch.equal(got, want)  # every other row as it was
    if scales is not None:
        assert torch.equal(scales.double(), swant)
    k = torch.full((n, g, hd), 9.0, device="cuda").to(dtype)
    v = k.clone()
    P.kv_read(pages, table, cu, n, dtype, scales=scales, starts=st, k=k, v=v, flag=flag)
    assert int(flag) == 0
    back = val.float().to(dtype)  # one float32 product, then the type's rounding
    if fmt == "int8":
        codes = torch.round(val / unit[..., None])
        back = (codes.float() * unit.float()[..., None]).to(dtype)
    assert torch.equal(k[2:109], back[2:109, 0]) and torch.equal(v[2:109], back[2:109, 1])
    assert bool((k[:2] == 9).all() and (k[109:] == 9).all() and (v[109:] == 9).all())


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_codes_next_to_borders(fmt):
    """Values within a float32 step of the border between two codes."""
    import scratch_llama_decoder_b200 as P
    gen = torch.Generator(device="cuda").manual_seed(3)
    n, hd = 4096, 64
    amax = torch.exp(4 * torch.randn(n, 1, generator=gen, device="cuda"))
    unit = (amax / 127) if fmt == "int8" else amax / 448
    steps = torch.randint(-126, 126, (n, hd), generator=gen, device="cuda") + 0.5
    x = (steps * unit).float()
    x = torch.nextafter(x, x + torch.randint(-1, 2, (n, hd), generator=gen, device="cuda"))
    x[:, 0] = amax[:, 0]
    x = x.clamp(-amax, amax)
    qkv = torch.zeros(n, 3, hd, device="cuda")
    qkv[:, 1] = x
    qkv[:, 2] = -x
    pages, scales = P.kv_pages(n // 64, 64, 1, hd, fmt)
    table = torch.arange(n // 64, dtype=torch.int32, device="cuda")[None]
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    P.kv_write(qkv.view(n, -1), cu, 1, pages, table, scales=scales)
    val, u = ref.stored(x, fmt)
    got = _values(pages, scales)[:, 0, 0].reshape(n, hd)
    assert torch.equal(scales[:, 0, 0].reshape(n).double(), u)
    assert torch.equal(got, val)
    assert torch.equal(_values(pages, scales)[:, 1, 0].reshape(n, hd), -val)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_extreme_and_nonfinite_rows(fmt):
    import scratch_llama_decoder_b200 as P
    rows = [[0.0] * 8, [math.nan] + [1.0] * 7, [math.inf] + [1.0] * 7, [-math.inf] + [0.0] * 7,
            [3.4e38, -3.4e38] + [1e30] * 6, [1e-45] * 8, [1e-40, -1e-39] + [0.0] * 6,
            [448.0, 449.0, 447.0, 0.001, -448.0, 0.0, 2 ** -9, 1.5 * 2 ** -10],
            [1.0, -0.0, 1e-38, 1e-30, 0.5, 0.25, 3.0, -127.0]]
    n = len(rows)
    x = torch.tensor(rows, device="cuda")
    qkv = torch.stack([x, x, x], 1).view(n, -1)
    pages, scales = P.kv_pages(1, 16, 1, 8, fmt)
    table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    P.kv_write(qkv, cu, 1, pages, table, scales=scales)
    val, unit = ref.stored(x, fmt)
    got = _values(pages, scales)[0, 0, 0, :n]
    assert torch.equal(torch.isnan(got), torch.isnan(val))
    assert torch.equal(got.nan_to_num(), val.nan_to_num())
    k, v = P.kv_read(pages, table, cu, n, torch.float32, scales=scales)
    # code * scale rounded to float32: e4m3's 3.4e38 / 2^120 = 255.8 has the code
    # 256 (steps of 16 there), and 256 * 2^120 = 2^128 is past the largest float32
    want = val.float()
    assert bool(torch.isnan(k[1:4]).all()) and torch.equal(k[4:, 0], want[4:])
    assert bool(torch.isfinite(want[5:]).all())


@pytest.mark.parametrize("fmt", FORMATS)
def test_bad_places_are_skipped_and_flagged(fmt):
    import scratch_llama_decoder_b200 as P
    ps, g, hd, h = 8, 2, 64, 2
    for table, starts, lens in (([[0, -1]], [0], [16]), ([[5, 0]], [0], [16]),
                                ([[0, 1 << 30]], [0], [16]), ([[0, 1]], [9], [8]),
                                ([[0, 1]], [-3], [8]), ([[0, 1]], [2147483647], [8])):
        store, scales = _filled(fmt, 6, ps, g, hd, 4)
        pages = store[2:5]  # 3 pages, with room around them
        sc = None if scales is None else scales[2:5]
        before = store.clone()
        t = torch.tensor(table, dtype=torch.int32, device="cuda")
        st = torch.tensor(starts, dtype=torch.int32, device="cuda")
        n = lens[0]
        cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        qkv = torch.randn(n, (h + 2 * g) * hd, device="cuda")
        flag = torch.zeros(1, dtype=torch.int32, device="cuda")
        P.kv_write(qkv, cu, h, pages, t, scales=sc, starts=st, flag=flag)
        assert int(flag) == 2
        assert torch.equal(store[:2].view(torch.uint8), before[:2].view(torch.uint8))
        assert torch.equal(store[5:].view(torch.uint8), before[5:].view(torch.uint8))
        flag.zero_()
        k, v = P.kv_read(pages, t, cu, n, torch.float32, scales=sc, starts=st, flag=flag)
        assert int(flag) == 2
        val = _values(pages, sc)
        for i in range(n):
            p = starts[0] + i
            page = table[0][p // ps] if 0 <= p < 2 * ps else -1
            ok = 0 <= page < 3
            wk = val[page, 0, :, p % ps].float() if ok else torch.zeros(g, hd, device="cuda")
            assert torch.equal(k[i], wk)


# ---------------------------------------------------------------- attention
def _attend(fmt, dtype, h, g, hd, ps, lens, seed=0, big=1.0):
    import scratch_llama_decoder_b200 as P
    gen = torch.Generator(device="cuda").manual_seed(seed)
    need = [-(-n // ps) for n in lens]
    n_pages = sum(need) + 2
    table = _tables(need, n_pages, seed)
    pages, scales = _filled(fmt, n_pages, ps, g, hd, seed + 1)
    q = (torch.randn(len(lens), h * hd, generator=gen, device="cuda") * big).to(dtype)
    # what lies past a sequence's length is not looked at
    for s, n in enumerate(lens):
        if n % ps:
            page = int(table[s, n // ps])
            if fmt in ("e4m3", "int8"):
                scales[page, :, :, n % ps:] = math.nan
                if fmt == "e4m3":
                    pages.view(torch.uint8)[page, :, :, n % ps:] = 0x7f  # NaN
            else:
                pages[page, :, :, n % ps:] = math.nan
    lt = torch.tensor(lens, dtype=torch.int32, device="cuda")
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = P.attention_paged(q, pages, table, lt, scales=scales, flag=flag)
    ro, rl, bo, bl = ref.paged(q, pages, scales, table, lens, h, dtype)
    live = torch.tensor([n > 0 for n in lens], device="cuda")
    ref.check(out, ro, bo, "out")
    ref.check(lse[live], rl[live], bl[live], "lse")
    assert bool((out[~live] == 0).all() and (lse[~live] == -math.inf).all())
    assert int(flag) == 0
    again = P.attention_paged(q, pages, table, lt, scales=scales)
    assert torch.equal(again[0], out) and torch.equal(again[1], lse)


LENS = [[1], [0], [63, 64, 65, 1, 0, 200], [1000, 3, 129], [17] * 40, [2500, 1, 1, 1]]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("hd", [32, 64, 128])
@pytest.mark.parametrize("h,g", [(4, 4), (8, 2), (8, 1), (3, 1)])
def test_attention(h, g, hd, dtype, fmt):
    for i, lens in enumerate(LENS):
        _attend(fmt, dtype, h, g, hd, (16, 64, 8)[i % 3], lens, seed=i)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("ps,h,g,hd", [(7, 4, 2, 64), (1, 2, 2, 64), (300, 4, 4, 32), (16, 20, 1, 64),
                                       (16, 34, 2, 32), (16, 4, 2, 40), (3, 2, 1, 2), (16, 6, 3, 96),
                                       (64, 17, 1, 128), (16, 4, 4, 126)])
def test_attention_odd_layouts(ps, h, g, hd, dtype, fmt):
    _attend(fmt, dtype, h, g, hd, ps, [130, 0, 1, 77], seed=ps)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", DTYPES)
def test_attention_large_scores(dtype, fmt):
    _attend(fmt, dtype, 8, 2, 64, 16, [500, 33], seed=5, big=20.0)


@pytest.mark.parametrize("fmt", FORMATS)
def test_bad_pages_are_left_out(fmt):
    import scratch_llama_decoder_b200 as P
    h, g, hd, ps = 8, 2, 64, 16
    for dtype in DTYPES:
        pages, scales = _filled(fmt, 8, ps, g, hd, 6)
        q = torch.randn(5, h * hd, device="cuda").to(dtype)
        table = torch.tensor([[0, -1, 1, 1 << 30], [8, 2, 3, -7], [-1, -1, -1, -1], [4, 5, 6, 7],
                              [4, 5, 6, 7]], dtype=torch.int32, device="cuda")
        lens = [64, 50, 10, 100000, -4]
        lt = torch.tensor(lens, dtype=torch.int32, device="cuda")
        flag = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = P.attention_paged(q, pages, table, lt, scales=scales, flag=flag)
        assert int(flag) == 2
        ro, rl, bo, bl = ref.paged(q, pages, scales, table, lens, h, dtype)
        ref.check(out, ro, bo, "out")
        live = torch.tensor([True, True, False, True, False], device="cuda")
        ref.check(lse[live], rl[live], bl[live], "lse")
        assert bool((out[~live] == 0).all() and (lse[~live] == -math.inf).all())


def test_strided_queries_and_tables():
    import scratch_llama_decoder_b200 as P
    h, g, hd, ps, lens = 8, 2, 64, 16, [100, 7, 40]
    for dtype in DTYPES:
        pages, scales = _filled("bf16", 20, ps, g, hd, 7)
        wide = torch.randn(3, (h + 2 * g) * hd + 5, device="cuda").to(dtype)
        q = wide[:, 1:1 + h * hd]
        table = _tables([7, 1, 3], 20, 8)
        big = torch.full((3, 50), -1, dtype=torch.int32, device="cuda")
        big[:, 3:3 + table.shape[1]] = table
        lt = torch.tensor(lens, dtype=torch.int32, device="cuda")
        got = P.attention_paged(q, pages, big[:, 3:3 + table.shape[1]], lt)
        want = P.attention_paged(q.contiguous(), pages, table, lt)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_long_cache_past_32_bit_offsets():
    """Pages whose element offsets pass 2^31 and 2^32."""
    import scratch_llama_decoder_b200 as P
    h, g, hd, ps = 8, 8, 128, 64
    n_pages = (1 << 32) // (2 * g * ps * hd) + 40  # 4.3 G elements of 1 byte
    pages = torch.zeros(n_pages, 2, g, ps, hd, dtype=torch.int8, device="cuda")
    scales = torch.zeros(n_pages, 2, g, ps, device="cuda")
    last = list(range(n_pages - 20, n_pages))
    table = torch.tensor([last], dtype=torch.int32, device="cuda")
    n = 20 * ps - 3
    gen = torch.Generator(device="cuda").manual_seed(9)
    qkv = torch.randn(n, 3 * h * hd, generator=gen, device="cuda").to(torch.bfloat16)
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    P.kv_write(qkv, cu, h, pages, table, scales=scales)
    assert int((scales[:-20] != 0).sum()) == 0
    k, v = P.kv_read(pages, table, cu, n, torch.bfloat16, scales=scales)
    x = qkv.view(n, 3, g, hd)
    val, unit = ref.stored(x[:, 1], "int8")
    assert float((k.double() - val).abs().max()) <= 2.0 ** -8 * float(val.abs().max())
    q = torch.randn(1, h * hd, generator=gen, device="cuda").to(torch.bfloat16)
    out, lse = P.attention_paged(q, pages, table, cu[1:], scales=scales)
    small = torch.arange(20, dtype=torch.int32, device="cuda")[None]
    o2, l2 = P.attention_paged(q, pages[-20:], small, cu[1:], scales=scales[-20:])
    assert torch.equal(out, o2) and torch.equal(lse, l2)


def test_graph_serves_other_lengths():
    import scratch_llama_decoder_b200 as P
    h, g, hd, ps = 8, 2, 64, 16
    pages, scales = _filled("int8", 200, ps, g, hd, 10)
    table = _tables([40, 40, 40, 40], 200, 11, spare=0)
    q = torch.randn(4, h * hd, device="cuda").to(torch.bfloat16)
    lens = torch.tensor([640, 1, 0, 64], dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    for _ in range(2):  # two captured calls replayed at once share nothing
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side):
            with torch.cuda.graph(graph, stream=side):
                res = P.attention_paged(q, pages, table, lens, scales=scales)
        graphs.append((graph, res, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for new in ([640, 1, 0, 64], [0, 0, 0, 0], [5, 600, 601, 640], [64, 65, 128, 129]):
        lens.copy_(torch.tensor(new, dtype=torch.int32))
        want = P.attention_paged(q, pages, table, lens, scales=scales)
        torch.cuda.synchronize()
        for graph, _, st in graphs:
            with torch.cuda.stream(st):
                for _ in range(5):
                    graph.replay()
        torch.cuda.synchronize()
        for _, res, _ in graphs:
            assert torch.equal(res[0], want[0]) and torch.equal(res[1], want[1])


@pytest.mark.parametrize("dtype,fmt", [(torch.float32, "f32"), (torch.bfloat16, "bf16"),
                                       (torch.bfloat16, "e4m3"), (torch.bfloat16, "int8"),
                                       (torch.float32, "int8")])
def test_prompts_then_tokens(dtype, fmt):
    """As a server runs them: prompts through packed attention, their k and v
    into the cache (the second one in two parts), then token by token: write,
    attend.  Every step's output is that of attention over the stored values
    of the whole sequence so far."""
    import scratch_llama_decoder_b200 as P
    h, g, hd, ps, prompt, steps = 8, 2, 64, 16, [33, 100, 1], 6
    gen = torch.Generator(device="cuda").manual_seed(12)
    w = (h + 2 * g) * hd
    total = [n + steps for n in prompt]
    seqs = [torch.randn(n, w, generator=gen, device="cuda").to(dtype) for n in total]
    need = [-(-n // ps) for n in total]
    table = _tables(need, sum(need) + 3, 13)
    pages, scales = P.kv_pages(sum(need) + 3, ps, g, hd, fmt)
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    batch = torch.cat([s[:n] for s, n in zip(seqs, prompt)])
    cu = [0, 33, 133, 134]
    out, lse = P.attention_packed(batch, ints(cu), h, g, flag=flag)
    ro, rl, bo, bl = ref.attention(batch, cu, h, g, dtype)
    ref.check(out, ro, bo, "prompt out")
    # sequence 1's first 60 rows, then the rest of it, apart from the others
    P.kv_write(batch[:93], ints([0, 33, 93]), h, pages, table, scales=scales, flag=flag)
    P.kv_write(batch[93:], ints([0, 0, 40, 41]), h, pages, table, scales=scales,
               starts=ints([33, 60, 0]), flag=flag)
    for t in range(steps):
        new = torch.stack([s[n + t] for s, n in zip(seqs, prompt)])
        P.kv_write(new, ints([0, 1, 2, 3]), h, pages, table, scales=scales,
                   starts=ints([n + t for n in prompt]), flag=flag)
        lens = [n + t + 1 for n in prompt]
        o, l = P.attention_paged(new[:, :h * hd], pages, table, ints(lens), scales=scales,
                                 flag=flag)
        ro, rl, bo, bl = ref.paged(new[:, :h * hd].contiguous(), pages, scales, table, lens, h,
                                   dtype)
        ref.check(o, ro, bo, "token out")
        ref.check(l, rl, bl, "token lse")
    assert int(flag) == 0
    # the cache holds the stored values of every row
    lens = total
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    k, v = P.kv_read(pages, table, ints(cu), cu[-1], torch.float32, scales=scales)
    kv = torch.cat(seqs).view(-1, h + 2 * g, hd)[:, h:].reshape(-1, 2, g, hd)
    val, _ = ref.stored(kv, fmt)
    assert float((k.double() - val[:, 0]).abs().max()) <= 2.0 ** -22
    assert float((v.double() - val[:, 1]).abs().max()) <= 2.0 ** -22
    if fmt in ("f32", "bf16"):  # then the last step is the packed attention's last row
        full, flse = P.attention_packed(torch.cat(seqs), ints(cu), h, g)
        last = torch.tensor(cu[1:], device="cuda") - 1
        ro, rl, bo, bl = ref.attention(torch.cat(seqs), cu, h, g, dtype)
        ref.check(o, ro[last], bo[last] * 2, "last token")
        ref.check(full[last], ro[last], bo[last], "last row")


def test_refused_arguments():
    import scratch_llama_decoder_b200 as P
    pages, scales = P.kv_pages(4, 16, 2, 64, "int8")
    table = torch.zeros(1, 2, dtype=torch.int32, device="cuda")
    q = torch.zeros(1, 8 * 64, device="cuda")
    lens = torch.ones(1, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    qkv = torch.zeros(1, 12 * 64, device="cuda")
    with pytest.raises(ValueError):
        P.attention_paged(q, pages, table, lens)  # no scales
    with pytest.raises(ValueError):
        P.attention_paged(q[:, :100], pages, table, lens, scales=scales)
    with pytest.raises(ValueError):
        P.attention_paged(q, pages, table, lens.long(), scales=scales)
    with pytest.raises(ValueError):
        P.attention_paged(q.expand(2, -1), pages, table, lens, scales=scales)
    with pytest.raises(ValueError):
        P.attention_paged(q, pages.transpose(0, 2), table, lens, scales=scales)
    with pytest.raises(ValueError):
        P.kv_write(qkv, cu, 4, pages, table, scales=scales)
    with pytest.raises(ValueError):
        P.kv_write(qkv, cu, 8, pages, table.cpu(), scales=scales)
    with pytest.raises(ValueError):
        P.kv_read(pages, table, cu, 1, torch.float16, scales=scales)
    with pytest.raises(ValueError):
        P.kv_pages(4, 16, 2, 64, "int4")


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", DTYPES)
def test_bad_pages_of_split_sequences(dtype, fmt):
    """Tables long enough for the split form: bad lengths, bad pages, none."""
    import scratch_llama_decoder_b200 as P
    h, g, hd, ps = 8, 2, 64, 16
    pages, scales = _filled(fmt, 70, ps, g, hd, 20)
    q = torch.randn(6, h * hd, device="cuda").to(dtype)
    table = torch.randint(0, 70, (6, 60), generator=torch.Generator().manual_seed(21))
    table[0, 5], table[0, 40], table[1, 0], table[2, :] = -1, 70, 1 << 30, -(1 << 31)
    table = table.to(torch.int32).cuda()
    lens = [960, 200, 900, (1 << 31) - 1, -(1 << 31), 0]
    lt = torch.tensor(lens, dtype=torch.int32, device="cuda")
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = P.attention_paged(q, pages, table, lt, scales=scales, flag=flag)
    assert int(flag) == 2
    ro, rl, bo, bl = ref.paged(q, pages, scales, table, lens, h, dtype)
    ref.check(out, ro, bo, "out")
    live = torch.tensor([True, True, False, True, False, False], device="cuda")
    ref.check(lse[live], rl[live], bl[live], "lse")
    assert bool((out[~live] == 0).all() and (lse[~live] == -math.inf).all())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("hd,h,g,cols", [(64, 4, 2, 60), (64, 4, 2, 70), (128, 20, 2, 70)])
def test_most_sequences(hd, h, g, cols, dtype, fmt):
    """8192 sequences, some long, in pages that all of them share; tables that
    are not split and tables that are."""
    import scratch_llama_decoder_b200 as P
    n, ps, n_pages = 8192, 16, 300
    pages, scales = _filled(fmt, n_pages, ps, g, hd, 22)
    gen = torch.Generator().manual_seed(23)
    lens = torch.randint(0, 40, (n,), generator=gen)
    some = torch.randperm(n, generator=gen)[:24]
    lens[some[:12]] = torch.randint(0, 961, (12,), generator=gen)
    lens[0], lens[-1] = 960, 0
    table = torch.randint(0, n_pages, (n, cols), generator=gen).to(torch.int32)
    q = torch.randn(n, h * hd, device="cuda").to(dtype)
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = P.attention_paged(q, pages, table.cuda(), lens.to(torch.int32).cuda(),
                                 scales=scales, flag=flag)
    assert int(flag) == 0
    some = torch.cat([some, torch.tensor([0, 1, n - 2, n - 1])])
    sl = lens[some].tolist()
    ro, rl, bo, bl = ref.paged(q[some.cuda()], pages, scales, table[some], sl, h, dtype)
    live = torch.tensor([x > 0 for x in sl], device="cuda")
    ref.check(out[some.cuda()], ro, bo, "out")
    ref.check(lse[some.cuda()][live], rl[live], bl[live], "lse")
    empty = (lens == 0).cuda()
    assert bool((out[empty] == 0).all() and (lse[empty] == -math.inf).all())
    assert bool(torch.isfinite(lse[~empty]).all())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("long", [False, True])
def test_a_nan_row_stays_with_its_readers(long, dtype, fmt):
    """A cached row that is not finite makes the outputs of the sequences and
    heads that read it NaN, and changes no other's bits; a prefix shared by
    sequences reads as if each had its own."""
    import scratch_llama_decoder_b200 as P
    h, g, hd, ps = 8, 2, 64, 16
    pages, scales = _filled(fmt, 90, ps, g, hd, 24)
    cols = 40 if long else 6
    table = torch.arange(80, dtype=torch.int32).view(2, 40)[:, :cols].repeat(2, 1)
    table[2:, :2] = table[:1, :2]  # sequences 2 and 3 share the first pages of 0
    table = table.cuda()
    lens = [cols * ps, cols * ps - 3, 31, cols * ps]
    lt = torch.tensor(lens, dtype=torch.int32, device="cuda")
    q = torch.randn(4, h * hd, device="cuda").to(dtype)
    want = P.attention_paged(q, pages, table, lt, scales=scales)
    ro, rl, bo, bl = ref.paged(q, pages, scales, table, lens, h, dtype)
    ref.check(want[0], ro, bo, "out")
    row = pages[1, :, 1, 3]  # position 19 of sequences 0, 2, 3, kv head 1
    if scales is None:
        row[0, 5] = math.nan
    else:
        scales[1, 0, 1, 3] = math.nan
    out, lse = P.attention_paged(q, pages, table, lt, scales=scales)
    o, w = (t.view(4, g, -1) for t in (out, want[0]))
    l, wl = (t.view(4, g, -1) for t in (lse, want[1]))
    for s in range(4):
        for i in range(g):
            if i == 1 and s != 1:
                assert bool(torch.isnan(o[s, i]).all() and torch.isnan(l[s, i]).all())
            else:
                assert torch.equal(o[s, i], w[s, i]) and torch.equal(l[s, i], wl[s, i])


def test_captured_steps_write_and_attend():
    """One captured step (write the new tokens, attend, move on) replayed: the
    positions advance on the device; two streams at once on their own caches."""
    import scratch_llama_decoder_b200 as P
    h, g, hd, ps, steps = 8, 2, 64, 16, 40
    runs = []
    side = torch.cuda.Stream()
    cu = torch.arange(4, dtype=torch.int32, device="cuda")
    for seed in (25, 26):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        pages, scales = P.kv_pages(130, ps, g, hd, "e4m3")
        table = _tables([40, 40, 40], 130, seed)
        first = torch.tensor([0, 15, 590], dtype=torch.int32, device="cuda")
        rows = torch.randn(steps, 3, (h + 2 * g) * hd, generator=gen, device="cuda")
        rows = rows.to(torch.bfloat16)
        pos, x = first.clone(), rows[0].clone()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side):
            with torch.cuda.graph(graph, stream=side):
                P.kv_write(x, cu, h, pages, table, scales=scales, starts=pos)
                pos.add_(1)
                out, lse = P.attention_paged(x[:, :h * hd], pages, table, pos, scales=scales)
                k, v = P.kv_read(pages, table, cu, 3, torch.float32, scales=scales, starts=pos - 1)
        runs.append((pages, scales, table, first, rows, pos, x, graph, out, lse, k, v,
                     torch.cuda.Stream(), []))
    torch.cuda.synchronize()
    for t in range(steps):
        for _, _, _, _, rows, _, x, graph, out, lse, k, v, st, got in runs:
            with torch.cuda.stream(st):
                x.copy_(rows[t])
                graph.replay()
                got.append([y.clone() for y in (out, lse, k, v)])
    torch.cuda.synchronize()
    for pages, scales, table, first, rows, pos, _, _, _, _, _, _, _, got in runs:
        assert torch.equal(pos, first + steps)
        p2, s2 = P.kv_pages(130, ps, g, hd, "e4m3")
        for t in range(steps):
            P.kv_write(rows[t], cu, h, p2, table, scales=s2, starts=first + t)
            o, l = P.attention_paged(rows[t][:, :h * hd], p2, table, first + t + 1, scales=s2)
            k, v = P.kv_read(p2, table, cu, 3, torch.float32, scales=s2, starts=first + t)
            for a, b in zip(got[t], (o, l, k, v)):
                assert torch.equal(a, b)
        assert torch.equal(p2.view(torch.uint8), pages.view(torch.uint8))
        assert torch.equal(s2, scales)


@pytest.mark.parametrize("dtype", DTYPES)
def test_offsets_that_decrease_write_inside_the_cache(dtype):
    """cu_seqlens of any contents: rows go to places of the tables or nowhere."""
    import scratch_llama_decoder_b200 as P
    h, g, hd, ps, n = 4, 2, 32, 8, 100
    qkv = torch.randn(n, (h + 2 * g) * hd, device="cuda").to(dtype)
    for cu in ([0, 60, 20, 100], [-50, 1 << 30, 5, -1], [100, 100, 0, 0],
               [(1 << 31) - 1, -(1 << 31), (1 << 31) - 1, 7]):
        for fmt in FORMATS:
            store, scales = _filled(fmt, 12, ps, g, hd, 27)
            before = store.clone()
            table = torch.tensor([[0, 1], [2, 3], [4, 5]], dtype=torch.int32, device="cuda")
            sc = None if scales is None else scales[3:9]
            cut = torch.tensor(cu, dtype=torch.int32, device="cuda")
            P.kv_write(qkv, cut, h, store[3:9], table, scales=sc)
            k, v = P.kv_read(store[3:9], table, cut, n, dtype, scales=sc)
            for part in (slice(0, 3), slice(9, 12)):
                assert torch.equal(store[part].view(torch.uint8), before[part].view(torch.uint8))
