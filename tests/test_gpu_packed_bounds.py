"""Packed attention on tcgen05 tiles at every head size and spacing it takes,
and bounds that pin the roundings the kernels avoid: D of a sequence's first
rows without the rounding of out, and the cache attention's weights in more
than bfloat16."""
import math

import pytest
import torch

from tests import packed_ref as ref
from tests.test_gpu_packed import _check, _data

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
U, R = ref.U, ref.R[BF]

# mean lengths far above those of the mma.sync kernels; 4 heads: no plan, 16: a plan
LONG = [900, 0, 1300, 1, 385]


@pytest.mark.parametrize("h,g", [(4, 2), (16, 4)])
@pytest.mark.parametrize("hd", [8, 16, 24, 40, 48, 56, 72, 80, 88, 96, 104, 112, 120])
def test_long_sequences_at_other_head_sizes(hd, h, g):
    qkv, dout, cu, cut = _data(LONG, h, g, hd, BF, seed=41 + hd)
    _check(qkv, dout, cu, cut, h, g)


@pytest.mark.parametrize("h,g", [(4, 2), (16, 4)])
@pytest.mark.parametrize("hd", [8, 32, 48, 64, 88, 128])
@pytest.mark.parametrize("pad,off", [(8, 0), (24, 8), (3, 1)])
def test_long_sequences_of_spaced_rows(pad, off, hd, h, g):
    """Rows apart, on 16 bytes (tensor maps) and not; nothing between them written."""
    import scratch_llama_decoder_b200 as P
    dense, dout, cu, cut = _data(LONG, h, g, hd, BF, seed=42)
    n, w = dense.shape
    base = torch.full((n * (w + pad) + off + 8,), 7.0, device="cuda").to(BF)
    qkv = base[off:off + n * (w + pad)].view(n, w + pad)[:, :w]
    qkv.copy_(dense)
    out, lse = _check(qkv, dout, cu, cut, h, g)
    store = torch.full_like(base, 7.0)
    dst = store[off:off + n * (w + pad)].view(n, w + pad)[:, :w]
    P.attention_packed_backward(qkv, cut, h, g, out, lse, dout, dqkv=dst)
    rx, bx = ref.backward(qkv, cu, h, g, out, lse, dout, BF)
    ref.check(dst, rx, bx, "spaced dqkv")
    dst.fill_(7.0)
    assert bool((store == 7.0).all())


def _equal(x, dout, lse, h, g, dtype, rows):
    """dqkv of sequences of one length, [s, length, ...] in 64 bits with the given lse,
    and its bounds, where D of the first `rows` rows is the quotient of sums over
    the kernel's own weights: off by their errors times |dP - D| and by the sums'."""
    s, m, _, hd = x.shape
    c, r, ex = 1 / math.sqrt(hd), ref.R[dtype], ref.EXP[dtype]
    dx = torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    bd = torch.zeros_like(dx)
    keep = torch.ones(m, m, dtype=torch.float64, device=x.device).tril()
    for i in range(h):
        j = i // (h // g)
        Q, K, V, G = (t.double() for t in (x[:, :, i], x[:, :, h + j], x[:, :, h + g + j],
                                           dout[:, :, i]))
        L = lse[:, :, i].double()[..., None]
        sc = Q @ K.transpose(1, 2) * c
        p = torch.exp(torch.where(keep > 0, sc - L, torch.full_like(sc, -math.inf)))
        dP = G @ V.transpose(1, 2)
        D = (p * dP).sum(2, keepdim=True)
        gap = (dP - D).abs()
        ds = p * (dP - D)
        # as packed_ref.backward
        ep = ((hd + 3) * U * (Q.abs() @ K.abs().transpose(1, 2)) * c
              + 3 * U * (sc.abs() + L.abs()) + ex) * p
        edp = (hd + 2) * U * (G.abs() @ V.abs().transpose(1, 2))
        eD = (ep * gap + p * edp + (2 * m + 8) * U * p * (gap + D.abs())).sum(2, keepdim=True)
        eds = p * (edp + eD) + ep * gap + (r + 3 * U) * ds.abs()
        sums = (m * (h // g) + 8) * U
        dx[:, :, i] = ds @ K * c
        bd[:, :, i] = (eds + sums * ds.abs()) @ K.abs() * c
        dx[:, :, h + j] += ds.transpose(1, 2) @ Q * c
        bd[:, :, h + j] += (eds + sums * ds.abs()).transpose(1, 2) @ Q.abs() * c
        dx[:, :, h + g + j] += p.transpose(1, 2) @ G
        bd[:, :, h + g + j] += (ep + (r + sums) * p).transpose(1, 2) @ G.abs()
    bd += ref.R[dtype] * dx.abs()
    if rows < m:  # later rows may take D from out: only dq of the first
        return dx[:, :rows, :h], bd[:, :rows, :h] + 1e-30
    return dx, bd + 1e-30


# lengths, sequences, rows whose D is their own: one tile of the mma.sync kernels (64
# rows) and of the tcgen05 ones (128)
FIRST = [(1, 3000, 1), (2, 1500, 2), (3, 1000, 3), (7, 900, 7), (64, 40, 64), (100, 12, 64),
         (700, 3, 64), (700, 12, 64)]


@pytest.mark.parametrize("hd", [32, 64, 72, 128])
@pytest.mark.parametrize("h,g", [(4, 2), (2, 2)])
@pytest.mark.parametrize("m,s,rows", FIRST)
def test_gradients_of_the_first_rows(m, s, rows, h, g, hd):
    """Row 0 has one weight, 1, whatever its score: its dq is 0 to the rounding of
    float32, not of out."""
    import scratch_llama_decoder_b200 as P
    qkv, dout, cu, cut = _data([m] * s, h, g, hd, BF, seed=43)
    out, lse = P.attention_packed(qkv, cut, h, g)
    dx = P.attention_packed_backward(qkv, cut, h, g, out, lse, dout)
    rx, bx = _equal(qkv.view(s, m, h + 2 * g, hd), dout.view(s, m, h, hd),
                    lse.view(h, s, m).permute(1, 2, 0), h, g, BF, rows)
    ref.check(dx.view(s, m, h + 2 * g, hd)[:, :rx.shape[1], :rx.shape[2]], rx, bx, (m, s))


@pytest.mark.parametrize("h,g", [(4, 2), (2, 2)])
@pytest.mark.parametrize("m,s,rows", FIRST[:5])
def test_float32_gradients_of_short_sequences(m, s, rows, h, g):
    import scratch_llama_decoder_b200 as P
    qkv, dout, cu, cut = _data([m] * s, h, g, 64, torch.float32, seed=44)
    out, lse = P.attention_packed(qkv, cut, h, g)
    dx = P.attention_packed_backward(qkv, cut, h, g, out, lse, dout)
    rx, bx = ref.backward(qkv[:60 * m], cu[:61], h, g, out[:60 * m], lse[:, :60 * m],
                          dout[:60 * m], torch.float32) if s > 60 else \
        ref.backward(qkv, cu, h, g, out, lse, dout, torch.float32)
    ref.check(dx[:rx.shape[0]], rx, bx, (m, s))
    # the last sequences as the first: the same rows give the same bits
    x2, d2 = qkv.flip(0).contiguous(), dout.flip(0).contiguous()
    x2, d2 = (t.view(s, m, -1).flip(1).reshape(t.shape) for t in (x2, d2))
    o2, l2 = P.attention_packed(x2, cut, h, g)
    dx2 = P.attention_packed_backward(x2, cut, h, g, o2, l2, d2)
    assert torch.equal(dx2.view(s, m, -1).flip(0), dx.view(s, m, -1))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "int8"])
@pytest.mark.parametrize("hd", [32, 64, 128])
@pytest.mark.parametrize("h,g", [(4, 4), (8, 2), (16, 1)])
@pytest.mark.parametrize("n", [1, 60, 500, 3000])
def test_cache_weights_keep_more_than_bfloat16(n, h, g, hd, fmt):
    """bfloat16 queries: a weight enters the product with v as two bfloat16 terms
    (2^-8 of 2^-8) over a bfloat16 cache, as one float16 (2^-11) over 8-bit codes.
    Beside it: scores by hd float32 sums, one exponential (2^-21), sums over n
    keys of which a tensor core may drop the last bit instead of rounding (2 U)."""
    import scratch_llama_decoder_b200 as P
    b, ps = 3, 16
    gen = torch.Generator(device="cuda").manual_seed(45)
    cols = -(-n // ps)
    pages, scales = P.kv_pages(b * cols, ps, g, hd, fmt)
    table = torch.randperm(b * cols, generator=gen, device="cuda").to(torch.int32).view(b, cols)
    rows = torch.randn(b * n, (h + 2 * g) * hd, generator=gen, device="cuda").to(BF)
    cu = torch.arange(0, b * n + 1, n, dtype=torch.int32, device="cuda")
    P.kv_write(rows, cu, h, pages, table, scales=scales)
    q = torch.randn(b, h * hd, generator=gen, device="cuda").to(BF)
    lens = torch.full((b,), n, dtype=torch.int32, device="cuda")
    out, lse = P.attention_paged(q, pages, table, lens, scales=scales)
    x = pages.double() if scales is None else pages.double() * scales.double()[..., None]
    x = x[table.long()].permute(0, 2, 3, 1, 4, 5).reshape(b, 2, g, cols * ps, hd)[..., :n, :]
    k, v = (x[:, i].repeat_interleave(h // g, 1) for i in (0, 1))
    z = q.double().view(b, h, 1, hd)
    sc = (z * k).sum(-1) / math.sqrt(hd)
    L = torch.logsumexp(sc, 2)
    p = torch.exp(sc - L[..., None])
    O = (p[..., None] * v).sum(2)
    es = (2 * (hd + 8) * U * (z.abs() * k.abs()).sum(-1) / math.sqrt(hd)
          + 8 * U * sc.abs()).amax(2) + 2.0 ** -21
    r = 2.0 ** -16 if fmt == "bf16" else 2.0 ** -11
    bound = (2 * es + (4 * n + 32) * U + r)[..., None] * (p[..., None] * v.abs()).sum(2)
    if fmt != "bf16":  # half a step of the least float16 weights, as in packed_ref.paged
        sv = scales[table.long()][:, :, 1].permute(0, 2, 1, 3).reshape(b, g, -1)[..., :n].double()
        sv = sv.repeat_interleave(h // g, 1)
        bound += 2.0 ** -38 * (p * sv).amax(2)[..., None] * (v.abs() / sv[..., None]).sum(2)
    ref.check(out.view(b, h, hd), O, bound + R * O.abs() + 1e-30, "out")
    ref.check(lse, L, es + (2 * n + 16) * U + 4 * U * L.abs() + 1e-30, "lse")
