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
