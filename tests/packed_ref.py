"""Plain 64-bit forms of the packed attention and the paged cache, and the
error bounds their 32-bit and bfloat16 kernels are held to.

Rounding units: u = 2^-24 (float32), r = finfo(bfloat16).eps / 2 = 2^-8.  A
dot product of n float32 products is off by at most (n + 1) u sum|a_i b_i|
whatever the order of its sum, a softmax weight by its score's absolute error
times itself plus the exponential's own (2^-12 covers the kernels' fastest,
a polynomial fitted to 7.5e-5; 4 u float32's expf and exp2f), and the
bfloat16 kernels round the weights (and dS) to bfloat16 before they enter a
product with the values: r more of each term.
"""
import math

import torch

U = 2.0 ** -24
R = {torch.float32: 0.0, torch.bfloat16: torch.finfo(torch.bfloat16).eps / 2}
EXP = {torch.float32: 4 * U, torch.bfloat16: 2.0 ** -12}


def split(qkv, h, g):
    """q [n, h, hd], k, v [n, g, hd] of q|k|v rows, in 64 bits."""
    n = qkv.shape[0]
    return qkv.double().reshape(n, h + 2 * g, qkv.shape[1] // (h + 2 * g)).split([h, g, g], 1)


def attention(qkv, cu, h, g, want=None):
    """out, lse and their error bounds for the rows of the sequences
    (elsewhere 0); cu: list of offsets; want: the kernel's type."""
    n, hd = qkv.shape[0], qkv.shape[1] // (h + 2 * g)
    q, k, v = split(qkv, h, g)
    out = torch.zeros(n, h, hd, dtype=torch.float64, device=qkv.device)
    lse = torch.zeros(h, n, dtype=torch.float64, device=qkv.device)
    ob, lb = torch.zeros_like(out), torch.zeros_like(lse)
    r, ex = (R[want], EXP[want]) if want is not None else (0.0, 0.0)
    for a, b in zip(cu[:-1], cu[1:]):
        if b <= a:
            continue
        m = b - a
        for i in range(h):
            j = i // (h // g)
            o, L, p, s, _ = _one(q[a:b, i], k[a:b, j], v[a:b, j])
            out[a:b, i], lse[i, a:b] = o, L
            # score error: the dot product's, and two roundings of the score
            es = ((hd + 3) * U * (q[a:b, i].abs() @ k[a:b, j].abs().t()) / math.sqrt(hd)
                  + 2 * U * s.abs()).tril().amax(1)
            # weights and their sum each move by es + ex; m terms are summed twice
            rel = 2 * (es + ex) + (2 * m + 16) * U + r
            ob[a:b, i] = rel[:, None] * (p @ v[a:b, j].abs()) + R[want or torch.float32] * o.abs()
            lb[i, a:b] = es + ex + (m + 8) * U + 4 * U * L.abs()
    return out.reshape(n, h * hd), lse, ob.reshape(n, h * hd) + 1e-30, lb + 1e-30


def _one(q, k, v):
    m, hd = q.shape
    s = q @ k.t() / math.sqrt(hd)
    keep = torch.ones(m, m, dtype=torch.bool, device=q.device).tril()
    z = s.masked_fill(~keep, -math.inf)
    L = torch.logsumexp(z, 1)
    p = torch.exp(z - L[:, None])
    return p @ v, L, p, s, keep


def backward(qkv, cu, h, g, out, lse, dout, want):
    """dqkv and its error bound, from the formulas with the given lse; D is the
    exact sum_j P_ij dP_ij.  A kernel may take it as dout . out instead: out is
    off by its own bound (attention's), D by that times |dout|, summed.  Or it
    may form the sum from its own weights: off by their errors times |dP - D|."""
    n, hd = qkv.shape[0], qkv.shape[1] // (h + 2 * g)
    c = 1 / math.sqrt(hd)
    q, k, v = split(qkv, h, g)
    o, do = (t.double().reshape(n, h, hd) for t in (out, dout))
    dx = torch.zeros(n, h + 2 * g, hd, dtype=torch.float64, device=qkv.device)
    bd = torch.zeros_like(dx)
    r, ex = R[want], EXP[want]
    for a, b in zip(cu[:-1], cu[1:]):
        if b <= a:
            continue
        m = b - a
        keep = torch.ones(m, m, dtype=torch.float64, device=qkv.device).tril()
        for i in range(h):
            j = i // (h // g)
            Q, K, V, O, G = q[a:b, i], k[a:b, j], v[a:b, j], o[a:b, i], do[a:b, i]
            L = lse[i, a:b].double()[:, None]
            s = Q @ K.t() * c
            p = torch.exp(torch.where(keep > 0, s - L, torch.full_like(s, -math.inf)))
            dP = G @ V.t()
            D = (p * dP).sum(1, keepdim=True)
            ds = p * (dP - D)
            # weight error (its score, L and their difference), then dS's
            ep = ((hd + 3) * U * (Q.abs() @ K.abs().t()) * c + 3 * U * (s.abs() + L.abs()) + ex) * p
            rel = 2 * (ep.sum(1, keepdim=True) + ex) + (2 * m + 16) * U + r
            eo = rel * (p @ V.abs()) + R[want] * O.abs()  # out's bound
            eD = (G.abs() * eo).sum(1, keepdim=True) + (ep * (dP - D).abs()).sum(1, keepdim=True)
            eds = (p * (hd + 2) * U * (G.abs() @ V.abs().t() + (G * O).abs().sum(1, keepdim=True))
                   + p * eD + ep * (dP - D).abs() + (r + 3 * U) * ds.abs())
            sums = (m * (h // g) + 8) * U
            dx[a:b, i] = ds @ K * c
            bd[a:b, i] = (eds + sums * ds.abs()) @ K.abs() * c
            dx[a:b, h + j] += ds.t() @ Q * c
            bd[a:b, h + j] += (eds + sums * ds.abs()).t() @ Q.abs() * c
            dx[a:b, h + g + j] += p.t() @ G
            bd[a:b, h + g + j] += (ep + (r + sums) * p).t() @ G.abs()
    bd += R[want] * dx.abs()
    return dx.reshape(n, qkv.shape[1]), bd.reshape(n, qkv.shape[1]) + 1e-30


def check(got, ref, bound, what, slack=1.0):
    """Every element within its bound; the worst ratio in the message."""
    e = (got.double() - ref).abs()
    ok = e <= slack * bound
    assert bool(ok.all()), (what, float((e / bound).nan_to_num(nan=float("inf")).max()),
                            int((~ok).sum()))


# ------------------------------------------------------------------- cache
def e4m3(y):
    """64-bit values to the nearest e4m3 number (|y| <= 448), ties to even."""
    _, e = torch.frexp(y.abs().clamp(min=2.0 ** -6))
    step = torch.exp2((e - 4).double())
    return torch.round(y / step) * step


def stored(x, fmt):
    """The values rows x [..., hd] have in a cache of the format, and scales."""
    x = x.double()
    if fmt in ("f32", "bf16"):
        return x.to({"f32": torch.float32, "bf16": torch.bfloat16}[fmt]).double(), None
    big = x.abs().amax(-1, keepdim=True)
    bad = ~torch.isfinite(x).all(-1, keepdim=True)
    if fmt == "int8":
        unit = (big / 127).float().double().clamp(min=2.0 ** -126)
        val = torch.round(x / unit) * unit
    else:
        e = torch.frexp(big / 448)  # mantissa in [1/2, 1), 64 bits: exact enough to compare
        e = torch.where(big > 448 * torch.exp2((e[1] - 1).double()), e[1], e[1] - 1)
        unit = torch.exp2(e.clamp(min=-126).double())
        unit = torch.where(big > 0, unit, torch.full_like(unit, 2.0 ** -126))
        val = e4m3(x / unit) * unit
    nan = torch.full((), math.nan, dtype=torch.float64, device=x.device)
    return torch.where(bad, nan, val), torch.where(bad, nan, unit)[..., 0]


def paged(q, pages, scales, table, lens, h, want):
    """out, lse and bounds of one token per sequence over its cached rows;
    positions whose page is outside the cache are left out.

    bfloat16 queries over an 8-bit cache: a key's weight times its v scale may
    be held in float16 (the codes fit it exactly), in units where the largest
    so far is 2^13 at least, of which 2^-25 is half the least step: each key is
    off by 2^-38 max_j(p_j scale_j) |code| at most beside the relative error,
    which matters where every weight but one is far below 2^-14 of the largest
    and that one's code is 0."""
    n_pages, _, g, ps, hd = pages.shape
    b = q.shape[0]
    x = pages.double() if scales is None else pages.double() * scales.double()[..., None]
    out = torch.zeros(b, h, hd, dtype=torch.float64, device=q.device)
    lse = torch.full((b, h), -math.inf, dtype=torch.float64, device=q.device)
    ob, lb = torch.zeros_like(out), torch.zeros_like(lse)
    qd = q.double().reshape(b, h, hd)
    r, ex = R[want], EXP[want]
    for s in range(b):
        n = min(max(lens[s], 0), table.shape[1] * ps)
        keep = [(int(table[s, t // ps]), t % ps) for t in range(n)]
        keep = [(p, t) for p, t in keep if 0 <= p < n_pages]
        if not keep:
            continue
        pi = torch.tensor([p for p, _ in keep], device=q.device)
        ti = torch.tensor([t for _, t in keep], device=q.device)
        kv = x[pi, :, :, ti]  # [m, 2, g, hd]
        m = len(keep)
        for i in range(h):
            k, v, z = kv[:, 0, i // (h // g)], kv[:, 1, i // (h // g)], qd[s, i]
            sc = k @ z / math.sqrt(hd)
            lse[s, i] = torch.logsumexp(sc, 0)
            p = torch.exp(sc - lse[s, i])
            out[s, i] = p @ v
            es = float(((hd + 5) * U * (k.abs() @ z.abs()) / math.sqrt(hd)
                        + 3 * U * sc.abs()).max())
            ob[s, i] = (2 * (es + ex) + (2 * m + 16) * U + r) * (p @ v.abs()) + \
                R[want] * out[s, i].abs()
            if scales is not None and want == torch.bfloat16:
                sv = scales[pi, 1, i // (h // g), ti].double()
                codes = pages[pi, 1, i // (h // g), ti].double().abs().sum(0)
                ob[s, i] += 2.0 ** -38 * float((p * sv).max()) * codes
            lb[s, i] = es + ex + (m + 8) * U + 4 * U * lse[s, i].abs()
    return out.reshape(b, -1), lse, ob.reshape(b, -1) + 1e-30, lb + 1e-30
