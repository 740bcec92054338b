"""Operators over sequences of different lengths, as they are measured.

Packed causal attention (a batch of prompts or documents laid end to end, with
its gradient), a paged key/value cache (written, quantised where its type is an
8-bit one, and read back) and the attention of one new token over that cache.
`run` computes each in its plain form (elementary torch operations in 32 bits)
or, where `own` is true, through the framework's kernels; `exact` gives the
same outputs from the definition in 64 bits.
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------- cases
def _lens(case):
    """Sequence lengths of a case: fixed by the case, so that its work is."""
    r = random.Random(case["lens_seed"])
    n = case["n_seq"]
    if case["op"] == "decode":  # spread over their logarithm up to the longest
        top = case["max_len"]
        got = [int(math.exp(r.uniform(math.log(max(1, top // 64)), math.log(top + 1))))
               for _ in range(n)]
        got[r.randrange(n)] = top
        if case["idle"]:  # slots of the batch that hold no request
            got[r.randrange(n)] = 0 if n > 1 else top
        return [min(x, top) for x in got]
    if case["rows"] == n:  # one new token of every request
        return [1] * n
    w = [r.expovariate(1.0) + 0.05 for _ in range(n)]
    got = [int(case["rows"] * x / sum(w)) for x in w]
    got[r.randrange(n)] += case["rows"] - sum(got)
    return got


def listed():
    att = dict(page_size=0, kv="", idle=False, max_len=0)
    pre = dict(att, op="prefill", dtype="bf16")
    trn = dict(att, op="train")
    cache = dict(op="cache", idle=False, max_len=0)
    dec = dict(op="decode", rows=0, dtype="bf16")
    return [
        # one short prompt of a chat turn: latency
        dict(pre, name="prefill short prompt", n_head=8, n_kv_head=2, head_dim=64, n_seq=1,
             rows=17, lens_seed=1),
        # a server's batch of prompts of different lengths, the 350M decoder's heads
        dict(pre, name="prefill ragged batch", n_head=16, n_kv_head=16, head_dim=64, n_seq=24,
             rows=16001, lens_seed=2),
        # two long documents, grouped heads
        dict(pre, name="prefill long documents", n_head=8, n_kv_head=2, head_dim=64, n_seq=2,
             rows=16384, lens_seed=5),
        # a training batch of packed documents: 8 x 2048 tokens of the 350M decoder
        dict(trn, name="train packed 350m", dtype="bf16", n_head=16, n_kv_head=16, head_dim=64,
             n_seq=40, rows=16384, lens_seed=4),
        # the 6-layer decoder's batch, 64 x 256 tokens, documents of about 128 tokens
        dict(trn, name="train packed head 32", dtype="bf16", n_head=8, n_kv_head=8, head_dim=32,
             n_seq=128, rows=16384, lens_seed=6),
        # the same in float32: the 8-layer float32 decoder
        dict(trn, name="train packed float32", dtype="f32", n_head=4, n_kv_head=4, head_dim=32,
             n_seq=64, rows=16384, lens_seed=7),
        # prompts written to an 8-bit float cache and read back
        dict(cache, name="cache e4m3 prompts", dtype="bf16", kv="e4m3", n_head=16, n_kv_head=16,
             head_dim=64, n_seq=24, rows=16001, page_size=64, lens_seed=8),
        # the new tokens of a decode batch, 8-bit integer cache: latency
        dict(cache, name="cache int8 new tokens", dtype="bf16", kv="int8", n_head=8, n_kv_head=2,
             head_dim=64, n_seq=33, rows=33, page_size=16, lens_seed=9),
        # one request early in its answer: latency
        dict(dec, name="decode one short", kv="bf16", n_head=8, n_kv_head=2, head_dim=64, n_seq=1,
             max_len=200, page_size=16, idle=False, lens_seed=10),
        # a batch of the grouped-head decoder within its context
        dict(dec, name="decode batch int8", kv="int8", n_head=8, n_kv_head=2, head_dim=64,
             n_seq=32, max_len=512, page_size=16, idle=True, lens_seed=11),
        # a large ragged batch with an 8-bit float cache
        dict(dec, name="decode ragged e4m3", kv="e4m3", n_head=16, n_kv_head=16, head_dim=64,
             n_seq=32, max_len=16384, page_size=64, idle=False, lens_seed=12),
        # one very long context, split over its length
        dict(dec, name="decode one long", kv="bf16", n_head=16, n_kv_head=16, head_dim=64,
             n_seq=1, max_len=100001, page_size=64, idle=False, lens_seed=13),
    ]


def _most(op):
    got = [work(c) for c in listed() if c["op"] == op]
    return max(g["bytes"] for g in got), max(g["flops"] for g in got)


def draw(rng):
    def log(lo, hi):
        return int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))

    while True:
        op = rng.choice(["prefill", "train", "cache", "decode"])
        h, g = rng.choice([(4, 4), (8, 8), (8, 2), (16, 16), (16, 4), (12, 4), (4, 1), (8, 1)])
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        c = dict(op=op, dtype=dtype, n_head=h, n_kv_head=g, head_dim=rng.choice([32, 64, 64, 128]),
                 lens_seed=rng.randrange(1 << 20), idle=False, max_len=0, page_size=0, kv="", rows=0)
        if op in ("prefill", "train"):
            c["n_seq"] = log(1, 128)
            c["rows"] = max(c["n_seq"], log(16, 16384))
        else:
            c["kv"] = rng.choice([dtype, "e4m3", "int8"])
            c["page_size"] = rng.choice([8, 16, 32, 64, 128])
            c["n_seq"] = log(1, 64)
            if op == "cache":
                c["rows"] = max(c["n_seq"], log(1, 16384))
            else:
                c["max_len"] = log(16, 100000)
                c["idle"] = rng.random() < 0.3 and c["n_seq"] > 1
        w, top = work(c), _most(op)
        f = 8 if dtype == "f32" and op != "cache" else 1  # float32 runs off the tensor cores
        if c["n_seq"] * c["max_len"] * g * c["head_dim"] > 6e8:
            continue  # the plain form lays all caches out to the longest one's length
        if w["bytes"] <= top[0] and w["flops"] * f <= max(top[1], 1):
            return c


def work(case):
    lens = _lens(case)
    h, g, hd = case["n_head"], case["n_kv_head"], case["head_dim"]
    b = 2 if case["dtype"] == "bf16" else 4
    if case["op"] in ("prefill", "train"):
        rows, pairs = sum(lens), sum(n * (n + 1) // 2 for n in lens)
        qkv, o, lse = rows * (h + 2 * g) * hd * b, rows * h * hd * b, rows * h * 4
        if case["op"] == "prefill":
            return {"bytes": qkv + o + lse, "flops": 4.0 * hd * pairs * h}
        # forward, then the gradient of q|k|v from that of the output
        return {"bytes": 2 * qkv + 2 * o + lse, "flops": 12.0 * hd * pairs * h}
    e, s = {"f32": (4, 0), "bf16": (2, 0), "e4m3": (1, 4), "int8": (1, 4)}[case["kv"]]
    if case["op"] == "cache":
        n = sum(lens) * 2 * g
        return {"bytes": n * (hd * b + 2 * (hd * e + s) + hd * b), "flops": 0.0}
    return {"bytes": sum(lens) * 2 * g * (hd * e + s) + case["n_seq"] * h * (2 * hd * b + 4),
            "flops": 4.0 * hd * sum(lens) * h}


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dt, dev = DT[case["dtype"]], "cuda"
    h, g, hd = case["n_head"], case["n_kv_head"], case["head_dim"]
    lens = _lens(case)
    st = dict(case=case, lens=lens)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    if case["op"] in ("prefill", "train", "cache"):
        rows = sum(lens)
        x = normal(rows, h + 2 * g, hd)
        if case["op"] == "cache":  # heads and positions of different sizes, as keys have
            x = x * torch.exp(normal(rows, h + 2 * g, 1))
        st["qkv"] = x.to(dt).reshape(rows, -1)
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        st["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev)
        if case["op"] == "train":
            st["dout"] = normal(rows, h * hd).to(dt)
    if case["op"] in ("cache", "decode"):
        ps = case["page_size"]
        # the cache holds earlier positions already where new tokens are written
        starts = [(7 * i * i + 3 * i) % (3 * ps) for i in range(len(lens))]
        starts = starts if case["op"] == "cache" else [0] * len(lens)
        need = [-(-(a + n) // ps) for a, n in zip(starts, lens)]
        n_pages = sum(need) + 3
        order = torch.randperm(n_pages, generator=gen, device=dev).to(torch.int32)
        cols = torch.arange(max(max(need), 1), device=dev)
        first = torch.tensor([sum(need[:i]) for i in range(len(need))], device=dev)
        used = cols[None] < torch.tensor(need, device=dev)[:, None]
        at = (first[:, None] + cols[None]).clamp(max=n_pages - 1)
        st["table"] = torch.where(used, order[at], torch.full_like(order[at], -1)).contiguous()
        st["starts"] = torch.tensor(starts, dtype=torch.int32, device=dev)
        shape = (n_pages, 2, g, ps, hd)
        st["scales"] = None
        if case["kv"] in ("e4m3", "int8"):
            st["scales"] = torch.exp2(torch.round(normal(*shape[:4]))) / 64
        if case["kv"] == "int8":
            st["pages"] = (normal(*shape) * 42).round().clamp(-127, 127).to(torch.int8)
            st["scales"] = st["scales"] * (1 + 0.3 * torch.rand(*shape[:4], generator=gen,
                                                                device=dev))
        elif case["kv"] == "e4m3":
            st["pages"] = (normal(*shape) * 64).clamp(-448, 448).to(torch.float8_e4m3fn)
        else:
            st["pages"] = normal(*shape).to(DT[case["kv"]])
        if case["op"] == "decode":
            st["q"] = normal(len(lens), h * hd).to(dt)
            st["kv_lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    return st


# ------------------------------------------------------------- plain forms
def _attend(q, k, v):
    """One sequence: q [n, H, hd], k and v [n, H, hd] in 32 bits -> o, lse, p."""
    n, hd = q.shape[0], q.shape[2]
    s = torch.matmul(q.transpose(0, 1), k.permute(1, 2, 0)) * (1.0 / math.sqrt(hd))
    i = torch.arange(n, device=q.device)
    s = s.masked_fill(i[None, :] > i[:, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - m)
    l = p.sum(-1, keepdim=True)
    p = p / l
    o = torch.matmul(p, v.transpose(0, 1)).transpose(0, 1)
    return o, (m + torch.log(l))[..., 0], p


def _plain_packed(st):
    c = st["case"]
    h, g, hd, dt = c["n_head"], c["n_kv_head"], c["head_dim"], DT[c["dtype"]]
    rep = h // g
    x = st["qkv"].float().view(-1, h + 2 * g, hd)
    outs, lses, grads, a = [], [], [], 0
    for n in st["lens"]:
        q, k, v = (t.repeat_interleave(r, 1) if r > 1 else t
                   for t, r in zip(x[a:a + n].split([h, g, g], 1), (1, rep, rep)))
        if n == 0:
            continue
        o, lse, p = _attend(q, k, v)
        outs.append(o.reshape(n, -1))
        lses.append(lse)
        if c["op"] == "train":
            do = st["dout"][a:a + n].float().view(n, h, hd)
            dv = torch.matmul(p.transpose(1, 2), do.transpose(0, 1))
            dp = torch.matmul(do.transpose(0, 1), v.permute(1, 2, 0))
            ds = p * (dp - (do * o).sum(-1).t()[..., None]) * (1.0 / math.sqrt(hd))
            dq = torch.matmul(ds, k.transpose(0, 1))
            dk = torch.matmul(ds.transpose(1, 2), q.transpose(0, 1))
            dk, dv = (t.view(g, rep, n, hd).sum(1) for t in (dk, dv))
            grads.append(torch.cat([dq, dk, dv], 0).transpose(0, 1).reshape(n, -1))
        a += n
    got = {"out": torch.cat(outs).to(dt), "lse": torch.cat(lses, 1)}
    if c["op"] == "train":
        got["dqkv"] = torch.cat(grads).to(dt)
    return got


def _quantise(x, kv):
    """x [..., hd] in 32 bits -> codes and scales, and the values they stand for."""
    amax = x.abs().amax(-1, keepdim=True)
    if kv == "e4m3":  # the least power of two that brings the largest within 448
        frac, e = torch.frexp(amax / 448)
        e = torch.where(frac > 0.5, e, e - 1).clamp(-126, 127)
        scale = torch.ldexp(torch.ones_like(amax), e)
        return (x / scale).to(torch.float8_e4m3fn), scale[..., 0]
    scale = (amax / 127).clamp(min=torch.finfo(torch.float32).tiny)
    # the quotient in 64 bits: values next to a border between two codes
    return torch.round(x.double() / scale.double()).to(torch.int8), scale[..., 0]


def _places(st):
    """(page, row in the page) of every packed row."""
    c = st["case"]
    n = torch.tensor(st["lens"], device="cuda")
    seq = torch.repeat_interleave(torch.arange(len(st["lens"]), device="cuda"), n)
    pos = torch.arange(len(seq), device="cuda") - st["cu"].long()[seq] + st["starts"].long()[seq]
    return st["table"][seq, pos // c["page_size"]].long(), pos % c["page_size"]


def _plain_cache(st):
    c = st["case"]
    h, g, hd, dt = c["n_head"], c["n_kv_head"], c["head_dim"], DT[c["dtype"]]
    kv = st["qkv"].view(-1, h + 2 * g, hd)[:, h:].float().view(-1, 2, g, hd)
    page, row = _places(st)
    if st["scales"] is None:
        st["pages"][page, :, :, row] = kv.to(st["pages"].dtype)
        back = st["pages"][page, :, :, row].float()
    else:
        codes, scale = _quantise(kv, c["kv"])
        st["pages"].view(torch.int8)[page, :, :, row] = codes.view(torch.int8)
        st["scales"][page, :, :, row] = scale
        back = st["pages"].view(torch.int8)[page, :, :, row].view(st["pages"].dtype).float()
        back = back * st["scales"][page, :, :, row][..., None]
    return {"k": back[:, 0].to(dt), "v": back[:, 1].to(dt)}


def _plain_decode(st):
    c = st["case"]
    h, g, hd, dt = c["n_head"], c["n_kv_head"], c["head_dim"], DT[c["dtype"]]
    b, table, ps = c["n_seq"], st["table"], c["page_size"]
    at = table.long().clamp(min=0)
    n = at.shape[1] * ps

    def rows(kv):  # [b, g, n, hd] of every sequence's pages
        x = st["pages"][:, kv]
        x = (x.view(torch.int8)[at].view(x.dtype) if st["scales"] is not None else x[at]).float()
        if st["scales"] is not None:
            x = x * st["scales"][:, kv][at][..., None]
        return x.permute(0, 2, 1, 3, 4).reshape(b, g, n, hd)

    live = torch.arange(n, device="cuda")[None] < st["kv_lens"][:, None]
    q = st["q"].float().view(b, g, h // g, hd)
    s = torch.matmul(q, rows(0).transpose(2, 3)) * (1.0 / math.sqrt(hd))
    s = s.masked_fill(~live[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - m.clamp(min=torch.finfo(torch.float32).min))
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p, rows(1)) / l.clamp(min=torch.finfo(torch.float32).tiny)
    return {"out": o.reshape(b, h * hd).to(dt), "lse": (m + torch.log(l)).view(b, h)}


def run(state):
    c = state["case"]
    h, g = c["n_head"], c["n_kv_head"]
    if own:
        import scratch_llama_decoder_b200 as P
        if c["op"] in ("prefill", "train"):
            out, lse = P.attention_packed(state["qkv"], state["cu"], h, g)
            got = {"out": out, "lse": lse}
            if c["op"] == "train":
                got["dqkv"] = P.attention_packed_backward(state["qkv"], state["cu"], h, g, out,
                                                          lse, state["dout"])
            return got
        if c["op"] == "cache":
            P.kv_write(state["qkv"], state["cu"], h, state["pages"], state["table"],
                       scales=state["scales"], starts=state["starts"])
            k, v = P.kv_read(state["pages"], state["table"], state["cu"],
                             state["qkv"].shape[0], state["qkv"].dtype, scales=state["scales"],
                             starts=state["starts"])
            return {"k": k, "v": v}
        out, lse = P.attention_paged(state["q"], state["pages"], state["table"],
                                     state["kv_lens"], scales=state["scales"])
        return {"out": out, "lse": lse}
    if c["op"] in ("prefill", "train"):
        return _plain_packed(state)
    return _plain_cache(state) if c["op"] == "cache" else _plain_decode(state)


# ------------------------------------------------------------ the definition
def exact(case, seed):
    st = prepare(case, seed)
    h, g, hd = case["n_head"], case["n_kv_head"], case["head_dim"]
    rep, root, lens = h // g, math.sqrt(hd), st["lens"]
    if case["op"] in ("prefill", "train"):
        rows = sum(lens)
        x = st["qkv"].double().view(rows, -1, hd)
        out = torch.zeros(rows, h, hd, dtype=torch.float64, device="cuda")
        lse = torch.zeros(h, rows, dtype=torch.float64, device="cuda")
        grad = torch.zeros_like(x)
        for s in range(len(lens)):
            a, b = int(st["cu"][s]), int(st["cu"][s + 1])
            keep = torch.ones(b - a, b - a, dtype=torch.bool, device="cuda").tril()
            for i in range(h if b > a else 0):
                q, k, v = x[a:b, i], x[a:b, h + i // rep], x[a:b, h + g + i // rep]
                z = torch.where(keep, q @ k.t() / root, torch.full((), -math.inf,
                                                                   dtype=torch.float64,
                                                                   device="cuda"))
                lse[i, a:b] = torch.logsumexp(z, 1)
                w = torch.exp(z - lse[i, a:b, None])
                out[a:b, i] = w @ v
                if case["op"] == "train":
                    do = st["dout"][a:b].double().view(b - a, h, hd)[:, i]
                    dw = do @ v.t()
                    dz = w * (dw - (w * dw).sum(1, keepdim=True)) / root
                    grad[a:b, i] = dz @ k
                    grad[a:b, h + i // rep] += dz.t() @ q
                    grad[a:b, h + g + i // rep] += w.t() @ do
        got = {"out": out.view(rows, -1), "lse": lse}
        if case["op"] == "train":
            got["dqkv"] = grad.view(rows, -1)
        return got
    if case["op"] == "cache":
        x = st["qkv"].double().view(-1, h + 2 * g, hd)
        k, v = x[:, h:h + g], x[:, h + g:]
        return {"k": _stored(k, case["kv"]), "v": _stored(v, case["kv"])}
    out = torch.zeros(len(lens), h, hd, dtype=torch.float64, device="cuda")
    lse = torch.full((len(lens), h), -math.inf, dtype=torch.float64, device="cuda")
    q = st["q"].double().view(-1, h, hd)
    for s, n in enumerate(lens):
        if n == 0:
            continue
        used = st["table"][s, :-(-n // case["page_size"])].tolist()
        kv = torch.cat([st["pages"][p].double() * (1.0 if st["scales"] is None else
                                                   st["scales"][p].double()[..., None])
                        for p in used], 2)[:, :, :n]
        for i in range(h):
            z = kv[0, i // rep] @ q[s, i] / root
            lse[s, i] = torch.logsumexp(z, 0)
            out[s, i] = torch.exp(z - lse[s, i]) @ kv[1, i // rep]
    return {"out": out.view(len(lens), -1), "lse": lse}


def _stored(x, kv):
    """The values an array of 64-bit rows [..., hd] has after its cache."""
    if kv in ("bf16", "f32"):
        return x.to(DT[kv]).double()
    big = x.abs().amax(-1, keepdim=True)
    if kv == "int8":
        unit = (big / 127).float().double().clamp(min=2.0 ** -126)
        return torch.round(x / unit) * unit
    unit = torch.exp2(torch.ceil(torch.log2(big / 448)).clamp(-126, 127))
    y = x / unit
    # e4m3: steps of 2^(e - 3) within a binade [2^e, 2^(e+1)), of 2^-9 below 2^-6
    _, e = torch.frexp(y.abs().clamp(min=2.0 ** -6))
    step = torch.exp2((e - 4).double())
    return torch.round(y / step) * step * unit
