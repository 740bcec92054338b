"""The host's test of overlapping rows against sets of bytes (no GPU), and the
refusal of a gradient array that overlaps an input."""
import ctypes as C
import os
import random
import shutil
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SHIM = """
#include "overlap.h"
extern "C" int one(uintptr_t p, int64_t ld, int64_t w, int64_t n, uintptr_t q, int64_t len) {
  return llm::overlap(p, ld, w, n, q, len);
}
extern "C" int two(uintptr_t a, int64_t ld, uintptr_t b, int64_t ld2, int64_t w, int64_t n) {
  return llm::rows_overlap((void *)a, ld, (void *)b, ld2, w, n);
}
"""


def test_overlap_against_byte_sets(tmp_path):
    if not shutil.which("g++"):
        pytest.skip("g++ not available")
    (tmp_path / "shim.cc").write_text(SHIM)
    so = str(tmp_path / "shim.so")
    subprocess.run(["g++", "-shared", "-fPIC", "-O1", "-I",
                    os.path.join(ROOT, "scratch_llama_decoder_b200", "csrc"), "-o", so,
                    str(tmp_path / "shim.cc")], check=True)
    lib = C.CDLL(so)
    lib.one.argtypes = [C.c_size_t, C.c_int64, C.c_int64, C.c_int64, C.c_size_t, C.c_int64]
    lib.two.argtypes = [C.c_size_t, C.c_int64, C.c_size_t, C.c_int64, C.c_int64, C.c_int64]
    rng = random.Random(1)
    seen = set()
    for _ in range(20000):
        n, w, ln = rng.randrange(1, 6), rng.randrange(1, 12), rng.randrange(1, 30)
        ld = w + rng.randrange(0, 15)
        ld2 = ld if rng.random() < 0.6 else w + rng.randrange(0, 15)
        p = 1 << 40
        q = p + rng.randrange(-90, 130)
        a = {p + r * ld + c for r in range(n) for c in range(w)}
        want = bool(a & set(range(q, q + ln)))
        assert bool(lib.one(p, ld, w, n, q, ln)) == want, (ld, w, n, q - p, ln)
        both = bool(a & {q + r * ld2 + c for r in range(n) for c in range(w)})
        assert bool(lib.two(p, ld, q, ld2, w, n)) == both, (ld, ld2, w, n, q - p)
        seen.add((want, both, ld == ld2))
    assert len(seen) == 8


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_gradient_that_overlaps_an_input_is_refused(dtype):
    """Rows that interleave are taken, rows that share an element are not."""
    import scratch_llama_decoder_b200 as P
    h, g, hd, n = 2, 1, 32, 50
    w = (h + 2 * g) * hd
    store = torch.randn(n, 2 * w + 8, device="cuda").to(dtype)
    qkv = store[:, :w]
    cu = torch.tensor([0, 20, n], dtype=torch.int32, device="cuda")
    out, lse = P.attention_packed(qkv, cu, h, g)
    dout = torch.randn(n, h * hd, device="cuda").to(dtype)
    want = P.attention_packed_backward(qkv, cu, h, g, out, lse, dout)
    for off in (0, 1, w - 1, w // 2):
        with pytest.raises(P.LLMError):
            P.attention_packed_backward(qkv, cu, h, g, out, lse, dout, dqkv=store[:, off:off + w])
    before = store[:, :w].clone()
    got = P.attention_packed_backward(qkv, cu, h, g, out, lse, dout, dqkv=store[:, w + 8:])
    assert torch.equal(got, want) and torch.equal(store[:, :w], before)
    flat = torch.empty(n * (h * hd + w), device="cuda").to(dtype)
    o2 = flat[:n * h * hd].view(n, h * hd)
    o2.copy_(out)
    for at, ok in ((n * h * hd, True), (n * h * hd - 1, False), (0, False)):
        dx = flat[at:at + n * w].view(n, w)
        if ok:
            P.attention_packed_backward(qkv, cu, h, g, o2, lse, dout, dqkv=dx)
            assert torch.equal(o2, out)
            continue
        for o, d in ((o2, dout), (out, o2)):
            with pytest.raises(P.LLMError):
                P.attention_packed_backward(qkv, cu, h, g, o, lse, d, dqkv=dx)
