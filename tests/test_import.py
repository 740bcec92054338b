"""The package imports, and its host calls work, where torch lacks the CUDA
entries (no GPU)."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_import_with_a_torch_built_without_cuda():
    code = ("import torch\n"
            "for n in [n for n in dir(torch._C) if n.startswith('_cuda_')]:\n"
            "    delattr(torch._C, n)\n"
            "import scratch_llama_decoder_b200 as P\n"
            "cfg = dict(vocab=64, d_model=64, n_layer=1, n_head=2, n_kv_head=1, d_ff=128, ctx=16,\n"
            "           batch=1)\n"
            "assert P.llm_workspace_bytes(cfg) > 0\n"
            "try:\n"
            "    P.attention_packed(torch.zeros(1, 96), torch.zeros(2, dtype=torch.int32), 1, 1)\n"
            "except ValueError:\n"
            "    print('refused')\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    assert r.stdout == "refused\n"
