"""The binding is imported where torch has no CUDA: its parameter blocks and checks need none."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_import_without_cuda_functions():
    code = ("import torch\n"
            "if hasattr(torch._C, '_cuda_getCurrentRawStream'): del torch._C._cuda_getCurrentRawStream\n"
            "from speculative_decoding_draft_bf16_gb300 import dtree\n"
            "print(dtree.Params(mode='ddtree', batch=1, L=4, V=64, dtype='bf16', K=4, B=8).mode)\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
