"""The package imports without a GPU and on a torch that was built without CUDA."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_import_on_a_torch_without_cuda():
    """Such a torch has none of the CUDA stream functions."""
    code = ("import torch\n"
            "for n in [n for n in dir(torch._C) if n.startswith('_cuda_getCurrent')]:\n"
            "    delattr(torch._C, n)\n"
            "import fp4_block_scaled_04_b200 as fq\n"
            "assert fq.fp4q_quantize_mxfp8 and fq.fp4q_dequantize\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
