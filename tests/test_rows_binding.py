"""The Python binding of the operators on vocabulary rows, as far as it goes without a GPU."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_import_on_a_torch_without_cuda():
    """A torch built without CUDA has none of the CUDA functions of its private module."""
    code = ("import torch\n"
            "for n in [n for n in dir(torch._C) if n.startswith('_cuda')]:\n"
            "    delattr(torch._C, n)\n"
            "import dflash2_draft_head_gb300 as df2\n"
            "assert df2.sample and df2.distill and df2.topk\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
