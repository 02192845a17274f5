"""The Python binding of the operators on vocabulary rows, as far as it goes without a GPU:
what it needs of torch when it is imported, and the row layouts that it takes."""
import ctypes
import os
import subprocess
import sys
from types import SimpleNamespace

import pytest
import torch

from dflash2_draft_head_gb300 import binding

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


def _fake(shape, stride):
    return SimpleNamespace(is_cuda=True, shape=torch.Size(shape), stride=lambda: stride)


@pytest.mark.parametrize("shape", [(0, 8), (5, 0, 8), (0, 5, 8), (5, 0, 3, 8), (2, 3, 0, 8), (0, 0, 8)])
def test_no_rows_in_any_leading_dimension(shape):
    t = torch.empty(shape)
    lead, rows, V, ld = binding._logit_rows(_fake(shape, t.stride()), "logits")
    assert (tuple(lead), rows, V) == (shape[:-1], 0, 8) and ld >= 8


@pytest.mark.parametrize("shape,stride,want", [
    ((4, 100), (104, 1), (4, 100, 104)), ((2, 3, 100), (312, 104, 1), (6, 100, 104)),
    ((1, 100), (7, 1), (1, 100, 100)), ((2, 1, 100), (104, 5, 1), (2, 100, 104)),
    ((100,), (1,), (1, 100, 100)),
])
def test_evenly_spaced_rows(shape, stride, want):
    assert binding._logit_rows(_fake(shape, stride), "logits")[1:] == want


def test_uneven_rows_are_refused():
    with pytest.raises(ValueError):
        binding._logit_rows(_fake((2, 3, 100), (400, 104, 1)), "logits")


class _Tensor(SimpleNamespace):
    """As much of a CUDA tensor as sample() looks at."""

    def data_ptr(self):
        return 1 << 20

    def is_contiguous(self):
        return True


@pytest.mark.parametrize("top_k,limit", [
    (0, None), (-1, None), (5, 5), (2 ** 21 - 1, 2 ** 21 - 1), (2 ** 31 - 1, None), (2 ** 31, None),
    (2 ** 32 + 5, None), (sys.maxsize, None), (-2 ** 32 + 5, None),
])
def test_a_top_k_beyond_32_bits_is_no_limit(monkeypatch, top_k, limit):
    """The C entry takes 32 bits: a number beyond them must not come out as a small one.  No
    row has more than 2^21 entries."""
    got = []

    def entry(*args):
        got.append(ctypes.c_int(args[8]).value)
        return 0

    rows, dev = torch.Size((2,)), SimpleNamespace(index=0)
    x = _Tensor(is_cuda=True, dtype=torch.float32, shape=torch.Size((2, 8)), stride=lambda: (8, 1),
                device=dev)
    u = _Tensor(is_cuda=True, dtype=torch.float32, shape=rows, device=dev)
    tok = _Tensor(is_cuda=True, dtype=torch.int32, shape=rows, device=dev)
    monkeypatch.setattr(binding, "lib", lambda: SimpleNamespace(dflash2_sample=entry))
    monkeypatch.setattr(binding, "_raw_stream", lambda i: 0)
    binding.sample(x, u, top_k=top_k, tokens=tok, probs=u)
    assert (got[0] if 0 < got[0] < 2 ** 21 else None) == limit
