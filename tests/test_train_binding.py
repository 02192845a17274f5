"""The Python binding of the training operators as far as it goes without a GPU: which device is
current at a call, and the lists of tensors that it takes."""
import contextlib
from types import SimpleNamespace

import pytest
import torch

from dflash2_draft_head_gb300 import binding


@pytest.mark.parametrize("current,index,switched", [(0, 0, []), (0, 1, [1]), (2, 0, [0])])
def test_the_tensors_device_is_current_at_the_call(monkeypatch, current, index, switched):
    """The library takes SMs and launches from the current device; the stream is the tensors'."""
    seen, inside = [], [current]

    @contextlib.contextmanager
    def device(k):
        seen.append(k)
        inside.append(k)
        yield
        inside.pop()

    monkeypatch.setattr(torch.cuda, "current_device", lambda: inside[-1])
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(binding, "_raw_stream", lambda k: 1000 + k)
    got = []

    def entry(*args):
        got.append((inside[-1], args))
        return 0

    binding._launch(index, entry, "a", 2)
    assert got == [(index, ("a", 2, 1000 + index))] and seen == switched


def test_a_failing_call_raises(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(binding, "_raw_stream", lambda k: 0)
    fake = SimpleNamespace(dflash2_status_string=lambda s: b"status", dflash2_last_error=lambda: b"why")
    monkeypatch.setattr(binding, "lib", lambda: fake)
    with pytest.raises(binding.Dflash2Error, match="status: why"):
        binding._launch(0, lambda *a: 2)


def test_inputs_on_another_device_are_refused():
    t = SimpleNamespace(dtype=torch.float32, get_device=lambda: 1, shape=(4,), is_cuda=True,
                        is_contiguous=lambda: True, data_ptr=lambda: 64, device="cuda:1")
    assert binding._on(t, "x", torch.float32, (4,), 1) == 64
    with pytest.raises(ValueError, match="x must be on device cuda:0"):
        binding._on(t, "x", torch.float32, (4,), 0)
    assert binding._on(None, "x", torch.float32, (4,), 0) is None


@pytest.mark.parametrize("lists", [
    dict(a=[torch.zeros(2)], b=[torch.zeros(2), torch.zeros(2)]), dict(a=[torch.zeros(2)], b=[]),
    dict(a=[torch.zeros(2)], b=[torch.zeros(2)]),
])
def test_lists_that_do_not_go_together(lists):
    with pytest.raises(ValueError):
        binding._Lists(**lists)


def test_what_is_no_tensor():
    with pytest.raises(TypeError):
        binding._Lists(a=[torch.zeros(2), None])
    with pytest.raises(TypeError):
        binding._Lists(a=[3.0])


@pytest.mark.parametrize("n,pairs", [(1, 0), (3, 1), (2001, 1000)])
def test_pairs(n, pairs):
    assert binding._pairs(torch.zeros(n, dtype=torch.int32)) == pairs


@pytest.mark.parametrize("shape", [(0,), (2,), (4,), (1, 3), ()])
def test_offsets_of_no_whole_pairs(shape):
    with pytest.raises(ValueError):
        binding._pairs(torch.zeros(shape, dtype=torch.int32))
