"""The 2-norm of lists of gradients against 64 bits.

Bound: a thread adds 64 squares in two chains of fused multiply-adds, 32 threads a tree of 5 and one
sum: 38 roundings of 2^-24 of the sum at most, half of it in the root, and the root's own: 1.2e-6."""
import numpy as np
import pytest
import torch

import dflash2_draft_head_gb300 as df2
from loss_rows import INF, NAN

pytestmark = pytest.mark.gpu
BOUND = 1.2e-6
KIND = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _built():
    df2.build_library()
    df2.lib()
    yield
    torch.cuda.synchronize()


def _lists(sizes, dtype, seed=0, offset=0, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    out = []
    for n in sizes:
        buf = torch.full((n + offset + 40,), NAN, dtype=KIND[dtype], device="cuda")
        t = buf[offset:offset + n]
        t.copy_(torch.randn(n, device="cuda", generator=g) * scale)
        out.append(t)
    return out


def _ref(ts):
    return float(np.sqrt(sum(float(t.double().square().sum()) for t in ts)))


def _check(ts, **kw):
    got = df2.grad_norm(ts, **kw)
    assert got.shape == (1,) and got.dtype == torch.float32
    want = _ref(ts)
    assert abs(got.item() - want) <= BOUND * want, (got.item(), want)
    return got


@pytest.mark.parametrize("offset", [0, 1, 3])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_sizes(dtype, offset):
    for sizes in ([1], [7], [0, 5, 0], [16383, 16384, 16385], [100003, 1, 33], [3_000_001],
                  [5] * 32, [5] * 33, [32 * 16384], [32 * 16384 + 1], [400_001, 7]):
        _check(_lists(sizes, dtype, sum(sizes), offset))


@pytest.mark.parametrize("count", [16, 17, 384, 385, 1000])
def test_numbers_of_tensors(count):
    rng = np.random.default_rng(count)
    _check(_lists([int(n) for n in rng.integers(0, 300, count)], "bf16"))


def test_shapes_and_no_elements():
    ts = [torch.randn(3, 4, 5, device="cuda"), torch.randn((), device="cuda")]
    _check(ts)
    assert df2.grad_norm([torch.empty(0, device="cuda")] * 3).item() == 0
    assert df2.grad_norm([torch.zeros(100000, device="cuda")]).item() == 0


@pytest.mark.parametrize("scale", [1e-40, 1e-30, 1e-21, 1e-13, 1e-10, 1e13, 1e17, 1e19, 1e30])
def test_squares_outside_fp32(scale):
    """From fp32's subnormal numbers (exact in both) with a norm that is a normal one, up to where
    the norm itself stays below 3.4e38."""
    _check(_lists([50000, 77], "f32", 3, scale=scale))
    mixed = _lists([20000], "f32", 4) + _lists([20000], "f32", 5, scale=scale)
    _check(mixed)


@pytest.mark.parametrize("bad", [NAN, INF, -INF])
def test_what_is_not_finite(bad):
    ts = _lists([20000, 50000, 3], "bf16")
    ts[1][40001] = bad
    got = df2.grad_norm(ts).item()
    assert np.isnan(got) if np.isnan(bad) else got == INF
    ts = [torch.full((1000,), 3e38, device="cuda")]      # the norm is beyond fp32
    assert df2.grad_norm(ts).item() == INF


def test_the_same_bits_every_time_and_given_outputs():
    ts = _lists([1_000_003, 77, 50000], "f32", 6)
    a = _check(ts)
    out = torch.full((1,), NAN, device="cuda")
    ws = torch.empty(4096, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        assert df2.grad_norm(ts, out=out, workspace=ws) is out
        assert torch.equal(a, out)


def test_two_streams_and_two_graphs_beside_one_another():
    """Each call has a workspace of its own."""
    lists = [_lists([1_500_000], "f32", k) for k in range(2)]
    want = [df2.grad_norm(ts) for ts in lists]
    streams = [torch.cuda.Stream() for _ in lists]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for k, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[k].append(df2.grad_norm(lists[k]))
    torch.cuda.synchronize()
    for k in range(2):
        assert all(torch.equal(want[k], x) for x in got[k])
    graphs, outs = [], []
    for ts in lists:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(df2.grad_norm(ts))
        graphs.append(graph)
    for _ in range(5):
        for graph, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, outs))


def test_refusals():
    g = torch.zeros(600000, device="cuda")
    for bad in [[], [g, g.bfloat16()], [g.half()], [g[::2]], [g.cpu()], [g, None]]:
        with pytest.raises((TypeError, ValueError)):
            df2.grad_norm(bad)
    with pytest.raises((TypeError, ValueError)):
        df2.grad_norm([g], out=torch.zeros(2, device="cuda"))
    for kw in [dict(workspace=torch.empty(8, dtype=torch.uint8, device="cuda")), dict(out=g[5:6])]:
        with pytest.raises(df2.Dflash2Error):
            df2.grad_norm([g], **kw)
