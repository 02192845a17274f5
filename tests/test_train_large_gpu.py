"""The operators of training on arrays whose offsets pass 32 bits, and on tensors of inference
mode."""
import pytest
import torch

import dflash2_draft_head_gb300 as df2
from loss_rows import equal_bits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    df2.build_library()
    df2.lib()
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    assert df2.take_device_faults() == 0


def test_rows_beyond_32_bits():
    """40000 x 151936 bf16 (12 GB): rows at the front, in the middle and at the end against the same
    rows in a batch that is split alike (lse, logp and gradient do not depend on the others)."""
    rows, V = 40000, 151936
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    z = torch.empty((rows, V), dtype=torch.bfloat16, device="cuda")
    for lo in range(0, rows, 4000):
        z[lo:lo + 4000].normal_(generator=g)
    tokens = torch.randint(0, V, (rows,), device="cuda", generator=g).to(torch.int32)
    old = torch.full((rows,), -12.0, device="cuda")
    A = torch.randn(rows, device="cuda", generator=g)
    pick = torch.tensor([0, 1, 14133, 14134, 28269, rows - 1], device="cuda")
    few = z[pick].repeat(1000, 1)
    loss, logp, lse, grad = df2.policy_loss(z, tokens, old, A, grad=True)
    part = df2.policy_loss(few, tokens[pick].repeat(1000), old[:6000].contiguous(),
                           A[pick].repeat(1000), grad=True)
    for whole, small in zip((loss, logp, lse, grad), part):
        assert equal_bits(whole[pick], small[-6:])
    del grad, few, part
    offsets = torch.tensor([0, rows // 2, rows], dtype=torch.int32, device="cuda")
    df2.preference_loss(z, tokens, offsets, grad=z)
    assert torch.isfinite(z[pick].float()).all()
    at = z[pick].float().gather(1, tokens[pick].long()[:, None]).squeeze(1)
    sign = torch.where(pick < rows // 2, -1.0, 1.0)  # up for the chosen sequence's tokens
    assert torch.equal(torch.sign(at), sign)


def test_a_tensor_beyond_32_bits():
    """2^32 + 4133 bf16 weights with 8-bit states (26 GB): the first and the last ones against the
    same elements in a tensor of their own, all rounded to the nearest (chance goes by place)."""
    n, tail = 2 ** 32 + 4133, 8192 + 4133
    start = n - tail                              # a multiple of the block of 32
    assert start % 32 == 0
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    p, grad = (torch.zeros(n, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    m, v = (torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in range(2))
    ms, vs = (torch.zeros((n + 31) // 32, dtype=torch.uint8, device="cuda") for _ in range(2))
    for part in (slice(0, tail), slice(start, n)):
        p[part].normal_(generator=g)
        grad[part].normal_(generator=g)
    norm = df2.grad_norm([grad])
    want = (grad[:tail].double().square().sum() + grad[start:].double().square().sum()).sqrt()
    assert abs(norm.item() - want.item()) <= 1.2e-6 * want.item()
    kw = dict(step=1, lr=1e-2, norm=norm, max_norm=1.0)
    small = []
    for lo in (0, start):
        one = [t[lo:lo + tail].clone() for t in (p, grad, m, v)]
        one += [torch.zeros((tail + 31) // 32, dtype=torch.uint8, device="cuda") for _ in range(2)]
        df2.adamw([one[0]], [one[1]], [one[2]], [one[3]], exp_avg_scale=[one[4]],
                  exp_avg_sq_scale=[one[5]], **kw)
        small.append(one)
    df2.adamw([p], [grad], [m], [v], exp_avg_scale=[ms], exp_avg_sq_scale=[vs], **kw)
    for one, lo in zip(small, (0, start)):
        for whole, part in zip((p, m, v), (one[0], one[2], one[3])):
            assert torch.equal(whole[lo:lo + tail], part)
        assert torch.equal(ms[lo // 32:(lo + tail + 31) // 32], one[4])
        assert torch.equal(vs[lo // 32:(lo + tail + 31) // 32], one[5])
    assert not p[2 ** 31:2 ** 31 + 100].any()
    # by chance: places 2^32 apart draw other numbers
    same = torch.full((4096,), 1.001, device="cuda").bfloat16()
    for lo in (0, 2 ** 32):
        p[lo:lo + 4096] = same
        grad[lo:lo + 4096] = 1.0
    df2.adamw([p], [grad], [m], [v], exp_avg_scale=[ms], exp_avg_sq_scale=[vs], step=2, lr=1e-3,
              seed=3)
    assert not torch.equal(p[:4096], p[2 ** 32:2 ** 32 + 4096])
    values = df2.state_decode(m, ms, dtype=torch.bfloat16)
    assert torch.equal(values[start:], df2.state_decode(m[start:].contiguous(), ms[start // 32:],
                                                        dtype=torch.bfloat16))


def test_tensors_of_inference_mode_are_taken():
    with torch.inference_mode():
        z = torch.randn(6, 500, device="cuda")
        tokens = torch.arange(6, dtype=torch.int32, device="cuda")
        f = torch.zeros(6, device="cuda")
        offsets = torch.tensor([0, 3, 6], dtype=torch.int32, device="cuda")
        want = df2.policy_loss(z, tokens, f, f + 1, grad=True)[3]
        y = z.clone()
        assert torch.equal(df2.policy_loss(y, tokens, f, f + 1, grad=y)[3], want)
        want = df2.preference_loss(z, tokens, offsets, grad=True)[4]
        y = z.clone()
        assert torch.equal(df2.preference_loss(y, tokens, offsets, grad=y)[4], want)
        p, m, v = (torch.zeros_like(z) for _ in range(3))
        df2.adamw([p], [want], [m], [v], step=1, lr=1e-3, norm=df2.grad_norm([want]))
        assert p.any() and m.any()
