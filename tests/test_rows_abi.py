"""Host-side argument checks of the operators on vocabulary rows (CPU only: every call
here is refused before any CUDA work, or has no rows and so launches nothing)."""
import ctypes

import pytest

from dflash2_draft_head_gb300 import binding, build_library


@pytest.fixture(scope="module")
def L():
    build_library()
    return binding.lib()


# fake addresses far apart: passed only to calls that launch nothing
P = [0x10000000 * (k + 1) for k in range(16)]
NAN, INF = float("nan"), float("inf")


def _sample(L, lg=P[0], ld=100, u=P[1], T=None, k=None, p=None, mp=None, t0=1.0, k0=0, p0=1.0,
            m0=0.0, rows=4, V=100, dt=0, tok=P[6], pr=P[7]):
    return L.dflash2_sample(lg, ld, u, T, k, p, mp, t0, k0, p0, m0, rows, V, dt, tok, pr, None)


@pytest.mark.parametrize("kw,code", [
    (dict(lg=None), 1), (dict(u=None), 1), (dict(tok=None), 1), (dict(rows=-1), 1), (dict(V=0), 1),
    (dict(dt=2), 1), (dict(ld=99), 1), (dict(ld=0), 1), (dict(lg=P[0] + 2), 1),
    (dict(lg=P[0] + 1, dt=1), 1), (dict(u=P[1] + 2), 1), (dict(T=P[2] + 1), 1),
    (dict(k=P[3] + 2), 1), (dict(p=P[4] + 3), 1), (dict(mp=P[5] + 2), 1), (dict(tok=P[6] + 1), 1),
    (dict(pr=P[7] + 2), 1), (dict(t0=-0.5), 1), (dict(t0=NAN), 1), (dict(p0=NAN), 1),
    (dict(m0=NAN), 1), (dict(tok=P[1]), 1), (dict(pr=P[6]), 1), (dict(tok=P[0] + 1596), 1),
    (dict(V=(1 << 21) + 1, ld=1 << 22), 2), (dict(rows=(1 << 24) + 1), 2),
    (dict(rows=0), 0), (dict(rows=0, lg=None, u=None, tok=None, pr=None), 0),
])
def test_sample_validation(L, kw, code):
    assert _sample(L, **kw) == code
    assert bool(L.dflash2_last_error()) == (code != 0)


def _distill(L, lg=P[0], ld=100, ids=P[1], y=P[2], w=P[3], rows=4, V=100, K=3, T=1.0, dt=0,
             loss=P[4], lse=P[5], g=P[6], gld=100, fl=P[7]):
    return L.dflash2_distill(lg, ld, ids, y, w, rows, V, K, T, dt, loss, lse, g, gld, fl, None)


def _back(L, lg=P[0], ld=100, ids=P[1], y=P[2], w=P[3], rows=4, V=100, K=3, T=1.0, dt=0,
          up=P[4], lse=P[5], g=P[6], gld=100, fl=P[7]):
    return L.dflash2_distill_backward(up, lg, ld, ids, y, w, lse, rows, V, K, T, dt, g, gld, fl,
                                      None)


COMMON = [
    (dict(lg=None), 1), (dict(ids=None), 1), (dict(y=None), 1), (dict(lse=None), 1),
    (dict(rows=-1), 1), (dict(V=0), 1), (dict(K=0), 1), (dict(dt=3), 1), (dict(ld=99), 1),
    (dict(gld=99), 1), (dict(T=0.0), 1), (dict(T=-1.0), 1), (dict(T=INF), 1), (dict(T=NAN), 1),
    (dict(T=1e-45), 1), (dict(lg=P[0] + 2), 1), (dict(g=P[6] + 2), 1), (dict(ids=P[1] + 2), 1),
    (dict(y=P[2] + 1), 1), (dict(w=P[3] + 2), 1), (dict(lse=P[5] + 1), 1), (dict(fl=P[7] + 2), 1),
    (dict(g=P[0] + 16), 1), (dict(g=P[0], gld=104), 1), (dict(g=P[1]), 1), (dict(fl=P[2]), 1),
    (dict(g=P[0] + 1596), 1), (dict(K=1025), 2),
    (dict(V=(1 << 28) + 1, ld=1 << 29, gld=1 << 29, lg=1 << 45, g=1 << 44), 2),
    (dict(rows=(1 << 24) + 1), 2), (dict(rows=0), 0),
]


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(loss=None), 1), (dict(loss=P[4] + 2), 1), (dict(loss=P[5]), 1), (dict(loss=P[3]), 1),
    (dict(rows=0, lg=None, ids=None, y=None, loss=None, lse=None), 0),
])
def test_distill_validation(L, kw, code):
    assert _distill(L, **kw) == code
    assert bool(L.dflash2_last_error()) == (code != 0)


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(up=None), 1), (dict(g=None), 1), (dict(up=P[4] + 1), 1), (dict(g=P[4]), 1),
    (dict(g=P[5]), 1),
])
def test_distill_backward_validation(L, kw, code):
    assert _back(L, **kw) == code
    assert bool(L.dflash2_last_error()) == (code != 0)


def test_last_error_names_the_call(L):
    assert _back(L, K=0) == 1
    assert ctypes.string_at(L.dflash2_last_error()).startswith(b"distill_backward")


def test_binding_refuses_host_tensors_before_any_call():
    import torch

    import dflash2_draft_head_gb300 as df2
    x, u = torch.zeros(2, 8), torch.zeros(2)
    ids, y = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, 3)
    with pytest.raises(ValueError):
        df2.sample(x, u)
    with pytest.raises(ValueError):
        df2.distill(x, ids, y)
    with pytest.raises(ValueError):
        df2.distill_backward(u, x, ids, y, u)
