"""Host-side argument checks of the losses on rewards and preferences, the gradients' norm and AdamW
(CPU only: every call here is refused before any CUDA work, or has nothing to do and so
launches nothing)."""
import ctypes

import pytest
import torch

import dflash2_draft_head_gb300 as df2
from dflash2_draft_head_gb300 import binding, build_library


@pytest.fixture(scope="module")
def L():
    build_library()
    return binding.lib()


# fake addresses far apart: passed only to calls that launch nothing
P = [0x10000000 * (k + 1) for k in range(24)]
NAN, INF = float("nan"), float("inf")


def _policy(L, lg=P[0], ld=100, tok=P[1], old=P[2], adv=P[3], ref=P[4], w=P[5], rows=4, V=100, T=1.0,
            lo=0.2, hi=0.2, kl=0.1, dt=0, loss=P[6], logp=P[7], lse=P[8], g=P[9], gld=100, fl=P[10]):
    return L.dflash2_policy_loss(lg, ld, tok, old, adv, ref, w, rows, V, T, lo, hi, kl, dt, loss,
                                 logp, lse, g, gld, fl, None)


def _policy_back(L, up=P[6], lg=P[0], ld=100, tok=P[1], old=P[2], adv=P[3], ref=P[4], w=P[5],
                 logp=P[7], lse=P[8], rows=4, V=100, T=1.0, lo=0.2, hi=0.2, kl=0.1, dt=0, g=P[9],
                 gld=100, fl=P[10]):
    return L.dflash2_policy_loss_backward(up, lg, ld, tok, old, adv, ref, w, logp, lse, rows, V, T,
                                          lo, hi, kl, dt, g, gld, fl, None)


ROWS = [
    (dict(lg=None), 1), (dict(tok=None), 1), (dict(lse=None), 1), (dict(rows=-1), 1), (dict(V=0), 1),
    (dict(dt=3), 1), (dict(ld=99), 1), (dict(gld=99), 1), (dict(lg=P[0] + 2), 1),
    (dict(g=P[9] + 2), 1), (dict(tok=P[1] + 2), 1), (dict(w=P[5] + 2), 1), (dict(lse=P[8] + 1), 1),
    (dict(fl=P[10] + 2), 1), (dict(ref=P[4] + 1), 1), (dict(g=P[0] + 16), 1),
    (dict(g=P[0], gld=104), 1), (dict(g=P[1]), 1), (dict(fl=P[1]), 1), (dict(fl=P[8]), 1),
    (dict(g=P[0] + 1596), 1), (dict(g=P[8] - 1596), 1),
    (dict(V=(1 << 28) + 1, ld=1 << 29, gld=1 << 29, lg=1 << 45, g=1 << 44), 2),
    (dict(rows=(1 << 24) + 1), 2),
]
POLICY = ROWS + [
    (dict(old=None), 1), (dict(adv=None), 1), (dict(ref=None), 1), (dict(T=0.0), 1),
    (dict(T=-1.0), 1), (dict(T=INF), 1), (dict(T=NAN), 1), (dict(T=1e-45), 1), (dict(lo=-0.1), 1),
    (dict(lo=NAN), 1), (dict(hi=-0.1), 1), (dict(hi=NAN), 1), (dict(kl=INF), 1), (dict(kl=NAN), 1),
    (dict(old=P[2] + 1), 1), (dict(adv=P[3] + 2), 1), (dict(logp=P[7] + 2), 1), (dict(logp=None), 1),
    (dict(rows=0), 0), (dict(rows=0, lg=None, tok=None, old=None, adv=None, lse=None), 0),
]


@pytest.mark.parametrize("kw,code", POLICY + [
    (dict(loss=None), 1), (dict(loss=P[6] + 2), 1), (dict(loss=P[7]), 1), (dict(lse=P[2]), 1),
])
def test_policy_validation(L, kw, code):
    assert _policy(L, **kw) == code
    assert bool(L.dflash2_last_error()) == (code != 0)


@pytest.mark.parametrize("kw,code", POLICY + [
    (dict(up=None), 1), (dict(g=None), 1), (dict(up=P[6] + 1), 1), (dict(g=P[6]), 1),
    (dict(g=P[7]), 1),
])
def test_policy_backward_validation(L, kw, code):
    assert _policy_back(L, **kw) == code
    assert bool(L.dflash2_last_error()) == (code != 0)


def _pref(L, lg=P[0], ld=100, tok=P[1], off=P[2], ref=P[4], w=P[5], rows=4, V=100, pairs=2, beta=0.1,
          e=0.0, margin=0.0, avg=0, dt=0, loss=P[6], seq=P[7], logp=P[11], lse=P[8], g=P[9], gld=100,
          fl=P[10]):
    return L.dflash2_preference_loss(lg, ld, tok, off, ref, w, rows, V, pairs, beta, e, margin, avg,
                                     dt, loss, seq, logp, lse, g, gld, fl, None)


def _pref_back(L, up=P[6], lg=P[0], ld=100, tok=P[1], off=P[2], ref=P[4], w=P[5], seq=P[7], lse=P[8],
               rows=4, V=100, pairs=2, beta=0.1, e=0.0, margin=0.0, avg=0, dt=0, g=P[9], gld=100,
               fl=P[10]):
    return L.dflash2_preference_loss_backward(up, lg, ld, tok, off, ref, w, seq, lse, rows, V, pairs,
                                              beta, e, margin, avg, dt, g, gld, fl, None)


PREF = ROWS + [
    (dict(off=None), 1), (dict(seq=None), 1), (dict(pairs=-1), 1), (dict(beta=INF), 1),
    (dict(beta=NAN), 1), (dict(margin=INF), 1), (dict(e=-0.01), 1), (dict(e=1.01), 1),
    (dict(e=NAN), 1), (dict(off=P[2] + 2), 1), (dict(seq=P[7] + 2), 1),
    (dict(pairs=(1 << 24) + 1), 2), (dict(rows=0, pairs=0), 0),
]


@pytest.mark.parametrize("kw,code", PREF + [
    (dict(loss=None), 1), (dict(logp=None), 1), (dict(loss=P[7] + 4), 1), (dict(seq=P[4]), 1),
    (dict(logp=P[8] + 4), 1), (dict(seq=P[2] + 16), 1), (dict(rows=0, off=None), 1),
    (dict(rows=0, loss=None), 1),
])
def test_preference_validation(L, kw, code):
    assert _pref(L, **kw) == code
    assert bool(L.dflash2_last_error()) == (code != 0)


@pytest.mark.parametrize("kw,code", PREF + [
    (dict(up=None), 1), (dict(g=None), 1), (dict(up=P[6] + 1), 1), (dict(g=P[6]), 1),
    (dict(g=P[7]), 1), (dict(rows=0), 0),
])
def test_preference_backward_validation(L, kw, code):
    assert _pref_back(L, **kw) == code
    assert bool(L.dflash2_last_error()) == (code != 0)


def _array(kind, v):
    return None if v is None else (kind * len(v))(*v)


def _ptrs(v):
    return _array(ctypes.c_void_p, v)


def _norm(L, grads=(P[0], P[1]), sizes=(100, 600000), dt=0, ws=P[2], wb=304, out=P[3], count=2):
    return L.dflash2_grad_norm(count, _ptrs(grads), _array(ctypes.c_int64, sizes), dt, ws, wb, out,
                               None)


@pytest.mark.parametrize("kw,code", [
    (dict(count=-1), 1), (dict(grads=None), 1), (dict(sizes=None), 1), (dict(sizes=(100, -1)), 1),
    (dict(sizes=(100, (1 << 40) + 1)), 2), (dict(dt=2), 1), (dict(out=None), 1), (dict(ws=None), 1),
    (dict(wb=303), 1), (dict(ws=P[2] + 4), 1), (dict(out=P[3] + 2), 1), (dict(grads=(P[0], None)), 1),
    (dict(grads=(P[0], P[1] + 2)), 1), (dict(grads=(P[0], P[1] + 1), dt=1), 1), (dict(out=P[1] + 796), 1),
    (dict(ws=P[0]), 1), (dict(out=P[2] + 300), 1),
])
def test_grad_norm_validation(L, kw, code):
    assert _norm(L, **kw) == code
    assert bool(L.dflash2_last_error())


def test_grad_norm_workspace(L):
    def need(*n):
        return L.dflash2_grad_norm_workspace_bytes(len(n), _array(ctypes.c_int64, n))
    assert need() == 0 and need(0, 0) == 0 and need(-1) == 0
    assert need(1) == 0 and need(32 * 16384) == 0 and need(*[1] * 32) == 0   # one launch does
    assert need(32 * 16384 + 1) == 264 and need(*[1] * 33) == 264
    assert need(31 * 16384 + 1, 0, 1) == 264
    assert need(1 << 40) == (1 << 40) // 16384 * 8


def _adamw(L, p=(P[0], P[1]), g=(P[2], P[3]), m=(P[4], P[5]), v=(P[6], P[7]), w=None, ms=None, vs=None,
           sizes=(100, 200), pdt=0, gdt=0, step_at=None, lr_at=None, step=1, lr=1e-3, b1=0.9, b2=0.999,
           eps=1e-8, wd=0.01, norm=None, most=0.0, scale=1.0, chance=0, count=2):
    return L.dflash2_adamw(count, _ptrs(p), _ptrs(g), _ptrs(m), _ptrs(v), _ptrs(w), _ptrs(ms),
                           _ptrs(vs), _array(ctypes.c_int64, sizes), pdt, gdt, step_at, lr_at, step,
                           lr, b1, b2, eps, wd, norm, most, scale, chance, 7, None)


SCALES = dict(ms=(P[8], P[9]), vs=(P[10], P[11]))


@pytest.mark.parametrize("kw,code", [
    (dict(count=-1), 1), (dict(sizes=None), 1), (dict(sizes=(100, -1)), 1),
    (dict(sizes=((1 << 40) + 1, 1)), 2), (dict(pdt=2), 1), (dict(gdt=-1), 1), (dict(b1=1.0), 1),
    (dict(b1=-0.1), 1), (dict(b1=NAN), 1), (dict(b2=1.0), 1), (dict(eps=0.0), 1), (dict(eps=-1.0), 1),
    (dict(eps=1e-60), 1), (dict(eps=1e60), 1), (dict(eps=NAN), 1), (dict(lr=INF), 1), (dict(lr=NAN), 1),
    (dict(wd=NAN), 1), (dict(scale=INF), 1), (dict(most=-1.0), 1), (dict(most=NAN), 1),
    (dict(most=1.0), 1), (dict(step=0), 1), (dict(step=-5), 1), (dict(ms=(P[8], P[9])), 1),
    (dict(vs=(P[8], P[9])), 1), (dict(w=(P[8], P[9])), 1), (dict(p=None), 1), (dict(g=None), 1),
    (dict(m=None), 1), (dict(v=None), 1), (dict(p=(P[0], None)), 1), (dict(w=(P[8], None), pdt=1), 1),
    (dict(p=(P[0], P[1] + 2)), 1), (dict(p=(P[0], P[1] + 1), pdt=1), 1), (dict(g=(P[2] + 2, P[3])), 1),
    (dict(m=(P[4] + 1, P[5])), 1), (dict(step_at=P[12] + 2), 1), (dict(lr_at=P[12] + 1), 1),
    (dict(norm=P[12] + 2), 1), (dict(p=(P[0], P[0])), 1), (dict(p=(P[0], P[0] + 396)), 1),
    (dict(g=(P[0], P[3])), 1), (dict(v=(P[4], P[7])), 1), (dict(norm=P[0] + 4), 1),
    (dict(step_at=P[4]), 1), (dict(lr_at=P[7] + 796), 1), (dict(m=(P[4], P[4] + 99)) | SCALES, 1),
    (dict(ms=(P[8], P[8] + 3), vs=(P[10], P[11])), 1), (dict(count=0, p=None, g=None, m=None, v=None,
                                                             sizes=None), 0),
    (dict(sizes=(0, 0), p=(None, None), g=(None, None), m=(None, None), v=(None, None)), 0),
])
def test_adamw_validation(L, kw, code):
    assert _adamw(L, **kw) == code
    assert bool(L.dflash2_last_error()) == (code != 0)


@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), 1), (dict(c=None), 1), (dict(s=None), 1), (dict(x=None), 1), (dict(dt=2), 1),
    (dict(x=P[2] + 2), 1), (dict(x=P[2] + 1, dt=1), 1), (dict(x=P[0] + 96), 1), (dict(x=P[1] - 396), 1),
    (dict(n=(1 << 40) + 1), 2), (dict(n=0, c=None, s=None, x=None), 0),
])
def test_state_validation(L, kw, code):
    a = dict(c=P[0], s=P[1], x=P[2], n=100, dt=0) | kw
    assert L.dflash2_state_decode(a["c"], a["s"], a["n"], 1, a["dt"], a["x"], None) == code
    assert bool(L.dflash2_last_error()) == (code != 0)
    assert L.dflash2_state_encode(a["x"], a["dt"], a["n"], 1, a["c"], a["s"], None) == code
    assert bool(L.dflash2_last_error()) == (code != 0)


def test_codes_and_scales_do_not_overlap(L):
    assert L.dflash2_state_encode(P[2], 0, 100, 0, P[0], P[0] + 99, None) == 1


def test_last_error_names_the_call(L):
    assert _policy_back(L, V=0) == 1
    assert ctypes.string_at(L.dflash2_last_error()).startswith(b"policy_loss_backward")
    assert _pref(L, pairs=-1) == 1
    assert ctypes.string_at(L.dflash2_last_error()).startswith(b"preference_loss:")


def test_binding_refuses_host_tensors_before_any_call():
    x, t, f = torch.zeros(2, 8), torch.zeros(2, dtype=torch.int32), torch.zeros(2)
    c = torch.zeros(8, dtype=torch.uint8)
    for call in (lambda: df2.policy_loss(x, t, f, f),
                 lambda: df2.policy_loss_backward(f, x, t, f, f, f, f),
                 lambda: df2.preference_loss(x, t, t),
                 lambda: df2.preference_loss_backward(f, x, t, t, f, f),
                 lambda: df2.grad_norm([f]), lambda: df2.grad_norm([]),
                 lambda: df2.adamw([f], [f], [f], [f], step=1, lr=1e-3),
                 lambda: df2.adamw([], [f], [], [], step=1, lr=1e-3),
                 lambda: df2.state_decode(c, c), lambda: df2.state_encode(f)):
        with pytest.raises(ValueError):
            call()
