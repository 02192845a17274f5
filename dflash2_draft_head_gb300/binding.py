"""ctypes binding of libdflash2.so (the C ABI declared in include/dflash2.h).

Argument marshalling only: shapes and dtypes are read from torch tensors,
outputs are allocated with torch when the caller does not pass them, and the
call goes to the CUDA library on the tensors' current stream.  There is no
fallback: if the library is missing or a call fails, an exception is raised.
"""
from __future__ import annotations

import array
import ctypes
import operator
import os
import threading

import torch
from torch.autograd.graph import increment_version  # for what autograd may have saved

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdflash2.so")

DF2_OK, DF2_ERR_INVALID_ARG, DF2_ERR_UNSUPPORTED, DF2_ERR_CUDA = 0, 1, 2, 3
DF2_F32, DF2_BF16 = 0, 1
FLAG_BAD_ID, FLAG_TIMEOUT, FLAG_OVERFLOW = 1, 2, 4

_lock = threading.Lock()
_lib = None


class Dflash2Error(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(msg)
        self.status = status


def lib() -> ctypes.CDLL:
    """The loaded library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"{LIB_PATH} is missing: build it first "
                    "(python -c 'import __graft_entry__ as g; g.build()')")
            L = ctypes.CDLL(LIB_PATH)
            vp, i = ctypes.c_void_p, ctypes.c_int
            L.dflash2_version.argtypes = []
            L.dflash2_version.restype = i
            L.dflash2_status_string.argtypes = [i]
            L.dflash2_status_string.restype = ctypes.c_char_p
            L.dflash2_last_error.argtypes = []
            L.dflash2_last_error.restype = ctypes.c_char_p
            L.dflash2_dynconv.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, i, vp]
            L.dflash2_dynconv.restype = i
            L.dflash2_project.argtypes = [vp, vp, vp, i, i, i, i, vp]
            L.dflash2_project.restype = i
            L.dflash2_project_workspace_bytes.argtypes = [i, i, i]
            L.dflash2_project_workspace_bytes.restype = ctypes.c_size_t
            L.dflash2_project_ws.argtypes = [vp, vp, vp, i, i, i, i, vp, ctypes.c_size_t, vp]
            L.dflash2_project_ws.restype = i
            L.dflash2_project_noalloc.argtypes = [vp, vp, vp, i, i, i, i, vp]
            L.dflash2_project_noalloc.restype = i
            L.dflash2_edges.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, vp, vp, vp, vp, vp]
            L.dflash2_edges.restype = i
            L.dflash2_select.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, vp, vp, vp,
                                         vp, vp, vp]
            L.dflash2_select.restype = i
            L.dflash2_predict_delta.argtypes = [vp, vp, vp, i, i, i, i, vp]
            L.dflash2_predict_delta.restype = i
            L.dflash2_dynconv_predicted.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, i, vp]
            L.dflash2_dynconv_predicted.restype = i
            L.dflash2_chain.argtypes = [vp, vp, vp, vp, vp, i, i, i, ctypes.c_float, vp, vp, vp,
                                        vp, vp]
            L.dflash2_chain.restype = i
            L.dflash2_topk.argtypes = [vp, i, i, i, i, vp, vp, vp]
            L.dflash2_topk.restype = i
            ll, f = ctypes.c_longlong, ctypes.c_float
            L.dflash2_sample.argtypes = [vp, ll, vp, vp, vp, vp, vp, f, i, f, f, i, i, i, vp, vp,
                                         vp]
            L.dflash2_sample.restype = i
            L.dflash2_distill.argtypes = [vp, ll, vp, vp, vp, i, i, i, f, i, vp, vp, vp, ll, vp,
                                          vp]
            L.dflash2_distill.restype = i
            L.dflash2_distill_backward.argtypes = [vp, vp, ll, vp, vp, vp, vp, i, i, i, f, i, vp,
                                                   ll, vp, vp]
            L.dflash2_distill_backward.restype = i
            d = ctypes.c_double
            L.dflash2_policy_loss.argtypes = [vp, ll, vp, vp, vp, vp, vp, i, i, f, f, f, f, i, vp,
                                              vp, vp, vp, ll, vp, vp]
            L.dflash2_policy_loss.restype = i
            L.dflash2_policy_loss_backward.argtypes = [vp, vp, ll, vp, vp, vp, vp, vp, vp, vp, i,
                                                       i, f, f, f, f, i, vp, ll, vp, vp]
            L.dflash2_policy_loss_backward.restype = i
            L.dflash2_preference_loss.argtypes = [vp, ll, vp, vp, vp, vp, i, i, i, f, f, f, i, i,
                                                  vp, vp, vp, vp, vp, ll, vp, vp]
            L.dflash2_preference_loss.restype = i
            L.dflash2_preference_loss_backward.argtypes = [vp, vp, ll, vp, vp, vp, vp, vp, vp, i,
                                                           i, i, f, f, f, i, i, vp, ll, vp, vp]
            L.dflash2_preference_loss_backward.restype = i
            L.dflash2_grad_norm_workspace_bytes.argtypes = [i, vp]
            L.dflash2_grad_norm_workspace_bytes.restype = ctypes.c_size_t
            L.dflash2_grad_norm.argtypes = [i, vp, vp, i, vp, ctypes.c_size_t, vp, vp]
            L.dflash2_grad_norm.restype = i
            L.dflash2_adamw.argtypes = [i, vp, vp, vp, vp, vp, vp, vp, vp, i, i, vp, vp, i, d, d,
                                        d, d, d, vp, d, d, i, ctypes.c_uint64, vp]
            L.dflash2_adamw.restype = i
            L.dflash2_state_decode.argtypes = [vp, vp, ll, i, i, vp, vp]
            L.dflash2_state_decode.restype = i
            L.dflash2_state_encode.argtypes = [vp, i, ll, i, vp, vp, vp]
            L.dflash2_state_encode.restype = i
            L.dflash2_select_plan.argtypes = [i, i, i, i, i, i, ctypes.POINTER(ctypes.c_int)]
            L.dflash2_select_plan.restype = i
            L.dflash2_probe_gather.argtypes = [vp, ctypes.c_longlong, i, vp, i, vp, vp]
            L.dflash2_probe_gather.restype = i
            L.dflash2_take_device_faults.argtypes = [ctypes.POINTER(ctypes.c_int32)]
            L.dflash2_take_device_faults.restype = i
            _lib = L
    return _lib


def _check(status: int):
    if status != DF2_OK:
        L = lib()
        raise Dflash2Error(status, f"{L.dflash2_status_string(status).decode()}: "
                                   f"{L.dflash2_last_error().decode()}")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(dev) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream)


def _raw_stream(index: int) -> int:
    """The current stream's handle without a Stream object around it (2 us a call).  Looked
    up at the call: a torch without CUDA has no such function."""
    return torch._C._cuda_getCurrentRawStream(index)


def _code(dt: torch.dtype) -> int:
    if dt == torch.bfloat16:
        return DF2_BF16
    if dt == torch.float32:
        return DF2_F32
    raise TypeError(f"unsupported dtype {dt}")


def _need(t, name, dtype=None):
    if t is None:
        return
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")


def version() -> int:
    return lib().dflash2_version()


def dynconv(x, hist, base, delta, out=None, out_dtype=None):
    """Grouped dynamic depthwise causal conv: x [S,n,C], hist [S,T-1,C] or None,
    base [T,C], delta [S,n,T,G] -> out [S,n,C]."""
    S, n, C = x.shape
    T = base.shape[0]
    G = delta.shape[-1]
    for t, nm in ((x, "x"), (hist, "hist"), (base, "base"), (delta, "delta")):
        _need(t, nm, x.dtype)
    if out is None:
        out = torch.empty((S, n, C), dtype=out_dtype or x.dtype, device=x.device)
    _need(out, "out")
    _check(lib().dflash2_dynconv(_ptr(x), _ptr(hist), _ptr(base), _ptr(delta), _ptr(out),
                                 S, n, C, T, G, _code(x.dtype), _code(out.dtype),
                                 _stream(x.device)))
    return out


def project_workspace_bytes(P: int, d: int, R: int) -> int:
    """Bytes of split-K workspace project(..., workspace=...) needs on this device."""
    return int(lib().dflash2_project_workspace_bytes(P, d, R))


def project(h, W, u=None, workspace=None):
    """u [P,R] fp32 = h [P,d] @ W[R,d]^T.  With `workspace` (a CUDA tensor of at
    least project_workspace_bytes(P, d, R) bytes) the split-K partial tiles are
    exchanged through it instead of through distributed shared memory."""
    P, d = h.shape
    R = W.shape[0]
    _need(h, "h")
    _need(W, "W", h.dtype)
    if u is None:
        u = torch.empty((P, R), dtype=torch.float32, device=h.device)
    _need(u, "u", torch.float32)
    if workspace is None:
        _check(lib().dflash2_project(_ptr(h), _ptr(W), _ptr(u), P, d, R, _code(h.dtype),
                                     _stream(h.device)))
    else:
        _need(workspace, "workspace")
        _check(lib().dflash2_project_ws(_ptr(h), _ptr(W), _ptr(u), P, d, R, _code(h.dtype),
                                        _ptr(workspace),
                                        workspace.numel() * workspace.element_size(),
                                        _stream(h.device)))
    return u


def project_noalloc(h, W, u=None):
    """project() through the library's fixed workspace (no device allocation by
    the library; u must be passed to avoid torch allocating it)."""
    P, d = h.shape
    R = W.shape[0]
    _need(h, "h")
    _need(W, "W", h.dtype)
    if u is None:
        u = torch.empty((P, R), dtype=torch.float32, device=h.device)
    _need(u, "u", torch.float32)
    _check(lib().dflash2_project_noalloc(_ptr(h), _ptr(W), _ptr(u), P, d, R, _code(h.dtype),
                                         _stream(h.device)))
    return u


def _edge_outputs(S, n, K, dev, edges_out, best_slot, best_score):
    E = max(n - 1, 0)
    if edges_out is True:
        edges_out = torch.empty((S, E, K, K), dtype=torch.float32, device=dev)
    elif edges_out is False:
        edges_out = None
    if best_slot is None:
        best_slot = torch.empty((S, E, K), dtype=torch.int32, device=dev)
    if best_score is None:
        best_score = torch.empty((S, E, K), dtype=torch.float32, device=dev)
    return edges_out, best_slot, best_score


def edges(cand_ids, u, A, B, unary, edges_out=None, best_slot=None, best_score=None,
          err_flag=None):
    """Edge scores + per-predecessor argmax.  cand_ids [S,n,K] int32, u [S*n,R] fp32,
    A, B [V,R], unary [S,n,K] fp32.  edges_out=True allocates the [S,n-1,K,K] matrix.
    Returns (edges_out or None, best_slot [S,n-1,K] int32, best_score [S,n-1,K] fp32)."""
    S, n, K = cand_ids.shape
    V, R = A.shape
    _need(cand_ids, "cand_ids", torch.int32)
    _need(u, "u", torch.float32)
    _need(A, "A")
    _need(B, "B", A.dtype)
    _need(unary, "unary", torch.float32)
    edges_out, best_slot, best_score = _edge_outputs(S, n, K, u.device, edges_out, best_slot,
                                                     best_score)
    _need(err_flag, "err_flag", torch.int32)
    _check(lib().dflash2_edges(_ptr(cand_ids), _ptr(u), _ptr(A), _ptr(B), _ptr(unary), S, n, K,
                               R, V, _code(A.dtype), _ptr(edges_out), _ptr(best_slot),
                               _ptr(best_score), _ptr(err_flag), _stream(u.device)))
    return edges_out, best_slot, best_score


def select(h, W, cand_ids, A, B, unary, u_out=None, edges_out=None, best_slot=None,
           best_score=None, err_flag=None):
    """Composite selector: project then edges.  h [S*n,d].
    Returns (u [S*n,R], edges_out or None, best_slot, best_score)."""
    S, n, K = cand_ids.shape
    d = h.shape[-1]
    V, R = A.shape
    _need(h, "h")
    _need(W, "W", h.dtype)
    _need(cand_ids, "cand_ids", torch.int32)
    _need(A, "A", h.dtype)
    _need(B, "B", h.dtype)
    _need(unary, "unary", torch.float32)
    if u_out is None:
        u_out = torch.empty((S * n, R), dtype=torch.float32, device=h.device)
    _need(u_out, "u_out", torch.float32)
    edges_out, best_slot, best_score = _edge_outputs(S, n, K, h.device, edges_out, best_slot,
                                                     best_score)
    _need(err_flag, "err_flag", torch.int32)
    _check(lib().dflash2_select(_ptr(h), _ptr(W), _ptr(cand_ids), _ptr(A), _ptr(B), _ptr(unary),
                                S, n, d, K, R, V, _code(h.dtype), _ptr(u_out), _ptr(edges_out),
                                _ptr(best_slot), _ptr(best_score), _ptr(err_flag),
                                _stream(h.device)))
    return u_out, edges_out, best_slot, best_score


def topk(logits, K, cand_ids=None, values=None):
    """Top-K candidates of every row: logits [..., V] (fp32 or bf16) ->
    (cand_ids [..., K] int32, values [..., K] fp32), descending, ties by index."""
    V = logits.shape[-1]
    lead = tuple(logits.shape[:-1])
    rows = 1
    for s in lead:
        rows *= s
    _need(logits, "logits")
    if cand_ids is None:
        cand_ids = torch.empty(lead + (K,), dtype=torch.int32, device=logits.device)
    if values is None:
        values = torch.empty(lead + (K,), dtype=torch.float32, device=logits.device)
    _need(cand_ids, "cand_ids", torch.int32)
    _need(values, "values", torch.float32)
    _check(lib().dflash2_topk(_ptr(logits), rows, V, K, _code(logits.dtype), _ptr(cand_ids),
                              _ptr(values), _stream(logits.device)))
    return cand_ids, values


def predict_delta(x, Wc, T, G, delta=None):
    """delta [S,n,T,G] = x [S,n,C] . Wc[T*G, C]^T in x's dtype (the conv's
    dynamic taps predicted from its input)."""
    S, n, C = x.shape
    _need(x, "x")
    _need(Wc, "Wc", x.dtype)
    if delta is None:
        delta = torch.empty((S, n, T, G), dtype=x.dtype, device=x.device)
    _need(delta, "delta", x.dtype)
    _check(lib().dflash2_predict_delta(_ptr(x), _ptr(Wc), _ptr(delta), S * n, C, T * G,
                                       _code(x.dtype), _stream(x.device)))
    return delta


def dynconv_predicted(x, hist, base, Wc, G, out=None, out_dtype=None):
    """The conv with its taps predicted from its input, fused: x [S,n,C], hist
    [S,T-1,C] or None, base [T,C], Wc [T*G,C] (bf16) -> out [S,n,C]; the same as
    dynconv(x, hist, base, predict_delta(x, Wc, T, G)) without delta in HBM."""
    S, n, C = x.shape
    T = base.shape[0]
    for t, nm in ((x, "x"), (hist, "hist"), (base, "base"), (Wc, "Wc")):
        _need(t, nm, x.dtype)
    if out is None:
        out = torch.empty((S, n, C), dtype=out_dtype or x.dtype, device=x.device)
    _need(out, "out")
    _check(lib().dflash2_dynconv_predicted(_ptr(x), _ptr(hist), _ptr(base), _ptr(Wc), _ptr(out),
                                           S, n, C, T, G, _code(x.dtype), _code(out.dtype),
                                           _stream(x.device)))
    return out


def chain(cand_ids, unary, edges, best_slot, p_min, start_slot=None, err_flag=None):
    """Greedy chain readout: (tokens [S,n] int32, probs [S,n] fp32, length [S] int32).
    cand_ids, unary [S,n,K]; edges [S,n-1,K,K] and best_slot [S,n-1,K] from
    select(..., edges_out=True) (None when n == 1); start_slot [S] int32 or None."""
    S, n, K = cand_ids.shape
    _need(cand_ids, "cand_ids", torch.int32)
    _need(unary, "unary", torch.float32)
    _need(edges, "edges", torch.float32)
    _need(best_slot, "best_slot", torch.int32)
    _need(start_slot, "start_slot", torch.int32)
    _need(err_flag, "err_flag", torch.int32)
    dev = cand_ids.device
    tokens = torch.empty((S, n), dtype=torch.int32, device=dev)
    probs = torch.empty((S, n), dtype=torch.float32, device=dev)
    length = torch.empty((S,), dtype=torch.int32, device=dev)
    _check(lib().dflash2_chain(_ptr(cand_ids), _ptr(unary), _ptr(edges), _ptr(best_slot),
                               _ptr(start_slot), S, n, K, float(p_min), _ptr(tokens), _ptr(probs),
                               _ptr(length), _ptr(err_flag), _stream(dev)))
    return tokens, probs, length


def _logit_rows(t, name):
    """(leading shape, rows, V, elements between two rows) of [..., V] logits: any
    spacing of the rows, but one, and elements that lie side by side."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    shape = t.shape
    V = shape[-1]
    if len(shape) == 2:
        ld, unit = t.stride()
        if (unit == 1 or V <= 1) and ld >= V:
            return shape[:1], shape[0], V, ld
    if 0 in shape[:-1]:  # the strides of a tensor without elements say nothing
        return shape[:-1], 0, V, max(V, 1)
    strides = t.stride()
    if V > 1 and strides[-1] != 1:
        raise ValueError(f"{name} must have its last dimension contiguous")
    rows, ld = 1, None
    for n, st in zip(reversed(shape[:-1]), reversed(strides[:-1])):
        if n != 1:
            if ld is None:
                ld = st
            elif st != ld * rows:
                raise ValueError(f"the rows of {name} must be evenly spaced")
        rows *= n
    return shape[:-1], rows, V, max(V, 1) if ld is None else ld


def _need_rows(t, name, dtype, shape):
    if t.dtype is dtype and t.is_cuda and t.shape == shape and t.is_contiguous():
        return t.data_ptr()
    _need(t, name, dtype)
    raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _out_rows(t, name, dtype, shape, dev, like=None):
    """(tensor, pointer) of an output with a value for every row, allocated for None
    (from `like`, another such fp32 tensor, where there is one: that takes less time)."""
    if t is None:
        if like is None:
            t = torch.empty(shape, dtype=dtype, device=dev)
        elif dtype is torch.float32:
            t = torch.empty_like(like)
        else:
            t = torch.empty_like(like, dtype=dtype)
        return t, t.data_ptr()
    return t, _need_rows(t, name, dtype, shape)


def _setting(v, name, dtype, shape):
    """(pointer, scalar) of a setting given for every row or once for all."""
    if isinstance(v, torch.Tensor):
        return _need_rows(v, name, dtype, shape), 0
    return None, v


def sample(logits, uniform, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, tokens=None,
           probs=None):
    """One token of every row: logits [..., V] (fp32 or bf16; the rows may be evenly
    spaced views), uniform [...] fp32 in [0, 1) -> (tokens [...] int32, probs [...]
    fp32, the token's share among the entries that top_k, top_p and min_p keep).
    Each setting is a number or a tensor [...] with one per row (top_k int32, the
    others fp32).  The same row and number give the same token in any batch."""
    shape, rows, V, ld = _logit_rows(logits, "logits")
    up = _need_rows(uniform, "uniform", torch.float32, shape)
    tp, t0 = _setting(temperature, "temperature", torch.float32, shape)
    kp, k0 = _setting(top_k, "top_k", torch.int32, shape)
    k0 = max(-1, min(k0, 0x7fffffff))  # the entry takes 32 bits; both ends are no limit
    pp, p0 = _setting(top_p, "top_p", torch.float32, shape)
    mp, m0 = _setting(min_p, "min_p", torch.float32, shape)
    dev = logits.device
    tokens, tokens_ptr = _out_rows(tokens, "tokens", torch.int32, shape, dev, uniform)
    probs, probs_ptr = _out_rows(probs, "probs", torch.float32, shape, dev, uniform)
    st = lib().dflash2_sample(logits.data_ptr(), ld, up, tp, kp, pp, mp, t0, k0, p0, m0, rows, V,
                              _code(logits.dtype), tokens_ptr, probs_ptr, _raw_stream(dev.index))
    if st != DF2_OK:
        _check(st)
    return tokens, probs


def _teacher(teacher_ids, teacher_logits, weight, shape):
    """K and the pointers of the teacher's entries and the weights."""
    K = teacher_ids.shape[-1]
    each = shape + (K,)
    return (K, _need_rows(teacher_ids, "teacher_ids", torch.int32, each),
            _need_rows(teacher_logits, "teacher_logits", torch.float32, each),
            None if weight is None else _need_rows(weight, "weight", torch.float32, shape))


def _grad_rows(grad, logits, ld):
    """The gradient tensor (allocated with the logits' strides when it is True), its
    pointer and the elements between two of its rows."""
    if grad is True:
        if logits.is_contiguous():
            grad = torch.empty_like(logits)
        else:
            grad = torch.empty_strided(logits.shape, logits.stride(), dtype=logits.dtype,
                                       device=logits.device)
        return grad, grad.data_ptr(), ld
    if grad.shape != logits.shape or grad.dtype != logits.dtype:
        raise ValueError("grad must have the shape and dtype of logits")
    return grad, grad.data_ptr(), _logit_rows(grad, "grad")[3]


def distill(logits, teacher_ids, teacher_logits, temperature=1.0, weight=None, grad=False,
            loss=None, lse=None, err_flag=None):
    """Distillation from a teacher's top K logits: logits [..., V] (fp32 or bf16; the
    rows may be evenly spaced views), teacher_ids [..., K] int32 and teacher_logits
    [..., K] fp32 as topk() returns them, weight [...] fp32 or None.  Returns
    (loss [...] fp32, lse [...] fp32, grad): loss[r] = weight[r] * KL(teacher's
    softmax over its K || student), lse for distill_backward, and with grad=True (or
    a tensor to write, which may be logits) the gradient of the sum of the losses;
    else None.  The results carry no autograd graph, also where logits do: hand the
    gradient on by logits.backward(grad)."""
    shape, rows, V, ld = _logit_rows(logits, "logits")
    K, ids_ptr, teacher_ptr, weight_ptr = _teacher(teacher_ids, teacher_logits, weight, shape)
    dev = logits.device
    loss, loss_ptr = _out_rows(loss, "loss", torch.float32, shape, dev, weight)
    lse, lse_ptr = _out_rows(lse, "lse", torch.float32, shape, dev, loss)
    _need(err_flag, "err_flag", torch.int32)
    given = isinstance(grad, torch.Tensor)
    if grad is None or grad is False:
        grad, grad_ptr, grad_ld = None, None, 0
    else:
        grad, grad_ptr, grad_ld = _grad_rows(grad, logits, ld)
    st = lib().dflash2_distill(logits.data_ptr(), ld, ids_ptr, teacher_ptr, weight_ptr, rows, V, K,
                               temperature, _code(logits.dtype), loss_ptr, lse_ptr, grad_ptr,
                               grad_ld, None if err_flag is None else err_flag.data_ptr(),
                               _raw_stream(dev.index))
    if st != DF2_OK:
        _check(st)
    if given:
        increment_version(grad)
    return loss, lse, grad


def distill_backward(grad_loss, logits, teacher_ids, teacher_logits, lse, temperature=1.0,
                     weight=None, grad=True, err_flag=None):
    """The gradient of distill() by its logits alone, from the gradient by its losses,
    grad_loss [...] fp32, and the lse [...] that it returned.  grad may be a tensor to
    write (also logits).  It carries no autograd graph."""
    shape, rows, V, ld = _logit_rows(logits, "logits")
    K, ids_ptr, teacher_ptr, weight_ptr = _teacher(teacher_ids, teacher_logits, weight, shape)
    up = _need_rows(grad_loss, "grad_loss", torch.float32, shape)
    lse_ptr = _need_rows(lse, "lse", torch.float32, shape)
    _need(err_flag, "err_flag", torch.int32)
    given = isinstance(grad, torch.Tensor)
    grad, grad_ptr, grad_ld = _grad_rows(grad, logits, ld)
    st = lib().dflash2_distill_backward(up, logits.data_ptr(), ld, ids_ptr, teacher_ptr,
                                        weight_ptr, lse_ptr, rows, V, K, temperature,
                                        _code(logits.dtype), grad_ptr, grad_ld,
                                        None if err_flag is None else err_flag.data_ptr(),
                                        _raw_stream(logits.device.index))
    if st != DF2_OK:
        _check(st)
    if given:
        increment_version(grad)
    return grad


def _launch(index: int, entry, *args):
    """Calls an entry whose last argument is the stream, with the tensors' device current."""
    if torch.cuda.current_device() == index:
        st = entry(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            st = entry(*args, _raw_stream(index))
    if st != DF2_OK:
        _check(st)


def _on(t, name, dtype, shape, index):
    """Pointer of an input of this type and shape on the device; None for None."""
    if t is None:
        return None
    if t.dtype is dtype and t.get_device() == index and t.shape == shape and t.is_contiguous():
        return t.data_ptr()
    _need_rows(t, name, dtype, shape)
    raise ValueError(f"{name} must be on device cuda:{index}, got {t.device}")


def _out_on(t, name, dtype, shape, dev, like=None):
    """(tensor, pointer) of an output, allocated for None (from `like`, a contiguous tensor of
    this type and shape, where there is one: that takes less time)."""
    if t is None:
        if like is None:
            t = torch.empty(shape, dtype=dtype, device=dev)
        else:
            t = torch.empty_like(like)
        return t, t.data_ptr()
    return t, _on(t, name, dtype, shape, dev.index)


def _grad_on(grad, logits, ld):
    """_grad_rows, with no gradient for None or False and on the logits' device."""
    if grad is None or grad is False:
        return None, None, 0
    grad, ptr, grad_ld = _grad_rows(grad, logits, ld)
    if grad.get_device() != logits.get_device():
        raise ValueError("grad must be on the device of logits")
    return grad, ptr, grad_ld


def _written(outs):
    """Raises the versions of the outputs that a caller gave, for autograd, which may have saved
    them.  Before the launch, which may fail when a part of it is under way."""
    for t in outs:
        if t is not None and isinstance(t, torch.Tensor):
            increment_version(t)


def policy_loss(logits, tokens, old_logp, advantage, ref_logp=None, temperature=1.0, clip_low=0.2,
                clip_high=0.2, kl_coef=0.0, weight=None, grad=False, loss=None, logp=None, lse=None,
                err_flag=None):
    """The clipped policy loss with a KL term at the drawn tokens: logits [..., V] (fp32 or
    bf16; the rows may be evenly spaced views), tokens [...] int32 (negative: not counted),
    old_logp, advantage, ref_logp [...] fp32 (ref_logp may be None where kl_coef is 0), weight
    [...] fp32 or None.  Returns (loss, logp, lse [...] fp32, grad): with rho = exp(logp -
    old_logp) and d = ref_logp - logp,
    loss = weight * (kl_coef * (exp(d) - d - 1) - min(rho * A, clamp(rho, 1 - clip_low,
    1 + clip_high) * A)); logp and lse for policy_loss_backward; and with grad=True (or a
    tensor to write, which may be logits) the gradient of the sum of the losses; else None.
    The results carry no autograd graph: hand the gradient on by logits.backward(grad)."""
    shape, rows, V, ld = _logit_rows(logits, "logits")
    dev = logits.device
    at, f32 = dev.index, torch.float32
    ins = (_on(tokens, "tokens", torch.int32, shape, at), _on(old_logp, "old_logp", f32, shape, at),
           _on(advantage, "advantage", f32, shape, at), _on(ref_logp, "ref_logp", f32, shape, at),
           _on(weight, "weight", f32, shape, at))
    given = (loss, logp, lse, grad)
    loss, loss_ptr = _out_on(loss, "loss", f32, shape, dev, old_logp)
    logp, logp_ptr = _out_on(logp, "logp", f32, shape, dev, old_logp)
    lse, lse_ptr = _out_on(lse, "lse", f32, shape, dev, old_logp)
    flag = None if err_flag is None else _on(err_flag, "err_flag", torch.int32, (1,), at)
    grad, grad_ptr, grad_ld = _grad_on(grad, logits, ld)
    _written(given)
    _launch(at, lib().dflash2_policy_loss, logits.data_ptr(), ld, *ins, rows, V, temperature,
            clip_low, clip_high, kl_coef, _code(logits.dtype), loss_ptr, logp_ptr, lse_ptr,
            grad_ptr, grad_ld, flag)
    return loss, logp, lse, grad


def policy_loss_backward(grad_loss, logits, tokens, old_logp, advantage, logp, lse, ref_logp=None,
                         temperature=1.0, clip_low=0.2, clip_high=0.2, kl_coef=0.0, weight=None,
                         grad=True, err_flag=None):
    """The gradient of policy_loss() by its logits alone, from the gradient by its losses,
    grad_loss [...] fp32, and the logp and lse [...] that it returned.  grad may be a tensor
    to write (also logits).  It carries no autograd graph."""
    shape, rows, V, ld = _logit_rows(logits, "logits")
    at, f32 = logits.device.index, torch.float32
    up = _on(grad_loss, "grad_loss", f32, shape, at)
    ins = (_on(tokens, "tokens", torch.int32, shape, at), _on(old_logp, "old_logp", f32, shape, at),
           _on(advantage, "advantage", f32, shape, at), _on(ref_logp, "ref_logp", f32, shape, at),
           _on(weight, "weight", f32, shape, at), _on(logp, "logp", f32, shape, at),
           _on(lse, "lse", f32, shape, at))
    flag = _on(err_flag, "err_flag", torch.int32, (1,), at)
    given = (grad,)
    grad, grad_ptr, grad_ld = _grad_on(grad, logits, ld)
    _written(given)
    _launch(at, lib().dflash2_policy_loss_backward, up, logits.data_ptr(), ld, *ins, rows, V,
            temperature, clip_low, clip_high, kl_coef, _code(logits.dtype), grad_ptr, grad_ld,
            flag)
    return grad


def _pairs(offsets):
    """Number of pairs that offsets [2 * pairs + 1] divides the rows into."""
    if offsets.dim() != 1 or offsets.numel() % 2 != 1:
        raise ValueError("offsets must have the shape [2 * pairs + 1], got "
                         f"{tuple(offsets.shape)}")
    return offsets.numel() // 2


def preference_loss(logits, tokens, offsets, ref_logp=None, beta=0.1, label_smoothing=0.0,
                    margin=0.0, average=False, weight=None, grad=False, loss=None, seq_logp=None,
                    logp=None, lse=None, err_flag=None):
    """The preference loss of pairs of sequences by their log ratios: logits [..., V] (fp32 or
    bf16; the rows may be evenly spaced views), tokens [...] int32 (negative: not counted, as
    a prompt's), offsets [2 * pairs + 1] int32: sequence s has the rows offsets[s] to
    offsets[s + 1] - 1, pair i consists of the chosen sequence i and the rejected one pairs + i;
    ref_logp [2 * pairs] fp32, the reference's sums of log-probabilities (means with average=True),
    or None; weight [pairs] fp32 or None.  With S the sequences' sums (means) and m = beta *
    ((S_c - ref_c) - (S_r - ref_r)) - margin, loss = weight * ((1 - label_smoothing) * log(1 +
    exp(-m)) + label_smoothing * log(1 + exp(m))).  Returns (loss [pairs], seq_logp [2 * pairs],
    logp [...], lse [...], grad): seq_logp and lse for preference_loss_backward; grad as
    policy_loss()'s."""
    shape, rows, V, ld = _logit_rows(logits, "logits")
    dev, pairs = logits.device, _pairs(offsets)
    at, f32 = dev.index, torch.float32
    ins = (_on(tokens, "tokens", torch.int32, shape, at),
           _on(offsets, "offsets", torch.int32, (2 * pairs + 1,), at),
           _on(ref_logp, "ref_logp", f32, (2 * pairs,), at),
           _on(weight, "weight", f32, (pairs,), at))
    given = (loss, seq_logp, logp, lse, grad)
    loss, loss_ptr = _out_on(loss, "loss", f32, (pairs,), dev, weight)
    seq_logp, seq_ptr = _out_on(seq_logp, "seq_logp", f32, (2 * pairs,), dev, ref_logp)
    logp, logp_ptr = _out_on(logp, "logp", f32, shape, dev)
    lse, lse_ptr = _out_on(lse, "lse", f32, shape, dev, logp)
    flag = _on(err_flag, "err_flag", torch.int32, (1,), at)
    grad, grad_ptr, grad_ld = _grad_on(grad, logits, ld)
    _written(given)
    _launch(at, lib().dflash2_preference_loss, logits.data_ptr(), ld, *ins, rows, V, pairs, beta,
            label_smoothing, margin, average, _code(logits.dtype), loss_ptr, seq_ptr, logp_ptr,
            lse_ptr, grad_ptr, grad_ld, flag)
    return loss, seq_logp, logp, lse, grad


def preference_loss_backward(grad_loss, logits, tokens, offsets, seq_logp, lse, ref_logp=None,
                             beta=0.1, label_smoothing=0.0, margin=0.0, average=False, weight=None,
                             grad=True, err_flag=None):
    """The gradient of preference_loss() by its logits alone, from the gradient by its losses,
    grad_loss [pairs] fp32, and the seq_logp and lse that it returned.  grad may be a tensor
    to write (also logits).  It carries no autograd graph."""
    shape, rows, V, ld = _logit_rows(logits, "logits")
    pairs, at, f32 = _pairs(offsets), logits.device.index, torch.float32
    up = _on(grad_loss, "grad_loss", f32, (pairs,), at)
    ins = (_on(tokens, "tokens", torch.int32, shape, at),
           _on(offsets, "offsets", torch.int32, (2 * pairs + 1,), at),
           _on(ref_logp, "ref_logp", f32, (2 * pairs,), at),
           _on(weight, "weight", f32, (pairs,), at),
           _on(seq_logp, "seq_logp", f32, (2 * pairs,), at), _on(lse, "lse", f32, shape, at))
    flag = _on(err_flag, "err_flag", torch.int32, (1,), at)
    given = (grad,)
    grad, grad_ptr, grad_ld = _grad_on(grad, logits, ld)
    _written(given)
    _launch(at, lib().dflash2_preference_loss_backward, up, logits.data_ptr(), ld, *ins, rows, V,
            pairs, beta, label_smoothing, margin, average, _code(logits.dtype), grad_ptr, grad_ld,
            flag)
    return grad


_device_of, _is_contiguous = torch.Tensor.get_device, torch.Tensor.is_contiguous
_data_ptr, _numel = torch.Tensor.data_ptr, torch.Tensor.numel
_dtype_of, _shape_of = operator.attrgetter("dtype"), operator.attrgetter("shape")


class _Lists:
    """Lists of tensors, one tensor of every list for each parameter, as arrays of pointers for a C
    entry.  The checks run over all of them at once, by functions that need no Python in
    between; only a failing one asks which list it was."""

    def __init__(self, **lists):
        self.lists = lists = {k: v for k, v in lists.items() if v is not None}
        self.n = n = len(next(iter(lists.values())))
        self.all = ts = [t for part in lists.values() for t in part]
        if len(ts) != n * len(lists) or any(len(part) != n for part in lists.values()):
            raise ValueError(f"all lists must have {n} tensors: " +
                             ", ".join(f"{name} has {len(part)}" for name, part in lists.items()))
        devices = set(map(_device_of, ts))  # a TypeError for what is no tensor
        self.index = index = ts[0].get_device()
        if devices != {index} or index < 0:
            self._blame(lambda t: t.get_device() == index >= 0,
                        "must be CUDA tensors on one device, that of all others")
        if not all(map(_is_contiguous, ts)):
            self._blame(_is_contiguous, "must be contiguous")
        self.dtypes, self.numels = list(map(_dtype_of, ts)), list(map(_numel, ts))
        self.at = {name: slice(k * n, k * n + n) for k, name in enumerate(lists)}

    def _blame(self, fine, what):
        raise ValueError(next(f"{name} {what}" for name, part in self.lists.items()
                              if not all(map(fine, part))))

    def dtype(self, name, dtype=None):
        """The type of a list: of all its tensors, and the given one, if any."""
        got = self.dtypes[self.at[name]]
        dtype = got[0] if dtype is None else dtype
        if got.count(dtype) != self.n:
            raise TypeError(f"{name} must be {dtype} all")
        return dtype

    def elements(self, name, want):
        if self.numels[self.at[name]] != want:
            raise ValueError(f"{name} must have {want} elements")

    def arrays(self, sizes):
        """(what has to live until the call returns, the sizes' address, the lists' by name)."""
        held = array.array("Q", sizes + list(map(_data_ptr, self.all)))
        at, step = held.buffer_info()[0], 8 * self.n
        return held, at, {name: at + step * (k + 1) for k, name in enumerate(self.lists)}


def grad_norm_workspace_bytes(grads) -> int:
    """Bytes of workspace that grad_norm() needs for these gradients."""
    sizes = array.array("Q", map(_numel, grads))
    return int(lib().dflash2_grad_norm_workspace_bytes(len(grads), sizes.buffer_info()[0]))


def grad_norm(grads, out=None, workspace=None):
    """The 2-norm of a list of gradients together (fp32 or bf16, one type) -> [1] fp32, without
    waiting for it.  workspace: a uint8 CUDA tensor of at least grad_norm_workspace_bytes(grads)
    bytes, allocated for None; calls that may run at the same time each need one of their own."""
    if len(grads) == 0:
        raise ValueError("grad_norm needs at least one tensor")
    ts, L = _Lists(grads=grads), lib()
    code = _code(ts.dtype("grads"))
    dev = ts.all[0].device
    held, sizes, ptrs = ts.arrays(ts.numels)
    given = (out,)
    out, out_ptr = _out_on(out, "out", torch.float32, (1,), dev)
    ws, ws_bytes = None, 0
    if workspace is not None:
        ws, ws_bytes = _on(workspace, "workspace", torch.uint8, workspace.shape, ts.index), \
            workspace.numel()
    else:
        ws_bytes = L.dflash2_grad_norm_workspace_bytes(ts.n, sizes)
        if ws_bytes > 0:
            workspace = torch.empty((ws_bytes,), dtype=torch.uint8, device=dev)
            ws = workspace.data_ptr()
    _written(given)
    _launch(ts.index, L.dflash2_grad_norm, ts.n, ptrs["grads"], sizes, code, ws, ws_bytes, out_ptr)
    return out


def adamw(params, grads, exp_avg, exp_avg_sq, step, lr, beta1=0.9, beta2=0.999, eps=1e-8,
          weight_decay=0.01, master=None, exp_avg_scale=None, exp_avg_sq_scale=None, norm=None,
          max_norm=None, grad_scale=1.0, seed=None):
    """One AdamW step over lists of tensors, in place: params and grads (each fp32 or bf16, one
    type a list), exp_avg and exp_avg_sq fp32 of as many elements, or uint8 with the lists
    exp_avg_scale and exp_avg_sq_scale ([(numel + 31) // 32] uint8 each): states in 8 bits, zeros
    to begin with (state_encode and state_decode go from values to them and back).  master: fp32
    copies of bf16 params, which take the step.  step: the step's number, 1 for the first, or an int32 CUDA
    tensor [1] with it; lr: a number or an fp32 CUDA tensor [1] (both for captured graphs; a
    step below 1 or an lr that is not finite is refused, in a tensor nothing is changed).
    norm: the gradients' norm (grad_norm); where it is not finite, nothing is changed (and a step
    tensor should not be raised for that call: step += torch.isfinite(norm) ahead of it); with
    max_norm it clips grads * grad_scale.  seed: an integer, by which 8-bit states, and bf16
    params without master, are rounded up or down with odds by the distance (else to the
    nearest, where 8-bit states and small steps of bf16 params get stuck)."""
    if len(params) == 0:
        if any(v is not None and len(v) for v in (grads, exp_avg, exp_avg_sq, master, exp_avg_scale,
                                                  exp_avg_sq_scale)):
            raise ValueError("params is empty, other lists are not")
        return
    f32, n = torch.float32, len(params)
    small = exp_avg_scale is not None or exp_avg_sq_scale is not None
    lists = [params, grads, exp_avg, exp_avg_sq]
    if master is not None:
        lists.append(master)
    if small:
        lists += [exp_avg_scale, exp_avg_sq_scale]
    try:
        ts = [t for part in lists for t in part]
        at = ts[0].get_device()
        dtypes, numels = list(map(_dtype_of, ts)), list(map(_numel, ts))
        sizes, states = numels[:n], [torch.uint8 if small else f32] * (2 * n)
        copies = [] if master is None else [f32] * n
        blocks = [-(-k // 32) for k in sizes] * 2 if small else []
        fine = (at >= 0 and set(map(_device_of, ts)) == {at} and all(map(_is_contiguous, ts)) and
                dtypes == dtypes[:1] * n + dtypes[n:n + 1] * n + states + copies +
                [torch.uint8] * len(blocks) and
                numels[2 * n:] == sizes * (2 if master is None else 3) + blocks and
                list(map(_shape_of, grads)) == list(map(_shape_of, params)) and
                set(map(len, lists)) == {n})
    except (AttributeError, TypeError):  # no tensors, or no list
        fine = False
    if not fine:
        _blame_adamw(params, grads, exp_avg, exp_avg_sq, master, exp_avg_scale, exp_avg_sq_scale)
    param_code, grad_code = _code(dtypes[0]), _code(dtypes[n])
    step_at, step = _setting_on(step, "step", torch.int32, at)
    if step_at is None and not 1 <= step < 1 << 31:  # the entry takes 32 bits
        raise ValueError(f"step={step}: the first step is 1, the last one 2^31 - 1")
    lr_at, lr = _setting_on(lr, "lr", f32, at)
    norm_at = _on(norm, "norm", f32, (1,), at)
    # before the launch, which may fail when a part of it is under way
    increment_version(ts[:n] + ts[2 * n:])
    held = array.array("Q", sizes + list(map(_data_ptr, ts)))  # lives until the call returns
    p, by = held.buffer_info()[0], 8 * n
    more = p + 5 * by  # behind sizes and the first four lists
    scales = more if master is None else more + by
    _launch(at, lib().dflash2_adamw, n, p + by, p + 2 * by, p + 3 * by, p + 4 * by,
            None if master is None else more, scales if small else None,
            scales + by if small else None, p, param_code, grad_code, step_at, lr_at, step, lr,
            beta1, beta2, eps, weight_decay, norm_at, 0.0 if max_norm is None else max_norm,
            grad_scale, seed is not None, 0 if seed is None else seed & 0xffffffffffffffff)


def _blame_adamw(params, grads, exp_avg, exp_avg_sq, master, exp_avg_scale, exp_avg_sq_scale):
    """Raises what is wrong with adamw()'s lists, one after the other."""
    ts = _Lists(params=params, grads=grads, exp_avg=exp_avg, exp_avg_sq=exp_avg_sq, master=master,
                exp_avg_scale=exp_avg_scale, exp_avg_sq_scale=exp_avg_sq_scale)
    small = exp_avg_scale is not None or exp_avg_sq_scale is not None
    state = torch.uint8 if small else torch.float32
    _code(ts.dtype("params"))
    _code(ts.dtype("grads"))
    if list(map(_shape_of, grads)) != list(map(_shape_of, params)):
        raise ValueError("grads must have the shapes of params")
    sizes = ts.numels[:ts.n]
    for name, dtype in (("exp_avg", state), ("exp_avg_sq", state), ("master", torch.float32)):
        if name in ts.lists:
            ts.dtype(name, dtype)
            ts.elements(name, sizes)
    for name in ("exp_avg_scale", "exp_avg_sq_scale"):
        if name not in ts.lists:
            raise ValueError("states in 8 bits need exp_avg_scale and exp_avg_sq_scale")
        ts.dtype(name, torch.uint8)
        ts.elements(name, [-(-n // 32) for n in sizes])
    raise ValueError("the lists of tensors do not go together")


def _setting_on(v, name, dtype, index):
    """(pointer, number) of a setting given as a tensor [1] on the device or as a number."""
    if isinstance(v, torch.Tensor):
        return _on(v, name, dtype, (1,), index), 0
    return None, v


def state_decode(codes, scale, squares=False, dtype=torch.float32, out=None):
    """The values of an 8-bit state of adamw(): codes uint8 of any shape, scale uint8
    [(numel + 31) // 32]; squares=True for exp_avg_sq.  Exact in fp32 and bf16."""
    index = codes.get_device()
    if index < 0:
        raise ValueError("codes must be a CUDA tensor")
    n = codes.numel()
    c = _on(codes, "codes", torch.uint8, codes.shape, index)
    s = _on(scale, "scale", torch.uint8, (-(-n // 32),), index)
    dtype = out.dtype if out is not None else dtype
    code = _code(dtype)
    given = (out,)
    out, out_ptr = _out_on(out, "out", dtype, codes.shape, codes.device)
    _written(given)
    _launch(index, lib().dflash2_state_decode, c, s, n, squares, code, out_ptr)
    return out


def state_encode(values, squares=False, codes=None, scale=None):
    """An 8-bit state of adamw() from values (fp32 or bf16, contiguous), to the nearest:
    (codes uint8 of the same shape, scale uint8 [(numel + 31) // 32])."""
    index = values.get_device()
    if index < 0:
        raise ValueError("values must be a CUDA tensor")
    n = values.numel()
    v = _on(values, "values", values.dtype, values.shape, index)
    code, given = _code(values.dtype), (codes, scale)
    codes, c = _out_on(codes, "codes", torch.uint8, values.shape, values.device)
    scale, s = _out_on(scale, "scale", torch.uint8, (-(-n // 32),), values.device)
    _written(given)
    _launch(index, lib().dflash2_state_encode, v, code, n, squares, c, s)
    return codes, scale


def take_device_faults() -> int:
    """Read and clear the library's device fault word (synchronises the device)."""
    v = ctypes.c_int32(0)
    _check(lib().dflash2_take_device_faults(ctypes.byref(v)))
    return int(v.value)


def probe_gather(table, row_bytes: int, ids, out=None):
    """Measurement aid: out[i] (int32 view of a uint32) = XOR of the 32-bit words of
    row ids[i] of `table` viewed as [rows, row_bytes] bytes."""
    _need(table, "table")
    _need(ids, "ids", torch.int32)
    nbytes = table.numel() * table.element_size()
    rows = nbytes // int(row_bytes)
    n_ids = ids.numel()
    if out is None:
        out = torch.empty((n_ids,), dtype=torch.int32, device=ids.device)
    _need(out, "out", torch.int32)
    _check(lib().dflash2_probe_gather(_ptr(table), rows, int(row_bytes), _ptr(ids), n_ids,
                                      _ptr(out), _stream(ids.device)))
    return out


def select_plan(S: int, n: int, d: int, K: int, R: int, dtype=torch.bfloat16) -> dict:
    """How select() runs these shapes on the current device: {"fused": bool,
    "cluster_size", "clusters", "rows_per_block"}."""
    out = (ctypes.c_int * 4)()
    _check(lib().dflash2_select_plan(S, n, d, K, R, _code(dtype), out))
    return {"fused": bool(out[0]), "cluster_size": out[1], "clusters": out[2],
            "rows_per_block": out[3]}
