"""ctypes binding of libdflash2.so (the C ABI declared in include/dflash2.h).

Argument marshalling only: shapes and dtypes are read from torch tensors,
outputs are allocated with torch when the caller does not pass them, and the
call goes to the CUDA library on the tensors' current stream.  There is no
fallback: if the library is missing or a call fails, an exception is raised.
"""
from __future__ import annotations

import ctypes
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
