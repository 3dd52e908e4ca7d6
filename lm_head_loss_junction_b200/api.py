"""Torch-tensor front end of libmls.

Each function checks tensor shapes/dtypes, allocates outputs with torch when
the caller does not pass them, and forwards raw pointers to the C ABI of the
same name (``mls_*``).  Every step of the computation runs in the library's
CUDA kernels; nothing here computes.
"""
from __future__ import annotations

import ctypes
import functools
from typing import List, Optional, Sequence, Tuple

import torch

from . import _lib
from ._lib import MLS_BF16, MLS_F32, check, i64_array, lib, ptr_array


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return MLS_BF16
    if t.dtype == torch.float32:
        return MLS_F32
    raise TypeError(f"unsupported dtype {t.dtype}; expected bfloat16 or float32")


def _stream_ptr(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _need(t: torch.Tensor, name: str, dtype=None, ndim=None):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims")


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


# ---------------------------------------------------------------- junction
def junction_fwd(x: torch.Tensor, o: torch.Tensor, E: torch.Tensor, *, out=None, scale_out=None,
                 variant: int = 0, status=None, stream=None) -> torch.Tensor:
    """y = [ (||E[x]|| / ||o||) o ; E[x] ] per token (see mls_junction_fwd; `variant`
    selects an ablation, see mls_junction_fwd_variant)."""
    _need(x, "x", torch.int32, 1)
    _need(o, "o", ndim=2)
    _need(E, "E", o.dtype, 2)
    T, D = o.shape
    V, delta = E.shape
    if x.shape[0] != T:
        raise ValueError("x and o disagree on T")
    y = out if out is not None else torch.empty((T, D + delta), dtype=o.dtype, device=o.device)
    _need(y, "out", o.dtype, 2)
    if scale_out is not None:
        _need(scale_out, "scale_out", torch.float32, 1)
    if variant:
        code = lib().mls_junction_fwd_variant(x.data_ptr(), T, o.data_ptr(), D, E.data_ptr(), V, delta,
                                              y.data_ptr(), _ptr(scale_out), int(variant), _dtype_code(o),
                                              _ptr(status), _stream_ptr(stream))
    else:
        code = lib().mls_junction_fwd(x.data_ptr(), T, o.data_ptr(), D, E.data_ptr(), V, delta, y.data_ptr(),
                                      _ptr(scale_out), _dtype_code(o), _ptr(status), _stream_ptr(stream))
    check("mls_junction_fwd", code)
    return y


def junction_bwd_workspace(T: int, V: int) -> int:
    n = ctypes.c_size_t()
    check("mls_junction_bwd_workspace", lib().mls_junction_bwd_workspace(T, V, ctypes.byref(n)))
    return n.value


def junction_bwd(x: torch.Tensor, o: torch.Tensor, E: torch.Tensor, dy: torch.Tensor, *,
                 want_de_rows: bool = True, dE: Optional[torch.Tensor] = None, accumulate_dE: bool = False,
                 do_out=None, de_out=None, workspace=None, variant: int = 0, status=None, stream=None):
    """Returns (do, de_rows or None, dE or None) (see mls_junction_bwd)."""
    _need(x, "x", torch.int32, 1)
    _need(o, "o", ndim=2)
    _need(E, "E", o.dtype, 2)
    _need(dy, "dy", o.dtype, 2)
    T, D = o.shape
    V, delta = E.shape
    if tuple(dy.shape) != (T, D + delta):
        raise ValueError("dy must be [T, D + delta]")
    do = do_out if do_out is not None else torch.empty_like(o)
    de = de_out
    if de is None and want_de_rows:
        de = torch.empty((T, delta), dtype=o.dtype, device=o.device)
    ws_bytes = 0
    if dE is not None:
        _need(dE, "dE", torch.float32, 2)
        ws_bytes = junction_bwd_workspace(T, V)
        if workspace is None:
            workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=o.device)
        ws_bytes = workspace.numel() * workspace.element_size()
    if variant:
        code = lib().mls_junction_bwd_variant(x.data_ptr(), T, o.data_ptr(), D, E.data_ptr(), V, delta,
                                              dy.data_ptr(), do.data_ptr(), _ptr(de), _ptr(dE),
                                              int(bool(accumulate_dE)), _ptr(workspace), ws_bytes, int(variant),
                                              _dtype_code(o), _ptr(status), _stream_ptr(stream))
    else:
        code = lib().mls_junction_bwd(x.data_ptr(), T, o.data_ptr(), D, E.data_ptr(), V, delta, dy.data_ptr(),
                                      do.data_ptr(), _ptr(de), _ptr(dE), int(bool(accumulate_dE)),
                                      _ptr(workspace), ws_bytes, _dtype_code(o), _ptr(status),
                                      _stream_ptr(stream))
    check("mls_junction_bwd", code)
    return do, de, dE


def junction_fwd_multi(x: torch.Tensor, o: Sequence[torch.Tensor], E: Sequence[torch.Tensor], *, out=None,
                       scale_out=None, status=None, stream=None) -> List[torch.Tensor]:
    """Every junction of a suite in one call: y[k] = junction(o[k], E[k]) (see mls_junction_fwd_multi)."""
    J = len(o)
    if len(E) != J or J < 1:
        raise ValueError("o and E must be non-empty lists of the same length")
    _need(x, "x", torch.int32, 1)
    T = x.shape[0]
    V = E[0].shape[0]
    D = [o[0].shape[1]]
    for k in range(J):
        _need(o[k], f"o[{k}]", o[0].dtype, 2)
        _need(E[k], f"E[{k}]", o[0].dtype, 2)
        if o[k].shape[0] != T or E[k].shape[0] != V or o[k].shape[1] != D[k]:
            raise ValueError(f"junction {k}: o must be [T, D_k] (D_k the previous junction's output width)")
        D.append(D[k] + E[k].shape[1])
    y = out if out is not None else [torch.empty((T, D[k + 1]), dtype=o[0].dtype, device=x.device)
                                     for k in range(J)]
    for k in range(J):
        _need(y[k], f"out[{k}]", o[0].dtype, 2)
    sc = None
    if scale_out is not None:
        sc = ptr_array([_ptr(t) for t in scale_out])
    code = lib().mls_junction_fwd_multi(x.data_ptr(), T, V, J, i64_array(D), ptr_array([t.data_ptr() for t in o]),
                                        ptr_array([t.data_ptr() for t in E]), ptr_array([t.data_ptr() for t in y]),
                                        sc, _dtype_code(o[0]), _ptr(status), _stream_ptr(stream))
    check("mls_junction_fwd_multi", code)
    return y


def junction_bwd_multi_workspace(T: int, V: int, J: int) -> int:
    n = ctypes.c_size_t()
    check("mls_junction_bwd_multi_workspace", lib().mls_junction_bwd_multi_workspace(T, V, J, ctypes.byref(n)))
    return n.value


def junction_bwd_multi(x: torch.Tensor, o: Sequence[torch.Tensor], E: Sequence[torch.Tensor],
                       dy: Sequence[torch.Tensor], *, do_out=None, de_out=None, dE=None, accumulate_dE=False,
                       workspace=None, status=None, stream=None):
    """Backward of every junction of a suite in one call (see mls_junction_bwd_multi).
    de_out / dE: lists (entries may be None) or None.  Returns (do list, de list, dE list)."""
    J = len(o)
    _need(x, "x", torch.int32, 1)
    T = x.shape[0]
    V = E[0].shape[0]
    D = [o[0].shape[1]] + [o[0].shape[1]] * J
    for k in range(J):
        D[k + 1] = D[k] + E[k].shape[1]
        if tuple(dy[k].shape) != (T, D[k + 1]):
            raise ValueError(f"dy[{k}] must be [T, D_k+1]")
    do = do_out if do_out is not None else [torch.empty_like(t) for t in o]
    de = de_out if de_out is not None else [None] * J
    tables = dE if dE is not None else [None] * J
    ws_bytes = 0
    if any(t is not None for t in tables):
        ws_bytes = junction_bwd_multi_workspace(T, V, J)
        if workspace is None:
            workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=x.device)
        ws_bytes = workspace.numel() * workspace.element_size()
    code = lib().mls_junction_bwd_multi(x.data_ptr(), T, V, J, i64_array(D), ptr_array([t.data_ptr() for t in o]),
                                        ptr_array([t.data_ptr() for t in E]), ptr_array([t.data_ptr() for t in dy]),
                                        ptr_array([t.data_ptr() for t in do]), ptr_array([_ptr(t) for t in de]),
                                        ptr_array([_ptr(t) for t in tables]), int(bool(accumulate_dE)),
                                        _ptr(workspace), ws_bytes, _dtype_code(o[0]), _ptr(status),
                                        _stream_ptr(stream))
    check("mls_junction_bwd_multi", code)
    return do, de, tables


# ---------------------------------------------------------------- multi-exit loss
def multiexit_loss_workspace(T: int, D: Sequence[int], V: int, dtype: torch.dtype) -> Tuple[int, int]:
    f = ctypes.c_size_t()
    b = ctypes.c_size_t()
    code = lib().mls_multiexit_loss_workspace(len(D), T, i64_array(D), V,
                                              MLS_BF16 if dtype == torch.bfloat16 else MLS_F32,
                                              ctypes.byref(f), ctypes.byref(b))
    check("mls_multiexit_loss_workspace", code)
    return f.value, b.value


def multiexit_loss_bwd_plan(T: int, D: Sequence[int], V: int, dtype: torch.dtype, ws_bytes: int):
    """(Tb, Vc, min_bytes): how the backward call splits its work for a workspace of ws_bytes
    (see mls_multiexit_loss_bwd_plan)."""
    tb = ctypes.c_int64()
    vc = ctypes.c_int64()
    mn = ctypes.c_size_t()
    code = lib().mls_multiexit_loss_bwd_plan(len(D), T, i64_array(D), V,
                                             MLS_BF16 if dtype == torch.bfloat16 else MLS_F32, int(ws_bytes),
                                             ctypes.byref(tb), ctypes.byref(vc), ctypes.byref(mn))
    check("mls_multiexit_loss_bwd_plan", code)
    return tb.value, vc.value, mn.value


def _loss_common(y, h, W):
    M = len(h)
    if len(W) != M or M < 1:
        raise ValueError("h and W must be non-empty lists of the same length")
    _need(y, "y", torch.int32, 1)
    T = y.shape[0]
    V = W[0].shape[0]
    dt = h[0].dtype
    D = []
    for m in range(M):
        _need(h[m], f"h[{m}]", dt, 2)
        _need(W[m], f"W[{m}]", dt, 2)
        if h[m].shape[0] != T or W[m].shape[0] != V or h[m].shape[1] != W[m].shape[1]:
            raise ValueError(f"exit {m}: h must be [T, D_m] and W [V, D_m]")
        D.append(h[m].shape[1])
    return M, T, V, D, dt


def _workspace(ws, nbytes, device):
    if ws is None:
        ws = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=device)
    return ws, ws.numel() * ws.element_size()


def multiexit_loss_fwd(y: torch.Tensor, h: List[torch.Tensor], W: List[torch.Tensor], alpha_d: float = 0.3, *,
                       losses=None, stats=None, workspace=None, exit_weights=None, distill="ce",
                       teacher_grad: bool = False, status=None, stream=None):
    """Returns (losses [2M], stats [3M-1, T], or [4M-2, T] for Jensen-Shannon or acceptance
    with the teacher gradient) (see mls_multiexit_loss_fwd; any option uses mls_multiexit_loss_fwd_opts)."""
    M, T, V, D, dt = _loss_common(y, h, W)
    dev = y.device
    if losses is None:
        losses = torch.empty(2 * M, dtype=torch.float32, device=dev)
    rows = 4 * M - 2 if (distill in ("js", "accept") and teacher_grad and M > 1) else 3 * M - 1
    if stats is None:
        stats = torch.empty((rows, T), dtype=torch.float32, device=dev)
    elif stats.shape[0] < rows:
        raise ValueError(f"stats needs {rows} rows")
    fwd_b, _ = multiexit_loss_workspace(T, D, V, dt)
    workspace, ws_bytes = _workspace(workspace, fwd_b, dev)
    args = (M, T, V, i64_array(D), y.data_ptr(), ptr_array([t.data_ptr() for t in h]),
            ptr_array([t.data_ptr() for t in W]), float(alpha_d), _dtype_code(h[0]), losses.data_ptr(),
            stats.data_ptr(), workspace.data_ptr(), ws_bytes)
    opts = _lib.loss_options(exit_weights, distill, teacher_grad)
    if opts is None:
        code = lib().mls_multiexit_loss_fwd(*args, _ptr(status), _stream_ptr(stream))
    else:
        code = lib().mls_multiexit_loss_fwd_opts(*args, ctypes.byref(opts), _ptr(status), _stream_ptr(stream))
    check("mls_multiexit_loss_fwd", code)
    return losses, stats


def multiexit_loss_bwd(y: torch.Tensor, h: List[torch.Tensor], W: List[torch.Tensor], stats: torch.Tensor,
                       alpha_d: float = 0.3, grad_scale: float = 1.0, *, dh=None, dW=None,
                       accumulate_dW: bool = False, workspace=None, exit_weights=None, distill="ce",
                       teacher_grad: bool = False, status=None, stream=None):
    """Returns (dh list, dW list) (see mls_multiexit_loss_bwd)."""
    M, T, V, D, dt = _loss_common(y, h, W)
    dev = y.device
    _need(stats, "stats", torch.float32, 2)
    if dh is None:
        dh = [torch.empty_like(t) for t in h]
    if dW is None:
        dW = [torch.empty((V, d), dtype=torch.float32, device=dev) for d in D]
    _, bwd_b = multiexit_loss_workspace(T, D, V, dt)
    workspace, ws_bytes = _workspace(workspace, bwd_b, dev)
    args = (M, T, V, i64_array(D), y.data_ptr(), ptr_array([t.data_ptr() for t in h]),
            ptr_array([t.data_ptr() for t in W]), float(alpha_d), _dtype_code(h[0]), stats.data_ptr(),
            float(grad_scale), ptr_array([t.data_ptr() for t in dh]), ptr_array([t.data_ptr() for t in dW]),
            int(bool(accumulate_dW)), workspace.data_ptr(), ws_bytes)
    opts = _lib.loss_options(exit_weights, distill, teacher_grad)
    if opts is None:
        code = lib().mls_multiexit_loss_bwd(*args, _ptr(status), _stream_ptr(stream))
    else:
        code = lib().mls_multiexit_loss_bwd_opts(*args, ctypes.byref(opts), _ptr(status), _stream_ptr(stream))
    check("mls_multiexit_loss_bwd", code)
    return dh, dW


def exit_agreement(h: List[torch.Tensor], W: List[torch.Tensor], stats: torch.Tensor, *, per_token=False,
                   want_top1=False, workspace=None, status=None, stream=None):
    """Agreement of every smaller exit with the largest (see mls_exit_agreement).

    Returns (metrics [3(M-1)] = mean beta, mean KL, mean top-1 agreement per
    smaller exit, per-token rows [3(M-1), T] or None, top-1 ids [M, T] or None).
    """
    M = len(h)
    if len(W) != M or M < 2:
        raise ValueError("need at least two exits")
    T, V, dt = h[0].shape[0], W[0].shape[0], h[0].dtype
    D = []
    for m in range(M):
        _need(h[m], f"h[{m}]", dt, 2)
        _need(W[m], f"W[{m}]", dt, 2)
        D.append(h[m].shape[1])
    _need(stats, "stats", torch.float32, 2)
    dev = h[0].device
    metrics = torch.empty(3 * (M - 1), dtype=torch.float32, device=dev)
    rows = torch.empty((3 * (M - 1), T), dtype=torch.float32, device=dev) if per_token else None
    top1 = torch.empty((M, T), dtype=torch.int32, device=dev) if want_top1 else None
    n = ctypes.c_size_t()
    check("mls_exit_agreement_workspace",
          lib().mls_exit_agreement_workspace(M, T, i64_array(D), V, _dtype_code(h[0]), ctypes.byref(n)))
    workspace, ws_bytes = _workspace(workspace, n.value, dev)
    code = lib().mls_exit_agreement(M, T, V, i64_array(D), ptr_array([t.data_ptr() for t in h]),
                                    ptr_array([t.data_ptr() for t in W]), _dtype_code(h[0]), stats.data_ptr(),
                                    metrics.data_ptr(), _ptr(rows), _ptr(top1), workspace.data_ptr(), ws_bytes,
                                    _ptr(status), _stream_ptr(stream))
    check("mls_exit_agreement", code)
    return metrics, rows, top1


# ---------------------------------------------------------------- single-exit LM-head operators
# A decoding step's call is shorter on the GPU than a careless wrapper is on the host, so these check each
# tensor with one expression, ask for the sizes of a shape once and take the raw stream.
def _head_fit(t, name, dtype, shape, dev):
    """Checks a tensor given by the caller: contiguous, of the dtype and shape, on the device of h."""
    if t.dtype is dtype and t.shape == shape and t.device == dev and t.is_contiguous():
        return
    _need(t, name, dtype)
    if t.device != dev:
        raise ValueError(f"{name} must be on the device of h")
    raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _head_common(h, W):
    _need(h, "h", ndim=2)
    _need(W, "W", h.dtype, 2)
    (T, D), (V, DW) = h.shape, W.shape
    if D != DW:
        raise ValueError("h must be [T, D] and W [V, D]")
    if W.device != h.device:
        raise ValueError("W must be on the device of h")
    return T, D, V, _dtype_code(h), h.device


def _head_stream(dev):
    return torch._C._cuda_getCurrentRawStream(dev.index)


def _head_ids(ids, T, dev):
    if ids.dim() not in (1, 2) or ids.shape[0] != T:
        raise ValueError("ids must be [T] or [T, N]")
    _head_fit(ids, "ids", torch.int32, ids.shape, dev)
    return 1 if ids.dim() == 1 else ids.shape[1]


def _head_workspace(ws, nbytes, dev):
    if ws is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=dev), nbytes
    _head_fit(ws, "workspace", ws.dtype, ws.shape, dev)
    return ws, ws.numel() * ws.element_size()


def _head_status(status, dev):
    """A word at least: flags would be lost in an empty tensor, or set in what lies behind an empty view."""
    if status is None:
        return
    _head_fit(status, "status", torch.int32, status.shape, dev)
    if status.numel() == 0:
        raise ValueError("status must have an element")


def _head_grads(h, W, dh, dW, dW_dtype, accumulate_dW, want_dh, want_dW):
    if not want_dh and dh is not None or not want_dW and dW is not None:
        raise ValueError("an output was given for a gradient that is not wanted")
    if dh is not None:
        _head_fit(dh, "dh", h.dtype, h.shape, h.device)
    elif want_dh:
        dh = torch.empty_like(h)
    if dW is not None:
        _head_fit(dW, "dW", dW.dtype, W.shape, h.device)
    elif want_dW:
        if accumulate_dW:
            raise ValueError("accumulate_dW needs dW")
        dW = torch.empty(*W.shape, dtype=dW_dtype, device=W.device)
    return dh, dW, _dtype_code(dW) if dW is not None else MLS_F32


def _elsewhere(h, stream):
    """Whether a call has to change the current device or stream first."""
    return stream is not None or h.is_cuda and h.device.index != torch.cuda.current_device()


def _moved(fn, h, stream, *args, **kw):
    """fn(*args, **kw) with the device of h current and, where one is given, on `stream`: launches and allocations
    both (a workspace from another stream's pool could be handed out again while this one still uses it)."""
    if stream is None:
        with torch.cuda.device(h.device):
            return fn(*args, **kw)
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=h.device)
    if stream.device != h.device:
        raise ValueError("stream must be of the device of h")
    with torch.cuda.stream(stream):
        return fn(*args, **kw)


def _code_of(dtype):
    return MLS_BF16 if dtype == torch.bfloat16 else MLS_F32


@functools.lru_cache(maxsize=1024)
def token_logprobs_workspace(T: int, D: int, V: int, N: int, top_k: int, dtype: torch.dtype) -> Tuple[int, int]:
    """(bytes, smallest accepted bytes) of token_logprobs (see mls_token_logprobs_workspace)."""
    n, least = ctypes.c_size_t(), ctypes.c_size_t()
    check("mls_token_logprobs_workspace",
          lib().mls_token_logprobs_workspace(T, D, V, N, top_k, _code_of(dtype), ctypes.byref(n),
                                             ctypes.byref(least)))
    return n.value, least.value


def token_logprobs(ids: Optional[torch.Tensor], h: torch.Tensor, W: torch.Tensor, *, top_k: int = 0, logp=None,
                   stats=None, top_ids=None, top_logp=None, workspace=None, status=None, stream=None):
    """Log probabilities of given tokens under softmax(h W^T), the entropy of that distribution and its top
    alternatives, without a T x V result (see mls_token_logprobs).

    ids: int32 [T] or [T, N] (-1: no token there), or None with top_k > 0.  Returns (logp of the shape of ids or
    None, stats [2, T] = log-sum-exp and entropy, top_ids [T, top_k] or None, top_logp [T, top_k] or None).
    """
    if _elsewhere(h, stream):
        return _moved(token_logprobs, h, stream, ids, h, W, top_k=top_k, logp=logp, stats=stats, top_ids=top_ids,
                      top_logp=top_logp, workspace=workspace, status=status)
    T, D, V, dt, dev = _head_common(h, W)
    f32 = torch.float32
    N = 0
    if ids is not None:
        N = _head_ids(ids, T, dev)
    elif logp is not None:
        raise ValueError("logp was given without ids")
    if not top_k and (top_ids is not None or top_logp is not None):
        raise ValueError("top_ids or top_logp was given without top_k")
    nbytes = token_logprobs_workspace(T, D, V, N, top_k, h.dtype)[0]
    if logp is not None:
        _head_fit(logp, "logp", f32, ids.shape, dev)
    elif N:
        logp = torch.empty(*ids.shape, dtype=f32, device=dev)
    if stats is not None:
        _head_fit(stats, "stats", f32, (2, T), dev)
    else:
        stats = torch.empty(2, T, dtype=f32, device=dev)
    if top_ids is not None:
        _head_fit(top_ids, "top_ids", torch.int32, (T, top_k), dev)
    elif top_k:
        top_ids = torch.empty(T, top_k, dtype=torch.int32, device=dev)
    if top_logp is not None:
        _head_fit(top_logp, "top_logp", f32, (T, top_k), dev)
    elif top_k:
        top_logp = torch.empty(T, top_k, dtype=f32, device=dev)
    _head_status(status, dev)
    workspace, ws_bytes = _head_workspace(workspace, nbytes, dev)
    check("mls_token_logprobs",
          lib().mls_token_logprobs(T, D, V, N, _ptr(ids), h.data_ptr(), W.data_ptr(), dt, _ptr(logp),
                                   stats.data_ptr(), top_k, _ptr(top_ids), _ptr(top_logp), workspace.data_ptr(),
                                   ws_bytes, _ptr(status), _head_stream(dev)))
    return logp, stats, top_ids, top_logp


@functools.lru_cache(maxsize=1024)
def token_logprobs_bwd_workspace(T: int, D: int, V: int, N: int, dtype: torch.dtype) -> Tuple[int, int]:
    """(bytes, smallest accepted bytes) of token_logprobs_bwd (see mls_token_logprobs_bwd_workspace)."""
    n, least = ctypes.c_size_t(), ctypes.c_size_t()
    check("mls_token_logprobs_bwd_workspace",
          lib().mls_token_logprobs_bwd_workspace(T, D, V, N, _code_of(dtype), ctypes.byref(n), ctypes.byref(least)))
    return n.value, least.value


def token_logprobs_bwd(ids: torch.Tensor, h: torch.Tensor, W: torch.Tensor, stats: torch.Tensor,
                       g_logp: torch.Tensor, g_entropy: Optional[torch.Tensor] = None, *, dh=None, dW=None,
                       dW_dtype: torch.dtype = torch.float32, accumulate_dW: bool = False, want_dh: bool = True,
                       want_dW: bool = True, workspace=None, status=None, stream=None):
    """Gradients of token_logprobs' log probabilities (g_logp, the shape of ids) and entropies (g_entropy [T])
    with respect to h and W (see mls_token_logprobs_bwd).  Returns (dh or None, dW or None); dW is fp32, or
    bf16 with dW_dtype=torch.bfloat16."""
    if _elsewhere(h, stream):
        return _moved(token_logprobs_bwd, h, stream, ids, h, W, stats, g_logp, g_entropy, dh=dh, dW=dW,
                      dW_dtype=dW_dtype, accumulate_dW=accumulate_dW, want_dh=want_dh, want_dW=want_dW,
                      workspace=workspace, status=status)
    T, D, V, dt, dev = _head_common(h, W)
    N = _head_ids(ids, T, dev)
    _head_fit(stats, "stats", torch.float32, (2, T), dev)
    _head_fit(g_logp, "g_logp", torch.float32, ids.shape, dev)
    if g_entropy is not None:
        _head_fit(g_entropy, "g_entropy", torch.float32, (T,), dev)
    _head_status(status, dev)
    dh, dW, dW_code = _head_grads(h, W, dh, dW, dW_dtype, accumulate_dW, want_dh, want_dW)
    workspace, ws_bytes = _head_workspace(workspace, token_logprobs_bwd_workspace(T, D, V, N, h.dtype)[0], dev)
    check("mls_token_logprobs_bwd",
          lib().mls_token_logprobs_bwd(T, D, V, N, ids.data_ptr(), h.data_ptr(), W.data_ptr(), dt,
                                       stats.data_ptr(), g_logp.data_ptr(), _ptr(g_entropy), _ptr(dh), _ptr(dW),
                                       dW_code, int(bool(accumulate_dW)), workspace.data_ptr(), ws_bytes,
                                       _ptr(status), _head_stream(dev)))
    return dh, dW


@functools.lru_cache(maxsize=1024)
def topk_distill_workspace(T: int, D: int, V: int, K: int, dtype: torch.dtype) -> Tuple[int, int, int, int]:
    """(forward bytes, smallest, backward bytes, smallest) of the distillation (see mls_topk_distill_workspace)."""
    v = [ctypes.c_size_t() for _ in range(4)]
    check("mls_topk_distill_workspace",
          lib().mls_topk_distill_workspace(T, D, V, K, _code_of(dtype), *[ctypes.byref(x) for x in v]))
    return tuple(x.value for x in v)


def _distill_common(y, teacher_ids, teacher_logits, token_weights, h, W, status):
    T, D, V, dt, dev = _head_common(h, W)
    if teacher_ids.dim() != 2:
        raise ValueError("teacher_ids must be [T, K]")
    K = teacher_ids.shape[1]
    _head_fit(y, "y", torch.int32, (T,), dev)
    _head_fit(teacher_ids, "teacher_ids", torch.int32, (T, K), dev)
    _head_fit(teacher_logits, "teacher_logits", torch.float32, (T, K), dev)
    if token_weights is not None:
        _head_fit(token_weights, "token_weights", torch.float32, (T,), dev)
    _head_status(status, dev)
    return T, D, V, K, dt, dev


def topk_distill_fwd(y: torch.Tensor, teacher_ids: torch.Tensor, teacher_logits: torch.Tensor, h: torch.Tensor,
                     W: torch.Tensor, alpha_d: float = 0.3, *, token_weights: Optional[torch.Tensor] = None,
                     losses=None, stats=None, workspace=None, status=None, stream=None):
    """Next-token cross-entropy mixed with the cross-entropy to a teacher's top logits (teacher_ids int32 [T, K],
    -1 where absent; teacher_logits f32 [T, K]; see mls_topk_distill_fwd).

    Returns (losses [3] = mean cross-entropy, mean distillation term, their mix; stats [3, T] = log-sum-exp and
    the two terms of every token)."""
    if _elsewhere(h, stream):
        return _moved(topk_distill_fwd, h, stream, y, teacher_ids, teacher_logits, h, W, alpha_d,
                      token_weights=token_weights, losses=losses, stats=stats, workspace=workspace, status=status)
    T, D, V, K, dt, dev = _distill_common(y, teacher_ids, teacher_logits, token_weights, h, W, status)
    nbytes = topk_distill_workspace(T, D, V, K, h.dtype)[0]
    if losses is not None:
        _head_fit(losses, "losses", torch.float32, (3,), dev)
    else:
        losses = torch.empty(3, dtype=torch.float32, device=dev)
    if stats is not None:
        _head_fit(stats, "stats", torch.float32, (3, T), dev)
    else:
        stats = torch.empty(3, T, dtype=torch.float32, device=dev)
    workspace, ws_bytes = _head_workspace(workspace, nbytes, dev)
    check("mls_topk_distill_fwd",
          lib().mls_topk_distill_fwd(T, D, V, K, y.data_ptr(), teacher_ids.data_ptr(), teacher_logits.data_ptr(),
                                     _ptr(token_weights), h.data_ptr(), W.data_ptr(), float(alpha_d), dt,
                                     losses.data_ptr(), stats.data_ptr(), workspace.data_ptr(), ws_bytes,
                                     _ptr(status), _head_stream(dev)))
    return losses, stats


def topk_distill_bwd(y: torch.Tensor, teacher_ids: torch.Tensor, teacher_logits: torch.Tensor, h: torch.Tensor,
                     W: torch.Tensor, stats: torch.Tensor, alpha_d: float = 0.3, grad_scale: float = 1.0, *,
                     token_weights: Optional[torch.Tensor] = None, dh=None, dW=None,
                     dW_dtype: torch.dtype = torch.float32, accumulate_dW: bool = False, want_dh: bool = True,
                     want_dW: bool = True, workspace=None, status=None, stream=None):
    """Gradients of topk_distill_fwd's mixed loss times grad_scale with respect to h and W (see
    mls_topk_distill_bwd).  Returns (dh or None, dW or None)."""
    if _elsewhere(h, stream):
        return _moved(topk_distill_bwd, h, stream, y, teacher_ids, teacher_logits, h, W, stats, alpha_d, grad_scale,
                      token_weights=token_weights, dh=dh, dW=dW, dW_dtype=dW_dtype, accumulate_dW=accumulate_dW,
                      want_dh=want_dh, want_dW=want_dW, workspace=workspace, status=status)
    T, D, V, K, dt, dev = _distill_common(y, teacher_ids, teacher_logits, token_weights, h, W, status)
    _head_fit(stats, "stats", torch.float32, (3, T), dev)
    dh, dW, dW_code = _head_grads(h, W, dh, dW, dW_dtype, accumulate_dW, want_dh, want_dW)
    workspace, ws_bytes = _head_workspace(workspace, topk_distill_workspace(T, D, V, K, h.dtype)[2], dev)
    check("mls_topk_distill_bwd",
          lib().mls_topk_distill_bwd(T, D, V, K, y.data_ptr(), teacher_ids.data_ptr(), teacher_logits.data_ptr(),
                                     _ptr(token_weights), h.data_ptr(), W.data_ptr(), float(alpha_d), dt,
                                     stats.data_ptr(), float(grad_scale), _ptr(dh), _ptr(dW), dW_code,
                                     int(bool(accumulate_dW)), workspace.data_ptr(), ws_bytes, _ptr(status),
                                     _head_stream(dev)))
    return dh, dW


def status_read(status: torch.Tensor, stream=None) -> Tuple[int, int]:
    """Synchronises, returns (status code, raw flag word) and clears the word."""
    out = ctypes.c_int32()
    code = lib().mls_status_read(status.data_ptr(), _stream_ptr(stream), ctypes.byref(out))
    return code, out.value


def new_status(device="cuda") -> torch.Tensor:
    return torch.zeros(1, dtype=torch.int32, device=device)
