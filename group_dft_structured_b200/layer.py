"""Torch-facing convenience around the C ABI: allocates outputs, the Fourier
weight buffer and the dW workspace with torch (device memory only) and calls
the library.  No arithmetic happens here.
"""

from __future__ import annotations

import contextlib

import torch

from . import (FEQL_ACT_NONE, FEQL_FP16, FEQL_FP16_SIMT, FEQL_FP32, feql_backward,
               feql_backward_dw, feql_backward_dw_workspace_bytes, feql_backward_dx,
               feql_ct_backward_act, feql_ct_backward_act_workspace_bytes, feql_ct_backward_dw,
               feql_ct_backward_dw_workspace_bytes, feql_ct_backward_dx, feql_ct_forward,
               feql_ct_forward_act, feql_ct_weight_fft, feql_ct_weight_fft_bytes, feql_forward,
               feql_mlp_forward, feql_mlp_weight_fft, feql_mlp_weight_fft_bytes,
               feql_norm_backward, feql_norm_backward_workspace_bytes, feql_norm_forward,
               feql_p4m_backward_act, feql_p4m_backward_act_workspace_bytes, feql_p4m_backward_dw,
               feql_p4m_backward_dw_workspace_bytes, feql_p4m_backward_dx, feql_p4m_forward,
               feql_p4m_forward_act, feql_p4m_weight_fft, feql_p4m_weight_fft_bytes,
               feql_scan_backward, feql_scan_backward_diff, feql_scan_forward,
               feql_scan_forward_diff, feql_scan_step, feql_scan_workspace_bytes,
               feql_weight_fft, feql_weight_fft_bytes)


def torch_dtype(mode: int):
    return torch.float16 if mode in (FEQL_FP16, FEQL_FP16_SIMT) else torch.float32


def weight_fft(W: torch.Tensor, mode: int, stream=None) -> torch.Tensor:
    D, C, _ = W.shape
    nbytes = feql_weight_fft_bytes(C, D, mode)
    if nbytes == 0:
        raise ValueError("unsupported (C, D, mode)")
    What = torch.empty(nbytes, dtype=torch.uint8, device=W.device)
    feql_weight_fft(W, What, C, D, mode, stream)
    return What


def forward(x: torch.Tensor, What: torch.Tensor, b, D: int, mode: int, out=None,
            stream=None) -> torch.Tensor:
    N, C, _ = x.shape
    y = out if out is not None else torch.empty((N, D, 4), dtype=x.dtype, device=x.device)
    feql_forward(x, What, b, y, N, C, D, mode, stream)
    return y


def backward_dx(dy: torch.Tensor, What: torch.Tensor, C: int, mode: int, out=None,
                stream=None) -> torch.Tensor:
    N, D, _ = dy.shape
    dx = out if out is not None else torch.empty((N, C, 4), dtype=dy.dtype, device=dy.device)
    feql_backward_dx(dy, What, dx, N, C, D, mode, stream)
    return dx


def dw_workspace(N: int, C: int, D: int, mode: int, device) -> torch.Tensor:
    nbytes = feql_backward_dw_workspace_bytes(N, C, D, mode)
    return torch.empty(max(nbytes, 16), dtype=torch.uint8, device=device)


def backward(x: torch.Tensor, dy: torch.Tensor, What: torch.Tensor, mode: int, ws=None,
             with_db: bool = True, stream=None):
    """dx, dW, db from one call (fused single pass over dy where supported)."""
    N, C, _ = x.shape
    D = dy.shape[1]
    if ws is None:
        ws = dw_workspace(N, C, D, mode, x.device)
    dx = torch.empty((N, C, 4), dtype=x.dtype, device=x.device)
    dW = torch.empty((D, C, 4), dtype=x.dtype, device=x.device)
    db = torch.empty((D,), dtype=x.dtype, device=x.device) if with_db else None
    feql_backward(x, dy, What, dx, dW, db, ws, ws.numel(), N, C, D, mode, stream)
    return dx, dW, db


def backward_dw(x: torch.Tensor, dy: torch.Tensor, mode: int, ws=None, out=None,
                with_db: bool = True, stream=None):
    N, C, _ = x.shape
    D = dy.shape[1]
    if ws is None:
        ws = dw_workspace(N, C, D, mode, x.device)
    if out is None:
        dW = torch.empty((D, C, 4), dtype=x.dtype, device=x.device)
        db = torch.empty((D,), dtype=x.dtype, device=x.device) if with_db else None
    else:
        dW, db = out
    feql_backward_dw(x, dy, dW, db, ws, ws.numel(), N, C, D, mode, stream)
    return dW, db


# --------------------------------------------------------- cyclic group C_T
# The group order T is the length of the last axis (T = 4 goes to the p4 path).

def ct_weight_fft(W: torch.Tensor, mode: int, stream=None) -> torch.Tensor:
    D, C, T = W.shape
    nbytes = feql_ct_weight_fft_bytes(T, C, D, mode)
    if nbytes == 0:
        raise ValueError("unsupported (T, C, D, mode)")
    What = torch.empty(nbytes, dtype=torch.uint8, device=W.device)
    feql_ct_weight_fft(T, W, What, C, D, mode, stream)
    return What


def ct_forward(x: torch.Tensor, What: torch.Tensor, b, D: int, mode: int, stream=None):
    N, C, T = x.shape
    y = torch.empty((N, D, T), dtype=x.dtype, device=x.device)
    feql_ct_forward(T, x, What, b, y, N, C, D, mode, stream)
    return y


def ct_backward_dx(dy: torch.Tensor, What: torch.Tensor, C: int, mode: int, stream=None):
    N, D, T = dy.shape
    dx = torch.empty((N, C, T), dtype=dy.dtype, device=dy.device)
    feql_ct_backward_dx(T, dy, What, dx, N, C, D, mode, stream)
    return dx


def ct_backward_dw(x: torch.Tensor, dy: torch.Tensor, mode: int, with_db: bool = True,
                   stream=None):
    N, C, T = x.shape
    D = dy.shape[1]
    nbytes = feql_ct_backward_dw_workspace_bytes(T, N, C, D, mode)
    ws = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=x.device)
    dW = torch.empty((D, C, T), dtype=x.dtype, device=x.device)
    db = torch.empty((D,), dtype=x.dtype, device=x.device) if with_db else None
    feql_ct_backward_dw(T, x, dy, dW, db, ws, ws.numel(), N, C, D, mode, stream)
    return dW, db


# --------------------------------------------------------- p4m (D4, order 8)

def p4m_weight_fft(W: torch.Tensor, mode: int, stream=None) -> torch.Tensor:
    D, C, _ = W.shape
    nbytes = feql_p4m_weight_fft_bytes(C, D, mode)
    if nbytes == 0:
        raise ValueError("unsupported (C, D, mode) for p4m")
    What = torch.empty(nbytes, dtype=torch.uint8, device=W.device)
    feql_p4m_weight_fft(W, What, C, D, mode, stream)
    return What


def p4m_forward(x: torch.Tensor, What: torch.Tensor, b, D: int, mode: int, stream=None):
    N, C, _ = x.shape
    y = torch.empty((N, D, 8), dtype=x.dtype, device=x.device)
    feql_p4m_forward(x, What, b, y, N, C, D, mode, stream)
    return y


def p4m_backward_dx(dy: torch.Tensor, What: torch.Tensor, C: int, mode: int, stream=None):
    N, D, _ = dy.shape
    dx = torch.empty((N, C, 8), dtype=dy.dtype, device=dy.device)
    feql_p4m_backward_dx(dy, What, dx, N, C, D, mode, stream)
    return dx


def p4m_backward_dw(x: torch.Tensor, dy: torch.Tensor, mode: int, with_db: bool = True,
                    stream=None):
    N, C, _ = x.shape
    D = dy.shape[1]
    nbytes = feql_p4m_backward_dw_workspace_bytes(N, C, D, mode)
    ws = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=x.device)
    dW = torch.empty((D, C, 8), dtype=x.dtype, device=x.device)
    db = torch.empty((D,), dtype=x.dtype, device=x.device) if with_db else None
    feql_p4m_backward_dw(x, dy, dW, db, ws, ws.numel(), N, C, D, mode, stream)
    return dW, db


# ------------------------------------------------------------ MLP block (p4)

def mlp_weight_fft(W1: torch.Tensor, W2: torch.Tensor, mode: int, stream=None) -> torch.Tensor:
    H, C, _ = W1.shape
    Co = W2.shape[0]
    nbytes = feql_mlp_weight_fft_bytes(C, H, Co, mode)
    if nbytes == 0:
        raise ValueError("unsupported (C, H, Co, mode) for the fused MLP block")
    What = torch.empty(nbytes, dtype=torch.uint8, device=W1.device)
    feql_mlp_weight_fft(W1, W2, What, C, H, Co, mode, stream)
    return What


def mlp_forward(x: torch.Tensor, What: torch.Tensor, b1, b2, H: int, Co: int, mode: int,
                stream=None) -> torch.Tensor:
    N, C, _ = x.shape
    y = torch.empty((N, Co, 4), dtype=x.dtype, device=x.device)
    feql_mlp_forward(x, What, b1, b2, y, N, C, H, Co, mode, stream)
    return y


# ------------------------------------------- operators between the layers
# These take CUDA tensors of any strides (a dense copy is made where needed) on
# one device, which need not be the current one, and run on torch's current
# stream of that device; what they return belongs to that stream.

_HERE = contextlib.nullcontext()


def _on(t: torch.Tensor):
    """The device guard of a call on ``t``'s device."""
    index = t.get_device()
    if index < 0:
        raise ValueError(f"expected CUDA tensors (libfeql.so kernels), got one on {t.device}")
    return _HERE if index == torch.cuda.current_device() else torch.cuda.device(index)


def _mode(t: torch.Tensor) -> int:
    if t.dtype == torch.float16:
        return FEQL_FP16
    if t.dtype == torch.float32:
        return FEQL_FP32
    raise TypeError(f"expected float16 or float32 data, not {t.dtype}")


def _take(t, name: str, shape, dtype, index: int):
    """``t`` checked and dense, on a 16-byte boundary; None stays None."""
    if t is None:
        return None
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} is {t.dtype}, expected {dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{index}")
    return _dense(t)


def _dense(t: torch.Tensor) -> torch.Tensor:
    """``t``, or a dense copy on a 16-byte boundary."""
    if not t.is_contiguous():
        t = t.detach().contiguous()
    return t if t.data_ptr() % 16 == 0 else t.detach().clone()


_sizes: dict = {}


def _bytes(query, index: int, *args) -> int:
    """query(*args) on device ``index``, asked once per sizes; 0 (refused) is asked anew."""
    key = (query, index, args)
    n = _sizes.get(key)
    if n is None:
        n = query(*args)
        if n:
            if len(_sizes) >= 4096:
                _sizes.clear()
            _sizes[key] = n
    return n


# The layer with activation and residual in its epilogue.  ``act`` is one of
# FEQL_ACT_*; the group order T is the length of x's last axis (p4m: 8).

def _layer_calls(p4m: bool):
    """The entry points of a group, each taking T first."""
    if p4m:
        return ((lambda T, *a: feql_p4m_weight_fft_bytes(*a)),
                (lambda T, *a: feql_p4m_forward_act(*a)),
                (lambda T, *a: feql_p4m_backward_act_workspace_bytes(*a)),
                (lambda T, *a: feql_p4m_backward_act(*a)))
    return (feql_ct_weight_fft_bytes, feql_ct_forward_act, feql_ct_backward_act_workspace_bytes,
            feql_ct_backward_act)


_CYCLIC_CALLS, _P4M_CALLS = _layer_calls(False), _layer_calls(True)


def _layer_input(x: torch.Tensor, mode: int, p4m: bool):
    if x.dim() != 3 or (p4m and x.shape[2] != 8):
        raise ValueError(f"x has shape {tuple(x.shape)}, expected "
                         f"{'(N, C, 8)' if p4m else '(N, C, T)'}")
    if x.dtype != torch_dtype(mode):
        raise TypeError(f"x is {x.dtype}, the mode's data is {torch_dtype(mode)}")
    return x.shape


def _forward_act(calls, p4m, x, What, b, D, mode, act, res, save_z):
    N, C, T = _layer_input(x, mode, p4m)
    nbytes, forward = _bytes(calls[0], -1, T, C, D, mode), calls[1]
    if nbytes == 0:
        raise ValueError("unsupported (T, C, D, mode)")
    with _on(x):
        at = x.get_device()
        x = _dense(x)
        What = _take(What, "What", (nbytes,), torch.uint8, at)
        b = _take(b, "b", (D,), x.dtype, at)
        res = _take(res, "res", (N, D, T), x.dtype, at)
        y = x.new_empty((N, D, T))
        slope = torch.empty_like(y) if save_z and act != FEQL_ACT_NONE else None
        forward(T, x, What, b, res, y, slope, N, C, D, act, mode)
    return y, slope


def _backward_act(calls, p4m, x, dy, slope, What, mode, act, with_dx, with_dw, with_db):
    N, C, T = _layer_input(x, mode, p4m)
    if dy.dim() != 3:
        raise ValueError(f"dy has shape {tuple(dy.shape)}, expected (N, D, T)")
    D = dy.shape[1]
    nbytes, workspace, backward = _bytes(calls[0], -1, T, C, D, mode), calls[2], calls[3]
    if nbytes == 0:
        raise ValueError("unsupported (T, C, D, mode)")
    dx = dW = db = None
    with _on(x):
        at = x.get_device()
        x = _dense(x)
        dy = _take(dy, "dy", (N, D, T), x.dtype, at)
        slope = _take(slope, "slope", (N, D, T), x.dtype, at)
        What = _take(What, "What", (nbytes,), torch.uint8, at)
        ws_bytes = _bytes(workspace, at, T, N, C, D, act, mode)
        ws = x.new_empty(ws_bytes, dtype=torch.uint8)
        if with_dx:
            dx = torch.empty_like(x)
        if with_dw or with_db:
            dW = x.new_empty((D, C, T))
        if with_db:
            db = x.new_empty(D)
        if with_dx or dW is not None:
            backward(T, x, dy, slope, What, dx, dW, db, ws, ws_bytes, N, C, D, act, mode)
    return dx, (dW if with_dw else None), db


def ct_forward_act(x: torch.Tensor, What: torch.Tensor, b, D: int, mode: int, act: int, res=None,
                   save_z: bool = False):
    """y = res + act(z), z = the C_T layer of x plus b: (y, slope).

    ``slope`` is act'(z), all that ct_backward_act takes of z; None without an
    activation, or unless ``save_z`` asks for what the backward pass needs of z.
    """
    return _forward_act(_CYCLIC_CALLS, False, x, What, b, D, mode, act, res, save_z)


def ct_backward_act(x: torch.Tensor, dy: torch.Tensor, slope, What: torch.Tensor, mode: int,
                    act: int, with_dx: bool = True, with_dw: bool = True, with_db: bool = True):
    """dx, dW, db of ct_forward_act (the residual's gradient is dy), None where not asked.

    ``slope``: as ct_forward_act returned it (not z).
    """
    return _backward_act(_CYCLIC_CALLS, False, x, dy, slope, What, mode, act, with_dx, with_dw,
                         with_db)


def p4m_forward_act(x: torch.Tensor, What: torch.Tensor, b, D: int, mode: int, act: int, res=None,
                    save_z: bool = False):
    """ct_forward_act of the p4m layer."""
    return _forward_act(_P4M_CALLS, True, x, What, b, D, mode, act, res, save_z)


def p4m_backward_act(x: torch.Tensor, dy: torch.Tensor, slope, What: torch.Tensor, mode: int,
                     act: int, with_dx: bool = True, with_dw: bool = True, with_db: bool = True):
    """ct_backward_act of the p4m layer."""
    return _backward_act(_P4M_CALLS, True, x, dy, slope, What, mode, act, with_dx, with_dw,
                         with_db)


def norm_forward(x: torch.Tensor, gamma=None, beta=None, eps: float = 1e-5,
                 save_stats: bool = True):
    """Layer norm of (N, C, T) features over C*T, affine per channel: (y, stats).

    ``stats`` (N, 2) fp32 (mean, reciprocal deviation) is what norm_backward
    takes; None without ``save_stats``.
    """
    if x.dim() != 3:
        raise ValueError(f"x has shape {tuple(x.shape)}, expected (N, C, T)")
    N, C, T = x.shape
    mode = _mode(x)
    with _on(x):
        at = x.get_device()
        x = _dense(x)
        gamma = _take(gamma, "gamma", (C,), x.dtype, at)
        beta = _take(beta, "beta", (C,), x.dtype, at)
        y = torch.empty_like(x)
        stats = x.new_empty((N, 2), dtype=torch.float32) if save_stats else None
        feql_norm_forward(x, gamma, beta, y, stats, N, C, T, eps, mode)
    return y, stats


def norm_backward(dy: torch.Tensor, x: torch.Tensor, stats: torch.Tensor, gamma=None,
                  with_params: bool = True):
    """dx, dgamma, dbeta (None, None without ``with_params``) of norm_forward."""
    if x.dim() != 3:
        raise ValueError(f"x has shape {tuple(x.shape)}, expected (N, C, T)")
    N, C, T = x.shape
    mode = _mode(x)
    with _on(x):
        at = x.get_device()
        x = _dense(x)
        dy = _take(dy, "dy", x.shape, x.dtype, at)
        stats = _take(stats, "stats", (N, 2), torch.float32, at)
        gamma = _take(gamma, "gamma", (C,), x.dtype, at)
        dx = torch.empty_like(x)
        dgamma = dbeta = None
        if with_params:
            dgamma, dbeta = x.new_empty(C), x.new_empty(C)
        nbytes = max(_bytes(feql_norm_backward_workspace_bytes, at, N, C, T, mode), 16)
        ws = x.new_empty(nbytes, dtype=torch.uint8)
        feql_norm_backward(x, dy, stats, gamma, dx, dgamma, dbeta, ws, nbytes, N, C, T, mode)
    return dx, dgamma, dbeta


def _scan_sizes(u: torch.Tensor, g: torch.Tensor, offsets):
    """(B, N, C, T, shared) of a dense (B, L, C, T) or packed (N, C, T) input."""
    if offsets is None:
        if u.dim() != 4:
            raise ValueError(f"u has shape {tuple(u.shape)}, expected (B, L, C, T), or "
                             "(N, C, T) with offsets")
        B, N = u.shape[0], u.shape[0] * u.shape[1]
    else:
        if u.dim() != 3:
            raise ValueError(f"u has shape {tuple(u.shape)}, expected (N, C, T) with offsets")
        if offsets.dim() != 1 or offsets.numel() < 1:
            raise ValueError("offsets has shape (B + 1,)")
        B, N = offsets.numel() - 1, u.shape[0]
    C, T = u.shape[-2:]
    if g.shape not in (u.shape, u.shape[:-1]):
        raise ValueError(f"g has shape {tuple(g.shape)}, expected {tuple(u.shape)} or, with one "
                         f"gate per channel, {tuple(u.shape[:-1])}")
    return B, N, C, T, g.dim() < u.dim()


def scan_forward(u: torch.Tensor, g: torch.Tensor, h0=None, offsets=None, save: bool = True):
    """h_l = a_l h_{l-1} + (1 - a_l) u_l with a = sigmoid(g): (h, hN, saved).

    Dense: u (B, L, C, T).  Packed: u (N, C, T) and ``offsets`` (B + 1,) int32,
    sequence b in rows offsets[b]..offsets[b + 1].  g has u's shape, or lacks its
    last axis (one gate per channel).  h0 and hN are (B, C, T) fp32 states;
    ``saved`` is what scan_backward takes: (h, h0), which it reads, for fp32 data, and
    for fp16 data, whose h is rounded, (h_{l-1} - u_l in fp32, None); None without
    ``save``.
    """
    B, N, C, T, shared = _scan_sizes(u, g, offsets)
    mode = _mode(u)
    with _on(u):
        at = u.get_device()
        u = _dense(u)
        g = _take(g, "g", g.shape, u.dtype, at)
        h0 = _take(h0, "h0", (B, C, T), torch.float32, at)
        offsets = _take(offsets, "offsets", (B + 1,), torch.int32, at)
        h = torch.empty_like(u)
        hN = u.new_empty((B, C, T), dtype=torch.float32)
        nbytes = max(_bytes(feql_scan_workspace_bytes, at, B, N, C, T, shared,
                            offsets is not None, mode), 16)
        ws = u.new_empty(nbytes, dtype=torch.uint8)
        if save and mode == FEQL_FP16:
            diff = torch.empty_like(u, dtype=torch.float32)
            feql_scan_forward_diff(u, g, h0, offsets, h, hN, diff, ws, nbytes, B, N, C, T, shared,
                                   mode)
            return h, hN, (diff, None)
        feql_scan_forward(u, g, h0, offsets, h, hN, ws, nbytes, B, N, C, T, shared, mode)
    return h, hN, ((h, h0) if save else None)


def scan_backward(dh: torch.Tensor, u, g: torch.Tensor, saved, dhN=None, offsets=None):
    """du, dg, dh0 of scan_forward on the same u, g and offsets.

    ``u`` is not read for fp16 data, and may be None there.
    """
    like = dh if u is None else u
    B, N, C, T, shared = _scan_sizes(like, g, offsets)
    mode = _mode(like)
    with _on(like):
        at = like.get_device()
        g = _take(g, "g", g.shape, like.dtype, at)
        dh = _take(dh, "dh", like.shape, like.dtype, at)
        dhN = _take(dhN, "dhN", (B, C, T), torch.float32, at)
        offsets = _take(offsets, "offsets", (B + 1,), torch.int32, at)
        kept = _take(saved[0], "saved", like.shape, torch.float32, at)
        du, dg = torch.empty_like(dh), torch.empty_like(g)
        dh0 = dh.new_empty((B, C, T), dtype=torch.float32)
        nbytes = max(_bytes(feql_scan_workspace_bytes, at, B, N, C, T, shared,
                            offsets is not None, mode), 16)
        ws = dh.new_empty(nbytes, dtype=torch.uint8)
        if mode == FEQL_FP16:
            feql_scan_backward_diff(dh, g, kept, dhN, offsets, du, dg, dh0, ws, nbytes, B, N, C, T,
                                    shared, mode)
        else:
            if u is None:
                raise ValueError("u is read for fp32 data")
            h0 = _take(saved[1], "h0", (B, C, T), torch.float32, at)
            feql_scan_backward(dh, _dense(u), g, kept, h0, dhN, offsets, du, dg, dh0, ws, nbytes,
                               B, N, C, T, shared, mode)
    return du, dg, dh0


def scan_step(u: torch.Tensor, g: torch.Tensor, state: torch.Tensor) -> torch.Tensor:
    """One token of each sequence: u (B, C, T), g (B, C, T) or (B, C); the fp32
    ``state`` (B, C, T) is updated in place and returned rounded to u's type."""
    if u.dim() != 3:
        raise ValueError(f"u has shape {tuple(u.shape)}, expected (B, C, T)")
    B, C, T = u.shape
    if g.shape not in (u.shape, u.shape[:-1]):
        raise ValueError(f"g has shape {tuple(g.shape)}, expected {(B, C, T)} or {(B, C)}")
    mode = _mode(u)
    with _on(u):
        if not state.is_contiguous() or state.data_ptr() % 16 != 0:
            raise ValueError("state is updated in place: it has to be dense and 16-byte aligned")
        at = u.get_device()
        u = _dense(u)
        g = _take(g, "g", g.shape, u.dtype, at)
        s = _take(state, "state", (B, C, T), torch.float32, at)
        h = torch.empty_like(u)
        feql_scan_step(u, g, s, h, B, C, T, g.dim() < 3, mode)
        if not state.is_inference():  # a graph that saved the state sees the change
            torch.autograd.graph.increment_version(state)
    return h
