"""Drop-in PyTorch module for the equivariant linear layer of the cyclic group
C_T (T = 4: the rotation group p4; any T in 2..16, T = 6 and 8 on the tensor
cores) and of p4m (rotations and reflections, point group D4), with autograd.

Flash EQ-Linear (arXiv abstract) presents the method as a plug-and-play
replacement for the EQ-Linear layers of existing equivariant models: the layer
computes the same function as the naive form, an ``nn.Linear`` whose (T*D) x
(T*C) weight is the group-circulant unrolling of W[D][C][T],

    A[d*T + t, c*T + s] = W[d, c, (t - s) mod T],   bias[d*T + t] = b[d],

acting on features laid out as (channel, group element) with the group index
innermost.  For p4m (group="p4m", 8 elements (r, m) at index 4 m + r) the
unrolling is A[d*8 + g, c*8 + h] = W[d, c, h^-1 g].  ``EqLinear.from_unrolled``
takes such a dense layer apart into (W, b); ``EqLinear.forward`` runs the
library's kernels.

Beside it stand the other parts of an equivariant network's block, each with
autograd: ``EqLinear``'s activation and residual (in the epilogue of its
products), ``EqNorm`` (layer norm), ``EqScan`` (gated linear recurrence over the
tokens), and ``EqScanBlock``, a residual block made of them.

Argument marshalling only: every step of the forward and backward passes runs
in libfeql.so through the C ABI (``layer`` allocates outputs with torch).
Tensors must live on a CUDA device; there is no CPU path.
"""

from __future__ import annotations

import math

import torch
from torch.autograd.function import once_differentiable

from . import ACTIVATIONS, FEQL_FP16, FEQL_FP32
from . import layer as _L


def mode_for(dtype: torch.dtype) -> int:
    if dtype == torch.float16:
        return FEQL_FP16
    if dtype == torch.float32:
        return FEQL_FP32
    raise TypeError(f"EqLinear computes in float16 or float32, not {dtype}")


def _p4m_index(r: int, m: int) -> int:
    return 4 * m + (r % 4)


def p4m_kernel_index(g: int, h: int) -> int:
    """Index of h^-1 g in p4m's point group D4, elements (r, m) at 4 m + r."""
    rg, mg = g % 4, g // 4
    rh, mh = h % 4, h // 4
    return _p4m_index((-1) ** mh * (rg - rh), mh ^ mg)


class EqLinearFunction(torch.autograd.Function):
    """y[n,d,t] = b[d] + sum_c sum_s W[d,c,(t-s) mod T] x[n,c,s] on (N, C, T) tensors
    (group "cyclic"), or the p4m group convolution W[d,c,h^-1 g] (group "p4m").

    ``What`` is the layer's Fourier weight buffer (``layer.ct_weight_fft`` of W),
    passed in so that callers who know that W is unchanged can reuse it.  Backward
    returns the gradients autograd asks for: dx from the dX pass, dW and db from
    the dW pass; for p4 with all of them needed, from the fused single pass.
    """

    @staticmethod
    def forward(ctx, x, W, b, What, mode: int, group: str = "cyclic"):
        D = W.shape[0]
        b = None if b is None else _L._dense(b)
        y = (_L.p4m_forward(x, What, b, D, mode) if group == "p4m"
             else _L.ct_forward(x, What, b, D, mode))
        ctx.save_for_backward(x, What)
        ctx.mode = mode
        ctx.group = group
        ctx.shape = (x.shape[1], D, x.shape[2])
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, What = ctx.saved_tensors
        C, D, T = ctx.shape
        need_x, need_W, need_b = ctx.needs_input_grad[:3]
        dy = _L._dense(dy)
        dx = dW = db = None
        if ctx.group == "p4m":
            if need_x:
                dx = _L.p4m_backward_dx(dy, What, C, ctx.mode)
            if need_W or need_b:
                dW, db = _L.p4m_backward_dw(x, dy, ctx.mode, with_db=need_b)
        elif T == 4 and need_x and need_W:
            dx, dW, db = _L.backward(x, dy, What, ctx.mode, with_db=need_b)
        else:
            if need_x:
                dx = _L.ct_backward_dx(dy, What, C, ctx.mode)
            if need_W or need_b:
                dW, db = _L.ct_backward_dw(x, dy, ctx.mode, with_db=need_b)
        return dx, (dW if need_W else None), (db if need_b else None), None, None, None


class EqLinearActFunction(torch.autograd.Function):
    """y = res + act(z), z = EqLinear(x) + b on (N, C, T) tensors; the arguments of
    EqLinearFunction, ``res`` (or None) and one of FEQL_ACT_*.  Backward: dz =
    dy act'(z) from the saved slopes, then dx, dW, db as asked for; dres = dy.
    ``train``: whether gradients are recorded (torch.is_grad_enabled() at the call,
    which a Function cannot see: without it weights that want gradients would have
    inference save for them)."""

    @staticmethod
    def forward(ctx, x, W, b, res, What, mode: int, group: str, act: int, train: bool = True):
        run = _L.p4m_forward_act if group == "p4m" else _L.ct_forward_act
        y, slope = run(x, What, b, W.shape[0], mode, act, res=res,
                       save_z=train and any(ctx.needs_input_grad[:3]))
        ctx.save_for_backward(x, What, slope)
        ctx.mode, ctx.group, ctx.act = mode, group, act
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, What, slope = ctx.saved_tensors
        need_x, need_W, need_b, need_res = ctx.needs_input_grad[:4]
        dx = dW = db = None
        if need_x or need_W or need_b:
            run = _L.p4m_backward_act if ctx.group == "p4m" else _L.ct_backward_act
            dx, dW, db = run(x, dy, slope, What, ctx.mode, ctx.act, with_dx=need_x,
                             with_dw=need_W, with_db=need_b)
        return dx, dW, db, (dy if need_res else None), None, None, None, None, None


class EqLinear(torch.nn.Module):
    """Equivariant linear layer of C_T (or p4m) on features (..., C*T), group index innermost.

    Parameters: ``weight`` [D][C][T] and ``bias`` [D] (or None), in float16
    (any T; the tensor cores serve T = 4, 8, p4m, and 6 with C and D multiples
    of 4) or float32.  ``group="p4m"`` selects the point
    group D4 (T = 8: rotations (r, 0) at 0..3, reflected (r, 1) at 4..7).  The
    weight is transformed at every call, by one small kernel; ``freeze()`` keeps the
    result for a model that is served.  ``activation`` ("relu", "gelu": the tanh form, "silu") is
    applied to the output and ``forward``'s ``residual`` added after it, both in
    the epilogue of the layer's products.
    """

    def __init__(self, in_channels: int, out_channels: int, group_order: int = 4,
                 bias: bool = True, dtype: torch.dtype = torch.float16, device=None,
                 group: str = "cyclic", activation: str = "none"):
        super().__init__()
        if activation not in ACTIVATIONS:
            raise ValueError(f"activation is one of {', '.join(ACTIVATIONS)}, not {activation!r}")
        self.activation = activation
        if group not in ("cyclic", "p4m"):
            raise ValueError(f"group is 'cyclic' or 'p4m', not {group!r}")
        if group == "p4m" and group_order != 8:
            raise ValueError("p4m has 8 group elements")
        self.group = group
        self.in_channels, self.out_channels = in_channels, out_channels
        self.group_order = group_order
        mode_for(dtype)
        self.weight = torch.nn.Parameter(
            torch.empty((out_channels, in_channels, group_order), dtype=dtype, device=device))
        self.bias = (torch.nn.Parameter(torch.empty((out_channels,), dtype=dtype, device=device))
                     if bias else None)
        self._frozen = False
        self._whats = {}  # stream: (what the weight was, its Fourier weight buffer, its memory)
        self.reset_parameters()

    def reset_parameters(self) -> None:
        # the bound nn.Linear uses for the unrolled layer: fan-in T*C
        bound = 1.0 / math.sqrt(self.group_order * self.in_channels)
        with torch.no_grad():
            self.weight.uniform_(-bound, bound)
            if self.bias is not None:
                self.bias.uniform_(-bound, bound)

    def fourier_weight(self) -> torch.Tensor:
        W = self.weight
        # Nothing tells reliably whether a weight has changed (a fused optimizer's step, a
        # replayed graph and a write through .data leave no version), so it is transformed
        # at every call unless it is declared constant.  A graph under capture has the
        # transform in itself, and nothing that it has yet to compute is kept.
        if (not self._frozen or (W.requires_grad and torch.is_grad_enabled())
                or torch.cuda.is_current_stream_capturing()):
            return self._transformed()
        key = (W.device, W.dtype, W.data_ptr(), None if W.is_inference() else W._version,
               tuple(W.shape))
        # a buffer to each stream: made, used and given back in its order alone; with the
        # weight's memory, which no other weight can have as long as the buffer is kept
        stream = torch.cuda.current_stream(W.device).cuda_stream
        kept = self._whats.get(stream)
        if kept is None or kept[0] != key:
            kept = (key, self._transformed(), W.detach())
            # (a new dict: other threads may be looking at this one)
            self._whats = {s: k for s, k in list(self._whats.items()) if k[0] == key}
            self._whats[stream] = kept
        return kept[1]

    def freeze(self, frozen: bool = True) -> "EqLinear":
        """Declares the weight constant from here on, as in a served model: its Fourier
        weight buffer is then kept (one for each stream that calls) wherever no gradient of
        the weight is recorded.  ``freeze(False)`` and ``train()`` end it."""
        self._frozen, self._whats = frozen, {}
        return self

    def train(self, mode: bool = True):
        if mode:
            self.freeze(False)
        return super().train(mode)

    def __getstate__(self):  # copies and files hold the weight alone
        return {**self.__dict__, "_whats": {}}

    def __setstate__(self, state):
        super().__setstate__({"_frozen": False, **state, "_whats": {}})

    def _transformed(self) -> torch.Tensor:
        wfft = _L.p4m_weight_fft if self.group == "p4m" else _L.ct_weight_fft
        # an ordinary tensor, which later calls may save for their backward pass
        with torch.inference_mode(False), torch.no_grad():
            return wfft(_L._dense(self.weight.detach()), mode_for(self.weight.dtype))

    def forward(self, x: torch.Tensor, residual: torch.Tensor | None = None) -> torch.Tensor:
        C, D, T = self.in_channels, self.out_channels, self.group_order
        if x.shape[-1] != C * T:
            raise ValueError(f"expected features of size C*T = {C * T}, got {x.shape[-1]}")
        if not x.is_cuda:
            raise RuntimeError("EqLinear runs on CUDA tensors only (libfeql.so kernels)")
        lead = x.shape[:-1]
        x3 = x.reshape(-1, C, T).contiguous()
        if x3.data_ptr() % 16 != 0:  # a part of a larger tensor
            x3 = x3.clone()  # (not _dense: in autograd's sight)
        if x3.dtype != self.weight.dtype:
            raise TypeError(f"input dtype {x3.dtype} differs from the weight's {self.weight.dtype}")
        if self.weight.device != x.device:
            raise ValueError(f"input on {x.device}, weight on {self.weight.device}")
        if residual is not None:
            if residual.shape != (*lead, D * T):
                raise ValueError(f"expected a residual of shape {(*lead, D * T)}, got "
                                 f"{tuple(residual.shape)}")
            residual = residual.reshape(-1, D, T)
        mode = mode_for(self.weight.dtype)
        with torch.cuda.device(x.device):  # which need not be the current one
            What = self.fourier_weight()
            if residual is None and self.activation == "none":
                y = EqLinearFunction.apply(x3, self.weight, self.bias, What, mode, self.group)
            else:
                y = EqLinearActFunction.apply(x3, self.weight, self.bias, residual, What, mode,
                                              self.group, ACTIVATIONS[self.activation],
                                              torch.is_grad_enabled())
        return y.reshape(*lead, D * T)

    def extra_repr(self) -> str:
        return (f"in_channels={self.in_channels}, out_channels={self.out_channels}, "
                f"group_order={self.group_order}, group={self.group}, "
                f"bias={self.bias is not None}"
                + (f", activation={self.activation}" if self.activation != "none" else ""))

    @classmethod
    def from_unrolled(cls, weight: torch.Tensor, bias: torch.Tensor | None, group_order: int,
                      atol: float = 0.0, group: str = "cyclic") -> "EqLinear":
        """The layer equal to the dense (T*D) x (T*C) map ``weight`` (+ ``bias``).

        ``weight`` must be group-circulant in the layout above (entries that
        should be equal may differ by ``atol``) and ``bias`` constant over the
        group index; otherwise ValueError.  Parameters keep weight's dtype and
        device.
        """
        T = group_order
        rows, cols = weight.shape
        if rows % T or cols % T:
            raise ValueError(f"dense shape {tuple(weight.shape)} is not a multiple of T = {T}")
        D, C = rows // T, cols // T
        A = weight.detach().reshape(D, T, C, T)  # [d][t][c][s]
        W = A[:, :, :, 0].permute(0, 2, 1).contiguous()  # W[d,c,u] = A[d, u, c, s=e]
        if group == "p4m":
            if T != 8:
                raise ValueError("p4m has 8 group elements")
            u = torch.tensor([[p4m_kernel_index(g, h) for h in range(8)] for g in range(8)],
                             device=weight.device)  # u[g][h] = h^-1 g
        else:
            t = torch.arange(T, device=weight.device)
            u = (t[:, None] - t[None, :]) % T  # u[t][s] = (t - s) mod T
        rebuilt = W[:, :, u].permute(0, 2, 1, 3)  # [d][t][c][s] = W[d, c, (t-s) mod T]
        if not torch.allclose(rebuilt, A, rtol=0.0, atol=atol):
            raise ValueError("weight is not group-circulant for this T")
        b = None
        if bias is not None:
            B = bias.detach().reshape(D, T)
            if not torch.allclose(B, B[:, :1].expand(D, T), rtol=0.0, atol=atol):
                raise ValueError("bias is not constant over the group index")
            b = B[:, 0].contiguous()
        m = cls(C, D, T, bias=b is not None, dtype=weight.dtype, device=weight.device,
                group=group)
        with torch.no_grad():
            m.weight.copy_(W)
            if b is not None:
                m.bias.copy_(b)
        return m


class EqNormFunction(torch.autograd.Function):
    """Layer norm of (N, C, T) features over C*T, affine per channel (``train`` as for
    EqLinearActFunction)."""

    @staticmethod
    def forward(ctx, x, gamma, beta, eps: float, train: bool = True):
        y, stats = _L.norm_forward(x, gamma, beta, eps,
                                   save_stats=train and any(ctx.needs_input_grad))
        ctx.save_for_backward(x, stats, gamma)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, stats, gamma = ctx.saved_tensors
        need_x, need_g, need_b = ctx.needs_input_grad[:3]
        dx, dgamma, dbeta = _L.norm_backward(dy, x, stats, gamma, with_params=need_g or need_b)
        return (dx if need_x else None, dgamma if need_g else None, dbeta if need_b else None,
                None, None)


class EqNorm(torch.nn.Module):
    """Layer norm of features (..., C*T), group index innermost: each token is
    normalised over all its C*T features, then scaled and shifted per channel
    (parameters ``weight`` [C] and ``bias`` [C], or neither without ``affine``).
    Statistics and parameters are shared over the group axis, so the module
    commutes with the group's action."""

    def __init__(self, channels: int, group_order: int = 4, eps: float = 1e-5,
                 affine: bool = True, dtype: torch.dtype = torch.float16, device=None):
        super().__init__()
        mode_for(dtype)
        self.channels, self.group_order, self.eps = channels, group_order, eps
        self.weight = self.bias = None
        if affine:
            self.weight = torch.nn.Parameter(torch.ones((channels,), dtype=dtype, device=device))
            self.bias = torch.nn.Parameter(torch.zeros((channels,), dtype=dtype, device=device))

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        C, T = self.channels, self.group_order
        if x.shape[-1] != C * T:
            raise ValueError(f"expected features of size C*T = {C * T}, got {x.shape[-1]}")
        y = EqNormFunction.apply(x.reshape(-1, C, T), self.weight, self.bias, self.eps,
                                 torch.is_grad_enabled())
        return y.reshape(x.shape)

    def extra_repr(self) -> str:
        return (f"channels={self.channels}, group_order={self.group_order}, eps={self.eps}, "
                f"affine={self.weight is not None}")


class EqScanFunction(torch.autograd.Function):
    """layer.scan_forward with autograd: (h, hN) of (u, g, h0, offsets); ``train`` as for
    EqLinearActFunction."""

    @staticmethod
    def forward(ctx, u, g, h0, offsets, train: bool = True):
        h, hN, saved = _L.scan_forward(u, g, h0, offsets,
                                       save=train and any(ctx.needs_input_grad[:3]))
        if saved is not None:
            # fp16 data: the backward pass reads neither u nor h0 (kept all the same, so that
            # a state that step() changes in between is refused in both types)
            ctx.save_for_backward(u if u.dtype == torch.float32 else None, g, saved[0], h0, offsets)
        ctx.set_materialize_grads(False)
        return h, hN

    @staticmethod
    @once_differentiable
    def backward(ctx, dh, dhN):
        u, g, kept, h0, offsets = ctx.saved_tensors
        if dh is None:
            dh = torch.zeros(kept.shape, dtype=g.dtype, device=g.device)
        du, dg, dh0 = _L.scan_backward(dh, u, g, (kept, h0), dhN, offsets)
        need = ctx.needs_input_grad
        return (du if need[0] else None, dg if need[1] else None, dh0 if need[2] else None, None,
                None)


class EqScan(torch.nn.Module):
    """Gated linear recurrence over the tokens, h = a h + (1 - a) u with
    a = sigmoid(gate), per feature of (..., C*T).

    ``forward(u, gate, state, offsets)``: u (B, L, C*T), or (N, C*T) rows of
    packed sequences with ``offsets`` (B + 1,) int32; gate of u's shape, or with
    C features (one gate per channel, shared over the group axis); state
    (B, C*T) fp32 or None (zero).  Returns h and the state after the last
    tokens.  ``step`` takes one token of each sequence, u (B, C*T), and updates
    the state in place (no autograd).
    """

    def __init__(self, channels: int, group_order: int = 4):
        super().__init__()
        self.channels, self.group_order = channels, group_order

    def _split(self, u, gate):
        C, T = self.channels, self.group_order
        if u.shape[-1] != C * T:
            raise ValueError(f"expected features of size C*T = {C * T}, got {u.shape[-1]}")
        if gate.shape[:-1] != u.shape[:-1] or gate.shape[-1] not in (C, C * T):
            raise ValueError(f"expected gates of shape {(*u.shape[:-1], C * T)} or "
                             f"{(*u.shape[:-1], C)}, got {tuple(gate.shape)}")
        lead = u.shape[:-1]
        shared = gate.shape[-1] == C and T > 1
        return u.reshape(*lead, C, T), gate if shared else gate.reshape(*lead, C, T)

    def forward(self, u: torch.Tensor, gate: torch.Tensor, state: torch.Tensor | None = None,
                offsets: torch.Tensor | None = None):
        C, T = self.channels, self.group_order
        uv, gv = self._split(u, gate)
        h0 = None if state is None else state.reshape(-1, C, T)
        h, hN = EqScanFunction.apply(uv, gv, h0, offsets, torch.is_grad_enabled())
        return h.reshape(u.shape), hN.reshape(-1, C * T)

    @torch.no_grad()
    def step(self, u: torch.Tensor, gate: torch.Tensor, state: torch.Tensor) -> torch.Tensor:
        C, T = self.channels, self.group_order
        uv, gv = self._split(u, gate)
        return _L.scan_step(uv, gv, state.view(-1, C, T)).reshape(u.shape)

    def extra_repr(self) -> str:
        return f"channels={self.channels}, group_order={self.group_order}"


class EqScanBlock(torch.nn.Module):
    """Residual block of an equivariant network whose tokens mix by a gated
    recurrence (the place of the attention or state-space mixer):

        n = norm1(x);  x = x + out(scan(value(n), gate(n)))
        x = x + fc2(gelu(fc1(norm2(x))))

    on features (B, L, C*T), or (N, C*T) rows of packed sequences with
    ``offsets``.  Every part commutes with the group's action on the group axis.
    ``step`` is the block on one token of each sequence, for generation: it takes
    and updates the (B, C*T) fp32 state that ``forward`` returns.
    """

    def __init__(self, channels: int, hidden: int, group_order: int = 4,
                 dtype: torch.dtype = torch.float16, device=None, group: str = "cyclic"):
        super().__init__()
        kw = {"dtype": dtype, "device": device}
        lin = {**kw, "group_order": group_order, "group": group}
        self.norm1 = EqNorm(channels, group_order, **kw)
        self.value = EqLinear(channels, channels, **lin)
        self.gate = EqLinear(channels, channels, **lin)
        self.scan = EqScan(channels, group_order)
        self.out = EqLinear(channels, channels, **lin)
        self.norm2 = EqNorm(channels, group_order, **kw)
        self.fc1 = EqLinear(channels, hidden, activation="gelu", **lin)
        self.fc2 = EqLinear(hidden, channels, **lin)
        with torch.no_grad():
            self.gate.bias.fill_(2.0)  # memories of some eight tokens to begin with

    def _mlp(self, x):
        return self.fc2(self.fc1(self.norm2(x)), residual=x)

    def freeze(self, frozen: bool = True) -> "EqScanBlock":
        """EqLinear.freeze of all its layers."""
        for m in self.modules():
            if isinstance(m, EqLinear):
                m.freeze(frozen)
        return self

    def forward(self, x: torch.Tensor, state: torch.Tensor | None = None,
                offsets: torch.Tensor | None = None):
        n = self.norm1(x)
        h, state = self.scan(self.value(n), self.gate(n), state, offsets)
        return self._mlp(self.out(h, residual=x)), state

    @torch.no_grad()
    def step(self, x: torch.Tensor, state: torch.Tensor) -> torch.Tensor:
        n = self.norm1(x)
        h = self.scan.step(self.value(n), self.gate(n), state)
        return self._mlp(self.out(h, residual=x))
