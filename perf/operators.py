"""Cases of the equivariant network operators beside the linear layer: layer norm, the linear
layer with bias, activation and residual in its epilogue, and the gated linear recurrence.

Features are (C, T) per token, the group index innermost.  ``run`` computes each operator in its
plain form (elementary torch operations in 32 bits, rounded once at the end) or, where ``own`` is
true, by the package's functions.
"""

import math

import torch

own = False

EPS = 1e-5
K0 = math.sqrt(2.0 / math.pi)   # the tanh form of GELU: z/2 (1 + tanh(K0 (z + K1 z^3)))
K1 = 0.044715
DT = {"fp16": torch.float16, "fp32": torch.float32}
ACTS = ("none", "relu", "gelu", "silu")


# ------------------------------------------------------------------------------- cases

def listed():
    return [
        # the norm in front of a small fp32 layer: one short launch
        {"name": "norm_fwd_small", "op": "norm", "train": False, "N": 256, "C": 16, "T": 4,
         "dtype": "fp32"},
        # a training step through the norm of the Swin stage-1 stream, 128 x 3136 tokens
        {"name": "norm_train_swin", "op": "norm", "train": True, "N": 401408, "C": 24, "T": 4,
         "dtype": "fp16"},
        # odd channel count, order-6 fibres, fp32
        {"name": "norm_train_odd", "op": "norm", "train": True, "N": 12608, "C": 67, "T": 6,
         "dtype": "fp32"},
        # fc1 of the ViT MLP with its activation (inference), 64 x 197 tokens
        {"name": "linear_fwd_vit_fc1", "op": "linear", "train": False, "group": "p4", "N": 12608,
         "C": 48, "D": 192, "T": 4, "dtype": "fp16", "act": "gelu", "res": False},
        # a wide layer closing a residual branch
        {"name": "linear_fwd_square_res", "op": "linear", "train": False, "group": "p4",
         "N": 65536, "C": 192, "D": 192, "T": 4, "dtype": "fp16", "act": "none", "res": True},
        # fc1 of the Swin stage-1 MLP: forward with the activation, then dx, dW, db
        {"name": "linear_train_swin", "op": "linear", "train": True, "group": "p4", "N": 401408,
         "C": 24, "D": 96, "T": 4, "dtype": "fp16", "act": "gelu", "res": False},
        # odd channel counts in fp32 with activation and residual
        {"name": "linear_train_fp32_odd", "op": "linear", "train": True, "group": "p4",
         "N": 3001, "C": 35, "D": 51, "T": 4, "dtype": "fp32", "act": "silu", "res": True},
        # the reflection group's layer in a residual block
        {"name": "linear_train_p4m", "op": "linear", "train": True, "group": "p4m", "N": 50000,
         "C": 12, "D": 48, "T": 8, "dtype": "fp16", "act": "silu", "res": True},
        # one token for each of 64 sequences being served
        {"name": "scan_step", "op": "scan", "train": False, "step": True, "packed": False,
         "B": 64, "L": 1, "C": 192, "T": 4, "gate": "element", "dtype": "fp16"},
        # one long sequence, as when a large image is read as a stream of tokens
        {"name": "scan_fwd_long", "op": "scan", "train": False, "step": False, "packed": False,
         "B": 1, "L": 65536, "C": 96, "T": 4, "gate": "element", "dtype": "fp16"},
        # training on the Swin stage-1 stream, one gate per channel
        {"name": "scan_train_swin", "op": "scan", "train": True, "step": False, "packed": False,
         "B": 128, "L": 3136, "C": 24, "T": 4, "gate": "channel", "dtype": "fp16"},
        # sequences of different lengths packed behind one another, odd channels, fp32
        {"name": "scan_train_packed", "op": "scan", "train": True, "step": False, "packed": True,
         "B": 37, "L": 700, "C": 33, "T": 6, "gate": "element", "dtype": "fp32"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "linear", "scan"))
    dtype = rng.choice(("fp16", "fp16", "fp32"))
    train = rng.random() < 0.6
    most = 401408 * 96 // (1 if dtype == "fp16" else 2)  # values of the largest listed tensor
    if op == "norm":
        T = rng.choice((1, 2, 3, 4, 4, 6, 8, 12, 16))
        C = max(_log(rng, 1, 1024), -(-16 // T))          # at least 16 features to a token
        N = _log(rng, 1, max(1, min(401408, most // (C * T))))
        return {"op": op, "train": train, "N": N, "C": C, "T": T, "dtype": dtype}
    if op == "linear":
        group, T = rng.choice((("p4", 4), ("p4", 4), ("p4m", 8), ("cyclic", 8), ("cyclic", 6),
                               ("cyclic", 3)))
        C, D = _log(rng, 2, 300), _log(rng, 2, 300)
        if group == "p4m":
            dtype = "fp16"                                # the one type of that layer
        if group == "p4" and dtype == "fp16":
            C, D = C + C % 2, D + D % 2                   # whole 16-byte rows
        cap = most // ((C + 2 * D) * T)
        if dtype == "fp32" or T == 3:                     # the CUDA-core layers: less work
            cap = min(cap, 2 * 10 ** 9 // (C * D * T))
        N = _log(rng, 1, max(1, min(401408, cap)))
        return {"op": op, "train": train, "group": group, "N": N, "C": C, "D": D, "T": T,
                "dtype": dtype, "act": rng.choice(ACTS[:1] + ACTS[2:]),
                "res": rng.random() < 0.5}
    T = rng.choice((1, 2, 4, 4, 6, 8, 3, 16))
    C = _log(rng, 1, 256)
    step = (not train) and rng.random() < 0.3
    B = _log(rng, 1, 512)
    cap = max(1, min(65536, most // (B * C * T)))
    L = 1 if step else _log(rng, 1, cap)
    return {"op": op, "train": train, "step": step, "packed": (not step) and rng.random() < 0.4,
            "B": B, "L": L, "C": C, "T": T, "gate": rng.choice(("channel", "element")),
            "dtype": dtype}


# ------------------------------------------------------------------------------ inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DT[case["dtype"]]

    def normal(*shape, std=1.0, mean=0.0, dtype=dt):
        v = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
        return v.mul_(std).add_(mean).to(dtype)

    s = dict(case)
    C, T = case["C"], case["T"]
    if case["op"] == "norm":
        N = case["N"]
        s["x"] = normal(N, C, T, mean=0.3)
        s["gamma"] = normal(C, std=0.1, mean=1.0)
        s["beta"] = normal(C, std=0.1)
        if case["train"]:
            s["dy"] = normal(N, C, T, std=0.1)
    elif case["op"] == "linear":
        N, D = case["N"], case["D"]
        s["x"] = normal(N, C, T)
        s["W"] = normal(D, C, T, std=1.0 / math.sqrt(T * C))
        s["b"] = normal(D, std=0.02)
        s["r"] = normal(N, D, T) if case["res"] else None
        if case["train"]:
            s["dy"] = normal(N, D, T, std=0.1)
    else:
        B, L = case["B"], case["L"]
        G = T if case["gate"] == "element" else None
        rows = (B * L,) if case["packed"] else (B, L)
        if case["step"]:
            rows = (B,)
        gate = rows + ((C,) if G is None else (C, T))
        s["u"] = normal(*rows, C, T)
        s["g"] = normal(*gate, std=1.5, mean=2.0)  # memories of a few to a few hundred tokens
        s["h0"] = normal(B, C, T, dtype=torch.float32)
        if case["packed"]:
            # B sequences that fill the B*L rows; some are empty, some much longer than others
            cut = torch.randint(0, B * L + 1, (B - 1,), generator=gen, device="cuda").sort().values
            ends = torch.tensor([0, B * L], device="cuda")
            s["offsets"] = torch.cat([ends[:1], cut, ends[1:]]).to(torch.int32)
        if case["train"]:
            s["dh"] = normal(*rows, C, T, std=0.1)
            s["dhN"] = normal(B, C, T, std=0.1, dtype=torch.float32)
    return s


def work(case):
    e = 2 if case["dtype"] == "fp16" else 4
    C, T = case["C"], case["T"]
    if case["op"] == "norm":
        n = case["N"] * C * T
        if case["train"]:  # x and y, then dy, x and dx
            return {"bytes": e * (5 * n + 6 * C), "flops": 24 * n}
        return {"bytes": e * (2 * n + 2 * C), "flops": 8 * n}
    if case["op"] == "linear":
        N, D = case["N"], case["D"]
        products = {"p4m": 12}.get(case["group"], 2 * T - 2 if T % 2 == 0 else 2 * T - 1)
        i, o = N * C * T, N * D * T
        bytes_ = e * (i + o * (2 if case["res"] else 1) + C * D * T + D)
        flops = 2.0 * products * N * C * D
        if case["train"]:  # the saved z, then x, dy, z and dx, dW, db (the residual's gradient is dy)
            bytes_ += e * (o + 2 * i + 2 * o + 2 * C * D * T + D)
            flops *= 3
        return {"bytes": bytes_, "flops": flops}
    n = case["B"] * case["L"] * C * T
    ng = n if case["gate"] == "element" else n // T
    state = 4 * case["B"] * C * T
    bytes_ = e * (2 * n + ng) + 2 * state
    flops = 8 * n
    if case["train"]:
        bytes_ += e * (3 * n + 2 * ng) + 2 * state
        flops += 20 * n
    return {"bytes": bytes_, "flops": flops}


# --------------------------------------------------------------------------------- run

def run(s):
    if s["op"] == "norm":
        return _own_norm(s) if own else _plain_norm(s)
    if s["op"] == "linear":
        return _own_linear(s) if own else _plain_linear(s)
    return _own_scan(s) if own else _plain_scan(s)


def _own_norm(s):
    from group_dft_structured_b200 import layer as L
    y, stats = L.norm_forward(s["x"], s["gamma"], s["beta"], EPS, save_stats=s["train"])
    if not s["train"]:
        return y
    dx, dgamma, dbeta = L.norm_backward(s["dy"], s["x"], stats, s["gamma"])
    return y, dx, dgamma, dbeta


def _own_linear(s):
    import group_dft_structured_b200 as F
    from group_dft_structured_b200 import layer as L
    mode = F.FEQL_FP16 if s["dtype"] == "fp16" else F.FEQL_FP32
    act = F.ACTIVATIONS[s["act"]]
    p4m = s["group"] == "p4m"
    What = s.get("What")
    if What is None or s["train"]:  # once per weight update; a served model keeps it
        What = s["What"] = (L.p4m_weight_fft if p4m else L.ct_weight_fft)(s["W"], mode)
    forward = L.p4m_forward_act if p4m else L.ct_forward_act
    y, z = forward(s["x"], What, s["b"], s["D"], mode, act, res=s["r"], save_z=s["train"])
    if not s["train"]:
        return y
    backward = L.p4m_backward_act if p4m else L.ct_backward_act
    dx, dW, db = backward(s["x"], s["dy"], z, What, mode, act)
    return y, dx, dW, db


def _own_scan(s):
    from group_dft_structured_b200 import layer as L
    if s["step"]:
        state = s["h0"].clone()
        return L.scan_step(s["u"], s["g"], state), state
    off = s.get("offsets")
    h, hN, ckpt = L.scan_forward(s["u"], s["g"], s["h0"], off, save=s["train"])
    if not s["train"]:
        return h, hN
    du, dg, dh0 = L.scan_backward(s["dh"], s["u"], s["g"], ckpt, s["dhN"], off)
    return h, hN, du, dg, dh0


def _plain_norm(s):
    x, gamma, beta = s["x"].float(), s["gamma"].float()[:, None], s["beta"].float()[:, None]
    d = x - x.mean((1, 2), keepdim=True)
    r = (d * d).mean((1, 2), keepdim=True).add(EPS).rsqrt()
    xh = d * r
    y = (xh * gamma + beta).to(s["x"].dtype)
    if not s["train"]:
        return y
    dy = s["dy"].float()
    g = dy * gamma
    dx = r * (g - g.mean((1, 2), keepdim=True) - xh * (g * xh).mean((1, 2), keepdim=True))
    dgamma, dbeta = (dy * xh).sum((0, 2)), dy.sum((0, 2))
    return tuple(v.to(s["x"].dtype) for v in (y, dx, dgamma, dbeta))


def _kernel_index(group, T):
    """u[t, s]: the weight element that takes group element s to t."""
    t = torch.arange(T, device="cuda")
    if group != "p4m":
        return (t[:, None] - t[None, :]) % T
    r, m = t % 4, t // 4  # element (r, m) at 4 m + r; h^-1 g
    rot = (1 - 2 * m[None, :]) * (r[:, None] - r[None, :])
    return 4 * (m[:, None] ^ m[None, :]) + rot % 4


def _unrolled(W, group):
    D, C, T = W.shape
    return W[:, :, _kernel_index(group, T)].permute(0, 2, 1, 3).reshape(D * T, C * T)


def _plain_linear(s):
    N, C, D, T = s["N"], s["C"], s["D"], s["T"]
    dt = s["x"].dtype
    A = _unrolled(s["W"].float(), s["group"])
    x = s["x"].float().reshape(N, C * T)
    z = (x @ A.t()).reshape(N, D, T) + s["b"].float()[:, None]
    if s["act"] == "none":
        a, slope = z, torch.ones_like(z)
    elif s["act"] == "relu":
        a, slope = z.clamp_min(0), (z > 0).float()
    else:
        v, dv = (z, 1.0) if s["act"] == "silu" else (2 * K0 * (z + K1 * z ** 3),
                                                   2 * K0 * (1 + 3 * K1 * z * z))
        p = 1 / (1 + torch.exp(-v))
        a, slope = z * p, p + z * p * (1 - p) * dv
    y = (a if s["r"] is None else s["r"].float() + a).to(dt)
    if not s["train"]:
        return y
    dz = (s["dy"].float() * slope).reshape(N, D * T)
    dx = (dz @ A).reshape(N, C, T).to(dt)
    dA = (dz.t() @ x).reshape(D, T, C, T).permute(0, 2, 1, 3).reshape(D, C, T * T)
    u = _kernel_index(s["group"], T).reshape(-1)
    dW = torch.zeros(D, C, T, device="cuda").index_add_(2, u, dA).to(dt)
    db = dz.reshape(N, D, T).sum((0, 2)).to(dt)
    return y, dx, dW, db


def _scan(a, b):
    """h_l = a_l h_{l-1} + b_l along axis 1, h_{-1} = 0, by halving: the pairs of neighbouring
    steps are steps of a scan of half the length, which gives every second h."""
    n = a.shape[1]
    if n == 1:
        return b
    a0, b0, a1, b1 = a[:, 0:n - 1:2], b[:, 0:n - 1:2], a[:, 1::2], b[:, 1::2]
    odd = _scan(a1 * a0, a1 * b0 + b1)
    h = torch.empty_like(b)
    h[:, 1::2] = odd
    h[:, 0] = b[:, 0]
    h[:, 2::2] = a[:, 2::2] * odd[:, :(n - 1) // 2] + b[:, 2::2]
    return h


def _plain_scan(s):
    C, T, B = s["C"], s["T"], s["B"]
    dt, shared = s["u"].dtype, s["gate"] == "channel"
    rows = (1, -1) if s["packed"] else (B, -1)
    u = s["u"].float().reshape(*rows, C * T)
    g = (s["g"].float()[..., None].expand(s["u"].shape) if shared else s["g"].float())
    a = (1 / (1 + torch.exp(-g))).reshape(*rows, C * T)
    c = (1 / (1 + torch.exp(g))).reshape(*rows, C * T)  # 1 - a, without its cancellation
    b = c * u
    h0 = s["h0"].reshape(B, C * T)
    # the first row of each sequence takes its initial state and nothing from the row before it
    # (a sequence of no rows returns its initial state)
    if s["packed"]:
        off = s["offsets"].long()
        first, last, full = off[:-1], off[1:] - 1, off[1:] > off[:-1]
        keep = torch.ones(u.shape[1], 1, device="cuda")
        keep[first[full]] = 0
        into = torch.zeros_like(u[0]).index_copy_(0, first[full], h0[full])[None]
    else:
        keep = torch.ones(u.shape[1], 1, device="cuda")
        keep[0] = 0
        into = torch.zeros_like(u)
        into[:, 0] = h0
    h = _scan(a * keep, b + a * into)
    if s["packed"]:
        hN = torch.where(full[:, None], h[0, last.clamp_min(0)], h0)
    else:
        hN = h[:, -1].clone()
    out = (h.to(dt).reshape(s["u"].shape), hN.reshape(B, C, T))
    if not s["train"]:
        return out
    dh = s["dh"].float().reshape(*rows, C * T)
    dhN = s["dhN"].reshape(B, C * T)
    if s["packed"]:
        dh = dh.index_add(1, last[full], dhN[full][None])
    else:
        dh = torch.cat([dh[:, :-1], dh[:, -1:] + dhN[:, None]], 1)
    after = torch.cat([(a * keep)[:, 1:], torch.zeros_like(a[:, :1])], 1)  # a of the next row
    delta = _scan(after.flip(1), dh.flip(1)).flip(1)
    before = torch.cat([torch.zeros_like(h[:, :1]), h[:, :-1]], 1) * keep + into
    du = c * delta
    dg = delta * (before - u) * a * c
    if s["packed"]:
        dh0 = torch.where(full[:, None], (a * delta)[0, first.clamp_max(u.shape[1] - 1)], dhN)
    else:
        dh0 = (a * delta)[:, 0]
    dg = dg.reshape(s["u"].shape)
    dg = (dg.sum(-1) if shared else dg).to(dt)
    return (*out, du.to(dt).reshape(s["u"].shape), dg, dh0.reshape(B, C, T))


# ------------------------------------------------------------------------------- exact

def exact(case, seed):
    s = prepare(case, seed)
    d = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v
         for k, v in s.items()}
    return {"norm": _exact_norm, "linear": _exact_linear, "scan": _exact_scan}[case["op"]](d)


def _exact_norm(s):
    N, C, T = s["x"].shape
    x = s["x"].reshape(N, C * T)
    F = C * T
    mu = x.sum(1) / F
    sigma = ((x * x).sum(1) / F - mu * mu + EPS).sqrt()  # moments: ample room in 64 bits
    gamma = s["gamma"].repeat_interleave(T)
    n = (x - mu[:, None]) / sigma[:, None]
    y = (n * gamma + s["beta"].repeat_interleave(T)).reshape(N, C, T)
    if not s["train"]:
        return y
    dy = s["dy"].reshape(N, F)
    # Jacobian of the normalisation: (I - 1 1^T / F - n n^T / F) / sigma
    g = dy * gamma
    dot1, dotn = g.sum(1, keepdim=True), torch.einsum("nf,nf->n", g, n)[:, None]
    dx = (g - (dot1 + n * dotn) / F) / sigma[:, None]
    dgamma = torch.einsum("nf,nf->f", dy, n).reshape(C, T).sum(1)
    return y, dx.reshape(N, C, T), dgamma, s["dy"].sum(2).sum(0)


def _exact_linear(s):
    N, C, T = s["x"].shape
    D = s["D"]
    W, p4m = s["W"], s["group"] == "p4m"

    def element(t, q):  # index of q^-1 t in the group
        if not p4m:
            return (t - q) % T
        sign = -1 if q >= 4 else 1
        return 4 * ((t // 4) ^ (q // 4)) + (sign * (t % 4 - q % 4)) % 4

    z = s["b"][None, :, None].expand(N, D, T).clone()
    for t in range(T):
        for q in range(T):
            z[:, :, t] += s["x"][:, :, q] @ W[:, :, element(t, q)].t()
    if s["act"] == "none":
        a, slope = z, torch.ones_like(z)
    elif s["act"] == "relu":
        a, slope = z * (z > 0), (z > 0).double()
    elif s["act"] == "silu":
        p = torch.sigmoid(z)
        a, slope = z * p, p * (1 + z * (1 - p))
    else:
        th = torch.tanh(K0 * (z + K1 * z ** 3))
        a = 0.5 * z * (1 + th)
        slope = 0.5 * (1 + th) + 0.5 * z * (1 - th * th) * K0 * (1 + 3 * K1 * z * z)
    y = a if s["r"] is None else a + s["r"]
    if not s["train"]:
        return y
    dz = s["dy"] * slope
    dx, dW = torch.zeros_like(s["x"]), torch.zeros_like(W)
    for t in range(T):
        for q in range(T):
            dx[:, :, q] += dz[:, :, t] @ W[:, :, element(t, q)]
            dW[:, :, element(t, q)] += dz[:, :, t].t() @ s["x"][:, :, q]
    return y, dx, dW, dz.sum(2).sum(0)


def _exact_scan(s):
    """Step by step over the tokens of every sequence at once."""
    C, T, B = s["C"], s["T"], s["B"]
    shared = s["gate"] == "channel"
    if s["packed"]:
        off = s["offsets"].tolist()
    else:
        L = 1 if s["step"] else s["L"]
        off = [i * L for i in range(B + 1)]
    longest = max(off[i + 1] - off[i] for i in range(B))
    if longest * (2 if s["train"] else 1) > 80000:
        return None
    u = s["u"].reshape(-1, C, T)
    a = torch.sigmoid(s["g"].reshape((-1, C, 1) if shared else (-1, C, T)))
    starts = torch.tensor(off[:-1], device="cuda")
    lens = torch.tensor(off[1:], device="cuda") - starts
    order = torch.argsort(lens, descending=True)
    alive = [0] * (longest + 1)  # how many sequences have a row l
    for n in lens.tolist():
        alive[n] += 1
    left, live = B, []
    for l in range(longest):
        left -= alive[l]
        live.append(left)
    begin = starts[order]
    state = s["h0"][order].clone()
    h, before = torch.zeros_like(u), torch.zeros_like(u) if s["train"] else None
    for l in range(longest):
        k = live[l]
        at = begin[:k] + l
        if before is not None:
            before[at] = state[:k]
        state[:k] = u[at] + a[at] * (state[:k] - u[at])
        h[at] = state[:k]
    hN = torch.empty_like(state)
    hN[order] = state
    if s["step"]:
        return h.reshape(s["u"].shape), hN
    if not s["train"]:
        return h.reshape(s["u"].shape), hN
    carry = s["dhN"][order].clone()
    dh = s["dh"].reshape(-1, C, T)
    du, dg = torch.zeros_like(u), torch.zeros_like(u)
    for l in range(longest - 1, -1, -1):
        k = live[l]
        at = begin[:k] + l
        delta = dh[at] + carry[:k]
        p = a[at]
        du[at] = (1 - p) * delta
        dg[at] = delta * (before[at] - u[at]) * p * (1 - p)
        carry[:k] = p * delta
    dh0 = torch.empty_like(carry)
    dh0[order] = carry
    dg = dg.reshape(s["u"].shape)
    return (h.reshape(s["u"].shape), hN, du.reshape(s["u"].shape), dg.sum(-1) if shared else dg,
            dh0)
