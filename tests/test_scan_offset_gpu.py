"""The recurrence's gradients where the states are close to the inputs (slowly varying
features with an offset), against float64.

dg = delta (h_{l-1} - u) a (1 - a) takes the difference from states of fp32, in fp16 data
too, so its bound has no half step of h.  What it has: the fp32 states' own error.  A step
multiplies by a and 1 - a, each off by a relative e (the hardware's exponential and
reciprocal for fp16 data, 20 * 2^-23, and the precise ones, 4 * 2^-23; with 4 roundings of
2^-24), so E_l = a E_{l-1} + e M_l, M_l = a M_{l-1} + (1 - a) |u_l|, runs through the rows as
the states do.  Then 2^-24 of the operands for the subtraction, a step e for each of a and
1 - a and 4 roundings for the products, the gradient's own error in delta, and half a step of
dg.  Here |h| is 10 to 1000 times |h - u|: half a step of h (2^-12 |h| at least) would be far
outside.
"""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import group_dft_structured_b200 as F
from group_dft_structured_b200 import layer as L
from group_dft_structured_b200.module import EqScan
from oracle import feql_ops_oracle as O

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {np.float16: 2.0 ** -11, np.float32: U}
TINY = {np.float16: 2.0 ** -25, np.float32: 0.0}
STEP = {np.float16: 20 * 2.0 ** -23 + 4 * U, np.float32: 4 * 2.0 ** -23 + 4 * U}


@pytest.fixture(scope="module", autouse=True)
def ready():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from group_dft_structured_b200 import build
    build.build()
    F.load()


def cuda(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def bound(u, g, dh, h0, dhN, off, dt):
    """dg of the definition and how far off it may be."""
    e, B = STEP[dt], len(off) - 1
    a, na = O.gates(np.broadcast_to(g[..., None], u.shape) if g.ndim < u.ndim else g)
    rdg = O.scan_backward(dh, u, g, h0, dhN, off)[1]
    h, _ = O.scan_forward(u, g, h0, off)
    before, Eb, Ed, delta = (np.zeros_like(u) for _ in range(4))
    for b in range(B):
        prev, M, E = h0[b], np.abs(h0[b]), np.zeros_like(h0[b])
        for l in range(off[b], off[b + 1]):
            before[l], Eb[l] = prev, E
            M = a[l] * M + na[l] * np.abs(u[l])
            E, prev = a[l] * E + e * M, h[l]
        c, M, E = dhN[b], np.abs(dhN[b]), np.zeros_like(dhN[b])
        for l in range(off[b + 1] - 1, off[b] - 1, -1):
            delta[l] = dh[l] + c
            Md = np.abs(dh[l]) + M
            Ed[l] = E + U * Md
            M, E, c = a[l] * Md, a[l] * Ed[l] + e * a[l] * Md, a[l] * delta[l]
    diff = np.abs(before - u)
    Eg = a * na * (np.abs(delta) * (Eb + U * (np.abs(before) + np.abs(u))) + Ed * diff
                   + (2 * e + 4 * U) * np.abs(delta) * diff)
    if g.ndim < u.ndim:
        Eg = Eg.sum(-1) + 16 * U * (np.abs(delta) * diff * a * na).sum(-1)
    return rdg, HALF[dt] * np.abs(rdg) + TINY[dt] + Eg


CASES = [  # rows of the sequences, C, T
    ([300, 300], 8, 4), ([300, 300], 24, 4), ([40] * 60, 6, 6), ([200], 5, 1), ([150, 150], 4, 2),
    ([120, 0, 900, 33], 3, 3), ([4000], 8, 4), ([0, 2500, 1], 4, 8),
]


@pytest.mark.parametrize("mean,noise", [(10.0, 0.1), (-3.0, 0.01), (100.0, 0.5)])
@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("dt", [np.float16, np.float32])
@pytest.mark.parametrize("rows,C,T", CASES)
def test_gates_gradient(rows, C, T, dt, shared, mean, noise):
    r = np.random.default_rng(sum(rows) + 7 * C + T)
    off = np.concatenate([[0], np.cumsum(rows)]).tolist()
    N, B = off[-1], len(rows)
    u = (mean + noise * r.standard_normal((N, C, T))).astype(dt)
    g = np.clip(2 + 1.5 * r.standard_normal((N, C) if shared else (N, C, T)), -8, 8).astype(dt)
    dh = r.standard_normal((N, C, T)).astype(dt)
    h0 = (mean + noise * r.standard_normal((B, C, T))).astype(np.float32)
    dhN = r.standard_normal((B, C, T)).astype(np.float32)
    dense = len(set(rows)) == 1
    shape = (lambda v: v.reshape(B, -1, *v.shape[1:])) if dense else (lambda v: v)
    U_, G_, D_ = (cuda(shape(v)) for v in (u, g, dh))
    o = None if dense else torch.tensor(off, dtype=torch.int32, device="cuda")
    _, _, saved = L.scan_forward(U_, G_, cuda(h0), o)
    dg = L.scan_backward(D_, U_, G_, saved, cuda(dhN), o)[1]
    ref, tol = bound(*(v.astype(np.float64) for v in (u, g, dh, h0, dhN)), off, dt)
    err = np.abs(dg.cpu().numpy().astype(np.float64).reshape(ref.shape) - ref)
    assert (err <= tol).all(), float((err / tol).max())


@pytest.mark.parametrize("shared", [False, True])
def test_states_beyond_fp16(shared):
    """An initial state that fp16 cannot hold: h saturates, the gradients do not."""
    r = np.random.default_rng(3)
    N, C, T = 60, 8, 4
    u = r.standard_normal((N, C, T)).astype(np.float16)
    g = r.standard_normal((N, C) if shared else (N, C, T)).astype(np.float16)
    dh = (1e-3 * r.standard_normal((N, C, T))).astype(np.float16)
    h0, dhN = np.full((1, C, T), 3e5, np.float32), np.zeros((1, C, T), np.float32)
    h, _, saved = L.scan_forward(cuda(u)[None], cuda(g)[None], cuda(h0))
    assert h.isinf().any()
    out = L.scan_backward(cuda(dh)[None], cuda(u)[None], cuda(g)[None], saved)
    assert all(torch.isfinite(t).all() for t in out)
    ref, tol = bound(*(v.astype(np.float64) for v in (u, g, dh, h0, dhN)), [0, N], np.float16)
    assert (np.abs(out[1][0].cpu().numpy().astype(np.float64) - ref) <= tol).all()


def test_saved_states_and_what_they_are_for():
    u = torch.randn(2, 70, 6, 4, device="cuda").half()
    h0 = torch.randn(2, 6, 4, device="cuda")
    h, hN, saved = L.scan_forward(u, u, h0)
    alone, last, none = L.scan_forward(u, u, h0, save=False)
    assert none is None and torch.equal(h, alone) and torch.equal(hN, last)
    assert saved[0].dtype == torch.float32
    assert torch.equal(saved[0][:, 0], h0 - u[:, 0].float())
    want = L.scan_backward(u, u, u, saved)
    for a, b in zip(L.scan_backward(u, None, u, saved), want):
        assert torch.equal(a, b)
    with pytest.raises(TypeError):
        L.scan_backward(u, u, u, (h, h0))  # the rounded states are not taken
    x = u.float()
    h, _, saved = L.scan_forward(x, x, h0)
    assert saved[0] is h
    with pytest.raises(ValueError):
        L.scan_backward(x, None, x, saved)


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_module_gradients_through_either_output(dtype):
    """Backward through h alone, through the state alone, and through both add up."""
    scan = EqScan(6, 4)
    u0 = (5 + 0.1 * torch.randn(3, 90, 24, device="cuda")).to(dtype)
    g0, s0 = torch.randn(3, 90, 6, device="cuda").to(dtype), torch.randn(3, 24, device="cuda")
    w, v = torch.randn(3, 90, 24, device="cuda").to(dtype), torch.randn(3, 24, device="cuda")
    grads = []
    for on in ((1, 0), (0, 1), (1, 1)):
        u, g, s = (t.clone().requires_grad_() for t in (u0, g0, s0))
        h, last = scan(u, g, s)
        outs = [(h, w), (last, v)]
        torch.autograd.backward(*zip(*[o for o, k in zip(outs, on) if k]))
        grads.append((u.grad, g.grad, s.grad))
    step = torch.finfo(dtype).eps
    for a, b, c in zip(*grads):  # three roundings of half a step, of a sum's parts
        size = a.double().abs() + b.double().abs()
        assert ((a.double() + b.double() - c.double()).abs() <= 2 * step * size + 1e-5).all()


def test_training_step_in_a_graph_and_on_another_stream():
    u = (4 + 0.1 * torch.randn(3, 1500, 8, 4, device="cuda")).half()
    g, dh = torch.randn(3, 1500, 8, device="cuda").half(), torch.randn_like(u)

    def both():
        h, hN, saved = L.scan_forward(u, g)
        return (h, hN, saved[0], *L.scan_backward(dh, u, g, saved))

    want = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = both()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = both()
    for t in out:
        t.fill_(7)
    graph.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(want, other, out):
        assert torch.equal(a, b) and torch.equal(a, c)
