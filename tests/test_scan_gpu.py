"""Gated linear recurrence on the GPU against the float64 oracle.

Tolerances.  A step multiplies by a and 1 - a, each off by a relative e: the
exponential of |g| <= 12 and the division are off by at most 20 * 2^-23 with the
hardware's functions (fp16 data) and 4 * 2^-23 with the precise ones, and the
products and sums add 4 roundings of 2^-24.  A state is the sum of the parts that
its rows gave, local ones and the carried one, each rounded by its own size, and
parts of both signs may cancel: so roundings count against the sum of the parts'
sizes, M_l = a M_{l-1} + (1 - a) |u|, not against |h|.  The error then obeys the
recurrence itself, E_l = a E_{l-1} + e M_l, which the tests run in float64; the
gradient's the same from the other end, with M_l = |dh_l| + a_{l+1} M_{l+1}.
The gates' gradient takes h_{l-1} from the forward's output: half a step of it off.
Outputs add half a step of their type.
"""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import group_dft_structured_b200 as F
from group_dft_structured_b200 import layer as L
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


def inputs(N, B, C, T, shared, dt, seed=0, mean=2.0):
    r = np.random.default_rng(900 + seed + N + 31 * C + T)
    u = r.standard_normal((N, C, T)).astype(dt)
    g = np.clip(r.standard_normal((N, C) if shared else (N, C, T)) * 1.5 + mean, -12, 12).astype(dt)
    dh = r.standard_normal((N, C, T)).astype(dt)
    h0 = r.standard_normal((B, C, T)).astype(np.float32)
    dhN = r.standard_normal((B, C, T)).astype(np.float32)
    return u, g, dh, h0, dhN


def within(got, ref, tol, what):
    got = got.detach().cpu().numpy().astype(np.float64)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    bad = ~(np.abs(got - ref) <= tol)
    worst = np.max(np.abs(got - ref) - tol) if got.size else 0
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, by {worst:.3g}"


def check(u, g, dh, h0, dhN, off, out):
    dt = u.dtype.type
    e = STEP[dt]
    h, hN, du, dg, dh0 = out
    B = len(off) - 1
    U64, G64, DH = u.astype(np.float64), g.astype(np.float64), dh.astype(np.float64)
    shape = (B, *u.shape[1:])
    H0 = np.zeros(shape) if h0 is None else h0.astype(np.float64)
    DN = np.zeros(shape) if dhN is None else dhN.astype(np.float64)
    rh, rhN = O.scan_forward(U64, G64, H0, off)
    rdu, rdg, rdh0 = O.scan_backward(DH, U64, G64, H0, DN, off)
    gf = np.broadcast_to(G64[..., None], u.shape) if g.ndim < u.ndim else G64
    a, na = O.gates(gf)
    Eh, EhN = np.zeros_like(rh), np.zeros(shape)
    before, Eb = np.zeros_like(rh), np.zeros_like(rh)
    Ed, Md, delta, Ed0 = (np.zeros_like(rh), np.zeros_like(rh), np.zeros_like(rh), np.zeros(shape))
    for b in range(B):
        prev, M = H0[b], np.abs(H0[b])
        for l in range(off[b], off[b + 1]):
            before[l], Eb[l] = prev, EhN[b]
            M = a[l] * M + na[l] * np.abs(U64[l])
            EhN[b] = a[l] * EhN[b] + e * M
            Eh[l], prev = EhN[b], rh[l]
        c, M = DN[b], np.abs(DN[b])
        for l in range(off[b + 1] - 1, off[b] - 1, -1):
            delta[l] = DH[l] + c
            Md[l] = np.abs(DH[l]) + M
            Ed[l] = Ed0[b] + U * Md[l]
            M = a[l] * Md[l]
            Ed0[b] = a[l] * Ed[l] + e * M
            c = a[l] * delta[l]
    half, tiny = HALF[dt], TINY[dt]
    within(h, rh, half * np.abs(rh) + tiny + Eh, "h")
    within(hN, rhN, U * np.abs(rhN) + EhN, "hN")
    if du is None:
        return
    within(du, rdu, half * np.abs(rdu) + tiny + na * (Ed + e * np.abs(delta)), "du")
    diff = np.abs(before - U64)
    Eb = Eb + half * np.abs(before) + tiny
    Eg = a * na * (np.abs(delta) * (Eb + U * (np.abs(before) + np.abs(U64))) + Ed * diff +
                   (2 * e + 4 * U) * np.abs(delta) * diff)
    if g.ndim < u.ndim:
        terms = np.abs(delta * (before - U64) * a * na).sum(-1)
        Eg = Eg.sum(-1) + 16 * U * terms
    within(dg, rdg, half * np.abs(rdg) + tiny + Eg, "dg")
    within(dh0, rdh0, U * np.abs(rdh0) + Ed0, "dh0")


def run(u, g, dh, h0, dhN, off=None, B=None):
    if off is None:  # dense: rows as (B, L)
        shape = lambda v: v.reshape(B, -1, *v.shape[1:])
        U_, G_, D_ = cuda(shape(u)), cuda(shape(g)), cuda(shape(dh))
        o = None
    else:
        U_, G_, D_ = cuda(u), cuda(g), cuda(dh)
        o = torch.tensor(off, dtype=torch.int32, device="cuda")
    h, hN, saved = L.scan_forward(U_, G_, cuda(h0), o)
    du, dg, dh0 = L.scan_backward(D_, U_, G_, saved, cuda(dhN), o)
    flat = (lambda t, v: t.reshape(v.shape))
    return flat(h, u), hN, flat(du, u), flat(dg, g), dh0


DENSE = [  # B, L, C, T
    (1, 1, 1, 1), (1, 2, 3, 1), (3, 5, 2, 2), (2, 31, 5, 3), (4, 64, 24, 4), (2, 257, 7, 4),
    (5, 49, 6, 6), (1, 300, 3, 5), (2, 700, 4, 12), (3, 130, 2, 16), (1, 129, 9, 7),
    (300, 9, 24, 4), (2, 2049, 8, 4), (1, 5000, 6, 4), (1, 4097, 5, 2), (1, 3001, 3, 3),
    (2, 1023, 2, 15), (1, 2500, 1, 8), (700, 3, 16, 8), (1, 40, 40, 13), (1, 34001, 2, 4),
]


@pytest.mark.parametrize("dt", [np.float16, np.float32])
@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("B,L_,C,T", DENSE)
def test_dense(B, L_, C, T, shared, dt):
    u, g, dh, h0, dhN = inputs(B * L_, B, C, T, shared, dt)
    off = [i * L_ for i in range(B + 1)]
    check(u, g, dh, h0, dhN, off, run(u, g, dh, h0, dhN, B=B))


PACKED = [
    ([0, 5, 5, 40, 41, 300], 300), ([0, 0, 0, 17], 17), ([3, 3, 50, 700, 700], 731),
    ([0, 0], 6), ([0, 1500, 1502, 1502, 2100], 2100), ([0, 3000], 3100),
    ([0, 1, 9000, 9000, 9100], 9107),
    (list(range(0, 200)) + [8000] + [8000 + i for i in range(60)], 8070),
    (list(range(0, 401)) + [900], 902),
]


@pytest.mark.parametrize("dt", [np.float16, np.float32])
@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("C,T", [(8, 4), (3, 6), (5, 1), (2, 3)])
@pytest.mark.parametrize("off,N", PACKED)
def test_packed(off, N, C, T, shared, dt):
    B = len(off) - 1
    u, g, dh, h0, dhN = inputs(N, B, C, T, shared, dt)
    check(u, g, dh, h0, dhN, off, run(u, g, dh, h0, dhN, off=off))


@pytest.mark.parametrize("shared", [False, True])
def test_without_states_and_long_memory(shared):
    # gates of about sigma(8): memories of thousands of tokens
    u, g, dh, _, _ = inputs(2 * 3000, 2, 8, 4, shared, np.float16, mean=8.0)
    off = [0, 3000, 6000]
    check(u, g, dh, None, None, off, run(u, g, dh, None, None, B=2))


@pytest.mark.parametrize("dt", [np.float16, np.float32])
@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("B,C,T", [(1, 1, 1), (64, 24, 4), (3, 7, 6), (1000, 33, 3)])
def test_step(B, C, T, shared, dt):
    u, g, _, h0, _ = inputs(B, B, C, T, shared, dt)
    state = cuda(h0)
    h = L.scan_step(cuda(u), cuda(g), state)
    off = list(range(B + 1))
    check(u, g, u, h0, None, off, (h, state, None, None, None))


def test_step_shows_in_the_state_version():
    """A graph that saved the state refuses to go on with the changed one."""
    from group_dft_structured_b200.module import EqScan
    scan = EqScan(8, 4)
    u = torch.randn(2, 5, 32, device="cuda").half().requires_grad_()
    gate = torch.randn(2, 5, 8, device="cuda").half()
    state = torch.zeros(2, 32, device="cuda")
    h, _ = scan(u, gate, state)
    scan.step(u.detach()[:, 0], gate[:, 0], state)
    with pytest.raises(RuntimeError, match="inplace"):
        h.float().sum().backward()
    with torch.inference_mode():
        held = torch.zeros(2, 32, device="cuda")
        scan.step(u.detach()[:, 0], gate[:, 0], held)
    assert torch.equal(held, state)


def test_steps_continue_a_scan():
    u, g, _, h0, _ = inputs(2 * 40, 2, 24, 4, False, np.float16)
    U_, G_ = cuda(u).view(2, 40, 24, 4), cuda(g).view(2, 40, 24, 4)
    h, hN, _ = L.scan_forward(U_, G_, cuda(h0), save=False)
    _, state, _ = L.scan_forward(U_[:, :33], G_[:, :33], cuda(h0), save=False)
    for l in range(33, 40):
        out = L.scan_step(U_[:, l], G_[:, l], state)
        # the two orders of summation differ by a few fp32 roundings of values below 8
        assert (out.float() - h[:, l].float()).abs().max() <= 2.0 ** -8
    assert (state - hN).abs().max() <= 1e-5


@pytest.mark.parametrize("T", [1, 4])
def test_infinite_gates_and_bad_values_stay_in_their_sequence(T):
    u, g, dh, h0, dhN = inputs(600, 3, 8, T, False, np.float32)
    off = [0, 200, 400, 600]
    clean = run(u, g, dh, h0, dhN, off=off)
    g[10], g[20] = np.inf, -np.inf      # shut and open: finite results, as the formula gives
    u[250, 2], g[300, 1] = np.nan, np.nan
    out = run(u, g, dh, h0, dhN, off=off)
    for i in (0, 2, 3):
        assert torch.equal(out[i][400:], clean[i][400:])
        assert torch.isfinite(out[i][:200]).all()
    assert torch.equal(out[1][2], clean[1][2]) and torch.equal(out[4][2], clean[4][2])
    assert torch.equal(out[0][20], cuda(u)[20])
    assert torch.equal(out[0][10], out[0][9])
    h = out[0][200:400]
    assert h[50:, 2].isnan().all() and torch.isfinite(h[:50]).all() and h[100:, 1].isnan().all()
    assert torch.isfinite(h[:, 3:]).all()


def test_offsets_beyond_the_rows_are_clamped():
    # nothing is read or written outside; the rows that lie inside are as always
    u, g, dh, h0, dhN = inputs(100, 2, 8, 4, False, np.float16)
    good = run(u, g, dh, h0, dhN, off=[0, 60, 100])
    over = run(u, g, dh, h0, dhN, off=[-7, 60, 1 << 30])
    for a, b in zip(good, over):
        assert torch.equal(a, b)


@pytest.mark.parametrize("packed", [False, True])
def test_repeatable_on_another_stream_and_in_a_graph(packed):
    B, L_ = 3, 700
    u, g, dh, h0, dhN = inputs(B * L_, B, 24, 4, True, np.float16)
    off = [0, 10, 1500, B * L_] if packed else None
    want = run(u, g, dh, h0, dhN, off=off, B=B)
    shape = (lambda v: v) if packed else (lambda v: v.reshape(B, L_, *v.shape[1:]))
    U_, G_, D_, H_, N_ = (cuda(v) for v in (shape(u), shape(g), shape(dh), h0, dhN))
    o = torch.tensor(off, dtype=torch.int32, device="cuda") if packed else None
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        h, hN, saved = L.scan_forward(U_, G_, H_, o)
        L.scan_backward(D_, U_, G_, saved, N_, o)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        h, hN, saved = L.scan_forward(U_, G_, H_, o)
        out = (h, hN, *L.scan_backward(D_, U_, G_, saved, N_, o))
    for _ in range(2):
        for t in out:
            t.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a.reshape(b.shape), b)


def test_strides_and_alignment():
    u, g, dh, h0, dhN = inputs(2 * 90, 2, 6, 4, False, np.float16)
    want = run(u, g, dh, h0, dhN, B=2)
    big = torch.empty(2, 90, 13, 4, dtype=torch.float16, device="cuda")
    U_, G_ = big[:, :, :6], big[:, :, 7:]
    U_.copy_(cuda(u).view(2, 90, 6, 4))
    G_.copy_(cuda(g).view(2, 90, 6, 4))
    odd = torch.empty(2 * 90 * 24 + 1, dtype=torch.float16, device="cuda")[1:].view(2, 90, 6, 4)
    odd.copy_(cuda(dh).view(2, 90, 6, 4))
    h, hN, saved = L.scan_forward(U_, G_, cuda(h0))
    out = (h, hN, *L.scan_backward(odd, U_, G_, saved, cuda(dhN)))
    for a, b in zip(out, want):
        assert torch.equal(a.reshape(b.shape), b)


def test_no_sequences_and_no_rows():
    e = torch.zeros(0, 5, 6, 4, dtype=torch.float16, device="cuda")
    h, hN, saved = L.scan_forward(e, e)
    du, dg, dh0 = L.scan_backward(e, e, e, saved)
    assert h.shape == du.shape == (0, 5, 6, 4) and hN.shape == dh0.shape == (0, 6, 4)
    e = torch.zeros(2, 0, 6, 4, dtype=torch.float16, device="cuda")
    h0 = torch.randn(2, 6, 4, device="cuda")
    h, hN, saved = L.scan_forward(e, e, h0)
    assert torch.equal(hN, h0)
    du, dg, dh0 = L.scan_backward(e, e, e, saved, h0)
    assert torch.equal(dh0, h0)


def test_refusals():
    u = torch.zeros(2, 5, 6, 4, dtype=torch.float16, device="cuda")
    off = torch.tensor([0, 10], dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError):
        L.scan_forward(u, u.float())
    with pytest.raises(TypeError):
        L.scan_forward(u, u, torch.zeros(2, 6, 4, dtype=torch.float16, device="cuda"))
    with pytest.raises(ValueError):
        L.scan_forward(u, u, torch.zeros(3, 6, 4, device="cuda"))
    with pytest.raises(TypeError):
        L.scan_forward(u.view(10, 6, 4), u.view(10, 6, 4), offsets=off.long())
    with pytest.raises(ValueError):
        L.scan_forward(u.view(10, 6, 4), u.view(10, 6, 4), offsets=off.cpu())
    with pytest.raises(ValueError):
        L.scan_forward(u, u, offsets=off)
    h, hN, saved = L.scan_forward(u, u)
    with pytest.raises(ValueError):
        L.scan_backward(u, u, u, (h[:, :4], None))
    with pytest.raises(ValueError):
        L.scan_backward(u[:, :4], u, u, saved)
    state = torch.zeros(6, 2, 4, device="cuda").permute(1, 0, 2)
    with pytest.raises(ValueError):
        L.scan_step(u[:, 0], u[:, 0], state)
    with pytest.raises(TypeError):
        L.scan_step(u[:, 0], u[:, 0], torch.zeros(2, 6, 4, device="cuda").half())


@pytest.mark.parametrize("dt", [np.float16, np.float32])
@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("B,L_", [(306, 530), (452, 261), (600, 300), (620, 2001)])
def test_last_round_of_sequences_cut(B, L_, shared, dt):
    """More sequences than run at a time: those of a short last round are cut."""
    C, T, K = 8, 4, 4  # K sequences, repeated
    u, g, dh, h0, dhN = inputs(K * L_, K, C, T, shared, dt)

    def tiled(v, per):
        v = v.reshape(K, per, *v.shape[1:]) if per else v
        return cuda(np.concatenate([v] * (B // K + 1))[:B])

    h, hN, saved = L.scan_forward(tiled(u, L_), tiled(g, L_), tiled(h0, 0))
    # backward may cut others than forward does: both kinds read the first one's h
    of = torch.arange(B, device="cuda") % K
    saved = (saved[0][:K][of], saved[1])
    du, dg, dh0 = L.scan_backward(tiled(dh, L_), tiled(u, L_), tiled(g, L_), saved, tiled(dhN, 0))
    out = (h, hN, du, dg, dh0)
    ends = [list(range(K)), [B - K + (k - B) % K for k in range(K)]]  # first and last of each
    like = (u, h0, u, g, h0)
    for pick in ends:
        check(u, g, dh, h0, dhN, [i * L_ for i in range(K + 1)],
              [t[pick].reshape(v.shape) for t, v in zip(out, like)])
    for t in out:  # whole or cut alike: the bits of one or of the other
        same = [(t == t[pick][of]).flatten(1).all(1) for pick in ends]
        assert bool((same[0] | same[1]).all())
