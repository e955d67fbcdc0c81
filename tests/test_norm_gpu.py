"""Layer norm of equivariant features on the GPU against the float64 oracle.

Tolerances.  With s = max|x| r of a row, xh = (x - mu) r is computed in fp32 from
a mean whose error is at most ~32 roundings of max|x|: 64 * 2^-24 * s with the
variance's, the subtraction's and the product's.  The output adds half a step of
its type, half a least subnormal of fp16, and the affine's fp32 rounding.
"""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import group_dft_structured_b200 as F
from group_dft_structured_b200 import layer as L
from oracle import feql_ops_oracle as O

pytestmark = pytest.mark.gpu

EPS = 1e-5
U = 2.0 ** -24
HALF = {np.float16: 2.0 ** -11, np.float32: U}
TINY = {np.float16: 2.0 ** -25, np.float32: 0.0}


@pytest.fixture(scope="module", autouse=True)
def ready():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from group_dft_structured_b200 import build
    build.build()
    F.load()


def inputs(N, C, T, dt, mean=0.3, scale=1.0, seed=0):
    r = np.random.default_rng(seed + 31 * N + 7 * C + T)
    x = (r.standard_normal((N, C, T)) * scale + mean).astype(dt)
    dy = r.standard_normal((N, C, T)).astype(dt)
    gamma = (1 + 0.1 * r.standard_normal(C)).astype(dt)
    beta = (0.1 * r.standard_normal(C)).astype(dt)
    return x, dy, gamma, beta


def cuda(a):
    return None if a is None else torch.from_numpy(a).cuda()


def f64(a):
    return None if a is None else a.astype(np.float64)


def within(got, ref, tol, what):
    got = got.detach().cpu().numpy().astype(np.float64)
    assert got.shape == ref.shape, what
    bad = np.abs(got - ref) > tol
    worst = np.max(np.abs(got - ref) - tol) if got.size else 0
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, by {worst:.3g}"


def check(x, dy, gamma, beta, got_y, got_stats, grads):
    dt = x.dtype.type
    N, C, T = x.shape
    X, DY, G, Bt = f64(x), f64(dy), f64(gamma), f64(beta)
    y, mu, r = O.norm_forward(X, G, Bt, EPS)
    g1 = np.ones(C) if G is None else np.abs(G)
    b1 = np.zeros(C) if Bt is None else np.abs(Bt)
    s = (np.abs(X).max(axis=(1, 2)) * r)[:, None, None] + 1
    within(got_y, y, HALF[dt] * np.abs(y) + TINY[dt] +
           64 * U * s * g1[None, :, None] + 4 * U * b1[None, :, None], "y")
    within(got_stats[:, 0], mu, 32 * U * np.abs(X).max(axis=(1, 2)), "mean")
    within(got_stats[:, 1], r, 64 * U * s[:, 0, 0] * r, "rstd")
    dx, dg, db = O.norm_backward(X, DY, G, EPS)
    xh = (X - mu[:, None, None]) * r[:, None, None]
    # each of dx's three terms is off by the error of xh and some 64 roundings
    gmax = (np.abs(DY) * g1[None, :, None]).max(axis=(1, 2))[:, None, None]
    xmax = np.abs(xh).max(axis=(1, 2))[:, None, None]
    within(grads[0], dx, HALF[dt] * np.abs(dx) + TINY[dt] +
           r[:, None, None] * 64 * U * gmax * (1 + 2 * s * (1 + xmax)), "dx")
    # fp32 sums of N T terms in a tree of at most ~N T / 1000 + 64 sequential adds
    depth = N * T / 1000 + 64
    mag = (np.abs(DY) * (np.abs(xh) + 64 * s)).sum(axis=(0, 2))
    within(grads[1], dg, HALF[dt] * np.abs(dg) + TINY[dt] + depth * U * mag, "dgamma")
    within(grads[2], db, HALF[dt] * np.abs(db) + TINY[dt] +
           depth * U * np.abs(DY).sum(axis=(0, 2)), "dbeta")


def run(x, dy, gamma, beta):
    X, G = cuda(x), cuda(gamma)
    y, stats = L.norm_forward(X, G, cuda(beta), EPS)
    return y, stats, L.norm_backward(cuda(dy), X, stats, G)


SHAPES = [
    (1, 1, 1), (5, 1, 2), (7, 3, 1), (300, 24, 4), (33, 16, 4), (129, 67, 6), (64, 5, 3),
    (257, 12, 8), (19, 192, 4), (1000, 11, 12), (9, 100, 16), (4, 1024, 4),
    (3, 1025, 8), (2, 513, 16), (5, 331, 3), (3, 4096, 4), (2, 2500, 16), (3, 4099, 8),
    (70, 9001, 4), (2, 20001, 3), (515, 8, 1), (40, 25, 5), (30, 510, 2),
]


@pytest.mark.parametrize("dt", [np.float16, np.float32])
@pytest.mark.parametrize("N,C,T", SHAPES)
def test_parity(N, C, T, dt):
    x, dy, gamma, beta = inputs(N, C, T, dt)
    check(x, dy, gamma, beta, *run(x, dy, gamma, beta))


@pytest.mark.parametrize("dt", [np.float16, np.float32])
@pytest.mark.parametrize("N,C,T", [(40, 4, 6), (333, 12, 10), (21, 340, 6), (50, 64, 2), (9, 96, 14),
                                   (6, 2731, 6), (17, 30, 6), (800, 2, 6), (11, 1540, 2)])
def test_pairs_of_a_channel(N, C, T, dt):
    """T even but no multiple of four: parameters and sums are shared by two."""
    x, dy, gamma, beta = inputs(N, C, T, dt)
    check(x, dy, gamma, beta, *run(x, dy, gamma, beta))


@pytest.mark.parametrize("dt", [np.float16, np.float32])
def test_parity_without_affine_and_many_rows(dt):
    x, dy, _, _ = inputs(40000, 6, 4, dt)
    check(x, dy, None, None, *run(x, dy, None, None))


@pytest.mark.parametrize("mean,scale", [(1000.0, 1.0), (0.0, 1e-4), (0.0, 8000.0), (-30000.0, 40.0)])
def test_rows_far_from_zero_and_small_or_large(mean, scale):
    x, dy, gamma, beta = inputs(77, 24, 4, np.float16, mean, scale)
    check(x, dy, gamma, beta, *run(x, dy, gamma, beta))


def test_constant_rows_give_beta():
    x = np.full((6, 24, 4), 3.25, np.float16)
    _, _, gamma, beta = inputs(6, 24, 4, np.float16)
    y, stats = L.norm_forward(cuda(x), cuda(gamma), cuda(beta), EPS)
    assert torch.equal(y, cuda(beta)[None, :, None].expand(6, 24, 4))
    assert torch.isfinite(stats).all()


def test_bad_rows_stay_alone():
    x, _, gamma, beta = inputs(50, 24, 4, np.float16)
    clean = L.norm_forward(cuda(x), cuda(gamma), cuda(beta), EPS)[0]
    x[3, 5, 1], x[20, 0, 0] = np.nan, np.inf
    y = L.norm_forward(cuda(x), cuda(gamma), cuda(beta), EPS)[0]
    keep = [i for i in range(50) if i not in (3, 20)]
    assert torch.equal(y[keep], clean[keep])
    assert y[3].isnan().all() and y[20].isnan().all()


def test_no_rows():
    x = torch.zeros(0, 24, 4, dtype=torch.float16, device="cuda")
    y, stats = L.norm_forward(x)
    dx, dg, db = L.norm_backward(x, x, stats)
    assert y.shape == dx.shape == (0, 24, 4) and not dg.any() and not db.any()


def test_strides_alignment_and_repeatability():
    x, dy, gamma, beta = inputs(333, 24, 4, np.float16)
    want = run(x, dy, gamma, beta)
    odd = torch.empty(333 * 96 + 1, dtype=torch.float16, device="cuda")[1:].view(333, 24, 4)
    odd.copy_(cuda(x))
    turned = cuda(dy).permute(2, 0, 1).contiguous().permute(1, 2, 0)
    y, stats = L.norm_forward(odd, cuda(gamma), cuda(beta), EPS)
    dx, dg, db = L.norm_backward(turned, odd, stats, cuda(gamma))
    for a, b in zip((y, stats, dx, dg, db), (want[0], want[1], *want[2])):
        assert torch.equal(a, b)


def test_another_stream_and_a_captured_graph():
    x, dy, gamma, beta = inputs(333, 24, 4, np.float16)
    want = run(x, dy, gamma, beta)
    X, DY, G, Bt = cuda(x), cuda(dy), cuda(gamma), cuda(beta)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        y, stats = L.norm_forward(X, G, Bt, EPS)
        L.norm_backward(DY, X, stats, G)
    side.synchronize()
    with torch.cuda.graph(graph, stream=side):
        y2, stats2 = L.norm_forward(X, G, Bt, EPS)
        grads = L.norm_backward(DY, X, stats2, G)
    assert torch.equal(y, want[0])
    for _ in range(2):
        for t in (y2, stats2, *grads):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((y2, stats2, *grads), (want[0], want[1], *want[2])):
            assert torch.equal(a, b)


def test_refusals():
    x = torch.zeros(4, 8, 4, dtype=torch.float16, device="cuda")
    with pytest.raises(ValueError):
        L.norm_forward(x, torch.zeros(7, dtype=torch.float16, device="cuda"))
    with pytest.raises(TypeError):
        L.norm_forward(x, torch.zeros(8, device="cuda"))
    with pytest.raises(ValueError):
        L.norm_forward(x, torch.zeros(8, dtype=torch.float16))
    with pytest.raises(F.FeqlError):
        L.norm_forward(x, eps=0.0)
    with pytest.raises(F.FeqlError):
        L.norm_forward(torch.zeros(4, 8, 17, dtype=torch.float16, device="cuda"))
    with pytest.raises(ValueError):
        L.norm_backward(x, x, torch.zeros(3, 2, device="cuda"))
