"""The layer with activation and residual in its epilogue, on the GPU against the
float64 oracles of the layer and of the activations.

Tolerances.  z is the layer's output before its rounding: within t max|z| (t =
5e-3 in fp16, 1e-5 in fp32, the layer's own bounds).  No activation's slope
exceeds 1.13, so y is within 1.13 t max|z| + half a step of y; no slope changes
by more than the change of z (ReLU's away from its corner), so the saved slope is
within t max|z| + half a step of it.  The backward pass is given slopes (rounded to
the data type): dz is then off by half a step, inside the layer's bound t on dx,
dW and db, which is relative to their largest value.
"""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import group_dft_structured_b200 as F
from group_dft_structured_b200 import layer as L
from oracle import feql_ct_oracle as OC
from oracle import feql_ops_oracle as OA
from oracle import feql_p4m_oracle as OP

pytestmark = pytest.mark.gpu

HALF = {np.float16: 2.0 ** -11, np.float32: 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def ready():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from group_dft_structured_b200 import build
    build.build()
    F.load()
    yield
    assert F.feql_device_status() == F.FEQL_OK


def cuda(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def host(t):
    return t.detach().cpu().numpy().astype(np.float64)


class Layer:
    def __init__(self, group, T, mode, N, C, D, seed=0):
        self.p4m = group == "p4m"
        self.mode = F.DTYPES[mode]
        self.dt = np.float16 if "16" in mode and "tf32" not in mode else np.float32
        self.tol = 5e-3 if self.dt == np.float16 else 1e-5
        self.O = OP if self.p4m else OC
        r = np.random.default_rng(77 + seed + N + 31 * C + 7 * D + T)
        n = lambda *s: r.standard_normal(s).astype(self.dt)
        self.x, self.dy, self.res, self.z = n(N, C, T), n(N, D, T), n(N, D, T), n(N, D, T)
        self.W = (r.standard_normal((D, C, T)) / np.sqrt(T * C)).astype(self.dt)
        self.b = (0.1 * r.standard_normal(D)).astype(self.dt)
        self.D = D
        fft = L.p4m_weight_fft if self.p4m else L.ct_weight_fft
        self.What = fft(cuda(self.W), self.mode)

    def forward(self, act, res, save_z):
        f = L.p4m_forward_act if self.p4m else L.ct_forward_act
        return f(cuda(self.x), self.What, cuda(self.b), self.D, self.mode, F.ACTIVATIONS[act],
                 res=cuda(self.res) if res else None, save_z=save_z)

    def backward(self, act, **kw):
        f = L.p4m_backward_act if self.p4m else L.ct_backward_act
        return f(cuda(self.x), cuda(self.dy), cuda(self.slope(act)), self.What, self.mode, F.ACTIVATIONS[act], **kw)

    def slope(self, act):
        """Slopes of some activation values, as the forward saves them."""
        if act == "none":
            return None
        return OA.act_slope(act, self.z.astype(np.float64)).astype(self.dt)

    def z64(self):
        return self.O.forward(*(v.astype(np.float64) for v in (self.x, self.W, self.b)))

    def check_forward(self, act, res, y, z):
        ref = self.z64()
        slack = self.tol * np.abs(ref).max()
        want = OA.act(act, ref) + (self.res.astype(np.float64) if res else 0)
        half = HALF[self.dt]
        assert (np.abs(host(y) - want) <= 1.13 * slack + half * np.abs(want) + 2.0 ** -24).all()
        if z is not None:
            s = OA.act_slope(act, ref)
            bad = np.abs(host(z) - s) > slack + half * np.abs(s) + 2.0 ** -24
            assert not (bad & ((act != "relu") | (np.abs(ref) > slack))).any()

    def check_backward(self, act, dx, dW, db):
        x, W, dy = (v.astype(np.float64) for v in (self.x, self.W, self.dy))
        dz = dy if act == "none" else dy * self.slope(act).astype(np.float64)
        rdW, rdb = self.O.backward_dw(x, dz)
        for got, ref in ((dx, self.O.backward_dx(dz, W)), (dW, rdW), (db, rdb)):
            if got is not None:
                assert self.O.rel_err(host(got), ref) <= self.tol


CASES = [
    ("cyclic", 4, "fp16", 1, 2, 2), ("cyclic", 4, "fp16", 127, 6, 10),
    ("cyclic", 4, "fp16", 300, 24, 96), ("cyclic", 4, "fp16", 129, 48, 192),
    ("cyclic", 4, "fp16", 40000, 24, 96), ("cyclic", 4, "fp16", 1000, 70, 130),
    ("cyclic", 4, "fp16", 257, 320, 34), ("cyclic", 4, "fp16_simt", 100, 7, 9),
    ("cyclic", 4, "fp32", 200, 35, 51), ("cyclic", 4, "fp32", 1, 1, 1),
    ("cyclic", 4, "fp32", 33, 520, 6), ("cyclic", 4, "fp32_3xtf32", 130, 16, 24),
    ("cyclic", 4, "fp32_simt", 65, 5, 3), ("cyclic", 8, "fp16", 200, 5, 7),
    ("cyclic", 8, "fp16", 513, 12, 48), ("cyclic", 6, "fp16", 300, 16, 64),
    ("cyclic", 6, "fp16", 300, 4, 92), ("cyclic", 6, "fp16", 100, 5, 7),
    ("cyclic", 8, "fp32", 90, 9, 33), ("cyclic", 3, "fp32", 70, 10, 11),
    ("cyclic", 12, "fp16", 50, 6, 5), ("cyclic", 16, "fp32", 40, 3, 4),
    ("p4m", 8, "fp16", 300, 12, 48), ("p4m", 8, "fp16", 77, 5, 9),
]


@pytest.mark.parametrize("res", [False, True])
@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu"])
@pytest.mark.parametrize("group,T,mode,N,C,D", CASES)
def test_parity(group, T, mode, N, C, D, act, res):
    m = Layer(group, T, mode, N, C, D)
    y, z = m.forward(act, res, True)
    assert (z is None) == (act == "none")
    m.check_forward(act, res, y, z)
    only_y, none = m.forward(act, res, False)
    assert none is None and torch.equal(only_y, y)
    m.check_backward(act, *m.backward(act))


@pytest.mark.parametrize("group,T,mode,N,C,D", [CASES[2], CASES[5], CASES[8], CASES[14], CASES[22]])
def test_gradient_subsets_and_repeatability(group, T, mode, N, C, D):
    m = Layer(group, T, mode, N, C, D)
    full = m.backward("gelu")
    for a, b in zip(full, m.backward("gelu")):
        assert torch.equal(a, b)
    m.check_backward("gelu", *m.backward("gelu", with_dx=False))
    m.check_backward("gelu", *m.backward("gelu", with_dw=False, with_db=False))
    m.check_backward("gelu", *m.backward("gelu", with_dw=False))
    assert m.backward("gelu", with_dx=False, with_dw=False, with_db=False) == (None, None, None)


@pytest.mark.parametrize("group,T,mode,N,C,D", [CASES[2], CASES[13], CASES[15], CASES[18], CASES[22]])
def test_without_activation_it_is_the_layer(group, T, mode, N, C, D):
    m = Layer(group, T, mode, N, C, D)
    plain = L.p4m_forward if m.p4m else L.ct_forward
    want = plain(cuda(m.x), m.What, cuda(m.b), D, m.mode)
    assert torch.equal(m.forward("none", False, False)[0], want)
    # the residual is added before the rounding: at most half a step from adding it after
    y = m.forward("none", True, False)[0]
    both = host(want) + m.res
    assert (np.abs(host(y) - both) <= HALF[m.dt] * (np.abs(both) + np.abs(host(want))) + 2.0 ** -24).all()


@pytest.mark.parametrize("act", ["gelu", "silu", "relu"])
def test_large_and_small_arguments(act):
    # an identity layer: z = x, so the activation is seen at chosen values
    C = 16
    W = np.zeros((C, C, 4), np.float32)
    W[np.arange(C), np.arange(C), 0] = 1
    v = np.concatenate([np.linspace(-100, 100, 401), np.geomspace(1e-30, 1e3, 200),
                        -np.geomspace(1e-30, 1e3, 200), [0.0, -0.0]]).astype(np.float32)
    x = np.resize(v, (13, C, 4))
    mode = F.FEQL_FP32_SIMT
    What = L.weight_fft(cuda(W), mode)
    z0 = L.forward(cuda(x), What, None, C, mode)  # what the layer makes of x
    y, slope = L.ct_forward_act(cuda(x), What, None, C, mode, F.ACTIVATIONS[act], save_z=True)
    ref = OA.act(act, host(z0))
    # 8 roundings and the argument of the exponential, off by 2^-23 |v| relative
    rel = 2.0 ** -24 * (8 + 4 * np.abs(host(z0)) * (1 + np.abs(host(z0)) ** 2))
    rel = np.minimum(rel, 1)
    # the reference's own 1 + tanh, of two numbers near 1, is off by 2 roundings of
    # 2^-53 (times |z| / 2), which shows where GELU itself is that small
    own = np.abs(host(z0)) * 2.0 ** -53 if act == "gelu" else 0
    assert (np.abs(host(y) - ref) <= rel * np.abs(ref) + own + 1e-36).all()
    dy = np.ones((13, C, 4), np.float32)
    dx, _, _ = L.ct_backward_act(cuda(x), cuda(dy), slope, What, mode, F.ACTIVATIONS[act])
    want = OA.act_slope(act, host(z0))
    assert np.isfinite(host(slope)).all() and np.isfinite(host(dx)).all()
    # the slope's 16 roundings and its exponential's argument, as above, at most 1.13 each
    assert (np.abs(host(slope) - want) <= 1.13 * np.minimum(rel + 2.0 ** -20, 1e-5)).all()
    assert np.abs(host(dx) - want).max() <= 2e-5 * 1.13


@pytest.mark.parametrize("act", ["gelu", "silu", "relu"])
def test_large_arguments_in_fp16(act):
    # z far beyond fp16's range, on the negative side where y is representable
    x = np.full((4, 16, 4), 6e4, np.float16)
    W = np.zeros((16, 16, 4), np.float16)
    W[:, :, 0] = np.where(np.arange(16) < 8, -6e4, -1.0)[:, None]
    for mode in (F.FEQL_FP16, F.FEQL_FP16_SIMT):
        What = L.weight_fft(cuda(W), mode)
        y, slope = L.ct_forward_act(cuda(x), What, None, 16, mode, F.ACTIVATIONS[act], save_z=True)
        assert not y.any() and not slope.any()


def test_relu_keeps_its_side_of_zero_in_fp16():
    # z > 0 below half the least subnormal is still on the side with slope 1
    x = np.full((4, 2, 4), 6e-8, np.float16)
    W = np.zeros((2, 2, 4), np.float16)
    W[:, :, 0] = 0.1
    What = L.weight_fft(cuda(W), F.FEQL_FP16_SIMT)
    for sign, want in ((1, 1.0), (-1, 0.0)):
        y, slope = L.ct_forward_act(cuda(x * np.float16(sign)), What, None, 2, F.FEQL_FP16_SIMT,
                                    F.FEQL_ACT_RELU, save_z=True)
        assert (slope == want).all() and not y.any()


def test_no_tokens():
    for group, T in (("cyclic", 4), ("cyclic", 8), ("cyclic", 3), ("p4m", 8)):
        m = Layer(group, T, "fp16", 0, 4, 8)
        y, z = m.forward("gelu", True, True)
        dx, dW, db = m.backward("gelu")
        assert y.shape == z.shape == (0, 8, T) and dx.shape == (0, 4, T)
        assert not dW.any() and not db.any()


def test_another_stream_and_a_captured_graph():
    m = Layer("cyclic", 4, "fp16", 3000, 24, 96)
    want = (*m.forward("gelu", True, True), *m.backward("gelu"))
    x, dy, z, res, b = cuda(m.x), cuda(m.dy), cuda(m.slope("gelu")), cuda(m.res), cuda(m.b)

    def both():
        y, zs = L.ct_forward_act(x, m.What, b, 96, m.mode, F.FEQL_ACT_GELU, res=res, save_z=True)
        return (y, zs, *L.ct_backward_act(x, dy, z, m.What, m.mode, F.FEQL_ACT_GELU))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = both()
    for _ in range(2):
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, c in zip(out, want):
            assert torch.equal(a, c)


def test_first_cuda_call_of_a_thread():
    # no runtime call has made a context current there
    import threading
    m = Layer("cyclic", 4, "fp16", 300, 24, 96)
    x, b, mode = cuda(m.x), cuda(m.b), m.mode
    want = L.ct_forward_act(x, m.What, b, 96, mode, F.FEQL_ACT_GELU)[0]
    y, got = torch.empty_like(want), []
    stream = torch.cuda.current_stream().cuda_stream
    t = threading.Thread(target=lambda: got.append(F.load().feql_ct_forward_act(
        4, x.data_ptr(), m.What.data_ptr(), b.data_ptr(), None, y.data_ptr(), None, 300, 24, 96,
        F.FEQL_ACT_GELU, mode, stream)))
    t.start()
    t.join()
    assert got == [F.FEQL_OK] and torch.equal(y, want)


def test_refusals():
    m = Layer("cyclic", 4, "fp16", 30, 4, 8)
    x, b, z = cuda(m.x), cuda(m.b), cuda(m.z)
    gelu = F.FEQL_ACT_GELU
    with pytest.raises(F.FeqlError):
        L.ct_forward_act(x, m.What, b, 8, m.mode, 9)
    with pytest.raises(TypeError):
        L.ct_forward_act(x, m.What, b, 8, F.FEQL_FP32, gelu)
    with pytest.raises(ValueError):
        L.ct_forward_act(x, m.What[:-16], b, 8, m.mode, gelu)
    with pytest.raises(ValueError):
        L.ct_forward_act(x, m.What, b, 8, m.mode, gelu, res=cuda(m.res)[:-1])
    with pytest.raises(TypeError):
        L.ct_forward_act(x, m.What, b, 8, m.mode, gelu, res=cuda(m.res).float())
    with pytest.raises(F.FeqlError):
        L.ct_backward_act(x, cuda(m.dy), None, m.What, m.mode, gelu)
    with pytest.raises(ValueError):
        L.ct_backward_act(x, cuda(m.dy), z[:, :4], m.What, m.mode, gelu)
    with pytest.raises(ValueError):
        L.p4m_forward_act(x, m.What, b, 8, m.mode, gelu)
    with pytest.raises((ValueError, F.FeqlError)):
        L.ct_forward_act(torch.zeros(4, 3, 4, dtype=torch.float16, device="cuda"), m.What, None, 8,
                         m.mode, gelu)  # odd channels on the tensor cores
