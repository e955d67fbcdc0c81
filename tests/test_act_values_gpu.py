"""The activations of the layer's epilogue at chosen values, in every kernel that has one.

A layer without activation and bias shows z itself: the same products, rounded once.
"""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import group_dft_structured_b200 as F
from group_dft_structured_b200 import layer as L

pytestmark = pytest.mark.gpu

# group, T, mode, channels: each kernel family and data type
LAYERS = [("cyclic", 4, "fp16", 16), ("cyclic", 4, "fp16", 70), ("cyclic", 8, "fp16", 12),
          ("cyclic", 6, "fp16", 16), ("p4m", 8, "fp16", 12), ("cyclic", 4, "fp16_simt", 7),
          ("cyclic", 6, "fp16", 5), ("cyclic", 4, "fp32_3xtf32", 24), ("cyclic", 4, "fp32_simt", 9),
          ("cyclic", 5, "fp32", 6)]


@pytest.fixture(scope="module", autouse=True)
def ready():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from group_dft_structured_b200 import build
    build.build()
    F.load()
    yield
    assert F.feql_device_status() == F.FEQL_OK


def calls(group):
    return ((L.p4m_weight_fft, L.p4m_forward, L.p4m_forward_act, L.p4m_backward_act)
            if group == "p4m" else
            (L.ct_weight_fft, L.ct_forward, L.ct_forward_act, L.ct_backward_act))


@pytest.mark.parametrize("save", [False, True])
@pytest.mark.parametrize("act", ["relu", "gelu", "silu"])
@pytest.mark.parametrize("group,T,mode,C", LAYERS)
def test_values_that_are_no_numbers_stay_so(group, T, mode, C, act, save):
    """A NaN in a token is a NaN in its outputs and slopes, and nowhere else; an
    infinity never ends as a finite value (z = -inf under ReLU excepted: 0)."""
    wfft, plain, forward, _ = calls(group)
    code = F.DTYPES[mode]
    dt = L.torch_dtype(code)
    r = np.random.default_rng(C + T)
    x = torch.from_numpy(r.standard_normal((300, C, T))).to(dt).cuda()
    W = torch.from_numpy(r.standard_normal((C, C, T)) / np.sqrt(C * T)).to(dt).cuda()
    res = torch.from_numpy(r.standard_normal((300, C, T))).to(dt).cuda()
    What = wfft(W, code)
    clean = [forward(x, What, None, C, code, F.ACTIVATIONS[act], res=q, save_z=save)
             for q in (None, res)]
    x[3, C // 2, 1], x[200, 0, 0], x[130, 1, 0] = float("nan"), float("inf"), float("-inf")
    z = plain(x, What, None, C, code)
    good = [i for i in range(300) if i not in (3, 130, 200)]
    assert z[3].isnan().all() and torch.isfinite(z[good]).all()
    for q, (y0, s0) in zip((None, res), clean):
        y, s = forward(x, What, None, C, code, F.ACTIVATIONS[act], res=q, save_z=save)
        assert torch.equal(y[good], y0[good]) and y[3].isnan().all()
        assert y[z.isnan()].isnan().all()
        assert not torch.isfinite(y[z == float("inf")]).any()
        if act != "relu":
            assert y[z == float("-inf")].isnan().all()
        if s is not None:
            assert torch.equal(s[good], s0[good])
            if act != "relu":  # ReLU's slope is 0 or 1, the side of a NaN is not 0
                assert s[z.isnan()].isnan().all()
                assert s[z == float("-inf")].isnan().all()


def act64(name, z):
    """act(z), act'(z), and what their arithmetic is made of: p, q, v, v'."""
    if name == "relu":
        one = (z > 0).astype(np.float64)
        return z * one, one, one, 1 - one, np.zeros_like(z), np.zeros_like(z)
    k0, k1 = np.sqrt(2 / np.pi), 0.044715
    v, dv = (z, np.ones_like(z)) if name == "silu" else (2 * k0 * (z + k1 * z ** 3),
                                                        2 * k0 * (1 + 3 * k1 * z * z))
    e = np.exp(-np.abs(v))
    p, q = np.where(v >= 0, 1, e) / (1 + e), np.where(v >= 0, e, 1) / (1 + e)
    return z * p, p + z * p * q * dv, p, q, v, dv


@pytest.mark.parametrize("act", ["relu", "gelu", "silu"])
@pytest.mark.parametrize("group,T,mode,C", LAYERS)
def test_an_identity_layer_shows_the_activation(group, T, mode, C, act):
    """Values that the layer passes on exactly (one group element of a fibre alone), to
    about a step of the type: the erf form of GELU, 5e-4 from the tanh form, would show.

    p = sigma(v) is off by the argument's three roundings, 2^-22 |v| of it, and by the
    exponential's and the reciprocal's 2^-21 together, relative; q = 1 - p in fp16 by
    that and a rounding of 2^-24, absolute.  y = z p, slope = p + y q v', and half a step.
    """
    wfft, plain, forward, _ = calls(group)
    code = F.DTYPES[mode]
    dt = L.torch_dtype(code)
    W = torch.zeros(C, C, T, device="cuda", dtype=dt)
    W[range(C), range(C), 0] = 1
    v = np.concatenate([np.linspace(-12, 12, 1201), np.geomspace(1e-3, 200, 300),
                        -np.geomspace(1e-3, 200, 300), [0.0, 60000.0, -60000.0]])
    x = torch.zeros(-(-len(v) // C), C, T, device="cuda", dtype=dt)
    x[..., 0] = torch.from_numpy(np.resize(v, x.shape[:2])).half().to(dt)
    What = wfft(W, code)
    z = plain(x, What, None, C, code)
    # Every bin of a fibre (v, 0, .., 0) is v itself, and the inverse adds up to three bins'
    # multiples of v by 1/T, 2/T and cosines: a power of two for T, exact; else each
    # constant, product and sum is off by 2^-24 of v at most, eight of them in all, in the
    # fibre's other elements too.
    exact = T != 6 and T != 5
    slack = 0 if exact else 8 * 2.0 ** -24 * x.abs().amax(2, keepdim=True)
    assert ((z - x).abs() <= slack + (0 if exact else torch.finfo(dt).eps / 2) * x.abs()).all()
    y, s = forward(x, What, None, C, code, F.ACTIVATIONS[act], save_z=True)
    Z = x.cpu().numpy().astype(np.float64)
    wy, ws, p, q, arg, dv = act64(act, Z)
    half = torch.finfo(dt).eps / 2
    tiny = 2.0 ** -25 if dt == torch.float16 else 2.0 ** -126
    eps = 2.0 ** -21 + 2.0 ** -22 * np.abs(arg)
    off = 0 if exact else 8 * 2.0 ** -24 * np.abs(Z).max(axis=2, keepdims=True)  # of z
    ty = half * np.abs(wy) + eps * np.abs(wy) + tiny + 1.13 * off
    ts = half * np.abs(ws) + eps * p + np.abs(wy * dv) * (2.0 ** -23 + 2 * eps * q + eps * p) \
        + tiny + 2.0 ** -23 + off
    if act == "relu":  # its slope is exact, on either side of a z that is not rounded
        ts = np.where(np.abs(Z) > off, 0.0, 1.0)
    assert (np.abs(y.cpu().numpy().astype(np.float64) - wy) <= ty).all()
    assert (np.abs(s.cpu().numpy().astype(np.float64) - ws) <= ts).all()
