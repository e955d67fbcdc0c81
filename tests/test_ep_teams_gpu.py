"""Layers on either side of the rule that deals out the tensor-core kernels' epilogue teams
(many input channels to an output, or few), in every kind of epilogue: against the layer
without activation, whose epilogue is another one.

Tolerance: the layer's z is known to half a step of its type (the plain layer's output);
no activation's slope exceeds 1.13 and none changes faster than z, so y is within 1.13 of
that half step and its own, and the saved slope within one half step of z and its own
(activations to 2^-20).
"""

import pytest

torch = pytest.importorskip("torch")

import group_dft_structured_b200 as F
from group_dft_structured_b200 import layer as L

pytestmark = pytest.mark.gpu

K0, K1 = (2 / torch.pi) ** 0.5, 0.044715


@pytest.fixture(scope="module", autouse=True)
def ready():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from group_dft_structured_b200 import build
    build.build()
    F.load()
    yield
    assert F.feql_device_status() == F.FEQL_OK


def act(name, z):
    if name == "none":
        return z, torch.ones_like(z)
    if name == "relu":
        return z.clamp_min(0), (z > 0).double()
    v, dv = (z, 1.0) if name == "silu" else (2 * K0 * (z + K1 * z ** 3),
                                            2 * K0 * (1 + 3 * K1 * z * z))
    p = torch.sigmoid(v)
    return z * p, p + z * p * (1 - p) * dv


@pytest.mark.parametrize("name", ["none", "relu", "gelu", "silu"])
@pytest.mark.parametrize("mode", ["fp16", "fp32_3xtf32"])
@pytest.mark.parametrize("N,C,D", [
    (1000, 192, 8), (1000, 96, 24), (40000, 96, 32), (300, 192, 96), (20000, 192, 192),
    (129, 256, 64), (700, 128, 64), (700, 126, 66), (30000, 64, 64), (500, 24, 96), (77, 2, 2),
    (1, 300, 16), (20000, 70, 34)])
def test_epilogue(N, C, D, mode, name):
    code = F.DTYPES[mode]
    dt = L.torch_dtype(code)
    torch.manual_seed(N + C + D)
    x = torch.randn(N, C, 4, device="cuda").to(dt)
    W = (torch.randn(D, C, 4, device="cuda") / (4 * C) ** 0.5).to(dt)
    b, res = torch.randn(D, device="cuda").to(dt), torch.randn(N, D, 4, device="cuda").to(dt)
    What = L.ct_weight_fft(W, code)
    z = L.ct_forward(x, What, b, D, code).double()
    half = torch.finfo(dt).eps / 2
    off = half * z.abs() + torch.finfo(dt).smallest_normal * half
    a, s = act(name, z)
    for r in (None, res):
        want = a if r is None else a + r.double()
        y, slope = L.ct_forward_act(x, What, b, D, code, F.ACTIVATIONS[name], res=r, save_z=True)
        tol = 1.13 * off + half * want.abs() + 2.0 ** -20 * (dt == torch.float16) * a.abs() \
            + 2.0 ** -25 * (dt == torch.float16) + 16 * 2.0 ** -24 * (a.abs() + want.abs())
        assert ((y.double() - want).abs() <= tol).all()
        only = L.ct_forward_act(x, What, b, D, code, F.ACTIVATIONS[name], res=r)[0]
        assert torch.equal(y, only)
        if slope is not None:
            tol = off + half * s.abs() + 2.0 ** -20 + 2.0 ** -25
            bad = ~((slope.double() - s).abs() <= tol)
            assert not (bad & ((name != "relu") | (z.abs() > off))).any()
