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
