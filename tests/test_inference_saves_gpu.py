"""What the modules save for a backward pass: nothing where no gradients are recorded, though
their parameters want them; the results are the same bits."""

import pytest

torch = pytest.importorskip("torch")

import group_dft_structured_b200 as F
from group_dft_structured_b200 import module as M
from group_dft_structured_b200.module import EqLinear, EqNorm, EqScan, EqScanBlock

pytestmark = pytest.mark.gpu

KINDS = [lambda: EqLinear(6, 6, 4, device="cuda", activation="gelu"),
         lambda: EqLinear(6, 6, 8, device="cuda", group="p4m", activation="silu"),
         lambda: EqNorm(6, device="cuda"), lambda: (lambda x, s=EqScan(6): s(x, x)[0]),
         lambda: (lambda x, b=EqScanBlock(6, 12, device="cuda"): b(x)[0])]


@pytest.fixture
def asked(monkeypatch):
    """Whether each call of the library was to save something."""
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from group_dft_structured_b200 import build
    build.build()
    F.load()
    seen = []
    for name, flag in (("ct_forward_act", "save_z"), ("p4m_forward_act", "save_z"),
                       ("norm_forward", "save_stats"), ("scan_forward", "save")):
        def wrapped(*a, _f=getattr(M._L, name), _k=flag, **kw):
            seen.append(kw[_k])
            return _f(*a, **kw)
        monkeypatch.setattr(M._L, name, wrapped)
    return seen


@pytest.mark.parametrize("make", KINDS)
@pytest.mark.parametrize("mode", [torch.no_grad, torch.inference_mode])
def test_nothing_is_saved_without_gradients(asked, make, mode):
    m = make()
    T = 8 if getattr(m, "group_order", 4) == 8 else 4
    x = torch.randn(2, 30, 6 * T, device="cuda").half().requires_grad_()
    want = m(x)
    assert any(asked)
    asked.clear()
    with mode():
        y = m(x)
    assert asked and not any(asked) and torch.equal(y, want)
    asked.clear()
    with torch.no_grad():
        with torch.enable_grad():
            m(x).sum().backward()
    assert any(asked) and x.grad.isfinite().all()
