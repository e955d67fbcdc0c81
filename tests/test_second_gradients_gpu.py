"""Gradients of gradients: no backward pass of the modules is differentiable itself, and each
says so rather than leave its part out."""

import pytest

torch = pytest.importorskip("torch")

import group_dft_structured_b200 as F
from group_dft_structured_b200.module import EqLinear, EqNorm, EqScan, EqScanBlock

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def ready():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from group_dft_structured_b200 import build
    build.build()
    F.load()


KW = dict(device="cuda", dtype=torch.float32)
MODULES = [lambda: EqLinear(4, 4, **KW), lambda: EqLinear(4, 4, activation="silu", **KW),
           lambda: EqNorm(4, **KW), lambda: (lambda x, scan=EqScan(4): scan(x, x)[0]),
           lambda: (lambda x, b=EqScanBlock(4, 8, **KW): b(x)[0])]


@pytest.mark.parametrize("make", MODULES)
def test_refused(make):
    m = make()
    x = torch.randn(2, 9, 16, device="cuda").requires_grad_()
    y = m(x).square()
    g, = torch.autograd.grad(y.sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        # a penalty on the gradient beside an ordinary loss, which alone has a gradient
        (y.sum() + g.square().sum()).backward()
