"""EqLinear on inputs and gradients that are parts of larger tensors, dense but off the
16-byte boundaries that the kernels read from."""

import pytest

torch = pytest.importorskip("torch")

import group_dft_structured_b200 as F
from group_dft_structured_b200.module import EqLinear

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def ready():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from group_dft_structured_b200 import build
    build.build()
    F.load()


@pytest.mark.parametrize("act", ["none", "gelu"])
@pytest.mark.parametrize("C,D,T,group,dtype", [
    (5, 7, 3, "cyclic", torch.float16), (5, 7, 3, "cyclic", torch.float32),
    (4, 8, 4, "cyclic", torch.float16), (3, 5, 4, "cyclic", torch.float32),
    (5, 7, 8, "p4m", torch.float16), (5, 7, 6, "cyclic", torch.float16)])
def test_parts_of_larger_tensors(C, D, T, group, dtype, act):
    torch.manual_seed(C * D)
    m = EqLinear(C, D, T, device="cuda", group=group, dtype=dtype, activation=act)
    big = torch.randn(1 + 41 * C * T, device="cuda").to(dtype)
    x = big[1:].view(41, C * T)
    assert x.is_contiguous() and x.data_ptr() % 16 != 0
    dy = torch.randn(1 + 41 * D * T, device="cuda").to(dtype)[1:].view(41, D * T)
    got = []
    for xi, di in ((x, dy), (x.clone(), dy.clone())):
        leaf = xi.detach().requires_grad_()
        m.zero_grad(set_to_none=True)
        y = m(leaf)
        y.backward(di)
        got.append((y.detach(), leaf.grad, m.weight.grad, m.bias.grad))
    for a, b in zip(*got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("act", ["none", "gelu"])
@pytest.mark.parametrize("C,D,T,group,dtype", [
    (5, 7, 3, "cyclic", torch.float16), (4, 8, 4, "cyclic", torch.float16),
    (3, 5, 4, "cyclic", torch.float32), (5, 7, 8, "p4m", torch.float16)])
def test_parameters_in_one_buffer(C, D, T, group, dtype, act):
    m = EqLinear(C, D, T, device="cuda", group=group, dtype=dtype, activation=act)
    x = torch.randn(41, C * T, device="cuda").to(dtype)
    want = m(x)
    flat = torch.empty(1 + m.weight.numel() + D, device="cuda", dtype=dtype)
    W, b = flat[1:1 + m.weight.numel()].view_as(m.weight), flat[1 + m.weight.numel():]
    with torch.no_grad():
        W.copy_(m.weight)
        b.copy_(m.bias)
    m.weight, m.bias = torch.nn.Parameter(W), torch.nn.Parameter(b)
    assert m.weight.data_ptr() % 16 != 0 and m.bias.data_ptr() % 16 != 0
    y = m(x)
    assert torch.equal(y, want)
    y.sum().backward()
    assert m.weight.grad.isfinite().all() and m.bias.grad.isfinite().all()


def test_gradients_that_are_slices_of_a_larger_one():
    m = EqLinear(5, 7, 3, device="cuda")
    x = torch.randn(9, 15, device="cuda").half().requires_grad_()
    parts = [m(x[i:i + 3]) for i in range(0, 9, 3)]
    torch.cat(parts).square().sum().backward()
    one = x.grad.clone()
    x.grad = None
    m.zero_grad(set_to_none=True)
    m(x).square().sum().backward()
    # the same products row by row
    assert torch.equal(one, x.grad)
