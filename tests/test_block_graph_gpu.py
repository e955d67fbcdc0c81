"""A training step of the block captured into a graph, the usual way: warm-up on a side
stream, gradients made inside the graph, inputs and weights changed in place between
replays.  (No eager graph of the same parameters is alive at the capture: torch would run
part of the captured backward pass on that graph's stream.)"""

import copy

import pytest

torch = pytest.importorskip("torch")

import group_dft_structured_b200 as F
from group_dft_structured_b200.module import EqScanBlock

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def ready():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from group_dft_structured_b200 import build
    build.build()
    F.load()
    yield
    assert F.feql_device_status() == F.FEQL_OK


def step(block, x, dy, off):
    y, state = block(x, None, off)
    ((y * dy).sum() + state.sum().to(y.dtype)).backward()
    return y


def eager(block, x, dy, off):
    """Outputs and gradients of a copy of the block."""
    b = copy.deepcopy(block)
    for p in b.parameters():
        p.grad = None
    y = step(b, x, dy, off).detach()
    return [y, *(p.grad for p in b.parameters())]


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("C,H,T,group,dtype", [
    (12, 24, 4, "cyclic", torch.float16), (12, 24, 4, "cyclic", torch.float32),
    (6, 10, 8, "p4m", torch.float16)])
def test_training_step(C, H, T, group, dtype, packed):
    torch.manual_seed(9)
    block = EqScanBlock(C, H, T, dtype=dtype, device="cuda", group=group)
    shape = (300, C * T) if packed else (3, 100, C * T)
    off = torch.tensor([0, 80, 80, 290], dtype=torch.int32, device="cuda") if packed else None
    x, dy = (torch.randn(shape, device="cuda").to(dtype) for _ in range(2))
    opt = torch.optim.SGD(block.parameters(), lr=1e-3)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            opt.zero_grad(set_to_none=True)
            step(block, x, dy, off)
            opt.step()
    torch.cuda.current_stream().wait_stream(side)
    opt.zero_grad(set_to_none=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = step(block, x, dy, off).detach()
    for _ in range(3):
        x.normal_()
        dy.normal_()
        if packed:
            off[1:3].add_(7)
        graph.replay()
        torch.cuda.synchronize()
        got = [y, *(p.grad for p in block.parameters())]
        for a, b in zip(got, eager(block, x, dy, off)):
            assert torch.equal(a, b)
        opt.step()  # in place: the next replay's weights


def test_graphed_callable():
    torch.manual_seed(10)
    block = EqScanBlock(12, 24, 4, device="cuda")
    x = torch.randn(2, 64, 48, device="cuda").half().requires_grad_()
    run = torch.cuda.make_graphed_callables(copy.deepcopy(block), (x.detach().clone().requires_grad_(),))
    twin = copy.deepcopy(block)
    for k in range(3):
        with torch.no_grad():
            x.copy_(torch.randn_like(x))
            for p, q in zip(run.parameters(), twin.parameters()):
                p.mul_(1.0 + 0.1 * k)
                q.copy_(p)
        outs = []
        for f, m in ((run, run), (twin, twin)):
            x.grad = None
            for p in m.parameters():
                p.grad = None
            y, s = f(x)
            (y.float().square().sum() + s.sum()).backward()
            outs.append([y.detach().clone(), s.detach().clone(), x.grad.clone(),
                         *(p.grad.clone() for p in m.parameters())])
        for a, b in zip(*outs):
            assert torch.equal(a, b)
