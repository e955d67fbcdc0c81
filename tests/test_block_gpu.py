"""The operators as a network uses them: the modules EqLinear (activation,
residual), EqNorm, EqScan and the residual block EqScanBlock made of them, with
autograd, against the same block in float64 on the CPU, against differences,
under the group's action, and token by token.

Tolerances, relative to the largest value of each tensor.  A layer is within 1e-5
(fp32) or 5e-3 (fp16) of its output's largest value; a path through the block
crosses at most five layers, and norms and gates pass an error on with a factor
of at most some two each: 10 layers' bounds for outputs, and 20 for gradients,
which cross the block twice.
"""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import group_dft_structured_b200 as F
from group_dft_structured_b200.module import (EqLinear, EqNorm, EqScan, EqScanBlock,
                                              p4m_kernel_index)
from oracle.feql_ops_oracle import K0, K1

LAYER = {torch.float16: 5e-3, torch.float32: 1e-5}


# ------------------------------------------------------------------ CPU ---

def test_constructors_refuse():
    with pytest.raises(ValueError):
        EqLinear(4, 4, activation="tanh")
    with pytest.raises(TypeError):
        EqNorm(4, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        EqNorm(4)(torch.zeros(3, 12, dtype=torch.float16))
    with pytest.raises(ValueError):
        EqScan(4)(torch.zeros(1, 3, 16), torch.zeros(1, 3, 8))
    with pytest.raises(ValueError):
        EqScan(4)(torch.zeros(1, 3, 12), torch.zeros(1, 3, 12))


def test_modules_have_no_cpu_path():
    x = torch.zeros(2, 3, 16, dtype=torch.float16)
    for f in (lambda: EqNorm(4)(x), lambda: EqScan(4)(x, x),
              lambda: EqLinear(4, 4, activation="gelu")(x)):
        with pytest.raises((ValueError, RuntimeError)):
            f()


# ------------------------------------------------------------------ GPU ---

@pytest.fixture
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from group_dft_structured_b200 import build
    build.build()
    F.load()
    torch.manual_seed(5)
    yield
    assert F.feql_device_status() == F.FEQL_OK


def unrolled(W, group):
    D, C, T = W.shape
    if group == "p4m":
        u = torch.tensor([[p4m_kernel_index(g, h) for h in range(8)] for g in range(8)])
    else:
        t = torch.arange(T)
        u = (t[:, None] - t[None, :]) % T
    return W[:, :, u].permute(0, 2, 1, 3).reshape(D * T, C * T)


class Reference:
    """The block in float64 on the CPU, from the block's own parameters."""

    def __init__(self, block, group, T):
        self.p = {k: v.detach().cpu().double().requires_grad_(True)
                  for k, v in block.named_parameters()}
        self.group, self.T = group, T

    def linear(self, name, x):
        A = unrolled(self.p[name + ".weight"], self.group)
        return x @ A.t() + self.p[name + ".bias"].repeat_interleave(self.T)

    def norm(self, name, x):
        d = x - x.mean(-1, keepdim=True)
        n = d / (d.square().mean(-1, keepdim=True) + 1e-5).sqrt()
        return (n * self.p[name + ".weight"].repeat_interleave(self.T)
                + self.p[name + ".bias"].repeat_interleave(self.T))

    def __call__(self, x, state, offsets):
        """x (N, C*T), state (B, C*T): y, state."""
        n = self.norm("norm1", x)
        u, a = self.linear("value", n), torch.sigmoid(self.linear("gate", n))
        rows, last = [None] * x.shape[0], []
        for b in range(len(offsets) - 1):
            h = state[b]
            for l in range(offsets[b], offsets[b + 1]):
                h = a[l] * h + (1 - a[l]) * u[l]
                rows[l] = h
            last.append(h)
        x = x + self.linear("out", torch.stack(rows))
        z = self.linear("fc1", self.norm("norm2", x))
        z = 0.5 * z * (1 + torch.tanh(K0 * (z + K1 * z ** 3)))
        return x + self.linear("fc2", z), torch.stack(last)


def off_by(got, ref):
    got, ref = got.detach().cpu().double(), ref.detach()
    return float((got - ref).abs().max() / ref.abs().max())


def make(C, H, T, group, dtype):
    block = EqScanBlock(C, H, T, dtype=dtype, device="cuda", group=group)
    with torch.no_grad():
        for p in (block.norm1, block.norm2):
            p.weight.add_(0.1 * torch.randn_like(p.weight))
            p.bias.add_(0.1 * torch.randn_like(p.bias))
    return block


@pytest.mark.gpu
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("C,H,T,group,dtype", [
    (12, 24, 4, "cyclic", torch.float16), (12, 24, 4, "cyclic", torch.float32),
    (6, 10, 8, "p4m", torch.float16), (8, 12, 6, "cyclic", torch.float16),
    (5, 7, 3, "cyclic", torch.float32)])
def test_block_and_its_gradients(gpu, C, H, T, group, dtype, packed):
    block = make(C, H, T, group, dtype)
    B, rows = 3, 120
    off = [0, 17, 17, rows] if packed else [0, 40, 80, rows]
    x = torch.randn(rows, C * T, device="cuda").to(dtype)
    s0 = torch.randn(B, C * T, device="cuda")
    dy, ds = torch.randn(rows, C * T).to(dtype), torch.randn(B, C * T)
    ref = Reference(block, group, T)
    xr, sr = x.cpu().double().requires_grad_(True), s0.cpu().double().requires_grad_(True)
    yr, lr = ref(xr, sr, off)
    ((yr * dy.double()).sum() + (lr * ds.double()).sum()).backward()
    xg, sg = x.clone().requires_grad_(True), s0.clone().requires_grad_(True)
    if packed:
        y, last = block(xg, sg, torch.tensor(off, dtype=torch.int32, device="cuda"))
    else:
        y, last = block(xg.view(B, -1, C * T), sg)
        y = y.reshape(rows, C * T)
    torch.autograd.backward([y, last], [dy.cuda(), ds.cuda()])
    t = LAYER[dtype]
    assert off_by(y, yr) <= 10 * t and off_by(last, lr) <= 10 * t
    assert off_by(xg.grad, xr.grad) <= 20 * t and off_by(sg.grad, sr.grad) <= 20 * t
    for k, v in block.named_parameters():
        assert off_by(v.grad, ref.p[k].grad) <= 20 * t, k


@pytest.mark.gpu
def test_gradient_against_differences(gpu):
    block = make(6, 8, 4, "cyclic", torch.float32)
    x, v = (torch.randn(2, 50, 24, device="cuda") for _ in range(2))
    dy = torch.randn(2, 50, 24, device="cuda")
    x.requires_grad_(True)
    (block(x)[0] * dy).sum().backward()
    slope = float((x.grad * v).sum())
    step = 1e-2
    with torch.no_grad():
        f = [float((block(x + s * v)[0].double() * dy).sum()) for s in (step, -step)]
    # differences are off by step^2 / 6 times a third derivative, about the size
    # of the values here, and by the outputs' fp32 error over the step
    size = float(dy.norm() * v.norm())
    assert abs((f[0] - f[1]) / (2 * step) - slope) <= (step ** 2 + 1e-5 / step) * size


@pytest.mark.gpu
@pytest.mark.parametrize("group,T", [("cyclic", 4), ("p4m", 8)])
def test_block_commutes_with_the_group(gpu, group, T):
    C = 8
    block = make(C, 16, T, group, torch.float16)
    x = torch.randn(2, 60, C, T, device="cuda").half()
    if group == "p4m":  # left translation by r: h -> r^-1 h on both halves
        turn = lambda v: torch.cat([v[..., :4].roll(1, -1), v[..., 4:].roll(1, -1)], -1)
    else:
        turn = lambda v: v.roll(1, -1)
    flat = lambda v: v.reshape(2, 60, C * T)
    with torch.no_grad():
        y, s = block(flat(x))
        yt, st = block(flat(turn(x).contiguous()))
    y, s = turn(y.view(2, 60, C, T)).double(), turn(s.view(2, C, T)).double()
    assert float((yt.view_as(y).double() - y).abs().max() / y.abs().max()) <= 10 * 5e-3
    assert float((st.view_as(s).double() - s).abs().max() / s.abs().max()) <= 10 * 5e-3


@pytest.mark.gpu
def test_block_token_by_token(gpu):
    block = make(12, 24, 4, "cyclic", torch.float16)
    x = torch.randn(5, 30, 48, device="cuda").half()
    with torch.no_grad():
        y, last = block(x)
        _, state = block(x[:, :20])
        state = state.clone()
        out = torch.stack([block.step(x[:, l], state) for l in range(20, 30)], 1)
    # the same kernels on other tile places: a few roundings apart
    assert float((out.float() - y[:, 20:].float()).abs().max() / y.abs().max()) <= 5e-3
    assert float((state - last).abs().max()) <= 5e-3


@pytest.mark.gpu
def test_some_gradients_only(gpu):
    block = make(6, 8, 4, "cyclic", torch.float16)
    x = torch.randn(2, 20, 24, device="cuda").half()
    for p in block.parameters():
        p.requires_grad_(False)
    x.requires_grad_(True)
    y, s = block(x)
    s.sum().backward()               # through the state alone
    assert x.grad.isfinite().all() and x.grad[:, -1].any()
    x2 = x.detach()
    block.fc1.weight.requires_grad_(True)
    block(x2)[0].sum().backward()
    assert block.fc1.weight.grad.any() and block.fc2.weight.grad is None


@pytest.mark.gpu
def test_rows_of_no_sequence_get_no_gradient(gpu):
    scan = EqScan(6, 4)
    u = torch.randn(30, 24, device="cuda").half().requires_grad_(True)
    g = torch.randn(30, 6, device="cuda").half().requires_grad_(True)
    off = torch.tensor([2, 11, 25], dtype=torch.int32, device="cuda")
    h, s = scan(u, g, offsets=off)
    h.sum().backward()
    for t in (h, u.grad, g.grad):
        assert not t[:2].any() and not t[25:].any() and t[2:25].any()


@pytest.mark.gpu
def test_two_blocks_on_two_streams(gpu):
    blocks = [make(12, 24, 4, "cyclic", torch.float16) for _ in range(2)]
    x = torch.randn(4, 500, 48, device="cuda").half()
    with torch.no_grad():
        want = [b(x)[0] for b in blocks]
        streams = [torch.cuda.Stream() for _ in blocks]
        got = [None, None]
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
        for _ in range(5):
            for i, (b, s) in enumerate(zip(blocks, streams)):
                with torch.cuda.stream(s):
                    got[i] = b(x)[0]
        torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
