"""Tensors of more than 2^31 values through the operators around the layer: the last
rows are what the same rows give by themselves."""

import pytest

torch = pytest.importorskip("torch")

import group_dft_structured_b200 as F
from group_dft_structured_b200 import layer as L

pytestmark = pytest.mark.gpu

C, T = 24, 4


@pytest.fixture(scope="module", autouse=True)
def ready():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB of device memory")
    from group_dft_structured_b200 import build
    build.build()
    F.load()
    yield
    torch.cuda.empty_cache()


def filled(*shape):
    """Varied fp16 values, quickly: a random block repeated."""
    t = torch.empty(shape, dtype=torch.float16, device="cuda")
    block = torch.randn(1 << 22, device="cuda").half()
    flat = t.view(-1)
    for i in range(0, flat.numel(), block.numel()):
        n = min(block.numel(), flat.numel() - i)
        flat[i:i + n] = block[:n]
    return t


def test_norm():
    N = (1 << 31) // (C * T) + 12345
    x, dy = filled(N, C, T), filled(N, C, T)
    y, stats = L.norm_forward(x)
    dx, _, _ = L.norm_backward(dy, x, stats)
    y1, s1 = L.norm_forward(x[-1000:])
    dx1, _, _ = L.norm_backward(dy[-1000:], x[-1000:], s1)
    assert torch.equal(y[-1000:], y1) and torch.equal(dx[-1000:], dx1)


def test_layer_with_activation():
    N, D = (1 << 31) // (4 * C * T) + 777, 4 * C
    x, W = filled(N, C, T), (torch.randn(D, C, T, device="cuda") * 0.1).half()
    res, mode, gelu = filled(N, D, T), F.FEQL_FP16, F.FEQL_ACT_GELU
    What = L.ct_weight_fft(W, mode)
    y, slope = L.ct_forward_act(x, What, None, D, mode, gelu, res=res, save_z=True)
    y1, slope1 = L.ct_forward_act(x[-500:], What, None, D, mode, gelu, res=res[-500:], save_z=True)
    assert torch.equal(y[-500:], y1) and torch.equal(slope[-500:], slope1)
    dx, _, _ = L.ct_backward_act(x, res, slope, What, mode, gelu)
    dx1, _, _ = L.ct_backward_act(x[-500:], res[-500:], slope1, What, mode, gelu)
    assert torch.equal(dx[-500:], dx1)


@pytest.mark.parametrize("packed", [False, True])
def test_scan(packed):
    B, n = 23, 1000000
    N = B * n
    assert N * C * T > 1 << 31
    shape = (N,) if packed else (B, n)
    u, g, dh = filled(*shape, C, T), filled(*shape, C, T), filled(*shape, C, T)
    off = torch.arange(0, N + 1, n, dtype=torch.int32, device="cuda") if packed else None
    h, hN, saved = L.scan_forward(u, g, None, off)
    du, dg, _ = L.scan_backward(dh, u, g, saved, None, off)
    last = lambda t: (t[-2000:] if packed else t[-1:, -2000:]).reshape(1, 2000, C, T)
    start = (h[-2001] if packed else h[-1, -2001])[None].float()
    h1, hN1, saved1 = L.scan_forward(last(u), last(g), start)
    du1, dg1, _ = L.scan_backward(last(dh), last(u), last(g), saved1)
    # the state before these rows was rounded to fp16 (values below 8: 2^-9 at most), and the
    # sums run in other tiles; gates of N(0, 1) forget within some tens of rows
    for a, b, lead in ((h, h1, 200), (du, du1, 0), (dg, dg1, 200)):
        a, b = last(a)[:, lead:].float(), b[:, lead:].float()
        assert (a - b).abs().max() <= 2.0 ** -9 * max(1.0, float(b.abs().max()))
    assert (hN[-1:] - hN1).abs().max() <= 1e-4
