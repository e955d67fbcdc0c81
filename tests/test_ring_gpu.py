"""Layers whose kernels have an odd number of input stages (wide ones, and split TF32):
the same bits at every call, with caches cold and with the loads' order as it comes."""

import pytest

torch = pytest.importorskip("torch")

import group_dft_structured_b200 as F
from group_dft_structured_b200 import layer as L

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


@pytest.mark.parametrize("mode,N,C,D", [
    ("fp32", 3000, 192, 192), ("fp32", 20000, 96, 96), ("fp32", 2000, 24, 96),
    ("fp32", 3000, 512, 128), ("fp32", 900, 70, 130), ("fp16", 3000, 192, 192),
    ("fp16", 20000, 384, 96), ("fp16", 3000, 96, 384)])
def test_the_same_at_every_call(mode, N, C, D):
    code = F.DTYPES[mode]
    dt = L.torch_dtype(code)
    torch.manual_seed(C + D)
    x, dy = torch.randn(N, C, 4, device="cuda").to(dt), torch.randn(N, D, 4, device="cuda").to(dt)
    W = (torch.randn(D, C, 4, device="cuda") / (4 * C) ** 0.5).to(dt)
    What = L.ct_weight_fft(W, code)
    gelu = F.FEQL_ACT_GELU

    def run():
        return (L.ct_forward(x, What, None, D, code), L.ct_backward_dx(dy, What, C, code),
                *L.ct_forward_act(x, What, None, D, code, gelu, res=dy, save_z=True),
                L.ct_forward_act(x, What, None, D, code, F.FEQL_ACT_RELU, res=dy)[0])

    # the layer itself, in float64 (its fp16 and fp32 bounds)
    t = torch.arange(4, device="cuda")
    A = W[:, :, (t[:, None] - t[None, :]) % 4].permute(0, 2, 1, 3).reshape(4 * D, 4 * C).double()
    ref = x.double().reshape(N, -1) @ A.t()
    want = run()
    off = (want[0].double().reshape(N, -1) - ref).abs().max() / ref.abs().max()
    assert off <= (5e-3 if dt == torch.float16 else 1e-5)
    big = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
    for i in range(40):
        big.fill_(i)  # the caches hold nothing of the layer
        for k, (a, b) in enumerate(zip(run(), want)):
            assert torch.equal(a, b), (i, k)
