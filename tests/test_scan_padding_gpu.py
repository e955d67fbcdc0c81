"""Packed sequences in buffers with many more rows than they cover: what lies before the
first and behind the last is zero in every output, and the sequences are as without it."""

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


def dirty(*like):
    """The next tensors of these sizes start from other values than zero."""
    for t in [torch.full_like(t, 7) for t in like for _ in range(3)]:
        del t


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("N,off", [
    (20000, [0, 700, 701, 1500]), (20000, [18000, 18200, 20000]), (20000, [9000, 9000, 9100]),
    (20000, [20000, 20000]), (20000, [0, 0]), (60000, [100, 30000]), (500, [499, 500]),
    (5000, list(range(1000, 1800, 2))), (70, [3, 9, 40])])
@pytest.mark.parametrize("C,T", [(24, 4), (5, 6), (3, 1)])
def test_rows_of_no_sequence(C, T, N, off, shared, dtype):
    torch.manual_seed(N + C)
    B = len(off) - 1
    u, dh = (torch.randn(N, C, T, device="cuda").to(dtype) for _ in range(2))
    g = torch.randn(N, C, *(() if shared else (T,)), device="cuda").to(dtype)
    h0, dhN = (torch.randn(B, C, T, device="cuda") for _ in range(2))

    def run(lo, hi):
        o = torch.tensor([v - lo for v in off], dtype=torch.int32, device="cuda")
        dirty(u[lo:hi], g[lo:hi])
        h, hN, saved = L.scan_forward(u[lo:hi], g[lo:hi], h0, o)
        return h, hN, *L.scan_backward(dh[lo:hi], u[lo:hi], g[lo:hi], saved, dhN, o)

    h, hN, du, dg, dh0 = run(0, N)
    for t in (h, du, dg):
        assert not t[:off[0]].any() and not t[off[-1]:].any()
        assert not t[:off[0]].isnan().any() and not t[off[-1]:].isnan().any()
    # the rows alone, cut into other segments: fp32 sums in another order
    alone = run(off[0], off[-1])
    eps = torch.finfo(dtype).eps
    for a, b in zip((h[off[0]:off[-1]], hN, du[off[0]:off[-1]], dg[off[0]:off[-1]], dh0), alone):
        if a.numel():
            assert ((a - b).abs().max() <= (eps + 64 * 2.0 ** -24) * b.abs().max()).item()
