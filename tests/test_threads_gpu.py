"""Calls from several host threads at once, of other sizes of the same kernels: each is as
if it were alone."""

import threading

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


def work(group, T, C, D, N):
    """One training step's calls of a layer with GELU, and their results alone."""
    x = torch.randn(N, C, T, device="cuda").half()
    dy, W = torch.randn(N, D, T, device="cuda").half(), torch.randn(D, C, T, device="cuda").half()
    W *= (C * T) ** -0.5
    wfft, forward, backward = ((L.p4m_weight_fft, L.p4m_forward_act, L.p4m_backward_act)
                               if group == "p4m" else
                               (L.ct_weight_fft, L.ct_forward_act, L.ct_backward_act))
    What = wfft(W, F.FEQL_FP16)

    def run():
        y, s = forward(x, What, None, D, F.FEQL_FP16, F.FEQL_ACT_GELU, res=dy, save_z=True)
        return y, s, *backward(x, dy, s, What, F.FEQL_FP16, F.FEQL_ACT_GELU)

    return run, run()


def mlp(C, H, N):
    x = torch.randn(N, C, 4, device="cuda").half()
    W1, W2 = (0.1 * torch.randn(*s, 4, device="cuda").half() for s in ((H, C), (C, H)))
    What = L.mlp_weight_fft(W1, W2, F.FEQL_FP16)
    run = lambda: (L.mlp_forward(x, What, None, None, H, C, F.FEQL_FP16),)
    return run, run()


JOBS = [lambda: [work("cyclic", 4, 24, 96, 300), work("cyclic", 4, 192, 192, 300)],
        lambda: [work("cyclic", 4, 16, 16, 200), work("cyclic", 4, 64, 128, 200)],
        lambda: [work("cyclic", 8, 8, 16, 200), work("cyclic", 8, 96, 64, 200)],
        lambda: [work("p4m", 8, 8, 16, 200), work("p4m", 8, 64, 96, 200)],
        lambda: [mlp(24, 96, 300), mlp(96, 384, 300)]]


@pytest.mark.parametrize("make", JOBS)
def test_two_threads(make):
    jobs, failed = make(), []
    torch.cuda.synchronize()

    def loop(run, want):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(300):
                    out = run()
                assert all(torch.equal(a, b) for a, b in zip(out, want))
        except BaseException as e:  # a thread's exception would be lost
            failed.append(repr(e))

    threads = [threading.Thread(target=loop, args=job) for job in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed


def raw(name, C, D, *args):
    """A C call's bound function and arguments, its tensors kept beside them."""
    lib, N = F.load(), 130
    x, dy = (torch.randn(N, k, 4, device="cuda").half() for k in (C, D))
    W = (0.1 * torch.randn(D, C, 4, device="cuda")).half()
    What, stream = L.ct_weight_fft(W, F.FEQL_FP16), torch.cuda.Stream()
    a = lambda t: t.data_ptr()
    if name == "forward":
        y, s = torch.empty_like(dy), torch.empty_like(dy)
        call = (lib.feql_forward_act, a(x), a(What), None, None, a(y), a(s), N, C, D,
                F.FEQL_ACT_GELU, F.FEQL_FP16, stream.cuda_stream)
        return call, (x, What, y, s, stream)
    ws = L.dw_workspace(N, C, D, F.FEQL_FP16, "cuda")
    dx, dW = torch.empty_like(x), torch.empty_like(W)
    call = (lib.feql_backward, a(x), a(dy), a(What), a(dx), a(dW), None, a(ws), ws.numel(), N, C,
            D, F.FEQL_FP16, stream.cuda_stream)
    return call, (x, dy, What, ws, dx, dW, stream)


@pytest.mark.parametrize("name,sizes", [
    ("forward", ((16, 16), (192, 96))), ("backward", ((16, 16), (64, 128))),
    ("backward", ((160, 32), (192, 256)))])
def test_c_calls_from_two_threads(name, sizes):
    """The calls alone, so close to one another that their host code overlaps."""
    calls, refused = [raw(name, *s) for s in sizes for _ in range(2)], []
    torch.cuda.synchronize()

    def loop(f, *args):
        bad = [st for st in (f(*args) for _ in range(4000)) if st != F.FEQL_OK]
        if bad:
            refused.append((len(bad), bad[0]))

    threads = [threading.Thread(target=loop, args=c) for c, _ in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not refused, refused
