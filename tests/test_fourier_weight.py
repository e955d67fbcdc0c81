"""EqLinear's Fourier weight buffer follows the weight: at every call, and where a frozen
layer keeps it, across inference mode, captured graphs and streams.  The first tests put a counting stand-in in the place of the
library's transform and need no GPU."""

import pytest

torch = pytest.importorskip("torch")

import group_dft_structured_b200 as F
from group_dft_structured_b200 import module as M
from group_dft_structured_b200.module import EqLinear


# ------------------------------------------------------------------ CPU ---

class Fake:
    """The weight transform and what torch says of streams."""

    def __init__(self, patch):
        self.calls, self.stream, self.capturing = 0, 1, False
        patch.setattr(M._L, "ct_weight_fft", self.transform)
        patch.setattr(torch.cuda, "is_current_stream_capturing", lambda: self.capturing)
        patch.setattr(torch.cuda, "current_stream",
                      lambda device=None: type("S", (), {"cuda_stream": self.stream}))

    def transform(self, W, mode, stream=None):
        self.calls += 1
        return 2 * W


@pytest.fixture
def fake(monkeypatch):
    return Fake(monkeypatch)


def frozen(C, D):
    return EqLinear(C, D).requires_grad_(False).freeze()


def test_at_every_call(fake):
    """Whatever changes the weight, seen or not by its version."""
    m = EqLinear(3, 5)
    for k in range(1, 4):
        assert torch.equal(m.fourier_weight(), 2 * m.weight) and fake.calls == 2 * k - 1
        m.weight.data.mul_(2)
        with torch.no_grad():
            assert torch.equal(m.fourier_weight(), 2 * m.weight) and fake.calls == 2 * k


def test_frozen_until_it_trains(fake):
    m = EqLinear(3, 5).freeze()
    with torch.no_grad():
        first = m.fourier_weight()
        assert m.fourier_weight() is first and fake.calls == 1
    m.fourier_weight()  # the weight's gradient is recorded: not kept
    assert fake.calls == 2
    with torch.no_grad():
        assert m.eval().fourier_weight() is first
        for end in (lambda: m.train(), lambda: m.freeze(False), lambda: torch.nn.Sequential(m).train()):
            m.freeze()
            kept = m.fourier_weight()
            assert m.fourier_weight() is kept
            end()
            assert m.fourier_weight() is not kept and m._whats == {}


def test_blocks_freeze_their_layers(fake):
    b = M.EqScanBlock(3, 5).requires_grad_(False)
    assert b.freeze() is b
    layers = [b.value, b.gate, b.out, b.fc1, b.fc2]
    assert all(m.fourier_weight() is m.fourier_weight() for m in layers)
    b.train()
    assert not any(m._frozen for m in layers)


def test_once_per_weight(fake):
    m = frozen(3, 5)
    first = m.fourier_weight()
    assert m.fourier_weight() is first and fake.calls == 1
    with torch.no_grad():
        m.weight.mul_(2)
    assert torch.equal(m.fourier_weight(), 2 * m.weight) and fake.calls == 2


def test_made_in_inference_mode_and_used_outside(fake):
    m = frozen(3, 5)
    with torch.inference_mode():
        What = m.fourier_weight()
    assert not What.is_inference()
    assert m.fourier_weight() is What and fake.calls == 1


def test_weights_made_in_inference_mode(fake):
    with torch.inference_mode():
        m = EqLinear(3, 5)
        m.fourier_weight()
        m.weight.mul_(2)
        assert torch.equal(m.fourier_weight(), 2 * m.weight)


def test_a_captured_transform_is_in_the_graph_alone(fake):
    m = frozen(3, 5)
    fake.capturing = True
    captured = m.fourier_weight()
    fake.capturing = False
    eager = m.fourier_weight()
    assert eager is not captured and fake.calls == 2
    fake.capturing = True  # with the eager one at hand
    assert m.fourier_weight() is not eager and fake.calls == 3
    fake.capturing = False
    assert m.fourier_weight() is eager and fake.calls == 3


def test_streams_do_not_share_a_buffer(fake):
    m = frozen(3, 5)
    first = m.fourier_weight()
    fake.stream = 2
    second = m.fourier_weight()
    assert second is not first and fake.calls == 2
    fake.stream = 1
    assert m.fourier_weight() is first and fake.calls == 2
    with torch.no_grad():
        m.weight.mul_(2)
    for stream in (2, 1):
        fake.stream = stream
        assert torch.equal(m.fourier_weight(), 2 * m.weight)
    assert fake.calls == 4 and len(m._whats) == 2


def test_copies_and_files_hold_the_weight_alone(fake):
    import copy
    import io
    m = frozen(3, 5)
    m.fourier_weight()
    size = lambda m: (lambda f: (torch.save(m, f), f.tell())[1])(io.BytesIO())
    fresh = frozen(3, 5)
    assert abs(size(m) - size(fresh)) < 64  # no buffer in it
    f = io.BytesIO()
    torch.save(m, f)
    f.seek(0)
    for other in (copy.deepcopy(m), torch.load(f, weights_only=False)):
        assert other._whats == {} and torch.equal(other.weight, m.weight)
        with torch.no_grad():
            other.weight.mul_(3)
        assert torch.equal(other.fourier_weight(), 2 * other.weight)
    assert len(m._whats) == 1


def test_another_weight_at_the_same_address(fake):
    m = frozen(40, 50)
    for k in range(1, 30):
        del m.weight
        m.weight = torch.nn.Parameter(torch.full((50, 40, 4), float(k), dtype=torch.float16),
                                      requires_grad=False)
        assert torch.equal(m.fourier_weight(), 2 * m.weight), k
    for k in range(1, 30):  # a weight of the moment, as torch.func.functional_call sets it
        m._parameters["weight"] = None
        m._parameters["weight"] = torch.full((50, 40, 4), float(k), dtype=torch.float16)
        assert torch.equal(m.fourier_weight(), 2 * m.weight), k


def test_threads_on_their_own_streams(fake, monkeypatch):
    """Many threads, each on a stream of its own, while the weight keeps changing."""
    import sys
    import threading
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: type(
        "S", (), {"cuda_stream": threading.get_ident()}))
    m, failed = frozen(3, 5), []

    def loop():
        try:
            for _ in range(300):
                with torch.no_grad():
                    m.weight.add_(1)
                m.fourier_weight()
        except BaseException as e:
            failed.append(repr(e))

    interval = sys.getswitchinterval()
    sys.setswitchinterval(1e-6)
    try:
        threads = [threading.Thread(target=loop) for _ in range(8)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    finally:
        sys.setswitchinterval(interval)
    assert not failed, failed
    assert torch.equal(m.fourier_weight(), 2 * m.weight)


# ------------------------------------------------------------------ GPU ---

@pytest.fixture
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from group_dft_structured_b200 import build
    build.build()
    F.load()
    torch.manual_seed(7)
    yield
    assert F.feql_device_status() == F.FEQL_OK


KINDS = [dict(), dict(activation="gelu"), dict(group="p4m", group_order=8, activation="relu")]


def layer(kind, **kw):
    m = EqLinear(16, 24, device="cuda", **kind, **kw)
    return m, torch.randn(70, 16 * m.group_order, device="cuda").half()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
def test_inference_then_training(gpu, kind):
    m, x = layer(kind)
    m.freeze()
    with torch.inference_mode():
        want = m(x).clone()
    y = m(x)
    y.sum().backward()
    assert torch.equal(y, want) and m.weight.grad.isfinite().all()


@pytest.mark.gpu
@pytest.mark.parametrize("warm", [False, True])
@pytest.mark.parametrize("kind", KINDS)
def test_captured_calls_follow_the_weight(gpu, kind, warm):
    m, x = layer(kind)
    m.freeze(warm)
    with torch.no_grad():
        if warm:
            m(x)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            y = m(x)
        eager = m(x)  # before any replay
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, eager)
        for _ in range(2):
            m.weight.mul_(-1.5)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, m(x)) and not torch.equal(y, eager)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
def test_two_streams_at_once(gpu, kind):
    """The first stream is far from done with its transform when the second calls."""
    m, x = layer(kind)
    m2, _ = layer(kind)
    m.freeze()
    with torch.no_grad():
        m2.weight.copy_(m.weight)
        if m.bias is not None:
            m2.bias.copy_(m.bias)
        want = m2(x)
        a, b = torch.cuda.Stream(), torch.cuda.Stream()
        for step in range(3):
            for s in (a, b):
                s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(a):
                torch.cuda._sleep(20000000)  # some 10 ms
                ya = m(x)
            with torch.cuda.stream(b):
                yb = m(x)
            torch.cuda.synchronize()
            assert torch.equal(ya, want) and torch.equal(yb, want), step
            m.weight.neg_()
            m2.weight.neg_()
            want = m2(x)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
def test_weights_of_the_moment(gpu, kind):
    m, x = layer(kind)
    for k in range(6):  # each freed before the next is made: the same address
        W = torch.randn_like(m.weight) * 0.1
        y = torch.func.functional_call(m, {"weight": W}, (x,))
        with torch.no_grad():
            m.weight.copy_(W)
            del W
            assert torch.equal(y, m(x)), k


@pytest.mark.gpu
@pytest.mark.parametrize("name,how", [("SGD", "fused"), ("SGD", "foreach"), ("AdamW", "fused"),
                                      ("AdamW", "foreach"), ("AdamW", "capturable")])
@pytest.mark.parametrize("kind", KINDS)
def test_optimizers_that_leave_no_version(gpu, kind, name, how):
    """Training goes on with the weights that a step has made, and so does what comes after."""
    m, x = layer(kind)
    # (fp16 states: an eps of 1e-8 would be 0 there and the step 0 / 0)
    eps = dict(eps=1e-3) if name == "AdamW" else {}
    opt = getattr(torch.optim, name)(m.parameters(), lr=1e-2, **{how: True}, **eps)
    for _ in range(3):
        with torch.no_grad():
            before = m(x)
        opt.zero_grad()
        m(x).float().square().mean().backward()
        opt.step()
        twin, _ = layer(kind)
        with torch.no_grad():
            for p, q in zip(twin.parameters(), m.parameters()):
                p.copy_(q)
            want = twin(x)
            assert torch.equal(m(x), want) and not torch.equal(want, before)
        assert torch.equal(m(x), want)


@pytest.mark.gpu
def test_steps_replayed_in_a_graph(gpu):
    """A captured training step moves the weights without a trace on the host."""
    m, x = layer(KINDS[1])
    opt = torch.optim.SGD(m.parameters(), lr=1e-2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def step():
        opt.zero_grad(set_to_none=True)
        m(x).float().square().mean().backward()
        opt.step()

    with torch.cuda.stream(side):
        for _ in range(2):
            step()
    torch.cuda.current_stream().wait_stream(side)
    opt.zero_grad(set_to_none=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        with torch.no_grad():
            before = m(x)
        graph.replay()
        torch.cuda.synchronize()
        twin, _ = layer(KINDS[1])
        with torch.no_grad():
            for p, q in zip(twin.parameters(), m.parameters()):
                p.copy_(q)
            assert torch.equal(m(x), twin(x)) and not torch.equal(m(x), before)
