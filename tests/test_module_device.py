"""EqLinear on a device that is not the current one: a stand-in for a second GPU's tensors
shows, without any GPU, under which device the library would be called."""

import contextlib

import pytest

torch = pytest.importorskip("torch")

from group_dft_structured_b200 import module as M
from group_dft_structured_b200.module import EqLinear


class Second(torch.Tensor):
    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda", 1))


@pytest.mark.parametrize("kind", [dict(), dict(activation="gelu")])
@pytest.mark.parametrize("residual", [False, True])
def test_calls_run_under_the_inputs_device(monkeypatch, kind, residual):
    current, seen = [0], []

    @contextlib.contextmanager
    def device(d):
        current.append(d.index)
        yield
        current.pop()

    def apply(x, W, b, *rest):
        seen.append(current[-1])
        return torch.zeros(x.shape[0], W.shape[0], W.shape[2])

    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(EqLinear, "fourier_weight", lambda self: seen.append(current[-1]))
    for f in (M.EqLinearFunction, M.EqLinearActFunction):
        monkeypatch.setattr(f, "apply", staticmethod(apply))
    m = EqLinear(3, 5, **kind)
    m._parameters["weight"] = m.weight.detach().as_subclass(Second)
    x = torch.zeros(7, 12, dtype=torch.float16).as_subclass(Second)
    res = torch.zeros(7, 20, dtype=torch.float16) if residual else None
    assert m(x, res).shape == (7, 20)
    assert seen == [1, 1] and current == [0]


def test_a_weight_elsewhere_is_refused():
    m = EqLinear(3, 5)
    with pytest.raises(ValueError):
        m(torch.zeros(7, 12, dtype=torch.float16).as_subclass(Second))
