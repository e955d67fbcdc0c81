"""The layer norm's parity cases with a comparison that a NaN fails."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import group_dft_structured_b200 as F
import test_norm_gpu as base

SHAPES = base.SHAPES + [(40, 4, 6), (333, 12, 10), (21, 340, 6), (9, 96, 14), (6, 2731, 6),
                        (11, 1540, 2), (40000, 6, 4)]


def within(got, ref, tol, what):
    got = got.detach().cpu().numpy().astype(np.float64)
    assert got.shape == ref.shape, what
    good = np.abs(got - ref) <= tol
    assert good.all(), f"{what}: {(~good).sum()} of {good.size} off"


def test_a_nan_is_off():
    ref, tol = np.zeros(3), np.ones(3)
    within(torch.tensor([0.0, 0.5, -1.0]), ref, tol, "values")
    with pytest.raises(AssertionError):
        within(torch.tensor([0.0, float("nan"), 0.0]), ref, tol, "values")


@pytest.mark.gpu
@pytest.mark.parametrize("affine", [True, False])
@pytest.mark.parametrize("dt", [np.float16, np.float32])
@pytest.mark.parametrize("N,C,T", SHAPES)
def test_parity(monkeypatch, N, C, T, dt, affine):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from group_dft_structured_b200 import build
    build.build()
    F.load()
    monkeypatch.setattr(base, "within", within)
    x, dy, gamma, beta = base.inputs(N, C, T, dt, seed=11)
    if not affine:
        gamma = beta = None
    base.check(x, dy, gamma, beta, *base.run(x, dy, gamma, beta))
