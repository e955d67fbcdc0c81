"""The layer's backward pass with activation or residual on no tokens."""

import pytest

torch = pytest.importorskip("torch")

import group_dft_structured_b200 as F
from group_dft_structured_b200 import build as B
from group_dft_structured_b200 import layer as L
from group_dft_structured_b200.module import EqLinear

P = 1 << 20  # aligned fake address; never dereferenced
GROUPS = [("cyclic", 4), ("cyclic", 8), ("cyclic", 6), ("cyclic", 3), ("p4m", 8)]


def test_input_gradient_of_no_tokens_needs_no_pointers():
    B.build()
    lib = F.load()
    for act in (F.FEQL_ACT_NONE, F.FEQL_ACT_RELU, F.FEQL_ACT_GELU):
        for dtype in (F.FEQL_FP16, F.FEQL_FP32):
            args = [None] * 7 + [P, 1 << 20, 0, 4, 4, act, dtype, None]
            assert lib.feql_backward_act(*args) == F.FEQL_OK
            assert lib.feql_ct_backward_act(3, *args) == F.FEQL_OK
    assert lib.feql_p4m_backward_act(*[None] * 8, 0, 0, 4, 4, 1, F.FEQL_FP16, None) == F.FEQL_OK
    # db without dW stays refused, and so do tokens without an output
    bad = [None] * 6 + [P, P, 1 << 20, 0, 4, 4, 1, F.FEQL_FP16, None]
    assert lib.feql_backward_act(*bad) == F.FEQL_ERR_INVALID_ARG
    bad = [P, P, P, P, None, None, None, P, 1 << 40, 8, 4, 4, 1, F.FEQL_FP16, None]
    assert lib.feql_backward_act(*bad) == F.FEQL_ERR_INVALID_ARG


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["none", "relu", "gelu"])
@pytest.mark.parametrize("group,T", GROUPS)
def test_each_gradient_alone(group, T, act):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    B.build()
    run = L.p4m_backward_act if group == "p4m" else L.ct_backward_act
    wfft = L.p4m_weight_fft if group == "p4m" else L.ct_weight_fft
    W = torch.randn(8, 4, T, device="cuda").half()
    x, dy = torch.zeros(0, 4, T, device="cuda").half(), torch.zeros(0, 8, T, device="cuda").half()
    slope = None if act == "none" else dy.clone()
    for with_dx in (False, True):
        for with_dw, with_db in ((False, False), (True, False), (False, True), (True, True)):
            dx, dW, db = run(x, dy, slope, wfft(W, F.FEQL_FP16), F.FEQL_FP16, F.ACTIVATIONS[act],
                             with_dx=with_dx, with_dw=with_dw, with_db=with_db)
            assert (dx is not None) == with_dx and (not with_dx or dx.shape == x.shape)
            assert (dW is not None) == with_dw and (not with_dw or not dW.any())
            assert (db is not None) == with_db and (not with_db or not db.any())


@pytest.mark.gpu
@pytest.mark.parametrize("kw", [dict(activation="gelu"), dict()])
@pytest.mark.parametrize("group,T", GROUPS)
def test_frozen_layer_on_no_tokens(group, T, kw):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    B.build()
    m = EqLinear(4, 8, T, group=group, device="cuda", **kw).requires_grad_(False)
    x = torch.zeros(0, 4 * T, device="cuda").half().requires_grad_()
    res = torch.zeros(0, 8 * T, device="cuda").half().requires_grad_()
    m(x, res).sum().backward()
    assert x.grad.shape == x.shape and res.grad.shape == res.shape
