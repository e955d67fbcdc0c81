"""Host-side checks of the operators around the layer, without a GPU: arguments
are refused before any CUDA call, and CPU tensors before any library call."""

import pytest

torch = pytest.importorskip("torch")

import group_dft_structured_b200 as F
from group_dft_structured_b200 import build as B
from group_dft_structured_b200 import layer as L

FP16, FP32 = F.FEQL_FP16, F.FEQL_FP32
INV, UNS = F.FEQL_ERR_INVALID_ARG, F.FEQL_ERR_UNSUPPORTED
P = 1 << 20  # aligned fake address; never dereferenced: every call below is refused first


@pytest.fixture(scope="module")
def lib():
    B.build()
    return F.load()


def test_norm_refusals(lib):
    f = lib.feql_norm_forward
    assert f(None, None, None, P, None, 8, 4, 4, 1e-5, FP16, None) == INV
    assert f(P, None, None, None, None, 8, 4, 4, 1e-5, FP16, None) == INV
    assert f(P, None, None, P, None, -1, 4, 4, 1e-5, FP16, None) == INV
    assert f(P, None, None, P, None, 8, 0, 4, 1e-5, FP16, None) == INV
    assert f(P, None, None, P, None, 8, 4, 0, 1e-5, FP16, None) == UNS
    assert f(P, None, None, P, None, 8, 4, 17, 1e-5, FP16, None) == UNS
    assert f(P, None, None, P, None, 8, 4, 4, 1e-5, 17, None) == INV
    for eps in (0.0, -1e-5, float("nan"), float("inf")):
        assert f(P, None, None, P, None, 8, 4, 4, eps, FP32, None) == INV
    assert f(P + 2, None, None, P, None, 8, 4, 4, 1e-5, FP16, None) == INV
    assert f(P, P + 8, None, P, None, 8, 4, 4, 1e-5, FP16, None) == INV
    assert f(P, None, None, P, P + 4, 8, 4, 4, 1e-5, FP16, None) == INV
    assert f(None, None, None, None, None, 0, 4, 4, 1e-5, FP16, None) == F.FEQL_OK
    b = lib.feql_norm_backward
    assert b(P, None, P, None, P, P, P, P, 1 << 30, 8, 4, 4, FP16, None) == INV
    assert b(P, P, None, None, P, P, P, P, 1 << 30, 8, 4, 4, FP16, None) == INV
    assert b(P, P, P, None, P, P, P, None, 1 << 30, 8, 4, 4, FP16, None) == INV
    assert b(P, P, P, None, P, P, P, P, 1 << 30, 1 << 31, 4, 4, FP16, None) == INV


def test_scan_refusals(lib):
    f = lib.feql_scan_forward
    assert f(None, P, None, None, P, None, P, 1 << 30, 2, 8, 4, 4, 0, FP16, None) == INV
    assert f(P, P, None, None, None, None, P, 1 << 30, 2, 8, 4, 4, 0, FP16, None) == INV
    assert f(P, P, None, None, P, None, P, 1 << 30, 3, 8, 4, 4, 0, FP16, None) == INV  # 8 rows, 3 sequences
    assert f(P, P, None, None, P, None, P, 1 << 30, 0, 8, 4, 4, 0, FP16, None) == INV
    assert f(P, P, None, None, P, None, P, 1 << 30, -1, 8, 4, 4, 0, FP16, None) == INV
    assert f(P, P, None, None, P, None, P, 1 << 30, 2, 8, 4, 17, 0, FP16, None) == UNS
    assert f(P, P, P + 4, None, P, None, P, 1 << 30, 2, 8, 4, 4, 0, FP16, None) == INV
    assert f(P, P, None, P + 4, P, None, P, 1 << 30, 2, 8, 4, 4, 0, FP16, None) == INV
    assert f(P, P, None, None, P, None, P, 1 << 30, 2, 8, 4, 4, 0, -1, None) == INV
    assert f(None, None, None, None, None, None, P, 1 << 30, 0, 0, 4, 4, 0, FP16, None) == F.FEQL_OK
    b = lib.feql_scan_backward
    assert b(P, P, P, None, None, None, None, P, P, None, P, 1 << 30, 2, 8, 4, 4, 0, FP16, None) == INV
    assert b(P, P, P, P, None, None, None, P, None, None, P, 1 << 30, 2, 8, 4, 4, 0, FP16, None) == INV
    s = lib.feql_scan_step
    assert s(P, P, None, P, 2, 4, 4, 0, FP16, None) == INV
    assert s(P, P, P, P, 2, 4, 17, 0, FP16, None) == UNS
    assert s(None, None, None, None, 0, 4, 4, 0, FP16, None) == F.FEQL_OK


def test_activation_refusals(lib):
    GELU = F.FEQL_ACT_GELU
    f = lib.feql_forward_act
    assert f(P, P, None, None, P, None, 8, 4, 4, -1, FP16, None) == INV
    assert f(P, P, None, None, P, None, 8, 4, 4, 4, FP16, None) == INV
    assert f(P, P, None, None, P, None, -1, 4, 4, GELU, FP16, None) == INV
    assert f(P, P, None, P + 8, P, None, 8, 4, 4, GELU, FP16, None) == INV
    assert f(P, P, None, None, P, P + 8, 8, 4, 4, GELU, FP16, None) == INV
    assert f(None, P, None, None, P, None, 8, 4, 4, GELU, FP16, None) == INV
    assert f(P, P, None, None, P, None, 8, 3, 4, GELU, FP16, None) == UNS
    assert f(None, None, None, None, None, None, 0, 4, 4, GELU, FP16, None) == F.FEQL_OK
    c = lib.feql_ct_forward_act
    assert c(17, P, P, None, None, P, None, 8, 4, 4, GELU, FP16, None) == UNS
    assert c(8, P, P, None, None, P, None, 8, 4, 4, 9, FP16, None) == INV
    assert c(3, P, None, None, None, P, None, 8, 4, 4, GELU, FP32, None) == INV
    m = lib.feql_p4m_forward_act
    assert m(P, P, None, None, P, None, 8, 4, 4, GELU, FP32, None) == UNS
    b = lib.feql_backward_act
    big = 1 << 40
    assert b(P, P, None, P, P, P, P, P, big, 8, 4, 4, GELU, FP16, None) == INV   # no slopes
    assert b(P, P, P, P, None, None, None, P, big, 8, 4, 4, GELU, FP16, None) == INV
    assert b(P, P, P, P, P, None, P, P, big, 8, 4, 4, GELU, FP16, None) == INV   # db without dW
    assert b(P, P, P, None, P, P, P, P, big, 8, 4, 4, GELU, FP16, None) == INV
    assert b(None, P, P, P, P, P, P, P, big, 8, 4, 4, GELU, FP16, None) == INV
    assert b(P, P, P, P, P, P, P, None, big, 8, 4, 4, GELU, FP16, None) == INV
    assert b(P, P, P + 2, P, P, P, P, P, big, 8, 4, 4, GELU, FP16, None) == INV
    assert b(P, P, P, P, P, P, P, P, big, 8, 4, 5, GELU, FP16, None) == UNS
    assert lib.feql_backward_act_workspace_bytes(8, 4, 4, 7, FP16) == 0
    assert lib.feql_p4m_backward_act_workspace_bytes(8, 4, 4, GELU, FP32) == 0


def test_layer_functions_refuse_cpu_tensors_and_wrong_shapes():
    x = torch.zeros(3, 4, 4, dtype=torch.float16)
    with pytest.raises(ValueError):
        L.norm_forward(x)
    with pytest.raises(TypeError):
        L.norm_forward(x.to(torch.bfloat16))
    with pytest.raises(ValueError):
        L.norm_forward(x[0])
    with pytest.raises(ValueError):
        L.scan_forward(x, x)  # packed rows without offsets
    with pytest.raises(ValueError):
        L.scan_forward(x[None], x[None][..., :2])
    with pytest.raises(ValueError):
        L.scan_step(x, x[..., 0], torch.zeros(3, 4, 4))
