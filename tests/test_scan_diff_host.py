"""Refusals of the recurrence's fp16 training calls, before any CUDA call."""

import pytest

import group_dft_structured_b200 as F
from group_dft_structured_b200 import build as B

FP16, FP32 = F.FEQL_FP16, F.FEQL_FP32
INV, UNS = F.FEQL_ERR_INVALID_ARG, F.FEQL_ERR_UNSUPPORTED
P = 1 << 20  # aligned fake address; never dereferenced: every call below is refused first
BIG = 1 << 30


@pytest.fixture(scope="module")
def lib():
    B.build()
    return F.load()


def test_forward_diff_refusals(lib):
    f = lib.feql_scan_forward_diff
    ok = lambda **k: [k.get(n, d) for n, d in (
        ("u", P), ("g", P), ("h0", None), ("off", None), ("h", P), ("hN", None), ("diff", P),
        ("ws", P), ("bytes", BIG), ("B", 2), ("N", 8), ("C", 4), ("T", 4), ("shared", 0),
        ("dtype", FP16), ("stream", None))]
    for bad in ({"u": None}, {"g": None}, {"h": None}, {"diff": None}, {"diff": P + 4},
                {"B": 3}, {"B": 0}, {"dtype": 17}, {"h0": P + 4}, {"off": P + 4}, {"C": 0}):
        assert f(*ok(**bad)) == INV, bad
    assert f(*ok(T=17)) == UNS
    assert f(*ok(dtype=FP32)) == UNS
    assert f(*ok(B=0, N=0, u=None, g=None, h=None, diff=None)) == F.FEQL_OK


def test_backward_diff_refusals(lib):
    f = lib.feql_scan_backward_diff
    ok = lambda **k: [k.get(n, d) for n, d in (
        ("dh", P), ("g", P), ("diff", P), ("dhN", None), ("off", None), ("du", P), ("dg", P),
        ("dh0", None), ("ws", P), ("bytes", BIG), ("B", 2), ("N", 8), ("C", 4), ("T", 4),
        ("shared", 0), ("dtype", FP16), ("stream", None))]
    for bad in ({"dh": None}, {"g": None}, {"diff": None}, {"du": None}, {"dg": None},
                {"diff": P + 8}, {"dhN": P + 4}, {"dh0": P + 2}, {"off": P + 4}, {"B": 3},
                {"B": -1}, {"N": -1}, {"dtype": -1}):
        assert f(*ok(**bad)) == INV, bad
    assert f(*ok(T=17)) == UNS
    assert f(*ok(dtype=FP32)) == UNS
    assert f(*ok(B=0, N=0, dh=None, g=None, diff=None, du=None, dg=None)) == F.FEQL_OK


def test_rounded_states_are_refused(lib):
    f = lib.feql_scan_backward
    args = [P, P, P, P, None, None, None, P, P, None, P, BIG, 2, 8, 4, 4, 0, FP16, None]
    assert f(*args) == UNS
