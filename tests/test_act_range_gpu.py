"""The value range of the layer's backward pass through an activation in fp16: every
finite dy, as the layer alone takes it, also where dy times a slope of up to 1.13 is
beyond fp16; and gradients among the subnormals.

Tolerances.  dx and dW: the fp16 layer's bound, 5e-3 of their largest value (dz's own
rounding of half a step is inside it).  db is a plain sum of dz over tokens and group
elements: each dz is rounded by half a step 2^-11 itself and at most four times on its way
through a fibre's butterflies (order 8: three stages; the plane's scale is exact), each
time by half a step of a value no larger than the fibre's sum of |dz|.  Below the normal
range a step is absolute: 2^-22 at most for dz, and at most 2^-19 a bin in the operand
planes (include/feql.h); dx[c] takes a bin of each dz[d] with the weights' sum over d and u.
"""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import group_dft_structured_b200 as F
from group_dft_structured_b200 import layer as L
from oracle import feql_ct_oracle as OC
from oracle import feql_p4m_oracle as OP

pytestmark = pytest.mark.gpu

# group, T, mode, N, C, D: the fused p4 backward, its two passes, orders 8 and 6, p4m, CUDA cores
LAYERS = [("cyclic", 4, "fp16", 300, 24, 96), ("cyclic", 4, "fp16", 300, 16, 16),
          ("cyclic", 4, "fp16", 200, 128, 64), ("cyclic", 4, "fp16", 150, 96, 192),
          ("cyclic", 8, "fp16", 200, 12, 20), ("cyclic", 6, "fp16", 200, 8, 16),
          ("p4m", 8, "fp16", 200, 12, 20), ("cyclic", 4, "fp16_simt", 100, 7, 9),
          ("cyclic", 5, "fp16", 100, 6, 7), ("cyclic", 6, "fp16", 100, 5, 7)]


@pytest.fixture(scope="module", autouse=True)
def ready():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from group_dft_structured_b200 import build
    build.build()
    F.load()
    yield
    assert F.feql_device_status() == F.FEQL_OK


def cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def host(t):
    return t.cpu().numpy().astype(np.float64)


def inputs(group, T, mode, N, C, D, seed):
    r = np.random.default_rng(seed + N + 31 * C + 7 * D + T)
    n = lambda s, *shape: (s * r.standard_normal(shape)).astype(np.float16)
    code = F.DTYPES[mode]
    W = n(0.25 / np.sqrt(T * D), D, C, T)
    wfft = L.p4m_weight_fft if group == "p4m" else L.ct_weight_fft
    backward = L.p4m_backward_act if group == "p4m" else L.ct_backward_act
    return r, n, W, wfft(cuda(W), code), code, backward, OP if group == "p4m" else OC


@pytest.mark.parametrize("parts", ["all", "dx", "dw"])
@pytest.mark.parametrize("act", ["gelu", "silu"])
@pytest.mark.parametrize("group,T,mode,N,C,D", LAYERS)
def test_largest_gradients(group, T, mode, N, C, D, act, parts):
    r, n, W, What, code, backward, O = inputs(group, T, mode, N, C, D, 5)
    x, dy = n(1e-2, N, C, T), n(1.0, N, D, T)
    slope = np.full((N, D, T), 0.5, np.float16)
    # the largest finite values in pairs of opposite sign, so that db stays finite, where
    # the slope is GELU's largest
    for d in range(0, D, 3):
        i, j = r.choice(N, 2, replace=False)
        t = r.integers(T)
        dy[i, d, t], dy[j, d, t] = 65504, -65504
        slope[i, d, t] = slope[j, d, t] = 1.1289
    dz = dy.astype(np.float64) * slope.astype(np.float64)
    assert np.abs(dz).max() > 65504
    X, W64 = x.astype(np.float64), W.astype(np.float64)
    rdx, (rdW, rdb) = O.backward_dx(dz, W64), O.backward_dw(X, dz)
    assert max(np.abs(v).max() for v in (rdx, rdW, rdb)) < 6e4
    dx, dW, db = backward(cuda(x), cuda(dy), cuda(slope), What, code, F.ACTIVATIONS[act],
                          with_dx=parts != "dw", with_dw=parts != "dx", with_db=parts != "dx")
    if dx is not None:
        assert O.rel_err(host(dx), rdx) <= 5e-3
    if dW is not None:
        assert O.rel_err(host(dW), rdW) <= 5e-3
        fibre = np.abs(dz).sum(2).sum(0)  # of channel d, over its tokens
        assert (np.abs(host(db) - rdb) <= 2.0 ** -11 * (5 * fibre + np.abs(rdb))).all()


@pytest.mark.parametrize("group,T,mode,N,C,D", LAYERS)
def test_smallest_gradients(group, T, mode, N, C, D):
    r, n, W, What, code, backward, O = inputs(group, T, mode, N, C, D, 6)
    x, dy = n(1.0, N, C, T), n(2.0 ** -17, N, D, T)
    slope = np.clip(n(0.4, N, D, T) + np.float16(0.5), -0.1, 1.1289).astype(np.float16)
    dz = dy.astype(np.float64) * slope.astype(np.float64)
    W64 = W.astype(np.float64)
    dx, dW, db = backward(cuda(x), cuda(dy), cuda(slope), What, code, F.FEQL_ACT_GELU)
    ref = O.backward_dx(dz, W64)
    reach = np.abs(W64).sum(axis=(0, 2))[None, :, None]  # of a bin's step, over d and u
    tol = 5e-3 * np.abs(ref).max() + (2.0 ** -22 + 2.0 ** -19) * reach + 2.0 ** -25
    assert (np.abs(host(dx) - ref) <= tol).all()
    rdW, rdb = O.backward_dw(x.astype(np.float64), dz)
    # each token's step times its x, or its step alone
    tol = 5e-3 * np.abs(rdW).max() + (2.0 ** -22 + 2.0 ** -19) * np.abs(x.astype(np.float64)).sum()
    assert (np.abs(host(dW) - rdW) <= tol + 2.0 ** -25).all()
    assert (np.abs(host(db) - rdb) <= (2.0 ** -22 + 2.0 ** -19) * N * T + 5e-3 * np.abs(rdb)).all()
