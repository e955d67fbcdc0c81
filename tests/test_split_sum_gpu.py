"""Weight gradients of the CUDA-core layers around the rule that picks the form of the sum
over the splits: a thread an output where they fill the GPU or the splits are few, else a
block for 32 outputs; sizes on either side, against float64.

Tolerance: the layer's fp32 bound, 1e-5 of the largest value (fp16 data: 5e-3).
"""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import group_dft_structured_b200 as F
from group_dft_structured_b200 import layer as L
from oracle import feql_ct_oracle as O

pytestmark = pytest.mark.gpu

# T, mode, N, C, D: one split; few; many on few outputs; many on more than 37888 (256 an SM)
CASES = [(4, "fp32", 3, 200, 190), (4, "fp32", 60, 33, 31), (4, "fp32", 100, 20, 30),
         (4, "fp32", 900, 35, 51), (4, "fp32", 400, 190, 199), (4, "fp32", 400, 192, 198),
         (4, "fp16_simt", 500, 17, 19), (4, "fp16_simt", 90, 200, 200), (4, "fp32", 5, 520, 514),
         (3, "fp32", 7, 160, 250), (3, "fp32", 120, 160, 161), (8, "fp32", 500, 20, 21),
         (16, "fp32", 300, 30, 33), (12, "fp16", 200, 40, 41), (5, "fp16", 9, 200, 200),
         (2, "fp32", 1, 1, 1), (7, "fp32", 0, 12, 11)]


@pytest.fixture(scope="module", autouse=True)
def ready():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from group_dft_structured_b200 import build
    build.build()
    F.load()


@pytest.mark.parametrize("with_db", [True, False])
@pytest.mark.parametrize("T,mode,N,C,D", CASES)
def test_weight_gradient(T, mode, N, C, D, with_db):
    code = F.DTYPES[mode]
    dt = np.float16 if "16" in mode else np.float32
    r = np.random.default_rng(N + C + 3 * D + T)
    x, dy = (r.standard_normal((N, k, T)).astype(dt) for k in (C, D))
    X, Y = (torch.from_numpy(v).cuda() for v in (x, dy))
    dW, db = L.ct_backward_dw(X, Y, code, with_db=with_db)
    again = L.ct_backward_dw(X, Y, code, with_db=with_db)
    assert torch.equal(dW, again[0]) and (db is None) == (not with_db)
    tol = 5e-3 if dt == np.float16 else 1e-5
    rdW, rdb = O.backward_dw(x.astype(np.float64), dy.astype(np.float64))
    for got, ref in ((dW, rdW), (db, rdb)):
        if got is not None:
            got = got.cpu().numpy().astype(np.float64)
            assert np.isfinite(got).all() and got.shape == ref.shape
            assert (np.abs(got - ref) <= tol * np.abs(ref).max()).all()
