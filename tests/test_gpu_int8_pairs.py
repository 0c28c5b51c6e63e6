"""The gradient's two products in one launch (tiles of 64 and of 128, and sizes whose
products take different tiles and so a launch each) against the definition and
against the products one at a time, bit for bit."""
import numpy as np
import pytest
import torch

import quantized_sgd_amd as q
from tests import plain_int8 as plain
from tests.test_gpu_int8 import DTYPES, levels, scales, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    q.lib()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,n,k", [(300, 500, 400), (1100, 70, 333), (1500, 1700, 1600), (300, 1700, 1600)])
def test_gradient_in_one_launch(m, n, k, dtype):
    print("pairs", m, n, k, dtype, flush=True)
    x, w, sw = values(m, k, dtype, 5), levels(n, k, 6, 1), scales(n, 7)
    gy = values(m, n, dtype, 8, 3, 1, 0.01)
    _, xq, sx = q.int8_linear(x, w, sw, keep=True)
    gx, gw = q.int8_linear_backward(gy, xq, sx, w, sw)
    g32, xq_, w_ = plain.to32(gy), xq.cpu().numpy(), w.cpu().numpy()
    gq, sg = plain.quantize_rows(g32, plain.to32(sw))
    hq, sh = plain.quantize_columns(g32, plain.to32(sx))
    assert plain.same(gx, plain.cast(plain.product(gq, sg, np.ascontiguousarray(w_.T)), dtype))
    assert plain.same(gw, torch.from_numpy(plain.product(hq, sh, np.ascontiguousarray(xq_.T))))
    gx1, _ = q.int8_linear_backward(gy, xq, sx, w, sw, need_gw=False)
    _, gw1 = q.int8_linear_backward(gy, xq, sx, w, sw, need_gx=False)
    assert torch.equal(gx1, gx) and torch.equal(gw1, gw)
