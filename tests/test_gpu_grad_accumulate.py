"""Gradient accumulation at sizes where dX and the accumulating weight gradients
share a launch of another plan than without, with exactly the queried workspace.
Integer inputs: every sum is exact in binary32 (below 2^24 steps), so the results
match the formulas in binary64 bit for bit, before and after accumulating."""
import numpy as np
import pytest

from block_util import Weight, f64, ints, put
from gpu_util import torch
from tensor_sharded_linear_plan_amd import binding as tsl
from test_gpu_grad import gated_grad, linear_grad

pytestmark = pytest.mark.gpu


def product(a, b):
    """In binary64 on the GPU: the sizes take numpy seconds."""
    t = torch()
    return (t.from_numpy(a).cuda() @ t.from_numpy(np.ascontiguousarray(b)).cuda()).cpu().numpy()


@pytest.mark.parametrize("M,K,N,order", [(1347, 1029, 3517, "kn"), (1369, 310, 3169, "kn"),
                                         (1203, 57, 5501, "nk")])
def test_linear(M, K, N, order):
    W = Weight("bf16", K, N, 3)
    sh = tsl.plan_linear(K, N, 1, tsl.COLUMN)[0]
    x, dy = ints(1, (M, K)), ints(2, (M, N))
    for acc, fill in ((0, 7.0), (1, 4.0)):
        dX, dW, db = linear_grad("bf16", W, sh, put(x, "bf16"), "none", None, put(dy, "bf16"),
                                 order=order, acc=acc, fill=fill)
        assert np.array_equal(f64(dX), product(dy, W.w.T))
        assert np.array_equal(f64(dW), product(x.T.copy(), dy) + acc * fill)
        assert np.array_equal(f64(db), dy.sum(0) + acc * fill)


@pytest.mark.parametrize("M,K,N,order", [(1024, 2048, 2048, "kn"), (1152, 2432, 2304, "nk")])
def test_gated(M, K, N, order):
    Wg, Wu = Weight("bf16", K, N, 5), Weight("bf16", K, N, 6)
    sh = tsl.plan_linear(K, N, 1, tsl.COLUMN)[0]
    x, g, u, dh = ints(1, (M, K)), ints(2, (M, N)), ints(3, (M, N)), ints(4, (M, N))
    zg, zu = dh * u * (g > 0), dh * np.maximum(g, 0)
    want = product(zg, Wg.w.T) + product(zu, Wu.w.T)
    for acc, fill in ((0, 7.0), (1, 4.0)):
        dX, dg, du = gated_grad("bf16", Wg, Wu, sh, put(x, "bf16"), "relu", put(g, "bf16"),
                                put(u, "bf16"), put(dh, "bf16"), order=order, acc=acc, fill=fill)
        assert np.array_equal(f64(dX), want)
        assert np.array_equal(f64(dg), product(x.T.copy(), zg) + acc * fill)
        assert np.array_equal(f64(du), product(x.T.copy(), zu) + acc * fill)
