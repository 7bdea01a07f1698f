"""Sum sets of more members together than one launch of the few-rows form holds:
each set's result and the padding around it, bit for bit (integer inputs)."""
import numpy as np
import pytest

from block_util import Weight, f64, ints, out, put, tsl, untouched
from test_gpu_few_rows import item, linear

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [1, 2, 4, 7])
@pytest.mark.parametrize("sets,members", [(33, 4), (64, 3), (70, 2), (9, 16)])
def test_sets(sets, members, M):
    K, N = 192, 40
    Ws = [Weight("q4", K, N, 10 + r) for r in range(5)]
    xs = [ints(20 + r, (M, K)) for r in range(3)]
    Xs = [put(x, "bf16") for x in xs]
    made = [item(W, Xs[0], Xs[0]) for W in Ws]
    items, eps, bufs, wants = [], [], [], []
    for s in range(sets):
        buf, Y = out(M, N, "f32")
        want = 0
        for r in range(members):
            w, x = (s + 2 * r) % 5, (s + r) % 3
            items.append(dict(made[w], X=Xs[x], ldx=Xs[x].stride(0), Y=Y, ldy=Y.stride(0),
                              sum_next=int(r + 1 < members)))
            eps.append(None)
            want = want + xs[x] @ Ws[w].w
        if s % 3 != 1:
            eps[-members] = dict(act=tsl.ACT_RELU)
            want = np.maximum(want, 0)
        bufs.append((buf, Y))
        wants.append(want)
    linear(items, eps, M)
    for (buf, Y), want in zip(bufs, wants):
        assert np.array_equal(f64(Y), want) and untouched(buf, M, N)
