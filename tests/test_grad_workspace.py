"""The backward passes accept the workspace their size queries ask for, on the
host alone: the workspace's address is odd, so a call of enough bytes ends in
TSL_ERR_MISALIGNED and one of too few in TSL_ERR_BUFFER_TOO_SMALL."""
import math
import random

import pytest

A = 1 << 44  # addresses a terabyte apart; never read
STEP = 1 << 40


def addr(i):
    return A + i * STEP


def up(v, a):
    return (v + a - 1) // a * a


def status(t, n_w, M, K, N, wdtype, act, outputs, order, accumulate):
    """Status of a call of exactly the queried bytes.  outputs: 1 dX, 2 the
    weight gradients, 3 both (linear: the bias gradient with each)."""
    sh = t.plan_linear(K, N, 1, t.COLUMN)[0]
    if n_w == 1:
        n = t.shard_linear_grad_workspace_size(sh, wdtype, M)
    else:
        n = t.shard_gated_grad_workspace_size(sh, sh, wdtype, M)
    sk, sn = (1, K) if order else (N, 1)
    a = dict(wdtype=wdtype, packed_t_bytes=STEP, M=M, X=addr(1), ldx=up(K, 8), act=act,
             dxdtype=t.BF16, dX=addr(2) if outputs & 1 else None, lddx=K, dwdtype=t.F32,
             dw_stride_k=sk, dw_stride_n=sn, accumulate_dw=accumulate, workspace=addr(3) + 1,
             ws_bytes=n, stream=0)
    dw = [addr(4), addr(5)] if outputs & 2 else [None, None]
    with pytest.raises(t.TslError) as e:
        if n_w == 1:
            t.shard_linear_grad(shard=sh, packed_t=addr(0), Z=addr(6), ldz=up(N, 8), dY=addr(7),
                                lddy=up(N, 8), dW=dw[0], db=addr(8), **a)
        else:
            t.shard_gated_grad(gate=sh, up=sh, packed_gate_t=addr(0), packed_up_t=addr(8),
                               G=addr(6), U=addr(9), ld_gu=up(N, 8), dH=addr(7), lddh=up(N, 8),
                               dW_gate=dw[0], dW_up=dw[1], **a)
    return e.value.status


# a weight gradient that accumulates is not split along k, and dX beside it in
# the launch then takes more partials than in a call that does not accumulate
@pytest.mark.parametrize("n_w,M,K,N,order", [(2, 1024, 2048, 2048, 0), (1, 1347, 1029, 3517, 0),
                                             (2, 2206, 1369, 2530, 0), (1, 1369, 310, 3169, 0),
                                             (1, 1203, 57, 5501, 1), (2, 1152, 2432, 2304, 0),
                                             (2, 1739, 2007, 5418, 1), (1, 4864, 512, 3456, 0)])
def test_accumulating_calls_fit_their_query(tsl_lib, n_w, M, K, N, order):
    t = tsl_lib
    for act in (t.ACT_NONE, t.ACT_RELU, t.ACT_SILU):
        for o in (order, 1 - order):
            for outputs in (1, 2, 3):
                for acc in (0, 1):
                    got = status(t, n_w, M, K, N, t.BF16, act, outputs, o, acc)
                    assert got == t.ERR_MISALIGNED, (act, o, outputs, acc)


def test_drawn_calls_fit_their_query(tsl_lib):
    t = tsl_lib
    rng = random.Random(5)

    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    for _ in range(400):
        small = rng.random() < .4  # where rounding's remainders are operands too
        wdtype = t.F32 if rng.random() < .2 else t.BF16
        most = 600 if wdtype == t.F32 else 6000
        M, K, N = (log(1, 64), log(16, most), log(16, 1024)) if small else \
            (log(1, most), log(16, most), log(16, most))
        c = (rng.choice([1, 2]), M, K, N, wdtype, rng.choice([t.ACT_NONE, t.ACT_RELU, t.ACT_GELU]),
             rng.choice([1, 2, 3]), rng.choice([0, 1]), rng.choice([0, 1]))
        assert status(t, *c) == t.ERR_MISALIGNED, c
