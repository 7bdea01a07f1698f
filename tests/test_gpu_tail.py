"""Large products of somewhat more tiles than whole rounds over the chip, whose
last columns run as a piece of their own, split along k: exact integer inputs,
so both pieces and the seam between them must match the formula (as in
test_gpu_epilogue.py and test_gpu_gated.py)."""
import numpy as np
import pytest

from block_util import DT, U, Weight, act, close, f64, ints, out, put, rne, untouched, ws
from gpu_util import torch
from tensor_sharded_linear_plan_amd import binding as tsl

pytestmark = pytest.mark.gpu


def partial_bytes(n, wk, M, K):
    """A workspace's part behind the binary16 activation copy of 4-bit weights."""
    if wk == "bf16":
        return n
    return n - (M * K * 2 + (M + 255) // 256 * 1024 + 255) // 256 * 256


@pytest.mark.parametrize("wk,M,K,N", [("bf16", 1670, 1536, 4728), ("bf16", 1972, 1600, 4387),
                                      ("q4", 1859, 1472, 4458), ("q4", 1567, 1536, 5143)])
def test_gated(wk, M, K, N):
    x = ints(1, (M, K))
    G, Up = Weight(wk, K, N, 2), Weight(wk, K, N, 3)
    sh = tsl.plan_linear(K, N, 1, tsl.COLUMN, 64 if wk == "q4" else 0)[0]
    (pg, nb), (pu, _) = G.pack(sh), Up.pack(sh)
    X = put(x, "bf16")
    bufs = [out(M, N, "bf16") for _ in range(3)]
    (hb, H), (gb, Go), (ub, Uo) = bufs
    it = dict(gate=sh, up=sh, packed_gate=pg, packed_up=pu, packed_bytes=nb, X=X, ldx=X.stride(0),
              H=H, ldh=H.stride(0), hdtype=tsl.BF16, G=Go, U=Uo, ld_gu=Go.stride(0))
    n = tsl.shard_gated_group_workspace_size([it], DT[wk], M)
    assert 0 < partial_bytes(n, wk, M, K) < M * 2 * N * 4  # a part of the columns is split
    for _ in range(2):
        tsl.shard_gated_group([it], tsl.ACT_SILU, DT[wk], tsl.BF16, M, ws(n), n)
    g, u = x @ G.w, x @ Up.w
    a, _, err = act(g, "silu")
    assert np.array_equal(f64(Go), rne(g, "bf16")) and np.array_equal(f64(Uo), rne(u, "bf16"))
    close(f64(H), a * u, (err + 2 * U * np.abs(a)) * np.abs(u), "bf16")
    assert all(untouched(b, M, N) for b, _ in bufs)


@pytest.mark.parametrize("wk,M,K,N,tp", [("bf16", 3570, 1344, 4629, 1), ("bf16", 3084, 1408, 5169, 1),
                                         ("q4", 3660, 1344, 4365, 1), ("q4", 3515, 1344, 4649, 1),
                                         ("q4", 3515, 1536, 4649, 2), ("bf16", 3084, 1536, 5169, 2)])
@pytest.mark.parametrize("k", ["bf16", "f32"])
def test_epilogue(wk, M, K, N, tp, k):
    W = Weight(wk, K, N, 5)
    x = ints(6, (M, K))
    X = put(x, "bf16")
    b = put(ints(7, (1, N), -9, 9) * 2.0 ** -3, k)[0]
    r = put(ints(8, (M, N), -9, 9), k)
    pb, P = out(M, N, k)
    items, eps = [], []
    for i, sh in enumerate(tsl.plan_linear(K, N, tp, tsl.ROW, 64 if wk == "q4" else 0)):
        buf, nb = W.pack(sh)
        items.append(dict(shard=sh, packed=buf, packed_bytes=nb, X=X[:, sh.k_off:], ldx=X.stride(0),
                          Y=r, ldy=r.stride(0), ydtype=DT[k], sum_next=int(i + 1 < tp)))
        eps.append(None)
    eps[0] = dict(act=tsl.ACT_RELU, bias=b, bias_dtype=DT[k], residual=r, res_dtype=DT[k],
                  ld_res=r.stride(0), pre=P, pre_dtype=DT[k], ld_pre=P.stride(0))
    res = f64(r)
    n = tsl.shard_linear_group_epilogue_workspace_size(items, eps, DT[wk], M)
    if tp == 1:
        assert 0 < partial_bytes(n, wk, M, K) < M * N * 4
    tsl.shard_linear_group_epilogue(items, eps, DT[wk], tsl.BF16, M, ws(n), n)
    z = x @ W.w + f64(b)
    assert np.array_equal(f64(P), rne(z, k))
    # every term is exact in binary32, and so is their sum
    assert np.array_equal(f64(r), rne(np.maximum(z, 0) + res, k))
    assert untouched(pb, M, N)
