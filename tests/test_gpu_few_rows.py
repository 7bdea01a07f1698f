"""Calls of one to nine rows of 4-bit weights, whose kernel packs several
32-k slices of the activations into one operand: every number of rows, k-ranges
with half a last record, ragged columns, sum sets, row indices, infinities.
Exact integer inputs (block_util.Weight), so results are compared bit for bit."""
import numpy as np
import pytest

from block_util import DEV, Weight, f64, ints, out, put, rne, rng, torch, tsl, untouched, ws

pytestmark = pytest.mark.gpu


def linear(items, eps, M):
    n = tsl.shard_linear_group_epilogue_workspace_size(items, eps, tsl.Q4G64, M)
    w = ws(n)
    tsl.shard_linear_group_epilogue(items, eps, tsl.Q4G64, tsl.BF16, M, w, n)


def item(W, x, Y, sh=None, k_off=0, **kw):
    sh = sh or tsl.plan_linear(W.K, W.N, 1, tsl.COLUMN, 64)[0]
    buf, nb = W.pack(sh)
    return dict(shard=sh, packed=buf, packed_bytes=nb, X=x[:, k_off:], ldx=x.stride(0), Y=Y,
                ldy=Y.stride(0), ydtype=tsl.F32, **kw)


@pytest.mark.parametrize("M", range(1, 10))
@pytest.mark.parametrize("K,N", [(64, 16), (128, 33), (192, 20003), (1088, 520), (2560, 96)])
def test_products(M, K, N):
    W, V = Weight("q4", K, N, 1), Weight("q4", K, N, 2)
    x = ints(3, (M, K))
    X = put(x, "bf16")
    yb, Y = out(M, N, "f32")
    pb, P = out(M, N, "f32")
    linear([item(W, X, Y)], [dict(act=tsl.ACT_RELU, pre=P, pre_dtype=tsl.F32, ld_pre=P.stride(0))], M)
    z = x @ W.w
    assert np.array_equal(f64(P), z) and np.array_equal(f64(Y), np.maximum(z, 0))
    bufs = [out(M, N, "bf16") for _ in range(3)]
    (hb, H), (gb, G), (ub, U) = bufs
    a, b = item(W, X, Y), item(V, X, Y)
    it = dict(gate=a["shard"], up=b["shard"], packed_gate=a["packed"], packed_up=b["packed"],
              packed_bytes=a["packed_bytes"], X=X, ldx=X.stride(0), H=H, ldh=H.stride(0),
              hdtype=tsl.BF16, G=G, U=U, ld_gu=G.stride(0))
    n = tsl.shard_gated_group_workspace_size([it], tsl.Q4G64, M)
    w = ws(n)
    tsl.shard_gated_group([it], tsl.ACT_RELU, tsl.Q4G64, tsl.BF16, M, w, n)
    u = x @ V.w
    assert np.array_equal(f64(G), rne(z, "bf16")) and np.array_equal(f64(U), rne(u, "bf16"))
    # z and u are whole multiples of 2^-7 below 2^10: binary32 rounds their
    # product once, by half a step, and bf16 once more
    assert np.all(np.abs(f64(H) - np.maximum(z, 0) * u) <=
                  (2.0 ** -8 + 2.0 ** -23) * np.abs(np.maximum(z, 0) * u))
    for buf in (yb, pb, hb, gb, ub):
        assert untouched(buf, M, N)


@pytest.mark.parametrize("M", [1, 4, 5, 8])
def test_sum_sets_and_indices(M):
    t = torch()
    N, T = 100, 11
    Y = out(M, N, "f32")[1]
    items, want = [], 0
    for i, K in enumerate((192, 64, 448)):
        W = Weight("q4", K, N, 20 + i)
        x = ints(30 + i, (T, K))
        idx = rng(40 + i).integers(-1, T + 1, size=M).astype(np.int32)
        items.append(item(W, put(x, "bf16"), Y, sum_next=int(i < 2), x_rows=T,
                          row_index=t.from_numpy(idx).to(DEV)))
        want = want + np.where(((idx >= 0) & (idx < T))[:, None], x[np.clip(idx, 0, T - 1)], 0) @ W.w
    linear(items, [dict(act=tsl.ACT_NONE), None, None], M)
    assert np.array_equal(f64(Y), want)


@pytest.mark.parametrize("M", [3, 7])
def test_rows_stay_apart(M):
    """Items of fewer rows than the call, and a row that is not finite."""
    K, N = 320, 72
    W = Weight("q4", K, N, 50)
    x = ints(51, (M, K))
    x[1, 70] = np.inf
    X = put(x, "bf16")
    bufs = [out(M, N, "f32") for _ in range(2)]
    linear([item(W, X, bufs[0][1]), item(W, X, bufs[1][1], rows=2)],
           [dict(act=tsl.ACT_NONE)] * 2, M)
    z = np.where(np.isfinite(x), x, 0) @ W.w
    for (buf, Y), m in zip(bufs, (M, 2)):
        y = f64(Y)
        keep = np.arange(m) != 1
        assert np.array_equal(y[:m][keep], z[:m][keep]) and not np.isfinite(y[1]).any()
        assert untouched(buf, m, N)


def test_repeats_and_replays():
    t = torch()
    M, K, N = 4, 4736, 200
    W = Weight("q4", K, N, 60, exact=False)
    X = put(rng(61).standard_normal((M, K)), "bf16")
    Y = out(M, N, "f32")[1]
    its, ep = [item(W, X, Y)], [dict(act=tsl.ACT_SILU)]
    linear(its, ep, M)
    want = Y.clone()
    g, side = t.cuda.CUDAGraph(), t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    with t.cuda.graph(g, stream=side):
        linear(its, ep, M)
    for _ in range(4):
        Y.fill_(-1)
        g.replay()
        t.cuda.synchronize()
        assert bool((Y == want).all())
        linear(its, ep, M)
        assert bool((Y == want).all())
