"""shard_gated_group on the GPU: act(X W_gate) * (X W_up) against the formula
in binary64.  Inputs are small integers (weights times a power of two), so
both products are exact in every kernel's arithmetic and the kept G and U must
match bit for bit; H then carries the activation's error (block_util.act), one
product's and the stored type's rounding."""
import numpy as np
import pytest

from block_util import (ACTS, DT, U, Weight, act, close, f64, ints, out, put, rne, rng, untouched,
                        ws)
from gpu_util import DEV, torch
from tensor_sharded_linear_plan_amd import binding as tsl

pytestmark = pytest.mark.gpu


def xkind(wk):
    return "f32" if wk == "f32" else "bf16"


def item(wk, x, K, N, seed, hk="bf16", save=False, exact=True, X=None, tp=1, rank=0):
    """(item, G weight, U weight, buffers) of one rank's gate and up column shards."""
    G, Up = Weight(wk, K, N * tp, seed, exact), Weight(wk, K, N * tp, seed + 1, exact)
    sh = tsl.plan_linear(K, N * tp, tp, tsl.COLUMN, 64 if wk == "q4" else 0)[rank]
    (pg, nb), (pu, _) = G.pack(sh), Up.pack(sh)
    X = put(x, xkind(wk)) if X is None else X
    M = x.shape[0]
    hb, H = out(M, N, hk)
    it = dict(gate=sh, up=sh, packed_gate=pg, packed_up=pu, packed_bytes=nb, X=X, ldx=X.stride(0),
              H=H, ldh=H.stride(0), hdtype=DT[hk])
    bufs = [(hb, H)]
    if save:
        bufs += [out(M, N, hk), out(M, N, hk)]
        it.update(G=bufs[1][1], U=bufs[2][1], ld_gu=bufs[1][1].stride(0))
    c = slice(rank * N, (rank + 1) * N)
    return it, G.w[:, c], Up.w[:, c], bufs


def run(items, name, wk, M):
    n = tsl.shard_gated_group_workspace_size(items, DT[wk], M)
    w = ws(n)
    tsl.shard_gated_group(items, ACTS[name], DT[wk], DT[xkind(wk)], M, w, n)
    return w


def check(x, wg, wu, bufs, name, hk, m):
    g, u = x @ wg, x @ wu
    a, _, err = act(g, name)
    H = bufs[0][1][:m]
    close(f64(H), a * u, (err + 2 * U * np.abs(a)) * np.abs(u), hk)
    if len(bufs) > 1:
        assert np.array_equal(f64(bufs[1][1][:m]), rne(g, hk))
        assert np.array_equal(f64(bufs[2][1][:m]), rne(u, hk))
    for b, v in bufs:
        assert untouched(b, m, v.shape[1])


CASES = [("f32", 1, 100, 33), ("f32", 20, 256, 48), ("bf16", 1, 256, 40), ("bf16", 2, 4096, 513),
         ("bf16", 4, 1000, 1792), ("bf16", 9, 640, 300), ("bf16", 32, 512, 1000),
         ("bf16", 33, 128, 70), ("bf16", 64, 2048, 33), ("bf16", 65, 1000, 257),
         ("bf16", 300, 512, 700), ("bf16", 512, 256, 1792), ("bf16", 40, 72, 8),
         ("bf16", 140, 2048, 64),
         ("q4", 1, 256, 40), ("q4", 1, 3584, 4736), ("q4", 3, 1024, 65), ("q4", 4, 128, 16),
         ("q4", 16, 1024, 260), ("q4", 40, 512, 1000), ("q4", 64, 192, 65), ("q4", 65, 128, 33),
         ("q4", 130, 2048, 300), ("q4", 257, 512, 1031), ("q4", 80, 64, 130)]


@pytest.mark.parametrize("wk,M,K,N", CASES)
@pytest.mark.parametrize("name,hk,save", [("silu", "bf16", False), ("gelu", "f32", True)])
def test_against_formula(wk, M, K, N, name, hk, save):
    x = ints(K + M, (M, K))
    it, wg, wu, bufs = item(wk, x, K, N, 3 * N, hk, save)
    run([it], name, wk, M)
    check(x, wg, wu, bufs, name, hk, M)


@pytest.mark.parametrize("name", list(ACTS))
@pytest.mark.parametrize("wk,M", [("f32", 3), ("bf16", 1), ("bf16", 12), ("bf16", 100), ("q4", 2),
                                  ("q4", 31), ("q4", 70)])
def test_activations(wk, M, name):
    x = ints(8, (M, 192))
    it, wg, wu, bufs = item(wk, x, 192, 100, 6, "bf16", True)
    run([it], name, wk, M)
    check(x, wg, wu, bufs, name, "bf16", M)


@pytest.mark.parametrize("wk,M", [("bf16", 2), ("bf16", 30), ("bf16", 100), ("q4", 1), ("q4", 90)])
def test_every_rank_of_a_layer(wk, M):
    """The four ranks' column shards side by side in one H."""
    t = torch()
    K, N, tp = 512, 80, 4
    x = ints(18, (M, K))
    X = put(x, "bf16")
    H = t.full((M, N * tp), 7.0, device=DEV)
    items = []
    for r in range(tp):
        it, wg, wu, _ = item(wk, x, K, N, 40, X=X, tp=tp, rank=r)
        it.update(H=H[:, r * N:], ldh=N * tp, hdtype=tsl.F32)
        items.append(it)
    run(items, "silu", wk, M)
    G, Up = Weight(wk, K, N * tp, 40).w, Weight(wk, K, N * tp, 41).w
    a, _, err = act(x @ G, "silu")
    close(f64(H), a * (x @ Up), (err + 2 * U * np.abs(a)) * np.abs(x @ Up), "f32")


@pytest.mark.parametrize("wk", ["q4", "bf16", "f32"])
@pytest.mark.parametrize("T", [1, 40, 300])
def test_experts_over_routed_rows(wk, T):
    """A mixture-of-experts layer: each expert over the tokens routed to it,
    read through the routing's row index; one expert gets no row of its own
    (an index outside X reads zeros)."""
    t = torch()
    E, top, K, N = 6, 2, 128, 96
    x = ints(28, (T, K))
    X = put(x, xkind(wk))
    topk = np.stack([rng(29 + i).permutation(E - 1)[:top] for i in range(T)]).astype(np.int32)
    off, row_slot, _ = tsl.moe_dispatch(topk, E, np.arange(E, dtype=np.int32))
    tok = np.concatenate([row_slot // top, [-1]]).astype(np.int32)  # the idle expert's row
    dtok = t.from_numpy(tok).to(DEV)
    R = len(tok)
    hb, H = out(R, N, "bf16")
    items, refs, most = [], [], 1
    for e in range(E):
        lo, hi = (int(off[e]), int(off[e + 1])) if e < E - 1 else (R - 1, R)
        if hi == lo:
            continue
        it, wg, wu, _ = item(wk, x, K, N, 100 + 2 * e, X=X)
        it.update(H=H[lo:], ldh=H.stride(0), rows=hi - lo, row_index=dtok[lo:], x_rows=T)
        items.append(it)
        refs.append((lo, hi, wg, wu))
        most = max(most, hi - lo)
    run(items, "silu", wk, most)
    for lo, hi, wg, wu in refs:
        xe = np.where((tok[lo:hi] >= 0)[:, None], x[np.maximum(tok[lo:hi], 0)], 0)
        a, _, err = act(xe @ wg, "silu")
        close(f64(H[lo:hi]), a * (xe @ wu), (err + 2 * U * np.abs(a)) * np.abs(xe @ wu), "bf16")
    assert untouched(hb, R, N) and not f64(H)[R - 1].any()


def test_many_experts_past_one_launch():
    """300 blocks in one call, streamed and in the GEMM regime."""
    for wk, M in (("q4", 1), ("q4", 66), ("bf16", 2), ("bf16", 34)):
        x = ints(38, (M, 64))
        X = put(x, "bf16")
        it, wg, wu, _ = item(wk, x, 64, 40, 44, X=X)
        H = torch().zeros((300, M, 40), device=DEV)
        items = [dict(it, H=H[i], ldh=40, hdtype=tsl.F32) for i in range(300)]
        run(items, "relu", wk, M)
        want = np.maximum(x @ wg, 0) * (x @ wu)
        # the product of two exact values, rounded once
        assert np.array_equal(f64(H), np.broadcast_to(rne(want, "f32"), H.shape)), (wk, M)


@pytest.mark.parametrize("wk,M", [("bf16", 3), ("bf16", 64), ("q4", 2), ("q4", 20), ("q4", 128)])
def test_random_values(wk, M):
    """Random values, gate without an activation (H = G U): the mean square
    error against |G| spread(U) + |U| spread(G), spread = sqrt(sum (x w)^2).
    Bounds of a product as in the epilogue's test: 2^-14 of the spread, or
    2^-11 sqrt(2 / 3) where the operands are binary16; binary32's own rounding
    of the product is far below either."""
    K, N = 1536, 333
    x = rng(5).standard_normal((M, K)).astype(np.float32)
    X = put(x, "bf16")
    it, wg, wu, bufs = item(wk, x, K, N, 33, "f32", False, False, X)
    run([it], "none", wk, M)
    x = f64(X)
    g, u = x @ wg, x @ wu
    scale = np.abs(g) * np.sqrt(x ** 2 @ wu ** 2) + np.abs(u) * np.sqrt(x ** 2 @ wg ** 2)
    e = np.sqrt(np.mean(((f64(bufs[0][1]) - g * u) / scale) ** 2))
    assert e < (2.0 ** -11 * np.sqrt(2 / 3) if wk == "q4" and M > 64 else 2.0 ** -14)


def test_non_finite_rows_stay_apart():
    for wk, M in (("q4", 3), ("q4", 70), ("bf16", 3), ("bf16", 70)):
        x = ints(48, (M, 128))
        X = put(x, "bf16")
        X[1, 3] = float("nan")
        it, wg, wu, bufs = item(wk, x, 128, 64, 50, X=X)
        run([it], "silu", wk, M)
        got = f64(bufs[0][1])
        assert np.isnan(got[1]).all() and np.isfinite(np.delete(got, 1, 0)).all(), (wk, M)


@pytest.mark.parametrize("wk,M", [("q4", 1), ("q4", 8), ("q4", 100), ("bf16", 1), ("bf16", 64)])
def test_captured_and_replayed(wk, M):
    t = torch()
    x = ints(58, (M, 2048))
    it, wg, wu, bufs = item(wk, x, 2048, 200, 60, "bf16", True)
    run([it], "silu", wk, M)
    want = [v.clone() for _, v in bufs]
    n = tsl.shard_gated_group_workspace_size([it], DT[wk], M)
    own, g, side = ws(n), t.cuda.CUDAGraph(), t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    with t.cuda.graph(g, stream=side):
        tsl.shard_gated_group([it], ACTS["silu"], DT[wk], tsl.BF16, M, own, n)
    for _ in range(3):
        for _, v in bufs:
            v.zero_()
        g.replay()
        t.cuda.synchronize()
        assert all(t.equal(a, b) for (_, a), b in zip(bufs, want))
        run([it], "silu", wk, M)
        t.cuda.synchronize()
