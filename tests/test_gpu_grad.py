"""Backward passes of the shard products with an epilogue and of the gated
block, on the GPU, against the formulas in binary64 and against differences.

Small integer inputs (weights times a power of two) with no activation or relu
make every dZ exact in its stored type and every sum exact in binary32, so the
results must match bit for bit (rounded once to their type).  With a smooth
activation each dZ is off by its stored type's half step h plus the slope's own
error: at most h + 2^-16 of it in bf16 (the slope's few hundred u are below
2^-16) and 2^-16 in binary32, which bounds the products' error by that times
sum |dZ| |W|, plus one u per term of the binary32 sum."""
import numpy as np
import pytest

from block_util import (ACTS, DT, HALF, U, Weight, act, close, f64, ints, out, put, rne, rng, tt,
                        untouched, ws)
from gpu_util import DEV, torch
from tensor_sharded_linear_plan_amd import binding as tsl

pytestmark = pytest.mark.gpu


def packed_t(W, sh):
    return W.pack(tsl.transpose_shard(sh), transposed=True)


def dw_out(K, N, kind, order, fill=7.0):
    """(buffer, [K][N] view, stride_k, stride_n) of a gradient in either order."""
    if order == "kn":
        buf, v = out(K, N, kind, fill=fill)
        return buf, v, v.stride(0), 1
    buf, v = out(N, K, kind, fill=fill)
    return buf, v.t(), 1, v.stride(0)


def linear_grad(wk, W, sh, X, name, Z, dY, xk="f32", wgk="f32", order="kn", want="xwb", acc=0,
                fill=7.0):
    M, K, N = dY.shape[0], sh.k_len, sh.n_len
    pt, nb = packed_t(W, sh)
    xb, dX = out(M, K, xk)
    wb, dW, sk, sn = dw_out(K, N, wgk, order, fill)
    db = torch().full((N,), fill, device=DEV)
    n = tsl.shard_linear_grad_workspace_size(sh, DT[wk], M)
    w = ws(n)
    tsl.shard_linear_grad(sh, DT[wk], pt if "x" in want else None, nb, M, X if "w" in want else None,
                          X.stride(0), ACTS[name], Z, 0 if Z is None else Z.stride(0), dY,
                          dY.stride(0), DT[xk], dX if "x" in want else None, dX.stride(0), DT[wgk],
                          dW if "w" in want else None, sk, sn, acc, db if "b" in want else None, w,
                          n)
    assert untouched(xb, M, K)
    r, c = (K, N) if order == "kn" else (N, K)
    assert untouched(wb, r, c, fill)
    return dX, dW, db


SHAPES = [(1, 64, 40), (3, 200, 513), (17, 72, 64), (33, 128, 100), (64, 257, 130), (65, 520, 33),
          (200, 96, 300), (300, 640, 256), (1000, 64, 70), (5, 8, 1)]


@pytest.mark.parametrize("M,K,N", SHAPES)
@pytest.mark.parametrize("wk,name,xk,wgk,order", [("bf16", "none", "f32", "f32", "kn"),
                                                  ("bf16", "relu", "bf16", "bf16", "nk"),
                                                  ("bf16", "none", "bf16", "f32", "nk"),
                                                  ("f32", "relu", "f32", "f32", "kn"),
                                                  ("f32", "none", "f32", "f32", "nk")])
def test_linear_exact(M, K, N, wk, name, xk, wgk, order):
    W = Weight(wk, K, N, M + K)
    sh = tsl.plan_linear(K, N, 1, tsl.COLUMN)[0]
    x, dy, z = ints(1, (M, K)), ints(2, (M, N)), ints(3, (M, N), -9, 9)
    Z = put(z, wk) if name != "none" else None
    dX, dW, db = linear_grad(wk, W, sh, put(x, wk), name, Z, put(dy, wk), xk, wgk, order)
    dz = dy * act(z, name)[1]
    assert np.array_equal(f64(dX), rne(dz @ W.w.T, xk))
    assert np.array_equal(f64(dW), rne(x.T @ dz, wgk))
    assert np.array_equal(f64(db), dz.sum(0))


@pytest.mark.parametrize("name", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("wk,M,K,N", [("bf16", 4, 136, 72), ("bf16", 100, 136, 200), ("f32", 50, 64, 40)])
def test_linear_smooth(name, wk, M, K, N):
    W = Weight(wk, K, N, 5)
    sh = tsl.plan_linear(K, N, 1, tsl.COLUMN)[0]
    X, dY, Z = (put(rng(s).standard_normal((M, c)) * k, wk)
                for s, c, k in ((6, K, 1), (7, N, 1), (8, N, 2.5)))
    dX, dW, db = linear_grad(wk, W, sh, X, name, Z, dY)
    x, z, dy = f64(X), f64(Z), f64(dY)
    dz = dy * act(z, name)[1]
    rel = 2.0 ** -16 + (HALF["bf16"] if wk == "bf16" else 0)
    # the slope near its zeros: within 2^-16 of the largest slope, 1.13
    err = rel * np.abs(dz) + 2.0 ** -16 * 1.13 * np.abs(dy)
    close(f64(dX), dz @ W.w.T, err @ np.abs(W.w.T) + N * U * (np.abs(dz) @ np.abs(W.w.T)), "f32")
    close(f64(dW), x.T @ dz, np.abs(x.T) @ err + M * U * (np.abs(x.T) @ np.abs(dz)), "f32")
    close(f64(db), dz.sum(0), 2.0 ** -16 * 2.2 * np.abs(dy).sum(0), "f32")


@pytest.mark.parametrize("wk,M", [("bf16", 20), ("bf16", 90), ("f32", 20)])
def test_linear_accumulates_and_parts(wk, M):
    """accumulate adds to dW and db; any subset of the outputs may be wanted
    and equals the full call's, bit for bit."""
    t = torch()
    K, N = 96, 136
    W = Weight(wk, K, N, 15)
    sh = tsl.plan_linear(K, N, 1, tsl.COLUMN)[0]
    X, dY, Z = (put(rng(s).standard_normal((M, c)), wk) for s, c in ((6, K), (7, N), (8, N)))
    x, dy = ints(1, (M, K)), ints(2, (M, N))
    _, dW, db = linear_grad(wk, W, sh, put(x, wk), "none", None, put(dy, wk), acc=1, fill=4.0)
    assert np.array_equal(f64(dW), 4 + x.T @ dy) and np.array_equal(f64(db), 4 + dy.sum(0))
    full = linear_grad(wk, W, sh, X, "silu", Z, dY)
    for want in ("x", "b", "xb"):
        got = linear_grad(wk, W, sh, X, "silu", Z, dY, want=want)
        for i, k in enumerate("xwb"):
            if k in want:
                assert t.equal(got[i], full[i]), want
    # dW alone may run in another launch: its sums may group k differently
    got = linear_grad(wk, W, sh, X, "silu", Z, dY, want="w")[1]
    assert float((got - full[1]).abs().max()) <= M * U * 40


def test_row_shard_and_replicated():
    """A row shard's backward reads the rank's block of W."""
    W = Weight("bf16", 256, 96, 25)
    M = 70
    for sh in tsl.plan_linear(256, 96, 2, tsl.ROW) + tsl.plan_linear(256, 96, 2, tsl.REPLICATED)[:1]:
        x, dy = ints(1, (M, sh.k_len)), ints(2, (M, 96))
        w = W.w[sh.k_off:sh.k_off + sh.k_len]
        dX, dW, db = linear_grad("bf16", W, sh, put(x, "bf16"), "none", None, put(dy, "bf16"))
        assert np.array_equal(f64(dX), dy @ w.T) and np.array_equal(f64(dW), x.T @ dy)
        t = tsl.transpose_shard(sh)
        assert (t.K, t.N, t.k_len, t.n_len) == (96, 256, 96, sh.k_len)
        assert tsl.transpose_shard(t).as_tuple()[4:10] == sh.as_tuple()[4:10]


def test_no_rows():
    W = Weight("bf16", 64, 48, 1)
    sh = tsl.plan_linear(64, 48, 1, tsl.COLUMN)[0]
    X, dY = put(np.zeros((1, 64)), "bf16")[:0], put(np.zeros((1, 48)), "bf16")[:0]
    for wgk, order in (("f32", "kn"), ("bf16", "nk")):
        pt, nb = packed_t(W, sh)
        wb, dW, sk, sn = dw_out(64, 48, wgk, order)
        db = torch().full((48,), 7.0, device=DEV)
        base = put(np.zeros((1, 64)), "bf16")
        args = (sh, tsl.BF16, pt, nb, 0, base, 64, tsl.ACT_NONE, None, 0, base, 64, tsl.F32, None, 0,
                DT[wgk], dW, sk, sn)
        if wgk == "f32":
            tsl.shard_linear_grad(*args, 1, db)
            assert bool((dW == 7).all()) and bool((db == 7).all())
        tsl.shard_linear_grad(*args, 0, db)
        assert not bool(dW.any()) and not bool(db.any())
        assert untouched(wb, *((64, 48) if order == "kn" else (48, 64)))


def gated_grad(wk, Wg, Wu, sh, X, name, G, Uv, dH, xk="f32", wgk="f32", order="kn", acc=0, fill=7.0,
               want="xw"):
    M, K, N = dH.shape[0], sh.k_len, sh.n_len
    (pg, nb), (pu, _) = packed_t(Wg, sh), packed_t(Wu, sh)
    xb, dX = out(M, K, xk)
    gb, dg, sk, sn = dw_out(K, N, wgk, order, fill)
    ub, du, _, _ = dw_out(K, N, wgk, order, fill)
    n = tsl.shard_gated_grad_workspace_size(sh, sh, DT[wk], M)
    w = ws(n)
    w_ = "w" in want
    tsl.shard_gated_grad(sh, sh, DT[wk], pg, pu, nb, M, X, X.stride(0), ACTS[name], G, Uv,
                         G.stride(0), dH, dH.stride(0), DT[xk], dX if "x" in want else None,
                         dX.stride(0), DT[wgk], dg if w_ else None, du if w_ else None, sk, sn, acc,
                         w, n)
    assert untouched(xb, M, K)
    r, c = (K, N) if order == "kn" else (N, K)
    assert untouched(gb, r, c, fill) and untouched(ub, r, c, fill)
    return dX, dg, du


@pytest.mark.parametrize("M,K,N", SHAPES)
@pytest.mark.parametrize("wk,name,xk,wgk,order", [("bf16", "relu", "f32", "f32", "kn"),
                                                  ("bf16", "none", "bf16", "bf16", "nk"),
                                                  ("f32", "relu", "f32", "f32", "nk")])
def test_gated_exact(M, K, N, wk, name, xk, wgk, order):
    Wg, Wu = Weight(wk, K, N, M), Weight(wk, K, N, M + 1)
    sh = tsl.plan_linear(K, N, 1, tsl.COLUMN)[0]
    x, g, u, dh = ints(1, (M, K)), ints(2, (M, N)), ints(3, (M, N)), ints(4, (M, N))
    dX, dg, du = gated_grad(wk, Wg, Wu, sh, put(x, wk), name, put(g, wk), put(u, wk), put(dh, wk), xk,
                            wgk, order)
    a, d, _ = act(g, name)
    zg, zu = dh * u * d, dh * a
    assert np.array_equal(f64(dX), rne(zg @ Wg.w.T + zu @ Wu.w.T, xk))
    assert np.array_equal(f64(dg), rne(x.T @ zg, wgk))
    assert np.array_equal(f64(du), rne(x.T @ zu, wgk))


@pytest.mark.parametrize("name", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("wk,M,K,N", [("bf16", 9, 136, 72), ("bf16", 130, 136, 200), ("f32", 40, 64, 40)])
def test_gated_smooth(name, wk, M, K, N):
    Wg, Wu = Weight(wk, K, N, 5), Weight(wk, K, N, 6)
    sh = tsl.plan_linear(K, N, 1, tsl.COLUMN)[0]
    X, G, Uv, dH = (put(rng(s).standard_normal((M, c)) * k, wk)
                    for s, c, k in ((6, K, 1), (7, N, 2.5), (8, N, 1), (9, N, 1)))
    dX, dg, du = gated_grad(wk, Wg, Wu, sh, X, name, G, Uv, dH)
    x, g, u, dh = f64(X), f64(G), f64(Uv), f64(dH)
    a, d, _ = act(g, name)
    zg, zu = dh * u * d, dh * a
    h = HALF["bf16"] if wk == "bf16" else 0
    eg = (2.0 ** -16 + h) * np.abs(zg) + 2.0 ** -16 * 1.13 * np.abs(dh * u)
    eu = (2.0 ** -16 + h) * np.abs(zu)
    mag = np.abs(zg) @ np.abs(Wg.w.T) + np.abs(zu) @ np.abs(Wu.w.T)
    close(f64(dX), zg @ Wg.w.T + zu @ Wu.w.T,
          eg @ np.abs(Wg.w.T) + eu @ np.abs(Wu.w.T) + 2 * N * U * mag, "f32")
    for got, zz, ez in ((dg, zg, eg), (du, zu, eu)):
        close(f64(got), x.T @ zz, np.abs(x.T) @ ez + M * U * (np.abs(x.T) @ np.abs(zz)), "f32")


def test_gated_accumulates_and_parts():
    t = torch()
    M, K, N = 80, 128, 72
    Wg, Wu = Weight("bf16", K, N, 5), Weight("bf16", K, N, 6)
    sh = tsl.plan_linear(K, N, 1, tsl.COLUMN)[0]
    x, g, u, dh = ints(1, (M, K)), ints(2, (M, N)), ints(3, (M, N)), ints(4, (M, N))
    ops = (put(x, "bf16"), "none", put(g, "bf16"), put(u, "bf16"), put(dh, "bf16"))
    _, dg, du = gated_grad("bf16", Wg, Wu, sh, *ops, acc=1, fill=3.0)
    assert np.array_equal(f64(dg), 3 + x.T @ (dh * u)) and np.array_equal(f64(du), 3 + x.T @ (dh * g))
    full = gated_grad("bf16", Wg, Wu, sh, *ops)
    assert t.equal(gated_grad("bf16", Wg, Wu, sh, *ops, want="x")[0], full[0])
    assert t.equal(gated_grad("bf16", Wg, Wu, sh, *ops, want="w")[1], full[1])


@pytest.mark.parametrize("name", ["silu", "gelu", "gelu_tanh"])
def test_against_differences(name):
    """The binary32 form against central differences of the definition."""
    M, K, N, h = 4, 16, 12, 1e-5
    Wg, Wu = Weight("f32", K, N, 5, False), Weight("f32", K, N, 6, False)
    sh = tsl.plan_linear(K, N, 1, tsl.COLUMN)[0]
    x, dh = rng(1).standard_normal((M, K)).astype("f4"), rng(2).standard_normal((M, N)).astype("f4")
    x, dh = x.astype(float) * 20, dh.astype(float)
    x = x.astype("f4").astype(float)

    def loss(x, wg, wu):
        return np.sum(dh * act(x @ wg, name)[0] * (x @ wu))
    G, Uv = put(x @ Wg.w, "f32"), put(x @ Wu.w, "f32")
    dX, dg, du = gated_grad("f32", Wg, Wu, sh, put(x, "f32"), name, G, Uv, put(dh, "f32"))
    for got, k in ((dX, 0), (dg, 1), (du, 2)):
        for i, j in ((0, 0), (3, 5), (2, 11)):
            a = [x, Wg.w, Wu.w]
            e = np.zeros_like(a[k])
            e[i, j] = h
            lo, hi = list(a), list(a)
            lo[k], hi[k] = a[k] - e, a[k] + e
            d = (loss(*hi) - loss(*lo)) / (2 * h)
            assert abs(d - f64(got)[i, j]) <= 2e-5 * max(1.0, np.abs(f64(got)).max())


def test_repeat_gives_the_same_bits_and_replays():
    t = torch()
    M, K, N = 200, 256, 320
    Wg, Wu = Weight("bf16", K, N, 5, False), Weight("bf16", K, N, 6, False)
    sh = tsl.plan_linear(K, N, 1, tsl.COLUMN)[0]
    X, G, Uv, dH = (put(rng(s).standard_normal((M, c)), "bf16")
                    for s, c in ((6, K), (7, N), (8, N), (9, N)))
    (pg, nb), (pu, _) = packed_t(Wg, sh), packed_t(Wu, sh)
    (pw, wnb), W = packed_t(Wg, sh), None
    dX, dX2 = out(M, K, "bf16")[1], out(M, K, "bf16")[1]
    dg, du, dw = (out(K, N, "f32")[1] for _ in range(3))
    db = t.empty(N, device=DEV)
    n = tsl.shard_gated_grad_workspace_size(sh, sh, tsl.BF16, M)
    n2 = tsl.shard_linear_grad_workspace_size(sh, tsl.BF16, M)
    w, w2 = ws(n), ws(n2)

    def step():
        tsl.shard_gated_grad(sh, sh, tsl.BF16, pg, pu, nb, M, X, X.stride(0), tsl.ACT_SILU, G, Uv,
                             G.stride(0), dH, dH.stride(0), tsl.BF16, dX, dX.stride(0), tsl.F32, dg,
                             du, dg.stride(0), 1, 0, w, n)
        tsl.shard_linear_grad(sh, tsl.BF16, pw, wnb, M, dX, dX.stride(0), tsl.ACT_GELU, G,
                              G.stride(0), dH, dH.stride(0), tsl.BF16, dX2, dX2.stride(0), tsl.F32,
                              dw, dw.stride(0), 1, 0, db, w2, n2)
    outs = (dX, dX2, dg, du, dw, db)
    step()
    want = [v.clone() for v in outs]
    step()
    assert all(t.equal(a, b) for a, b in zip(outs, want))
    g, side = t.cuda.CUDAGraph(), t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    with t.cuda.graph(g, stream=side):
        step()
    for _ in range(3):
        for v in outs:
            v.zero_()
        g.replay()
        t.cuda.synchronize()
        assert all(t.equal(a, b) for a, b in zip(outs, want))
        step()
        t.cuda.synchronize()


@pytest.mark.parametrize("M", [1, 64, 65])
@pytest.mark.parametrize("acc", [0, 1])
def test_bias_gradient_alone(M, acc):
    """The sums of one and of several blocks of rows, with no product at all."""
    N = 100
    W = Weight("bf16", 64, N, 1)
    sh = tsl.plan_linear(64, N, 1, tsl.COLUMN)[0]
    dy = ints(2, (M, N))
    X = put(ints(1, (M, 64)), "bf16")
    db = linear_grad("bf16", W, sh, X, "none", None, put(dy, "bf16"), want="b", acc=acc, fill=5.0)[2]
    assert np.array_equal(f64(db), dy.sum(0) + 5 * acc)
