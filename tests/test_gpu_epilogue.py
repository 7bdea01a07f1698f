"""shard_linear_group_epilogue on the GPU: act(X W + bias) + residual against
the formula in binary64.  Inputs are small integers (weights times a power of
two), so X W + bias is exact in every kernel's arithmetic and the kept
pre-activation must match bit for bit; what is left is the activation's error
(block_util.act), the addition's and the stored type's rounding.  Random
values and the binary16 path's rounding are checked by their mean square."""
import numpy as np
import pytest

from block_util import (ACTS, DT, U, Weight, act, close, f64, ints, out, put, rne, rng, tt,
                        untouched, ws)
from gpu_util import DEV, torch
from tensor_sharded_linear_plan_amd import binding as tsl

pytestmark = pytest.mark.gpu


def xkind(wk):
    return "f32" if wk == "f32" else "bf16"


def problem(wk, M, K, N, tp=1, seed=1, exact=True, x=None):
    """X, the ROW shards of W over tp ranks, their packed copies."""
    W = Weight(wk, K, N, seed, exact)
    x = ints(seed + 1, (M, K)) if x is None else x
    X = put(x, xkind(wk))
    shards = tsl.plan_linear(K, N, tp, tsl.ROW, 64 if wk == "q4" else 0)
    items = []
    for r, sh in enumerate(shards):
        buf, nb = W.pack(sh)
        items.append(dict(shard=sh, packed=buf, packed_bytes=nb, X=X[:, sh.k_off:],
                          ldx=X.stride(0), sum_next=int(r + 1 < tp)))
    return W, X, items


def run(items, eps, wk, M, **kw):
    n = tsl.shard_linear_group_epilogue_workspace_size(items, eps, DT[wk], M)
    w = ws(n)
    tsl.shard_linear_group_epilogue(items, eps, DT[wk], DT[xkind(wk)], M, w, n, **kw)
    return w


def epilogue(M, N, name, bk=None, rk=None, pk=None, seed=50):
    """(epilogue dict, its bias, residual and kept pre-activation buffers)."""
    e = dict(act=ACTS[name])
    b = r = p = pbuf = None
    if bk:
        b = put(ints(seed, (1, N), -9, 9) * 2.0 ** -3, bk)[0]
        e.update(bias=b, bias_dtype=DT[bk])
    if rk:
        r = put(rng(seed + 1).standard_normal((M, N)), rk)
        e.update(residual=r, res_dtype=DT[rk], ld_res=r.stride(0))
    if pk:
        pbuf, p = out(M, N, pk)
        e.update(pre=p, pre_dtype=DT[pk], ld_pre=p.stride(0))
    return e, b, r, p, pbuf


def check(Y, p, x, w, b, r, name, yk, pk):
    z = x @ w + (0 if b is None else f64(b))
    if p is not None:
        assert np.array_equal(f64(p), rne(z, pk))
    v, _, err = act(z, name)
    if r is not None:
        v = v + f64(r)
        err = err + U * np.abs(v)
    close(f64(Y), v, err, yk)


# every kernel family: fp32, streaming (resident and windowed, k split or
# not), the GEMMs over full, ragged and split tiles
CASES = [("f32", 1, 192, 40, 1), ("f32", 33, 100, 33, 1), ("f32", 7, 1024, 17, 2),
         ("bf16", 1, 256, 40, 1), ("bf16", 3, 2048, 513, 1), ("bf16", 5, 1000, 260, 1),
         ("bf16", 17, 640, 1100, 1), ("bf16", 32, 512, 64, 2), ("bf16", 33, 128, 70, 1),
         ("bf16", 65, 1000, 257, 1), ("bf16", 130, 4096, 96, 1), ("bf16", 300, 256, 1031, 1),
         ("bf16", 200, 512, 320, 4), ("bf16", 1, 2048, 4112, 8), ("bf16", 40, 80, 8, 1),
         ("q4", 1, 256, 40, 1), ("q4", 2, 4096, 700, 1), ("q4", 1, 4736, 513, 1),
         ("q4", 16, 1024, 260, 1), ("q4", 40, 512, 1000, 2), ("q4", 64, 192, 65, 1),
         ("q4", 65, 128, 33, 1), ("q4", 130, 2048, 300, 1), ("q4", 257, 512, 1031, 1),
         ("q4", 100, 1024, 520, 4), ("q4", 70, 640, 100, 2), ("q4", 4, 4096, 1024, 4)]


@pytest.mark.parametrize("wk,M,K,N,tp", CASES)
@pytest.mark.parametrize("name,bk,rk,pk,yk", [("none", "bf16", "bf16", None, "bf16"),
                                              ("silu", None, None, "f32", "f32"),
                                              ("gelu", "f32", None, "bf16", "bf16")])
def test_against_formula(wk, M, K, N, tp, name, bk, rk, pk, yk):
    W, X, items = problem(wk, M, K, N, tp, seed=K + N)
    e, b, r, p, pbuf = epilogue(M, N, name, bk, rk, pk)
    ybuf, Y = out(M, N, yk)
    items[0].update(Y=Y, ldy=Y.stride(0), ydtype=DT[yk])
    run(items, [e] + [None] * (tp - 1), wk, M)
    check(Y, p, f64(X), W.w, b, r, name, yk, pk)
    assert untouched(ybuf, M, N) and (pbuf is None or untouched(pbuf, M, N))


@pytest.mark.parametrize("name", list(ACTS))
@pytest.mark.parametrize("wk,M", [("f32", 5), ("bf16", 2), ("bf16", 20), ("bf16", 70), ("q4", 1),
                                  ("q4", 30), ("q4", 90)])
def test_activations_and_residuals(wk, M, name):
    K, N = 128, 144
    W, X, items = problem(wk, M, K, N, seed=9)
    for rk, yk in (("f32", "bf16"), ("bf16", "f32"), ("f32", "f32")):
        e, b, r, p, _ = epilogue(M, N, name, "bf16", rk, "f32")
        Y = out(M, N, yk)[1]
        items[0].update(Y=Y, ldy=Y.stride(0), ydtype=DT[yk])
        run(items, [e], wk, M)
        check(Y, p, f64(X), W.w, b, r, name, yk, "f32")


@pytest.mark.parametrize("wk,M,tp", [("f32", 4, 1), ("bf16", 2, 1), ("bf16", 20, 2), ("bf16", 80, 2),
                                     ("q4", 1, 4), ("q4", 50, 1), ("q4", 100, 2), ("q4", 3, 16),
                                     ("bf16", 70, 16)])
def test_residual_in_place(wk, M, tp):
    """The residual stream updated in place: Y is the residual.  16 ranks are
    more than one sum launch or joined product takes."""
    K, N = 1024, 200
    W, X, items = problem(wk, M, K, N, tp, seed=21)
    for k in ("bf16", "f32"):
        e, b, r, p, _ = epilogue(M, N, "none", "f32", k, None)
        apart = out(M, N, k)[1]
        items[0].update(Y=apart, ldy=apart.stride(0), ydtype=DT[k])
        run(items, [e] + [None] * (tp - 1), wk, M)
        check(apart, None, f64(X), W.w, b, r, "none", k, None)
        items[0].update(Y=r, ldy=r.stride(0))
        run(items, [e] + [None] * (tp - 1), wk, M)
        assert torch().equal(r, apart)


@pytest.mark.parametrize("wk,M", [("bf16", 3), ("bf16", 64), ("q4", 2), ("q4", 20), ("q4", 128)])
def test_random_values(wk, M):
    """Random weights and activations: the mean square error against the
    product's own spread sqrt(sum (x w)^2).  binary32 accumulation: far below
    2^-14 of it; binary16 operands (4-bit weights above 64 rows) round each
    factor by at most 2^-11, independently: below 2^-11 sqrt(2 / 3)."""
    K, N = 1536, 333
    x = rng(5).standard_normal((M, K))
    W, X, items = problem(wk, M, K, N, seed=33, exact=False, x=x)
    Y = out(M, N, "f32")[1]
    items[0].update(Y=Y, ldy=Y.stride(0), ydtype=tsl.F32)
    run(items, [dict(act=tsl.ACT_NONE)], wk, M)
    want = f64(X) @ W.w
    spread = np.sqrt((f64(X) ** 2) @ (W.w ** 2))
    e = np.sqrt(np.mean(((f64(Y) - want) / spread) ** 2))
    assert e < (2.0 ** -11 * np.sqrt(2 / 3) if wk == "q4" and M > 64 else 2.0 ** -14)


@pytest.mark.parametrize("wk,M", [("f32", 6), ("bf16", 4), ("bf16", 24), ("bf16", 90), ("q4", 3),
                                  ("q4", 30), ("q4", 100)])
def test_group_of_mixed_items(wk, M):
    """Items with, without and with other epilogues, own row counts and rows
    read through an index, in one call."""
    t = torch()
    K, rows = 256, [M, 1, (M + 1) // 2, M]
    Ns = [96, 33, 200, 96]
    x = ints(3, (M, K))
    X = put(x, xkind(wk))
    idx = rng(4).integers(-1, M + 1, size=rows[2]).astype(np.int32)  # -1 and M read zeros
    dix = t.from_numpy(idx).to(DEV)
    items, eps, checks = [], [], []
    for i, N in enumerate(Ns):
        W = Weight(wk, K, N, 60 + i)
        sh = tsl.plan_linear(K, N, 1, tsl.COLUMN, 64 if wk == "q4" else 0)[0]
        buf, nb = W.pack(sh)
        e, b, r, p, _ = epilogue(rows[i], N, ["gelu", "none", "silu", "relu"][i],
                                 "bf16" if i != 1 else None, "bf16" if i == 2 else None, "f32",
                                 seed=70 + i)
        ybuf, Y = out(rows[i], N, "bf16")
        items.append(dict(shard=sh, packed=buf, packed_bytes=nb, X=X, ldx=X.stride(0), Y=Y,
                          ldy=Y.stride(0), ydtype=tsl.BF16, rows=rows[i],
                          row_index=dix if i == 2 else None, x_rows=M if i == 2 else 0))
        eps.append(e if i != 1 else None)
        xi = x[:rows[i]] if i != 2 else np.where(((idx >= 0) & (idx < M))[:, None],
                                                 x[np.clip(idx, 0, M - 1)], 0)
        checks.append((Y, p if i != 1 else None, xi, W.w, b, r,
                       ["gelu", "none", "silu", "relu"][i], ybuf, rows[i], N))
    run(items, eps, wk, M)
    for Y, p, xi, w, b, r, name, ybuf, m, n in checks:
        check(Y, p, xi, w, b, r, name, "bf16", "f32")
        assert untouched(ybuf, m, n)


def test_many_items_past_one_launch():
    """More items than one launch's table holds (300 in the GEMM regime, 300
    streamed), every one with a bias of its own."""
    t = torch()
    K, N = 128, 32
    for wk, M in (("q4", 70), ("bf16", 36), ("q4", 2), ("bf16", 2)):
        W = Weight(wk, K, N, 80)
        X = put(ints(81, (M, K)), "bf16")
        sh = tsl.plan_linear(K, N, 1, tsl.COLUMN, 64 if wk == "q4" else 0)[0]
        buf, nb = W.pack(sh)
        bias = t.arange(300 * N, device=DEV, dtype=t.float32).view(300, N) / 16
        Y = t.zeros((300, M, N), device=DEV)
        items = [dict(shard=sh, packed=buf, packed_bytes=nb, X=X, ldx=X.stride(0), Y=Y[i], ldy=N,
                      ydtype=tsl.F32) for i in range(300)]
        run(items, [dict(bias=bias[i], act=tsl.ACT_RELU) for i in range(300)], wk, M)
        want = np.maximum((f64(X) @ W.w)[None] + f64(bias)[:, None, :], 0)
        assert np.array_equal(f64(Y), want), (wk, M)


@pytest.mark.parametrize("wk,M", [("q4", 1), ("q4", 70), ("bf16", 3), ("bf16", 40), ("f32", 3)])
def test_infinities_stay_in_their_rows(wk, M):
    """An infinite residual or activation reaches its own outputs only."""
    K, N = 128, 64
    W, X, items = problem(wk, M, K, N, seed=91)
    r = put(np.zeros((M, N)), "f32")
    r[0, 5] = float("inf")
    Y = out(M, N, "f32")[1]
    items[0].update(Y=Y, ldy=Y.stride(0), ydtype=tsl.F32)
    run(items, [dict(residual=r, res_dtype=tsl.F32, ld_res=r.stride(0), act=tsl.ACT_SILU)], wk, M)
    got = f64(Y)
    assert np.isinf(got[0, 5])
    got[0, 5] = 0
    assert np.isfinite(got).all()


def test_same_as_plain_group_without_epilogues():
    """All-null epilogues: the products of shard_linear_group, bit for bit."""
    t = torch()
    for wk, M in (("q4", 1), ("q4", 33), ("q4", 200), ("bf16", 2), ("bf16", 100), ("f32", 9)):
        x = rng(7).standard_normal((M, 512))
        W, X, items = problem(wk, M, 512, 300, 2, seed=5, exact=False, x=x)
        got = []
        for f in ("plain", "epilogue"):
            Y = out(M, 300, "bf16")[1]
            items[0].update(Y=Y, ldy=Y.stride(0), ydtype=tsl.BF16)
            if f == "plain":
                n = tsl.shard_linear_group_workspace_size(items, DT[wk], M)
                tsl.shard_linear_group(items, DT[wk], DT[xkind(wk)], M, ws(n), n)
            else:
                run(items, [None, None], wk, M)
            got.append(Y)
        assert t.equal(*got), (wk, M)


@pytest.mark.parametrize("wk,M,tp", [("q4", 1, 2), ("q4", 4, 4), ("q4", 80, 2), ("bf16", 1, 1),
                                     ("bf16", 16, 1), ("bf16", 48, 2), ("f32", 5, 1)])
def test_captured_and_replayed(wk, M, tp):
    t = torch()
    K, N = 2048, 272
    W, X, items = problem(wk, M, K, N, tp, seed=13)
    e, b, r, p, _ = epilogue(M, N, "silu", "bf16", "bf16", "bf16")
    Y = out(M, N, "bf16")[1]
    items[0].update(Y=Y, ldy=Y.stride(0), ydtype=tsl.BF16)
    eps = [e] + [None] * (tp - 1)
    keep = run(items, eps, wk, M)
    want = Y.clone()
    n = tsl.shard_linear_group_epilogue_workspace_size(items, eps, DT[wk], M)
    g, side = t.cuda.CUDAGraph(), t.cuda.Stream()
    own = ws(n)
    side.wait_stream(t.cuda.current_stream())
    with t.cuda.graph(g, stream=side):
        tsl.shard_linear_group_epilogue(items, eps, DT[wk], DT[xkind(wk)], M, own, n)
    for _ in range(3):
        Y.zero_()
        g.replay()
        t.cuda.synchronize()
        assert t.equal(Y, want)
        run(items, eps, wk, M)
        t.cuda.synchronize()
    del keep


@pytest.mark.parametrize("wk,M,T", [("f32", 4, 3), ("bf16", 5, 9), ("bf16", 20, 50), ("bf16", 70, 40),
                                    ("q4", 3, 7), ("q4", 30, 9), ("q4", 66, 200)])
def test_sum_set_read_through_row_indices(wk, M, T):
    """The members of a set read different rows of different matrices."""
    t = torch()
    K, N = 256, 72
    e, b, r, p, _ = epilogue(M, N, "silu", "f32", "f32", "f32")
    Y = out(M, N, "f32")[1]
    items, want = [], f64(b)[None, :]
    for i in range(2):
        W = Weight(wk, K, N, 140 + i)
        x = ints(150 + i, (T, K))
        idx = rng(160 + i).integers(-1, T + 1, size=M).astype(np.int32)
        sh = tsl.plan_linear(K, N, 1, tsl.ROW, 64 if wk == "q4" else 0)[0]
        buf, nb = W.pack(sh)
        X = put(x, xkind(wk))
        items.append(dict(shard=sh, packed=buf, packed_bytes=nb, X=X, ldx=X.stride(0), Y=Y,
                          ldy=Y.stride(0), ydtype=tsl.F32, sum_next=1 - i,
                          row_index=t.from_numpy(idx).to(DEV), x_rows=T))
        want = want + np.where(((idx >= 0) & (idx < T))[:, None], x[np.clip(idx, 0, T - 1)], 0) @ W.w
    run(items, [e, None], wk, M)
    assert np.array_equal(f64(p), want)
    v, _, err = act(want, "silu")
    close(f64(Y), v + f64(r), err + U * np.abs(v + f64(r)), "f32")


@pytest.mark.parametrize("wk,M", [("f32", 3), ("bf16", 4), ("bf16", 40), ("q4", 4), ("q4", 70)])
def test_accumulating_items_beside_epilogues(wk, M):
    """A plain accumulating product and one with an epilogue in one call, in
    the workspace the size query asks for."""
    K, N = 1024, 96
    W, X, (a,) = problem(wk, M, K, N, seed=171)
    Y1, Y2 = out(M, N, "f32", fill=2.0)[1], out(M, N, "f32")[1]
    items = [dict(a, Y=Y1, ldy=Y1.stride(0), ydtype=tsl.F32, accumulate=1),
             dict(a, Y=Y2, ldy=Y2.stride(0), ydtype=tsl.F32)]
    run(items, [None, dict(act=tsl.ACT_RELU)], wk, M)
    z = f64(X) @ W.w
    assert np.array_equal(f64(Y1), z + 2) and np.array_equal(f64(Y2), np.maximum(z, 0))
