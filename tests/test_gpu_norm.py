"""add_rms_norm and its backward pass on the GPU against the definition in
binary64, over widths that take each register shape, odd widths and unaligned
rows, part counts, types, zero and non-finite rows, and in-place residuals.

Tolerances count roundings.  The library works in binary32 (half a step
u = 2^-24): the rank sum of R parts and a residual is off by at most R u of
the sum of its terms' magnitudes; rstd comes from n squares added in an order
of at most 64 adds per thread and 16 across, each u, halved by the square
root, so y is off by well under 64 u of itself plus the sum's error; the
stored type adds its own half step.
"""
import numpy as np
import pytest

from gpu_util import DEV, torch
from tensor_sharded_linear_plan_amd import binding as tsl

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "e4m3": 2.0 ** -4}
DT = {"f32": tsl.F32, "bf16": tsl.BF16, "e4m3": tsl.E4M3}


def tt(name):
    t = torch()
    return {"f32": t.float32, "bf16": t.bfloat16, "e4m3": t.float8_e4m3fn}[name]


def rows(m, n, kind, seed, std=1.0, ld=None, off=0):
    """[m][n] rows of `kind` at a stride of ld, starting `off` elements into
    their allocation; the padding holds NaN."""
    t = torch()
    ld = ld or n
    g = t.Generator().manual_seed(seed)
    buf = t.full((off + m * ld,), float("nan"))
    v = buf[off:].view(m, ld)
    v[:, :n] = t.randn((m, n), generator=g) * std
    return buf.to(tt(kind)).to(DEV)[off:].view(m, ld)[:, :n]


def blank(m, n, kind, ld=None, off=0):
    t = torch()
    ld = ld or n
    buf = t.full((off + m * ld + 8,), 3.0, device=DEV).to(tt(kind))
    return buf, buf[off:off + m * ld].view(m, ld)[:, :n]


def f64(x):
    return x.detach().cpu().double().numpy()


def norm_ref(parts, res, w, eps):
    r = sum(f64(p) for p in parts)
    mag = sum(np.abs(f64(p)) for p in parts)
    if res is not None:
        r, mag = r + f64(res), mag + np.abs(f64(res))
    rstd = 1 / np.sqrt(np.mean(r * r, axis=1, keepdims=True) + eps)
    y = r * rstd * (1 if w is None else f64(w))
    return r, mag, rstd, y


def run_norm(m, n, parts=2, pk="f32", rk="bf16", wk="bf16", yk="bf16", group=0, pad=0, off=0,
             res=True, keep=True, seed=1, eps=1e-6, edit=None):
    t = torch()
    ld = n + pad
    P = [rows(m, n, pk, seed + i, 0.7, ld, off) for i in range(parts)]
    R = rows(m, n, rk, seed + 90, 2.0, ld, off) if res else None
    W = (1 + 0.2 * rows(1, n, "f32", seed + 91)[0]).to(tt(wk)) if wk else None
    if edit:
        edit(P, R)
    sbuf, S = blank(m, n, rk, ld, off)
    ybuf, Y = blank(m, n, yk, ld, off)
    groups = -(-n // group) if group else 1
    sc = t.full((m, groups), -1.0, device=DEV) if yk == "e4m3" else None
    rs = t.full((m,), -1.0, device=DEV)
    ref = norm_ref(P, R, W, eps)
    tsl.add_rms_norm(P, DT[pk], ld, m, n, R, DT[rk], ld, S if keep else None, ld, W,
                     DT[wk] if wk else 0, eps, DT[yk], Y, ld, sc, group, rs)
    # nothing outside the rows is written
    for buf, v, k in ((sbuf, S, rk), (ybuf, Y, yk)):
        chk = buf.float()
        mask = t.zeros_like(chk, dtype=t.bool)
        mask[off:off + m * ld].view(m, ld)[:, :n] = True
        assert bool((chk[~mask] == 3.0).all())
    return ref, S, Y, sc, rs


def check_norm(out, yk, rk, group, terms, keep=True):
    (r, mag, rstd, y), S, Y, sc, rs = out
    esum = terms * U * mag                       # binary32 sum of `terms` values
    if keep:
        assert np.all(np.abs(f64(S) - r) <= esum + HALF[rk] * (np.abs(r) + esum) + 1e-40)
    rel = 64 * U                                 # rstd and the three products
    n = r.shape[1]
    # the sum's error also moves rstd: by at most its root-mean-square share
    drms = np.sqrt(np.mean(esum ** 2, axis=1, keepdims=True)) * rstd
    assert np.all(np.abs(f64(rs)[:, None] - rstd) <= (rel + drms) * rstd)
    wgt = np.abs(y) / np.maximum(np.abs(r), 1e-300)
    ey = np.abs(y) * (rel + drms) + esum * wgt
    if yk != "e4m3":
        assert np.all(np.abs(f64(Y) - y) <= ey + HALF[yk] * (np.abs(y) + ey) + 1e-40)
        return
    g = group or n
    s = f64(sc)
    for i in range(s.shape[1]):
        blk = slice(i * g, min(n, (i + 1) * g))
        top = np.abs(y[:, blk]).max(axis=1)
        et = ey[:, blk].max(axis=1)
        assert np.all(np.abs(s[:, i] - top / 448) <= et / 448 + 4 * U * top / 448)
        got = f64(Y.float())[:, blk] * s[:, i:i + 1]
        # half a step of e4m3; below 2^-6 (in units of s) the step is 2^-9
        step = np.maximum(HALF["e4m3"] * np.abs(y[:, blk]), 2.0 ** -10 * s[:, i:i + 1])
        assert np.all(np.abs(got - y[:, blk]) <= step * (1 + 1e-3) + 2 * ey[:, blk])


@pytest.mark.parametrize("m,n,pad,off", [(1, 3584, 0, 0), (3, 1, 0, 0), (5, 7, 1, 0), (2, 64, 8, 0),
                                         (6, 509, 3, 0), (4, 512, 0, 8), (3, 513, 7, 0),
                                         (2, 2049, 7, 0), (3, 4097, 0, 1), (2, 8192, 8, 0),
                                         (2, 8200, 0, 0), (1, 16385, 0, 0), (2, 32768, 0, 0),
                                         (513, 96, 0, 0)])
@pytest.mark.parametrize("yk,group", [("bf16", 0), ("f32", 0), ("e4m3", 0), ("e4m3", 64)])
def test_shapes(m, n, pad, off, yk, group):
    out = run_norm(m, n, parts=2, yk=yk, group=group, pad=pad, off=off, seed=n)
    check_norm(out, yk, "bf16", group, 3)


@pytest.mark.parametrize("parts", [1, 3, 8, 64])
@pytest.mark.parametrize("pk,rk,wk,res", [("f32", "f32", "f32", True), ("bf16", "bf16", None, True),
                                          ("bf16", "f32", "bf16", False)])
def test_parts_and_types(parts, pk, rk, wk, res):
    out = run_norm(4, 1000, parts=parts, pk=pk, rk=rk, wk=wk, yk="f32", res=res, seed=parts)
    check_norm(out, "f32", rk, 0, parts + 1)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("n", [128, 200, 2000])
def test_e4m3_groups(group, n):
    out = run_norm(7, n, yk="e4m3", group=group, seed=group + n)
    check_norm(out, "e4m3", "bf16", group, 3)


@pytest.mark.parametrize("yk,group", [("bf16", 0), ("e4m3", 0), ("e4m3", 32)])
def test_zero_rows(yk, group):
    """A row of zeros: r = 0, y = 0, rstd = eps^-1/2, scales 0."""
    def zero(P, R):
        for p in P:
            p[1] = 0
        R[1] = 0
    (r, mag, rstd, y), S, Y, sc, rs = run_norm(3, 96, yk=yk, group=group, edit=zero)
    assert not f64(S)[1].any() and not f64(Y.float())[1].any()
    assert abs(float(rs[1]) - 1e3) < 1e-2
    if sc is not None:
        assert not f64(sc)[1].any() and bool((sc[0] > 0).all())


def test_zero_row_eps_zero_is_nan_there_only():
    def zero(P, R):
        P[0][1] = 0
        P[1][1] = 0
        R[1] = 0
    (r, _, _, y), S, Y, _, _ = run_norm(3, 96, yk="f32", eps=0.0, edit=zero)
    assert np.isnan(f64(Y)[1]).all() and np.isfinite(f64(Y)[[0, 2]]).all()


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_non_finite_row(bad):
    """Only the row with the value is touched by it; its e4m3 codes are NaN."""
    def put(P, R):
        P[0][1, 5] = bad
    (r, _, _, y), S, Y, sc, rs = run_norm(3, 100, yk="e4m3", group=32, edit=put)
    got = f64(Y.float())
    assert np.isfinite(got[[0, 2]]).all() and np.isfinite(f64(sc)[[0, 2]]).all()
    # inf: rstd 0, so the inf's own y is NaN and its group's codes with it
    assert np.isnan(got[1, :32]).all() and not np.isfinite(f64(sc)[1, 0])


def test_tiny_values_keep_scales():
    """Row maxima near the smallest binary32 numbers: codes stay in range."""
    t = torch()
    w = t.full((64,), 1e-38, device=DEV)
    P = rows(2, 64, "f32", 3)
    Y = t.empty((2, 64), dtype=tt("e4m3"), device=DEV)
    sc = t.empty(2, device=DEV)
    tsl.add_rms_norm([P], tsl.F32, 64, 2, 64, None, tsl.F32, 0, None, 0, w, tsl.F32, 1e-6,
                     tsl.E4M3, Y, 64, sc, 0)
    assert bool((Y.float().abs().amax(1) == 448).all()) or bool((sc == 0).all())
    assert bool(t.isfinite(Y.float()).all())


def test_in_place_residual_and_repeat():
    t = torch()
    P = [rows(5, 640, "f32", 11 + i) for i in range(4)]
    R = rows(5, 640, "bf16", 20)
    keep = R.clone()
    Y1, Y2 = (t.empty((5, 640), dtype=t.bfloat16, device=DEV) for _ in range(2))
    S = t.empty_like(R)
    args = (P, tsl.F32, 640, 5, 640)
    tsl.add_rms_norm(*args, R, tsl.BF16, 640, S, 640, None, 0, 1e-5, tsl.BF16, Y1, 640)
    tsl.add_rms_norm(*args, R, tsl.BF16, 640, R, 640, None, 0, 1e-5, tsl.BF16, Y2, 640)
    assert t.equal(R, S) and t.equal(Y1, Y2) and not t.equal(R, keep)


def test_row_offsets_past_4_gib():
    """Rows whose byte offsets need more than 32 bits (a stride of 2^29 elements)."""
    t = torch()
    ld, m, n = 1 << 29, 5, 128
    buf = t.empty(4 * ld + n, dtype=t.bfloat16, device=DEV)
    v = t.as_strided(buf, (m, n), (ld, 1))
    src = rows(m, n, "bf16", 5)
    v.copy_(src)
    Y1, Y2 = (t.empty((m, n), dtype=t.float32, device=DEV) for _ in range(2))
    for x, l, y in ((v, ld, Y1), (src, n, Y2)):
        tsl.add_rms_norm([x], tsl.BF16, l, m, n, None, tsl.F32, 0, None, 0, None, 0, 1e-6,
                         tsl.F32, y, n)
    assert t.equal(Y1, Y2)


# ---- backward ------------------------------------------------------------------

def grad_ref(x, dy, w, rstd, dres):
    t = dy * w
    xh = x * rstd
    dx = rstd * (t - xh * np.mean(t * xh, axis=1, keepdims=True))
    return dx + (0 if dres is None else dres), np.sum(dy * xh, axis=0)


@pytest.mark.parametrize("m,n,pad,off", [(1, 3584, 0, 0), (3, 1, 0, 0), (9, 77, 3, 0),
                                         (4100, 64, 0, 0), (1030, 520, 0, 0), (5, 2056, 0, 0),
                                         (7, 8191, 1, 1), (2, 16000, 0, 0), (2, 32768, 0, 0)])
@pytest.mark.parametrize("kind,dres,rs", [("bf16", True, True), ("f32", False, False)])
def test_grad(m, n, pad, off, kind, dres, rs):
    t = torch()
    ld, eps = n + pad, 1e-5
    x, dy = rows(m, n, kind, 31, 2.0, ld, off), rows(m, n, kind, 32, 1.0, ld, off)
    W = (1 + 0.2 * rows(1, n, "f32", 33)[0]).to(tt(kind))
    D = rows(m, n, kind, 34, 1.0, ld, off) if dres else None
    r64 = 1 / np.sqrt(np.mean(f64(x) ** 2, axis=1, keepdims=True) + eps)
    rstd = t.from_numpy(r64[:, 0].astype(np.float32)).to(DEV) if rs else None
    if rs:
        r64 = r64.astype(np.float32).astype(np.float64)
    buf, dx = blank(m, n, kind, ld, off)
    nws = tsl.add_rms_norm_grad_workspace_size(m, n)
    ws = t.empty(max(nws, 256), dtype=t.uint8, device=DEV)
    got = []
    for acc in (0, 1, 0):
        dw = t.full((n,), 2.0, device=DEV)
        tsl.add_rms_norm_grad(m, n, dy, DT[kind], ld, x, DT[kind], ld, W, DT[kind], eps, rstd, D,
                              ld, dx, DT[kind], ld, dw, acc, ws, nws)
        got.append(dw.clone())
    assert t.equal(got[0], got[2])  # the same bits again
    X, DY, w = f64(x), f64(dy), f64(W)
    want, dwant = grad_ref(X, DY, w, r64, None if D is None else f64(D))
    # binary32: every term within a few u of the largest thing added, plus the
    # mean's n adds (at most 64 in a row)
    mag = r64 * (np.abs(DY * w) + np.abs(X * r64) * np.mean(np.abs(DY * w * X * r64), axis=1,
                                                            keepdims=True))
    tol = 80 * U * mag + 2 * U * np.abs(want)
    assert np.all(np.abs(f64(dx) - want) <= tol + HALF[kind] * (np.abs(want) + tol) + 1e-40)
    # dw: at most m/groups adds per row group and groups/16 + 16 after that
    tolw = (64 + m / 64) * U * np.sum(np.abs(DY * X * r64), axis=0)
    assert np.all(np.abs(f64(got[0]) - dwant) <= tolw + 1e-40)
    assert np.all(np.abs(f64(got[1]) - (dwant + 2)) <= tolw + 4 * U * (np.abs(dwant) + 2))


def test_grad_against_differences():
    """Central differences of the forward definition in binary64."""
    t = torch()
    m, n, eps, h = 3, 24, 1e-3, 1e-5
    x, dy, w = rows(m, n, "f32", 51), rows(m, n, "f32", 52), rows(1, n, "f32", 53)[0]
    dx, dw = t.empty((m, n), device=DEV), t.empty(n, device=DEV)
    nws = tsl.add_rms_norm_grad_workspace_size(m, n)
    ws = t.empty(max(nws, 256), dtype=t.uint8, device=DEV)
    tsl.add_rms_norm_grad(m, n, dy, tsl.F32, n, x, tsl.F32, n, w, tsl.F32, eps, None, None, 0, dx,
                          tsl.F32, n, dw, 0, ws, nws)
    X, W, DY = f64(x), f64(w), f64(dy)

    def loss(a, b):
        return np.sum(DY * a / np.sqrt(np.mean(a * a, axis=1, keepdims=True) + eps) * b)
    for i, j in ((0, 0), (1, 7), (2, 23)):
        e = np.zeros_like(X)
        e[i, j] = h
        d = (loss(X + e, W) - loss(X - e, W)) / (2 * h)
        assert abs(d - f64(dx)[i, j]) < 1e-5 * (1 + abs(d))
        ew = np.zeros_like(W)
        ew[j] = h
        d = (loss(X, W + ew) - loss(X, W - ew)) / (2 * h)
        assert abs(d - f64(dw)[j]) < 1e-5 * (1 + abs(d))


def test_grad_no_rows_and_parts_of_it():
    t = torch()
    x = rows(4, 40, "bf16", 61)
    dw = t.full((40,), 5.0, device=DEV)
    tsl.add_rms_norm_grad(0, 40, x, tsl.BF16, 40, x, tsl.BF16, 40, None, 0, 1e-6, None, None, 0,
                          None, 0, 0, dw, 0, None, 0)
    assert not bool(dw.any())
    a, b = t.empty((4, 40), device=DEV), t.empty((4, 40), device=DEV)
    nws = tsl.add_rms_norm_grad_workspace_size(4, 40)
    ws = t.empty(max(nws, 256), dtype=t.uint8, device=DEV)
    dy = rows(4, 40, "bf16", 62)
    args = (4, 40, dy, tsl.BF16, 40, x, tsl.BF16, 40, None, 0, 1e-6, None)
    tsl.add_rms_norm_grad(*args, None, 0, a, tsl.F32, 40, None)
    tsl.add_rms_norm_grad(*args, None, 0, b, tsl.F32, 40, dw, 0, ws, nws)
    assert t.equal(a, b)
    # dres may be dX itself
    c = rows(4, 40, "f32", 63)
    want, apart = a + c, t.empty((4, 40), device=DEV)
    tsl.add_rms_norm_grad(*args, c, 40, apart, tsl.F32, 40, None)
    tsl.add_rms_norm_grad(*args, c, 40, c, tsl.F32, 40, None)
    assert t.equal(c, apart)
    # the last product and the addition of dres are one fused multiply-add,
    # rounded once: with p the exact product, c = p + dres within u |c|, while
    # `want` rounds p first (u |a|) and the sum after it (u |want|)
    assert bool(((c - want).abs() <= U * (a.abs() + 2.001 * want.abs())).all())


def test_graph_and_streams():
    """Captured and replayed with eager calls in between, on a side stream."""
    t = torch()
    m, n = 33, 1024
    P = [rows(m, n, "f32", 70 + i) for i in range(2)]
    R = rows(m, n, "bf16", 75)
    S, Y = (t.empty((m, n), dtype=t.bfloat16, device=DEV) for _ in range(2))
    rs, dx = t.empty(m, device=DEV), t.empty((m, n), dtype=t.bfloat16, device=DEV)
    dw = t.empty(n, device=DEV)
    nws = tsl.add_rms_norm_grad_workspace_size(m, n)
    ws = t.empty(max(nws, 256), dtype=t.uint8, device=DEV)

    def step():
        tsl.add_rms_norm(P, tsl.F32, n, m, n, R, tsl.BF16, n, S, n, None, 0, 1e-6, tsl.BF16, Y, n,
                         None, 0, rs)
        tsl.add_rms_norm_grad(m, n, Y, tsl.BF16, n, S, tsl.BF16, n, None, 0, 1e-6, rs, R, n, dx,
                              tsl.BF16, n, dw, 0, ws, nws)
    step()
    want = [v.clone() for v in (S, Y, rs, dx, dw)]
    g = t.cuda.CUDAGraph()
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    with t.cuda.graph(g, stream=side):
        step()
    for k in range(3):
        for v in (S, Y, rs, dx, dw):
            v.zero_()
        g.replay()
        t.cuda.synchronize()
        assert all(t.equal(a, b) for a, b in zip((S, Y, rs, dx, dw), want)), k
        step()
        t.cuda.synchronize()
