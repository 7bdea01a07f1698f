"""cache_attention on the GPU against its definition in binary64 over the values
that the cache holds.

Tolerance, u = 2^-24, w = 2^-11 (half a step of binary16; operands of sequences
of more than `FEW` query rows a K/V head are rounded to it, others enter exactly).  With
a = sum |q| over a run of 64, the logit's terms s (128 + c) q and 128 s q are
bounded by 271 |s| a and b q by |b| a; a sum of n terms is off by at most n u of
their magnitudes, n = 72, so the logit by
    e = scale sum_runs (72 u (271 |s| + |b|) a) [+ scale 2 w sum |q| |k|],
and the logit's products with scale and its exponential's by 8 u (|x| + 2).
A probability is off by the factor exp(+-e), the quotient by exp(2 e); the
weighted sum over n tokens by (n + 8) u of sum p (271 |s| + |b|) [and 2 w of
sum p |v|].  The result is then rounded once."""
import numpy as np
import pytest

import attn_util as au
from gpu_util import DEV, torch
from tensor_sharded_linear_plan_amd import binding as tsl

pytestmark = pytest.mark.gpu

W16 = 2.0 ** -11
FEW = 64


@pytest.fixture(params=[False, True], ids=["", "roomy"], autouse=True)
def roomy(request, monkeypatch):
    """Every test twice: with page tables of the sizes in use, and as wide as for long
    contexts, by which records of prompts are expanded once for all tiles."""
    monkeypatch.setitem(globals(), "ROOMY", request.param)


def widened(pages, batch, d):
    t = torch()
    w = max(2200 * 32 // (pages.page_tokens * pages.heads), 1) + batch.table.shape[1]
    table = t.full((max(len(batch.n), 1), w), -1, dtype=t.int32, device=DEV)
    table[:len(batch.n), :batch.max_pages] = d["page_table"][:, :batch.max_pages]
    d.update(page_table=table, ld_table=w, max_pages=w, max_context=w * pages.page_tokens)


def run(pages, batch, hq, q, scale, window=0, sinks=0, okind="bf16", pad=0, head_major=False,
        stream=None, **kw):
    Q = q if isinstance(q, au.Operand) else au.Operand(batch.rows, hq, pages.d, "bf16", pad,
                                                       head_major, values=q)
    O = au.Operand(batch.rows, hq, pages.d, okind, pad, head_major)
    d = batch.dict(**kw)
    if ROOMY and not kw:
        widened(pages, batch, d)
    n = tsl.cache_attention_workspace_size(pages.dict, d, hq, window, sinks)
    ws = torch().full((n + 256,), 0xFF, dtype=torch().uint8, device=DEV) if n else None
    tsl.cache_attention(pages.dict, d, hq, Q.view, Q.ld, Q.head, scale, window, sinks, au.DT[okind],
                        O.view, O.ld, O.head, ws, n, stream)
    if n:
        assert bool((ws[n:] == 0xFF).all())
    return Q, O


def bounds(q, k, v, ks, vs, scale, mag, rounded):
    """The error bound of the module's docstring for one sequence: [n][hq][d]."""
    n, hq, d = q.shape
    ctx, h, _ = k.shape
    g, runs = hq // h, d // 64
    err = np.zeros_like(mag)
    for x in range(hq):
        a = np.abs(q[:, x]).reshape(n, runs, 64).sum(-1)
        s, b = (np.abs(np.nan_to_num(t[:, x // g])) for t in ks)
        kk = np.abs(np.nan_to_num(k[:, x // g]))
        logit = abs(scale) * (np.abs(q[:, x]) @ kk.T)
        e = abs(scale) * 72 * au.U * (a @ (271 * s + b).T) + 8 * au.U * (logit + 2)
        if rounded:
            e = e + 2 * W16 * logit
        e = e.max(1, initial=0)[:, None]
        s, b = (np.abs(np.nan_to_num(t[:, x // g])) for t in vs)
        big = np.repeat((271 * s + b).max(0, initial=0), 64, -1)[None]
        err[:, x] = np.expm1(2 * e) * mag[:, x] + (ctx + 8) * au.U * big
        if rounded:
            err[:, x] += (2 * W16 + 4 * au.U * ctx) * mag[:, x]
    return err


def check(O, Q, batch, K, V, hq, scale, window, sinks, okind, rounded):
    q, got = Q.get(), O.get()
    at = 0
    worst = 0.0
    for s, (n, c) in enumerate(zip(batch.n, batch.ctx)):
        row = int(batch.start[s])
        k, v = K[at:at + c], V[at:at + c]
        (_, *ks), (_, *vs) = au.quantise(k), au.quantise(v)
        want, mag = au.attend(q[row:row + n], au.held(k), au.held(v), scale, window, sinks, c - n)
        err = bounds(q[row:row + n], au.held(k), au.held(v), ks, vs, scale, mag, rounded)
        g = got[row:row + n]
        au.within(g, want, err + au.HALF[okind] * (np.abs(want) + err) + 1e-38, s)
        if n:
            nd, nw = np.linalg.norm(np.nan_to_num(g - want)), np.linalg.norm(np.nan_to_num(want))
            worst = max(worst, nd / nw if nw else 0.0)
        at += c
    live = list(batch.live())
    assert O.rest_untouched(live)
    # all outputs together: roundings are independent, so their norm is that of
    # one half step a value at most, and what the operands add stays below it
    assert worst <= au.HALF[okind] + (2 * W16 if rounded else 2.0 ** -12), worst


def data(batch, heads, d, hq, seed, kscale=1.0):
    r = au.rng(seed)
    n = sum(max(c, 0) for c in batch.ctx)
    K = au.rne((r.standard_normal((n, heads, d)) + r.standard_normal((1, heads, d))) * kscale, "bf16")
    V = au.rne(r.standard_normal((n, heads, d)) * r.uniform(0.3, 1.5, (n, 1, 1)), "bf16")
    q = r.standard_normal((batch.rows, hq, d))
    return K, V, q


CASES = [
    # d, hq, hkv, page, rows, contexts, window, sinks, out, pad, head-major
    (128, 28, 4, 64, [1], [1], 0, 0, "bf16", 0, False),
    (128, 28, 4, 64, [1], [1000], 0, 0, "f32", 0, False),
    (128, 8, 8, 32, [1, 1, 1, 1, 1], [31, 32, 33, 1, 257], 0, 0, "bf16", 1, False),
    (64, 32, 8, 32, [1, 1, 0, 1], [700, 65, 9, 40], 0, 0, "f32", 0, False),
    (256, 4, 2, 64, [1, 2], [100, 333], 0, 0, "bf16", 0, True),
    (128, 7, 1, 128, [3, 5, 1], [3, 129, 400], 0, 0, "bf16", 0, True),
    (64, 5, 1, 256, [4], [2100], 0, 0, "f32", 1, False),
    (128, 16, 2, 64, [1, 1, 2], [500, 90, 301], 64, 0, "bf16", 0, False),
    (128, 16, 2, 64, [1, 1, 2], [500, 90, 301], 100, 4, "f32", 0, False),
    (64, 8, 8, 32, [1, 3], [2000, 60], 1, 0, "bf16", 0, False),
    (64, 8, 8, 32, [1, 3], [2000, 60], 33, 70, "f32", 0, False),
    (128, 64, 1, 64, [1], [300], 0, 0, "bf16", 0, False),
]


@pytest.mark.parametrize("d,hq,hkv,page,rows,ctx,window,sinks,okind,pad,hm", CASES)
def test_attend_few_rows(d, hq, hkv, page, rows, ctx, window, sinks, okind, pad, hm):
    b = au.Batch(rows, ctx, page, seed=d + hq, lead=1, tail=2)
    pages = au.Pages(b.n_pages, page, hkv, d)
    K, V, q = data(b, hkv, d, hq, d + hq + page)
    au.fill(pages, b, K, V)
    Q, O = run(pages, b, hq, q, d ** -0.5, window, sinks, okind, pad, hm)
    check(O, Q, b, K, V, hq, d ** -0.5, window, sinks, okind, d < 256 and max(rows) * hq // hkv > FEW)


LONG = [
    (128, 4, 2, 64, [40], [40], 0, 0, "bf16", 0, False),
    (128, 28, 4, 64, [33, 70, 1], [33, 100, 200], 0, 0, "f32", 0, False),
    (64, 32, 8, 32, [300], [300], 0, 0, "bf16", 1, False),
    (64, 8, 1, 32, [129, 0, 64], [700, 50, 64], 0, 0, "f32", 0, True),
    (256, 3, 1, 128, [90], [200], 0, 0, "bf16", 0, False),
    (128, 8, 2, 128, [257], [257], 50, 0, "f32", 0, False),
    (128, 8, 2, 128, [200, 31], [600, 31], 64, 5, "bf16", 0, False),
    (64, 2, 2, 64, [500], [500], 7, 130, "f32", 0, False),
    (128, 7, 1, 256, [100], [1500], 0, 0, "bf16", 0, False),
    # several tiles of 128 rows, the records expanded for each or once for all
    (128, 8, 2, 64, [130], [130], 0, 0, "f32", 0, False),
    (128, 28, 4, 64, [100, 3, 70, 60], [400, 50, 60, 60], 0, 0, "bf16", 0, False),
    (64, 32, 8, 32, [600], [1000], 100, 5, "f32", 1, False),
    (128, 64, 4, 64, [300, 2, 50], [900, 40, 300], 130, 40, "bf16", 0, False),
    (64, 8, 1, 32, [70, 55], [3000, 900], 0, 0, "bf16", 0, True),
    (128, 4, 4, 128, [700, 40, 390], [700, 300, 391], 0, 0, "f32", 0, False),
    (64, 4, 4, 64, [513], [600], 33, 200, "bf16", 0, False),
    (128, 16, 2, 32, [65, 64], [1025, 64], 1, 0, "f32", 0, False),
    (128, 12, 1, 32, [43], [2400], 700, 64, "bf16", 0, False),
]


@pytest.mark.parametrize("d,hq,hkv,page,rows,ctx,window,sinks,okind,pad,hm", LONG)
def test_attend_prompts(d, hq, hkv, page, rows, ctx, window, sinks, okind, pad, hm):
    b = au.Batch(rows, ctx, page, seed=d + hq, lead=3, tail=1)
    pages = au.Pages(b.n_pages, page, hkv, d)
    K, V, q = data(b, hkv, d, hq, d + hq + page + 1)
    au.fill(pages, b, K, V)
    Q, O = run(pages, b, hq, q, d ** -0.5, window, sinks, okind, pad, hm)
    check(O, Q, b, K, V, hq, d ** -0.5, window, sinks, okind, True)


@pytest.mark.parametrize("d,hq,hkv,window,sinks", [(128, 28, 4, 0, 0), (64, 8, 2, 0, 0), (64, 8, 2, 60, 3),
                                                   (128, 8, 8, 0, 0), (128, 32, 1, 100, 0), (256, 4, 2, 0, 0)])
def test_generated_tokens_beside_a_prompt(d, hq, hkv, window, sinks):
    """Sequences of one or a few rows in one call with long ones, in any order."""
    g = hq // hkv
    few = FEW // g  # rows that the kernel of few rows takes
    rows = [1, 300, 1, few, few + 1, 0, 2, 64 + 130 // g]
    ctx = [700, 300, 1, few + 90, few + 90, 50, 333, 700]
    b = au.Batch(rows, ctx, 64, seed=6, lead=2, tail=2)
    pages = au.Pages(b.n_pages, 64, hkv, d)
    K, V, q = data(b, hkv, d, hq, 61)
    au.fill(pages, b, K, V)
    Q, O = run(pages, b, hq, q, d ** -0.5, window, sinks, "f32")
    check(O, Q, b, K, V, hq, d ** -0.5, window, sinks, "f32", True)


@pytest.mark.parametrize("rows,ctx", [([1, 1, 2], [64, 1024, 513]), ([40, 256], [296, 256])])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_equal_weights_give_the_exact_mean(rows, ctx, d):
    """q = 0: every visible token has the same weight.  Values that are small
    multiples of a power of two sum without rounding, so the result is the
    binary32 quotient of the sum and the count (three roundings: the
    reciprocal, the product and, joined ranges, their sums' scale)."""
    hq, hkv, page = 4, 2, 64
    b = au.Batch(rows, ctx, page, seed=d)
    pages = au.Pages(b.n_pages, page, hkv, d)
    n = sum(ctx)
    r = au.rng(d)
    V = r.integers(0, 16, size=(n, hkv, d)).astype(np.float64)
    V[..., 0::64], V[..., 1::64] = 0, 15  # s = 1, b = 0: codes are the values
    V = (V - 8) / 8
    K = r.standard_normal((n, hkv, d))
    au.fill(pages, b, K, V)
    for window, sinks in ((0, 0), (40, 3)):
        Q, O = run(pages, b, hq, np.zeros((b.rows, hq, d)), 1.0, window, sinks, "f32")
        got, at = O.get(), 0
        for s, (m, c) in enumerate(zip(b.n, b.ctx)):
            row = int(b.start[s])
            want, _ = au.attend(np.zeros((m, hq, d)), K[at:at + c], V[at:at + c], 1.0, window, sinks, c - m)
            # the reference's own weights 1 / n are rounded to binary64
            au.within(got[row:row + m], want, 4 * au.U * np.abs(want) + c * 2.0 ** -53, s)
            at += c


@pytest.mark.parametrize("rows", [1, 3, 70, 130])
@pytest.mark.parametrize("d", [64, 128])
def test_tokens_out_of_sight_do_not_count(rows, d):
    """Pages hold NaN (0xFF) wherever no token was written; tokens past a row, or
    outside its window, that read NaN; a page that is not there."""
    t = torch()
    hq, hkv, page, c = 8, 2, 32, 200
    b = au.Batch([rows, rows], [c, c], page, seed=3)
    pages = au.Pages(b.n_pages, page, hkv, d)
    K, V, q = data(b, hkv, d, hq, 9)
    K[150, 0, 3] = np.nan      # K of a token: NaN rows where it is seen
    V[c + 60, 1, 5] = np.inf   # V of a token: its run of 64 columns
    K[c - 1], V[c - 1] = np.inf, np.nan  # the last token, seen by the last row alone
    au.fill(pages, b, K, V)
    for window, sinks in ((0, 0), (49, 0), (49, 61), (20, 2)):
        Q, O = run(pages, b, hq, q, d ** -0.5, window, sinks, "f32")
        check(O, Q, b, K, V, hq, d ** -0.5, window, sinks, "f32", rows * 4 > 16)
    # without page 2 of sequence 1 its tokens 64 .. 95 are not there
    table = b.table.copy()
    table[1, 2] = -5
    b.dev[2] = t.from_numpy(table).to(DEV)
    Q, O = run(pages, b, hq, q, d ** -0.5, 0, 0, "f32")
    k, v = au.held(K[c:]), au.held(V[c:])
    keep = np.r_[0:64, 96:c]
    qq = Q.get()[rows:]
    for i in range(rows):
        n = int((keep <= c - rows + i).sum())
        want, mag = au.attend(qq[i:i + 1], k[keep[:n]], v[keep[:n]], d ** -0.5, 0, 0, n - 1)
        err = bounds(qq[i:i + 1], k[keep[:n]], v[keep[:n]], au.quantise(K[c:][keep[:n]])[1:],
                     au.quantise(V[c:][keep[:n]])[1:], d ** -0.5, mag, rows * 4 > 16)
        au.within(O.get()[rows + i:rows + i + 1], want, err + au.U * np.abs(want) + 1e-38, i)


@pytest.mark.parametrize("rows", [2, 50, 200])
def test_rows_that_see_nothing(rows):
    """Rows before position 0, contexts of zero, tables without pages: zeros."""
    d, hq, hkv, page = 128, 4, 2, 32
    b = au.Batch([rows, rows, rows], [rows + 10, rows - 1, 0], page, seed=4)
    pages = au.Pages(b.n_pages, page, hkv, d)
    K, V, q = data(b, hkv, d, hq, 21)
    au.fill(pages, b, K, V)
    Q, O = run(pages, b, hq, q, d ** -0.5, 0, 0, "f32")
    got = O.get()
    assert (got[rows] == 0).all() and (got[2 * rows:] == 0).all()
    assert np.isfinite(got).all() and (got[:rows] != 0).any() and (got[rows + 1:2 * rows] != 0).any()
    Q, O = run(pages, b, hq, q, d ** -0.5, 0, 0, "bf16", max_pages=0)
    assert (O.get() == 0).all()


@pytest.mark.parametrize("rows", [1, 40, 110])
def test_strong_and_weak_logits(rows):
    """Logits hundreds apart in either direction and order, a negative and a zero
    scale: the running maximum follows."""
    d, hq, hkv, page, c = 64, 4, 1, 64, 500
    b = au.Batch([rows], [c], page)
    K, V, q = data(b, hkv, d, hq, 31)
    for ramp in (np.linspace(0, 6, c), np.linspace(6, 0, c), np.where(np.arange(c) == 250, 6, 0)):
        Kr = au.rne(K * 0.05 + ramp[:, None, None] * np.sign(q[0, 0])[None, None], "bf16")
        pages = au.Pages(b.n_pages, page, hkv, d)
        au.fill(pages, b, Kr, V)
        for scale in (0.25, -0.25, 0.0):
            Q, O = run(pages, b, hq, q, scale, 0, 0, "f32")
            got = O.get()
            assert np.isfinite(got).all()
            want, mag = au.attend(Q.get(), au.held(Kr), au.held(V), scale, 0, 0, c - rows)
            err = bounds(Q.get(), au.held(Kr), au.held(V), au.quantise(Kr)[1:], au.quantise(V)[1:],
                         scale, mag, rows * 4 > 16)
            au.within(got, want, err + au.U * np.abs(want) + 1e-38, scale)


def test_equal_calls_give_equal_bits_and_sizes_are_hints():
    """Repeated calls, and calls told a wrong largest context."""
    d, hq, hkv, page = 128, 28, 4, 64
    b = au.Batch([1, 1, 1], [3000, 17, 900], page)
    pages = au.Pages(b.n_pages, page, hkv, d)
    K, V, q = data(b, hkv, d, hq, 41)
    au.fill(pages, b, K, V)
    Q, first = run(pages, b, hq, q, d ** -0.5)
    check(first, Q, b, K, V, hq, d ** -0.5, 0, 0, "bf16", False)
    for _ in range(3):
        assert torch().equal(run(pages, b, hq, q, d ** -0.5)[1].buf, first.buf)
    for hint in (1, 64, 300, 700, 10 ** 9):
        Q, O = run(pages, b, hq, q, d ** -0.5, max_context=hint)
        check(O, Q, b, K, V, hq, d ** -0.5, 0, 0, "bf16", False)


def test_large_magnitudes():
    """Keys, values and queries far from one: powers of two from 2^-60 to 2^60."""
    d, hq, hkv, page, c = 128, 8, 2, 64, 300
    for rows in (1, 64, 128):
        b = au.Batch([rows], [c], page)
        K, V, q = data(b, hkv, d, hq, 51)
        for ke, ve, qe in ((60, -60, -60), (-60, 60, 60), (0, 100, 0), (0, -100, 0), (20, 16, -20)):
            pages = au.Pages(b.n_pages, page, hkv, d)
            k, v = K * 2.0 ** ke, V * 2.0 ** ve
            au.fill(pages, b, k, v)
            Q, O = run(pages, b, hq, q * 2.0 ** qe, d ** -0.5, 0, 0, "f32")
            check(O, Q, b, k, v, hq, d ** -0.5, 0, 0, "f32", rows > 4)


@pytest.mark.parametrize("hint", [1, 64, 300, 620, 10 ** 9])
def test_prompts_longer_than_they_were_said_to_be(hint):
    """Records are expanded once for the sequences that the workspace has room
    for, and per tile for the others: the results are right either way."""
    d, hq, hkv, page = 64, 64, 8, 64
    b = au.Batch([200, 150, 1, 120], [250, 610, 70, 130], page)
    pages = au.Pages(b.n_pages, page, hkv, d)
    K, V, q = data(b, hkv, d, hq, 71)
    au.fill(pages, b, K, V)
    for window, sinks in ((0, 0), (77, 9)):
        Q, O = run(pages, b, hq, q, d ** -0.5, window, sinks, "f32", max_context=hint)
        check(O, Q, b, K, V, hq, d ** -0.5, window, sinks, "f32", True)


def test_room_for_the_records_of_one_prompt():
    """Tables for 262144 tokens, of which one sequence's records fill what is taken
    for them: the others' are expanded per tile."""
    d, hq, hkv, page = 128, 16, 8, 128
    b = au.Batch([200, 1, 210, 0, 195], [200, 300, 211, 40, 400], page, extra_cols=2048)
    pages = au.Pages(b.n_pages, page, hkv, d)
    K, V, q = data(b, hkv, d, hq, 72)
    au.fill(pages, b, K, V)
    Q, O = run(pages, b, hq, q, d ** -0.5, 0, 0, "f32", max_context=262144, max_pages=2048)
    check(O, Q, b, K, V, hq, d ** -0.5, 0, 0, "f32", True)


@pytest.mark.parametrize("rows", [1, 60, 512])
@pytest.mark.parametrize("ke,ve", [(30, 50), (-30, -50), (0, 100), (0, -100)])
def test_later_tokens_of_another_magnitude(rows, ke, ve):
    """The first 256 tokens and the others differ by powers of two: rows among the
    first are as exact as without the others, rows behind them see both."""
    d, hq, hkv, page, c, half = 64, 8, 2, 64, 512, 256
    b = au.Batch([rows], [c], page)
    K, V, q = data(b, hkv, d, hq, 81)
    K[half:] *= 2.0 ** ke
    V[half:] *= 2.0 ** ve
    q[max(0, rows - (c - half)):] *= 2.0 ** -max(ke, 0)
    pages = au.Pages(b.n_pages, page, hkv, d)
    au.fill(pages, b, K, V)
    Q, O = run(pages, b, hq, q, d ** -0.5, 0, 0, "f32")
    check(O, Q, b, K, V, hq, d ** -0.5, 0, 0, "f32", rows > 12)
    if rows == c:
        got, qq = O.get()[:half], Q.get()[:half]
        k, v = K[:half], V[:half]
        want, mag = au.attend(qq, au.held(k), au.held(v), d ** -0.5, 0, 0, 0)
        err = bounds(qq, au.held(k), au.held(v), au.quantise(k)[1:], au.quantise(v)[1:], d ** -0.5, mag, True)
        au.within(got, want, err + au.U * np.abs(want) + 1e-38)


@pytest.mark.parametrize("longest", [1, 3, 300])
def test_a_thousand_sequences(longest):
    d, hq, hkv, page = 64, 4, 2, 32
    r = au.rng(91)
    rows = [1] * 1100
    rows[1050], rows[3], rows[77] = longest, 0, 2
    ctx = [int(x) for x in r.integers(1, 70, 1100)]
    ctx[1050] = 310
    b = au.Batch(rows, ctx, page, seed=9, lead=1, tail=1)
    pages = au.Pages(b.n_pages, page, hkv, d)
    K, V, q = data(b, hkv, d, hq, 92)
    au.fill(pages, b, K, V)
    Q, O = run(pages, b, hq, q, d ** -0.5, 0, 0, "f32")
    check(O, Q, b, K, V, hq, d ** -0.5, 0, 0, "f32", longest > 24)


@pytest.mark.parametrize("rows", [1, 5, 150])
def test_far_pages_and_strides(rows):
    """Pages past 2^32 bytes, rows and heads of the operands past 2^31 elements."""
    d, hq, hkv, page = 64, 8, 2, 4096
    b = au.Batch([rows], [5000], page)
    n = 2 ** 32 // (page // 32 * hkv * 36 * d) + 40
    pages = au.Pages(n, page, hkv, d)
    K, V, q = data(b, hkv, d, hq, 95)
    b.dev[2] = torch().from_numpy(np.int32(n - 1) - b.table).to(DEV)  # the last pages
    au.fill(pages, b, K, V)
    far = 2 ** 30 + 8
    strides = (far, d) if rows == 5 else (hq * d, d) if rows == 1 else (d, 2 ** 29 + 8)
    Q = au.Operand(b.rows, hq, d, "bf16", strides=strides, values=q)
    d_ = b.dict()
    O = au.Operand(b.rows, hq, d, "bf16", strides=strides)
    nws = tsl.cache_attention_workspace_size(pages.dict, d_, hq)
    ws = torch().empty(nws, dtype=torch().uint8, device=DEV)
    tsl.cache_attention(pages.dict, d_, hq, Q.view, Q.ld, Q.head, 0.125, 0, 0, tsl.BF16, O.view, O.ld,
                        O.head, ws, nws)
    check(O, Q, b, K, V, hq, 0.125, 0, 0, "bf16", rows > 12)


@pytest.mark.parametrize("rows", [3, 60, 200])
def test_queries_that_are_not_finite(rows):
    """A row whose query is NaN or infinite in one head: the other heads of it and
    the other rows are as they would be."""
    d, hq, hkv, page, c = 128, 8, 2, 64, 300
    b = au.Batch([rows, rows], [c, c], page, seed=8)
    pages = au.Pages(b.n_pages, page, hkv, d)
    K, V, q = data(b, hkv, d, hq, 97)
    au.fill(pages, b, K, V)
    Q = au.Operand(b.rows, hq, d, "bf16", values=q)
    for bad in (np.nan, np.inf, -np.inf):
        q2 = q.copy()
        q2[1, 3, 7], q2[rows + rows // 2, 0, 100] = bad, bad
        _, O = run(pages, b, hq, q2, d ** -0.5, 0, 0, "f32")
        got = O.get()
        for i, x in ((1, 3), (rows + rows // 2, 0)):
            if np.isnan(bad):
                assert np.isnan(got[i, x]).all()
            got[i, x] = 0  # not compared
        at = 0
        for s in range(2):
            qq = Q.get()[s * rows:(s + 1) * rows]
            k, v = K[at:at + c], V[at:at + c]
            want, mag = au.attend(qq, au.held(k), au.held(v), d ** -0.5, 0, 0, c - rows)
            err = bounds(qq, au.held(k), au.held(v), au.quantise(k)[1:], au.quantise(v)[1:], d ** -0.5, mag,
                         rows * 4 > FEW)
            i, x = ((1, 3), (rows // 2, 0))[s]
            want[i, x] = 0
            au.within(got[s * rows:(s + 1) * rows], want, err + au.U * np.abs(want) + 1e-38, s)
            at += c


def test_two_calls_at_once():
    """Two streams, a workspace each, the same cache: each as by itself."""
    t = torch()
    d, hq, hkv, page = 128, 16, 2, 64
    b = au.Batch([1, 130, 1, 2], [3000, 900, 40, 700], page, seed=12)
    pages = au.Pages(b.n_pages, page, hkv, d)
    K, V, q = data(b, hkv, d, hq, 98)
    au.fill(pages, b, K, V)
    kinds = ((1, 0, 0), (-0.5, 100, 4))
    alone = [run(pages, b, hq, q * f, d ** -0.5, w, s, "f32") for f, w, s in kinds]
    seqs, calls = b.dict(), []
    if ROOMY:
        widened(pages, b, seqs)
    for k in range(8):
        f, w, s = kinds[k % 2]
        n = tsl.cache_attention_workspace_size(pages.dict, seqs, hq, w, s)
        calls.append((w, s, au.Operand(b.rows, hq, d, "bf16", values=q * f), au.Operand(b.rows, hq, d, "f32"),
                      n, t.empty(max(n, 256), dtype=t.uint8, device=DEV)))
    streams = [t.cuda.Stream() for _ in kinds]
    t.cuda.synchronize()
    for k, (w, s, Q, O, n, ws) in enumerate(calls):
        tsl.cache_attention(pages.dict, seqs, hq, Q.view, Q.ld, Q.head, d ** -0.5, w, s, tsl.F32, O.view,
                            O.ld, O.head, ws, n, streams[k % 2].cuda_stream)
    t.cuda.synchronize()
    for k, c in enumerate(calls):
        assert t.equal(c[3].buf, alone[k % 2][1].buf), k


@pytest.mark.parametrize("rows", [1, 60, 150])
@pytest.mark.parametrize("ve", [-100, 90])
def test_missing_pages_among_values_of_any_magnitude(rows, ve):
    t = torch()
    d, hq, hkv, page, c = 64, 8, 2, 32, 320
    b = au.Batch([rows], [c], page, seed=14)
    pages = au.Pages(b.n_pages, page, hkv, d)
    K, V, q = data(b, hkv, d, hq, 99)
    V = V * 2.0 ** ve
    au.fill(pages, b, K, V)
    table = b.table.copy()
    table[0, [0, 4, 9]] = -1, b.n_pages, -7
    b.dev[2] = t.from_numpy(table).to(DEV)
    keep = np.r_[32:128, 160:288]
    for window, sinks in ((0, 0), (200, 40)):
        Q, O = run(pages, b, hq, q, d ** -0.5, window, sinks, "f32")
        got, qq = O.get(), Q.get()
        for i in range(rows):
            pos = c - rows + i
            j = keep[(keep <= pos) & ((keep > pos - window) | (keep < sinks) | (window == 0))]
            want, mag = au.attend(qq[i:i + 1], au.held(K[j]), au.held(V[j]), d ** -0.5, 0, 0, len(j) - 1)
            err = bounds(qq[i:i + 1], au.held(K[j]), au.held(V[j]), au.quantise(K[j])[1:],
                         au.quantise(V[j])[1:], d ** -0.5, mag, rows * 4 > FEW)
            au.within(got[i:i + 1], want, err + au.U * np.abs(want) + 1e-38, i)


@pytest.mark.parametrize("rows", [1, 60, 150])
@pytest.mark.parametrize("d", [64, 128])
def test_large_values_without_weight(rows, d):
    """128 tokens whose logits leave them no weight (e^-512 d / 64) and whose values
    are 2^40 times the others': the others keep their bits."""
    hq, hkv, page, c = 4, 1, 64, 600
    b = au.Batch([rows], [c], page, seed=15)
    pages = au.Pages(b.n_pages, page, hkv, d)
    K, V, q = data(b, hkv, d, hq, 100, kscale=0.05)
    q[:] = 1.0
    for lo in (0, 256):
        k, v = K.copy(), V.copy()
        k[lo:lo + 128] = -8.0
        v[lo:lo + 128] *= 2.0 ** 40
        rest = np.r_[0:lo, lo + 128:c]
        au.fill(pages, b, k, v)
        Q, O = run(pages, b, hq, q, 1.0, 0, 0, "f32")
        got, qq = O.get(), Q.get()
        for i in range(0, rows, 7):
            j = rest[rest <= c - rows + i]
            want, mag = au.attend(qq[i:i + 1], au.held(k[j]), au.held(v[j]), 1.0, 0, 0, len(j) - 1)
            err = bounds(qq[i:i + 1], au.held(k[j]), au.held(v[j]), au.quantise(k[j])[1:],
                         au.quantise(v[j])[1:], 1.0, mag, rows * 4 > FEW)
            au.within(got[i:i + 1], want, err + au.U * np.abs(want) + 1e-38, (lo, i))
