"""cache_append and cache_read on the GPU: codes, scales and biases bit for bit
against the quantiser in binary64, read from the pages by the layout's
description, and what must keep its bits."""
import numpy as np
import pytest

import attn_util as au
from gpu_util import DEV, torch
from tensor_sharded_linear_plan_amd import binding as tsl

pytestmark = pytest.mark.gpu


def rows_of(batch):
    """(sequence, position, row) of every live row that has a place."""
    out = []
    for s, (n, c) in enumerate(zip(batch.n, batch.ctx)):
        for i in range(n):
            out.append((s, c - n + i, int(batch.start[s]) + i))
    return out


def append(pages, batch, K, V, kind, pad=0, head_major=False, **kw):
    k = au.Operand(batch.rows, pages.heads, pages.d, kind, pad, head_major, values=K)
    v = au.Operand(batch.rows, pages.heads, pages.d, kind, pad, head_major, values=V)
    tsl.cache_append(pages.dict, batch.dict(**kw), au.DT[kind], k.view, k.ld, k.head, v.view, v.ld,
                     v.head)
    return k.get(), v.get()


def check_pages(pages, batch, k, v):
    kc, vc, ks, vs = pages.unpack()
    touched = np.zeros(kc.shape[:2], bool)
    for s, pos, row in rows_of(batch):
        if pos < 0:
            continue
        p, t = batch.table[s, pos // pages.page_tokens], pos % pages.page_tokens
        touched[p, t] = True
        for x, c, (sc, bi) in ((k[row], kc, ks), (v[row], vc, vs)):
            q, a, b = au.quantise(x)
            assert np.array_equal(c[p, t], q), (s, pos)
            assert np.array_equal(sc[p, t], a, equal_nan=True)
            assert np.array_equal(bi[p, t], b, equal_nan=True)
    # everything else is as it was: codes 15, scales and biases NaN (0xFF bytes)
    for c in (kc, vc):
        assert (c[~touched] == 15).all()
    for sc, bi in (ks, vs):
        assert np.isnan(sc[~touched]).all() and np.isnan(bi[~touched]).all()
    assert bool((pages.buf[pages.bytes:] == pages.fill).all())


@pytest.mark.parametrize("d,heads,page,kind,rows,ctx,pad,head_major", [
    (128, 2, 64, "bf16", [1], [1], 0, False),
    (128, 1, 32, "bf16", [1, 1, 1, 1], [1, 32, 33, 100], 0, False),
    (64, 3, 32, "bf16", [5, 0, 40, 31], [5, 7, 71, 64], 1, False),
    (256, 2, 64, "f32", [3, 65, 1], [3, 200, 65], 0, True),
    (128, 2, 128, "f32", [17, 130], [17, 300], 2, False),
    (64, 1, 256, "bf16", [100], [100], 0, True),
])
def test_append(d, heads, page, kind, rows, ctx, pad, head_major):
    b = au.Batch(rows, ctx, page, seed=d + page, lead=2, tail=3)
    pages = au.Pages(b.n_pages, page, heads, d)
    r = au.rng(d * heads)
    shape = (b.rows, heads, d)
    K = r.standard_normal(shape) * 2 + r.standard_normal((1, heads, d))
    V = r.standard_normal(shape) * 0.1
    k, v = append(pages, b, K, V, kind, pad, head_major)
    check_pages(pages, b, k, v)
    # and back, in both types; rows of no sequence keep what they had
    for okind in ("f32", "bf16"):
        ko = au.Operand(b.rows, heads, d, okind, pad, head_major)
        vo = au.Operand(b.rows, heads, d, okind, pad, head_major)
        tsl.cache_read(pages.dict, b.dict(), au.DT[okind], ko.view, ko.ld, ko.head, vo.view, vo.ld,
                       vo.head)
        live = b.live()
        for o, x in ((ko, k), (vo, v)):
            assert np.array_equal(o.get()[live], au.rne(au.held(x[live]), okind))
            assert o.rest_untouched(list(live))


def test_tokens_one_at_a_time_equal_all_at_once():
    d, heads, page, n = 128, 2, 64, 75
    r = au.rng(4)
    K, V = r.standard_normal((n, heads, d)), r.standard_normal((n, heads, d))
    b = au.Batch([n], [n], page, seed=1)
    one, all_ = (au.Pages(b.n_pages, page, heads, d) for _ in range(2))
    append(all_, b, K, V, "bf16")
    for i in range(n):
        step = au.Batch([1], [i + 1], page, seed=1)
        step.table, step.max_pages, step.dev = b.table, b.max_pages, [step.dev[0], step.dev[1], b.dev[2]]
        append(one, step, K[i:i + 1], V[i:i + 1], "bf16")
    assert torch().equal(one.buf, all_.buf)


def test_borders_of_codes_and_scales():
    """Quotients on and next to the borders between codes, constant runs, tiny
    and huge ones, and runs that are not finite."""
    d, heads, page = 64, 1, 32
    rows = []
    base = np.arange(64) / 4.0                                  # s = 1.05 -> 1.0469
    rows.append(base)
    rows.append(np.concatenate([[0, 15], np.arange(62) % 30 / 2]))  # s = 1: ties at k + 1/2
    for k in range(6):                                          # one ulp beside the ties
        tie = np.concatenate([[0, 15], np.arange(62) % 30 / 2]).astype(np.float32)
        tie[2 + k::6] = np.nextafter(tie[2 + k::6], np.float32(99 if k % 2 else -99))
        tie[2:] = np.clip(tie[2:], 0, 15)
        rows.append(tie)
    rows.append(np.full(64, 3.25))                              # constant: s = 0
    rows.append(np.full(64, -0.0))
    rows.append(base * 1e-40)                                   # scales below the normals
    rows.append(base * 1e37)
    rows.append(np.where(np.arange(64) % 2, 3e38, -3e38))       # max - b past binary32
    for bad in (np.nan, np.inf, -np.inf):
        x = base.copy()
        x[17] = bad
        rows.append(x)
    rows.append(np.where(np.arange(64) == 5, 1e30, 1.0))        # one outlier
    rows.append(-1000 + base / 64)                              # far from zero, little spread
    K = np.stack(rows)[:, None, :]
    n = len(rows)
    for kind in ("f32", "bf16"):
        b = au.Batch([n], [n], page)
        pages = au.Pages(b.n_pages, page, heads, d)
        k, v = append(pages, b, K, K[::-1], kind)
        check_pages(pages, b, k, v)
    r = au.rng(11)  # many random runs: no code off by one
    K, V = (r.standard_normal((2000, 2, 64)) * np.exp2(r.integers(-20, 20, size=(2000, 2, 1)))
            for _ in range(2))
    b = au.Batch([2000], [2000], 256)
    pages = au.Pages(b.n_pages, 256, 2, 64)
    k, v = append(pages, b, K, V, "f32")
    check_pages(pages, b, k, v)


def test_places_that_are_not_there():
    """Positions before 0, past the table and in pages outside the cache: nothing
    is written, and they read as zeros."""
    t, d, heads, page = torch(), 128, 2, 32
    b = au.Batch([40, 10, 70, 5], [100, 4, 70, 12], page, seed=2)
    table = b.table.copy()
    table[0, 2] = -1                 # positions 64 .. 95 of sequence 0
    table[2, 1] = b.n_pages          # 32 .. 63 of sequence 2
    table[2, 2] = 2 ** 31 - 1        # 64 .. 69
    b.dev[2] = t.from_numpy(table).to(DEV)
    pages = au.Pages(b.n_pages, page, heads, d)
    r = au.rng(5)
    K, V = r.standard_normal((b.rows, heads, d)), r.standard_normal((b.rows, heads, d))
    short = dict(max_pages=3)        # the table's first three columns only: 96 tokens
    k, v = append(pages, b, K, V, "bf16", **short)
    there = [(s, p, row) for s, p, row in rows_of(b)
             if 0 <= p < 96 and 0 <= table[s, p // page] < b.n_pages]
    kc, vc, ks, vs = pages.unpack()
    for s, p, row in there:
        assert np.array_equal(kc[table[s, p // page], p % page], au.quantise(k[row])[0])
    assert int((~np.isnan(ks[0])).sum()) == len(there) * heads * d // 64
    ko = au.Operand(b.rows, heads, d, "f32")
    vo = au.Operand(b.rows, heads, d, "f32")
    tsl.cache_read(pages.dict, b.dict(**short), tsl.F32, ko.view, ko.ld, ko.head, vo.view, vo.ld, vo.head)
    want_k, want_v = np.zeros_like(k), np.zeros_like(v)
    for s, p, row in there:
        want_k[row], want_v[row] = au.rne(au.held(k[row]), "f32"), au.rne(au.held(v[row]), "f32")
    assert np.array_equal(ko.get(), want_k) and np.array_equal(vo.get(), want_v)


def test_read_one_side_and_row_limits():
    d, heads, page = 64, 2, 32
    b = au.Batch([9, 4], [20, 4], page, tail=2)
    pages = au.Pages(b.n_pages, page, heads, d)
    r = au.rng(6)
    k, v = append(pages, b, r.standard_normal((b.rows, heads, d)), r.standard_normal((b.rows, heads, d)),
                  "bf16")
    for side in (0, 1):
        o = au.Operand(b.rows, heads, d, "f32")
        arg = [None, 0, 0] * 2
        arg[3 * side:3 * side + 3] = [o.view, o.ld, o.head]
        tsl.cache_read(pages.dict, b.dict(max_rows=6), tsl.F32, *arg)
        got, want = o.get(), au.rne(au.held((k, v)[side]), "f32")
        live = list(range(6)) + list(range(9, 13))  # rows 6 .. 8 of the first are past max_rows
        assert np.array_equal(got[live], want[live])
        assert o.rest_untouched(live)
    # nothing to do
    none = au.Batch([], [], page)
    e = au.Operand(1, heads, d, "bf16")
    tsl.cache_append(pages.dict, none.dict(), tsl.BF16, e.view, e.ld, e.head, e.view, e.ld, e.head)
