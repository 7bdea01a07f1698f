"""cache_attention where one wave of the kernel of few rows walks a long range of
tokens: binary32 results, near-equal weights.

Tolerance, u = 2^-24.  V's codes are summed as z + c, z 128 for a quarter of the
tokens and 16 for the others (44 on average; c averages 7.5), beside the same sum
without c, and every 8 records the difference is taken.  Within those 256 tokens
of weight w the 16 partial sums of either grow evenly to A = 256 w s 51.5 and
A' = 256 w s 44; were every rounding at its bound u and all of one sign, the
difference would be off by 8.5 u (A + A').  With normal values (s = 4.75 / 15 of
their deviation v), w = 1 / n and n / 256 such differences, each independent of
the others, the result is off by
    8.5 u 256 (0.317 v) 95.5 / n sqrt(n / 256) = 2.5e-4 v / sqrt(n),
where the result itself, a mean of n independent values, is v / sqrt(n): 2^-12 of
its norm, for any n.  (Roundings of random sign come to a tenth of that.)  What
else is rounded is small beside it: p s to 16 bits of random sign, 2^-17 of
terms that are 2 v / n each; the logits (see test_gpu_attend), whose e = 72 u
271 s a scale <= 2^-14 at |q| = 2^-6, moves weights by 2 e of random sign."""
import numpy as np
import pytest

import attn_util as au
from gpu_util import DEV, torch
from tensor_sharded_linear_plan_amd import binding as tsl

pytestmark = pytest.mark.gpu

BOUND = 2.0 ** -12
Q = 2.0 ** -6


def filled(ctx, d, hkv, seed, page=256):
    b = au.Batch([1], [ctx], page, seed=seed)
    pages = au.Pages(b.n_pages, page, hkv, d)
    r = au.rng(seed)
    K, V = (au.rne(r.standard_normal((ctx, hkv, d)), "bf16") for _ in "kv")
    au.fill(pages, b, K, V)
    return b, pages, au.held(K), au.held(V), r


def call(pages, seqs, hq, q, window=0, sinks=0, kind="f32"):
    rows, _, d = q.shape
    op, o = au.Operand(rows, hq, d, "bf16", values=q), au.Operand(rows, hq, d, kind)
    n = tsl.cache_attention_workspace_size(pages.dict, seqs, hq, window, sinks)
    ws = torch().full((n + 256,), 0xFF, dtype=torch().uint8, device=DEV)
    tsl.cache_attention(pages.dict, seqs, hq, op.view, op.ld, op.head, d ** -0.5, window, sinks,
                        au.DT[kind], o.view, o.ld, o.head, ws, n)
    assert bool((ws[n:] == 0xFF).all())
    return op.get(), o.get(), n


def error(got, want):
    assert np.isfinite(got).all()
    return np.linalg.norm(got - want) / np.linalg.norm(want)


@pytest.mark.parametrize("d,hq,hkv,rows,ctx", [
    (64, 4, 1, 1, 32768), (64, 4, 1, 1, 131072), (64, 8, 1, 5, 32768), (128, 6, 2, 1, 32768),
    (128, 2, 1, 1, 131072), (128, 16, 1, 4, 32768), (256, 2, 1, 1, 32768), (256, 5, 1, 3, 20000)])
@pytest.mark.parametrize("window", [0, 30000])
def test_one_wave_walks_all_of_a_long_context(d, hq, hkv, rows, ctx, window):
    """Told of 64 tokens, a call gives each tile to one wave, however many there are."""
    b, pages, K, V, r = filled(ctx, d, hkv, d + hq)
    b = au.Batch([rows], [ctx], 256, seed=d + hq)
    q = r.standard_normal((rows, hq, d)) * Q
    qq, got, n = call(pages, b.dict(max_context=64), hq, q, window, 4 if window else 0)
    assert n == 0
    want, _ = au.attend(qq, K, V, d ** -0.5, window, 4 if window else 0, ctx - rows)
    assert error(got, want) <= BOUND


@pytest.mark.parametrize("n,d,hkv,ctx", [(256, 128, 8, 8192), (600, 64, 8, 5000), (1030, 64, 2, 8192)])
def test_as_many_tiles_as_waves(n, d, hkv, ctx):
    """A batch whose tiles fill the chip; the sequences share their pages."""
    t = torch()
    b, pages, K, V, r = filled(ctx, d, hkv, n)
    hq = 2 * hkv
    q = r.standard_normal((1, hq, d)) * Q
    seqs = b.dict(n_seqs=n, rows=n, row_start=t.arange(n + 1, dtype=t.int32, device=DEV),
                  context=t.full((n,), ctx, dtype=t.int32, device=DEV),
                  page_table=b.dev[2].repeat(n, 1))
    qq, got, _ = call(pages, seqs, hq, np.broadcast_to(q, (n, hq, d)))
    want, _ = au.attend(qq[:1], K, V, d ** -0.5, 0, 0, ctx - 1)
    for s in range(n):
        assert error(got[s:s + 1], want) <= BOUND, s


@pytest.mark.parametrize("rows,ctx", [(90, 200), (40, 12000)])
def test_many_rows_of_heads_of_256(rows, ctx):
    """Any number of rows with heads of 256 goes the same way."""
    b, pages, K, V, r = filled(ctx, 256, 1, rows)
    b = au.Batch([rows], [ctx], 256, seed=rows)
    q = r.standard_normal((rows, 3, 256)) * Q
    qq, got, _ = call(pages, b.dict(), 3, q)
    want, _ = au.attend(qq, K, V, 1 / 16, 0, 0, ctx - rows)
    assert error(got, want) <= BOUND


@pytest.mark.parametrize("every", [8, 2])
def test_records_that_are_not_there(every):
    """Each record that a settlement would follow is missing: the others' sums are
    settled all the same."""
    t, d, hkv, ctx = torch(), 64, 1, 32768
    b, pages, K, V, r = filled(ctx, d, hkv, 5, page=32)
    table = b.table.copy()
    table[0, every - 1:ctx // 32:every] = -1
    b.dev[2] = t.from_numpy(table).to(DEV)
    keep = np.flatnonzero(np.repeat(table[0, :ctx // 32] >= 0, 32))
    q = r.standard_normal((1, 4, d)) * Q
    qq, got, _ = call(pages, b.dict(max_context=64), 4, q)
    want, _ = au.attend(qq, K[keep], V[keep], d ** -0.5, 0, 0, len(keep) - 1)
    assert error(got, want) <= BOUND
