"""cache_attention over values of very different size: what a value keeps beside
larger ones, with and without weight.

Keys are 0, but for some tokens whose logits are -512 (or 512 for a row whose query
has the other sign): the others' weights are equal, and theirs e^-512, or 1 and the
others' nothing.  So probabilities are exact and a result is the mean of values.

Tolerance, u = 2^-24: sequences of more than 64 query rows a K/V head take values
rounded to binary16, half a step 2^-11, in units in which the largest of its record
(of 128 neighbours at most) is 2^10.9 or more: a scale, a bias and the value are
each off by half of 2^-24 units at least, so by 3 2^-25 2^-10.9 of the largest
together.  The sum over the tokens adds (ctx + 8) u of the terms.  Others' sums
(test_gpu_attend_long) are off by 15.7 u 52 s <= 2^-14 of a value's size 3 s, less
than 2^-11 of the terms' mean."""
import numpy as np
import pytest

import attn_util as au
import test_gpu_attend as ta

pytestmark = pytest.mark.gpu


@pytest.fixture(params=[False, True], ids=["", "roomy"], autouse=True)
def roomy(request, monkeypatch):
    monkeypatch.setattr(ta, "ROOMY", request.param, raising=False)


def setup(rows, d, ctx, big, V, signs, hq=4, kind="bf16"):
    """Rows at the end of ctx tokens, of which `big` (a mask) have keys of -8; what
    each row's result is, its terms' mean size."""
    b = au.Batch([rows], [ctx], 64, seed=ctx)
    pages = au.Pages(b.n_pages, 64, 1, d)
    K = np.where(big[:, None, None], -8.0, 0.0) * np.ones((1, 1, d))
    au.fill(pages, b, K, V, kind)
    q = np.ones((rows, hq, d)) * signs[:, None, None]
    Q, O = ta.run(pages, b, hq, q, 64 / d, 0, 0, "f32")
    got, held = O.get(), au.held(V)[:, 0]
    want, mag = np.zeros((rows, d)), np.zeros((rows, d))
    for i in range(rows):
        see = (np.arange(ctx) <= ctx - rows + i) & (big if signs[i] < 0 else ~big)
        want[i], mag[i] = held[see].mean(0), np.abs(held[see]).mean(0)
    return got, want[:, None], mag[:, None]


@pytest.mark.parametrize("rows", [1, 60, 150])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("k", [0, 12, 16, 18, 20, 21])
def test_small_runs_beside_a_large_one(rows, d, k):
    """Every record's last token has values of -64.5 .. 55, the others' are 2^-k
    times such (scale and bias of 8 bits): to 2^-22 of the largest they keep theirs."""
    ctx = 620
    r = au.rng(k)
    c = r.integers(0, 16, size=(ctx, 1, d))
    c[..., 0::64], c[..., 1::64] = 0, 15
    V = c * (255 / 32) - 64.5
    big = np.arange(ctx) % 32 == 31
    V[~big] *= 2.0 ** -k
    got, want, mag = setup(rows, d, ctx, big, V, np.ones(rows), kind="f32")
    au.within(got, np.broadcast_to(want, got.shape),
              (2.0 ** -11 + (ctx + 8) * au.U) * mag + 3 * 2.0 ** -25 * 2.0 ** -10.9 * 64.5 + 1e-38, k)


@pytest.mark.parametrize("rows", [1, 60, 150])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("be,e", [(40, 0), (100, 0), (100, -60), (98, -100), (-100, 20)])
@pytest.mark.parametrize("where", ["first", "middle", "turns", "fives"])
def test_values_without_weight(rows, d, be, e, where):
    """2^be values that most rows pass over without weight, and every third row
    gives all its weight, before, among or in turn with the others' 2^e."""
    ctx = 600
    t = np.arange(ctx)
    big = {"first": t < 128, "middle": (t >= 256) & (t < 384), "turns": t // 32 % 2 == 1,
           "fives": t % 5 == 0}[where]
    r = au.rng(d + rows)
    V = au.rne(r.standard_normal((ctx, 1, d)) * np.where(big, 2.0 ** be, 2.0 ** e)[:, None, None], "bf16")
    signs = np.where(np.arange(rows) % 3 == 1, -1.0, 1.0)
    got, want, mag = setup(rows, d, ctx, big, V, signs)
    size = np.where(signs < 0, 2.0 ** be, 2.0 ** e)[:, None, None] * 8
    if where in ("turns", "fives") and rows > 1:
        # the two kinds are neighbours: what the large ones leave of the small is not
        # kept, the large ones are
        keep = signs < 0 if be > e else signs > 0
        got, want, mag, size = got[keep], want[keep], mag[keep], size[keep]
    au.within(got, np.broadcast_to(want, got.shape),
              (2.0 ** -11 + (ctx + 8) * au.U) * mag + 3 * 2.0 ** -25 * 2.0 ** -10.9 * size + 1e-38, where)
