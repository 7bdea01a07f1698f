"""cache_attention at sizes whose products are large though their sums are not.
Tolerances are those of test_gpu_attend."""
import pytest

import attn_util as au
import test_gpu_attend as ta

pytestmark = pytest.mark.gpu


def call(monkeypatch, b, hq, hkv, d, window=0, sinks=0, kind="f32", page=32, seed=0, rounded=False, **kw):
    monkeypatch.setattr(ta, "ROOMY", False, raising=False)
    pages = au.Pages(b.n_pages, page, hkv, d)
    K, V, q = ta.data(b, hkv, d, hq, seed)
    au.fill(pages, b, K, V)
    Q, O = ta.run(pages, b, hq, q, d ** -0.5, window, sinks, kind, **kw)
    ta.check(O, Q, b, K, V, hq, d ** -0.5, window, sinks, kind, rounded)


def test_a_prompt_of_heads_of_256_beside_hundreds_of_tokens(monkeypatch):
    rows = [1] * 600
    rows[411] = 1024
    b = au.Batch(rows, [1024 if n > 1 else 20 + i % 90 for i, n in enumerate(rows)], 32, seed=2, lead=1, tail=2)
    call(monkeypatch, b, 32, 4, 256, seed=21)


@pytest.mark.parametrize("window,sinks", [(0, 0), (150, 40)])
def test_tiles_over_several_waves_of_heads_of_256(monkeypatch, window, sinks):
    """Prompts of lengths that leave tiles in every position of a wave's part: begun
    and ended in it, begun, ended, and neither."""
    b = au.Batch([1, 300, 17, 2, 90], [2500, 300, 900, 64, 1500], 32, seed=3, lead=2, tail=1)
    call(monkeypatch, b, 6, 2, 256, window, sinks, seed=22)
    b = au.Batch([1], [12000], 32, seed=4)  # one tile over all waves
    call(monkeypatch, b, 2, 1, 256, window, sinks, seed=23)


def test_hundreds_of_sequences_of_a_few_more_rows_than_few(monkeypatch):
    """72 query rows a K/V head each: more tiles than workgroups that run at once."""
    r = au.rng(6)
    ctx = [int(x) for x in r.integers(9, 400, 300)]
    b = au.Batch([9] * 300, ctx, 32, seed=7, lead=1, tail=1)
    call(monkeypatch, b, 16, 2, 128, seed=24, rounded=True)
    # ... of which one alone has them, in ranges of tokens
    rows = [1] * 400
    rows[123] = 40
    b = au.Batch(rows, [3000 if n > 1 else 50 for n in rows], 32, seed=8)
    call(monkeypatch, b, 16, 2, 128, seed=25, rounded=True)


def test_two_thousand_prompts(monkeypatch):
    r = au.rng(9)
    ctx = [128 + int(x) for x in r.integers(0, 40, 2048)]
    call(monkeypatch, au.Batch([128] * 2048, ctx, 32, seed=10), 1, 1, 64, seed=26, rounded=True)


@pytest.mark.parametrize("d,hq,hkv,rows,ctx,window", [
    (64, 300, 1, [1, 2], [900, 40], 0),       # one token's heads over several tiles
    (128, 260, 2, [1], [3000], 500),
    (256, 130, 1, [1, 3], [300, 900], 0),
    (64, 400, 200, [1, 1, 40], [70, 1, 90], 0),
    (128, 150, 150, [70], [70], 20)])
def test_many_heads(monkeypatch, d, hq, hkv, rows, ctx, window):
    b = au.Batch(rows, ctx, 32, seed=11, lead=1, tail=1)
    call(monkeypatch, b, hq, hkv, d, window, 3, seed=27,
         rounded=d < 256 and max(rows) * hq // hkv > ta.FEW)


def test_told_of_no_context_at_all(monkeypatch):
    for d, rows in ((64, [1, 3]), (128, [90, 2]), (256, [20, 1])):
        b = au.Batch(rows, [400, 333], 32, seed=12)
        call(monkeypatch, b, 4, 2, d, seed=28, rounded=d < 256, max_context=0)
