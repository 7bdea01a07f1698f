"""Runs of binary32 whose values lie closer together than a bf16's step: the bias,
rounded, may lie above all of them, and then the scale of the header's formula is
negative.  Codes, scales and biases bit for bit as that says, what is read back, and
attention over them."""
import numpy as np
import pytest

import attn_util as au
import test_gpu_attend as ta
from tensor_sharded_linear_plan_amd import binding as tsl

pytestmark = pytest.mark.gpu


def quantise(x):
    """cache_append's formula in full: any scale but 0 divides."""
    r = x.reshape(x.shape[:-1] + (x.shape[-1] // 64, 64))
    b = au.rne(r.min(-1), "bf16")
    s = au.rne(((r.max(-1).astype(np.float32) - b.astype(np.float32)).astype(np.float32) /
                np.float32(15)).astype(np.float64), "bf16")
    c = np.rint((r - b[..., None]) / np.where(s != 0, s, 1.0)[..., None])
    c = np.where((s != 0)[..., None], np.clip(c, 0, 15), 0)
    return c.reshape(x.shape).astype(np.int64), s, b


def narrow(n, heads, d, seed):
    """Runs around values whose bf16 lies above or below them, spread by less than a
    step, by a few, and not at all; among them tiny ones."""
    r = au.rng(seed)
    runs = (n, heads, d // 64, 1)
    mid = r.choice([1.006, 1.002, -1.006, 100.3, -7.77, 2.0 ** -20 * 1.006, 3.0], runs) * \
        r.choice([1.0, 1.001, 0.999], runs)
    step = np.abs(mid) * r.choice([0.0, 2.0 ** -20, 2.0 ** -12, 2.0 ** -9, 2.0 ** -7, 2.0 ** -5], runs)
    x = (mid + step * r.uniform(-1, 1, (n, heads, d // 64, 64))).astype(np.float32)
    one = r.random((n, heads, d // 64)) < 0.1  # one value beside equal ones
    x[one] = x[one][:, :1]
    x[one, 17] *= np.float32(1 + 2.0 ** -20)
    return x.reshape(n, heads, d).astype(np.float64)


@pytest.mark.parametrize("d,heads", [(64, 2), (128, 1), (256, 1)])
def test_narrow_runs(d, heads):
    n, page = 400, 64
    b = au.Batch([n], [n], page, seed=d)
    pages = au.Pages(b.n_pages, page, heads, d)
    x = [narrow(n, heads, d, d + i) for i in (0, 1)]
    ops = [au.Operand(n, heads, d, "f32", values=v) for v in x]
    k, v = ops
    tsl.cache_append(pages.dict, b.dict(), tsl.F32, k.view, k.ld, k.head, v.view, v.ld, v.head)
    kc, vc, ks, vs = pages.unpack()
    at = (b.table[0, np.arange(n) // page], np.arange(n) % page)
    out = [au.Operand(n, heads, d, "f32") for _ in x]
    ko, vo = out
    tsl.cache_read(pages.dict, b.dict(), tsl.F32, ko.view, ko.ld, ko.head, vo.view, vo.ld, vo.head)
    some = 0
    for val, codes, (sc, bi), o in ((x[0], kc, ks, ko), (x[1], vc, vs, vo)):
        c, s, bias = quantise(val)
        some += int((s < 0).sum())
        assert np.array_equal(codes[at], c) and np.array_equal(sc[at], s) and np.array_equal(bi[at], bias)
        held = au.values(c, s, bias)
        assert np.array_equal(o.get(), au.rne(held, "f32"))
    assert some > 50


@pytest.mark.parametrize("rows", [1, 60])
@pytest.mark.parametrize("d", [64, 128])
def test_attention_over_narrow_runs(monkeypatch, rows, d):
    """Steps of either sign in the products: 1 and 60 rows (240 query rows a K/V
    head) of 4 heads over 300 tokens, by test_gpu_attend's bounds."""
    hq, n, page = 4, 300, 64
    b = au.Batch([rows], [n], page, seed=3)
    pages = au.Pages(b.n_pages, page, 1, d)
    K, V = narrow(n, 1, d, 5) / 8, narrow(n, 1, d, 6)
    au.fill(pages, b, K, V, "f32")
    q = au.rng(7).standard_normal((rows, hq, d))
    (kc, *ks), (vc, *vs) = quantise(au.rne(K, "f32")), quantise(au.rne(V, "f32"))
    k, v = au.values(kc, *ks), au.values(vc, *vs)
    many = rows * hq > ta.FEW
    for roomy in (False, True):
        monkeypatch.setattr(ta, "ROOMY", roomy, raising=False)
        Q, O = ta.run(pages, b, hq, q, d ** -0.5, 0, 0, "f32")
        want, mag = au.attend(Q.get(), k, v, d ** -0.5, 0, 0, n - rows)
        err = ta.bounds(Q.get(), k, v, ks, vs, d ** -0.5, mag, many)
        au.within(O.get(), want, err + au.U * np.abs(want) + 1e-38, roomy)
