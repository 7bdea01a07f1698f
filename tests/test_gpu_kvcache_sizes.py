"""cache_append and cache_read of many sequences beside a long one."""
import numpy as np
import pytest

import attn_util as au
from gpu_util import torch
from tensor_sharded_linear_plan_amd import binding as tsl

pytestmark = pytest.mark.gpu


def test_a_long_prompt_beside_two_thousand_tokens():
    """A workgroup for each record of the longest, of every sequence and head, would
    be 2^24 of them and more."""
    d, heads, page, n, long = 64, 8, 32, 2048, 32768
    rows = [1] * n
    rows[777] = long
    ctx = [long if m > 1 else 1 + i % 70 for i, m in enumerate(rows)]
    b = au.Batch(rows, ctx, page, seed=1, lead=1, tail=2)
    pages = au.Pages(b.n_pages, page, heads, d)
    r = au.rng(2)
    K, V = (r.standard_normal((b.rows, heads, d), dtype=np.float32) for _ in "kv")
    k, v = (au.Operand(b.rows, heads, d, "bf16", values=x) for x in (K, V))
    tsl.cache_append(pages.dict, b.dict(), tsl.BF16, k.view, k.ld, k.head, v.view, v.ld, v.head)
    ko, vo = (au.Operand(b.rows, heads, d, "f32") for _ in "kv")
    tsl.cache_read(pages.dict, b.dict(), tsl.F32, ko.view, ko.ld, ko.head, vo.view, vo.ld, vo.head)
    torch().cuda.synchronize()
    live = b.live()
    for o, x in ((ko, k), (vo, v)):
        assert np.array_equal(o.get()[live], au.rne(au.held(x.get()[live]), "f32"))
        assert o.rest_untouched(list(live))
