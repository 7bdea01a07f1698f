"""Arguments that the attention operators refuse, on the host alone (every call
here ends in its checks, before anything is enqueued), and the library's
exported names."""
import ctypes
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A, STEP = 1 << 40, 1 << 32


def addr(i):
    return A + i * STEP


def status(t, f, *a, **kw):
    with pytest.raises(t.TslError) as e:
        f(*a, **kw)
    return e.value.status


def test_library_exports_its_header_and_nothing_else(tsl_lib):
    text = open(os.path.join(ROOT, "include", "tsl_attn.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = set(re.findall(r"^\s*(?:const\s+)?\w+\s*\*?\s*(\w+)\s*\(", text, flags=re.M))
    assert names == set(tsl_lib.ATTN_EXPORTS)
    out = subprocess.run(["nm", "-D", "--defined-only", tsl_lib.ATTN_LIBRARY], capture_output=True,
                         text=True, check=True).stdout
    defined = {l.split()[-1] for l in out.splitlines() if l.strip()}
    assert {n for n in defined if not n.startswith("__hip_cuid_")} == names
    assert ctypes.sizeof(tsl_lib.Rotary) == 48 and tsl_lib.Rotary.style.offset == 44
    assert ctypes.sizeof(tsl_lib.RotateItem) == 64 and tsl_lib.RotateItem.ydtype.offset == 56
    assert ctypes.sizeof(tsl_lib.Cache) == 32 and tsl_lib.Cache.head_dim.offset == 24
    assert ctypes.sizeof(tsl_lib.Seqs) == 56 and tsl_lib.Seqs.max_pages.offset == 52
    # a status with a HIP text behind it reads the library's own
    assert tsl_lib.TslError(tsl_lib.ERR_HIP, "rotate_heads").status == tsl_lib.ERR_HIP


def test_rotate_refusals(tsl_lib):
    t = tsl_lib
    INV, UNS, MIS = t.ERR_INVALID_ARG, t.ERR_UNSUPPORTED, t.ERR_MISALIGNED

    def call(M=4, inverse=0, n=1, rot=(), **kw):
        it = dict(X=addr(0), ldx=512, x_head=64, Y=addr(1), ldy=512, y_head=64, n_heads=8, xdtype=1,
                  ydtype=1)
        r = dict(positions=addr(2), ld_pos=4, axes=1, pair_axis=None, freq=addr(3), rot_dim=64,
                 head_dim=64, style=0)
        it.update(kw)
        r.update(dict(rot))
        items = [dict(it, X=addr(10 + 2 * i) if i else it["X"], Y=addr(11 + 2 * i) if i else it["Y"])
                 for i in range(n)]
        return status(t, t.rotate_heads, items, M, r, inverse, stream=0)

    for kw in (dict(X=None), dict(Y=None), dict(M=-1), dict(inverse=2), dict(n=0), dict(n_heads=0),
               dict(xdtype=2), dict(ydtype=3), dict(ldx=500), dict(x_head=60), dict(ldy=448 + 63),
               dict(ldx=-1), dict(y_head=-64),
               # heads outermost, too near
               dict(ldx=64, x_head=255),
               dict(rot=dict(positions=None)), dict(rot=dict(freq=None)), dict(rot=dict(axes=0)),
               dict(rot=dict(rot_dim=63)), dict(rot=dict(rot_dim=66)), dict(rot=dict(rot_dim=0)),
               dict(rot=dict(style=2)), dict(rot=dict(axes=2, ld_pos=3)),
               dict(rot=dict(pair_axis=[0] * 31 + [1])),
               # overlaps: shifted in place, other types or strides in place, the tables
               dict(Y=addr(0) + 128), dict(Y=addr(0), ydtype=0), dict(Y=addr(0), ldy=1024),
               dict(Y=addr(2) - 128), dict(Y=addr(3) - 64)):
        assert call(**kw) == INV, kw
    for kw in (dict(n=9), dict(M=1 << 22), dict(rot=dict(axes=5, ld_pos=8)),
               dict(rot=dict(head_dim=514, rot_dim=64), x_head=514, ldx=8 * 514, y_head=514, ldy=8 * 514),
               dict(n_heads=2000, ldx=1 << 20, ldy=1 << 20)):
        assert call(**kw) == UNS, kw
    for kw in (dict(X=addr(0) + 1), dict(Y=addr(1) + 1), dict(rot=dict(positions=addr(2) + 2)),
               dict(rot=dict(freq=addr(3) + 1))):
        assert call(**kw) == MIS, kw
    with pytest.raises(ValueError):
        call(rot=dict(pair_axis=[0]))
    # two items: one's Y on the other's X
    it = dict(X=addr(0), ldx=512, x_head=64, Y=addr(0), ldy=512, y_head=64, n_heads=8, xdtype=1, ydtype=1)
    r = dict(positions=addr(2), freq=addr(3), rot_dim=64, head_dim=64)
    assert status(t, t.rotate_heads, [it, dict(it, Y=addr(1))], 4, r, stream=0) == INV
    t.rotate_heads([it], 0, r, stream=0)


def cache(**kw):
    return dict(dict(pages=addr(0), n_pages=8, page_tokens=64, n_kv_heads=2, head_dim=128), **kw)


def seqs(**kw):
    return dict(dict(n_seqs=2, rows=6, max_rows=4, max_context=4096, row_start=addr(1),
                     context=addr(1) + 4096, page_table=addr(1) + 8192, ld_table=64, max_pages=64), **kw)


BAD_CACHE = [(dict(pages=None), "INVALID_ARG"), (dict(n_pages=0), "INVALID_ARG"),
             (dict(n_kv_heads=0), "INVALID_ARG"), (dict(head_dim=0), "INVALID_ARG"),
             (dict(page_tokens=0), "INVALID_ARG"), (dict(head_dim=96), "UNSUPPORTED"),
             (dict(page_tokens=48), "UNSUPPORTED"), (dict(page_tokens=16), "UNSUPPORTED"),
             (dict(page_tokens=8192), "UNSUPPORTED"), (dict(n_pages=1 << 31), "UNSUPPORTED"),
             (dict(pages=addr(0) + 16), "MISALIGNED")]
BAD_SEQS = [(dict(n_seqs=-1), "INVALID_ARG"), (dict(rows=-1), "INVALID_ARG"),
            (dict(max_rows=-1), "INVALID_ARG"), (dict(max_context=-1), "INVALID_ARG"),
            (dict(max_pages=-1), "INVALID_ARG"), (dict(row_start=None), "INVALID_ARG"),
            (dict(context=None), "INVALID_ARG"), (dict(page_table=None), "INVALID_ARG"),
            (dict(ld_table=3), "INVALID_ARG"), (dict(n_seqs=65536), "UNSUPPORTED"),
            (dict(rows=1 << 22), "UNSUPPORTED"), (dict(max_pages=1 << 25, ld_table=1 << 25), "UNSUPPORTED"),
            (dict(row_start=addr(1) + 2), "MISALIGNED"), (dict(page_table=addr(1) + 8193), "MISALIGNED")]


def test_append_and_read_refusals(tsl_lib):
    t = tsl_lib

    def call(c=(), q=(), f=None, **kw):
        a = dict(dtype=1, K=addr(2), ldk=256, k_head=128, V=addr(3), ldv=256, v_head=128)
        a.update(kw)
        return [status(t, g, cache(**dict(c)), seqs(**dict(q)), stream=0, **a)
                for g in ((f,) if f else (t.cache_append, t.cache_read))]

    code = lambda n: getattr(t, "ERR_" + n)  # noqa: E731
    for kw, e in BAD_CACHE:
        assert set(call(c=kw)) == {code(e)}, kw
    for kw, e in BAD_SEQS:
        assert set(call(q=kw)) == {code(e)}, kw
    for kw, e in ((dict(dtype=2), "INVALID_ARG"), (dict(ldk=255), "INVALID_ARG"),
                  (dict(k_head=120), "INVALID_ARG"), (dict(ldv=-256), "INVALID_ARG"),
                  (dict(K=None, V=None), "INVALID_ARG"), (dict(K=addr(0) + 256), "INVALID_ARG"),
                  (dict(K=addr(2) + 8), "MISALIGNED"), (dict(ldk=260), "MISALIGNED"),
                  (dict(ldv=262, dtype=0), "MISALIGNED"), (dict(v_head=132), "INVALID_ARG")):
        assert set(call(**kw)) == {code(e)}, kw
    assert call(f=t.cache_append, K=None) == [code("INVALID_ARG")]
    for kw in (dict(K=addr(3)), dict(K=addr(3) + 512), dict(V=addr(1)), dict(V=addr(1) + 8192)):
        assert call(f=t.cache_read, **kw) == [code("INVALID_ARG")], kw
    for kw in (dict(n_seqs=0), dict(rows=0), dict(max_rows=0)):
        t.cache_append(cache(), seqs(**kw), 1, addr(2), 256, 128, addr(3), 256, 128, stream=0)
    assert status(t, t.cache_size, cache(head_dim=100)) == t.ERR_UNSUPPORTED
    assert t.cache_size(cache(pages=None)) == 8 * 2 * 2 * 36 * 128


def test_attention_refusals(tsl_lib):
    t = tsl_lib
    need = t.cache_attention_workspace_size(cache(), seqs(), 8)
    assert need > 0

    def call(c=(), q=(), **kw):
        a = dict(n_q_heads=8, Q=addr(2), ldq=1024, q_head=128, scale=0.1, window=0, sinks=0, odtype=1,
                 O=addr(3), ldo=1024, o_head=128, workspace=addr(4), ws_bytes=1 << 24)
        a.update(kw)
        return status(t, t.cache_attention, cache(**dict(c)), seqs(**dict(q)),
                      stream=0, **a)

    code = lambda n: getattr(t, "ERR_" + n)  # noqa: E731
    for kw, e in BAD_CACHE:
        assert call(c=kw) == code(e), kw
    for kw, e in BAD_SEQS:
        assert call(q=kw) == code(e), kw
    for kw, e in ((dict(Q=None), "INVALID_ARG"), (dict(O=None), "INVALID_ARG"),
                  (dict(n_q_heads=0), "INVALID_ARG"), (dict(n_q_heads=7), "NOT_DIVISIBLE"),
                  (dict(n_q_heads=2048, ldq=1 << 20, ldo=1 << 20), "UNSUPPORTED"),
                  (dict(window=-1), "INVALID_ARG"), (dict(sinks=-1), "INVALID_ARG"),
                  (dict(window=(1 << 30) + 1), "UNSUPPORTED"), (dict(sinks=(1 << 30) + 1), "UNSUPPORTED"),
                  (dict(scale=float("nan")), "INVALID_ARG"), (dict(scale=float("inf")), "INVALID_ARG"),
                  (dict(scale=3e38), "INVALID_ARG"),
                  (dict(odtype=2), "INVALID_ARG"), (dict(ldq=1023), "INVALID_ARG"),
                  (dict(q_head=100), "INVALID_ARG"), (dict(ldo=900), "INVALID_ARG"),
                  (dict(Q=addr(2) + 8), "MISALIGNED"), (dict(O=addr(3) + 2), "MISALIGNED"),
                  (dict(ldq=1028), "MISALIGNED"), (dict(ldo=1026), "MISALIGNED"),
                  (dict(workspace=None), "BUFFER_TOO_SMALL"), (dict(ws_bytes=need - 1), "BUFFER_TOO_SMALL"),
                  (dict(workspace=addr(4) + 16), "MISALIGNED"),
                  # overlaps
                  (dict(O=addr(2)), "INVALID_ARG"), (dict(O=addr(2) + 1024), "INVALID_ARG"),
                  (dict(O=addr(0) + 4096), "INVALID_ARG"), (dict(workspace=addr(2)), "INVALID_ARG"),
                  (dict(workspace=addr(3) + 256), "INVALID_ARG"), (dict(workspace=addr(0)), "INVALID_ARG"),
                  (dict(O=addr(1)), "INVALID_ARG")):
        assert call(**kw) == code(e), kw
    for kw in (dict(n_seqs=0), dict(rows=0), dict(max_rows=0)):
        t.cache_attention(cache(), seqs(**kw), 8, addr(2), 1024, 128, 0.1, 0, 0, 1, addr(3), 1024, 128,
                          stream=0)


def test_workspace_size_goes_by_the_sizes_alone(tsl_lib):
    """The size is a function of the sizes alone, and 0 where a tile is one range."""
    t = tsl_lib
    size = lambda w=0, **kw: t.cache_attention_workspace_size(cache(), seqs(**kw), 8, w, 0)  # noqa: E731
    assert size(max_context=64) == 0
    assert size() == size(row_start=None, context=None, page_table=None) > 0
    assert size(max_pages=1) == 0                # 64 tokens at most
    assert size(max_context=10 ** 9) == size()   # 64 pages of 64
    assert size(w=16, max_context=10 ** 6, max_pages=10 ** 4, ld_table=10 ** 4) == 0
