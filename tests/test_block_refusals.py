"""Arguments the epilogue products and the gated block refuse, and their size
queries, on the host alone: every call here ends in its checks."""
import ctypes
import os
import re
import subprocess

import pytest

from conftest import ROOT

A = 1 << 32  # addresses of the right alignment; never read
STEP = 1 << 24


def addr(i):
    return A + i * STEP


def declared():
    text = open(os.path.join(ROOT, "include", "tsl_block.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return set(re.findall(r"^\s*(?:const\s+)?\w+\s*\*?\s*(\w+)\s*\(", text, flags=re.M))


def test_library_exports_its_header_and_nothing_else(tsl_lib):
    names = declared()
    assert names == set(tsl_lib.BLOCK_EXPORTS)
    out = subprocess.run(["nm", "-D", "--defined-only", tsl_lib.BLOCK_LIBRARY],
                         capture_output=True, text=True, check=True).stdout
    defined = {l.split()[-1] for l in out.splitlines() if l.strip()}
    assert {n for n in defined if not n.startswith("__hip_cuid_")} == names
    assert ctypes.sizeof(tsl_lib.Epilogue) == 56 and tsl_lib.Epilogue.act.offset == 40
    assert ctypes.sizeof(tsl_lib.GatedItem) == 120 and tsl_lib.GatedItem.hdtype.offset == 112
    # a status with a HIP text behind it reads the library's own
    assert tsl_lib.TslError(tsl_lib.ERR_HIP, "add_rms_norm").status == tsl_lib.ERR_HIP


def linear(t, M=4, **kw):
    sh = t.plan_linear(128, 64, 1, t.COLUMN)[0]
    it = dict(shard=sh, packed=addr(0), packed_bytes=1 << 20, X=addr(1), ldx=128, Y=addr(2), ldy=64,
              ydtype=t.BF16)
    ep = dict(act=t.ACT_SILU, bias=addr(3), bias_dtype=t.BF16, residual=addr(4), res_dtype=t.BF16,
              ld_res=64, pre=addr(5), pre_dtype=t.F32, ld_pre=64)
    it.update({k: v for k, v in kw.items() if k in it or k == "accumulate"})
    ep.update({k: v for k, v in kw.items() if k not in it and k != "accumulate"})
    with pytest.raises(t.TslError) as e:
        t.shard_linear_group_epilogue([it], [ep], t.BF16, t.BF16, M, None, 0, stream=0)
    return e.value.status


def test_epilogue_refusals(tsl_lib):
    t = tsl_lib
    INV = t.ERR_INVALID_ARG
    for kw in (dict(act=5), dict(act=-1), dict(bias_dtype=2), dict(res_dtype=3), dict(pre_dtype=2),
               dict(ld_res=63), dict(ld_pre=63), dict(accumulate=1, ydtype=t.F32), dict(M=-1),
               dict(X=None), dict(ydtype=3),
               # outputs on inputs or on each other
               dict(pre=addr(1)), dict(pre=addr(2)), dict(pre=addr(3)), dict(pre=addr(4) + 256),
               dict(bias=addr(2)), dict(residual=addr(2), ld_res=72),
               dict(residual=addr(2), res_dtype=t.F32), dict(residual=addr(2) + 128), dict(Y=addr(1))):
        assert linear(t, **kw) == INV, kw
    for kw in (dict(bias=addr(3) + 1), dict(residual=addr(4) + 1), dict(pre=addr(5) + 2),
               dict(ldx=132), dict(X=addr(1) + 8)):
        assert linear(t, **kw) == t.ERR_MISALIGNED, kw
    assert linear(t, ld_res=1 << 31) == t.ERR_UNSUPPORTED
    assert linear(t, packed_bytes=16) == t.ERR_BUFFER_TOO_SMALL


def test_epilogues_of_a_sum_set(tsl_lib):
    """Only the first member of a set may carry one."""
    t = tsl_lib
    shards = t.plan_linear(256, 64, 2, t.ROW)
    items = [dict(shard=sh, packed=addr(8 + r), packed_bytes=1 << 20, X=addr(1) + 256 * r, ldx=256,
                  Y=addr(2), ldy=64, sum_next=1 - r) for r, sh in enumerate(shards)]
    ep = dict(act=t.ACT_RELU)
    for eps in ([None, ep], [ep, ep]):
        with pytest.raises(t.TslError) as e:
            t.shard_linear_group_epilogue(items, eps, t.BF16, t.BF16, 4, None, 0, stream=0)
        assert e.value.status == t.ERR_INVALID_ARG
    with pytest.raises(ValueError):
        t.shard_linear_group_epilogue(items, [ep], t.BF16, t.BF16, 4, None, 0, stream=0)


def gated(t, M=4, act=2, wdtype=None, up=None, **kw):
    sh = t.plan_linear(128, 64, 1, t.COLUMN)[0]
    it = dict(gate=sh, up=up or sh, packed_gate=addr(0), packed_up=addr(1), packed_bytes=1 << 20,
              X=addr(2), ldx=128, H=addr(3), ldh=64, hdtype=t.BF16, G=addr(4), U=addr(5), ld_gu=64)
    it.update(kw)
    with pytest.raises(t.TslError) as e:
        t.shard_gated_group([it], act, t.BF16 if wdtype is None else wdtype, t.BF16, M, None, 0,
                            stream=0)
    return e.value.status


def test_gated_refusals(tsl_lib):
    t = tsl_lib
    for kw in (dict(act=7), dict(M=-1), dict(G=None), dict(U=None), dict(ld_gu=63), dict(ldh=63),
               dict(hdtype=2), dict(packed_up=None), dict(X=None), dict(rows=5),
               dict(up=t.plan_linear(128, 80, 1, t.COLUMN)[0]),
               dict(up=t.plan_linear(192, 64, 1, t.COLUMN)[0], ldx=192),
               dict(H=addr(2)), dict(G=addr(3)), dict(U=addr(4) + 128), dict(G=addr(2)),
               dict(row_index=addr(6), x_rows=0), dict(row_index=addr(4), x_rows=4)):
        assert gated(t, **kw) == t.ERR_INVALID_ARG, kw
    for kw in (dict(G=addr(4) + 1), dict(H=addr(3) + 1), dict(row_index=addr(6) + 2, x_rows=4)):
        assert gated(t, **kw) == t.ERR_MISALIGNED, kw
    assert gated(t, wdtype=t.F32) == t.ERR_UNSUPPORTED
    assert gated(t, ld_gu=1 << 31) == t.ERR_UNSUPPORTED
    assert gated(t, packed_bytes=64) == t.ERR_BUFFER_TOO_SMALL
    sh = t.plan_linear(96, 64, 1, t.COLUMN)[0]  # k not in whole groups of 64
    assert gated(t, wdtype=t.Q4G64, gate=sh, up=sh) == t.ERR_GROUP_ALIGN


def test_size_queries_and_empty_calls(tsl_lib):
    t = tsl_lib
    sh = t.plan_linear(4096, 4096, 1, t.COLUMN, 64)[0]
    it = dict(gate=sh, up=sh, packed_gate=addr(0), packed_up=addr(1), packed_bytes=1 << 30,
              X=addr(2), ldx=4096, H=addr(20), ldh=4096)
    assert t.shard_gated_group_workspace_size([it], t.Q4G64, 0) == 0
    # above 64 rows at least the binary16 activation copy
    assert t.shard_gated_group_workspace_size([it], t.Q4G64, 100) >= 100 * 4096 * 2
    # a call of no rows enqueues nothing, with no workspace
    t.shard_gated_group([it], t.ACT_SILU, t.Q4G64, t.BF16, 0, None, 0, stream=0)
    lin = dict(shard=sh, packed=addr(0), packed_bytes=1 << 30, X=addr(2), ldx=4096, Y=addr(20),
               ldy=4096)
    t.shard_linear_group_epilogue([lin], [dict(act=t.ACT_GELU)], t.Q4G64, t.BF16, 0, None, 0,
                                  stream=0)
    # short and missing workspaces
    for M in (100, 2000):
        need = t.shard_gated_group_workspace_size([it], t.Q4G64, M)
        for w, n in ((None, 0), (addr(40), need - 1)):
            with pytest.raises(t.TslError) as e:
                t.shard_gated_group([it], t.ACT_SILU, t.Q4G64, t.BF16, M, w, n, stream=0)
            assert e.value.status == t.ERR_BUFFER_TOO_SMALL
    with pytest.raises(t.TslError):
        t.shard_gated_group_workspace_size([dict(it, rows=9)], t.Q4G64, 4)
