"""The size limits of include/tsl_block.h, on the host alone: the workspace's
address is odd, so a call within the limits ends in TSL_ERR_MISALIGNED."""
import pytest

A = 1 << 45  # addresses far apart; never read
STEP = 1 << 42


def linear(t, M, K, N, wdtype, lddy=None, lddx=None):
    up = lambda v: (v + 7) // 8 * 8  # noqa: E731
    sh = t.plan_linear(K, N, 1, t.COLUMN)[0]
    with pytest.raises(t.TslError) as e:
        t.shard_linear_grad(sh, wdtype, A, STEP, M, A + STEP, up(K), t.ACT_NONE, None, 0,
                            A + 2 * STEP, lddy or up(N), t.F32, A + 3 * STEP, lddx or K, t.F32,
                            A + 4 * STEP, N, 1, 0, A + 5 * STEP, A + 6 * STEP + 1, STEP, stream=0)
    return e.value.status


def test_backward_limits(tsl_lib):
    t = tsl_lib
    last = (1 << 22) - 65
    for M, K, N in ((last, 16, 16), (16, last, 16), (16, 16, last), (1 << 20, 1 << 14, 16)):
        assert linear(t, M, K, N, t.BF16) == t.ERR_MISALIGNED, (M, K, N)
    for M, K, N in ((last + 1, 16, 16), (16, last + 1, 16), (16, 16, last + 1),
                    (1 << 20, (1 << 14) + 1, 16), (1 << 20, 16, (1 << 14) + 1)):
        assert linear(t, M, K, N, t.BF16) == t.ERR_UNSUPPORTED, (M, K, N)
        sh = t.plan_linear(K, N, 1, t.COLUMN)[0]
        for f in (lambda: t.shard_linear_grad_workspace_size(sh, t.BF16, M),
                  lambda: t.shard_gated_grad_workspace_size(sh, sh, t.BF16, M)):
            with pytest.raises(t.TslError) as e:
                f()
            assert e.value.status == t.ERR_UNSUPPORTED
    assert linear(t, 1 << 18, 1 << 14, 16, t.F32) == t.ERR_MISALIGNED
    assert linear(t, 1 << 18, (1 << 14) + 4, 16, t.F32) == t.ERR_UNSUPPORTED
    assert linear(t, 16, 16, 16, t.BF16, lddy=(1 << 22) - 8) == t.ERR_MISALIGNED
    assert linear(t, 16, 16, 16, t.BF16, lddx=(1 << 31) - 1) == t.ERR_MISALIGNED
    for kw in (dict(lddy=1 << 22), dict(lddx=1 << 31)):
        assert linear(t, 16, 16, 16, t.BF16, **kw) == t.ERR_UNSUPPORTED, kw


def test_epilogue_strides(tsl_lib):
    t = tsl_lib
    sh = t.plan_linear(130, 64, 1, t.COLUMN)[0]  # X is copied to whole stages: needs workspace
    it = dict(shard=sh, packed=A, packed_bytes=STEP, X=A + STEP, ldx=136, Y=A + 2 * STEP, ldy=64)
    for field, ld in (("residual", "ld_res"), ("pre", "ld_pre")):
        for stride, want in (((1 << 31) - 1, t.ERR_MISALIGNED), (1 << 31, t.ERR_UNSUPPORTED)):
            ep = {field: A + 3 * STEP, ld: stride}
            n = t.shard_linear_group_epilogue_workspace_size([it], [ep], t.BF16, 200)
            assert n > 0
            with pytest.raises(t.TslError) as e:
                t.shard_linear_group_epilogue([it], [ep], t.BF16, t.BF16, 200, A + 4 * STEP + 1, n,
                                              stream=0)
            assert e.value.status == want
