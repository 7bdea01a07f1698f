"""Arguments the products' backward passes refuse, and their size queries, on
the host alone: every call here ends in its checks."""
import pytest

A = 1 << 32
STEP = 1 << 24


def addr(i):
    return A + i * STEP


def status(t, f, **kw):
    with pytest.raises(t.TslError) as e:
        f(stream=0, **kw)
    return e.value.status


def linear_args(t, **kw):
    sh = t.plan_linear(128, 64, 1, t.COLUMN)[0]
    a = dict(shard=sh, wdtype=t.BF16, packed_t=addr(0), packed_t_bytes=1 << 20, M=10, X=addr(1),
             ldx=128, act=t.ACT_SILU, Z=addr(2), ldz=64, dY=addr(3), lddy=64, dxdtype=t.BF16,
             dX=addr(4), lddx=128, dwdtype=t.F32, dW=addr(5), dw_stride_k=64, dw_stride_n=1,
             accumulate_dw=0, db=addr(6), workspace=addr(7), ws_bytes=1 << 22)
    a.update(kw)
    return a


def test_linear_grad_refusals(tsl_lib):
    t = tsl_lib
    bad = lambda **kw: status(t, t.shard_linear_grad, **linear_args(t, **kw))  # noqa: E731
    for kw in (dict(M=-1), dict(act=9), dict(wdtype=3), dict(dX=None, dW=None, db=None),
               dict(dY=None), dict(X=None), dict(Z=None), dict(packed_t=None), dict(lddy=56),
               dict(ldz=56), dict(ldx=120), dict(lddx=127), dict(dxdtype=2), dict(dwdtype=3),
               dict(dw_stride_k=63), dict(dw_stride_k=64, dw_stride_n=2),
               dict(dw_stride_k=1, dw_stride_n=127), dict(accumulate_dw=2),
               # outputs on inputs, on each other and on the workspace
               dict(dX=addr(1)), dict(dX=addr(2)), dict(dX=addr(3)), dict(dW=addr(4)),
               dict(db=addr(5)), dict(dX=addr(0)), dict(dW=addr(7)), dict(X=addr(7)),
               dict(db=addr(3))):
        assert bad(**kw) == t.ERR_INVALID_ARG, kw
    for kw in (dict(wdtype=t.Q4G64), dict(accumulate_dw=1, dwdtype=t.BF16), dict(M=1 << 22),
               dict(lddy=1 << 22), dict(ldx=1 << 22)):
        assert bad(**kw) == t.ERR_UNSUPPORTED, kw
    for kw in (dict(X=addr(1) + 8), dict(dY=addr(3) + 2), dict(Z=addr(2) + 8), dict(lddy=68),
               dict(ldx=132), dict(packed_t=addr(0) + 128), dict(dX=addr(4) + 1),
               dict(dW=addr(5) + 2), dict(db=addr(6) + 1), dict(workspace=addr(7) + 64)):
        assert bad(**kw) == t.ERR_MISALIGNED, kw
    for kw in (dict(packed_t_bytes=100), dict(workspace=None), dict(ws_bytes=256)):
        assert bad(**kw) == t.ERR_BUFFER_TOO_SMALL, kw


def test_gated_grad_refusals(tsl_lib):
    t = tsl_lib
    sh = t.plan_linear(128, 64, 1, t.COLUMN)[0]

    def bad(**kw):
        a = dict(gate=sh, up=sh, wdtype=t.BF16, packed_gate_t=addr(0), packed_up_t=addr(1),
                 packed_t_bytes=1 << 20, M=10, X=addr(2), ldx=128, act=t.ACT_SILU, G=addr(3),
                 U=addr(4), ld_gu=64, dH=addr(5), lddh=64, dxdtype=t.BF16, dX=addr(6), lddx=128,
                 dwdtype=t.F32, dW_gate=addr(7), dW_up=addr(8), dw_stride_k=64, dw_stride_n=1,
                 accumulate_dw=0, workspace=addr(9), ws_bytes=1 << 22)
        a.update(kw)
        return status(t, t.shard_gated_grad, **a)
    for kw in (dict(G=None), dict(U=None), dict(dH=None), dict(dW_gate=None), dict(dW_up=None),
               dict(dX=None, dW_gate=None, dW_up=None), dict(packed_up_t=None), dict(ld_gu=56),
               dict(up=t.plan_linear(128, 80, 1, t.COLUMN)[0]),
               dict(up=t.plan_linear(64, 64, 1, t.COLUMN)[0]), dict(dX=addr(3)), dict(dW_up=addr(7)),
               dict(dX=addr(1)), dict(dW_up=addr(4) + 64), dict(U=addr(9) + 1024)):
        assert bad(**kw) == t.ERR_INVALID_ARG, kw
    for kw in (dict(U=addr(4) + 8), dict(ld_gu=68), dict(packed_up_t=addr(1) + 16)):
        assert bad(**kw) == t.ERR_MISALIGNED, kw
    assert bad(wdtype=t.Q4G64) == t.ERR_UNSUPPORTED


def test_sizes_and_transposes(tsl_lib):
    t = tsl_lib
    col = t.plan_shards(512, 8, 4, 64, 1024, 4)
    for sh in col:
        tr = t.transpose_shard(sh)
        assert (tr.K, tr.N) == (sh.N, sh.K)
        assert (tr.k_off, tr.k_len, tr.n_off, tr.n_len) == (sh.n_off, sh.n_len, sh.k_off, sh.k_len)
        assert t.pack_shard_size(tr, t.BF16) >= sh.k_len * sh.n_len * 2
        if sh.strategy == t.COLUMN:
            assert tr.strategy == t.ROW and tr.combine == t.COMBINE_SUM
        elif sh.strategy == t.ROW:
            assert tr.strategy == t.COLUMN and tr.combine == t.COMBINE_CONCAT
        else:
            assert tr.strategy == sh.strategy
    with pytest.raises(t.TslError):
        t.transpose_shard(t.Shard())
    sh = col[t.GATE]
    last = 0
    for M in (1, 64, 65, 4096):  # at least the transposed copies, and it grows with M
        n = t.shard_gated_grad_workspace_size(sh, sh, t.BF16, M)
        assert n >= 2 * (M + 63) // 64 * 64 * (2 * 256 + 512) and n >= last
        assert t.shard_linear_grad_workspace_size(sh, t.BF16, M) > 0
        last = n
    assert t.shard_linear_grad_workspace_size(sh, t.F32, 0) >= 0
    for f in (lambda: t.shard_linear_grad_workspace_size(sh, t.Q4G64, 4),
              lambda: t.shard_linear_grad_workspace_size(sh, t.BF16, -1),
              lambda: t.shard_gated_grad_workspace_size(sh, col[t.DOWN], t.BF16, 4)):
        with pytest.raises(t.TslError):
            f()
