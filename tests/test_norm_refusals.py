"""Arguments add_rms_norm and its backward pass refuse, on the host alone:
every call here ends in its checks, before anything is enqueued."""
import pytest

A = 1 << 30  # an address of the right alignment; never read


@pytest.fixture
def call(tsl_lib):
    def norm(**kw):
        a = dict(parts=[A], pdtype=0, ld_part=64, M=2, n=64, residual=A + (1 << 20), rdtype=1,
                 ldr=64, sum_out=A + (2 << 20), ld_sum=64, weight=A + (3 << 20), wdtype=1, eps=1e-6,
                 ydtype=1, Y=A + (4 << 20), ldy=64, scales=None, group=0, rstd=None, stream=0)
        a.update(kw)
        with pytest.raises(tsl_lib.TslError) as e:
            tsl_lib.add_rms_norm(**a)
        return e.value.status
    return norm


def test_norm_refusals(tsl_lib, call):
    t = tsl_lib
    INV, UNS, MIS = t.ERR_INVALID_ARG, t.ERR_UNSUPPORTED, t.ERR_MISALIGNED
    for kw in (dict(parts=[]), dict(parts=[A] * 65), dict(parts=[None]), dict(Y=None), dict(M=-1),
               dict(n=0), dict(eps=-1.0), dict(eps=float("nan")), dict(pdtype=2), dict(pdtype=3),
               dict(rdtype=3), dict(wdtype=7), dict(ydtype=2), dict(ld_part=63), dict(ldr=63),
               dict(ld_sum=63), dict(ldy=63), dict(group=32), dict(scales=A + (5 << 20)),
               dict(ydtype=3), dict(ydtype=3, scales=A + (5 << 20), group=48),
               # overlaps: y on the part, the residual, the weight; sum on y; scales on y
               dict(Y=A), dict(Y=A + (1 << 20) + 128), dict(Y=A + (3 << 20)),
               dict(sum_out=A + (4 << 20)), dict(sum_out=A + (1 << 20), ld_sum=128),
               dict(ydtype=3, scales=A + (4 << 20)), dict(rstd=A)):
        assert call(**kw) == INV, kw
    for kw in (dict(n=32769, ld_part=40000, ldr=40000, ld_sum=40000, ldy=40000), dict(M=1 << 22),
               dict(ldy=1 << 31)):
        assert call(**kw) == UNS, kw
    for kw in (dict(parts=[A + 2]), dict(residual=A + (1 << 20) + 1), dict(Y=A + (4 << 20) + 1),
               dict(weight=A + (3 << 20) + 1), dict(rstd=A + (6 << 20) + 2)):
        assert call(**kw) == MIS, kw
    # no rows: accepted, nothing enqueued
    t.add_rms_norm([A], 0, 64, 0, 64, None, 0, 0, None, 0, None, 0, 1e-6, 1, A, 64, stream=0)


def test_norm_grad_refusals(tsl_lib):
    t = tsl_lib
    need = t.add_rms_norm_grad_workspace_size(2, 64)  # at least one partial row

    def call(**kw):
        a = dict(M=2, n=64, dY=A, dydtype=1, lddy=64, X=A + (1 << 20), xdtype=1, ldx=64,
                 weight=A + (2 << 20), wdtype=1, eps=1e-6, rstd=A + (3 << 20), dres=A + (4 << 20),
                 ld_dres=64, dX=A + (5 << 20), dxdtype=1, lddx=64, dW=A + (6 << 20),
                 accumulate_dw=0, workspace=A + (7 << 20), ws_bytes=1 << 20, stream=0)
        a.update(kw)
        with pytest.raises(t.TslError) as e:
            t.add_rms_norm_grad(**a)
        return e.value.status
    for kw in (dict(dY=None), dict(X=None), dict(dX=None, dres=None, dW=None), dict(dX=None),
               dict(M=-1), dict(n=0), dict(rstd=None, eps=-1.0), dict(dydtype=2), dict(xdtype=3),
               dict(wdtype=2), dict(dxdtype=2), dict(accumulate_dw=2), dict(lddy=63), dict(ldx=8),
               dict(lddx=63), dict(ld_dres=63), dict(dX=A), dict(dX=A + (1 << 20)),
               dict(dres=A + (5 << 20), ld_dres=72), dict(dW=A + (5 << 20)),
               dict(workspace=A + (1 << 20))):
        assert call(**kw) == t.ERR_INVALID_ARG, kw
    for kw in (dict(workspace=None), dict(ws_bytes=need - 1)):
        assert call(**kw) == t.ERR_BUFFER_TOO_SMALL, kw
    for kw in (dict(dY=A + 1), dict(rstd=A + (3 << 20) + 2), dict(dW=A + (6 << 20) + 2),
               dict(workspace=A + (7 << 20) + 16)):
        assert call(**kw) == t.ERR_MISALIGNED, kw
    assert call(n=40000, lddy=40000, ldx=40000, lddx=40000, ld_dres=40000) == t.ERR_UNSUPPORTED
    with pytest.raises(t.TslError):
        t.add_rms_norm_grad_workspace_size(-1, 4)
    assert need >= 64 * 4 and need <= t.add_rms_norm_grad_workspace_size(4000, 64)
