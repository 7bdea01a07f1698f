"""Operands of one item of a grouped call that another item writes: refused on
the host, before anything is enqueued."""
import pytest

A = 1 << 32  # addresses of the right alignment; never read
STEP = 1 << 24


def addr(i):
    return A + i * STEP


def status(t, items, eps):
    with pytest.raises(t.TslError) as e:
        # a workspace too short for the call: what passes the checks ends there
        t.shard_linear_group_epilogue(items, eps, t.F32, t.F32, 300, None, 0, stream=0)
    return e.value.status


def item(t, y):
    sh = t.plan_linear(4096, 64, 1, t.COLUMN)[0]
    return dict(shard=sh, packed=addr(0), packed_bytes=1 << 30, X=addr(100), ldx=4096, Y=addr(y),
                ldy=64, ydtype=t.F32)


def test_residual_that_another_item_updates(tsl_lib):
    t = tsl_lib
    one = dict(residual=addr(200), res_dtype=t.F32, ld_res=64)
    two = dict(residual=addr(201), res_dtype=t.F32, ld_res=64)
    # both items read what the first one writes
    assert status(t, [item(t, 200), item(t, 201)], [one, dict(one)]) == t.ERR_INVALID_ARG
    assert status(t, [item(t, 201), item(t, 200)], [dict(one), one]) == t.ERR_INVALID_ARG
    # and the other way round: each in place of the other
    assert status(t, [item(t, 200), item(t, 201)], [two, one]) == t.ERR_INVALID_ARG
    # a bias that lies in an output
    assert status(t, [item(t, 200), item(t, 201)],
                  [dict(bias=addr(201), bias_dtype=t.F32), None]) == t.ERR_INVALID_ARG
    # an item whose residual and bias are one array, its own output
    assert status(t, [item(t, 200)], [dict(one, bias=addr(200), bias_dtype=t.F32)]) == \
        t.ERR_INVALID_ARG


def test_residuals_in_place_and_shared_are_taken(tsl_lib):
    """Each item's residual its own output, and one residual read by two items."""
    t = tsl_lib
    one = dict(residual=addr(200), res_dtype=t.F32, ld_res=64)
    two = dict(residual=addr(201), res_dtype=t.F32, ld_res=64)
    for eps in ([one, two], [dict(one, residual=addr(300)), dict(two, residual=addr(300))]):
        items = [item(t, 200), item(t, 201)]
        need = t.shard_linear_group_epilogue_workspace_size(items, eps, t.F32, 300)
        assert need > 0  # so that the call ends at its workspace
        assert status(t, items, eps) == t.ERR_BUFFER_TOO_SMALL
