"""The layer-block entry points of the binding take any shard with as_tuple, as
the grouped products do (host only: every call ends in its checks)."""
import pytest

A = 1 << 32  # addresses of the right alignment; never read


class Other:
    """A caller's own shard record."""

    def __init__(self, shard):
        self.fields = shard.as_tuple()

    def as_tuple(self):
        return self.fields


def test_any_shard_with_as_tuple(tsl_lib):
    t = tsl_lib
    sh = t.plan_linear(256, 96, 2, t.COLUMN)[1]
    o = Other(sh)
    assert t.transpose_shard(o).as_tuple() == t.transpose_shard(sh).as_tuple()
    assert t.shard_linear_grad_workspace_size(o, t.BF16, 70) == \
        t.shard_linear_grad_workspace_size(sh, t.BF16, 70)
    assert t.shard_gated_grad_workspace_size(o, sh, t.BF16, 70) == \
        t.shard_gated_grad_workspace_size(sh, o, t.BF16, 70)

    def item(g, u):
        return dict(gate=g, up=u, packed_gate=A, packed_up=2 * A, packed_bytes=1 << 20, X=3 * A,
                    ldx=256, H=4 * A, ldh=48)
    assert t.shard_gated_group_workspace_size([item(o, sh)], t.F32, 9) == \
        t.shard_gated_group_workspace_size([item(sh, sh)], t.F32, 9)
    linear = dict(shard=o, packed=A, packed_bytes=1 << 20, X=3 * A, ldx=256, Y=4 * A, ldy=48)
    # calls, up to a check that fails: the shard has been read by then
    for f, args in (
            (t.shard_linear_group_epilogue, ([dict(linear, ldy=47)], [None], t.BF16, t.BF16, 4)),
            (t.shard_gated_group, ([dict(item(o, o), ldh=47)], t.ACT_SILU, t.BF16, t.BF16, 4)),
            (t.shard_linear_grad, (o, t.BF16, A, 1 << 20, 4, 3 * A, 256, t.ACT_NONE, None, 0, 4 * A,
                                   47, t.F32, 5 * A, 256, t.F32, None, 0, 0)),
            (t.shard_gated_grad, (o, o, t.BF16, A, 2 * A, 1 << 20, 4, 3 * A, 256, t.ACT_NONE, 4 * A,
                                  5 * A, 48, 6 * A, 47, t.F32, 7 * A, 256, t.F32, None, None, 0, 0))):
        with pytest.raises(t.TslError) as e:
            f(*args, stream=0)
        assert e.value.status == t.ERR_INVALID_ARG
